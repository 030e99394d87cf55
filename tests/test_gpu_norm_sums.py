"""GPU test of the norms' weight gradients over many rows: the bound does not grow with the rows."""
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_20_amd as kda
    kda.load_library()


@pytest.mark.parametrize("R,D,types", [(6200000, 70, (BF, BF)), (3100000, 500, (BF, BF)), (1540000, 640, (BF, FP)), (384000, 4096, (BF, BF)), (384000, 3000, (FP, FP)),
                                       (390000, 5000, (BF, BF)), (340001, 8704, (BF, BF)), (409 * 1500, 4100, (FP, FP))])
def test_weight_gradients_of_many_equal_rows(R, D, types):
    """R times one row: every sum is R times that row's term, and its additions round the same way again and again.  At most 64 rows are
    added up in float32, so the bound is that of few rows (block_ref: 64 roundings for a term, 64 for the sum) whatever R; a chain of the
    1500 rows that a workgroup would have here is off by up to 1500 / 4 of them."""
    import gated_delta_rule_20_amd as kda
    dtype, x_dtype = types
    gen = torch.Generator().manual_seed(D)
    rnd = lambda t, *s: torch.randn(s, generator=gen).to(t).cuda()  # noqa: E731
    one = dict(x=rnd(x_dtype, 1, D), y=rnd(dtype, 1, D), dx=rnd(x_dtype, 1, D), dn=rnd(dtype, 1, D))
    post, res, pre = (1 + 0.3 * rnd(FP, D) for _ in range(3))
    many = {k: t.expand(R, D).contiguous() for k, t in one.items()}
    got = kda.block_norm_bwd(many["x"], many["y"], many["dx"], many["dn"], post_weight=post, res_scale=res, pre_weight=pre, scale=0.7)
    f = ref.f64
    want, tol = ref.norm_bwd(f(one["x"]), f(one["y"]), None, f(post), f(res), f(pre), 0.7, 1e-6, f(one["dx"]), f(one["dn"]))
    for name, t in (("dpost", got.dpost_weight), ("dres", got.dres_scale), ("dpre", got.dpre_weight)):
        ref.close(t, R * want[name], R * tol[name], FP, name)
    for name, t, ty in (("dx", got.dx, x_dtype), ("dy", got.dy, dtype)):
        assert torch.equal(t[:1].expand(R, D), t), name
        ref.close(t[:1], want[name], tol[name], ty, name)


@pytest.mark.parametrize("R,D,types", [(262145, 33, (FP, FP)), (131073, 300, (BF, FP)), (262144, 40, (BF, BF)), (65537, 600, (BF, BF)), (16385, 2100, (BF, BF)),
                                       (8193, 16384, (BF, BF))])
def test_first_rows_of_further_workgroups(R, D, types):
    """One row more than the first workgroups take (most of the others have none then), or none more."""
    import gated_delta_rule_20_amd as kda
    dtype, x_dtype = types
    gen = torch.Generator(device="cuda").manual_seed(R)
    rnd = lambda t, *s: torch.randn(s, generator=gen, device="cuda").to(t)  # noqa: E731
    x, y, gate, dx, dn = rnd(x_dtype, R, D), rnd(dtype, R, D), rnd(dtype, R, D), rnd(x_dtype, R, D), rnd(dtype, R, D)
    post, res, pre = (1 + 0.3 * rnd(FP, D) for _ in range(3))
    ws = torch.full((kda.block_norm_bwd_workspace_size(x),), 0xFF, dtype=torch.uint8, device="cuda")      # (NaN)
    got = kda.block_norm_bwd(x, y, dx, dn, gate=gate, post_weight=post, res_scale=res, pre_weight=pre, scale=0.7, workspace=ws)
    f = ref.f64
    sums = None
    for at in range(0, R, 4096):
        rows = slice(at, at + 4096)
        want, tol = ref.norm_bwd(f(x[rows]), f(y[rows]), f(gate[rows]), f(post), f(res), f(pre), 0.7, 1e-6, f(dx[rows]), f(dn[rows]))
        part = [(want[k], tol[k]) for k in ("dpost", "dres", "dpre")]
        sums = part if sums is None else [(a + c, b + d) for (a, b), (c, d) in zip(sums, part)]
        if at % 65536 == 0 or at + 4096 >= R:
            for k, t, ty in (("dx", got.dx, x_dtype), ("dy", got.dy, dtype), ("dgate", got.dgate, dtype)):
                ref.close(t[rows], want[k], tol[k], ty, (k, at))
    for (want, tol), t, name in zip(sums, (got.dpost_weight, got.dres_scale, got.dpre_weight), ("dpost", "dres", "dpre")):
        ref.close(t, want, tol, FP, name)
