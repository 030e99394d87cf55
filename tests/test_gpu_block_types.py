"""GPU tests of the types that the norms around a block return where activations come in 8 bits, and of a recurrent model's training
step in every combination of types, each call of it against its definition in float64 (block_ref)."""
import itertools

import numpy as np
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
TYPES = [(FP, FP), (BF, BF), (BF, FP)]
IDS = ["fp32", "bf16", "bf16-fp32"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_20_amd as kda
    kda.load_library()


def _kda():
    import gated_delta_rule_20_amd as kda
    return kda


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("y", [False, True])
@pytest.mark.parametrize("given", ["dn dx_new", "dn", "dx_new"])
@pytest.mark.parametrize("types", TYPES, ids=IDS)
def test_types_of_the_gradients(types, given, y, packed):
    """Without ``dtype`` every gradient has the type of what it is the gradient of, and the values of a call that names both types."""
    kda = _kda()
    dtype, x_dtype = types
    R, D = 23, 200
    gen = torch.Generator().manual_seed(1)
    rnd = lambda t, *s: torch.randn(s, generator=gen).to(t).cuda()  # noqa: E731
    weights = dict(pre_weight=1 + 0.1 * rnd(FP, D))
    if y:
        weights.update(post_weight=1 + 0.1 * rnd(FP, D), res_scale=0.5 + 0.1 * rnd(FP, D))
    ys, gate = (rnd(dtype, R, D), rnd(dtype, R, D)) if y else (None, None)
    x1, n, saved = kda.block_norm_fwd(rnd(x_dtype, R, D), ys, gate=gate, n_out=torch.empty(R, D, dtype=dtype, device="cuda"), pack=True,
                                      **weights)
    assert x1.dtype == x_dtype and n.dtype == dtype
    if packed:
        x1, ys, gate = saved
    dx_new = rnd(x_dtype, R, D) if "dx_new" in given else None
    dn = rnd(dtype, R, D) if "dn" in given.split() else None
    x1 = x1 if dn is not None else None
    got = kda.block_norm_bwd(x1, ys, dx_new, dn, gate=gate, **weights)
    want = kda.block_norm_bwd(x1, ys, dx_new, dn, gate=gate, dtype=dtype, dx=torch.empty(R, D, dtype=x_dtype, device="cuda"), **weights)
    for name, a, b, t in zip(got._fields, got, want, (x_dtype, dtype, dtype, FP, FP, FP)):
        assert (a is None) == (b is None), name
        if a is not None:
            assert a.dtype == b.dtype == t and torch.equal(a, b), name


@pytest.mark.parametrize("types", TYPES, ids=IDS)
def test_packed_activations_know_their_type(types):
    """Every call that packs says what it packed, also into a Packed of the caller's."""
    kda = _kda()
    dtype, x_dtype = types
    x, y = torch.randn(5, 40, device="cuda").to(x_dtype), torch.randn(5, 40, device="cuda").to(dtype)
    new = lambda: kda.Packed(torch.empty(5, 40, dtype=torch.int8, device="cuda"), torch.empty(5, 1, device="cuda"))  # noqa: E731
    mine = new()
    assert mine.dtype is None and kda.act_pack(y, out=mine) is mine and mine.dtype == dtype == kda.act_pack(y).dtype
    for pack in (True, kda.BlockNormSaved(new(), new(), new())):
        saved = kda.block_norm_fwd(x, y, gate=y, pre_weight=torch.ones(40, device="cuda"), pack=pack)[2]
        assert [p.dtype for p in saved] == [x_dtype, dtype, dtype]
    for pack in (True, new()):
        assert kda.gated_scan_fwd(y[None], y[None], cu_seqlens=torch.tensor([0, 5], dtype=torch.int32, device="cuda"),
                                  pack=pack if pack is True else kda.Packed(*(t[None] for t in pack)))[2].dtype == dtype


class Checked:
    """The package's calls, each against the definition with the inputs that it got."""

    def __init__(self, types, cu, pack):
        self.kda, self.types, self.cu, self.pack, self.calls = _kda(), types, cu, pack, 0
        self.cu_dev = torch.tensor(cu, dtype=torch.int32, device="cuda")

    def value(self, t):
        return ref.values(*t) if isinstance(t, self.kda.Packed) else ref.f64(t)

    def close(self, names, got, want, tol, types):
        self.calls += 1
        for name, a, b, t, ty in zip(names, got, want, tol, types):
            if b is None:
                assert a is None, name
                continue
            assert a.dtype == ty, (name, a.dtype)
            ref.close(a, b, t, ty, f"call {self.calls}: {name}")

    def norm_fwd(self, x, y=None, gate=None, post_weight=None, res_scale=None, pre_weight=None):
        dtype, x_dtype = self.types
        n_out = torch.empty(x.shape, dtype=dtype, device="cuda") if pre_weight is not None else None
        x1, n, saved = self.kda.block_norm_fwd(x, y, gate=gate, post_weight=post_weight, res_scale=res_scale, pre_weight=pre_weight, n_out=n_out,
                                               pack=True)
        f = ref.f64
        if y is not None:
            want, tol = ref.norm_fwd(f(x), f(y), f(gate), f(post_weight), f(res_scale), 1.0, 1e-6)
            self.close(["x'"], [x1], [want], [tol], [x_dtype])
        if n is not None:
            want, tol = ref.norm_n(f(x1), f(pre_weight), 1e-6)
            self.close(["n"], [n], [want], [tol], [dtype])
        return x1, n, saved if self.pack else (x1, y, gate)

    def norm_bwd(self, x1, y, dx1, dn, gate=None, post_weight=None, res_scale=None, pre_weight=None):
        dtype, x_dtype = self.types
        got = self.kda.block_norm_bwd(x1, y, dx1, dn, gate=gate, post_weight=post_weight, res_scale=res_scale, pre_weight=pre_weight)
        f = ref.f64
        want, tol = ref.norm_bwd(self.value(x1), None if y is None else self.value(y), None if gate is None else self.value(gate),
                                 f(post_weight), f(res_scale), f(pre_weight), 1.0, 1e-6, f(dx1), f(dn))
        names = ("dx", "dy", "dgate", "dpost", "dres", "dpre")
        self.close(names, got, [want.get(k) for k in names], [tol.get(k) for k in names], (x_dtype, dtype, dtype, FP, FP, FP))
        return got

    def scan_fwd(self, x, z, A):
        h, hT, h8 = self.kda.gated_scan_fwd(x, z, A_log=A, complement=True, cu_seqlens=self.cu_dev, pack=True)
        want, wT, tol, tT = ref.scan(ref.f64(x), ref.f64(z), ref.f64(A), -5.0, True, self.cu, None)
        self.close(("h", "final state"), (h, hT), (want, wT), (tol, tT), (self.types[0], FP))
        return h, h8 if self.pack else h

    def scan_bwd(self, x, z, h, d_h, A, rows):
        C = A.shape[0]
        drows = torch.empty_like(rows)
        got = self.kda.gated_scan_bwd(x, z, h, d_h, A_log=A, complement=True, cu_seqlens=self.cu_dev, dx=drows[:, :C], dg=drows[:, C:])
        want, tol = ref.scan_bwd(self.value(x), ref.f64(z), self.value(h), ref.f64(d_h), ref.f64(A), -5.0, True, self.cu, None, None)
        self.close(("dx", "dg", "dA_log", "dh0"), got, want, tol, (self.types[0], self.types[0], FP, FP))
        return drows, got[2]


@pytest.mark.parametrize("last", [False, True], ids=["no-last-norm", "last-norm"])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("types", TYPES, ids=IDS)
def test_training_step_call_by_call(types, packed, last):
    """Two blocks forwards and backwards as a training step joins them (n = norm(x); (v, z) = n Win; h = scan(v, z);
    x = x + res Sigmoid(n Wgate) norm(h Wout)), with a norm behind the last block or none: then no gradient of n names the blocks' type."""
    dtype, x_dtype = types
    D, C, lens = 48, 40, (70, 1, 0, 100)
    T = sum(lens)
    gen = torch.Generator().manual_seed(2)
    rnd = lambda t, *s: torch.randn(s, generator=gen).to(t).cuda()  # noqa: E731
    layers = [dict(pre=1 + 0.1 * rnd(FP, D), win=(rnd(FP, D, 2 * C) / D ** 0.5).to(dtype), A=0.3 * rnd(FP, C), wout=(rnd(FP, C, D) / C ** 0.5).to(dtype),
                   wgate=(rnd(FP, D, D) / D ** 0.5).to(dtype), post=1 + 0.1 * rnd(FP, D), res=0.7 + 0.1 * rnd(FP, D)) for _ in range(2)]
    pres = [layers[1]["pre"], 1 + 0.1 * rnd(FP, D) if last else None]
    ops = Checked(types, np.concatenate([[0], np.cumsum(lens)]).tolist(), packed)
    x, n, (first, _, _) = ops.norm_fwd(rnd(x_dtype, T, D), pre_weight=layers[0]["pre"])
    kept = []
    for p, nxt in zip(layers, pres):
        rows = n @ p["win"]
        h, hs = ops.scan_fwd(rows[:, :C], rows[:, C:], p["A"])
        y, gate = h @ p["wout"], n @ p["wgate"]
        x, n2, saved = ops.norm_fwd(x, y, gate=gate, post_weight=p["post"], res_scale=p["res"], pre_weight=nxt)
        kept.append((n, rows, h, hs, ops.kda.act_pack(rows[:, :C]) if packed else rows[:, :C], saved))
        n = n2
    dx, dn = rnd(x_dtype, T, D), rnd(dtype, T, D) if last else None
    for p, nxt, (n, rows, h, hs, vs, (xs, ys, gs)) in reversed(list(zip(layers, pres, kept))):
        b = ops.norm_bwd(xs, ys, dx, dn, gate=gs, post_weight=p["post"], res_scale=p["res"], pre_weight=nxt)
        drows, _ = ops.scan_bwd(vs, rows[:, C:], hs, b.dy @ p["wout"].t(), p["A"], rows)
        dx, dn = b.dx, drows @ p["win"].t() + b.dgate @ p["wgate"].t()
        assert (n.t() @ drows).dtype == (h.t() @ b.dy).dtype == (n.t() @ b.dgate).dtype == dtype
    b = ops.norm_bwd(first, None, dx, dn, pre_weight=layers[0]["pre"])
    assert b.dx.dtype == x_dtype and ops.calls == (12 if last else 11)


def test_calls_that_name_no_type_are_refused():
    kda = _kda()
    untyped = lambda t: kda.Packed(*kda.act_pack(t))  # noqa: E731
    w = dict(pre_weight=torch.ones(40, device="cuda"))
    x, y = torch.randn(5, 40, device="cuda"), torch.randn(5, 40, device="cuda").to(BF)
    with pytest.raises(ValueError, match="dtype"):
        kda.block_norm_bwd(None, untyped(y), x, None)
    assert kda.block_norm_bwd(None, untyped(y), x, None, dtype=BF).dy.dtype == BF
    with pytest.raises(ValueError, match="dx"):
        kda.block_norm_bwd(untyped(x), None, None, y, **w)
    got = kda.block_norm_bwd(untyped(x), None, None, y, dx=torch.empty_like(x), **w)
    assert got.dx.dtype == FP
    # what one type settles of the other is no guess: a bf16 stream has bf16 blocks, fp32 blocks have an fp32 stream
    assert kda.block_norm_bwd(None, untyped(y), y, None).dy.dtype == BF
    assert kda.block_norm_bwd(untyped(x), None, None, x, **w).dx.dtype == FP


def test_all_combinations_of_what_names_a_type():
    """Whatever subset of the tensors is given, named types agree with the full call's."""
    kda = _kda()
    for dtype, x_dtype in TYPES:
        x, y = torch.randn(3, 16, device="cuda").to(x_dtype), torch.randn(3, 16, device="cuda").to(dtype)
        p = lambda t, on: kda.act_pack(t) if on else t  # noqa: E731
        for px, py, pg, gate in itertools.product((False, True), repeat=4):
            got = kda.block_norm_bwd(p(x, px), p(y, py), None, y, gate=p(y, pg) if gate else None, pre_weight=torch.ones(16, device="cuda"))
            assert got.dx.dtype == x_dtype and got.dy.dtype == dtype and (not gate or got.dgate.dtype == dtype)
