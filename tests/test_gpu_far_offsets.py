"""GPU tests on arrays of more than 2^32 elements: the last rows give what the same rows give alone, bit for bit, with decays and
gradients of their own, so that a row read or written at a wrapped offset shows."""
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
    yield
    torch.cuda.empty_cache()


def _rnd(gen, t, *s):
    return torch.randn(s, generator=gen).to(t).cuda()


@pytest.mark.parametrize("complement", [False, True])
def test_scan(complement):
    """x and g as the halves of wide rows, dx and dg too.  The last rows begin at a multiple of 4096, where nothing but zeros lies
    before, so that their segments join in the same order as alone."""
    import gated_delta_rule_20_amd as kda
    T, C, tail = 266240 + 1000, 16400, 1000
    assert T * C > 1 << 32
    gen = torch.Generator().manual_seed(1)
    rows = torch.zeros(T, 2 * C, dtype=BF, device="cuda")
    rows[:, C:] = -0.5
    rows[-tail:, :C] = _rnd(gen, BF, tail, C)
    rows[-tail:, C:] = -torch.exp(_rnd(gen, FP, tail, C) - 2).to(BF)
    x, g = rows[:, :C], rows[:, C:]
    last = rows[-tail:].clone()
    h, hT, h8 = kda.gated_scan_fwd(x[None], g[None], complement=complement, pack=True)
    w, wT, w8 = kda.gated_scan_fwd(last[None, :, :C], last[None, :, C:], complement=complement, pack=True)
    assert torch.equal(h[0, -tail:], w[0]) and torch.equal(hT, wT) and (h[0, :-tail] == 0).all()
    assert torch.equal(h8.codes[0, -tail:], w8.codes[0]) and torch.equal(h8.scales[0, -tail:], w8.scales[0])
    assert (h8.codes[0, :-tail] == 0).all() and (h8.scales[0, :-tail] == 0).all()
    d_h = torch.zeros(1, T, C, dtype=BF, device="cuda")
    d_h[0, -tail:] = _rnd(gen, BF, tail, C)
    dhT = _rnd(gen, FP, 1, C)
    drows = torch.full((T, 2 * C), 7.0, dtype=BF, device="cuda")
    x8 = kda.act_pack(x[None])
    # (expected values of the same rows alone, from elements and from codes)
    for saved, hs, xs, lx in (("elements", h, x[None], last[None, :, :C]), ("codes", h8, x8, kda.act_pack(last[None, :, :C]))):
        kw = dict(complement=complement, dfinal_state=dhT)
        drows.fill_(7.0)
        _, _, _, dh0 = kda.gated_scan_bwd(xs if complement else None, g[None], hs, d_h, dx=drows[None, :, :C], dg=drows[None, :, C:], **kw)
        dx, dg, _, _ = kda.gated_scan_bwd(lx if complement else None, last[None, :, C:], w if saved == "elements" else w8,
                                          d_h[:, -tail:].contiguous(), **kw)
        assert torch.equal(drows[-tail:, :C], dx[0]) and torch.equal(drows[-tail:, C:], dg[0]), saved
        assert dg.abs().max() > 0 and (drows[:-tail - 1000] == 0).all() and (dh0 == 0).all(), saved


def test_step_slots():
    import gated_delta_rule_20_amd as kda
    n_slots, C = 270000, 16400
    assert n_slots * C > 1 << 32
    gen = torch.Generator().manual_seed(2)
    pool = torch.zeros(n_slots, C, device="cuda")
    few = _rnd(gen, FP, 3, C)
    slots = torch.tensor([n_slots - 1, 5, n_slots - 40000], dtype=torch.int32, device="cuda")
    pool[slots.long()] = few
    x, g = _rnd(gen, BF, 3, C), -torch.exp(_rnd(gen, BF, 3, C))
    h = kda.gated_scan_step(x, g, pool, slots=slots)
    assert torch.equal(h, kda.gated_scan_step(x, g, few)) and torch.equal(pool[slots.long()], few)
    pool[slots.long()] = 0
    assert (pool == 0).all()


@pytest.mark.parametrize("R,D", [(1049600, 4096), (2800000, 1537), (525000, 8192), (262400, 16384)])
def test_norm_gradients(R, D):
    """By rows (whole and ragged), by rows with weights in LDS, by columns."""
    import gated_delta_rule_20_amd as kda
    assert R * D > 1 << 32
    tail = 7
    gen = torch.Generator().manual_seed(D)
    last = dict(x=_rnd(gen, BF, tail, D), y=_rnd(gen, BF, tail, D), gate=_rnd(gen, BF, tail, D), dx=_rnd(gen, BF, tail, D), dn=_rnd(gen, BF, tail, D))
    post, res, pre = (1 + 0.3 * _rnd(gen, FP, D) for _ in range(3))
    far = {}
    for k, t in last.items():
        far[k] = torch.zeros(R, D, dtype=BF, device="cuda")
        far[k][-tail:] = t
    weights = dict(post_weight=post, res_scale=res, pre_weight=pre, scale=0.7)
    f = ref.f64
    for packed in (False, True):
        pack = lambda t: kda.act_pack(t) if packed else t  # noqa: E731
        call = lambda d, **kw: kda.block_norm_bwd(pack(d["x"]), pack(d["y"]), d["dx"], d["dn"], gate=pack(d["gate"]), **weights, **kw)  # noqa: E731
        got, alone = call(far), call(last)
        for name, a, b in zip(("dx", "dy", "dgate"), got, alone):
            assert torch.equal(a[-tail:], b) and (a[:-tail] == 0).all(), (name, packed)
        val = lambda t: ref.values(*kda.act_pack(t)) if packed else f(t)  # noqa: E731
        want, tol = ref.norm_bwd(val(last["x"]), val(last["y"]), val(last["gate"]), f(post), f(res), f(pre), 0.7, 1e-6, f(last["dx"]), f(last["dn"]))
        for name, t in (("dpost", got.dpost_weight), ("dres", got.dres_scale), ("dpre", got.dpre_weight)):
            ref.close(t, want[name], tol[name], FP, f"{name} packed={packed}")
        del got, alone


def test_norm_forward_from_strided_rows():
    """y and the gate as the halves of wide rows, packed copies of all three."""
    import gated_delta_rule_20_amd as kda
    R, D, tail = 525000, 8190, 5
    gen = torch.Generator().manual_seed(3)
    wide = torch.zeros(R, 2 * D, dtype=BF, device="cuda")
    wide[-tail:] = _rnd(gen, BF, tail, 2 * D)
    x = torch.zeros(R, D, dtype=BF, device="cuda")
    x[-tail:] = _rnd(gen, BF, tail, D)
    w = 1 + 0.1 * _rnd(gen, FP, D)
    call = lambda x, wide: kda.block_norm_fwd(x, wide[:, :D], gate=wide[:, D:], post_weight=w, pre_weight=w, pack=True)  # noqa: E731
    a, n, saved = call(x, wide)
    b, m, kept = call(x[-tail:].clone(), wide[-tail:].clone())
    assert torch.equal(a[-tail:], b) and torch.equal(n[-tail:], m) and (n[:-tail] == 0).all()
    for p, q in zip(saved, kept):
        assert torch.equal(p.codes[-tail:], q.codes) and torch.equal(p.scales[-tail:], q.scales) and (p.codes[:-tail] == 0).all()
