"""GPU tests of the norms around a block (kda_block_norm_fwd / _bwd) against their definition in float64, within bounds counted
in roundings (block_ref)."""
import numpy as np
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


def _kda():
    import gated_delta_rule_20_amd as kda
    return kda


def _inputs(R, D, dtype, x_dtype, gate, post, res, pre, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    d = dict(x=(2 * rnd(R, D)).to(x_dtype), y=(1.5 * rnd(R, D)).to(dtype), gate=(2 * rnd(R, D)).to(dtype) if gate else None,
             post=1 + 0.3 * rnd(D) if post else None, res=0.5 + 0.3 * rnd(D) if res else None,
             pre=1 + 0.3 * rnd(D) if pre else None, dx=rnd(R, D).to(x_dtype), dn=rnd(R, D).to(dtype) if pre else None)
    return {k: v if v is None else v.cuda() for k, v in d.items()}


def _kw(d, scale=0.7, eps=1e-6):
    return dict(gate=d["gate"], post_weight=d["post"], res_scale=d["res"], pre_weight=d["pre"], scale=scale, eps=eps)


SIZES = [(1, 1), (3, 5), (2, 8), (5, 127), (7, 512), (4, 513), (9, 1000), (130, 1024), (3, 2051), (600, 64), (33, 4096), (2, 4097),
         (5, 8192), (3, 10001), (2, 16384), (7, 390), (6, 511), (11, 1999), (4, 3001), (3, 6), (9, 4094)]
TYPES = [(FP, FP), (BF, BF), (BF, FP)]
PARTS = [(True, True, True, True), (True, False, False, True), (False, True, False, True), (False, False, True, False),
         (True, True, False, False), (False, False, False, True)]


@pytest.mark.parametrize("types", TYPES, ids=["fp32", "bf16", "bf16-fp32"])
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_forward_and_backward(case, types):
    kda = _kda()
    R, D = SIZES[case]
    for k, parts in enumerate(PARTS):
        if D > 2000 and k not in (0, 1 + case % 5):
            continue
        d = _inputs(R, D, *types, *parts, seed=10 * case + k)
        x1, n, saved = kda.block_norm_fwd(d["x"], d["y"], pack=True, **_kw(d))
        want, tol = ref.norm_fwd(*(ref.f64(d[a]) for a in ("x", "y", "gate", "post", "res")), 0.7, 1e-6)
        ref.close(x1, want, tol, types[1], f"x' {parts}")
        if d["pre"] is None:
            assert n is None
        else:
            ref.close(n, *ref.norm_n(ref.f64(x1), ref.f64(d["pre"]), 1e-6), types[0], f"n {parts}")
        for t, p in zip((x1, d["y"], d["gate"]), saved):
            if t is None:
                assert p is None
                continue
            q = kda.act_pack(t)
            assert torch.equal(p.codes, q.codes) and torch.equal(p.scales, q.scales)
        plain = kda.block_norm_fwd(d["x"], d["y"], **_kw(d))
        assert torch.equal(plain[0], x1) and (n is None or torch.equal(plain[1], n))
        for packed in (False, True):
            kw = _kw(d)
            xs, ys = (saved.x_new, saved.y) if packed else (x1, d["y"])
            kw["gate"] = saved.gate if packed else d["gate"]
            got = kda.block_norm_bwd(xs, ys, d["dx"], d["dn"], dtype=types[0], **kw)
            val = lambda t: None if t is None else ref.values(*t) if isinstance(t, kda.Packed) else ref.f64(t)  # noqa: E731
            want, tol = ref.norm_bwd(val(xs), val(ys), val(kw["gate"]), *(ref.f64(d[a]) for a in ("post", "res", "pre")), 0.7,
                                     1e-6, ref.f64(d["dx"]), ref.f64(d["dn"]))
            for name, t, ty in zip(("dx", "dy", "dgate", "dpost", "dres", "dpre"), got, (types[1], types[0], types[0], FP, FP, FP)):
                if name not in want:
                    assert t is None, name
                    continue
                assert t.dtype == ty
                ref.close(t, want[name], tol[name], ty, f"{name} {parts} packed={packed}")


@pytest.mark.parametrize("types", TYPES, ids=["fp32", "bf16", "bf16-fp32"])
def test_first_and_last_norm(types):
    """No block before (y None): x' is x itself.  Only one of the two gradients given."""
    kda = _kda()
    R, D = 37, 300
    d = _inputs(R, D, *types, True, True, True, True, seed=3)
    n_out = torch.empty(R, D, dtype=types[0], device="cuda")
    x1, n = kda.block_norm_fwd(d["x"], pre_weight=d["pre"], n_out=n_out)
    assert x1 is d["x"] and n is n_out
    ref.close(n, *ref.norm_n(ref.f64(d["x"]), ref.f64(d["pre"]), 1e-6), types[0], "n")
    for dx in (None, d["dx"]):
        got = kda.block_norm_bwd(d["x"], None, dx, d["dn"], pre_weight=d["pre"])
        zero = np.zeros((R, D)) if dx is None else ref.f64(dx)
        want, tol = ref.norm_bwd(ref.f64(d["x"]), None, None, None, None, ref.f64(d["pre"]), 1.0, 1e-6, zero, ref.f64(d["dn"]))
        ref.close(got.dx, want["dx"], tol["dx"], types[1], "dx")
        ref.close(got.dpre_weight, want["dpre"], tol["dpre"], FP, "dpre")
        assert got.dy is None and got.dgate is None
    got = kda.block_norm_bwd(None, d["y"], d["dx"], None, **_kw(d))
    want, tol = ref.norm_bwd(None, *(ref.f64(d[a]) for a in ("y", "gate", "post", "res", "pre")), 0.7, 1e-6, ref.f64(d["dx"]), None)
    assert torch.equal(got.dx, d["dx"]) and (got.dpre_weight == 0).all()
    ref.close(got.dy, want["dy"], tol["dy"], types[0], "dy")
    none = kda.block_norm_bwd(None, d["y"], d["dx"], None, need_dweights=False, **_kw(d))
    assert torch.equal(none.dy, got.dy) and none[3:] == (None, None, None)


def test_gradients_against_differences():
    """Central differences of <dx', x'> + <dn, n> in float64."""
    kda = _kda()
    d = _inputs(6, 40, FP, FP, True, True, True, True, seed=7)
    x1, _ = kda.block_norm_fwd(d["x"], d["y"], **_kw(d))
    got = kda.block_norm_bwd(x1, d["y"], d["dx"], d["dn"], **_kw(d))
    names = ("x", "y", "gate", "post", "res", "pre")
    base = [ref.f64(d[k]) for k in names]

    def loss(x, y, gate, post, res, pre):
        v = ref.norm_fwd(x, y, gate, post, res, 0.7, 1e-6)[0]
        return (v * ref.f64(d["dx"])).sum() + (ref.norm_n(v, pre, 1e-6)[0] * ref.f64(d["dn"])).sum()
    rng = np.random.default_rng(0)
    for i, grad in enumerate(got):
        v, eps = rng.standard_normal(base[i].shape), 1e-5
        lo, hi = list(base), list(base)
        lo[i], hi[i] = base[i] - eps * v, base[i] + eps * v
        num, ana = (loss(*hi) - loss(*lo)) / (2 * eps), (ref.f64(grad) * v).sum()
        # x' was rounded to float32 before the gradients: 1e-6 of each
        assert abs(num - ana) <= 1e-5 * np.abs(ref.f64(grad) * v).sum() + 1e-7, names[i]


def test_in_place_strides_and_guards():
    """x' over x, dx over dx'; y and the gate as parts of wider rows, their gradients into parts of one; nothing else written."""
    kda = _kda()
    for R, D, dtype in ((50, 45, BF), (20, 1003, FP), (70, 2048, BF)):
        d = _inputs(R, D, dtype, dtype, True, True, True, True, seed=D)
        a = kda.block_norm_fwd(d["x"], d["y"], **_kw(d))
        ga = kda.block_norm_bwd(a[0], d["y"], d["dx"], d["dn"], **_kw(d))
        wide = torch.full((R, 2 * D + 5), 7.0, dtype=dtype, device="cuda")
        yv, gv = wide[:, 1:1 + D], wide[:, 3 + D:3 + 2 * D]
        yv.copy_(d["y"])
        gv.copy_(d["gate"])
        x = torch.full((R * D + 512,), 7.0, dtype=dtype, device="cuda")
        xv = x[256:-256].view(R, D)
        xv.copy_(d["x"])
        kw = _kw(d)
        kw["gate"] = gv
        b = kda.block_norm_fwd(xv, yv, x_out=xv, **kw)
        assert torch.equal(a[0], xv) and torch.equal(a[1], b[1])
        assert (x[:256] == 7).all() and (x[-256:] == 7).all()
        out = torch.full((R, 2 * D + 5), 7.0, dtype=dtype, device="cuda")
        dx = d["dx"].clone()
        gb = kda.block_norm_bwd(xv, yv, dx, d["dn"], dx=dx, dy=out[:, 1:1 + D], dgate=out[:, 3 + D:3 + 2 * D], **kw)
        assert all(torch.equal(p, q) for p, q in zip(ga, gb))
        assert (out[:, 0] == 7).all() and (out[:, 1 + D:3 + D] == 7).all() and (out[:, 3 + 2 * D:] == 7).all()


def test_zero_rows_extremes_and_nan():
    """Rows of zeros (eps 0 too), gates far out, a NaN row that stays in its row; no rows at all."""
    kda = _kda()
    d = _inputs(9, 200, FP, FP, True, True, False, True, seed=1)
    d["x"][3], d["y"][3], d["gate"][4], d["gate"][5] = 0.0, 0.0, 200.0, -200.0
    for eps in (0.0, 1e-6):
        x1, n = kda.block_norm_fwd(d["x"], d["y"], **_kw(d, eps=eps))
        assert (n[3] == 0).all() and (x1[3] == 0).all() and torch.isfinite(n).all()
        assert torch.equal(x1[5], d["x"][5])               # the gate is closed
        g = kda.block_norm_bwd(x1, d["y"], d["dx"], d["dn"], **_kw(d, eps=eps))
        assert (g.dgate[4] == 0).all() and (g.dgate[5] == 0).all() and (g.dy[5] == 0).all()
        assert eps == 0.0 or all(torch.isfinite(t).all() for t in g if t is not None)
    a = kda.block_norm_fwd(d["x"], d["y"], **_kw(d))
    ga = kda.block_norm_bwd(a[0], d["y"], d["dx"], d["dn"], **_kw(d))
    y = d["y"].clone()
    y[7, 20] = float("nan")
    b = kda.block_norm_fwd(d["x"], y, **_kw(d))
    gb = kda.block_norm_bwd(b[0], y, d["dx"], d["dn"], **_kw(d))
    keep = torch.arange(9) != 7
    for p, q in ((a[0], b[0]), (a[1], b[1]), (ga.dx, gb.dx), (ga.dy, gb.dy), (ga.dgate, gb.dgate)):
        assert torch.equal(p[keep.cuda()], q[keep.cuda()])
    assert torch.isnan(b[1][7]).all()
    e = torch.empty(0, 200, device="cuda")
    x1, n = kda.block_norm_fwd(e, e, post_weight=d["post"], pre_weight=d["pre"])
    assert x1.shape == n.shape == (0, 200)
    g = kda.block_norm_bwd(e, e, e, e, post_weight=d["post"], pre_weight=d["pre"])
    assert (g.dpost_weight == 0).all() and (g.dpre_weight == 0).all()


def test_repeats_streams_and_graph():
    kda = _kda()
    d = _inputs(1500, 640, BF, FP, True, True, True, True, seed=2)

    def both():
        x1, n, saved = kda.block_norm_fwd(d["x"], d["y"], pack=True, **_kw(d))
        kw = _kw(d)
        kw["gate"] = saved.gate
        return [x1, n, *kda.block_norm_bwd(saved.x_new, saved.y, d["dx"], d["dn"], **kw)]
    first = both()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, both()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = kda.block_norm_fwd(d["x"], d["y"], stream=side, **_kw(d))
    side.synchronize()
    assert torch.equal(other[0], first[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for i in range(3):
        d["y"].copy_(torch.randn(1500, 640, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(kept, both())), i


@pytest.mark.parametrize("types", TYPES, ids=["fp32", "bf16", "bf16-fp32"])
def test_workspace_size_is_enough(types):
    kda = _kda()
    for R, D in ((3, 16), (700, 4095), (700, 4097), (2000, 5000), (300, 8192), (40, 8193)):
        d = _inputs(R, D, *types, False, True, True, True, seed=1)
        x1, _, saved = kda.block_norm_fwd(d["x"], d["y"], pack=True, **_kw(d))
        want = kda.block_norm_bwd(x1, d["y"], d["dx"], d["dn"], **_kw(d))
        for x in (x1, saved.x_new):
            ws = torch.empty(kda.block_norm_bwd_workspace_size(x), dtype=torch.uint8, device="cuda")
            kda.block_norm_bwd(x, d["y"], d["dx"], d["dn"], workspace=ws, **_kw(d))
        got = kda.block_norm_bwd(x1, d["y"], d["dx"], d["dn"], workspace=ws, **_kw(d))
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(want, got))


def test_many_wide_rows():
    """Rows too wide for one workgroup's registers, more of them than workgroups; rows do not depend on their neighbours, dx over
    dx', one weight's gradient only, a captured call."""
    kda = _kda()
    R, D = 1100, 8201
    d = _inputs(R, D, BF, BF, True, True, True, True, seed=5)
    x1, _, saved = kda.block_norm_fwd(d["x"], d["y"], pack=True, **_kw(d))
    got = kda.block_norm_bwd(x1, d["y"], d["dx"], d["dn"], **_kw(d))
    want, tol = ref.norm_bwd(*(ref.f64(t) for t in (x1, d["y"], d["gate"], d["post"], d["res"], d["pre"])), 0.7, 1e-6,
                             ref.f64(d["dx"]), ref.f64(d["dn"]))
    for name, t, ty in zip(("dx", "dy", "dgate", "dpost", "dres", "dpre"), got, (BF, BF, BF, FP, FP, FP)):
        ref.close(t, want[name], tol[name], ty, name)
    cut = slice(1030, 1041)
    kw = _kw(d)
    kw["gate"] = d["gate"][cut]
    dx = d["dx"][cut].clone()
    part = kda.block_norm_bwd(x1[cut], d["y"][cut], dx, d["dn"][cut], dx=dx, **kw)
    assert all(torch.equal(a[cut], b) for a, b in zip(got[:3], part[:3]))
    assert kda.block_norm_bwd_workspace_size(x1, weights=0) > 0
    none = kda.block_norm_bwd(x1, d["y"], d["dx"], d["dn"], need_dweights=False, **_kw(d))
    assert all(torch.equal(a, b) for a, b in zip(got[:3], none[:3])) and none[3:] == (None, None, None)
    kw["gate"] = saved.gate
    ws = torch.empty(kda.block_norm_bwd_workspace_size(saved.x_new), dtype=torch.uint8, device="cuda")
    call = lambda: kda.block_norm_bwd(saved.x_new, saved.y, d["dx"], d["dn"], workspace=ws, **kw)  # noqa: E731
    first = call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for _ in range(3):
        ws.fill_(0xA5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_large_offsets():
    """Rows behind 2^32 bytes give what the same rows give alone."""
    kda = _kda()
    R, D = 150000, 16384
    y = torch.zeros(R, D, dtype=BF, device="cuda")
    tail = torch.randn(5, D, device="cuda").to(BF)
    y[-5:] = tail
    w = torch.ones(D, device="cuda")
    x1, n = kda.block_norm_fwd(y, y, post_weight=w, pre_weight=w, x_out=y)
    a, b = kda.block_norm_fwd(tail, tail, post_weight=w, pre_weight=w)
    assert torch.equal(x1[-5:], a) and torch.equal(n[-5:], b) and (n[:-5] == 0).all()
