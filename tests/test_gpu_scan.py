"""GPU tests of the gated scan (kda_gated_scan_fwd / _bwd / _step) against its definition in float64, within bounds counted in
roundings (block_ref)."""
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


def _inputs(lens, C, dtype, g_dtype, logits, states, seed=0, slow=False):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    T = sum(lens)
    g = 2 * rnd(T, C) - 2 if logits else -torch.exp(rnd(T, C) * 2 - (6 if slow else 2))
    if not logits and T > 3:
        g[T // 2] = -60.0                      # a token that forgets everything
        g[T // 3, ::3] = 0.0                   # and ones that keep it
        g[T // 4, ::5] = 0.7                   # counts as 0
    N = len(lens)
    d = dict(x=rnd(T, C).to(dtype), g=g.to(g_dtype), A=0.4 * rnd(C) if logits else None, h0=rnd(N, C) if states else None,
             dh=rnd(T, C).to(dtype), dhT=rnd(N, C) if states else None)
    d = {k: v if v is None else v.cuda() for k, v in d.items()}
    d["cu"] = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64).tolist()
    d["cu_dev"] = torch.tensor(d["cu"], dtype=torch.int32).cuda()
    return d


def _fwd_ref(d, complement, g_min=-5.0):
    return ref.scan(ref.f64(d["x"]), ref.f64(d["g"]), ref.f64(d["A"]), g_min, complement, d["cu"], ref.f64(d["h0"]))


LENS = [((1,), 1), ((0, 1, 2, 0), 3), ((128,), 128), ((127,), 130), ((129,), 7), ((5, 0, 300, 1, 64), 100), ((1,) * 200, 24),
        ((2000,), 9), ((300, 700), 257), ((64, 64, 64, 64, 256), 1000), ((17, 260), 2056)]


@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("logits", [False, True])
@pytest.mark.parametrize("types", [(FP, FP), (BF, BF), (BF, FP)], ids=["fp32", "bf16", "bf16-fp32"])
@pytest.mark.parametrize("case", range(len(LENS)))
def test_forward(case, types, logits, complement):
    lens, C = LENS[case]
    states = (case + logits + complement) % 2 == 0
    d = _inputs(lens, C, *types, logits, states, seed=case)
    h, hT = _kda().gated_scan_fwd(d["x"], d["g"], A_log=d["A"], complement=complement, cu_seqlens=d["cu_dev"],
                                  initial_state=d["h0"])
    want, wT, tol, tT = _fwd_ref(d, complement)
    assert h.dtype == types[0] and hT.dtype == FP
    ref.close(h, want, tol, types[0], "h")
    ref.close(hT, wT, tT, FP, "final state")


@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("logits", [False, True])
@pytest.mark.parametrize("types", [(FP, FP), (BF, BF), (BF, FP)], ids=["fp32", "bf16", "bf16-fp32"])
@pytest.mark.parametrize("case", range(len(LENS)))
def test_backward(case, types, logits, complement):
    kda = _kda()
    lens, C = LENS[case]
    states, packed = (case + logits) % 2 == 0, (case + complement) % 3 == 0
    d = _inputs(lens, C, *types, logits, states, seed=50 + case)
    h = torch.from_numpy(_fwd_ref(d, complement)[0]).to(types[0]).cuda()
    hs, xs = (kda.act_pack(h), kda.act_pack(d["x"])) if packed else (h, d["x"])
    got = kda.gated_scan_bwd(xs if complement else None, d["g"], hs, d["dh"], A_log=d["A"], complement=complement,
                             cu_seqlens=d["cu_dev"], initial_state=d["h0"], dfinal_state=d["dhT"])
    val = lambda t: ref.values(*t) if isinstance(t, kda.Packed) else ref.f64(t)  # noqa: E731
    want, tol = ref.scan_bwd(val(xs), ref.f64(d["g"]), val(hs), ref.f64(d["dh"]), ref.f64(d["A"]), -5.0, complement, d["cu"],
                             ref.f64(d["h0"]), ref.f64(d["dhT"]))
    for name, a, b, t, ty in zip(("dx", "dg", "dA_log", "dinitial_state"), got, want, tol, (*types, FP, FP)):
        if b is None:
            assert a is None
            continue
        assert a.dtype == ty
        ref.close(a, b, t, ty, name)
    # without dg: the same dx and dinitial_state, h and x not read
    dx, dg, dA, dh0 = kda.gated_scan_bwd(None, d["g"], None, d["dh"], A_log=d["A"], complement=complement,
                                         cu_seqlens=d["cu_dev"], dfinal_state=d["dhT"], need_dg=False)
    assert dg is None and dA is None and torch.equal(dx, got[0]) and torch.equal(dh0, got[3])


def test_gradients_against_differences():
    """Gradients of a scalar of (h, final state) by central differences of the float64 definition."""
    kda = _kda()
    d = _inputs((40, 3, 90), 6, FP, FP, True, True, seed=3)
    for complement in (False, True):
        h, _ = kda.gated_scan_fwd(d["x"], d["g"], A_log=d["A"], complement=complement, cu_seqlens=d["cu_dev"], initial_state=d["h0"])
        dx, dg, dA, dh0 = kda.gated_scan_bwd(d["x"], d["g"], h, d["dh"], A_log=d["A"], complement=complement,
                                             cu_seqlens=d["cu_dev"], initial_state=d["h0"], dfinal_state=d["dhT"])
        base = [ref.f64(d[k]) for k in ("x", "g", "A", "h0")]

        def loss(x, g, A, h0):
            h, hT, _, _ = ref.scan(x, g, A, -5.0, complement, d["cu"], h0)
            return (h * ref.f64(d["dh"])).sum() + (hT * ref.f64(d["dhT"])).sum()
        gen = np.random.default_rng(0)
        for i, grad in enumerate((dx, dg, dA, dh0)):
            v = gen.standard_normal(base[i].shape)
            eps = 1e-5
            lo, hi = [b.copy() for b in base], [b.copy() for b in base]
            lo[i] -= eps * v
            hi[i] += eps * v
            num, ana = (loss(*hi) - loss(*lo)) / (2 * eps), (ref.f64(grad) * v).sum()
            # float32 gradients: each within about 1e-5 of itself here; differences of second order in 64 bits
            assert abs(num - ana) <= 2e-5 * np.abs(ref.f64(grad) * v).sum() + 1e-6, (complement, i, num, ana)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_batch_equals_packed(dtype):
    """[B, T, C] without offsets is B packed sequences of T tokens, bit for bit, forwards and backwards."""
    kda = _kda()
    for B, T, C in ((3, 100, 40), (2, 256, 136), (5, 1, 8), (70, 3, 17)):
        d = _inputs((T,) * B, C, dtype, dtype, True, True, seed=B)
        v = lambda t: t.view(B, T, C)  # noqa: E731
        kw = dict(A_log=d["A"], complement=True, initial_state=d["h0"])
        a = kda.gated_scan_fwd(d["x"], d["g"], cu_seqlens=d["cu_dev"], **kw)
        b = kda.gated_scan_fwd(v(d["x"]), v(d["g"]), **kw)
        assert torch.equal(v(a[0]), b[0]) and torch.equal(a[1], b[1])
        kw["dfinal_state"] = d["dhT"]
        a = kda.gated_scan_bwd(d["x"], d["g"], a[0], d["dh"], cu_seqlens=d["cu_dev"], **kw)
        b = kda.gated_scan_bwd(v(d["x"]), v(d["g"]), b[0], v(d["dh"]), **kw)
        assert all(torch.equal(p.reshape(q.shape), q) for p, q in zip(a, b))


def test_slow_decay_keeps_float32():
    """States that fade over 10^4 tokens stay accurate to float32.  With k = 8 independent roundings a token the error is about
    8 sqrt(10^4) 2^-25 = 2.4e-5 of the state at the most likely worst; a rounded e^g would be off by 10^4 2^-25 = 3e-4."""
    kda = _kda()
    T, C = 30000, 16
    gen = torch.Generator().manual_seed(5)
    x = torch.rand(T, C, generator=gen).cuda()
    g = (-1e-4 * (1 + 0.1 * torch.rand(C, generator=gen))).expand(T, C).contiguous().cuda()
    h, hT = kda.gated_scan_fwd(x[None], g[None])
    a, H = np.exp(ref.f64(g)[0]), np.zeros(C)
    xs, want = ref.f64(x), np.zeros((T, C))
    for t in range(T):
        H = a * H + xs[t]
        want[t] = H
    assert np.linalg.norm(ref.f64(h)[0] - want) <= 2.4e-5 * np.linalg.norm(want)
    assert np.linalg.norm(ref.f64(hT)[0] - H) <= 2.4e-5 * np.linalg.norm(H)
    dx = kda.gated_scan_bwd(None, g[None], None, x.flip(0).contiguous()[None], need_dg=False)[0]
    assert np.linalg.norm(ref.f64(dx)[0][::-1] - want) <= 2.4e-5 * np.linalg.norm(want)


def test_edges_of_decays_and_values():
    """-inf forgets (also a large state), values above 0 count as 0, underflow is 0; a NaN or infinity stays in its channel and
    sequence."""
    kda = _kda()
    lens, C = (150, 90, 200), 20
    d = _inputs(lens, C, FP, FP, False, True, seed=9)
    g = d["g"].clone()
    g[10, :4], g[180], g[70, 4] = float("-inf"), -200.0, -1e-30
    x = d["x"].clone()
    x[5, 0] = 3e30
    d["x"], d["g"] = x, g
    h, hT = kda.gated_scan_fwd(x, g, cu_seqlens=d["cu_dev"], initial_state=d["h0"])
    want, wT, tol, tT = _fwd_ref(d, False)
    ref.close(h, want, tol, FP, "h")
    ref.close(hT, wT, tT, FP, "final state")
    bad = x.clone()
    bad[160, 3], bad[20, 7] = float("nan"), float("inf")
    g2 = g.clone()
    g2[260, 11] = float("nan")
    h2, hT2 = kda.gated_scan_fwd(bad, g2, cu_seqlens=d["cu_dev"], initial_state=d["h0"])
    touched = torch.zeros_like(h, dtype=torch.bool)
    touched[160:240, 3] = touched[20:150, 7] = touched[260:440, 11] = True
    assert torch.equal(h2[~touched], h[~touched]) and not torch.isfinite(h2[160:180, 3]).any()
    assert not torch.isfinite(h2[20:30, 7]).any() and torch.isnan(h2[260:440, 11]).all()
    dy = d["dh"].clone()
    dy[100, 5] = float("nan")
    a = kda.gated_scan_bwd(None, g, h, d["dh"], cu_seqlens=d["cu_dev"], initial_state=d["h0"])
    b = kda.gated_scan_bwd(None, g, h, dy, cu_seqlens=d["cu_dev"], initial_state=d["h0"])
    keep = torch.ones_like(h, dtype=torch.bool)
    keep[:101, 5] = False
    assert torch.equal(a[0][keep], b[0][keep]) and torch.equal(a[1][keep], b[1][keep]) and torch.isnan(b[0][75:101, 5]).all()


@pytest.mark.parametrize("dtype", [FP, BF])
def test_strided_rows(dtype):
    """x and g as parts of wider rows (odd offsets, odd strides), dx and dg into parts of one: the same bits as dense ones, and
    nothing else is written."""
    kda = _kda()
    T, C = 333, 45
    d = _inputs((200, 133), C, dtype, dtype, True, True, seed=4)
    kw = dict(A_log=d["A"], complement=True, cu_seqlens=d["cu_dev"], initial_state=d["h0"])
    wide = torch.randn(T, 2 * C + 7, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    wide[:, 3:3 + C], wide[:, 3 + C:3 + 2 * C] = d["x"], d["g"]
    xv, gv = wide[:, 3:3 + C], wide[:, 3 + C:3 + 2 * C]
    a = kda.gated_scan_fwd(d["x"], d["g"], **kw)
    b = kda.gated_scan_fwd(xv, gv, **kw)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga = kda.gated_scan_bwd(d["x"], d["g"], a[0], d["dh"], **kw)
    out = torch.full((T, 2 * C + 7), 7.0, dtype=dtype, device="cuda")
    gb = kda.gated_scan_bwd(xv, gv, a[0], d["dh"], dx=out[:, 3:3 + C], dg=out[:, 3 + C:3 + 2 * C], **kw)
    assert all(torch.equal(p, q) for p, q in zip(ga, gb))
    rest = torch.ones(2 * C + 7, dtype=torch.bool)
    rest[3:3 + 2 * C] = False
    assert (out[:, rest.cuda()] == 7).all()
    # an odd number of bytes before the first element is not offered by torch; odd elements are
    s = kda.gated_scan_step(xv[:9], gv[:9], torch.zeros(9, C, device="cuda"), A_log=d["A"])
    t = kda.gated_scan_step(d["x"][:9], d["g"][:9], torch.zeros(9, C, device="cuda"), A_log=d["A"])
    assert torch.equal(s, t)


@pytest.mark.parametrize("g", [0.0, 3.0, -1e-7, -0.09, -1.5, float("-inf")])
def test_constant_decays_over_many_segments(g):
    """The same decay everywhere, over segments, blocks of them and blocks of blocks; whole numbers while nothing decays."""
    kda = _kda()
    T, C = 9000, 5
    x = torch.randint(-2, 3, (T, C), generator=torch.Generator().manual_seed(1)).float()
    gs = torch.full((T, C), g)
    h, hT = kda.gated_scan_fwd(x.cuda()[None], gs.cuda()[None])
    if g >= 0:
        assert torch.equal(h[0].cpu(), x.cumsum(0))
    want, wT, tol, tT = ref.scan(ref.f64(x), ref.f64(gs), None, -5.0, False, [0, T], None)
    ref.close(h[0], want, tol, FP, "h")
    ref.close(hT, wT, tT, FP, "final state")
    back = kda.gated_scan_bwd(None, gs.cuda()[None], None, x.flip(0).cuda()[None], need_dg=False)[0]
    ref.close(back[0].flip(0), want, tol, FP, "dx")


def test_rows_outside_sequences_and_broken_offsets():
    """Rows before the first and behind the last sequence stay as they were; offsets that break their rules write nothing
    outside the outputs (guards on both sides)."""
    kda = _kda()
    T, C = 400, 33
    gen = torch.Generator().manual_seed(2)

    def guarded(rows, cols, dtype):
        buf = torch.full((rows * cols + 512,), 7.0, dtype=dtype, device="cuda")
        return buf, buf[256:256 + rows * cols].view(rows, cols)
    x, g, dh = (torch.randn(T, C, generator=gen).cuda() for _ in range(3))
    for cu in ([50, 130, 130, 300], [0, 300, 100, 400], [390, 400, 500, 900], [-5, 40, 41, 2000], [400, 0, 400, 0], [7, 7, 7, 7]):
        cus = torch.tensor(cu, dtype=torch.int32).cuda()
        N = len(cu) - 1
        bh, h = guarded(T, C, FP)
        bT, hT = guarded(N, C, FP)
        kda.gated_scan_fwd(x, g, cu_seqlens=cus, out=h, final_state=hT)
        bx, dx = guarded(T, C, FP)
        bg, dg = guarded(T, C, FP)
        b0, dh0 = guarded(N, C, FP)
        kda.gated_scan_bwd(None, g, x, dh, cu_seqlens=cus, dx=dx, dg=dg, dinitial_state=dh0)
        for buf in (bh, bT, bx, bg, b0):
            assert (buf[:256] == 7).all() and (buf[-256:] == 7).all(), cu
        if cu == sorted(cu) and 0 <= cu[0] and cu[-1] <= T:
            outside = torch.ones(T, dtype=torch.bool)
            outside[cu[0]:cu[-1]] = False
            for t in (h, dx, dg):
                assert (t[outside.cuda()] == 7).all(), cu


def test_states_in_place_and_empty_calls():
    kda = _kda()
    d = _inputs((40, 0, 300), 50, BF, BF, False, True, seed=6)
    a = kda.gated_scan_fwd(d["x"], d["g"], cu_seqlens=d["cu_dev"], initial_state=d["h0"])
    state = d["h0"].clone()
    b = kda.gated_scan_fwd(d["x"], d["g"], cu_seqlens=d["cu_dev"], initial_state=state, final_state=state)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], state) and torch.equal(state[1], d["h0"][1])
    ga = kda.gated_scan_bwd(None, d["g"], a[0], d["dh"], cu_seqlens=d["cu_dev"], initial_state=d["h0"], dfinal_state=d["dhT"])
    grad = d["dhT"].clone()
    gb = kda.gated_scan_bwd(None, d["g"], a[0], d["dh"], cu_seqlens=d["cu_dev"], initial_state=d["h0"], dfinal_state=grad,
                            dinitial_state=grad)
    assert torch.equal(ga[0], gb[0]) and torch.equal(ga[1], gb[1]) and torch.equal(ga[3], grad)
    # workspaces of the user's: overlapping states need a copy there
    size = kda.gated_scan_fwd_workspace_size(d["x"], cu_seqlens=d["cu_dev"], same_states=True)
    state = d["h0"].clone()
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    b = kda.gated_scan_fwd(d["x"], d["g"], cu_seqlens=d["cu_dev"], initial_state=state, final_state=state, workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], state)
    with pytest.raises(kda.KDAError, match="workspace"):
        kda.gated_scan_fwd(d["x"], d["g"], cu_seqlens=d["cu_dev"], initial_state=state, final_state=state,
                           workspace=ws[:kda.gated_scan_fwd_workspace_size(d["x"], cu_seqlens=d["cu_dev"])])
    grad = d["dhT"].clone()
    ws = torch.empty(kda.gated_scan_bwd_workspace_size(d["dh"], cu_seqlens=d["cu_dev"], same_states=True), dtype=torch.uint8, device="cuda")
    gb = kda.gated_scan_bwd(None, d["g"], a[0], d["dh"], cu_seqlens=d["cu_dev"], initial_state=d["h0"], dfinal_state=grad,
                            dinitial_state=grad, workspace=ws)
    assert torch.equal(ga[0], gb[0]) and torch.equal(ga[3], grad)
    e = torch.empty(2, 0, 50, dtype=BF, device="cuda")
    h, hT = kda.gated_scan_fwd(e, e, initial_state=d["h0"][:2].contiguous())
    assert h.shape == (2, 0, 50) and torch.equal(hT, d["h0"][:2])
    g = kda.gated_scan_bwd(None, e, e, e, A_log=torch.zeros(50, device="cuda"), dfinal_state=d["h0"][:2].contiguous())
    assert torch.equal(g[3], d["h0"][:2]) and (g[2] == 0).all()
    z = kda.gated_scan_fwd(e, e)[1]
    assert (z == 0).all()


@pytest.mark.parametrize("dtype", [FP, BF])
def test_packed_output(dtype):
    """The forward's 8-bit copy of h is what act_pack makes of the returned h; rows outside every sequence are left alone."""
    kda = _kda()
    for lens, C in (((300, 1, 0, 77), 200), ((513,), 129), ((64, 64), 128), ((10,), 5)):
        d = _inputs(lens, C, dtype, dtype, False, False, seed=C)
        h, _, p = kda.gated_scan_fwd(d["x"], d["g"], cu_seqlens=d["cu_dev"], pack=True)
        q = kda.act_pack(h)
        assert torch.equal(p.codes, q.codes) and torch.equal(p.scales, q.scales)
    T = 300
    x = torch.randn(T, 140, device="cuda").to(dtype)
    cu = torch.tensor([20, 60, 250], dtype=torch.int32, device="cuda")
    mine = kda.Packed(torch.full((T, 140), 9, dtype=torch.int8, device="cuda"), torch.full((T, 2), 9.0, device="cuda"))
    h = torch.zeros_like(x)
    kda.gated_scan_fwd(x, -x.abs(), cu_seqlens=cu, out=h, pack=mine)
    q = kda.act_pack(h)
    assert torch.equal(mine.codes[20:250], q.codes[20:250]) and torch.equal(mine.scales[20:250], q.scales[20:250])
    for t in mine:
        assert (t[:20] == 9).all() and (t[250:] == 9).all()


@pytest.mark.parametrize("types", [(FP, FP), (BF, BF), (BF, FP)], ids=["fp32", "bf16", "bf16-fp32"])
def test_step(types):
    kda = _kda()
    for N, C, logits, complement in ((1, 1, False, False), (3, 2048, True, False), (70, 2051, False, True), (300, 40, True, True)):
        d = _inputs((N,), C, *types, logits, False, seed=N)
        n_slots = N + 3
        gen = torch.Generator().manual_seed(N)
        state = torch.randn(n_slots, C, generator=gen).cuda()
        slots = torch.randperm(n_slots, generator=gen)[:N].to(torch.int32)
        if N > 4:
            slots[1], slots[2], slots[-1] = -1, n_slots, slots[0]      # empty, empty, named twice
        new = torch.full_like(state, 7.0)
        h = kda.gated_scan_step(d["x"], d["g"], state, A_log=d["A"], complement=complement, slots=slots.cuda(), new_state=new)
        seen = {}
        for n, s in enumerate(slots.tolist()):
            if not 0 <= s < n_slots or s in seen:
                assert (h[n] == 0).all()
                continue
            seen[s] = n
        rows = list(seen.values())
        at = torch.tensor(list(seen.keys()))
        S = ref.f64(state)[at.numpy()]
        want, _, tol, _ = ref.scan(ref.f64(d["x"])[rows], ref.f64(d["g"])[rows], ref.f64(d["A"]), -5.0, complement,
                                   list(range(len(rows) + 1)), S)
        ref.close(h[rows], want, tol, types[0], "h")
        ref.close(new[at.cuda()], want, tol, FP, "state")
        untouched = [s for s in range(n_slots) if s not in seen]
        assert (new[untouched] == 7).all()
        inplace = state.clone()
        h2 = kda.gated_scan_step(d["x"], d["g"], inplace, A_log=d["A"], complement=complement, slots=slots.cuda())
        assert torch.equal(h2, h) and torch.equal(inplace[at.cuda()], new[at.cuda()])


def test_step_continues_forward():
    """Tokens decoded one by one from a prefill's final state match the prefill of the whole, to float32."""
    kda = _kda()
    N, T, C = 4, 40, 70
    d = _inputs((T,) * N, C, FP, FP, True, True, seed=8)
    v = lambda t: t.view(N, T, C)  # noqa: E731
    whole, last = kda.gated_scan_fwd(v(d["x"]), v(d["g"]), A_log=d["A"], initial_state=d["h0"])
    cut = 25
    _, state = kda.gated_scan_fwd(v(d["x"])[:, :cut].contiguous(), v(d["g"])[:, :cut].contiguous(), A_log=d["A"],
                                  initial_state=d["h0"])
    for t in range(cut, T):
        h = kda.gated_scan_step(v(d["x"])[:, t], v(d["g"])[:, t], state, A_log=d["A"])
        assert torch.allclose(h, whole[:, t], rtol=1e-5, atol=1e-5)
    assert torch.allclose(state, last, rtol=1e-5, atol=1e-5)


def test_repeats_bit_for_bit_streams_and_graph():
    """Results do not depend on the order of workgroups; a given stream is used; a captured call replays on fresh inputs."""
    kda = _kda()
    d = _inputs((3000, 1, 777), 520, BF, BF, True, True, seed=11)
    kw = dict(A_log=d["A"], complement=True, cu_seqlens=d["cu_dev"], initial_state=d["h0"])

    def both():
        h, hT, p = kda.gated_scan_fwd(d["x"], d["g"], pack=True, **kw)
        return [h, hT, *p, *kda.gated_scan_bwd(d["x"], d["g"], p, d["dh"], dfinal_state=d["dhT"], **kw)]
    first = both()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, both()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = kda.gated_scan_fwd(d["x"], d["g"], stream=side, **kw)
    side.synchronize()
    assert torch.equal(other[0], first[0]) and torch.equal(other[1], first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for i in range(3):
        d["x"].copy_(torch.randn_like(d["x"].float()))
        d["dh"].copy_(torch.randn_like(d["x"].float()))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(kept, both())), i


def test_many_sequences():
    """Thousands of packed sequences (the offsets are searched), empty ones among them and at the end, also as a batch of equal
    lengths."""
    kda = _kda()
    gen = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 4, (3000,), generator=gen).tolist() + [500] + [0] * 700 + [70, 0, 0]
    d = _inputs(lens, 36, BF, BF, True, True, seed=1)
    h, hT = kda.gated_scan_fwd(d["x"], d["g"], A_log=d["A"], cu_seqlens=d["cu_dev"], initial_state=d["h0"])
    want, wT, tol, tT = _fwd_ref(d, False)
    ref.close(h, want, tol, BF, "h")
    ref.close(hT, wT, tT, FP, "final state")
    hs = torch.from_numpy(want).to(BF).cuda()
    got = kda.gated_scan_bwd(None, d["g"], hs, d["dh"], A_log=d["A"], cu_seqlens=d["cu_dev"], initial_state=d["h0"],
                             dfinal_state=d["dhT"])
    want, tol = ref.scan_bwd(None, ref.f64(d["g"]), ref.f64(hs), ref.f64(d["dh"]), ref.f64(d["A"]), -5.0, False, d["cu"],
                             ref.f64(d["h0"]), ref.f64(d["dhT"]))
    for name, a, b, t, ty in zip(("dx", "dg", "dA_log", "dinitial_state"), got, want, tol, (BF, BF, FP, FP)):
        ref.close(a, b, t, ty, name)


def test_one_activation_packed_the_other_not():
    kda = _kda()
    d = _inputs((400, 7), 150, BF, BF, True, True, seed=2)
    h = torch.from_numpy(_fwd_ref(d, True)[0]).to(BF).cuda()
    for hs, xs in ((kda.act_pack(h), d["x"]), (h, kda.act_pack(d["x"]))):
        got = kda.gated_scan_bwd(xs, d["g"], hs, d["dh"], A_log=d["A"], complement=True, cu_seqlens=d["cu_dev"], initial_state=d["h0"],
                                 dfinal_state=d["dhT"])
        val = lambda t: ref.values(*t) if isinstance(t, kda.Packed) else ref.f64(t)  # noqa: E731
        want, tol = ref.scan_bwd(val(xs), ref.f64(d["g"]), val(hs), ref.f64(d["dh"]), ref.f64(d["A"]), -5.0, True, d["cu"],
                                 ref.f64(d["h0"]), ref.f64(d["dhT"]))
        for name, a, b, t, ty in zip(("dx", "dg", "dA_log", "dinitial_state"), got, want, tol, (BF, BF, FP, FP)):
            ref.close(a, b, t, ty, name)


@pytest.mark.parametrize("g_min", [-0.05, -1.0, -300.0])
def test_lower_bounds_of_the_gate(g_min):
    """Decays that never come near e^-0.1, that straddle it, and that underflow."""
    kda = _kda()
    for complement in (False, True):
        d = _inputs((300,), 40, FP, FP, True, True, seed=4)
        kw = dict(A_log=d["A"], g_min=g_min, complement=complement, cu_seqlens=d["cu_dev"], initial_state=d["h0"])
        h, hT = kda.gated_scan_fwd(d["x"], d["g"], **kw)
        want, wT, tol, tT = _fwd_ref(d, complement, g_min)
        ref.close(h, want, tol, FP, "h")
        ref.close(hT, wT, tT, FP, "final state")
        got = kda.gated_scan_bwd(d["x"], d["g"], h, d["dh"], **kw)
        want, tol = ref.scan_bwd(ref.f64(d["x"]), ref.f64(d["g"]), ref.f64(h), ref.f64(d["dh"]), ref.f64(d["A"]), g_min, complement,
                                 d["cu"], ref.f64(d["h0"]), None)
        for name, a, b, t in zip(("dx", "dg", "dA_log", "dinitial_state"), got, want, tol):
            ref.close(a, b, t, FP, name)


def test_calls_at_once():
    """Calls on several streams, each with its own workspace, wait for their own segments only; one caller's workspace serves calls
    that follow one another, of other sizes too."""
    kda = _kda()
    sizes = [(6000, 384), (3000, 1024), (9000, 130), (20000, 64)]
    data = [_inputs((T,), C, BF, BF, True, False, seed=T) for T, C in sizes]
    call = lambda d, **kw: kda.gated_scan_fwd(d["x"], d["g"], A_log=d["A"], cu_seqlens=d["cu_dev"], **kw)  # noqa: E731
    want = [call(d) for d in data]
    streams = [torch.cuda.Stream() for _ in sizes]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [call(d, stream=s) for d, s in zip(data, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    need = max(kda.gated_scan_fwd_workspace_size(d["x"], cu_seqlens=d["cu_dev"]) for d in data)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for d, b in zip(data, want):
            a = call(d, workspace=ws)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_large_offsets():
    """More than 2^32 bytes of rows: the last rows are computed from their own inputs."""
    kda = _kda()
    T, C = 70000, 16400                                    # 2.3 GB a tensor of bf16, rows behind 2^31 bytes
    x = torch.zeros(T, C, dtype=BF, device="cuda")
    g = torch.full((T, C), -0.5, dtype=BF, device="cuda")
    tail = torch.randn(300, C, device="cuda").to(BF)
    x[-300:] = tail
    h, hT = kda.gated_scan_fwd(x[None], g[None])
    want, wT = kda.gated_scan_fwd(tail[None], g[None, :300])
    assert (h[0, :-300] == 0).all()
    # the same recurrence from a zero state; tiles start elsewhere, so float32 roundings may differ before the rounding to bf16
    assert torch.allclose(h[0, -300:].float(), want[0].float(), rtol=2.0 ** -7, atol=1e-5)
    assert torch.allclose(hT, wT, rtol=1e-5, atol=1e-5)
