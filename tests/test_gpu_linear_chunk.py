"""GPU tests of kda_linear_chunk_fwd and kda_linear_chunk_bwd against the recurrence in float64.

Every element is held to linear_ref.bound.  That bound takes each rounding at its worst and all of one sign; since
roundings of a sum's terms are independent, the 2-norm of the difference is also held to what they come to together:
a rounding to bf16 is at most 2^-8 and 2^-8 / sqrt(3) in the mean square, and an output sees at most three (score or
state operand of its two parts, and itself), so 2^-8; float32 results (states, dg, all results of float32
calls) to 1e-5."""
import numpy as np
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu

TOL2 = {torch.bfloat16: 2.0 ** -8, torch.float32: 1e-5}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_20_amd as kda
    kda.load_library()


def _inputs(lens, H, Hk, Dk, Dv, dtype, per_head, states=True, seed=0, decay=0.3, tail=0, head=0):
    """Packed sequences; `head` / `tail` rows before and behind them belong to none."""
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    R, N = head + sum(lens) + tail, len(lens)
    cu = [head + sum(lens[:i]) for i in range(N + 1)]
    d = dict(q=rnd(R, Hk, Dk).to(dtype), k=(rnd(R, Hk, Dk) / Dk ** 0.5).to(dtype), v=rnd(R, H, Dv).to(dtype),
             do=rnd(R, H, Dv).to(dtype),
             g=-torch.rand((H,) if per_head else (R, H), generator=gen) * 2 * decay,
             h0=rnd(N, H, Dk, Dv) if states else None, dhT=rnd(N, H, Dk, Dv) if states else None,
             cu=torch.tensor(cu, dtype=torch.int32))
    return {x: y if y is None else y.cuda() for x, y in d.items()}, cu


def _forward_check(d, cu, o, hT, scale):
    a = {x: ref.f64(d[x]) for x in ("q", "k", "v", "g", "h0")}
    ro, rs = ref.forward(a["q"], a["k"], a["v"], a["g"], scale, cu, a["h0"])
    mo, ms = ref.forward(abs(a["q"]), abs(a["k"]), abs(a["v"]), a["g"], abs(scale), cu,
                         None if a["h0"] is None else abs(a["h0"]))
    n = max([cu[i + 1] - cu[i] for i in range(len(cu) - 1)])
    go, gs = ref.f64(o).reshape(ro.shape), ref.f64(hT)
    rows = slice(cu[0], cu[-1])
    assert np.all(np.abs(go - ro)[rows] <= ref.bound(ro, mo, o.dtype, n)[rows])
    assert np.all(np.abs(gs - rs) <= ref.bound(rs, ms, torch.float32, n))
    assert ref.rel2(go[rows], ro[rows]) <= TOL2[o.dtype]
    assert ref.rel2(gs, rs) <= TOL2[torch.float32]


def _backward_check(d, cu, got, scale):
    a = {x: ref.f64(d[x]) for x in ("q", "k", "v", "g", "do", "h0", "dhT")}
    m = {x: y if y is None or x == "g" else np.abs(y) for x, y in a.items()}
    order = ("q", "k", "v", "g", "do")
    want = ref.backward(*(a[x] for x in order), scale, cu, a["h0"], a["dhT"])
    mags = ref.backward(*(m[x] for x in order), abs(scale), cu, m["h0"], m["dhT"])
    n = max([cu[i + 1] - cu[i] for i in range(len(cu) - 1)])
    rows = slice(cu[0], cu[-1])
    for name, x, r, mag in zip(("dq", "dk", "dv", "dg", "dh0"), got, want, mags):
        y = ref.f64(x).reshape(r.shape)
        if name == "dg":
            # dg's terms are differences of running sums over up to 32 chunks, which the largest of them bounds
            mag = np.full_like(mag, mag.max()) if mag.size else mag
        if name != "dh0" and not (name == "dg" and r.ndim == 1):
            y, r, mag = y[rows], r[rows], mag[rows]
        if r.size == 0:
            continue
        assert np.all(np.abs(y - r) <= ref.bound(r, mag, x.dtype, n)), name
        if name == "dg" and r.ndim == 1:
            # A sum over tokens whose values cancel: an error of e |dg_t| a token is e sum |dg_t| here, whatever is left
            # of the sum itself.  sum |dg_t|, per head:
            every = ref.backward(*(a[x] for x in order[:3]), np.broadcast_to(a["g"], d["v"].shape[:2]), a["do"], scale, cu,
                                 a["h0"], a["dhT"])[3]
            assert np.linalg.norm(y - r) <= TOL2[x.dtype] * np.linalg.norm(np.abs(every).sum(0)), name
            continue
        assert ref.rel2(y, r) <= TOL2[x.dtype], name


LENS = [[1], [63], [64], [65], [130, 0, 1, 31, 32, 33], [0], [300, 257], [1100], [520, 3, 700, 256, 512], [2100]]
HEADS = [(2, 2, 64, 64), (2, 1, 128, 64), (3, 3, 64, 128), (2, 2, 128, 128)]


def _fwd(d, scale, **kw):
    import gated_delta_rule_20_amd as kda
    return kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], scale=scale, cu_seqlens=d["cu"], initial_state=d["h0"], **kw)


def _bwd(d, scale, **kw):
    import gated_delta_rule_20_amd as kda
    return kda.linear_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], scale=scale, cu_seqlens=d["cu"],
                                initial_state=d["h0"], dfinal_state=d["dhT"], **kw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,Hk,Dk,Dv", HEADS)
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_forward(lens, H, Hk, Dk, Dv, dtype):
    per_head, states = len(lens) % 2 == 0, lens != [300, 257]
    d, cu = _inputs(lens, H, Hk, Dk, Dv, dtype, per_head, states, seed=len(lens))
    o, hT = _fwd(d, 0.8)
    _forward_check(d, cu, o, hT, 0.8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,Hk,Dk,Dv", HEADS)
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_backward(lens, H, Hk, Dk, Dv, dtype):
    per_head, states = len(lens) % 2 == 1, lens != [300, 257]
    d, cu = _inputs(lens, H, Hk, Dk, Dv, dtype, per_head, states, seed=10 + len(lens))
    _backward_check(d, cu, _bwd(d, 0.8), 0.8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T", [(3, 70), (2, 600), (1, 1), (2, 0)])
def test_batched_layout(B, T, dtype):
    import gated_delta_rule_20_amd as kda
    d, cu = _inputs([T] * B, 2, 2, 64, 64, dtype, False, seed=B)
    x = {n: d[n].view((B, T) + d[n].shape[1:]) for n in ("q", "k", "v", "g", "do")}
    o, hT = kda.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], initial_state=d["h0"])
    assert o.shape == x["v"].shape
    _forward_check(d, cu, o, hT, 1.0)
    got = kda.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], initial_state=d["h0"], dfinal_state=d["dhT"])
    assert got[0].shape == x["q"].shape and got[3].shape == x["g"].shape
    _backward_check(d, cu, got, 1.0)


@pytest.mark.parametrize("decay", [0.0, 0.01, 30.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_decay_range(decay, dtype):
    """No decay, hardly any, and one that forgets within a token; with resets (-inf, -200, -1e30) and values above 0."""
    d, cu = _inputs([700, 90], 2, 2, 64, 64, dtype, False, seed=3, decay=decay)
    g = d["g"]
    g[5], g[64], g[100, 0], g[128, 1], g[300:310] = -float("inf"), -200.0, -1e30, -float("inf"), -90.0
    g[700] = -float("inf")
    g[400] = 3.0
    o, hT = _fwd(d, 1.0)
    _forward_check(d, cu, o, hT, 1.0)
    _backward_check(d, cu, _bwd(d, 1.0), 1.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_sequences(dtype):
    """More packed sequences than are searched (128): empty and one-token ones and one long enough to be cut."""
    r = np.random.RandomState(0)
    lens = r.randint(0, 5, 1300).tolist()
    lens[700], lens[1299] = 500, 130
    d, cu = _inputs(lens, 2, 1, 64, 64, dtype, False, seed=17, head=3, tail=5)
    o, hT = _fwd(d, 1.0)
    _forward_check(d, cu, o, hT, 1.0)
    _backward_check(d, cu, _bwd(d, 1.0), 1.0)


def test_rows_outside_the_sequences_stay():
    d, cu = _inputs([70, 0, 300], 2, 1, 64, 64, torch.bfloat16, False, seed=4, head=9, tail=77)
    for x in ("q", "k", "v", "do", "g"):        # what is there must not reach the sequences either
        d[x][:9] = float("nan")
        d[x][cu[-1]:] = float("inf")
    out = torch.full_like(d["v"], 7.0)
    o, hT = _fwd(d, 1.0, out=out)
    assert o is out and bool((out[:9] == 7.0).all()) and bool((out[cu[-1]:] == 7.0).all())
    outs = dict(dq=torch.full_like(d["q"], 7.0), dk=torch.full_like(d["k"], 7.0), dv=torch.full_like(d["v"], 7.0),
                dg=torch.full_like(d["g"], 7.0))
    got = _bwd(d, 1.0, **outs)
    for x in outs.values():
        assert bool((x[:9] == 7.0).all()) and bool((x[cu[-1]:] == 7.0).all())
    clean = {n: (x if x is None or x.shape[0] != d["q"].shape[0] else torch.nan_to_num(x, 0.0, 0.0, 0.0))
             for n, x in d.items()}
    _forward_check(clean, cu, torch.nan_to_num(o), hT, 1.0)
    _backward_check(clean, cu, got, 1.0)


@pytest.mark.parametrize("lens", [[700, 90], [100, 90]], ids=str)
def test_states_in_place(lens):
    """final_state = initial_state and dinitial_state = dfinal_state give the same bits as separate arrays."""
    d, cu = _inputs(lens, 2, 2, 128, 64, torch.bfloat16, False, seed=5)
    o, hT = _fwd(d, 1.0)
    got = _bwd(d, 1.0)
    keep = d["h0"].clone(), d["dhT"].clone()
    o2, h2 = _fwd(d, 1.0, final_state=d["h0"])
    assert torch.equal(o2, o) and torch.equal(h2, hT) and h2 is d["h0"]
    d["h0"] = keep[0]
    got2 = _bwd(d, 1.0, dinitial_state=d["dhT"])
    assert all(torch.equal(x, y) for x, y in zip(got, got2))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_checkpoints(dtype):
    """Slots at multiples of checkpoint_every chunks strictly inside a sequence; the others are left as they were."""
    lens = [1000, 128, 129, 0, 64]
    d, cu = _inputs(lens, 2, 2, 64, 64, dtype, True, seed=6)
    ck = torch.full((5, 3, 2, 64, 64), 7.0, device="cuda")
    _fwd(d, 1.0, checkpoints=ck, checkpoint_every=2)
    a = {x: ref.f64(d[x]) for x in ("q", "k", "v", "g", "h0")}
    _, _, want = ref.forward(a["q"], a["k"], a["v"], a["g"], 1.0, cu, a["h0"], every=128)
    _, _, mags = ref.forward(abs(a["q"]), abs(a["k"]), abs(a["v"]), a["g"], 1.0, cu, abs(a["h0"]), every=128)
    got = ref.f64(ck)
    for s in range(5):
        for j in range(3):
            w = want.get((s, 128 * (j + 1)))
            if w is None:
                assert np.all(got[s, j] == 7.0)
            else:
                assert np.all(np.abs(got[s, j] - w) <= ref.bound(w, mags[s, 128 * (j + 1)], torch.float32, 1000))


def test_resume_equals_one_call():
    """A sequence in two calls, the second from the first one's final state: the chunks fall alike, so outputs are close
    to one call's within their own bounds."""
    import gated_delta_rule_20_amd as kda
    d, cu = _inputs([600], 2, 2, 64, 64, torch.float32, False, seed=7)
    parts, S = [], d["h0"]
    for a, b in ((0, 37), (37, 600)):
        o, S = kda.linear_chunk_fwd(*(d[x][None, a:b].contiguous() for x in ("q", "k", "v", "g")), initial_state=S)
        parts.append(o[0])
    _forward_check(d, cu, torch.cat(parts), S, 1.0)


def test_gradients_against_differences():
    """Directional derivatives of a loss of the float64 recurrence (central differences) against the kernel's float32
    gradients: the step 1e-5 leaves 1e-10 of the third derivative and 1e-11 of rounding, far below float32's 1e-6."""
    d, cu = _inputs([70, 5], 2, 1, 64, 64, torch.float32, False, seed=8)
    a = {x: ref.f64(d[x]) for x in ("q", "k", "v", "g", "do", "h0", "dhT")}

    def loss(b):
        o, S = ref.forward(b["q"], b["k"], b["v"], b["g"], 0.8, cu, b["h0"])
        return float((o * a["do"]).sum() + (S * a["dhT"]).sum())

    got = dict(zip(("q", "k", "v", "g", "h0"), _bwd(d, 0.8)))
    r = np.random.RandomState(9)
    for x, grad in got.items():
        u = r.randn(*a[x].shape)
        e = 1e-5
        diff = (loss({**a, x: a[x] + e * u}) - loss({**a, x: a[x] - e * u})) / (2 * e)
        terms = ref.f64(grad) * u
        assert abs(diff - terms.sum()) <= 1e-5 * np.abs(terms).sum(), x


def test_without_dg_and_state_gradient():
    d, cu = _inputs([400, 9], 2, 2, 64, 64, torch.bfloat16, False, seed=11)
    got = _bwd(d, 1.0)
    less = _bwd(d, 1.0, need_dg=False)
    assert less[3] is None
    for i in (2, 4):
        assert torch.equal(less[i], got[i])
    # the state enters dq and dk with fewer terms where dg is not wanted; both hold to their own bounds
    _backward_check(d, cu, (*less[:3], got[3], less[4]), 1.0)


def test_broken_offsets_stay_inside():
    """cu_seqlens that decreases, leaves the rows or overlaps: wrong results, but no access outside the tensors (each
    output has a guard behind it)."""
    import gated_delta_rule_20_amd as kda
    d, _ = _inputs([900], 2, 1, 64, 64, torch.float32, True, seed=12)
    for cu in ([-5, 400, 100, 5000, 20], [0, 900, 0, 900, 0], [900, 900, 900, 0, 900], [2 ** 31 - 1, -2 ** 31, 7, 800, 900]):
        cu = torch.tensor(cu, dtype=torch.int32).cuda()
        buf = torch.full((900 + 64, 2, 64), 7.0, device="cuda")
        h = torch.zeros((4, 2, 64, 64), device="cuda")
        kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], cu_seqlens=cu, initial_state=h, out=buf[:900])
        assert bool((buf[900:] == 7.0).all())
        dv = torch.full((900 + 64, 2, 64), 7.0, device="cuda")
        kda.linear_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], cu_seqlens=cu, initial_state=h, dfinal_state=h, dv=dv[:900])
        assert bool((dv[900:] == 7.0).all())
    # the same with more sequences than are searched
    cu = torch.from_numpy(np.random.RandomState(3).randint(-100, 1100, 401).astype(np.int32)).cuda()
    h = torch.zeros((400, 2, 64, 64), device="cuda")
    buf, dv = torch.full((900 + 64, 2, 64), 7.0, device="cuda"), torch.full((900 + 64, 2, 64), 7.0, device="cuda")
    kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], cu_seqlens=cu, initial_state=h, out=buf[:900])
    kda.linear_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], cu_seqlens=cu, initial_state=h, dfinal_state=h, dv=dv[:900])
    assert bool((buf[900:] == 7.0).all()) and bool((dv[900:] == 7.0).all())


def test_non_finite_stays_in_its_sequence_and_chunk():
    d, cu = _inputs([200, 200], 2, 2, 64, 64, torch.bfloat16, False, seed=13)
    o, hT = _fwd(d, 1.0)
    d["v"][130], d["k"][150] = float("inf"), float("nan")     # in the first sequence's third chunk
    o2, h2 = _fwd(d, 1.0)
    assert torch.equal(o2[:128], o[:128]) and torch.equal(o2[200:], o[200:]) and torch.equal(h2[1], hT[1])
    assert not bool(torch.isfinite(o2[150:200]).any())


def test_graph_replays():
    """Forward and backward captured on static buffers, replayed on fresh inputs, equal to eager calls bit for bit."""
    d, cu = _inputs([700, 90], 2, 1, 64, 64, torch.bfloat16, True, seed=14)
    names = ("q", "k", "v", "g", "do", "h0", "dhT")
    run = lambda x: (*_fwd(x, 1.0), *_bwd(x, 1.0))  # noqa: E731
    run(d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(d)
    for i in range(3):
        fresh, _ = _inputs([700, 90], 2, 1, 64, 64, torch.bfloat16, True, seed=20 + i)
        for x in names:
            d[x].copy_(fresh[x])
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, run(fresh)):
            assert torch.equal(x, y)


def test_streams_at_once():
    """Calls on several streams at the same time equal the same calls one after another."""
    jobs = [_inputs([500 + 40 * i, 64], 2, 2, 64, 128, torch.bfloat16, False, seed=30 + i)[0] for i in range(4)]
    want = [(*_fwd(d, 1.0), *_bwd(d, 1.0)) for d in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = []
    for d, s in zip(jobs, streams):
        with torch.cuda.stream(s):
            got.append((*_fwd(d, 1.0, stream=s), *_bwd(d, 1.0, stream=s)))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_binding_refusals():
    """Shapes, types, layouts and devices that the binding turns away before the library is called."""
    import gated_delta_rule_20_amd as kda
    d, _ = _inputs([64], 4, 2, 64, 64, torch.bfloat16, True, seed=15)
    q, k, v, g = (d[x][None] if x != "g" else d[x] for x in ("q", "k", "v", "g"))
    ok = dict(initial_state=d["h0"])
    kda.linear_chunk_fwd(q, k, v, g, **ok)
    wide = torch.zeros((1, 64, 2, 128), dtype=torch.bfloat16, device="cuda")
    bad = [((q.float(), k, v, g), {}, "k must be"), ((q, k[:, :9], v, g), {}, "q's shape"), ((q, k, v[:, :9], g), {}, "leading axes"),
           ((q, k, v[:, :, :3].contiguous(), g[:3]), {}, "multiple"), ((q, k, v, g[:3]), {}, "g must be"), ((q, k, v, g.cpu()), {}, "device"),
           ((q, k, v, g.bfloat16()), {}, "g must be"), ((wide[..., :64], k, v, g), {}, "contiguous"),
           ((q, k, v, g), dict(initial_state=d["h0"][:, :2]), "contiguous|initial_state"),
           ((q, k, v, g), dict(cu_seqlens=d["cu"].long()), "cu_seqlens"), ((q, k, v, g), dict(cu_seqlens=d["cu"][:1]), "cu_seqlens"),
           ((q, k, v, g), dict(out=v.float()), "out"), ((q, k, v, g), dict(out=v[:, :9].contiguous()), "out"),
           ((q, k, v, g), dict(checkpoints=torch.zeros((1, 1, 4, 64, 64), device="cuda")), "checkpoints"),
           ((q[0], k[0], v[0], g), {}, "q must be")]
    for args, kw, msg in bad:
        with pytest.raises(ValueError, match=msg):
            kda.linear_chunk_fwd(*args, **kw)
    with pytest.raises(kda.KDAError, match="head dims"):
        x = torch.zeros((1, 8, 2, 32), dtype=torch.bfloat16, device="cuda")
        kda.linear_chunk_fwd(x, x, x, g[:2])
    with pytest.raises(kda.KDAError, match="workspace"):
        long = torch.zeros((1, 4096, 1, 64), device="cuda")
        kda.linear_chunk_fwd(long, long, long, g[:1].contiguous(), workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="d_o"):
        kda.linear_chunk_bwd(q, k, v, g, d["do"][None][:, :9])
    with pytest.raises(ValueError, match="dfinal_state"):
        kda.linear_chunk_bwd(q, k, v, g, d["do"][None], dfinal_state=d["h0"][0])


def test_long_packed_call_beyond_4_gib():
    """Rows whose byte offset passes 2^32 in q, k, v and o: the last sequence of a long batch equals a call of its own."""
    import gated_delta_rule_20_amd as kda
    H, D, T = 64, 128, 270000                          # 64 * 128 * 2 bytes a row: 4.4 GB
    gen = torch.Generator(device="cuda").manual_seed(16)
    x = torch.randn((T, H, D), generator=gen, device="cuda", dtype=torch.bfloat16)
    y = torch.randn((T, H, D), generator=gen, device="cuda", dtype=torch.bfloat16)
    g = -torch.rand(H, generator=gen, device="cuda") * 0.5
    cu = torch.tensor([0, T - 200, T], dtype=torch.int32, device="cuda")
    o, hT = kda.linear_chunk_fwd(x, y, x, g, scale=0.1, cu_seqlens=cu)
    tail = [t[-200:][None].contiguous() for t in (x, y, x)]
    o1, h1 = kda.linear_chunk_fwd(*tail, g, scale=0.1)
    # the calls cut the 200 tokens into segments differently, so states agree to float32 and outputs to a rounding
    assert ref.rel2(ref.f64(hT[1]), ref.f64(h1[0])) <= 1e-5
    assert ref.rel2(ref.f64(o[-200:]), ref.f64(o1[0])) <= TOL2[torch.bfloat16]
    del o, hT
    got = kda.linear_chunk_bwd(x, y, x, g, y, scale=0.1, cu_seqlens=cu, need_dg=False)
    one = kda.linear_chunk_bwd(*tail, g, tail[1], scale=0.1, need_dg=False)
    for a, b in zip(got[:3], one[:3]):
        assert ref.rel2(ref.f64(a[-200:]), ref.f64(b[0])) <= TOL2[torch.bfloat16]
