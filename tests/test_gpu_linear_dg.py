"""GPU tests of the decays' gradient (dg of kda_linear_chunk_bwd) where its terms differ widely in size, against the
recurrence in float64.

dg_u = e^{g_u} <S_{u-1}, dS_u> is a sum over pairs s < u <= t of what token s (or the entering state) writes and token t (or
the leaving state's gradient) reads.  The kernel adds the pairs of one chunk directly; what crosses the whole chunk, w = e^{G_end}
<S, dS>, it takes from R = <state, its gradient>, which is formed anew at every anchor (every 512 tokens, and at a
sequence's end) and carried backwards from there by the chunks' own terms.  So an element is off by float32 roundings of its own
terms (``mags``: the formula on absolute values) and, unless w is known to be 0, of the terms that R has
passed since its anchor."""
import numpy as np
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16]
TOL2 = 1e-5          # dg is a float32 result; the 2-norm that test_gpu_linear_chunk.py holds all of them to


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_20_amd as kda
    kda.load_library()


def _inputs(lens, H, dtype, g, h0=None, dhT=None, do=1.0, seed=0, Hk=None, D=64):
    """Packed sequences with log-decays g [R, H]; h0, dhT, do: sizes of the entering states, of the leaving ones' gradients
    and of the outputs' gradients (None: not given)."""
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    R, N, Hk = sum(lens), len(lens), Hk or H
    cu = [sum(lens[:i]) for i in range(N + 1)]
    d = dict(q=rnd(R, Hk, D).to(dtype), k=(rnd(R, Hk, D) / 8).to(dtype), v=rnd(R, H, D).to(dtype),
             do=(do * rnd(R, H, D)).to(dtype), g=g.float(), h0=None if h0 is None else h0 * rnd(N, H, D, D),
             dhT=None if dhT is None else dhT * rnd(N, H, D, D))
    return {x: y if y is None else y.cuda() for x, y in d.items()}, cu


def _run(d, cu):
    import gated_delta_rule_20_amd as kda
    return kda.linear_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], initial_state=d["h0"], dfinal_state=d["dhT"],
                                cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())


def _want(d, cu):
    """dg, and the terms' magnitudes, in float64."""
    a = {x: ref.f64(y) for x, y in d.items()}
    m = {x: y if y is None or x == "g" else np.abs(y) for x, y in a.items()}
    return tuple(ref.backward(x["q"], x["k"], x["v"], x["g"], x["do"], 1.0, cu, x["h0"], x["dhT"])[3] for x in (a, m))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", [1e2, 1e4, 1e6])
@pytest.mark.parametrize("at,T", [(0, 64), (0, 61), (64, 128), (70, 130)])
def test_large_state_before_a_strong_decay(at, T, size, dtype):
    """One token forgets all but e^-17 of a state that is far larger than what the chunk adds; nothing but the leaving
    state's gradient reads it.  e^-17 is below a float32's half step of 1, but what it leaves of the state is not
    below the rounding of the chunk's own terms."""
    H = 2
    g = torch.full((T, H), -0.001)
    g[at] = -17.0
    d, cu = _inputs([T], H, dtype, g, h0=size, dhT=1.0, do=0.0, seed=T + at)
    got = ref.f64(_run(d, cu)[3])
    want, mags = _want(d, cu)
    assert ref.rel2(got, want) <= TOL2
    # up to and with the strong decay: what the state's rest contributes, alone
    tol = ref.bound(want, mags.max(0, keepdims=True), torch.float32, T)
    assert np.all(np.abs(got - want) <= tol)
    if size == 1e6:                                        # there the bound is below the values themselves
        assert np.all(np.abs(want[at]) > 2 * tol[at])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("part", ["pairs", "keys", "queries"])
def test_small_elements_among_large_ones(part, dtype):
    """Sequences of one chunk whose dg has no w: pairs of tokens alone, with what the tokens leave for the final state's
    gradient (no outputs' gradients), with what they read from the entering state.  Tokens that forget nearly everything have a
    dg far below their neighbours', made of small terms only, and every element is held to float32 of its own
    terms; the first one without an entering state is 0."""
    H = 3
    lens = [1, 2, 15, 16, 17, 31, 32] + ([33, 48, 49, 63, 64] if dtype == torch.bfloat16 else [])
    R = sum(lens)
    r = np.random.RandomState(5)
    g = -0.002 * torch.rand((R, H), generator=torch.Generator().manual_seed(6))
    for i in r.choice(R, R // 6, replace=False):
        g[i, r.randint(H)] = float(r.choice([-5.0, -12.0, -17.0, -25.0]))
    d, cu = _inputs(lens, H, dtype, g, h0=1.0 if part == "queries" else None, dhT=1.0 if part == "keys" else None,
                    do=0.0 if part == "keys" else 1.0, seed=7)
    got = ref.f64(_run(d, cu)[3])
    want, mags = _want(d, cu)
    err, tol = np.abs(got - want), ref.bound(want, mags, torch.float32, 64)
    assert np.all(err <= tol), (float((err / np.maximum(mags, 1e-30)).max()), int((err > tol).sum()))
    assert ref.rel2(got, want) <= TOL2


def _interval_bound(d, cu, want, mags):
    """Element bound with R's way: its own terms, and those of the 512 tokens that R is carried over (an anchor lies at
    every multiple of 512 tokens and at the end), as magnitudes of q . dq and k . dk, which hold all of a token's y
    and z, and of R itself, which is among the interval's elements."""
    m = {x: None if y is None else np.abs(ref.f64(y)) if x != "g" else ref.f64(y) for x, y in d.items()}
    H = m["v"].shape[1]
    q, k = ref.widen(m["q"], H), ref.widen(m["k"], H)
    mq, mk = ref.backward(q, k, m["v"], m["g"], m["do"], 1.0, cu, m["h0"], m["dhT"])[:2]
    token = (q * mq).sum(-1) + (k * mk).sum(-1)
    passed = np.zeros_like(mags)
    for a, b in zip(cu[:-1], cu[1:]):
        for i in range(a, b, 512):
            rows = slice(i, min(i + 512, b))
            passed[rows] = token[rows].sum(0) + mags[rows].max(0)
    n = max(b - a for a, b in zip(cu[:-1], cu[1:]))
    return ref.bound(want, mags + passed, torch.float32, n)


def _many(n):
    return np.random.RandomState(9).randint(0, 9, n).tolist()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens", [[5000, 0, 1, 3300, 511, 700], [600, *_many(70), 4990, *_many(140), 3200]], ids=["searched", "tabulated"])
@pytest.mark.parametrize("Hk,states", [(32, True), (16, False)])
def test_segments_of_several_anchors(lens, Hk, states, dtype):
    """Enough tokens and heads that a workgroup's segment (1024 tokens) holds two anchors, on sequences of several segments
    among short ones: all gradients of the first and the last two value heads against the recurrence.  Decays forget over
    some 100 to 1000 tokens, and now and then at once, so states reach across anchors and segments."""
    H, R = 32, sum(lens)
    assert R * H > 512 * 512                                # from here on segments are longer than an anchor's interval
    gen = torch.Generator().manual_seed(10)
    g = -0.004 * torch.rand((R, H), generator=gen)
    g[torch.rand((R, H), generator=gen) < 1e-3] = -9.0
    size = 1.0 if states else None
    d, cu = _inputs(lens, H, dtype, g, h0=size, dhT=size, seed=11, Hk=Hk)
    got = [ref.f64(x) for x in _run(d, cu)]
    group = H // Hk
    for first in (0, H - 2):
        heads, kheads = slice(first, first + 2), slice(first // group, (first + 1) // group + 1)
        sub = {x: None if y is None else (y[:, kheads] if x in ("q", "k") else y[:, heads]).contiguous() for x, y in d.items()}
        a = [ref.f64(sub[x]) for x in ("q", "k", "v", "g", "do")]
        want = ref.backward(*a, 1.0, cu, ref.f64(sub["h0"]), ref.f64(sub["dhT"]))
        mags = ref.backward(*(y if i == 3 else np.abs(y) for i, y in enumerate(a)), 1.0, cu,
                            *(None if sub[x] is None else np.abs(ref.f64(sub[x])) for x in ("h0", "dhT")))
        for name, x, w, m, hs in zip(("dq", "dk", "dv", "dg", "dh0"), got, want, mags, (kheads, kheads, heads, heads, heads)):
            x = x[:, hs]
            t = dtype if name in ("dq", "dk", "dv") else torch.float32
            tol = _interval_bound(sub, cu, w, m) if name == "dg" else ref.bound(w, m, t, max(lens))
            assert np.all(np.abs(x - w) <= tol), name
            assert ref.rel2(x, w) <= (2.0 ** -8 if t == torch.bfloat16 else TOL2), name


@pytest.mark.parametrize("H", [2, 32])
@pytest.mark.parametrize("name,where", [("v", "before"), ("k", "before"), ("do", "behind"), ("q", "behind")])
def test_non_finite_gradients(name, where, H):
    """An infinity among q, k, v or d_o reaches no other sequence.  In its own it reaches what the formula carries it to
    (v and k by the state: dq and dg behind them; q and d_o by its gradient: dk, dv and dg before them), its
    own chunk, and dg of up to 512 tokens before it; all else keeps its bits."""
    lens = [2100, 300] if H == 2 else [9000, 300]
    at = lens[0] - 200
    gen = torch.Generator().manual_seed(13)
    g = -0.01 * torch.rand((sum(lens), H), generator=gen)
    d, cu = _inputs(lens, H, torch.bfloat16, g, seed=14)
    clean = _run(d, cu)
    d[name][at] = float("inf")
    got = _run(d, cu)
    chunk, n = at // 64 * 64, lens[0]
    for x, y in zip(got[:4], clean):
        assert torch.equal(x[n:], y[n:])
    assert torch.equal(got[4][1], clean[4][1])
    dq, dk, dv, dg = (torch.eq(x, y).flatten(1).all(1).cpu() for x, y in zip(got[:4], clean))
    if where == "before":                                  # the state behind it, so nothing of dk and dv but its own chunk's
        assert dq[:chunk].all() and dg[:max(0, at - 512)].all()
        rest = torch.arange(n + lens[1])
        rest = (rest < chunk) | (rest >= chunk + 64)
        assert dk[rest].all() and dv[rest].all()
    else:                                                  # the gradient of the state before it
        assert dk[chunk + 64:].all() and dv[chunk + 64:].all() and dg[chunk + 64:].all()
        rest = torch.arange(n + lens[1])
        assert dq[(rest < chunk) | (rest >= chunk + 64)].all()
    assert not torch.isfinite(torch.cat([x[chunk:chunk + 64].flatten().float() for x in got[:4]])).all()
