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
