"""GPU tests of kda_linear_recurrent_step against the recurrence in float64.

Bounds, per element, from the roundings: with x = g log2(e) the decay e^g carries the rounding of x
(|x| 2^-24, so |g| 2^-24 relative) and the hardware exponential's (taken as 2^-22); S' adds two products, each rounded,
and their sum; o sums Dk products in any order and rounds once to its type."""
import numpy as np
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_20_amd as kda
    kda.load_library()


def _inputs(N, H, Hk, Dk, Dv, dtype, per_head, slots, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    d = dict(q=rnd(N, Hk, Dk).to(dtype), k=rnd(N, Hk, Dk).to(dtype), v=rnd(N, H, Dv).to(dtype),
             g=-torch.rand((H,) if per_head else (N, H), generator=gen) * 4, state=rnd(slots, H, Dk, Dv))
    return {x: y.cuda() for x, y in d.items()}


def _check(d, o, new, slots, scale):
    """o [N, H, Dv] and the states of the named slots against float64; the other slots are untouched."""
    H = d["v"].shape[1]
    q, k, v, S0 = ref.widen(ref.f64(d["q"]), H), ref.widen(ref.f64(d["k"]), H), ref.f64(d["v"]), ref.f64(d["state"])
    g = np.broadcast_to(np.minimum(ref.f64(d["g"]), 0.0), v.shape[:2])
    got_o, got_s = ref.f64(o), ref.f64(new)
    seen = set()
    for n, slot in enumerate(slots):
        if not 0 <= slot < S0.shape[0] or slot in seen:
            assert np.all(got_o[n] == 0.0)
            continue
        seen.add(slot)
        a = np.exp(g[n])[:, None, None]
        old, add = a * S0[slot], k[n][:, :, None] * v[n][:, None, :]
        S = old + add
        gm = np.where(np.isfinite(g[n]), np.abs(g[n]), 0.0)[:, None, None]
        tol = np.abs(old) * (gm * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -24) + np.abs(add) * 2.0 ** -24 + np.abs(S) * 2.0 ** -24
        tol = 1.01 * tol + 1e-37
        assert np.all(np.abs(got_s[slot] - S) <= tol), (n, slot)
        ro = scale * np.einsum("hkv,hk->hv", S, q[n])
        Dk = S.shape[1]
        to = abs(scale) * np.einsum("hkv,hk->hv", tol + np.abs(S) * (Dk + 3) * 2.0 ** -24, np.abs(q[n]))
        to = 1.01 * (to + ref.HALF[o.dtype] * (np.abs(ro) + to))
        assert np.all(np.abs(got_o[n] - ro) <= to), (n, slot)
    return seen


CASES = [  # N, H, Hk, Dk, Dv
    (1, 1, 1, 64, 64), (3, 4, 2, 64, 128), (5, 6, 1, 128, 64), (2, 3, 3, 128, 128), (70, 4, 4, 128, 128), (300, 1, 1, 64, 64),
    (33, 9, 3, 128, 64), (65, 5, 5, 64, 128)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("N,H,Hk,Dk,Dv", CASES)
def test_step_in_place(N, H, Hk, Dk, Dv, per_head, dtype):
    import gated_delta_rule_20_amd as kda
    d = _inputs(N, H, Hk, Dk, Dv, dtype, per_head, N + 1)
    state = d["state"].clone()
    o = kda.linear_recurrent_step(d["q"], d["k"], d["v"], d["g"], state, scale=0.7)
    _check(d, o, state, range(N), 0.7)
    assert torch.equal(state[N], d["state"][N])


@pytest.mark.parametrize("N,H", [(9, 2), (150, 3), (600, 1)])
def test_slots_padding_and_repeats(N, H):
    """Rows with slots out of range or named before are empty places; unnamed slots keep their content."""
    import gated_delta_rule_20_amd as kda
    S = N + 40
    d = _inputs(N, H, 1, 64, 64, torch.float32, False, S, seed=1)
    slots = torch.randperm(S, generator=torch.Generator().manual_seed(2))[:N].to(torch.int32)
    slots[0], slots[3], slots[-1] = -1, S, 2 ** 31 - 1
    slots[5] = slots[1]
    slots[N - 2] = slots[1]
    state = d["state"].clone()
    o = kda.linear_recurrent_step(d["q"], d["k"], d["v"], d["g"], state, slots=slots.cuda())
    seen = _check(d, o, state, slots.tolist(), 1.0)
    rest = [s for s in range(S) if s not in seen]
    assert torch.equal(state[rest], d["state"][rest])
    # into another pool: the read one keeps its content, unnamed slots of the written one too
    new = torch.full_like(state, 7.0)
    o2 = kda.linear_recurrent_step(d["q"], d["k"], d["v"], d["g"], d["state"], slots=slots.cuda(), new_state=new)
    assert torch.equal(o2, o) and torch.equal(new[sorted(seen)], state[sorted(seen)])
    assert bool((new[rest] == 7.0).all())


def test_decay_extremes():
    """g = 0 keeps the state, -inf and everything below -177 forgets it, g above 0 counts as 0."""
    import gated_delta_rule_20_amd as kda
    d = _inputs(4, 2, 2, 64, 64, torch.float32, False, 4, seed=3)
    d["g"] = torch.tensor([[0.0, -float("inf")], [-200.0, -1e30], [5.0, -103.0], [-0.0, -1e-30]]).cuda()
    state = d["state"].clone()
    o = kda.linear_recurrent_step(d["q"], d["k"], d["v"], d["g"], state)
    _check(d, o, state, range(4), 1.0)


def test_step_far_in_a_large_pool():
    """Slots whose byte offset passes 2^32."""
    import gated_delta_rule_20_amd as kda
    H, S = 16, 4200          # 1 MiB per slot
    state = torch.zeros((S, H, 128, 128), device="cuda")
    d = _inputs(2, H, H, 128, 128, torch.bfloat16, True, 1, seed=4)
    d["state"] = torch.randn((2, H, 128, 128), generator=torch.Generator().manual_seed(5)).cuda()
    state[4199], state[4097] = d["state"][0], d["state"][1]
    o = kda.linear_recurrent_step(d["q"], d["k"], d["v"], d["g"], state,
                                  slots=torch.tensor([4199, 4097], dtype=torch.int32).cuda())
    _check(d, o, state[[4199, 4097]], [0, 1], 1.0)
    assert float(state[:4097].abs().max()) == 0.0


def test_step_graph_replays():
    import gated_delta_rule_20_amd as kda
    d = _inputs(20, 4, 4, 64, 64, torch.bfloat16, False, 24, seed=6)
    slots = torch.arange(20, dtype=torch.int32).cuda()
    state, o = d["state"].clone(), torch.empty_like(d["v"])
    run = lambda: kda.linear_recurrent_step(d["q"], d["k"], d["v"], d["g"], state, slots=slots, out=o)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(3):
        fresh = _inputs(20, 4, 4, 64, 64, torch.bfloat16, False, 24, seed=7 + i)
        for x in ("q", "k", "v", "g"):
            d[x].copy_(fresh[x])
        before = state.clone()
        graph.replay()
        torch.cuda.synchronize()
        eager = before.clone()
        eo = kda.linear_recurrent_step(d["q"], d["k"], d["v"], d["g"], eager, slots=slots)
        assert torch.equal(o, eo) and torch.equal(state, eager)
