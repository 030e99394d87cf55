"""GPU test of packed scans with very many empty sequences: their states pass through, and the sequences around them are computed as
without them."""
import pytest
import torch

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


@pytest.mark.parametrize("T,at,empty,C", [(12800, 100, 1 << 25, 128), (12800, 6464, 1 << 25, 100), (700, 700, (1 << 20) + 5, 7), (700, 0, 1 << 21, 130),
                                          (0, 0, (1 << 20) + 300, 33)])
def test_empty_sequences_between_two(T, at, empty, C):
    """Rows [0, at) are one sequence, [at, T) another, with `empty` in between (so the segments behind wait for none of that work)."""
    import gated_delta_rule_20_amd as kda
    gen = torch.Generator().manual_seed(T + at)
    rnd = lambda t, *s: torch.randn(s, generator=gen).to(t).cuda()  # noqa: E731
    x, g, d_h = rnd(BF, T, C), -torch.exp(rnd(BF, T, C) - 4), rnd(BF, T, C)
    cu = torch.full((empty + 3,), at, dtype=torch.int32, device="cuda")
    cu[0], cu[-1] = 0, T
    two = torch.tensor([0, at, T], dtype=torch.int32, device="cuda")
    h0 = torch.empty(empty + 2, C, device="cuda").normal_()
    ends = lambda t: t[[0, -1]].contiguous()  # noqa: E731
    h, hT = kda.gated_scan_fwd(x, g, cu_seqlens=cu, initial_state=h0)
    w, wT = kda.gated_scan_fwd(x, g, cu_seqlens=two, initial_state=ends(h0))
    assert torch.equal(h, w) and torch.equal(ends(hT), wT) and torch.equal(hT[1:-1], h0[1:-1])
    dx, dg, _, dh0 = kda.gated_scan_bwd(None, g, w, d_h, cu_seqlens=cu, initial_state=h0, dfinal_state=hT)
    want = kda.gated_scan_bwd(None, g, w, d_h, cu_seqlens=two, initial_state=ends(h0), dfinal_state=ends(hT))
    assert torch.equal(dx, want[0]) and torch.equal(dg, want[1]) and torch.equal(ends(dh0), want[3]) and torch.equal(dh0[1:-1], hT[1:-1])
    # without entering states, and in place
    hT = kda.gated_scan_fwd(x, g, cu_seqlens=cu, final_state=hT)[1]
    assert (hT[1:-1] == 0).all() and torch.equal(ends(hT), kda.gated_scan_fwd(x, g, cu_seqlens=two)[1])
    before = h0[1:-1].clone()
    kda.gated_scan_fwd(x, g, cu_seqlens=cu, initial_state=h0, final_state=h0)
    assert torch.equal(ends(h0), wT) and torch.equal(h0[1:-1], before)


def test_many_short_sequences():
    """More than 2^20 sequences of 0 to 2 tokens: as a loop over the tokens says (whole numbers: nothing is rounded)."""
    import gated_delta_rule_20_amd as kda
    N, C = (1 << 20) + 77, 5
    gen = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 3, (N,), generator=gen)
    cu = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)])
    T = int(cu[-1])
    x = torch.randint(-3, 4, (T, C), generator=gen).float()
    h0 = torch.randint(-3, 4, (N, C), generator=gen).float()
    seq = torch.repeat_interleave(torch.arange(N), lens)
    second = torch.arange(T) > cu[seq]
    want = h0[seq] + x
    want[second] += x[:-1][second[1:]]
    h, hT = kda.gated_scan_fwd(x.cuda(), torch.zeros(T, C, device="cuda"), cu_seqlens=cu.int().cuda(), initial_state=h0.cuda())
    last = h0.clone()
    last[lens > 0] = want[cu[1:][lens > 0] - 1]
    assert torch.equal(h.cpu(), want) and torch.equal(hT.cpu(), last)
    dx, dg, _, dh0 = kda.gated_scan_bwd(None, torch.zeros(T, C, device="cuda"), h, x.cuda(), cu_seqlens=cu.int().cuda(), initial_state=h0.cuda(),
                                        dfinal_state=h0.cuda())
    grad = h0[seq] + x
    first_of_two = torch.cat([second[1:], torch.zeros(1, dtype=torch.bool)])
    grad[first_of_two] += x[1:][first_of_two[:-1]]
    start = h0.clone()
    start[lens > 0] = grad[cu[:-1][lens > 0]]
    assert torch.equal(dx.cpu(), grad) and torch.equal(dh0.cpu(), start)
    prev = h0[seq]
    prev[second] = want[:-1][second[1:]]
    assert torch.equal(dg.cpu(), grad * prev)
