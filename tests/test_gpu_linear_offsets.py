"""GPU test of linear attention with cu_seqlens that break their rules: results are wrong then, but nothing outside the outputs
and the workspace is written.  Every output and the workspace, which has exactly the size that is asked for, lie between two
guards."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

GUARD = 1 << 16      # bytes on either side
FILL = 0x5A


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_20_amd as kda
    kda.load_library()


class _Guarded:
    """Tensors cut out of larger buffers of one byte value."""

    def __init__(self):
        self.kept = []

    def __call__(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        buf = torch.full((2 * GUARD + n,), FILL, dtype=torch.uint8, device="cuda")
        self.kept.append((buf, n))
        return buf[GUARD:GUARD + n].view(dtype).view(shape)

    def check(self):
        for i, (buf, n) in enumerate(self.kept):
            assert bool((buf[:GUARD] == FILL).all()), i
            assert bool((buf[GUARD + n:] == FILL).all()), i


RULES_BROKEN = {
    "negative": [-5, 400, 100, 5000, 20], "repeated": [0, 900, 0, 900, 0], "backwards": [900, 900, 900, 0, 900],
    "limits": [2 ** 31 - 1, -2 ** 31, 7, 800, 900], "overlapping": [0, 900] * 60,
    "many": np.random.RandomState(3).randint(-100, 1100, 401).tolist(), "many overlapping": [0, 900] * 200,
}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,Hk,per_head", [(2, 1, False), (2, 2, True), (20, 20, False)])
@pytest.mark.parametrize("cu", RULES_BROKEN.values(), ids=RULES_BROKEN.keys())
def test_nothing_outside_is_written(cu, H, Hk, per_head, dtype):
    import gated_delta_rule_20_amd as kda
    T, D, N = 900, 64, len(cu) - 1
    gen = torch.Generator().manual_seed(12)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    q, k, v, do = (rnd(T, n, D).to(dtype).cuda() for n in (Hk, Hk, H, H))
    g = (-0.1 * torch.rand((H,) if per_head else (T, H), generator=gen)).cuda()
    h0, dhT = rnd(N, H, D, D).cuda(), rnd(N, H, D, D).cuda()
    offsets = torch.tensor(cu, dtype=torch.int32).cuda()
    new = _Guarded()
    bytes_of = lambda n: new((n,), torch.uint8)  # noqa: E731
    o, hT = new(v.shape, dtype), new(h0.shape, torch.float32)
    ck = new((N, 2, H, D, D), torch.float32)
    kda.linear_chunk_fwd(q, k, v, g, cu_seqlens=offsets, initial_state=h0, out=o, final_state=hT, checkpoints=ck, checkpoint_every=2,
                         workspace=bytes_of(kda.linear_chunk_fwd_workspace_size(q, v, cu_seqlens=offsets)))
    for need_dg in (True, False):
        n = kda.linear_chunk_bwd_workspace_size(q, v, cu_seqlens=offsets, g_per_head=per_head, need_dg=need_dg, dfinal_state=True)
        kda.linear_chunk_bwd(q, k, v, g, do, cu_seqlens=offsets, initial_state=h0, dfinal_state=dhT, need_dg=need_dg,
                             dq=new(q.shape, dtype), dk=new(k.shape, dtype), dv=new(v.shape, dtype),
                             dg=new(g.shape, torch.float32) if need_dg else None, dinitial_state=new(h0.shape, torch.float32),
                             workspace=bytes_of(n))
    torch.cuda.synchronize()
    new.check()
    # the same call with states updated in place
    a, b = new(h0.shape, torch.float32), new(h0.shape, torch.float32)
    a.copy_(h0)
    b.copy_(dhT)
    kda.linear_chunk_fwd(q, k, v, g, cu_seqlens=offsets, initial_state=a, out=o, final_state=a,
                         workspace=bytes_of(kda.linear_chunk_fwd_workspace_size(q, v, cu_seqlens=offsets)))
    kda.linear_chunk_bwd(q, k, v, g, do, cu_seqlens=offsets, initial_state=h0, dfinal_state=b, dinitial_state=b, dq=new(q.shape, dtype),
                         dk=new(k.shape, dtype), dv=new(v.shape, dtype), dg=new(g.shape, torch.float32),
                         workspace=bytes_of(kda.linear_chunk_bwd_workspace_size(q, v, cu_seqlens=offsets, g_per_head=per_head,
                                                                                dfinal_state=True)))
    torch.cuda.synchronize()
    new.check()
