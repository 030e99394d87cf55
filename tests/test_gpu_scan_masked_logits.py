"""GPU tests of the gated scan where logits mask tokens: infinities and the types' largest values."""
import math

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


@pytest.mark.parametrize("value", [-math.inf, math.inf, "lowest", "highest", -1e30, -3e4, 1e30, -150.0, -90.0, -80.0])
@pytest.mark.parametrize("types", [(FP, FP), (BF, BF), (BF, FP)], ids=["fp32", "bf16", "bf16-fp32"])
@pytest.mark.parametrize("T", [50, 900])
def test_masked_tokens(T, types, value):
    """Logits far out shut or open the gate: such tokens keep (or decay) the state, have no gradient of their logit, and leave the sum
    of A_log's as it is without them (z Sigmoid'(z) goes to 0).  float64 stands in with logits where exp(A) z = +-40 at least: there
    Sigmoid' is below 5e-18, z times it below 1e-15, and the decays differ by 2e-17 from the limit's."""
    import gated_delta_rule_20_amd as kda
    dtype, g_dtype = types
    C = 37
    top = torch.finfo(g_dtype).max
    value = {"lowest": -top, "highest": top}.get(value, value)
    gen = torch.Generator().manual_seed(T)
    rnd = lambda t, *s: torch.randn(s, generator=gen).to(t).cuda()  # noqa: E731
    x, z, d_h, A = rnd(dtype, T, C), rnd(g_dtype, T, C) - 1, rnd(dtype, T, C), 0.3 * rnd(FP, C)
    h0, dhT = rnd(FP, 1, C), rnd(FP, 1, C)
    masked = (torch.rand(T, C, generator=gen) < 0.3).cuda()
    masked[T // 2:T // 2 + 10] = True
    z = torch.where(masked, torch.full_like(z, value), z)
    z64 = ref.f64(z).copy()
    z64[masked.cpu().numpy()] = math.copysign(max(40.0 * math.exp(3.0), 0.0), value) if abs(value) > 1e3 else float(z[masked][0])
    for complement in (False, True):
        kw = dict(A_log=A, complement=complement, initial_state=h0)
        h, hT = kda.gated_scan_fwd(x[None], z[None], **kw)
        want, wT, tol, tT = ref.scan(ref.f64(x), z64, ref.f64(A), -5.0, complement, [0, T], ref.f64(h0))
        ref.close(h[0], want, tol, dtype, "h")
        ref.close(hT, wT, tT, FP, "final state")
        dx, dg, dA, dh0 = kda.gated_scan_bwd(x[None], z[None], h, d_h[None], dfinal_state=dhT, **kw)
        want, tol = ref.scan_bwd(ref.f64(x), z64, ref.f64(h[0]), ref.f64(d_h), ref.f64(A), -5.0, complement, [0, T], ref.f64(h0), ref.f64(dhT))
        if abs(value) > 1e3:
            assert (dg[0][masked] == 0).all()
            want[1][masked.cpu().numpy()] = 0
        # Sigmoid' below float32's smallest normal number, 2^-126, may count as 0: dg = e (h - x) 5 e^A Sigmoid' with |e| and |h - x| at
        # most the sums of what goes into them, and z T times as much in dA
        sums = [np.abs(ref.f64(a)).sum(0) + np.abs(ref.f64(b)[0]) for a, b in ((d_h, dhT), (x, h0))]
        flushed = 2.0 ** -126 * 5 * np.exp(ref.f64(A)) * sums[0] * 2 * sums[1]
        tol = (tol[0], tol[1] + flushed, tol[2] + flushed * T * 803, tol[3])
        for name, a, b, t, ty in zip(("dx", "dg", "dA_log", "dinitial_state"), (dx[0], dg[0], dA, dh0), want, tol, (dtype, g_dtype, FP, FP)):
            ref.close(a, b, t, ty, f"{name} complement={complement}")
