"""GPU tests of activations in 8 bits (kda_act_pack / kda_act_unpack): codes and scales are the format's, bit for bit."""
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


def _check(x, p):
    codes, scales = ref.pack(x.float().cpu().numpy().reshape(-1, x.shape[-1]))
    assert np.array_equal(p.codes.cpu().numpy().reshape(codes.shape), codes)
    assert np.array_equal(p.scales.cpu().numpy().reshape(scales.shape), scales, equal_nan=True)


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (2, 128), (5, 129), (37, 1001), (4, 6, 64), (2, 3, 5, 128), (300, 4096), (1, 100000)])
def test_pack_and_unpack(shape, dtype):
    kda = _kda()
    gen = torch.Generator().manual_seed(len(shape) + shape[-1])
    x = (torch.randn(shape, generator=gen) * torch.exp2(20 * torch.rand(shape[-1], generator=gen) - 10)).to(dtype).cuda()
    p = kda.act_pack(x)
    _check(x, p)
    for out in (FP, BF):
        got = kda.act_unpack(p, dtype=out)
        want = torch.from_numpy(ref.values(p.codes, p.scales)).to(FP).to(out)   # exact product, rounded to fp32, then to out
        assert torch.equal(got.cpu(), want)
    # a value is off by half a code at most: amax / 254, and the roundings of scale and code (2 ulp)
    group = np.repeat(ref.f64(p.scales), 128, axis=-1)[..., :shape[-1]]
    assert np.all(np.abs(ref.values(*p) - ref.f64(x)) <= group * (0.5 + 127 * 4 * ref.U))


def test_special_values():
    """Zeros, groups too small for a scale, values at the border of rounding, infinities and NaN (their group only)."""
    kda = _kda()
    x = torch.randn(12, 300)
    x[0] = 0.0
    x[1, :128] = 1e-39
    x[2, 3], x[3, 130], x[4, 299] = float("nan"), float("inf"), float("-inf")
    x[5] = torch.arange(300) * 0.5                         # halves: ties go to the even code
    x[5, 127], x[5, 255], x[5, 299] = 127.0, 127.0, 127.0
    x[6] = 3.4e38 * torch.sign(x[6])
    x[7] = -0.0
    x[8, :128] = 2.0 ** -118
    x[9, :128] = 2.0 ** -119
    x = x.cuda()
    p = kda.act_pack(x)
    _check(x, p)
    v = kda.act_unpack(p, dtype=FP)
    assert torch.isnan(v[2, :128]).all() and torch.isfinite(v[2, 128:]).all()
    assert torch.isnan(v[3, 128:256]).all() and torch.isfinite(v[3, :128]).all() and torch.isnan(v[4, 256:]).all()
    assert (v[0] == 0).all() and (v[1, :128] == 0).all() and (v[9, :128] == 0).all() and (v[8, :128] != 0).all()


def test_strides_guards_streams_and_outputs():
    kda = _kda()
    wide = torch.randn(40, 300, device="cuda")
    part = wide[:, 11:11 + 141]
    p = kda.act_pack(part)
    _check(part.contiguous(), p)
    view = torch.randn(6, 10, 200, device="cuda").to(BF)[:, 2:7]
    with pytest.raises(ValueError, match="evenly"):
        kda.act_pack(view)
    codes = torch.full((40 * 141 + 64,), 9, dtype=torch.int8, device="cuda")
    scales = torch.full((80 + 64,), 9.0, device="cuda")
    out = kda.Packed(codes[32:-32].view(40, 141), scales[32:-32].view(40, 2))
    assert kda.act_pack(part, out=out) is out and torch.equal(out.codes, p.codes) and torch.equal(out.scales, p.scales)
    for t in (codes, scales):
        assert (t[:32] == 9).all() and (t[-32:] == 9).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q = kda.act_pack(part, stream=side)
    side.synchronize()
    assert torch.equal(q.codes, p.codes)
    res = torch.full((40 * 141 + 64,), 9.0, device="cuda")
    kda.act_unpack(p, out=res[32:-32].view(40, 141))
    assert (res[:32] == 9).all() and (res[-32:] == 9).all()
    e = kda.act_pack(torch.empty(0, 5, device="cuda"))
    assert e.codes.shape == (0, 5) and kda.act_unpack(e).shape == (0, 5)


def test_large_offsets():
    kda = _kda()
    R, D = 600000, 8192                                    # 4.9 GB of codes
    x = torch.zeros(R, D, dtype=BF, device="cuda")
    x[-3:] = torch.randn(3, D, device="cuda").to(BF)
    p = kda.act_pack(x)
    _check(x[-3:], kda.Packed(p.codes[-3:], p.scales[-3:]))
    v = kda.act_unpack(p)
    want = kda.act_unpack(kda.Packed(p.codes[-3:].contiguous(), p.scales[-3:].contiguous()))
    assert torch.equal(v[-3:], want) and (v[:10] == 0).all()
