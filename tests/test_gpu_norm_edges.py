"""GPU tests of the norm where its numbers come to an end: subnormal scales, and what its
quantized values are beside ties."""
import pytest
import torch

import bit_quantized_gemm_gb300 as qg

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_quantized_gemm_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    qg.check_device_error()


@pytest.mark.parametrize("top", [1, 60, 100, 127, 180, 190, 191, 317, 1000, 20000, 2 ** 22, 2 ** 23, 2 ** 30])
def test_int8_scales_of_a_few_subnormal_units(top):
    # Rows of 1 and -1 alone, K a power of two, eps 0: the norm is exact (1/sqrt(1) = 1), so that y is sign *
    # weight, here up to `top` units of 2^-149 (from 2^23 units on they are normal numbers). The quantizer has the same
    # definition but for its quotient, which is this call's, too, where the scale is subnormal. A scale that rounds
    # to 0 (up to 63 units) gives q = 0.
    k = 2048
    g = torch.Generator(device=DEV)
    g.manual_seed(top)
    sign = torch.where(torch.rand(5, k, generator=g, device=DEV) < 0.5, -1.0, 1.0)
    units = torch.randint(0, top + 1, (k,), generator=g, device=DEV)
    units[7] = top
    w = (units.double() * 2.0 ** -149).to(F32)
    assert torch.equal(w.double(), units.double() * 2.0 ** -149) or top > 2 ** 24
    q, scale, bs, h, _ = qg.rmsnorm_quantize_act(sign, w, 0.0, block_sums=True, q16=True)
    y = sign.double() * w.double()
    want_s = (y.abs().amax(dim=1).cpu() / 127).to(F32).to(DEV)      # (a double's quotient by 127 rounds as fp32's would)
    assert torch.equal(scale, want_s)
    assert torch.equal(h.to(torch.int32), q.to(torch.int32))
    assert torch.equal(bs, q.view(5, k // 32, 32).sum(dim=2, dtype=torch.int32))
    want, ws, wbs, wh = qg.quantize_act(sign * w, block_sums=True, q16=True)
    assert torch.equal(scale, ws)
    if float(scale[0]) == 0:
        assert top < 64 and not bool(q.any())
    elif float(scale[0]) < 2.0 ** -126:
        assert torch.equal(q, want) and torch.equal(h, wh) and torch.equal(bs, wbs)
    else:
        assert bool(((q.int() - want.int()).abs() <= 1).all())      # a product with fl(1/s): beside ties
    s = scale.double()[:, None]
    near = torch.where(s > 0, (y / torch.where(s > 0, s, torch.ones_like(s))).clamp(-127, 127), torch.zeros_like(y))
    assert bool(((q.double() - near).abs() <= 0.5 + 2.0 ** -15).all())
