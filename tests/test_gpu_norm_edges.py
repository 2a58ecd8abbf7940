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


@pytest.mark.parametrize("m,k,dtype,wdtype", [(70, 5120, BF16, BF16), (9, 17408, BF16, F32), (64, 2560, F32, BF16),
                                              (3, 32784, F32, F32)])
def test_e4m3_is_the_nearest_value_but_beside_ties(m, k, dtype, wdtype):
    # The root is a factor of every y of a row and of its scale: what is off in y / s is two roundings of y, two of
    # the largest y, the constant's and the product's of s, fl(1/s) and its product, 8 * 2^-24. (Exact ties are common
    # with bf16 rows and weights, whose products have few bits: which way one goes is not said.)
    g = torch.Generator(device=DEV)
    g.manual_seed(m + k)
    x = torch.randn(m, k, generator=g, device=DEV).to(dtype)
    w = (1 + 0.2 * torch.randn(k, generator=g, device=DEV)).to(wdtype)
    q, _, _ = qg.rmsnorm_quantize_act_fp8(x, w)
    t = x.double().cpu() * w.double().cpu()
    kb = -(-k // 128)
    p = torch.zeros(m, kb * 128, dtype=torch.float64)
    p[:, :k] = t
    top = p.view(m, kb, 128).abs().amax(dim=2).repeat_interleave(128, 1)[:, :k]
    v = 448 * t / top
    values = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()     # 0 up to 448
    middles = (values[1:] + values[:-1]) / 2
    near = values[torch.bucketize(v.abs(), middles)] * v.sign()
    tie = torch.zeros_like(v, dtype=torch.bool)
    for i in (0, 1):        # the middle below and the one above
        at = middles[(torch.bucketize(v.abs(), middles) - 1 + i).clamp(0, len(middles) - 1)]
        tie |= (v.abs() - at).abs() <= 2.0 ** -21 * at
    far = q.float().double().cpu() != near
    assert not bool((far & ~tie).any())
    assert int(far.sum()) <= int(tie.sum())


def test_sums_of_squares_beyond_fp32():
    # (their sum is fp32: 1 / sqrt is 0 or, with eps 0, infinite; the rows beside keep their bits)
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    x = torch.randn(6, 640, generator=g, device=DEV)
    w = 1 + 0.2 * torch.randn(640, generator=g, device=DEV)
    want, ws, _ = qg.rmsnorm_quantize_act_fp8(x, w, 0.0)
    want8, ws8 = qg.rmsnorm_quantize_act(x, w, 0.0)[:2]
    x[1] *= 2.0 ** 70
    x[4] *= 2.0 ** -90
    q, s, _ = qg.rmsnorm_quantize_act_fp8(x, w, 0.0)
    q8, s8 = qg.rmsnorm_quantize_act(x, w, 0.0)[:2]
    rest = [0, 2, 3, 5]
    assert torch.equal(q[rest].view(torch.uint8), want[rest].view(torch.uint8)) and torch.equal(s[:, rest], ws[:, rest])
    assert torch.equal(q8[rest], want8[rest]) and torch.equal(s8[rest], ws8[rest])
    assert bool((s[:, 1] == 0).all()) and not bool(q[1].float().any()) and s8[1] == 0 and not bool(q8[1].any())
    assert not bool(s[:, 4].isfinite().any()) and not bool(s8[4].isfinite())
