"""GPU tests of the norm and of the gate into 8-bit activations, against 64 bits.

What a value y may be off by, relative to itself (half units of fp32, 2^-24):
  norm: the sum of squares is a chain of 16, a butterfly of 5, a chain of at most
  4 and a butterfly of 5: 30, halved by the root; the quotient by K (2 ulp, 4 half
  units) and + eps 1, halved; the refined reciprocal root 4 (1.5 times the square of
  the hardware's 2^-22.9 vanishes; the step's own roundings), two products 2.
  Together 24: below 2^-19.
  gate: (8 + |g|) * 2^-23, as the header states.
The scale adds its constant's rounding and a product (int8: a quotient), 2 * 2^-24.
A quantized value times its scale is then off from y by that, and by half a step:
2^-4 of the value or 2^-10 of the scale (e4m3), half the scale (int8).
"""
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


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def rows(g, m, k, dtype, pad=0, loud=1.0):
    x = torch.randn(m, k + pad, generator=g, device=DEV) * loud
    x *= torch.where(torch.rand(k + pad, generator=g, device=DEV) < 0.01, 20.0, 1.0)
    return x.to(dtype)[:, :k]


def exact_norm(h, w, eps):
    h = h.double()
    return h / torch.sqrt(h.square().mean(dim=1, keepdim=True) + eps) * w.double()


def blocks_of(y):
    m, k = y.shape
    kb = -(-k // 128)
    p = torch.zeros(m, kb * 128, dtype=y.dtype, device=y.device)
    p[:, :k] = y
    return p.view(m, kb, 128)


def check_e4m3(q, scale, y, off):
    """q, scale against y (64 bits); off: what |y| may be off by, relative."""
    m, k = y.shape
    top = blocks_of(y.abs()).amax(dim=2).t()
    off_top = blocks_of(off.expand_as(y)).amax(dim=2).t()
    want = top / 448
    assert bool(((scale.double() - want).abs() <= (off_top + 2.0 ** -23) * want).all())
    s = scale.double().t().repeat_interleave(128, 1)[:, :k]
    far = (q.double() * s - y).abs()
    assert bool((far <= torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * s) * (1 + 2.0 ** -10) + off * y.abs()).all())


def check_int8(q, scale, y, off):
    want = y.abs().amax(dim=1) / 127
    assert bool(((scale.double() - want).abs() <= (off + 2.0 ** -23) * want).all())
    far = (q.double() * scale.double()[:, None] - y).abs()
    assert bool((far <= (0.5 + 2.0 ** -10) * scale.double()[:, None] + off * y.abs()).all())


SIZES = [(1, 16), (3, 144), (1, 5120), (64, 2560), (7, 496), (130, 8192), (33, 8208), (2, 17408), (9, 17424),
         (1000, 272), (2, 65536), (3, 32784), (700, 1040), (5, 11200), (200, 11200), (3, 16384)]


@pytest.mark.parametrize("m,k", SIZES)
@pytest.mark.parametrize("dtype,wdtype,residual", [(BF16, BF16, True), (BF16, F32, False), (F32, BF16, True),
                                                   (F32, F32, False)])
def test_norm_e4m3(m, k, dtype, wdtype, residual):
    g = gen(m * 7 + k)
    x = rows(g, m, k, dtype, 16 * (m % 3))
    w = (1 + 0.2 * torch.randn(k, generator=g, device=DEV)).to(wdtype)
    res = rows(g, m, k, dtype, 16, 4.0) if residual else None
    q, scale, total = qg.rmsnorm_quantize_act_fp8(x, w, 1e-5, residual=res)
    h = x
    if residual:
        h = (x.float() + res.float()).to(dtype)
        assert torch.equal(total, h)
    else:
        assert total is None
    y = exact_norm(h, w, 1e-5)
    check_e4m3(q, scale, y, torch.tensor(2.0 ** -19, dtype=torch.float64, device=DEV))


@pytest.mark.parametrize("m,k", [(1, 32), (5, 160), (1, 17408), (64, 5120), (200, 2560), (33, 8224), (2, 65536),
                                 (900, 288)])
@pytest.mark.parametrize("dtype,residual", [(BF16, True), (F32, False), (F32, True)])
def test_norm_int8(m, k, dtype, residual):
    g = gen(m * 5 + k)
    x = rows(g, m, k, dtype, 16 * (m % 2))
    w = (1 + 0.2 * torch.randn(k, generator=g, device=DEV)).to(BF16)
    res = rows(g, m, k, dtype, 0, 4.0) if residual else None
    q, scale, bs, h16, total = qg.rmsnorm_quantize_act(x, w, residual=res, block_sums=True, q16=True)
    h = (x.float() + res.float()).to(dtype) if residual else x
    if residual:
        assert torch.equal(total, h)
    check_int8(q, scale, exact_norm(h, w, 1e-6), 2.0 ** -19)
    assert torch.equal(h16.to(torch.int32), q.to(torch.int32))
    assert torch.equal(bs, q.view(m, k // 32, 32).sum(dim=2, dtype=torch.int32))
    # the fp16 copy alone
    q2, s2, _, h2, _ = qg.rmsnorm_quantize_act(x, w, residual=res, q16=True, int8=False)
    assert q2 is None and torch.equal(h2, h16) and torch.equal(s2, scale)


def test_norm_of_exact_values_has_the_quantizers_bits():
    # rows of one magnitude 2^a, K a power of two, eps 0: every step of the norm is exact, so that y is
    # sign * weight and the quantizers' own bits have to come out
    g = gen(1)
    k = 2048
    sign = torch.where(torch.rand(12, k, generator=g, device=DEV) < 0.5, -1.0, 1.0)
    x = sign * torch.tensor([2.0 ** a for a in range(-6, 6)], device=DEV)[:, None]
    w = torch.randn(k, generator=g, device=DEV)
    for dtype in (BF16, F32):
        q, scale, _ = qg.rmsnorm_quantize_act_fp8(x.to(dtype), w, 0.0)
        want, ws = qg.quantize_act_fp8(sign * w)
        assert torch.equal(q.view(torch.uint8), want.view(torch.uint8)) and torch.equal(scale, ws)
        q, scale, bs, h, _ = qg.rmsnorm_quantize_act(x.to(dtype), w, 0.0, block_sums=True, q16=True)
        want, ws, wbs, wh = qg.quantize_act(sign * w, block_sums=True, q16=True)
        assert torch.equal(q, want) and torch.equal(scale, ws) and torch.equal(bs, wbs) and torch.equal(h, wh)


@pytest.mark.parametrize("k", [256, 5120, 11216, 16384, 17408])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_bits_of_a_row(k, dtype):
    # alone, in batches, on their stored sum, in place: the same bits (K of the int8 norm: a multiple of 32)
    k = k // 32 * 32
    g = gen(k)
    x, res = rows(g, 1700, k, dtype), rows(g, 1700, k, dtype, 0, 3.0)
    w = torch.randn(k, generator=g, device=DEV)
    q, scale, total = qg.rmsnorm_quantize_act_fp8(x, w, residual=res)
    q8, s8, _, _, _ = qg.rmsnorm_quantize_act(x, w, residual=res)
    for rows_ in (slice(5, 6), slice(1690, 1700), slice(100, 400)):
        a, b, c = qg.rmsnorm_quantize_act_fp8(x[rows_], w, residual=res[rows_])
        assert torch.equal(a.view(torch.uint8), q[rows_].view(torch.uint8))
        assert torch.equal(b, scale[:, rows_]) and torch.equal(c, total[rows_])
        a, b, _ = qg.rmsnorm_quantize_act_fp8(total[rows_], w)
        assert torch.equal(a.view(torch.uint8), q[rows_].view(torch.uint8)) and torch.equal(b, scale[:, rows_])
        a, b, _, _, _ = qg.rmsnorm_quantize_act(x[rows_], w, residual=res[rows_])
        assert torch.equal(a, q8[rows_]) and torch.equal(b, s8[rows_])
    kb, m = scale.shape
    room = torch.full((kb, m + 12), 7.0, device=DEV)
    mine, out_q = res.clone(), torch.empty_like(q)
    a, b, c = qg.rmsnorm_quantize_act_fp8(x, w, residual=mine, out=(out_q, room[:, :m], mine))
    assert c is mine and torch.equal(mine, total) and torch.equal(out_q.view(torch.uint8), q.view(torch.uint8))
    mine = x.clone()
    a, b, c = qg.rmsnorm_quantize_act(mine, w, residual=res, out=(q8.clone(), s8.clone(), None, None, mine))[:3]
    assert torch.equal(a, q8) and torch.equal(b, s8) and torch.equal(mine, total)
    assert torch.equal(room[:, :m], scale) and bool((room[:, m:] == 7.0).all())


def test_norm_of_zero_tiny_and_non_finite_rows():
    g = gen(3)
    x = rows(g, 8, 512, F32)
    x[0] = 0
    x[1] *= 1e-30       # below eps: y is about 1e-27
    x[2, 7] = float("nan")
    x[3, 300] = float("inf")
    x[4, 3] = float("-inf")
    w = torch.randn(512, generator=g, device=DEV)
    q, scale, _ = qg.rmsnorm_quantize_act_fp8(x, w)
    assert bool((scale[:, 0] == 0).all()) and bool((q[0].float() == 0).all())
    # NaN and infinities by the formula: r is NaN, or 0 with the infinity's own y NaN and the others 0
    assert bool(scale[:, 2].isnan().all())
    assert scale[:, 3].isnan().tolist() == [False, False, True, False] and bool((scale[[0, 1, 3], 3] == 0).all())
    assert scale[:, 4].isnan().tolist() == [True, False, False, False] and bool((scale[1:, 4] == 0).all())
    wt, wts = torch.ones(130, 512, device=DEV).to(torch.float8_e4m3fn), torch.ones(2, 4, device=DEV)
    assert bool(qg.gemm_fp8(q, scale, wt, wts)[2:5].isnan().all())
    ok = [1, 5, 6, 7]
    check_e4m3(q[ok], scale[:, ok], exact_norm(x[ok], w, 1e-6), torch.tensor(2.0 ** -19, dtype=torch.float64, device=DEV))
    q8, s8, bs, _, _ = qg.rmsnorm_quantize_act(x, w, block_sums=True)
    assert s8[0] == 0 and bool((q8[0] == 0).all()) and bool(s8[2:5].isnan().all())
    assert bool((q8[2:5] == 0).all()) and bool((bs[2:5] == 0).all())
    check_int8(q8[ok], s8[ok], exact_norm(x[ok], w, 1e-6), 2.0 ** -19)


def off_gate(gate):
    return (8 + gate.double().abs()) * 2.0 ** -23


@pytest.mark.parametrize("m,k,dtype,pad", [(1, 16, BF16, 0), (1, 9728, BF16, 0), (3, 144, F32, 16), (65, 528, BF16, 48),
                                           (7, 17408, F32, 0), (2000, 272, BF16, 0), (2, 65536, BF16, 0)])
def test_gate(m, k, dtype, pad):
    g = gen(m + k)
    x = (torch.randn(m, 2 * k + pad, generator=g, device=DEV) * 3).to(dtype)[:, :2 * k]
    q, scale = qg.silu_mul_quantize_act_fp8(x)
    gate, up = x[:, :k].double(), x[:, k:].double()
    check_e4m3(q, scale, gate * torch.sigmoid(gate) * up, off_gate(gate))
    a, b = qg.silu_mul_quantize_act_fp8(x[m // 2:m // 2 + 1])
    assert torch.equal(a.view(torch.uint8), q[m // 2:m // 2 + 1].view(torch.uint8))
    assert torch.equal(b, scale[:, m // 2:m // 2 + 1])


def test_gate_far_values():
    # gates from -87 (e^g at the edge of fp32) to 80, blocks alike so that small results have scales of their own
    gate = torch.cat([torch.full((128,), v) for v in (-87.0, -60.0, -20.0, -1e-3, 0.0, 1e-30, 30.0, 80.0)])
    up = torch.linspace(-3, 3, 1024)
    x = torch.cat([gate, up])[None].to(DEV)
    q, scale = qg.silu_mul_quantize_act_fp8(x)
    gd, ud = x[:, :1024].double(), x[:, 1024:].double()
    y = gd * torch.sigmoid(gd) * ud
    s = scale[:, 0].double()
    want = blocks_of(y.abs()).amax(dim=2)[0] / 448
    normal = want > 2.0 ** -126
    assert bool(((s - want).abs()[normal] <= (off_gate(gd).view(8, 128).amax(dim=1) + 2.0 ** -23)[normal] * want[normal]).all())
    assert s[4] == 0 and bool((q[0, 512:640].float() == 0).all())
    # infinities and NaN follow the formula: silu(inf) = inf, silu(-inf) and NaN are NaN
    x = torch.ones(4, 64, device=DEV)
    x[0, 3], x[1, 3], x[2, 3], x[3, 40] = float("inf"), float("-inf"), float("nan"), float("inf")
    _, scale = qg.silu_mul_quantize_act_fp8(x)
    assert scale[0, 0] == float("inf") and bool(scale[0, 1:3].isnan().all()) and scale[0, 3] == float("inf")
