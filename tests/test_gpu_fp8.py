"""GPU tests of the FP8 calls: quantize_act_fp8 bit for bit against the
definition, gemm_fp8 and linear_fp8 against 64-bit products within a bound
derived from the number of roundings.

Bound of a product: a block's fp32 tensor sum of at most 128 exact products is
off by at most one unit in the last place (2^-23 of the running magnitude,
which the sum of |terms| bounds) per addition; scaling it and adding it to the
chain rounds three times more (s * ws, the product inside the fmaf counted
once, the sum). So |err| <= (128 + 3 + KB) * 2^-23 * sum |terms|, and bf16
outputs add half a unit, 2^-8 * |y| (2^-9, doubled for the sum of both).
"""
import pytest
import torch

import bit_quantized_gemm_gb300 as qg

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BLOCK = 128


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_quantized_gemm_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    qg.check_device_error()


def blocks(k):
    return -(-k // BLOCK)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def activations(seed, m, k, dtype=torch.bfloat16, pad=0):
    g = gen(seed)
    x = torch.randn(m, k + pad, generator=g, device=DEV)
    x *= torch.where(torch.rand(k + pad, generator=g, device=DEV) < 0.01, 20.0, 1.0)
    return x.to(dtype)[:, :k]


def weights(seed, n, k, pad=0):
    g = gen(seed)
    w = (torch.randn(n, k + pad, generator=g, device=DEV) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    ws = torch.rand(blocks(n), blocks(k), generator=g, device=DEV) * 1e-3 + 1e-5
    return w[:, :k], ws


def reference_quantize(x):
    """The definition in fp32 on the CPU: the scale's product, IEEE division, then nearest-even e4m3."""
    inv = torch.tensor(1.0) / torch.tensor(448.0)
    x = x.float().cpu()
    m, k = x.shape
    q = torch.empty(m, k, dtype=torch.float8_e4m3fn)
    s = torch.empty(blocks(k), m)
    for b in range(blocks(k)):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        s[b] = part.abs().amax(dim=1) * inv
        y = torch.where(s[b][:, None] == 0, torch.zeros(()), part / s[b][:, None])
        q[:, b * BLOCK:(b + 1) * BLOCK] = y.clamp(-448, 448).to(torch.float8_e4m3fn)
    return q, s


def same_bits(a, b):
    """Equal as values, NaN equal to NaN (e4m3 and fp32)."""
    a, b = a.float().cpu(), b.float().cpu()
    return bool(((a == b) | (a.isnan() & b.isnan())).all()) and bool((a.signbit() == b.signbit())[~a.isnan()].all())


def check_product(out, q, scale, w, ws):
    m, k = q.shape
    n = w.shape[0]
    kb = blocks(k)
    a = q.double() * scale.double().t().repeat_interleave(BLOCK, 1)[:, :k]
    b = w.double() * ws.double().repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    y, mag = a @ b.t(), a.abs() @ b.abs().t()
    bound = (128 + 3 + kb) * 2.0 ** -23 * mag
    if out.dtype == torch.bfloat16:
        bound += 2.0 ** -8 * y.abs()
    assert out.shape == (m, n)
    assert bool(((out.double() - y).abs() <= bound).all())


# ------------------------------------------------------------------- quantizer
@pytest.mark.parametrize("m,k,dtype,pad", [
    (1, 16, torch.bfloat16, 0), (1, 5120, torch.bfloat16, 0), (3, 144, torch.float32, 0),
    (5, 496, torch.bfloat16, 16), (16, 17408, torch.bfloat16, 0), (257, 2576, torch.float32, 48),
    (1000, 640, torch.bfloat16, 80), (2, 65536, torch.float32, 0),
])
def test_quantize_bits(m, k, dtype, pad):
    x = activations(m + k, m, k, dtype, pad)
    x[m // 2, : min(k, 200)] = 0          # a zero block
    q, s = qg.quantize_act_fp8(x)
    rq, rs = reference_quantize(x)
    assert same_bits(s, rs) and same_bits(q, rq)


def test_quantize_ties_and_tiny_scales():
    # quotients on and beside every rounding boundary of e4m3 (absmax 448: s = 1), and blocks whose
    # scale is subnormal or underflows to zero
    grid = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mid = (grid[1:] + grid[:-1]) / 2
    up, down = torch.tensor(float("inf")), torch.tensor(float("-inf"))
    vals = torch.cat([mid, torch.nextafter(mid, up), torch.nextafter(mid, down), grid])
    vals = torch.cat([vals, -vals])
    rows = []
    for i in range(0, len(vals), 112):
        row = torch.zeros(128)
        part = vals[i:i + 112]
        row[:len(part)] = part
        row[127] = 448.0
        rows.append(row)
    x = torch.stack(rows)
    x = torch.cat([x, x * 3.0, x * 1e-3, x * 2.0 ** -130, x * 2.0 ** -140, x * 2.0 ** -149]).to(DEV)
    q, s = qg.quantize_act_fp8(x)
    rq, rs = reference_quantize(x)
    assert same_bits(s, rs) and same_bits(q, rq)


def test_quantize_non_finite():
    x = activations(3, 4, 512, torch.float32)
    x[0, 5] = float("nan")
    x[1, 130] = float("inf")
    x[2, 300] = float("-inf")
    q, s = qg.quantize_act_fp8(x)
    rq, rs = reference_quantize(x)
    assert same_bits(s, rs) and same_bits(q, rq)
    w, ws = weights(4, 40, 512)
    out = qg.gemm_fp8(q, s, w, ws)
    assert bool(out[:3].isnan().all()) and bool(out[3].isfinite().all())


# --------------------------------------------------------------------- product
SHAPES = [
    (1, 16, 1), (1, 128, 64), (2, 272, 129), (7, 1024, 100), (8, 5120, 1000), (16, 2576, 515),
    (17, 640, 257), (33, 1040, 384), (64, 2560, 640), (65, 384, 130), (100, 4096, 1000),
    (128, 1168, 333), (129, 512, 4096), (200, 656, 777), (256, 2560, 2560), (300, 1296, 1500),
    (777, 2576, 1003), (1024, 512, 5000), (2048, 768, 2560),
]


@pytest.mark.parametrize("m,k,n", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemm(m, k, n, dtype):
    q, s = qg.quantize_act_fp8(activations(m + n, m, k))
    w, ws = weights(k + n, n, k)
    out = qg.gemm_fp8(q, s, w, ws, out_dtype=dtype)
    check_product(out, q, s, w, ws)


@pytest.mark.parametrize("m,k,n", [(1, 17408, 5120), (64, 5120, 17408), (2048, 2560, 9728), (2048, 9728, 2560)])
def test_gemm_layer_sizes(m, k, n):
    q, s = qg.quantize_act_fp8(activations(m, m, k))
    w, ws = weights(n, n, k)
    check_product(qg.gemm_fp8(q, s, w, ws), q, s, w, ws)


@pytest.mark.parametrize("m,k,n", [(1, 16, 40000), (9, 400, 30001), (16, 2576, 25003), (32, 144, 48000), (64, 656, 20001)])
def test_gemm_more_tiles_than_sms(m, k, n):
    # few tokens and many weight rows: a CTA takes several tiles after one another
    x = activations(m, 200, k)
    w, ws = weights(n, n, k)
    q, s = qg.quantize_act_fp8(x)
    all_rows = qg.gemm_fp8(q, s, w, ws, out_dtype=torch.float32)
    out = qg.linear_fp8(x[:m], w, ws, out_dtype=torch.float32)
    q, s = qg.quantize_act_fp8(x[:m])
    check_product(out, q, s, w, ws)
    assert torch.equal(out, all_rows[:m])
    assert torch.equal(qg.gemm_fp8(q, s, w, ws, out_dtype=torch.float32), out)


@pytest.mark.parametrize("m", [1, 5, 64, 130, 600])
def test_gemm_strides(m):
    # weight rows inside a wider buffer, output rows inside a wider one whose rest stays as it was
    k, n = 640, 333
    q, s = qg.quantize_act_fp8(activations(m, m, k))
    w, ws = weights(n, n, k, pad=96)
    for dtype, ld in [(torch.bfloat16, 347), (torch.bfloat16, 344), (torch.float32, 335), (torch.float32, 336)]:
        room = torch.full((m, ld), 7.0, dtype=dtype, device=DEV)
        qg.gemm_fp8(q, s, w, ws, out=room[:, :n])
        check_product(room[:, :n], q, s, w, ws)
        assert bool((room[:, n:] == 7.0).all())
    # scales of a larger batch: rows further apart
    wide = torch.full((s.shape[0], m + 13 + (-(m + 13)) % 4), float("nan"), device=DEV)
    wide[:, :m] = s
    assert torch.equal(qg.gemm_fp8(q, wide[:, :m], w, ws), qg.gemm_fp8(q, s, w, ws))


def test_gemm_scales_by_block():
    # ones everywhere: each output is the exact sum over blocks of 128 * s * ws, powers of two
    m, k, n = 130, 400, 300
    q = torch.ones(m, k, device=DEV).to(torch.float8_e4m3fn)
    s = torch.ones(4, 132, device=DEV)[:, :m]
    s *= (2.0 ** (torch.arange(4, device=DEV) * 2))[:, None]
    s[:, 1::2] *= 4
    ws = torch.tensor([[1, 2, 4, 8], [16, 32, 64, 128], [256, 512, 1024, 2048]], device=DEV).float()
    w = torch.ones(n, k, device=DEV).to(torch.float8_e4m3fn)
    for rows in (1, 16, 130):
        out = qg.gemm_fp8(q[:rows], s[:, :rows] if rows == m else s[:, :rows].contiguous() if rows % 4 == 0
                          else torch.cat([s[:, :rows], s[:, :3]], 1)[:, :rows], w, ws, out_dtype=torch.float32)
        count = torch.tensor([128., 128., 128., 16.], device=DEV)
        y = (s[:, :rows].t() * count) @ ws.repeat_interleave(128, 0)[:n].t()
        assert torch.equal(out, y)


def test_gemm_rows_do_not_depend_on_their_batch():
    # the bits of a row are the same alone, in every batch size and at every place
    k, n, most = 2576, 1111, 700
    q, s = qg.quantize_act_fp8(activations(9, most, k))
    w, ws = weights(9, n, k)
    whole = qg.gemm_fp8(q, s, w, ws, out_dtype=torch.float32)
    for m0, m in [(0, 1), (5, 1), (8, 3), (4, 16), (100, 17), (40, 64), (12, 100), (256, 128), (300, 200), (64, 400)]:
        room = torch.zeros(s.shape[0], m + (-m) % 4, device=DEV)
        room[:, :m] = s[:, m0:m0 + m]
        part = qg.gemm_fp8(q[m0:m0 + m].contiguous(), room[:, :m], w, ws, out_dtype=torch.float32)
        assert torch.equal(part, whole[m0:m0 + m])


# ----------------------------------------------------------------------- layer
@pytest.mark.parametrize("m,k,n,dtype,pad", [
    (1, 5120, 640, torch.bfloat16, 0), (3, 144, 65, torch.float32, 16), (16, 2576, 1000, torch.bfloat16, 48),
    (64, 1024, 257, torch.float32, 0), (150, 656, 500, torch.bfloat16, 0), (513, 2560, 1280, torch.bfloat16, 16),
])
def test_linear_is_quantize_then_gemm(m, k, n, dtype, pad):
    x = activations(m, m, k, dtype, pad)
    w, ws = weights(n, n, k)
    q, s = qg.quantize_act_fp8(x)
    for out_dtype in (torch.bfloat16, torch.float32):
        two = qg.gemm_fp8(q, s, w, ws, out_dtype=out_dtype)
        for _ in range(3):
            assert torch.equal(qg.linear_fp8(x, w, ws, out_dtype=out_dtype), two)


def test_linear_on_another_stream_and_in_a_graph():
    m, k, n = 24, 1280, 900
    w, ws = weights(1, n, k)
    xs = [activations(i, m, k) for i in range(4)]
    want = [qg.linear_fp8(x, w, ws) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [qg.linear_fp8(x, w, ws, stream=side) for x in xs]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    static, out = xs[0].clone(), torch.empty_like(want[0])
    work = torch.empty(qg.linear_fp8_workspace_bytes(m, k), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qg.linear_fp8(static, w, ws, out=out, workspace=work)
    for x, y in zip(xs, want):
        static.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y)


def test_refusals_of_the_binding():
    x = activations(1, 4, 256)
    w, ws = weights(2, 130, 256)
    q, s = qg.quantize_act_fp8(x)
    bad = [
        lambda: qg.quantize_act_fp8(x.t()), lambda: qg.quantize_act_fp8(x.half()),
        lambda: qg.linear_fp8(x, w, ws[:1]), lambda: qg.linear_fp8(x, w[:, :128], ws),
        lambda: qg.linear_fp8(x, w.float(), ws), lambda: qg.gemm_fp8(q, s.t(), w, ws),
        lambda: qg.gemm_fp8(q, s[:1], w, ws), lambda: qg.gemm_fp8(q, s, w, ws, out=torch.empty(4, 129, device=DEV)),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(qg.QGError):
        qg.quantize_act_fp8(activations(1, 4, 200)[:, :200].contiguous())      # K % 16
    with pytest.raises(qg.QGError):
        qg.linear_fp8(x, w, ws, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
