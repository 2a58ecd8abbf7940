"""GPU tests of the product grouped by expert. A row has the bits of gemm_fp8 with its
expert's weights, so most cases compare bits; one compares with 64 bits on its own."""
import pytest
import torch

import bit_quantized_gemm_gb300 as qg

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_quantized_gemm_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    qg.check_device_error()


def inputs(seed, m, e, k, n, pad=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(m, k, generator=g, device=DEV).to(BF16)
    q, scale = qg.quantize_act_fp8(x)
    w = (torch.randn(e, n + pad, k + 16 * pad, generator=g, device=DEV) * 100).clamp(-448, 448).to(E4M3)[:, :n, :k]
    ws = torch.rand(e, -(-n // 128), -(-k // 128), generator=g, device=DEV) * 1e-3 + 1e-5
    return q, scale, w, ws


def offsets_of(counts, first=0):
    return torch.tensor([first] + counts, device=DEV).cumsum(0)


def by_expert(q, scale, offsets, w, ws, out):
    edges = offsets.tolist()
    for e in range(w.shape[0]):
        lo, hi = edges[e], edges[e + 1]
        if hi > lo:
            s = torch.empty(scale.shape[0], (hi - lo + 3) // 4 * 4, device=DEV)[:, :hi - lo].copy_(scale[:, lo:hi])
            out[lo:hi] = qg.gemm_fp8(q[lo:hi].contiguous(), s, w[e], ws[e], out_dtype=out.dtype)
    return out


def bits(t):
    return t.view(torch.int16 if t.dtype == BF16 else torch.int32)


COUNTS = [
    ([1], 16, 1), ([3], 272, 64), ([0, 1, 0], 128, 100), ([2, 0, 5, 1], 640, 129), ([1] * 8, 2560, 2432),
    ([0] * 63 + [9], 384, 257), ([17, 15, 33, 1], 1040, 300), ([64, 65, 3, 0, 130], 1216, 333),
    ([127, 129, 128, 1], 656, 1003), ([300, 0, 513], 512, 640), ([5, 700, 2, 31, 90, 0], 1296, 515),
    ([1000], 2576, 777), ([2048, 4], 256, 2560), ([7] * 100, 400, 200), ([0, 0], 128, 64),
]


@pytest.mark.parametrize("counts,k,n", COUNTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_grouped_has_the_bits_of_each_product(counts, k, n, dtype):
    m = max(sum(counts), 1)
    q, scale, w, ws = inputs(m + k + n, m, len(counts), k, n)
    off = offsets_of(counts)
    out = torch.full((m, n), 7.0, device=DEV, dtype=dtype)
    want = by_expert(q, scale, off, w, ws, out.clone())
    got = qg.gemm_fp8_grouped(q, scale, off, w, ws, out=out)
    assert got is out and torch.equal(bits(out), bits(want))


@pytest.mark.parametrize("m,counts,first", [(50, [3, 0, 9], 4), (400, [130, 100, 9], 61), (33, [0, 0, 0], 0)])
def test_rows_of_no_expert_are_left(m, counts, first):
    q, scale, w, ws = inputs(m, m, len(counts), 512, 260, pad=3)
    off = offsets_of(counts, first)
    room = torch.full((m, 300), 7.0, device=DEV, dtype=BF16)
    want = by_expert(q, scale, off, w, ws, room.clone()[:, :260])
    qg.gemm_fp8_grouped(q, scale, off, w, ws, out=room[:, :260])
    assert torch.equal(bits(room[:, :260].contiguous()), bits(want.contiguous()))
    assert bool((room[:, 260:] == 7.0).all())


@pytest.mark.parametrize("off", [[-5, 3, 900], [0, 40, 20], [10, 5, 60], [100, 200, 300], [2 ** 40, 2 ** 41, -1]])
def test_offsets_outside_the_rows(off):
    # out-of-range offsets are clamped, an expert that ends before it begins has no rows
    m = 60
    q, scale, w, ws = inputs(m, m, 2, 384, 200)
    offsets = torch.tensor(off, device=DEV)
    out = torch.full((m, 200), 7.0, device=DEV, dtype=F32)
    want = by_expert(q, scale, offsets.clamp(0, m), w, ws, out.clone())
    qg.gemm_fp8_grouped(q, scale, offsets, w, ws, out=out)
    assert torch.equal(bits(out), bits(want))


def test_many_experts_and_a_wide_one():
    m, e = 1500, 1024
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    q, scale, w, ws = inputs(5, m, e, 256, 96)
    counts = torch.bincount(torch.randint(0, e, (m - 600,), generator=g, device=DEV), minlength=e)
    counts[700] += 600
    off = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    out = torch.empty(m, 96, device=DEV, dtype=BF16)
    want = by_expert(q, scale, off, w, ws, torch.empty_like(out))
    qg.gemm_fp8_grouped(q, scale, off, w, ws, out=out)
    assert torch.equal(bits(out), bits(want))


@pytest.mark.parametrize("e", [31, 32, 33, 127, 128, 129, 256])
@pytest.mark.parametrize("rows", [3, 40])
def test_numbers_of_experts(e, rows):
    # (their offsets are read in groups)
    counts = [(i * 7) % (2 * rows) for i in range(e)]
    m = sum(counts)
    q, scale, w, ws = inputs(e, m, e, 144, 72)
    off = offsets_of(counts)
    out = torch.empty(m, 72, device=DEV, dtype=F32)
    want = by_expert(q, scale, off, w, ws, torch.empty_like(out))
    qg.gemm_fp8_grouped(q, scale, off, w, ws, out=out)
    assert torch.equal(bits(out), bits(want))


def test_against_64_bits():
    # the bound of gemm_fp8's own tests: (128 + 3 + KB) * 2^-23 of the sum of magnitudes
    counts, k, n = [40, 3, 200], 1296, 390
    q, scale, w, ws = inputs(2, 243, 3, k, n)
    out = qg.gemm_fp8_grouped(q, scale, offsets_of(counts), w, ws, out_dtype=F32)
    kb, lo = -(-k // 128), 0
    for e, c in enumerate(counts):
        a = q[lo:lo + c].double() * scale[:, lo:lo + c].double().t().repeat_interleave(128, 1)[:, :k]
        b = w[e].double() * ws[e].double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
        bound = (128 + 3 + kb) * 2.0 ** -23 * (a.abs() @ b.abs().t())
        assert bool(((out[lo:lo + c].double() - a @ b.t()).abs() <= bound).all())
        lo += c


def test_non_finite_rows_stay_to_themselves():
    q, scale, w, ws = inputs(3, 40, 2, 512, 130)
    want = qg.gemm_fp8_grouped(q, scale, offsets_of([18, 22]), w, ws, out_dtype=F32)
    scale[2, 17] = float("nan")
    scale[0, 30] = float("inf")
    out = qg.gemm_fp8_grouped(q, scale, offsets_of([18, 22]), w, ws, out_dtype=F32)
    keep = [i for i in range(40) if i not in (17, 30)]
    assert torch.equal(out[keep], want[keep])
    assert bool(out[17].isnan().all()) and not bool(out[30].isfinite().any())
