"""GPU tests of token_logprobs on long rows against the definition in 64 bits.

Tolerances. A thread adds up to 16 terms of a chunk and the sums of up to 32
chunks; these are scaled at most 32 times to a higher maximum (the exponential
2^-22, the product 2^-24 each time, relative) before they go into a compensated
sum. A term e^d, d = x - m, is off by 2^-22 and by its rounded argument, 2 |d|
2^-24. The compensated sum, the scalings of it (each follows a rise of the maximum
by one or more, so that all of them weigh less than 1 / (1 - 1/e) of one) and the
tree of threads, warps and pieces add no more than 32 roundings. For |d| <= 24,
below which terms weigh nothing beside these, S and T are off by
    (16 + 32 + 32 * 5 + 4 + 48 + 32) 2^-24 < 2e-5
of their sums of magnitudes. So log S is off by 2e-5, x - m - log S by two more
roundings, and H = log S - T / S by 2e-5 (1 + 2 |T / S|).
"""
import math

import pytest
import torch

import bit_quantized_gemm_gb300 as qg
from bit_quantized_gemm_gb300 import _lib

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_quantized_gemm_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    qg.check_device_error()
    torch.cuda.empty_cache()


def near(got, want, tol, what):
    got = got.double()
    assert torch.equal(got.isnan(), want.isnan()), what
    sure = want.isfinite()
    assert torch.equal(got[~sure & ~want.isnan()], want[~sure & ~want.isnan()]), what
    assert bool(((got - want).abs() <= tol)[sure].all()), \
        "%s: off by %.3g" % (what, float(((got - want).abs() - tol)[sure].max()))


def check(x, ids, top, got=None, rows_at_once=32):
    """The definition in 64 bits, some rows at a time; `got`: the outputs to compare (computed when None)."""
    given, entropy, order, vals = got if got is not None else qg.token_logprobs(x, ids, top=top)
    for r in range(0, x.shape[0], rows_at_once):
        part, pid = x[r:r + rows_at_once].double(), ids[r:r + rows_at_once]
        m, v = part.shape
        bad = ~(part < INF).all(dim=1, keepdim=True)
        empty = (part == -INF).all(dim=1, keepdim=True)
        zero = torch.zeros((), dtype=torch.float64, device=DEV)
        peak = torch.where(bad | empty, zero, part.amax(dim=1, keepdim=True))
        d = part - peak
        e = torch.exp(d)
        total = torch.where(empty, zero + 1, e.sum(dim=1, keepdim=True))
        t_over_s = torch.where(e > 0, e * d, zero).sum(dim=1, keepdim=True) / total
        lp = torch.where(bad, zero + math.nan, d - total.log())
        want = torch.gather(lp, 1, pid.clamp(0, v - 1))
        want = torch.where(pid < 0, zero, torch.where(pid >= v, zero + math.nan, want))
        near(given[r:r + rows_at_once], want, 2e-5 + 2 * 2.0 ** -24 * want.abs(), "given")
        want = torch.where(bad, zero + math.nan, torch.where(empty, zero, total.log() - t_over_s))[:, 0]
        near(entropy[r:r + rows_at_once], want, 2e-5 * (1 + 2 * t_over_s[:, 0].abs()), "entropy")
        if top:
            best = torch.sort(part, dim=1, descending=True, stable=True).indices[:, :top]
            want = torch.gather(lp, 1, best)
            best = torch.where((want == -INF) | want.isnan(), -1, best)
            assert torch.equal(order[r:r + rows_at_once], best), "top ids"
            near(vals[r:r + rows_at_once], want, 2e-5 + 2 * 2.0 ** -24 * want.abs(), "top")


def some_ids(m, v, count):
    g = torch.Generator(device=DEV)
    g.manual_seed(m + v)
    return torch.randint(0, v, (m, count), generator=g, device=DEV)


# Peaks where a thread starts and a constant background below them: every step of its sum rounds
# the same way, which random logits never show. (Chains of 4096 such terms are off by 1e-4 and more.)
@pytest.mark.parametrize("below", [9.14, 11.0, 12.61])
@pytest.mark.parametrize("m,v,pieces,dtype", [
    (1, 1 << 24, 16, torch.float32), (1, 1 << 24, 16, torch.bfloat16),
    (512, 1 << 20, 1, torch.bfloat16), (512, 1 << 20, 1, torch.float32),
])
def test_peaks_above_a_constant_background(m, v, pieces, dtype, below):
    x = torch.full((m, v), -below, device=DEV).to(dtype)
    x.view(m, pieces, v // pieces)[:, :, :4096] = 0.0
    check(x, some_ids(m, v, 2), 0, rows_at_once=4)


# A maximum that rises in every chunk, by little and by much: the sums so far are scaled each time.
@pytest.mark.parametrize("rise", [1e-3, 0.3, 4.0, 40.0, 1e4])
@pytest.mark.parametrize("m,v", [(1, 1 << 24), (500, 262143)])
def test_rising_maximum(m, v, rise):
    x = (torch.arange(v, device=DEV, dtype=torch.float64) * (rise / v)).float()[None].repeat(m, 1)
    check(x, some_ids(m, v, 2), 0, rows_at_once=4)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("v,pitch", [(40003, 40003), (131072, 131072), (131072, 131077)])
def test_rows_in_other_batches_and_places(v, pitch, dtype):
    # a row alone, in small and large batches (16 pieces down to one) and at other addresses: the
    # alternatives are the same, the floats within twice the error of one call
    g = torch.Generator(device=DEV)
    g.manual_seed(v)
    most = 520
    x = torch.randn(most, pitch, generator=g, device=DEV).mul_(2.5).to(dtype)[:, :v]
    x[3, ::7] = x[3, 0]                     # ties
    x[4] = -INF
    x[4, v // 2] = 1.0
    ids = some_ids(most, v, 2)
    whole = qg.token_logprobs(x, ids, top=20)
    for r0, m in [(0, 1), (3, 1), (4, 2), (1, 7), (0, 16), (2, 40), (5, 62), (30, 100), (100, 200), (17, 500)]:
        part = qg.token_logprobs(x[r0:r0 + m], ids[r0:r0 + m].contiguous(), top=20)
        assert torch.equal(part[2], whole[2][r0:r0 + m])
        for a, b, t in [(part[0], whole[0], 0), (part[1], whole[1], 2), (part[3], whole[3], 0)]:
            b = b[r0:r0 + m].double()
            # (|T / S| is at most the entropy's own size: both of its terms are positive)
            near(a, b, 4e-5 * (1 + t * b.abs()) + 4 * 2.0 ** -24 * b.abs(), "batch of %d from %d" % (m, r0))
    moved = torch.empty(70 * pitch + 8, dtype=dtype, device=DEV)
    for shift in range(1, 8):
        place = moved[shift:shift + 70 * pitch].view(70, pitch)[:, :v]
        place.copy_(x[:70])
        part = qg.token_logprobs(place, ids[:70].contiguous(), top=20)
        assert torch.equal(part[2], whole[2][:70])
        for a, b, t in [(part[0], whole[0], 0), (part[1], whole[1], 2), (part[3], whole[3], 0)]:
            b = b[:70].double()
            near(a, b, 4e-5 * (1 + t * b.abs()) + 4 * 2.0 ** -24 * b.abs(), "at an address + %d" % shift)


# One CTA over a whole long row: 32 to 128 chunks, candidates that are ranked after up to 64 of them,
# more candidates than their buffer holds (ascending rows), and the values around the aligned part of a
# row, which come last but may have the lowest indices.
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("v,pitch", [(131072, 131072), (200003, 200003), (262143, 262151)])
def test_whole_rows(v, pitch, dtype):
    m = 512
    sms = torch.cuda.get_device_properties(DEV).multi_processor_count
    if sms == 152:
        assert _lib.logprobs_pieces(m, v, sms) == 1
    g = torch.Generator(device=DEV)
    g.manual_seed(pitch)
    x = torch.randn(m, pitch, generator=g, device=DEV).mul_(2.5)[:, :v]
    up = torch.arange(v, device=DEV).float() / v
    x[0:6] = up                                     # ascending, with runs of equal values in bf16
    x[6:12] = -up
    x[12:18] = 0.0                                  # all equal
    x[18:24] = (torch.arange(v, device=DEV) % 3).float()
    for r in range(24, 48):                         # the largest in the unaligned ends, ties among them
        x[r, :8] = 30.0
        x[r, v - 8:] = 30.0
        x[r, v // 2] = 30.0 + r % 2
    x[48:56, 1:] = 5.0                              # a first value that ties with all the rest, or not
    x[48:56, 0] = torch.tensor([5.0, 6.0, 4.0, 5.0, -INF, 5.0, 6.0, 5.0], device=DEV)
    x[56:64] = -INF                                 # nothing, one value, a few
    x[57, v - 1] = 2.0
    x[58, 0] = 2.0
    x[59, ::v // 20] = 1.0
    x[60, 5000:5040] = 3.0
    x[64:72, ::2] = -INF
    x[72, v // 3] = math.nan
    x[73, v - 1] = INF
    x[74:80, : v - 3000] = -INF                     # only the last chunks have any
    x[80:86] = up * up * 40.0                       # a maximum that rises to the end
    x[86:90] = torch.finfo(dtype).min
    x[87, 77] = 0.0
    x = x.to(dtype)
    if pitch != v:
        room = torch.zeros(m, pitch, dtype=dtype, device=DEV)
        room[:, :v] = x
        x = room[:, :v]
    ids = some_ids(m, v, 3)
    ids[::5, 1] = -1
    ids[::7, 2] = v
    for top in (0, 1, 5, 32):
        check(x, ids, top)
