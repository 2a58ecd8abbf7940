"""GPU tests of token_logprobs against the definition in 64 bits.

Tolerances, from fp32 statistics over V values whose terms are e^(x-m) <= 1:
a term is off by a few units (the exponential, its rounded argument: for
x - m >= -104 at most 104 * 2^-24 relative) and fp32 partial sums of at most
2^7 terms each are joined in a tree, so log S is off by at most
(104 + 128 + 64) * 2^-24 < 2e-5 and in practice far less; x - m - log S rounds
twice more, at most 2^-24 * |value| each. Entropy carries the same relative
error in both of its terms.
"""
import math

import pytest
import torch

import bit_quantized_gemm_gb300 as qg

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


def reference(x, ids, top):
    """The definition in 64 bits, on the CPU."""
    x = x.double().cpu()
    ids = ids.cpu()
    m, v = x.shape
    bad = ~(x < INF).all(dim=1)
    empty = (x == -INF).all(dim=1)
    peak = torch.where(empty | bad, torch.zeros(m).double(), x.amax(dim=1))
    e = torch.exp(x - peak[:, None])
    log_s = torch.where(empty, torch.zeros(m).double(), torch.log(e.sum(dim=1)))
    lp = (x - peak[:, None]) - log_s[:, None]
    lp[bad] = math.nan
    entropy = -torch.where(lp > -INF, lp.exp() * lp, torch.zeros(()).double()).sum(dim=1)
    entropy[empty] = 0.0
    entropy[bad] = math.nan
    given = torch.gather(lp, 1, ids.clamp(0, v - 1))
    given[ids < 0] = 0.0
    given[ids >= v] = math.nan
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top]
    vals = torch.gather(lp, 1, order)
    order = torch.where((vals == -INF) | vals.isnan(), torch.full_like(order, -1), order)
    pad = top - order.shape[1]
    if pad > 0:
        fill = torch.where(bad, math.nan, -INF).double()[:, None].expand(m, pad)
        order = torch.cat([order, torch.full((m, pad), -1)], 1)
        vals = torch.cat([vals, fill], 1)
    return given, entropy, order, vals


def close(a, b, what):
    a = a.double().cpu()
    fine = b.isfinite()
    assert torch.equal(a.isnan(), b.isnan()), what
    assert torch.equal(a[~fine & ~b.isnan()], b[~fine & ~b.isnan()]), what
    assert bool(((a - b).abs()[fine] <= 2e-5 + 4 * 2.0 ** -24 * b.abs()[fine]).all()), what


def check(x, ids, top):
    given, entropy, order, vals = qg.token_logprobs(x, ids, top=top)
    two = ids if ids.dim() == 2 else ids[:, None]
    rg, re, ro, rv = reference(x, two, top)
    close(given.view(two.shape), rg, "given")
    close(entropy, re, "entropy")
    assert torch.equal(order.cpu(), ro), "top ids"
    close(vals, rv, "top")


def logits(seed, m, v, dtype, pad=0, scale=2.5):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(m, v + pad, generator=g, device=DEV) * scale
    x[:, :: max(1, v // 5)] += 9.0
    return x.to(dtype)[:, :v]


def some_ids(seed, m, v, count):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randint(0, v, (m, count), generator=g, device=DEV)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,v,count,top,pad", [
    (1, 1, 1, 0, 0), (1, 1, 1, 3, 0), (2, 7, 2, 7, 0), (3, 31, 1, 32, 0), (1, 1000, 0, 1, 0), (5, 4097, 3, 20, 1),
    (2, 32768, 1, 20, 0), (9, 50001, 4, 5, 61), (1, 131072, 1, 20, 0), (1, 262143, 2, 32, 0), (64, 20011, 1, 1, 128),
    (300, 8191, 1, 5, 0), (1025, 1536, 2, 32, 3), (200, 65537, 1, 2, 0),
])
def test_against_64_bits(m, v, count, top, pad, dtype):
    check(logits(m + v, m, v, dtype, pad), some_ids(v, m, v, count), top)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("v", [5, 1024, 30001, 140001])
def test_masks(v, dtype):
    # rows left with nothing, with one value, with fewer than `top`, NaN and +inf, the type's lowest value
    x = logits(v, 12, v, dtype)
    low = torch.finfo(dtype).min
    x[0] = -INF
    x[1] = -INF
    x[1, v // 2] = 3.0
    x[2] = -INF
    x[2, -3:] = torch.tensor([1.0, 2.0, 1.0], device=DEV).to(dtype)
    x[3, v - 1] = math.nan
    x[4, 0] = INF
    x[5] = low
    x[6, 1:] = low
    x[7, ::2] = -INF
    x[8] = -INF
    x[8, 0] = math.nan
    x[9, : v - 1] = -INF
    x[10] = torch.finfo(dtype).max
    ids = some_ids(1, 12, v, 3)
    ids[:, 1] = v // 2
    ids[11, 0], ids[11, 1], ids[11, 2] = -1, v, -(2 ** 40)
    ids[10, 2] = 2 ** 40
    ids[3, 0] = -1
    check(x, ids, 5)
    check(x, ids, 32)


@pytest.mark.parametrize("v", [33, 5000, 70000, 131072])
def test_ties_go_to_the_lowest_index(v):
    x = torch.zeros(8, v, device=DEV)
    x[1] = (torch.arange(v, device=DEV) % 3).float()
    x[2] = torch.arange(v, device=DEV).float() / v           # ascending
    x[3] = -x[2]                                             # descending
    x[4, v - 20:] = 1.0
    x[5] = (torch.arange(v, device=DEV) % 2).float() * -0.0  # both zeros are equal
    x[6, v // 3:v // 3 + 40] = 2.0
    x[7, 5:] = -INF
    for dtype in (torch.float32, torch.bfloat16):
        for top in (1, 5, 32):
            check(x.to(dtype), torch.zeros(8, 1, dtype=torch.int64, device=DEV), top)


def test_one_dimensional_ids_and_extreme_rows():
    x = logits(2, 6, 3000, torch.float32, scale=30.0)
    x[1] *= 1e30                       # a point mass
    x[2] *= 1e-30                      # uniform to rounding
    x[3] -= 3e38 / 4
    ids = some_ids(3, 6, 3000, 1)[:, 0]
    check(x, ids, 4)
    given = qg.token_logprobs(x, ids, top=4)[0]
    assert given.shape == (6,)


def test_rows_do_not_depend_on_their_batch_and_repeat():
    x = logits(4, 70, 40003, torch.bfloat16)
    ids = some_ids(5, 70, 40003, 2)
    first = qg.token_logprobs(x, ids, top=8)
    again = qg.token_logprobs(x, ids, top=8)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = qg.token_logprobs(x, ids, top=8, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, other))


def test_long_buffer():
    # rows further apart than 2^31 elements in all: offsets are 64-bit
    m, v, ld = 9, 1000, 1 << 28
    room = torch.empty(m * ld, dtype=torch.bfloat16, device=DEV)
    x = room.view(m, ld)[:, :v]
    x.copy_(logits(6, m, v, torch.bfloat16))
    check(x, some_ids(7, m, v, 2), 5)
    del x, room
    torch.cuda.empty_cache()


def test_refusals_of_the_binding():
    x = logits(1, 4, 100, torch.float32)
    ids = some_ids(1, 4, 100, 2)
    for call in [lambda: qg.token_logprobs(x.t(), ids), lambda: qg.token_logprobs(x.double(), ids),
                 lambda: qg.token_logprobs(x, ids[:3]), lambda: qg.token_logprobs(x, ids.int()),
                 lambda: qg.token_logprobs(x, ids.t())]:
        with pytest.raises(ValueError):
            call()
    for top in (-1, 33):
        with pytest.raises(qg.QGError):
            qg.token_logprobs(x, ids, top=top)
