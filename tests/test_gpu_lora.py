"""GPU tests of the low-rank adapters against 64 bits.

Bound: every addition of products in fp32 is off by at most one unit, 2^-23 of the sum
of |terms|, so a chain of c of them by c * 2^-23.
h, by tensor cores, bf16 rows: one of eight parts of K, in steps of 64, then 8 sums. Of
fp32: one of 64 shares of K, in steps of 32 with three products a value, then 16 sums.
A row at a time (few_rows): 64 products a lane at most (K in parts of 1024, K / 1024 of them), 5 sums
of lanes and K / 1024 of parts.
scaling * h: 2^-24, and by tensor cores 2^-17 for its two bf16 numbers (2^-24 for the three of
fp32 outputs). The second product: that often rank, up to 16, products. The sum with base rounds once to fp32 and once to the output: half a
step, 2^-8 (bf16) or 2^-24.
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


def inputs(seed, m, k, n, rank, count, x=BF16, out=BF16, pad=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    xs = torch.randn(m, k + pad, generator=g, device=DEV).to(x)[:, :k]
    base = torch.randn(m, n + pad, generator=g, device=DEV).to(out)[:, :n]
    a = (torch.randn(count, rank, k, generator=g, device=DEV) / k ** 0.5).to(BF16)
    b = torch.randn(count, n, rank, generator=g, device=DEV).to(BF16)
    scaling = 0.25 + torch.rand(count, generator=g, device=DEV)
    ids = torch.randint(-1, count, (m,), generator=g, device=DEV)
    return base, xs, a, b, ids, scaling


def few_rows(rank):
    """Rows up to which they are taken one at a time."""
    return 128 if rank <= 32 else 32 if rank <= 64 else 16


def check(got, base, x, a, b, ids, scaling):
    m, k, rank, count = x.shape[0], x.shape[1], a.shape[1], a.shape[0]
    if m <= few_rows(rank):
        c1 = 64 + 5 + -(-k // 1024)
    elif x.dtype == BF16:
        c1 = 64 * -(-(-(-k // 64)) // 8) + 8
    else:
        c1 = 3 * 32 * -(-(-(-k // 32)) // 64) + 16
    numbers = 2 if got.dtype == BF16 else 3
    c2 = numbers * 16 * -(-rank // 16)
    off = 2.0 ** -16.9 if numbers == 2 else 2.0 ** -23
    half = 2.0 ** -8 if got.dtype == BF16 else 2.0 ** -24
    assert got.shape == base.shape and got.dtype == base.dtype
    for i in range(-1, count):
        rows = (ids == i).nonzero()[:, 0]
        if not len(rows):
            continue
        if i < 0:
            assert torch.equal(got[rows], base[rows])
            continue
        f = 1.0 if scaling is None else float(scaling[i])
        xd, ad, bd = x[rows].double(), a[i].double(), b[i].double()
        h, hm = xd @ ad.t(), xd.abs() @ ad.abs().t()
        y = base[rows].double() + f * (h @ bd.t())
        bound = f * ((c1 * 2.0 ** -23 * hm + off * h.abs()) @ bd.abs().t())
        bound += c2 * 2.0 ** -23 * f * (h.abs() @ bd.abs().t())
        bound += (half + 2.0 ** -24) * (y.abs() + bound)
        assert bool(((got[rows].double() - y).abs() <= bound).all())


CASES = [
    (1, 16, 1, 8, 1), (1, 17408, 5120, 16, 3), (5, 272, 100, 16, 2), (16, 2560, 333, 8, 20), (31, 528, 256, 24, 4),
    (64, 5120, 1000, 16, 64), (33, 1040, 257, 32, 5), (100, 640, 129, 64, 3), (65, 2064, 520, 128, 9),
    (300, 256, 72, 40, 7), (700, 1280, 2000, 64, 2), (40, 65536, 64, 16, 3), (128, 2560, 2000, 32, 9),
    (32, 5120, 777, 64, 6), (33, 5120, 777, 64, 6), (16, 1296, 2048, 128, 4), (17, 1296, 2048, 128, 4), (3, 17408, 640, 72, 2),
]


@pytest.mark.parametrize("m,k,n,rank,count", CASES)
@pytest.mark.parametrize("x,out", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
def test_adapters(m, k, n, rank, count, x, out):
    base, xs, a, b, ids, scaling = inputs(m + k + n, m, k, n, rank, count, x, out)
    check(qg.add_lora(base, xs, a, b, ids, scaling), base, xs, a, b, ids, scaling)
    # runs of rows, and no scaling
    ids = ids.sort().values
    check(qg.add_lora(base, xs, a, b, ids), base, xs, a, b, ids, None)


@pytest.mark.parametrize("n", [64, 77, 200])
def test_strides_and_in_place(n):
    base, xs, a, b, ids, scaling = inputs(n, 90, 512, n, 16, 4, pad=16)
    want = qg.add_lora(base, xs, a, b, ids, scaling)
    check(want, base, xs, a, b, ids, scaling)
    room = torch.full((90, n + 24), 7.0, device=DEV, dtype=BF16)
    got = qg.add_lora(base, xs, a, b, ids, scaling, out=room[:, :n])
    assert torch.equal(got, want) and bool((room[:, n:] == 7.0).all())
    room[:, :n] = base
    got = qg.add_lora(room[:, :n], xs, a, b, ids, scaling, out=room[:, :n])
    assert torch.equal(got, want) and bool((room[:, n:] == 7.0).all())
    # rows that start off 16-byte boundaries
    odd = torch.full((90, n + 25), 7.0, device=DEV, dtype=BF16)
    got = qg.add_lora(base, xs, a, b, ids, scaling, out=odd[:, 3:3 + n])
    assert torch.equal(got, want) and bool((odd[:, :3] == 7.0).all()) and bool((odd[:, 3 + n:] == 7.0).all())


@pytest.mark.parametrize("x", [BF16, F32])
@pytest.mark.parametrize("rank,n", [(24, 304), (64, 304), (128, 2000)])
def test_bits_of_a_row_do_not_depend_on_the_others(x, rank, n):
    # (of calls of few rows, and of calls of more)
    few = few_rows(rank)
    base, xs, a, b, ids, scaling = inputs(1, 500, 1296, n, rank, 6, x)
    for many in (False, True):
        last = 500 if many else few
        want = qg.add_lora(base[:last], xs[:last], a, b, ids[:last], scaling)
        for rows in ((slice(3, 499), slice(100, 400), slice(9, 10 + few)) if many
                     else (slice(7, 8), slice(few // 4, few // 2), slice(1, few))):
            got = qg.add_lora(base[rows], xs[rows], a, b, ids[rows].contiguous(), scaling)
            assert torch.equal(got, want[rows])
        turn = torch.randperm(last, device=DEV)
        got = qg.add_lora(base[turn], xs[turn], a, b, ids[turn], scaling)
        assert torch.equal(got, want[turn])


@pytest.mark.parametrize("x,out,rank", [(BF16, BF16, 64), (BF16, F32, 128), (F32, BF16, 8), (BF16, BF16, 72)])
@pytest.mark.parametrize("m,n", [(129, 64), (200, 1000), (384, 5120), (1000, 328), (2049, 136), (130, 1), (257, 63),
                                 (999, 333), (300, 2051)])
def test_many_rows(m, n, x, out, rank):
    # runs of rows, some without an adapter; a tile of rows of one adapter, of several, of none
    base, xs, a, b, ids, scaling = inputs(m + n, m, 528, n, rank, 9, x, out)
    runs = torch.randint(-2, 9, (m // 60 + 1,), device=DEV).repeat_interleave(60)[:m].contiguous()
    for which in (runs, ids, torch.full_like(ids, 3), torch.full_like(ids, -1)):
        got = qg.add_lora(base, xs, a, b, which, scaling)
        check(got, base, xs, a, b, which.clamp(min=-1), scaling)
        mine = base.clone()
        assert qg.add_lora(mine, xs, a, b, which, scaling, out=mine) is mine
        assert torch.equal(mine, got)


@pytest.mark.parametrize("n", [200, 10000, 10001])
@pytest.mark.parametrize("count", [3, 4, 5, 9, 128])
@pytest.mark.parametrize("out,rank", [(BF16, 16), (F32, 72)])
def test_many_rows_of_many_adapters(n, count, out, rank):
    # more adapters in 128 rows than accumulators or slots, in several tiles of a CTA
    base, xs, a, b, _, scaling = inputs(8, 300, 272, n, rank, count, BF16, out)
    ids = torch.arange(300, device=DEV) * 37 % count
    check(qg.add_lora(base, xs, a, b, ids, scaling), base, xs, a, b, ids, scaling)
    runs = (torch.arange(300, device=DEV) // 23) % (count + 1) - 1
    check(qg.add_lora(base, xs, a, b, runs, scaling), base, xs, a, b, runs, scaling)


@pytest.mark.parametrize("rank", [16, 64, 128])
def test_a_workspace_of_many_rows_is_one_of_fewer(rank):
    base, xs, a, b, ids, scaling = inputs(9, 300, 2064, 520, rank, 5)
    ws = torch.full((qg.add_lora_workspace_bytes(300, 2064, rank),), 255, dtype=torch.uint8, device=DEV)
    for m in (300, 129, 128, 40, 17, 16, 1, 33, 200):
        got = qg.add_lora(base[:m], xs[:m], a, b, ids[:m].contiguous(), scaling, workspace=ws)
        assert torch.equal(got, qg.add_lora(base[:m], xs[:m], a, b, ids[:m].contiguous(), scaling))


def test_rows_without_an_adapter_keep_their_bits():
    base, xs, a, b, ids, scaling = inputs(4, 50, 256, 96, 8, 3)
    base.view(torch.int16)[:, 5] = 0x7FA3      # a NaN with a payload
    base.view(torch.int16)[:, 6] = -32768      # -0
    ids[:] = torch.tensor([-1, 3, 2 ** 40, -2 ** 40, 99] * 10, device=DEV)
    got = qg.add_lora(base, xs, a, b, ids, scaling)
    assert torch.equal(got.view(torch.int16), base.view(torch.int16))


def test_non_finite_values_stay_to_their_rows_and_adapters():
    base, xs, a, b, ids, scaling = inputs(5, 64, 256, 96, 8, 4, F32, F32)
    ids = torch.arange(64, device=DEV) % 5 - 1
    want = qg.add_lora(base, xs, a, b, ids, scaling)
    a[2, 3, 100], b[3, 40, 2] = float("nan"), float("inf")
    xs[6, 9] = float("inf")             # row 6 has adapter 0
    got = qg.add_lora(base, xs, a, b, ids, scaling)
    fine = (ids != 2) & (ids != 3)
    fine[6] = False
    assert torch.equal(got[fine], want[fine])
    assert bool(got[ids == 2].isnan().all())
    assert torch.equal(got[ids == 3][:, :40], want[ids == 3][:, :40])
    assert not bool(got[ids == 3][:, 40].isfinite().any()) and not bool(got[6].isfinite().any())
    # (an infinite h alone: h * b is infinite, not NaN)
    xs[6] = 0
    a[0] = 0
    a[0, 1, 0], xs[6, 0] = 1.0, float("inf")
    b[0, :, 1] = 1.0
    xs[6, 1:] = 0
    got = qg.add_lora(base, xs, a, b, ids, scaling)
    assert got[6].isnan().all() or got[6].isinf().all()
