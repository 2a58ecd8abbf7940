"""GPU tests of the adapters with many rows (tensor cores) where the other tests take few: strides,
what lies around the outputs, addresses off 16 bytes; and values at the end of their range on both paths."""
import pytest
import torch

import bit_quantized_gemm_gb300 as qg
from test_gpu_lora import BF16, DEV, F32, check, few_rows, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_quantized_gemm_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    qg.check_device_error()


TYPES = [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)]
INF = float("inf")


def around(m, n, dtype, left):
    """Outputs [m, n] inside a buffer of sevens, `left` columns in, with a few rows more."""
    es = 2 if dtype == BF16 else 4
    ld = (left + n + 16) * es // 16 * 16 // es + 16 // es * (left == 0)
    room = torch.full((m + 3, ld + (left > 0)), 7.0, device=DEV, dtype=dtype)
    return room, room[:m, left:left + n]


def untouched(room, m, n, left):
    return (bool((room[:m, :left] == 7.0).all()) and bool((room[:m, left + n:] == 7.0).all())
            and bool((room[m:] == 7.0).all()))


@pytest.mark.parametrize("x,out", TYPES)
@pytest.mark.parametrize("rank", [16, 64, 72])
@pytest.mark.parametrize("m,n", [(129, 64), (200, 200), (300, 77), (131, 1000), (257, 2056)])
def test_strides_in_place_and_what_lies_around(m, n, rank, x, out):
    base, xs, a, b, ids, scaling = inputs(m + n + rank, m, 512, n, rank, 4, x, out, pad=16)
    assert base.stride(0) == n + 16 and xs.stride(0) == 528
    want = qg.add_lora(base, xs, a, b, ids, scaling)
    check(want, base, xs, a, b, ids, scaling)
    # the same bits from contiguous inputs
    assert torch.equal(qg.add_lora(base.contiguous(), xs.contiguous(), a, b, ids, scaling), want)
    for left in (0, 3):     # rows on 16-byte boundaries (where N allows), and off them
        room, mine = around(m, n, out, left)
        got = qg.add_lora(base, xs, a, b, ids, scaling, out=mine)
        assert torch.equal(got, want) and untouched(room, m, n, left)
        mine.copy_(base)
        got = qg.add_lora(mine, xs, a, b, ids, scaling, out=mine)
        assert torch.equal(got, want) and untouched(room, m, n, left)
    # an aligned base, outputs off it, and the other way round
    _, odd = around(m, n, out, 1)
    odd.copy_(base)
    assert torch.equal(qg.add_lora(odd, xs, a, b, ids, scaling), want)


ROWS = [8, 130, 300]        # one at a time; by tensor cores


@pytest.mark.parametrize("x,out", TYPES)
@pytest.mark.parametrize("rank", [8, 24, 72])
@pytest.mark.parametrize("m", ROWS)
def test_non_finite_values_stay_to_their_rows_and_adapters(m, rank, x, out):
    base, xs, a, b, _, scaling = inputs(m + rank, m, 272, 96, rank, 4, x, out)
    ids = torch.arange(m, device=DEV) % 5 - 1
    want = qg.add_lora(base, xs, a, b, ids, scaling)
    assert bool(want.isfinite().all())
    # NaN in an adapter's A, in one column's B, in a row of x (row 1 has adapter 0)
    a[2, rank - 1, 100], b[3, 40, rank // 2], xs[1, 9] = float("nan"), float("nan"), float("nan")
    got = qg.add_lora(base, xs, a, b, ids, scaling)
    fine = (ids != 2) & (ids != 3)
    fine[1] = False
    assert torch.equal(got[fine], want[fine])
    assert bool(got[ids == 2].isnan().all()) and bool(got[1].isnan().all())
    rest = torch.arange(96, device=DEV) != 40
    assert torch.equal(got[ids == 3][:, rest], want[ids == 3][:, rest]) and bool(got[ids == 3][:, 40].isnan().all())


@pytest.mark.parametrize("x,out", TYPES)
@pytest.mark.parametrize("rank", [8, 24, 72])
@pytest.mark.parametrize("m", ROWS)
def test_an_infinite_activation(m, rank, x, out):
    # every rank's weight of its column is positive: h is +-inf, and every product with B has its sign
    base, xs, a, b, _, scaling = inputs(m + rank, m, 272, 96, rank, 4, x, out)
    ids = torch.arange(m, device=DEV) % 5 - 1
    a[0, :, 100] = a[0, :, 100].abs() + 0.125
    b[0] = b[0].abs() + 0.125
    want = qg.add_lora(base, xs, a, b, ids, scaling)
    xs[1, 100], xs[6, 100] = INF, -INF
    got = qg.add_lora(base, xs, a, b, ids, scaling)
    assert bool((got[1] == INF).all()) and bool((got[6] == -INF).all())
    fine = torch.ones(m, dtype=torch.bool, device=DEV)
    fine[1] = fine[6] = False
    assert torch.equal(got[fine], want[fine])


@pytest.mark.parametrize("x,out", TYPES)
@pytest.mark.parametrize("m", ROWS)
def test_values_at_the_end_of_their_range(m, x, out):
    # finite numbers that round to infinity as bf16 (above 2^128 - 2^119), as activations and as h: with weights that
    # bring them back the outputs are ordinary numbers
    rank, top = 16, torch.finfo(x).max
    base, xs, a, b, _, scaling = inputs(m, m, 272, 96, rank, 2, x, out)
    ids = torch.arange(m, device=DEV) % 3 - 1
    scaling.fill_(1.0)
    xs[:, 100] = top * torch.where(torch.arange(m, device=DEV) % 2 == 0, 1.0, -1.0)
    a[:, :, 100] = 2.0 ** -126
    check(qg.add_lora(base, xs, a, b, ids, scaling), base, xs, a, b, ids, scaling)
    xs.zero_()
    xs[:, 3] = 2.0 ** 64
    a.zero_()
    a[:, :, 3] = 2.0 ** 63
    scaling.fill_(2.0 - 2.0 ** -23)         # scaling * h: the largest fp32 number
    b.mul_(2.0 ** -100)
    check(qg.add_lora(base, xs, a, b, ids, scaling), base, xs, a, b, ids, scaling)


@pytest.mark.parametrize("x,out", TYPES)
@pytest.mark.parametrize("rank", [8, 24, 72])
@pytest.mark.parametrize("m", ROWS)
def test_an_infinite_weight_of_an_adapter(m, rank, x, out):
    # few rows: the sign of the sum's terms; many: not finite. Everything else keeps its bits
    base, xs, a, b, _, scaling = inputs(m + rank, m, 272, 96, rank, 4, x, out)
    ids = torch.arange(m, device=DEV) % 5 - 1
    xs[:, 100] = torch.where(torch.arange(m, device=DEV) % 2 == 0, 1.5, -1.5)
    b[2] = b[2].abs() + 0.125
    a[3, rank // 2] = 0
    a[3, rank // 2, 100] = 1.0
    want = qg.add_lora(base, xs, a, b, ids, scaling)
    a[2, :, 100] = INF              # adapter 2: h = +-inf
    b[3, 40, rank // 2] = -INF      # adapter 3: one column
    got = qg.add_lora(base, xs, a, b, ids, scaling)
    fine = (ids != 2) & (ids != 3)
    rest = torch.arange(96, device=DEV) != 40
    assert torch.equal(got[fine], want[fine]) and torch.equal(got[ids == 3][:, rest], want[ids == 3][:, rest])
    two, three = got[ids == 2], got[ids == 3][:, 40]
    if m <= few_rows(rank) or x == BF16:        # (one product for a bf16 activation)
        assert torch.equal(two, (xs[ids == 2][:, 100:101] * INF).to(out).expand_as(two))
    else:
        assert not bool(two.isfinite().any())
    if m <= few_rows(rank):
        assert torch.equal(three, (xs[ids == 3][:, 100] * -INF).to(out))
    else:
        assert not bool(three.isfinite().any())


@pytest.mark.parametrize("x,out,rank", [(BF16, BF16, 16), (F32, F32, 64), (BF16, F32, 72), (F32, BF16, 128)])
@pytest.mark.parametrize("m,n", [(130, 77), (700, 1000), (2100, 328)])
def test_captured_and_replayed_with_other_ids(m, n, x, out, rank):
    # two graphs of many rows that share a workspace, replayed in turn on other inputs and ids
    base, xs, a, b, ids, scaling = inputs(m, m, 528, n, rank, 9, x, out)
    ws = torch.full((qg.add_lora_workspace_bytes(m, 528, rank),), 255, dtype=torch.uint8, device=DEV)
    outs = [torch.empty_like(base) for _ in range(2)]
    qg.add_lora(base, xs, a, b, ids, scaling, out=outs[0], workspace=ws)
    torch.cuda.synchronize()
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qg.add_lora(base, xs, a, b, ids, scaling, out=o, workspace=ws)
        graphs.append(g)
    turn = torch.arange(m, device=DEV)
    for other in (turn % 9, torch.full_like(ids, -1), torch.full_like(ids, 8), turn // 100 % 11 - 1, turn * 37 % 40 - 3):
        ids.copy_(other)
        base.neg_()
        xs.mul_(-1.0)
        for g, o in zip(graphs, outs):
            o.fill_(7.0)
            g.replay()
        torch.cuda.synchronize()
        want = qg.add_lora(base, xs, a, b, ids, scaling)
        check(want, base, xs, a, b, torch.where(ids < 9, ids, -1).clamp(min=-1), scaling)
        assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("n", [96, 77])
def test_rows_without_an_adapter_keep_their_bits_among_others(n, out):
    # many rows, every second one without an adapter: NaN with payloads, -0, subnormal numbers of base stay
    base, xs, a, b, ids, scaling = inputs(n, 300, 256, n, 16, 3, BF16, out)
    word = torch.int16 if out == BF16 else torch.int32
    shift = 0 if out == BF16 else 16
    for col, v in ((5, 0x7FA3), (6, -0x8000), (7, 0x0001), (8, -0x7FFF)):
        base.view(word)[:, col] = v << shift
    ids[::2] = torch.tensor([-1, 3, 2 ** 40, -2 ** 40, 99] * 30, device=DEV)
    ids[1::2] = torch.arange(150, device=DEV) % 3
    for mine in (None, base.clone()):       # to other memory, and in place
        got = qg.add_lora(base if mine is None else mine, xs, a, b, ids, scaling, out=mine)
        assert torch.equal(got.view(word)[::2], base.view(word)[::2])
        assert bool(got[1::2, 5].isnan().all()) and bool(got[1::2, 9:].isfinite().all())
        assert not bool((got[1::2, 9:] == base[1::2, 9:]).all())
