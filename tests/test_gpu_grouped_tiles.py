"""GPU tests of every tile of the product grouped by expert: the bits of gemm_fp8 with each expert's weights, and what
lies around the outputs."""
import pytest
import torch

import bit_quantized_gemm_gb300 as qg
from bit_quantized_gemm_gb300 import _lib
from test_gpu_grouped import BF16, DEV, F32, bits, by_expert, inputs, offsets_of
from test_grouped_plans import FIRST, TILES, counts_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_quantized_gemm_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    qg.check_device_error()


# 33 blocks of K with a last one of 16 values (more than a warp's 32 weight scales), 3 with one of 16; 32 whole ones
@pytest.mark.parametrize("k", [272, 4096, 4112])
@pytest.mark.parametrize("i", [0, 1])
@pytest.mark.parametrize("tile,m,experts,ns,several", TILES)
def test_every_tile(tile, m, experts, ns, several, i, k):
    n = ns[i]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert _lib.gemm_fp8_grouped_tile(m, n, experts, sms) == tile
    q, scale, w, ws = inputs(m + n + k, m, experts, k, n)
    off = offsets_of(counts_of(m, experts), FIRST)
    assert any(int(o) % 4 for o in off)     # (a row of scales starts on four rows)
    for dtype in (BF16, F32):
        room = torch.full((m + 2, n + 8), 7.0, device=DEV, dtype=dtype)
        want = by_expert(q, scale, off, w, ws, room.clone()[:m, :n])
        got = qg.gemm_fp8_grouped(q, scale, off, w, ws, out=room[:m, :n])
        assert torch.equal(bits(got.contiguous()), bits(want.contiguous()))
        assert bool((room[:, n:] == 7.0).all()) and bool((room[m:] == 7.0).all())
        assert bool((got[:FIRST] == 7.0).all()) and bool((got[int(off[-1]):] == 7.0).all())


@pytest.mark.parametrize("k", [272, 4112])
@pytest.mark.parametrize("tile,m,experts,ns,several", [t for t in TILES if t[4]])
def test_a_replayed_tile(tile, m, experts, ns, several, k):
    # captured once, replayed with other numbers of rows: all at one expert, none at all, the first again
    n = ns[1]
    q, scale, w, ws = inputs(m + n, m, experts, k, n)
    first = offsets_of(counts_of(m, experts), FIRST)
    off, out = first.clone(), torch.full((m, n), 7.0, device=DEV, dtype=BF16)
    qg.gemm_fp8_grouped(q, scale, off, w, ws, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qg.gemm_fp8_grouped(q, scale, off, w, ws, out=out)
    one = torch.full_like(first, m)
    one[:2] = 0
    for offsets in (one, torch.zeros_like(first), first):
        off.copy_(offsets)
        out.fill_(7.0)
        graph.replay()
        assert torch.equal(bits(out), bits(by_expert(q, scale, offsets, w, ws, torch.full_like(out, 7.0))))
