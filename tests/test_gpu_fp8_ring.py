"""GPU tests of the FP8 kernels' rings over many rounds: the token scales of a
block come through the ring with its operands and are read by other warps than
the ones that ask for the next round's, so a slot that is rewritten too early
shows as another block's scale.

Every value is exact, so that nothing but the right scale passes: operands are
whole numbers of at most 2, scales powers of two (a token's from 1 to 8, another
one from block to block; a weight block's 1 or 2), so that a block's sum is at
most 512, an output at most 512 * 16 * 512 < 2^24 and every step of the chain is
a whole number in fp32.
"""
import pytest
import torch

import bit_quantized_gemm_gb300 as qg
from bit_quantized_gemm_gb300 import _lib

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_quantized_gemm_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    qg.check_device_error()


def exact_case(m, k, n):
    g = torch.Generator(device=DEV)
    g.manual_seed(m + k + n)
    kb, nb = -(-k // 128), -(-n // 128)
    q = torch.randint(-2, 3, (m, k), generator=g, device=DEV).float()
    w = torch.randint(-2, 3, (n, k), generator=g, device=DEV).float()
    room = torch.zeros(kb, -(-m // 4) * 4, device=DEV)
    s = room[:, :m]
    s.copy_(2.0 ** torch.randint(0, 4, (kb, m), generator=g, device=DEV))
    ws = 2.0 ** torch.randint(0, 2, (nb, kb), generator=g, device=DEV)
    a = q.double() * s.double().t().repeat_interleave(128, 1)[:, :k]
    b = w.double() * ws.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return q.to(torch.float8_e4m3fn), s, w.to(torch.float8_e4m3fn), ws, (a @ b.t()).float()


@pytest.mark.parametrize("m,k,n", [
    # up to 64 tokens: tiles of 64 weight rows, of 128, and several tiles a CTA
    (1, 17408, 5120), (16, 17408, 5120), (24, 17408, 5120), (64, 17408, 5120),
    (3, 5120, 17408), (16, 5120, 17408), (32, 5120, 17408), (64, 5120, 17408), (7, 2576, 40001),
    # more: single CTAs and pairs, short tails of K, several tiles a CTA
    (65, 17408, 5120), (128, 17408, 5120), (512, 17408, 5120), (777, 2576, 5003), (1024, 9744, 2560),
    (2048, 2560, 9728), (4096, 4240, 4864),
    # the longest chains: products of scales pass through two to four buffers 512 times
    (200, 65536, 1500), (2000, 65536, 2500), (600, 65424, 5000),
])
def test_scales_of_many_rounds(m, k, n):
    q, s, w, ws, want = exact_case(m, k, n)
    out = [qg.gemm_fp8(q, s, w, ws, out_dtype=torch.float32) for _ in range(5)]
    for y in out:
        assert torch.equal(y, want)


@pytest.mark.parametrize("m,k,n", [(1, 17408, 5120), (64, 17408, 5120), (64, 5120, 17408), (128, 17408, 5120),
                                   (2048, 2560, 9728)])
def test_layer_calls_in_a_row(m, k, n):
    # one workspace, rewritten by each call's quantizer: every call gives the bits of the two separate ones
    g = torch.Generator(device=DEV)
    g.manual_seed(m)
    x = (torch.randn(m, k, generator=g, device=DEV) * 3).to(torch.bfloat16)
    w = (torch.randn(n, k, generator=g, device=DEV) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    ws = torch.rand(-(-n // 128), -(-k // 128), generator=g, device=DEV) * 1e-3 + 1e-5
    work = torch.empty(qg.linear_fp8_workspace_bytes(m, k), dtype=torch.uint8, device=DEV)
    q, s = qg.quantize_act_fp8(x)
    two = qg.gemm_fp8(q, s, w, ws)
    out = [qg.linear_fp8(x, w, ws, workspace=work) for _ in range(5)]
    for y in out:
        assert torch.equal(y, two)


# Every tile of the kernel above 64 tokens, with more tiles than CTAs (or pairs) at once: rows that
# leave by TMA and by element stores, an odd last block of K, more than 32 blocks (the weight scales of
# the next 32 follow), more than 2048 tokens (a second group of the tile order), a short last token tile.
@pytest.mark.parametrize("m,k,n,tile", [
    (25600, 272, 64, (128, 64)), (20001, 656, 40, (128, 64)), (4890, 4208, 398, (128, 64)),
    (777, 2576, 5003, (128, 128)), (300, 4208, 17408, (128, 128)), (5390, 4240, 775, (128, 128)),
    (5390, 400, 776, (128, 128)),
    (700, 656, 9000, (256, 128)), (4970, 4208, 778, (256, 128)), (4970, 272, 776, (256, 128)),
    (2048, 4208, 9728, (256, 256)), (5783, 4240, 1164, (256, 256)), (5783, 400, 1163, (256, 256)),
])
def test_every_tile(m, k, n, tile):
    sms = torch.cuda.get_device_properties(DEV).multi_processor_count
    if sms == 152:
        assert _lib.gemm_fp8_tile(m, n, sms) == tile
    q, s, w, ws, want = exact_case(m, k, n)
    for dtype in (torch.float32, torch.bfloat16):
        for _ in range(2):
            assert torch.equal(qg.gemm_fp8(q, s, w, ws, out_dtype=dtype), want.to(dtype))
