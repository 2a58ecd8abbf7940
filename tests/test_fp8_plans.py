"""What the FP8 GEMM's tiles and the pieces of token_logprobs are chosen to be: the rules
that the GPU tests rely on to reach every variant (host only)."""
import pytest

import bit_quantized_gemm_gb300 as qg
from bit_quantized_gemm_gb300 import _lib
from bit_quantized_gemm_gb300 import build as qbuild


@pytest.fixture(scope="module", autouse=True)
def _built():
    qbuild.build()


@pytest.mark.parametrize("sms", [1, 2, 3, 76, 132, 152])
def test_tiles_follow_the_tokens(sms):
    for m in (1, 16, 17, 32, 33, 64, 65, 128, 129, 1000, 8192, 1 << 24):
        for n in (1, 64, 65, 128, 5120, 9728, 17408, 131072, 1 << 24):
            tokens, rows = _lib.gemm_fp8_tile(m, n, sms)
            if m <= 64:
                assert tokens == (16 if m <= 16 else 32 if m <= 32 else 64) and rows in (64, 128)
                assert (rows == 64) == (-(-n // 64) <= sms)
            else:
                assert (tokens, rows) in ((128, 64), (128, 128), (256, 128), (256, 256))
                assert tokens == 128 or sms > 1


def test_pieces():
    for v in (1, 100, 4096, 4097, 32768, 131072, 1 << 24):
        last = 16
        for m in (1, 2, 16, 37, 38, 61, 62, 200, 493, 494, 4096, 1 << 24):
            pieces = _lib.logprobs_pieces(m, v, 152)
            assert pieces in (1, 2, 4, 8, 16) and pieces <= last
            assert pieces == 1 or v > 4096 * (pieces // 2)
            last = pieces
    # 16 pieces were slower than 8 from about 42 rows on (61 rows of 131072: 16.4 and 14.4 us)
    assert [_lib.logprobs_pieces(m, 131072, 152) for m in (1, 31, 37, 42, 61, 64)] == [16, 16, 16, 8, 8, 8]
    assert _lib.logprobs_pieces(494, 1 << 24, 152) == 1


def test_refusals():
    for call in (lambda: _lib.gemm_fp8_tile(0, 1, 152), lambda: _lib.gemm_fp8_tile(1, (1 << 24) + 1, 152),
                 lambda: _lib.gemm_fp8_tile(1, 1, 0), lambda: _lib.logprobs_pieces(1, 0, 152),
                 lambda: _lib.logprobs_pieces(1, 1, 5000)):
        with pytest.raises(qg.QGError):
            call()
