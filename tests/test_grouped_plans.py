"""What the tile of the product grouped by expert is chosen to be: the rule that the GPU tests rely on to
reach every variant (host only)."""
import random

import pytest

import bit_quantized_gemm_gb300 as qg
from bit_quantized_gemm_gb300 import _lib
from bit_quantized_gemm_gb300 import build as qbuild

# tile (rows x weight rows), rows, experts, N of odd length and of 16-byte rows, whether a CTA (or pair) gets several tiles
TILES = [
    ((16, 64), 100, 5, (515, 520), False),      # (as many tiles as SMs at most, by the rule)
    ((16, 128), 400, 32, (515, 520), True),
    ((32, 128), 1000, 32, (257, 264), True),
    ((128, 64), 12001, 5, (129, 136), True),
    ((128, 128), 12001, 8, (257, 264), True),
    ((128, 256), 12001, 8, (515, 520), True),
    ((256, 128), 5000, 3, (257, 264), False),
    ((256, 128), 20001, 4, (71, 72), True),
    ((256, 256), 12001, 3, (515, 520), True),
]
FIRST, BEHIND = 3, 5        # rows of no expert in front of the first and behind the last


def counts_of(m, experts):
    """Rows of very unequal experts, one of them without any."""
    r = random.Random(m + experts)
    part = [r.random() ** 2 + 0.02 for _ in range(experts)]
    part[experts // 2] = 0
    counts = [int((m - FIRST - BEHIND) * p / sum(part)) for p in part]
    counts[-1] += m - FIRST - BEHIND - sum(counts)
    return counts


@pytest.fixture(scope="module", autouse=True)
def _built():
    qbuild.build()


@pytest.mark.parametrize("sms", [1, 2, 3, 76, 132, 148, 152])
def test_tiles_follow_the_rows(sms):
    small, large = ((16, 64), (16, 128), (32, 128)), ((128, 64), (128, 128), (128, 256), (256, 128), (256, 256))
    for experts in (1, 2, 9, 64, 1024):
        for m in (1, 8, 100, 512, 2048, 2049, 16384, 1 << 24):
            for n in (1, 64, 65, 2432, 5120, 1 << 24):
                tile = _lib.gemm_fp8_grouped_tile(m, n, experts, sms)
                assert tile in small + large and (tile[0] < 256 or sms > 1)
                most = min(m, experts) + m // 16        # tiles of 16 rows, at most
                if -(-n // 64) * most <= sms:
                    assert tile == (16, 64)
                elif -(-n // 128) * most <= sms or m // experts <= 12:
                    assert tile == (16, 128)
                else:
                    assert tile == (32, 128) if m // experts <= 32 else tile in large


@pytest.mark.parametrize("sms", [148, 152])
@pytest.mark.parametrize("tile,m,experts,ns,several", TILES)
def test_the_cases_reach_their_tiles(tile, m, experts, ns, several, sms):
    counts = counts_of(m, experts)
    assert sum(counts) == m - FIRST - BEHIND and counts[experts // 2] == 0
    for n in ns:
        assert _lib.gemm_fp8_grouped_tile(m, n, experts, sms) == tile
        tiles = sum(-(-c // tile[0]) for c in counts) * -(-n // tile[1])
        assert (tiles > sms // (2 if tile[0] == 256 else 1)) == several
    assert {t[0] for t in TILES} == {(16, 64), (16, 128), (32, 128), (128, 64), (128, 128), (128, 256), (256, 128),
                                     (256, 256)}


def test_refusals():
    for args in ((0, 1, 1, 152), (1, 0, 1, 152), (1, (1 << 24) + 1, 1, 152), ((1 << 24) + 1, 1, 1, 152), (1, 1, 0, 152),
                 (1, 1, 1025, 152), (1, 1, 1, 0), (1, 1, 1, 4097)):
        with pytest.raises(qg.QGError):
            _lib.gemm_fp8_grouped_tile(*args)
