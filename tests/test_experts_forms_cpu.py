"""The forms that the GPU tests of 4-bit products run reach every branch of the
dispatch, whose rules are read from the sources here."""

import re

from test_dense_sources_cpu import code
from w4_forms import FORMS

W4, TC, SHARED = code("k_w4.cu"), code("k_w4_tc.cu"), code("experts.cuh")


def constant(text, name):
    return int(re.search(rf"\b{name}\s*=\s*(\d+)", text).group(1))


STREAM, ROWS = constant(SHARED, "kW4Stream"), constant(SHARED, "kW4Rows")
TILE, STAGES, TOKENS = constant(code("dense_cluster.cuh"), "kRows"), constant(TC, "kStages"), constant(TC, "kMostTokens")


def two_tiles(n, k):
    m = re.search(r"const bool two = a\.N >= (\d+) && a\.K >= (\d+);", W4)
    return n >= int(m.group(1)) and k >= int(m.group(2))


def split(rows, k, n):
    """CTAs along K, and tiles of tokens."""
    m = re.search(r"int n = (\d+);\s*while \(n > 1 && \(tiles \* n > (\d+) \|\| n > pairs\)\) --n;", TC)
    ttiles = -(-rows // TOKENS)
    tiles, s = -(-n // TILE) * ttiles, int(m.group(1))
    while s > 1 and (tiles * s > int(m.group(2)) or s > -(-k // 128)):
        s -= 1
    return s, ttiles


def test_streaming_instances():
    """Each number of eights of tokens with each number of tiles of weight rows,
    and remainders along every axis in the larger ones."""
    small = [f for f in FORMS if f[0] <= STREAM]
    assert {(rows > 8, two_tiles(n, k)) for rows, k, n in small} == {(a, b) for a in (False, True) for b in (False, True)}
    big = [f for f in small if two_tiles(f[2], f[1])]
    assert any(k % 128 for _, k, _ in big) and any(n % 32 for _, _, n in big) and any(n % 8 for _, _, n in big)


def test_clusters_and_rings():
    mid = [f for f in FORMS if STREAM < f[0] <= ROWS]
    assert {split(*f)[0] for f in mid} == {1, 2, 3, 4}
    # rings that wrap, in a cluster of each size that can
    assert {split(*f)[0] for f in mid if -(-f[1] // 128) // split(*f)[0] > STAGES} >= {1, 2, 3, 4}
    assert {split(*f)[1] for f in mid} == {1, 2}
    assert {k % 128 for _, k, _ in mid} == {0, 32, 64, 96}
    assert any(n % 8 and split(rows, k, n)[0] == 1 for rows, k, n in mid) and any(n % 8 and split(rows, k, n)[0] > 1 for rows, k, n in mid)


def test_unpacked_products():
    large = [f for f in FORMS if f[0] > ROWS]
    assert any(n % 8 for _, _, n in large) and any(n % 8 == 0 for _, _, n in large)
