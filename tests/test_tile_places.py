"""The arithmetic by which the tensor-core kernels find a tile (expert_tiles.cuh), on the CPU: quotients by a reciprocal that
is known before, quotients in float32 that are one off at most and are put right, and the tiles of uneven segments, which have
to cover each row and channel tile once."""
import random

import numpy as np
import pytest

F = np.float32


def by_reciprocal(n, d):
    """operator/ of a Divisor."""
    q = n * (0xFFFFFFFF // d) >> 32
    return q + (n - q * d >= d)


def divide(n, d, ulps=0):
    """divide(): the quotient is taken in float32, here with an error of its own besides (the approximate one is within 2)."""
    q = F(n) / F(d)
    q = F(q + q * F(ulps * 2.0 ** -23))
    q = max(int(q), 0)
    rest = n - q * d
    if rest < 0:
        q, rest = q - 1, rest + d
    elif rest >= d:
        q, rest = q + 1, rest - d
    return q, rest


def place_of(local, at, tiles, ctiles, ulps):
    before = at // 8 * 8
    channel, tile = divide(local - before * ctiles, min(8, tiles - before), ulps)
    return before + tile, channel


def test_quotients_by_a_known_reciprocal():
    rng = random.Random(0)
    divisors = list(range(1, 260)) + [2 ** k + s for k in range(8, 32) for s in (-1, 0, 1)] + [rng.randrange(1, 2 ** 32) for _ in range(500)]
    for d in divisors:
        most = (2 ** 32 - 1) // d
        ns = [rng.randrange(2 ** 32) for _ in range(40)] + [0, 1, 2 ** 31, 2 ** 32 - 1]
        ns += [k * d + s for k in (1, 2, 3, most // 2, most) for s in (-1, 0, 1)]
        for n in ns:
            if 0 <= n < 2 ** 32:
                assert by_reciprocal(n, d) == n // d, (n, d)


@pytest.mark.parametrize("ulps", [-3, 0, 3])
def test_small_quotients_in_float32(ulps):
    rng = random.Random(1)
    for d in list(range(1, 300)) + [2 ** k + s for k in range(9, 27) for s in (-1, 0, 1)] + [rng.randrange(1, 2 ** 26) for _ in range(500)]:
        for q in (0, 1, 7, 8, 255, 4096, 2 ** 19):
            for rest in {0, 1 % d, d // 2, d - 1}:
                n = q * d + rest
                if n < 2 ** 31:
                    assert divide(n, d, ulps) == (q, rest), (n, d)


@pytest.mark.parametrize("tile", [32, 64, 128, 256, 288])
@pytest.mark.parametrize("ctiles", [1, 3, 8, 55])
def test_tiles_cover_every_segment_once(tile, ctiles):
    rng = random.Random(tile + ctiles)
    segments = [0, 1, 31, 32, 33, tile - 1, tile, tile + 1, 0, 8 * tile, 8 * tile + 1, 17 * tile - 5] + [rng.randrange(12 * tile) for _ in range(12)]
    first = [0]
    for rows in segments:
        first.append(first[-1] + -(-rows // tile))
    covered = [[0] * ((rows + 31) // 32) for rows in segments]   # by groups of 32 rows, times channel tiles
    seen = set()
    for item in range(first[-1] * ctiles):
        at = by_reciprocal(item, ctiles)
        e = max(i for i in range(len(segments)) if first[i] <= at and segments[i])
        tiles = first[e + 1] - first[e]
        j, channel = place_of(item - first[e] * ctiles, at - first[e], tiles, ctiles, rng.choice([-3, 0, 3]))
        assert 0 <= j < tiles and 0 <= channel < ctiles
        assert (e, j, channel) not in seen
        seen.add((e, j, channel))
        each, more = divide((segments[e] + 31) // 32, tiles)
        start = j * each + min(j, more)
        m = min(32 * (each + (j < more)), segments[e] - 32 * start)
        assert 0 < m <= tile
        for g in range(start, start + (m + 31) // 32):
            covered[e][g] += 1
    assert len(seen) == first[-1] * ctiles
    assert all(n == ctiles for e in covered for n in e)
