"""How the 8-bit cache's attention kernels lay out and share their work, as
the device code does it (integer arithmetic restated here): the closed form for
the units before a tile, the search for a run's start, and which block joins
the partial states of a tile that several runs share."""
import random

import pytest


def seq_tiles(n, r, RT):
    return (n * r + RT - 1) // RT


def tile_units(n, ln, r, RT, KT, rt):
    see = ln - n + (min(n * r, (rt + 1) * RT) - 1) // r + 1
    return (see + KT - 1) // KT if see > 0 else 0


def floor_sum(n, m, a, b):
    s = 0
    while True:
        s += n * (n - 1) // 2 * (a // m) + n * (b // m)
        a, b = a % m, b % m
        top = a * n + b
        if top < m:
            return s
        n, b, m, a = top // m, top % m, a, m


def units_before(n, ln, r, RT, KT, k):
    s = 0
    if k <= 4:
        return sum(tile_units(n, ln, r, RT, KT, rt) for rt in range(k))
    if k == seq_tiles(n, r, RT):
        k -= 1
        s += tile_units(n, ln, r, RT, KT, k)
    c = RT - 1 + r * (ln - n + KT)
    k0 = (-c + RT - 1) // RT if c < 0 else 0
    return s + (floor_sum(k - k0, r * KT, RT, c + RT * k0) if k0 < k else 0)


def cta_of(s, N, C):
    return ((s + 1) * C - 1) // N


def empty_tiles(n, ln, r, RT):
    if n <= ln:
        return 0
    return seq_tiles(n, r, RT) if ln == 0 else min(seq_tiles(n, r, RT) - 1, (r * (n - ln) + RT) // RT - 1)


COST = 2  # places a tile takes beyond its units


def places_before(n, ln, r, k):
    return units_before(n, ln, r, 128, 128, k) + COST * max(k - empty_tiles(n, ln, r, 128), 0)


def find_tile(n, ln, r, off):
    a, z = 0, seq_tiles(n, r, 128)
    while z - a > 1:
        step = (z - a + 31) // 32
        last = max(i for i in range(32) if a + i * step < z and places_before(n, ln, r, a + i * step) <= off)
        a += last * step
        z = min(z, a + step)
    return a, max(off - places_before(n, ln, r, a) - COST, 0)


def _sequences(rng, count):
    for _ in range(count):
        r = rng.choice([1, 2, 3, 5, 7, 8, 16, 20, 64])
        yield rng.randint(1, 900), rng.choice([0, 1, rng.randint(0, 300), rng.randint(0, 5000)]), r


@pytest.mark.parametrize("RT,KT", [(128, 128), (256, 128), (8, 64), (16, 64), (32, 64)])
def test_closed_form(RT, KT):
    for n, ln, r in _sequences(random.Random(RT), 300):
        units = [tile_units(n, ln, r, RT, KT, rt) for rt in range(seq_tiles(n, r, RT))]
        at = 0
        for k in range(len(units) + 1):
            assert units_before(n, ln, r, RT, KT, k) == at
            at += units[k] if k < len(units) else 0
        assert empty_tiles(n, ln, r, RT) == sum(u == 0 for u in units)
        assert sorted(units[:empty_tiles(n, ln, r, RT)]) == [0] * empty_tiles(n, ln, r, RT)


def test_search_for_a_place():
    for n, ln, r in _sequences(random.Random(3), 200):
        at = 0
        for k in range(seq_tiles(n, r, 128)):
            units = tile_units(n, ln, r, 128, 128, k)
            if units:
                for i in {0, units // 2, units - 1}:
                    assert find_tile(n, ln, r, at + COST + i) == (k, i)
                assert find_tile(n, ln, r, at) == (k, 0) and find_tile(n, ln, r, at + COST - 1) == (k, 0)
                at += units + COST


def test_closed_form_at_the_largest_sizes():
    n, ln, r = 1 << 24, 1 << 26, 64
    for k in (5, 1 << 20, seq_tiles(n, r, 128) - 1, seq_tiles(n, r, 128)):
        got = units_before(n, ln, r, 128, 128, k)
        assert 0 < got < 1 << 44
        assert units_before(n, ln, r, 128, 128, k) - units_before(n, ln, r, 128, 128, k - 1) == tile_units(
            n, ln, r, 128, 128, k - 1)


def test_every_unit_is_run_and_every_shared_tile_joined_once():
    """A run that starts inside a tile's units holds its state in the block's
    first slot, the run that holds the tile's first unit (and not its last) in
    the second; exactly one block, that of the tile's second run, joins them."""
    rng = random.Random(5)
    for _ in range(300):
        C = rng.choice([1, 2, 7, 152])
        tiles = [rng.choice([1, 2, 3, rng.randint(1, 40), rng.randint(1, 400)]) for _ in range(rng.randint(1, 60))]
        N = sum(tiles) + COST * len(tiles)
        starts = [sum(tiles[:i]) + COST * (i + 1) for i in range(len(tiles))]  # places of the first units
        runs = [(c * N // C, (c + 1) * N // C) for c in range(C)]
        joined, done = {}, []
        for c, (lo, hi) in enumerate(runs):
            if lo >= hi:
                continue
            i = max(k for k, s in enumerate(starts) if s - COST <= lo)
            first = max(lo - starts[i], 0)
            units = sum(max(0, min(hi, s + n) - max(lo, s)) for s, n in zip(starts, tiles))
            at, k = first, i
            for _ in range(units):  # the run's walk
                done.append((k, at))
                at += 1
                if at == tiles[k]:
                    at, k = 0, k + 1
            if first == 0:
                continue
            start = lo - first
            assert start == starts[i]
            c0 = cta_of(start, N, C)
            if c != cta_of((c0 + 1) * N // C, N, C):
                continue
            c1 = cta_of(start + tiles[i] - 1, N, C)
            assert i not in joined
            joined[i] = [k for k in range(c0, c1 + 1) if runs[k][0] < runs[k][1]]
        assert done == [(k, i) for k, n in enumerate(tiles) for i in range(n)]
        for i, s in enumerate(starts):
            over = [c for c, (lo, hi) in enumerate(runs) if lo < s + tiles[i] and hi > s and lo < hi]
            assert (joined.get(i) == over) if len(over) > 1 else i not in joined
            for c in over[1:]:
                assert runs[c][0] > s  # its first slot
            if len(over) > 1:
                assert runs[over[0]][0] <= s and runs[over[0]][1] < s + tiles[i]  # its second slot
