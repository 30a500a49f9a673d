"""How the 8-bit cache's attention kernels share their work, restated from the
device code step by step: the places that tiles take, the cut into runs, the
search for a run's start (32 sequences at a time), a run's walk, the table of run
starts and what both merge kernels make of it. The constants come from the
sources."""
import os
import random
import re
from collections import namedtuple

import pytest

from tests.test_kv8_partition import empty_tiles, seq_tiles, tile_units, units_before

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_grouped_expert_moe_gb300", "csrc")


def _constant(name, file):
    with open(os.path.join(CSRC, file)) as f:
        found = re.findall(r"constexpr int %s = (\d+);" % name, f.read())
    assert len(found) == 1, (name, file, found)
    return int(found[0])


SPLIT_COST, TILES_COST = _constant("kTileCost", "kv8_split.cu"), _constant("kTileCost", "kv8_tiles.cu")
SPLIT_CTAS, TILES_CTAS = _constant("kMaxCtas", "kv8_split.cu"), _constant("kMaxCtas", "kv8_tiles.cu")
ROWS, KEYS = _constant("kRows", "kv8_tiles.cu"), _constant("kKeys", "kv8_tiles.cu")

Place = namedtuple("Place", "b g rt i nb tile lo n len units")
Kind = namedtuple("Kind", "RT KT cost")
SPLIT = [Kind(rows, keys, SPLIT_COST) for keys, most in ((64, 16), (128, 32)) for rows in (8, 16, 32) if rows <= most]
TILES = [Kind(2 * ROWS, KEYS, TILES_COST), Kind(ROWS, KEYS, TILES_COST)]


def test_the_constants_are_the_ones_meant():
    assert (SPLIT_COST, TILES_COST, ROWS, KEYS) == (4, 3, 128, 128)


def places_before(n, ln, r, k, kind):
    return units_before(n, ln, r, kind.RT, kind.KT, k) + kind.cost * max(k - empty_tiles(n, ln, r, kind.RT), 0)


def run_start(N, C, c):
    return c * (N // C) + min(c, N % C)


def find_run(seqs, Hkv, r, kind, c, C):
    """find_run of one warp; seqs: (lo, n, len) per sequence."""
    RT, KT, cost = kind
    B = len(seqs)
    total, before, units, tiles, at = 0, 0, 0, 0, 0
    base, phase = 0, 0
    while base < B:
        chunk = []
        for lane in range(32):
            b = base + lane
            v1 = w1 = nt1 = lo = n = ln = 0
            if b < B:
                lo, n, ln = seqs[b]
                nt1 = seq_tiles(n, r, RT)
                w1 = units_before(n, ln, r, RT, KT, nt1)
                v1 = w1 + cost * (nt1 - empty_tiles(n, ln, r, RT))
            chunk.append((v1, w1, nt1, lo, n, ln))
        reach = min(B, 32)  # the scan takes log2 steps that reach this far, its total that lane's
        vi, wi, ti = ([sum(x[k] for x in chunk[:i + 1]) * Hkv for i in range(reach)] for k in range(3))
        base += 32
        if phase == 0:
            total += vi[-1]
            if base < B:
                continue
            at = run_start(total, C, c)
            phase = 1
            if B > 32:
                base = 0
                continue
        hit = [i for i in range(reach) if before + vi[i] > at]
        if hit:
            L = hit[0]
            v1, w1, nt1, lo, n, ln = chunk[L]
            off = at - (before + vi[L] - v1 * Hkv)
            units += wi[L] - w1 * Hkv
            tiles += ti[L] - nt1 * Hkv
            g = off // v1
            off -= g * v1
            a, z = 0, nt1
            while z - a > 1:
                step = (z - a + 31) // 32
                last = max(i for i in range(32)
                           if a + i * step < z and places_before(n, ln, r, a + i * step, kind) <= off)
                a += last * step
                z = min(z, a + step)
            first = units_before(n, ln, r, RT, KT, a)
            i = max(off - first - cost * (max(a - empty_tiles(n, ln, r, RT), 0) + 1), 0)
            return Place(base - 32 + L, g, a, i, tile_units(n, ln, r, RT, KT, a), tiles + g * nt1 + a, lo, n, ln,
                         units + g * w1 + first + i)
        before += vi[-1]
        units += wi[-1]
        tiles += ti[-1]
    return Place(-1, 0, 0, 0, 0, 0, 0, 0, 0, units)


def walk(seqs, Hkv, r, kind, start, count):
    """The (tile, unit) pairs of a run: Cursor.advance."""
    b, g, rt, i, nb, tile, _, n, ln, _ = start
    out = []
    for j in range(count):
        out.append(((b, g, rt), tile, i, nb))
        if j + 1 == count:
            break
        i += 1
        if i < nb:
            continue
        i = 0
        while True:
            tile += 1
            rt += 1
            if rt >= seq_tiles(n, r, kind.RT):
                rt = 0
                g += 1
                if g >= Hkv:
                    g = 0
                    while True:
                        b += 1
                        _, n, ln = seqs[b]
                        if n != 0:
                            break
                        # a sequence without tokens has no tiles
            nb = tile_units(n, ln, r, kind.RT, kind.KT, rt)
            if nb:
                break
    return out


def _batch(rng, kind):
    B = rng.choice([1, 1, 2, 3, 8, 31, 32, 33, 40, 64, 65, 100])
    r = rng.choice([1, 2, 3, 5, 8, 20, 64])
    Hkv = rng.choice([1, 1, 2, 3, 8])
    rows = kind.RT // r + 1
    seqs, lo = [], 0
    for _ in range(B):
        n = rng.choice([0, 1, 1, rng.randint(0, 3 * rows), rng.randint(0, 2 * rows)])
        ln = rng.choice([0, 1, rng.randint(0, 200), rng.randint(0, 3000), n, max(n - 3, 0), n + rng.randint(0, 700)])
        seqs.append((lo, n, ln))
        lo += n
    return seqs, Hkv, r


def _all_units(seqs, Hkv, r, kind):
    out, tile = [], 0
    for b, (_, n, ln) in enumerate(seqs):
        for g in range(Hkv):
            for rt in range(seq_tiles(n, r, kind.RT)):
                nb = tile_units(n, ln, r, kind.RT, kind.KT, rt)
                out += [((b, g, rt), tile, i, nb) for i in range(nb)]
                tile += 1
    return out, tile


def _runs(seqs, Hkv, r, kind, C):
    starts = [find_run(seqs, Hkv, r, kind, c, C) for c in range(C + 1)]
    runs = [walk(seqs, Hkv, r, kind, a, z.units - a.units) for a, z in zip(starts, starts[1:])]
    info = [(a.tile if a.b >= 0 else 0, bool(w), a.i if a.b >= 0 else 0) for a, w in zip(starts, runs)]
    return runs, info


@pytest.mark.parametrize("C", [1, 2, 7, 76, 152])
@pytest.mark.parametrize("kind", SPLIT + TILES)
def test_runs_cover_every_unit_once(kind, C):
    rng = random.Random(C * 1000 + kind.RT)
    for _ in range(12):
        seqs, Hkv, r = _batch(rng, kind)
        runs, _ = _runs(seqs, Hkv, r, kind, C)
        want, _ = _all_units(seqs, Hkv, r, kind)
        assert [u for w in runs for u in w] == want
        # no run is longer than the places it was dealt
        N = len(want) + kind.cost * len({u[1] for u in want})
        assert max(map(len, runs)) <= -(-N // C)


@pytest.mark.parametrize("C", [1, 2, 7, 148, 152])
@pytest.mark.parametrize("kind", SPLIT)
def test_split_merge_takes_the_runs_of_a_tile(kind, C):
    """Every (run, tile) has a slot of its own within the workspace, and the merge
    of each tile reads exactly those of the runs that worked on it."""
    rng = random.Random(C * 1000 + kind.RT + 1)
    for _ in range(12):
        seqs, Hkv, r = _batch(rng, kind)
        runs, info = _runs(seqs, Hkv, r, kind, C)
        units, tiles = _all_units(seqs, Hkv, r, kind)
        worked = [(c, t) for c, w in enumerate(runs) for t in sorted({u[1] for u in w})]
        slots = [c + t for c, t in worked]
        assert len(set(slots)) == len(slots)
        rows, B = sum(n for _, n, _ in seqs) * r, len(seqs)
        assert max(slots, default=0) < SPLIT_CTAS + (rows // kind.RT + min(rows, B)) * Hkv
        for t in {u[1] for u in units}:
            c1 = max(c for c, (tile, live, _) in enumerate(info) if live and tile <= t)
            c0 = max(c for c, (tile, live, i) in enumerate(info) if live and tile <= t and (tile < t or i == 0))
            assert list(range(c0, c1 + 1)) == [c for c, x in worked if x == t]


@pytest.mark.parametrize("kind,C", [(k, C) for k in TILES for C in (1, 2, 7, 74, 76, 152)
                                    if C <= TILES_CTAS * ROWS // k.RT])  # runs of one or two blocks
def test_tiles_merge_joins_every_shared_tile_once(kind, C):
    """A run leaves at most two partial states, and a tile that several runs
    share is joined by one of them alone, from all of their slots."""
    rng = random.Random(C * 1000 + kind.RT + 2)
    for _ in range(25):
        seqs, Hkv, r = _batch(rng, kind)
        runs, info = _runs(seqs, Hkv, r, kind, C)
        units, _ = _all_units(seqs, Hkv, r, kind)
        state, whole = {}, set()  # (run, slot) -> tile; tiles finished by their run
        for c, w in enumerate(runs):
            for t in sorted({u[1] for u in w}):
                mine = [u for u in w if u[1] == t]
                mid, ends = mine[0][2] > 0, mine[-1][2] == mine[-1][3] - 1
                if not mid and ends:
                    whole.add(t)
                else:
                    assert (c, 0 if mid else 1) not in state
                    state[c, 0 if mid else 1] = t
        joined = {}
        for c, (tile, live, i) in enumerate(info):
            if not live or i == 0:
                continue
            earlier = [k for k in range(c) if info[k][1]]
            if not earlier:
                continue
            c0 = earlier[-1]
            later = sum(1 for k in range(c, C) if info[k][1] and info[k][0] == tile)
            if info[c0][0] == tile and info[c0][2] > 0:
                continue
            assert tile not in joined
            joined[tile] = [(k, 1 if k == c0 else 0) for k in range(c0, c + later)]
        for t in {u[1] for u in units}:
            held = sorted(k for k, x in state.items() if x == t)
            assert (t in whole) == (not held)
            assert joined.get(t, []) == held
        assert not whole & set(joined)


@pytest.mark.parametrize("kind", SPLIT + TILES)
def test_fewer_places_than_runs(kind):
    """One row over one position, and a batch of such: most runs have nothing."""
    for B in (1, 5, 40):
        seqs = [(b, 1, 1) for b in range(B)]
        runs, info = _runs(seqs, 1, 1, kind, 152)
        assert [u for w in runs for u in w] == _all_units(seqs, 1, 1, kind)[0]
        assert sum(live for _, live, _ in info) <= B
