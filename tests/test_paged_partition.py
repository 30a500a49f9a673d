"""How the paged attention kernel deals its work out (integer arithmetic
restated here): the two searches for a run's start against an enumeration of
all units, and what the merge kernel makes of the runs' heads."""
import os
import random
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_grouped_expert_moe_gb300", "csrc")
with open(os.path.join(CSRC, "paged_attn.cu")) as f:
    SRC = f.read()


def _constant(name):
    return int(re.search(rf"\b{name} = (\d+)", SRC).group(1))


KEYS, SMALL_TILES = _constant("kKeys"), _constant("kSmallTiles")


def seq_tiles(n, r, RT):
    return (n * r + RT - 1) // RT


def tile_units(n, ln, r, RT, rt):
    see = ln - n + (min(n * r, (rt + 1) * RT) - 1) // r + 1
    return (see + KEYS - 1) // KEYS if see > 0 else 0


def starts(N, C, c):
    return c * (N // C) + min(c, N % C)


def enumerate_units(ns, lens, H, r, RT, cost):
    """Every place: (b, g, rt, i, tile, units before, whether it is a unit and not a tile's cost)."""
    out, tile, units = [], 0, 0
    for b, (n, ln) in enumerate(zip(ns, lens)):
        for g in range(H):
            for rt in range(seq_tiles(n, r, RT)):
                nb = tile_units(n, ln, r, RT, rt)
                if nb:
                    out += [(b, g, rt, 0, tile, units, False)] * cost
                    out += [(b, g, rt, i, tile, units + i, True) for i in range(nb)]
                units += nb
                tile += 1
    return out, units


def find_small(ns, lens, H, r, RT, cost, c, C):
    """Lane k has `per` sequences from per k on, one tile each."""
    B = len(ns)
    per = (B + 31) >> 5
    nb = [(ln + KEYS - 1) // KEYS if n > 0 else 0 for n, ln in zip(ns, lens)]
    lanes = [range(min(k * per, B), min(k * per + per, B)) for k in range(32)]
    v = [sum(nb[b] + cost for b in bs if nb[b]) for bs in lanes]
    w = [sum(nb[b] for b in bs) for bs in lanes]
    t = [sum(ns[b] > 0 for b in bs) for bs in lanes]
    N = sum(v) * H
    at = starts(N, C, c)
    hits = [k for k in range(32) if sum(v[:k + 1]) * H > at]
    if not hits:
        return None, sum(w) * H
    L = hits[0]
    off, units, tile, b = at - sum(v[:L]) * H, sum(w[:L]) * H, sum(t[:L]) * H, L * per
    while nb[b] == 0 or off >= (nb[b] + cost) * H:
        off -= (nb[b] + cost) * H if nb[b] else 0
        units += nb[b] * H
        tile += H if ns[b] else 0
        b += 1
    g = off // (nb[b] + cost)
    i = max(off - g * (nb[b] + cost) - cost, 0)
    return (b, g, 0, i, tile + g), units + g * nb[b] + i


def find_tiles(ns, lens, H, r, RT, cost, c, C):
    sums = []
    for n, ln in zip(ns, lens):
        nb = [tile_units(n, ln, r, RT, rt) for rt in range(seq_tiles(n, r, RT))]
        sums.append((sum(x + cost for x in nb if x), sum(nb)))
    N = sum(s[0] for s in sums) * H
    off = starts(N, C, c)
    if off >= N:
        return None, sum(s[1] for s in sums) * H
    b = units = tile = 0
    while off >= sums[b][0] * H:
        off -= sums[b][0] * H
        units += sums[b][1] * H
        tile += seq_tiles(ns[b], r, RT) * H
        b += 1
    g = off // sums[b][0]
    off -= g * sums[b][0]
    units += g * sums[b][1]
    tile += g * seq_tiles(ns[b], r, RT)
    rt = 0
    while True:  # 32 tiles at a time
        nb = [tile_units(ns[b], lens[b], r, RT, rt + k) if rt + k < seq_tiles(ns[b], r, RT) else 0 for k in range(32)]
        v = [x + cost if x else 0 for x in nb]
        hits = [k for k in range(32) if sum(v[:k + 1]) > off]
        if hits:
            break
        off -= sum(v)
        units += sum(nb)
        rt += 32
    k = hits[0]
    i = max(off - sum(v[:k]) - cost, 0)
    return (b, g, rt + k, i, tile + rt + k), units + sum(nb[:k]) + i


def _calls(rng, count, single):
    for _ in range(count):
        B, H, r = rng.randint(1, 70 if single else 6), rng.randint(1, 3), rng.choice([1, 2, 3, 5, 8, 64])
        RT = rng.choice([128, 256])
        lens = [rng.choice([0, 1, 128, 129, rng.randint(0, 900)]) for _ in range(B)]
        most = RT // r if single else 700 // r + 1
        ns = [rng.choice([0, rng.randint(0, most), min(ln, rng.randint(0, most))]) for ln in lens]
        yield ns, lens, H, r, RT, rng.choice([1, 3]), rng.choice([1, 3, 76, 152])


def _check(find, single):
    rng = random.Random(7)
    for ns, lens, H, r, RT, cost, C in _calls(rng, 150, single):
        places, total = enumerate_units(ns, lens, H, r, RT, cost)
        N = len(places)
        for c in {0, C // 2, max(C - 1, 0), C} | {rng.randint(0, C) for _ in range(4)}:
            at = starts(N, C, c)
            got, units = find(ns, lens, H, r, RT, cost, c, C)
            if at >= N:
                assert got is None and units == total
            else:
                b, g, rt, i, tile, before, _ = places[at]
                assert (got, units) == ((b, g, rt, i, tile), before), (ns, lens, H, r, RT, cost, C, c)


def test_starts_of_single_tiles():
    _check(find_small, True)


def test_starts_among_several_tiles():
    _check(find_tiles, False)


def test_single_tiles_by_either_search():
    rng = random.Random(8)
    for ns, lens, H, r, RT, cost, C in _calls(rng, 60, True):
        for c in range(0, C + 1, max(1, C // 5)):
            assert find_small(ns, lens, H, r, RT, cost, c, C) == find_tiles(ns, lens, H, r, RT, cost, c, C)


def test_the_merge_joins_every_cut_tile_once_from_all_of_its_runs():
    rng = random.Random(9)
    cut = 0
    for ns, lens, H, r, RT, cost, C in _calls(rng, 200, False):
        places, _ = enumerate_units(ns, lens, H, r, RT, cost)
        N, heads, runs = len(places), [], {}
        for c in range(C):
            mine = places[starts(N, C, c):starts(N, C, c + 1)]
            units = [p for p in mine if p[6]]
            heads.append((mine[0][4], 1 | (2 if mine[0][3] > 0 else 0)) if units else (-1, 0))
            for p in units:
                runs.setdefault(p[4], set()).add(c)
        want = {t: sorted(cs) for t, cs in runs.items() if len(cs) > 1}
        got = {}
        for t in range(C):
            tile, what = heads[t]
            before = heads[t - 1] if t else (-1, 0)
            if what & 2 and not (before[1] & 2 and before[0] == tile):
                c1 = t
                while c1 + 1 < C and heads[c1 + 1][1] and heads[c1 + 1][0] == tile:
                    c1 += 1
                assert tile not in got
                got[tile] = list(range(t - 1, c1 + 1))
        assert got == want, (ns, lens, H, r, RT, cost, C)
        cut += len(want)
    assert cut > 200
