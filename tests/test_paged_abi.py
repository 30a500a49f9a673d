"""What the entry points of rotary positions and the paged KV cache refuse on
the host, before any CUDA call (the fake device addresses are never
dereferenced), the table of turns, and how the attention kernel's ring is laid
out."""
import ctypes
import glob
import math
import os
import random
import re

import numpy as np
import pytest
import torch

from oracle import paged

REF = ctypes.byref
ADDR = [0x100000 * (i + 1) for i in range(12)]
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_grouped_expert_moe_gb300", "csrc")

ROPE = dict(T=8, Hq=16, Hk=2, D=256)


def _spec(m, **kw):
    f = dict(turns=0x7000000, q_gain=None, k_gain=None, rot=64, layout=0, norm=0, eps=1e-6, gain_offset=0.0, magnitude=1.0)
    f.update(kw)
    return m.RopeSpecC(*f.values())


def _rope(m, sh, spec, q=ADDR[0], k=ADDR[1], pos=ADDR[2], qo=ADDR[3], ko=ADDR[4]):
    return m.lib().moe_rope(REF(sh) if sh else None, REF(spec) if spec else None, q, k, pos, qo, ko, None)


@pytest.mark.parametrize("kw,code", [
    (dict(), 1), (dict(T=-1), 2), (dict(T=(1 << 24) + 1), 2), (dict(Hq=0, Hk=0), 2), (dict(Hq=-1), 2), (dict(Hk=4097), 2),
    (dict(T=1 << 24, Hq=65, Hk=0), 2), (dict(D=0), 2), (dict(D=72), 2), (dict(D=272), 2), (dict(D=80), 1),
    (dict(q_stride=4096), 1), (dict(q_stride=4088), 2), (dict(k_stride=516), 2), (dict(qo_stride=4092), 2),
    (dict(ko_stride=-512), 2), (dict(ko_stride=504), 2)])
def test_rope_shapes(moelib, kw, code):
    # without positions a good shape gets as far as the pointer checks
    assert _rope(moelib, moelib.rope_shape(**{**ROPE, **kw}), _spec(moelib), pos=None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(rot=0), 1), (dict(rot=8), 2), (dict(rot=272), 2), (dict(rot=-16), 2), (dict(rot=256), 1), (dict(layout=2), 2),
    (dict(layout=-1), 2), (dict(norm=4), 2), (dict(norm=-1), 2), (dict(norm=3), 1), (dict(norm=1, eps=0.0), 2),
    (dict(norm=1, eps=-1.0), 2), (dict(eps=0.0), 1), (dict(eps=math.inf), 2), (dict(gain_offset=math.nan), 2),
    (dict(magnitude=math.inf), 2), (dict(turns=None), 1), (dict(turns=0x7000008), 1), (dict(q_gain=0x8000002), 1),
    (dict(k_gain=0x8000008), 1)])
def test_rope_specs(moelib, kw, code):
    assert _rope(moelib, moelib.rope_shape(**ROPE), _spec(moelib, **kw), q=None) == code
    sh = moelib.paged_shape(**PAGED)
    assert _append(moelib, sh, spec=_spec(moelib, **kw), k=None) == code


def test_rope_arguments(moelib):
    m, sh, sp = moelib, moelib.rope_shape(**ROPE), _spec(moelib)
    for kw in (dict(q=None), dict(k=None), dict(pos=None), dict(qo=None), dict(ko=None), dict(q=ADDR[0] + 8),
               dict(k=ADDR[1] + 2), dict(pos=ADDR[2] + 2), dict(qo=ADDR[3] + 8), dict(ko=ADDR[4] + 4)):
        assert _rope(m, sh, sp, **kw) == 1, kw
    assert _rope(m, None, sp) == 1 and _rope(m, sh, None) == 1
    assert _rope(m, m.rope_shape(0, 16, 2, 256), sp, None, None, None, None, None) == 0
    assert _rope(m, m.rope_shape(4, 0, 2, 256), sp, q=None, qo=None, k=None) == 1


@pytest.mark.parametrize("kw,code", [
    (dict(rot=8), 2), (dict(rot=0), 2), (dict(rot=512), 2), (dict(scaling=4), 1), (dict(scaling=-1), 1),
    (dict(reserved=1), 1), (dict(base=1.0), 1), (dict(base=math.nan), 1), (dict(base=math.inf), 1), (dict(factor=0.5), 1),
    (dict(factor=math.nan), 1), (dict(scaling=2, original=0), 1), (dict(scaling=3, original=-5), 1),
    (dict(scaling=2, low=0.0), 1), (dict(scaling=2, low=4.0), 1), (dict(scaling=3, high=math.inf), 1), (dict(), 0),
    (dict(scaling=3), 0), (dict(original=0, low=0.0), 0)])
def test_frequencies_refused(moelib, kw, code):
    f = dict(rot=64, scaling=0, original=4096, reserved=0, base=1e4, factor=2.0, low=1.0, high=4.0, given=None)
    f.update(kw)
    c, t, mag = moelib.RopeFrequencies(*f.values()), (ctypes.c_uint64 * 128)(), ctypes.c_float()
    L = moelib.lib()
    assert L.moe_rope_table(REF(c), t, REF(mag)) == code
    assert L.moe_rope_table(None, t, REF(mag)) == 1 and L.moe_rope_table(REF(c), None, REF(mag)) == 1
    bad = (ctypes.c_double * 32)(*([0.1] * 31 + [math.inf]))
    c.given = bad
    assert L.moe_rope_table(REF(c), t, REF(mag)) == (code or 1)


@pytest.mark.parametrize("rot,base,scaling,factor,original,low,high", [
    (64, 1e7, "plain", 1.0, 0, 1.0, None), (128, 1e4, "linear", 4.0, 0, 1.0, None), (64, 5e5, "bands", 8.0, 8192, 1.0, None),
    (128, 1e4, "bands", 32.0, 4096, 0.5, 20.0), (128, 1e4, "ramp", 32.0, 32768, 1.0, None), (16, 1e6, "ramp", 4.0, 64, 2.0, 8.0)])
def test_table_of_turns(moelib, rot, base, scaling, factor, original, low, high):
    """Turns within 2^-54 of the oracle's (fp64 on both sides, two roundings of up to 2^-53 of values below 0.16, and
    pow's last place)."""
    m = moelib
    t = m.rope_table(rot, base, getattr(m, f"ROPE_{scaling.upper()}"), factor, original, low, high, device="cpu")
    w, magnitude = paged.frequencies(rot, base, scaling, factor, original, low, high)
    assert t.rot == rot and t.turns.shape == (rot // 2,) and t.magnitude == pytest.approx(magnitude, rel=1e-7)
    for got, want in zip(t.turns.tolist(), w):
        assert abs((got % (1 << 64)) / 2.0 ** 64 - want / (2 * math.pi)) <= 2.0 ** -54


def test_given_frequencies(moelib):
    """Whole turns count for nothing, and a negative frequency turns the other way."""
    w = [0.0, 1.0, -1.0, 2 * math.pi + 1.0, -0.25, 1e-9, 3.0, 100.0]
    t = moelib.rope_table(16, freqs=w, device="cpu").turns.tolist()
    for got, want in zip(t, w):
        d = (got / 2.0 ** 64 - want / (2 * math.pi)) % 1.0
        assert min(d, 1 - d) <= 2.0 ** -48
    with pytest.raises(moelib.MoeError, match="7 frequencies for 8 pairs"):
        moelib.rope_table(16, freqs=w[:7], device="cpu")


# ----------------------------------------------------------- paged cache ---

PAGED = dict(B=2, T=8, Hq=16, Hkv=2, D=256, page=64, n_pages=100, max_pages=40)


def _cache(m, **kw):
    c = m.PagedCacheC(0x1000000, 0x2000000, 0x3000000)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [dict(k_pages=None), dict(v_pages=None), dict(tables=None), dict(k_pages=0x1000008), dict(v_pages=0x2000002),
              dict(tables=0x3000002)]


def _append(m, sh, spec=None, q=ADDR[0], k=ADDR[1], v=ADDR[2], off=ADDR[3], st=ADDR[4], pos=None, c=1, qo=ADDR[5],
            status=None):
    c = _cache(m) if c == 1 else c
    return m.lib().moe_paged_append(REF(sh) if sh else None, REF(spec) if spec else None, q, k, v, off, st, pos,
                                    REF(c) if c else None, qo, status, None)


@pytest.mark.parametrize("kw,code", [
    (dict(), 0), (dict(B=0), 2), (dict(B=4097), 2), (dict(T=-1), 2), (dict(T=(1 << 24) + 1), 2), (dict(Hkv=0), 2),
    (dict(Hkv=3), 2), (dict(Hq=0), 2), (dict(Hq=130), 2), (dict(Hq=128), 0), (dict(Hq=258), 2), (dict(D=64), 0),
    (dict(D=96), 2), (dict(D=512), 2), (dict(page=16), 0), (dict(page=256), 0), (dict(page=8), 2), (dict(page=512), 2),
    (dict(page=48), 2), (dict(n_pages=0), 2), (dict(n_pages=1 << 30), 2), (dict(n_pages=(1 << 30) - 1), 0),
    (dict(max_pages=0), 2), (dict(max_pages=1 << 20), 0), (dict(max_pages=(1 << 20) + 1), 2), (dict(tree_words=8), 0),
    (dict(tree_words=9), 2), (dict(tree_words=-1), 2), (dict(q_stride=4096), 0), (dict(q_stride=4100), 2),
    (dict(q_stride=4088), 2), (dict(kv_stride=512), 0), (dict(kv_stride=504), 2), (dict(B=4096, Hkv=32, Hq=32), 2)])
def test_paged_shapes(moelib, kw, code):
    m, L = moelib, moelib.lib()
    sh, n = m.paged_shape(**{**PAGED, **kw}), ctypes.c_size_t()
    assert L.moe_paged_workspace_bytes(REF(sh), REF(n)) == code
    # with a null cache a good shape gets as far as the pointer checks
    assert _append(m, sh, c=None) == (code or 1)
    assert L.moe_paged_keep(REF(sh), None, *ADDR[:3], 8, None, None, None) == (code or 1)
    assert L.moe_paged_attn(REF(sh), ADDR[0], None, ADDR[1], ADDR[2], None, 0.1, ADDR[3], ADDR[4], 1 << 40, None) == (code or 1)


def test_append_arguments(moelib):
    m, sh = moelib, moelib.paged_shape(**PAGED)
    for kw in (dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(off=None), dict(st=None), dict(q=ADDR[0] + 8),
               dict(k=ADDR[1] + 2), dict(v=ADDR[2] + 8), dict(off=ADDR[3] + 2), dict(st=ADDR[4] + 1), dict(pos=ADDR[6] + 2),
               dict(qo=ADDR[5] + 4), dict(status=ADDR[7] + 2)):
        assert _append(m, sh, **kw) == 1, kw
    assert _append(m, None) == 1
    for kw in BAD_CACHES:
        assert _append(m, sh, c=_cache(m, **kw)) == 1, kw
    assert _append(m, m.paged_shape(**{**PAGED, "T": 0}), None, None, None, None, None, None, qo=None) == 0


def test_keep_arguments(moelib):
    m, sh = moelib, moelib.paged_shape(**PAGED)

    def keep(c=None, st=ADDR[0], kept=ADDR[1], path=ADDR[2], width=8, out=None, status=None, sh=sh):
        return m.lib().moe_paged_keep(REF(sh) if sh else None, REF(c or _cache(m)), st, kept, path, width, out, status, None)

    for kw in (dict(st=None), dict(kept=None), dict(path=None), dict(st=ADDR[0] + 2), dict(kept=ADDR[1] + 1),
               dict(path=ADDR[2] + 2), dict(out=ADDR[3] + 2), dict(status=ADDR[4] + 2), dict(sh=None)):
        assert keep(**kw) == 1, kw
    assert keep(width=-1) == 2 and keep(width=513) == 2
    for kw in BAD_CACHES:
        assert keep(c=_cache(m, **kw)) == 1, kw


def test_attention_arguments(moelib):
    m, L, sh = moelib, moelib.lib(), moelib.paged_shape(**PAGED)
    q, off, ln, o, ws = ADDR[:5]
    need = m.paged_workspace_bytes(sh)

    def attn(q=q, c=None, off=off, ln=ln, tree=None, scale=0.0625, o=o, ws=ws, n=need, sh=sh):
        return L.moe_paged_attn(REF(sh) if sh else None, q, REF(c or _cache(m)), off, ln, tree, scale, o, ws, n, None)

    for kw in (dict(q=None), dict(off=None), dict(ln=None), dict(o=None), dict(ws=None), dict(sh=None), dict(q=q + 8),
               dict(o=o + 4), dict(off=off + 2), dict(ln=ln + 1), dict(ws=ws + 16), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=math.inf), dict(scale=math.nan), dict(tree=ADDR[5])):
        assert attn(**kw) == 1, kw
    tree = m.paged_shape(**{**PAGED, "tree_words": 1})
    assert attn(sh=tree) == 1 and attn(sh=tree, tree=ADDR[5] + 4) == 1
    for kw in BAD_CACHES:
        assert attn(c=_cache(m, **kw)) == 1, kw
    assert attn(n=need - 1) == 3
    for block, limit in [(-1, 10 ** 6), (0, 0), (0, -5), (0, 10 ** 10)]:
        assert L.moe_paged_attn_test_stall(REF(sh), q, REF(_cache(m)), off, ln, None, 0.0625, o, ws, need, block, limit,
                                           None) == 1
    assert L.moe_paged_workspace_bytes(None, REF(ctypes.c_size_t())) == 1
    assert L.moe_paged_workspace_bytes(REF(sh), None) == 1


@pytest.mark.parametrize("scale", [3.4028234e38, 2.36e38, 1e39])
def test_a_scale_whose_base_2_form_passes_fp32(moelib, scale):
    """scale log2(e) would be infinite: refused (as invalid, not for the workspace, which is too small here)."""
    m, L, sh = moelib, moelib.lib(), moelib.paged_shape(**PAGED)
    for s, code in ((scale, 1), (2.3e38, 3)):
        assert L.moe_paged_attn(REF(sh), ADDR[0], REF(_cache(m)), ADDR[1], ADDR[2], None, s, ADDR[3], ADDR[4], 0, None) == code


def test_a_workspace_serves_calls_of_any_number_of_tokens(moelib):
    sizes = {moelib.paged_workspace_bytes(moelib.paged_shape(**{**PAGED, "T": T, "tree_words": w}))
             for T in (0, 1, 50, 4000, 1 << 20) for w in (0, 4)}
    assert len(sizes) == 1


def test_binding_refuses_tensors_of_the_wrong_kind(moelib, monkeypatch):
    """The checks the C entry points cannot make: type, sizes, strides, device."""
    m = moelib
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    bf = dict(dtype=torch.bfloat16)
    sh = m.paged_shape(B=1, T=3, Hq=4, Hkv=2, D=64, page=16, n_pages=5, max_pages=4, kv_stride=256)
    cache = m.paged_alloc_cache(sh, "cpu")
    assert cache.k.shape == (5, 2, 16, 64) and cache.tables.shape == (1, 4)
    x = torch.zeros(3, 256, **bf)
    q, k, v = torch.zeros(3, 4, 64, **bf), x[:, :128].view(3, 2, 64), x[:, 128:].view(3, 2, 64)
    i32 = dict(dtype=torch.int32)
    # a cache of CPU tensors is refused by every call
    for call in (lambda: m.paged_append(sh, None, q, k, v, torch.zeros(2, **i32), torch.zeros(1, **i32), cache, q),
                 lambda: m.paged_attn(sh, q, cache, torch.zeros(2, **i32), torch.zeros(1, **i32), q,
                                      torch.zeros(1 << 20, dtype=torch.uint8)),
                 lambda: m.paged_keep(sh, cache, torch.zeros(1, **i32), torch.zeros(1, **i32), torch.zeros(1, 3, **i32))):
        with pytest.raises(m.MoeError, match="not on the current device") as e:
            call()
        assert e.value.status == m.MOE_ERR_INVALID_ARG
    with pytest.raises(m.MoeError, match="not on the current device"):
        m.rope(m.rope_shape(3, 4, 0, 64), m.rope_spec(), q, None, None, q, None)
    for text, c in [("k is torch.float16", (cache.k.half(), cache.v, cache.tables)),
                    ("v has shape", (cache.k, cache.v[:4], cache.tables)),
                    ("k has strides", (cache.k.transpose(1, 2), cache.v, cache.tables)),
                    ("tables is torch.int64", (cache.k, cache.v, cache.tables.long())),
                    ("pages are", (cache.k[0], cache.v, cache.tables)),
                    ("pages are", (cache.k, cache.v, cache.tables[0]))]:
        with pytest.raises(m.MoeError, match=text):
            m.PagedCache(*c)
    g = torch.ones(64, **bf)
    for text, kw in [("q_gain is torch.float32", dict(q_gain=g.float())), ("k_gain has shape", dict(q_gain=g, k_gain=g[:32])),
                     ("q_gain has shape", dict(q_gain=g.view(1, 64))), ("k_gain has strides", dict(k_gain=x[:, 0]))]:
        with pytest.raises(m.MoeError, match=text):
            m.rope_spec(**kw)


# ------------------------------------------------------- the kernel's plan ---

def _order(tiles, bufs):
    """The order of the products S and O of a run of tiles of so many units, as the issuing and loading warps go: S ahead
    of O as far as there are buffers, but not over a tile's end."""
    out, u = [], 0
    for nu in tiles:
        for j in range(1 - bufs, nu):
            if j + bufs - 1 < nu:
                out.append(("S", u + j + bufs - 1))
            if j >= 0:
                out.append(("O", u + j))
        u += nu
    return out


@pytest.mark.parametrize("bufs", [2, 3])
def test_places_in_the_ring_are_the_order_of_use(bufs):
    """V's place as the warps that look through it have it; no S is written before O has taken the weights that lay
    there; a stage of the ring (one, two or four to a place) is always the same loading warp's."""
    rng = random.Random(5)
    for _ in range(500):
        tiles = [rng.randint(1, rng.choice([1, 2, 12])) for _ in range(rng.randint(1, 6))]
        order = _order(tiles, bufs)
        at = {x: i for i, x in enumerate(order)}
        assert len(at) == len(order) == 2 * sum(tiles)
        u = 0
        for nu in tiles:
            for j in range(nu):
                assert at["O", u + j] == 2 * (u + j) + 1 + min(bufs - 1, nu - 1 - j)
                assert u + j < bufs or at["S", u + j] > at["O", u + j - bufs]
                assert at["S", u + j] < at["O", u + j]
            u += nu
        for parts in (1, 2, 4):
            for place in range(len(order)):
                assert all((place * parts + h) % 8 % 2 == (place * parts + h) % 2 for h in range(parts))


def test_bits_of_values_that_are_not_finite_fit():
    """The units of a tile that some of its rows do not see, at most 8, for tiles of 128 and 256 rows."""
    rng = random.Random(6)
    most = 0
    for _ in range(20000):
        RT, r, tree = rng.choice([128, 256]), rng.randint(1, 64), rng.random() < 0.5
        n = rng.randint(1, 512 if tree else 3000)
        ln = n + rng.randint(-n, 1000)
        rt = rng.randrange((n * r + RT - 1) // RT)
        see = ln - n + (min(n * r, (rt + 1) * RT) - 1) // r + 1
        if see <= 0:
            continue
        part = max(ln - n + (0 if tree else rt * RT // r + 1), 0)
        last = (see + 127) // 128 - 1
        if (last + 1) * 128 > part:
            most = max(most, last - part // 128)
    assert 3 <= most < 8


SOURCES = sorted(glob.glob(os.path.join(CSRC, "paged*")) + glob.glob(os.path.join(CSRC, "rope*")))


def _code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_load_takes_the_non_coherent_path(path):
    """Blocks may be resident while the kernel before them still writes what
    they read (programmatic dependent launch): see tests/test_kv8_loads.py."""
    assert len(SOURCES) >= 5
    found = re.findall(r"__ldg\b|ldg_nc\w*|ld\.global\.nc[.\w]*|ld\.global\.\w+\.nc[.\w]*", _code(path))
    assert not found, found


@pytest.mark.parametrize("path", [p for p in SOURCES if p.endswith(".cu")], ids=os.path.basename)
def test_nothing_is_read_before_the_dependency_wait(path):
    for kernel in re.split(r"__global__", _code(path))[1:]:
        head = kernel.split("griddepcontrol.wait")[0]
        assert len(head) < len(kernel), kernel[:120]
        assert not re.findall(r"\bld\(|ld_u64\(|ld_once_v4\(|__ldcg|\bld\.global", head), head[-400:]
