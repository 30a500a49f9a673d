"""What the 8-bit KV cache's entry points refuse on the host, before any CUDA
call (the fake device addresses are never dereferenced)."""
import ctypes

import pytest
import torch

REF = ctypes.byref
GOOD = dict(B=2, T=8, Hq=16, Hkv=2, D=256, L_max=4096, block=64, format=0, q_stride=0, kv_stride=0)
ADDR = [0x100000 * (i + 1) for i in range(8)]


@pytest.mark.parametrize("kw,code", [
    (dict(), 0), (dict(B=0), 2), (dict(B=4097), 2), (dict(T=-1), 2), (dict(T=(1 << 24) + 1), 2),
    (dict(T=1 << 24), 0), (dict(T=1 << 24, B=1, Hkv=64, Hq=64), 0), (dict(T=1 << 24, B=1, Hkv=65, Hq=65), 2),
    (dict(Hkv=0), 2), (dict(Hkv=3), 2), (dict(Hq=0), 2), (dict(Hq=130), 2), (dict(Hq=128), 0), (dict(Hq=258), 2),
    (dict(B=4096, Hkv=32, Hq=32), 2), (dict(B=16, Hkv=4096, Hq=4096), 0), (dict(B=1, Hkv=4097, Hq=4097), 2),
    (dict(D=64), 0), (dict(D=128), 0), (dict(D=96), 2), (dict(D=512), 2), (dict(L_max=0), 2), (dict(L_max=1 << 26), 0),
    (dict(L_max=(1 << 26) + 1), 2), (dict(block=16), 0), (dict(block=32), 0), (dict(block=8), 2), (dict(block=128), 2),
    (dict(format=1), 0), (dict(format=2), 2), (dict(format=-1), 2), (dict(q_stride=4096), 0), (dict(q_stride=4100), 2),
    (dict(q_stride=4088), 2), (dict(q_stride=-4096), 2), (dict(kv_stride=512), 0), (dict(kv_stride=5120), 0),
    (dict(kv_stride=504), 2), (dict(kv_stride=514), 2)])
def test_shapes(moelib, kw, code):
    sh = moelib.kv8_shape(**{**GOOD, **kw})
    n = ctypes.c_size_t()
    L = moelib.lib()
    assert L.moe_kv8_workspace_bytes(REF(sh), REF(n)) == code
    # with a null cache a good shape gets as far as the pointer checks
    assert L.moe_kv8_write(REF(sh), *ADDR[:4], None, None, None) == (code or 1)
    assert L.moe_kv8_read(REF(sh), None, *ADDR[:4], None, None) == (code or 1)
    assert L.moe_kv8_attn(REF(sh), ADDR[0], None, ADDR[1], ADDR[2], 0.1, ADDR[3], ADDR[4], 1 << 40, None) == (code or 1)


def _cache(moelib, **kw):
    c = moelib.Kv8CacheC(0x1000000, 0x2000000, 0x3000000, 0x4000000)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [dict(k_codes=None), dict(v_codes=None), dict(k_scales=None), dict(v_scales=None), dict(k_codes=0x1000008),
              dict(v_codes=0x2000001), dict(k_scales=0x3000002), dict(v_scales=0x4000001)]


def test_write_and_read_arguments(moelib):
    L, sh, c = moelib.lib(), moelib.kv8_shape(**GOOD), _cache(moelib)
    k, v, off, st = ADDR[:4]

    def write(k=k, v=v, off=off, st=st, c=c, status=None, sh=sh):
        return L.moe_kv8_write(REF(sh) if sh else None, k, v, off, st, REF(c) if c else None, status, None)

    def read(k=k, v=v, off=off, st=st, c=c, status=None, sh=sh):
        return L.moe_kv8_read(REF(sh) if sh else None, REF(c) if c else None, off, st, k, v, status, None)

    for call in (write, read):
        for kw in (dict(k=None), dict(v=None), dict(off=None), dict(st=None), dict(c=None), dict(sh=None),
                   dict(k=k + 8), dict(v=v + 2), dict(off=off + 2), dict(st=st + 1), dict(status=0x900002)):
            assert call(**kw) == 1, kw
        for kw in BAD_CACHES:
            assert call(c=_cache(moelib, **kw)) == 1, kw
        assert call(sh=moelib.kv8_shape(**{**GOOD, "T": 0}), k=None, v=None, off=None, st=None) == 0


def test_attention_arguments(moelib):
    L, sh, c = moelib.lib(), moelib.kv8_shape(**GOOD), _cache(moelib)
    q, off, ln, o, ws = ADDR[:5]
    need = moelib.kv8_workspace_bytes(sh)

    def attn(q=q, c=c, off=off, ln=ln, scale=0.0625, o=o, ws=ws, n=need, sh=sh):
        return L.moe_kv8_attn(REF(sh) if sh else None, q, REF(c) if c else None, off, ln, scale, o, ws, n, None)

    for kw in (dict(q=None), dict(off=None), dict(ln=None), dict(o=None), dict(ws=None), dict(c=None), dict(sh=None),
               dict(q=q + 8), dict(o=o + 4), dict(off=off + 2), dict(ln=ln + 1), dict(ws=ws + 16), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan"))):
        assert attn(**kw) == 1, kw
    for kw in BAD_CACHES:
        assert attn(c=_cache(moelib, **kw)) == 1, kw
    assert attn(n=need - 1) == 3
    for block, limit in [(-1, 10 ** 6), (0, 0), (0, -5), (0, 10 ** 10)]:
        assert L.moe_kv8_attn_test_stall(REF(sh), q, REF(c), off, ln, 0.0625, o, ws, need, block, limit, None) == 1
    assert L.moe_kv8_workspace_bytes(None, REF(ctypes.c_size_t())) == 1
    assert L.moe_kv8_workspace_bytes(REF(sh), None) == 1


def test_binding_refuses_tensors_of_the_wrong_kind(moelib, monkeypatch):
    """The checks the C entry points cannot make: type, sizes, strides, device."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # CPU tensors are "on" device -1
    sh = moelib.kv8_shape(B=1, T=3, Hq=4, Hkv=2, D=64, L_max=20, block=16, kv_stride=256)
    x = torch.zeros(3, 256, dtype=torch.bfloat16)
    k, v = x[:, :128].view(3, 2, 64), x[:, 128:].view(3, 2, 64)
    off, st = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    cache = moelib.kv8_alloc_cache(sh, "cpu")
    assert cache.k.shape == (1, 2, 20, 64) and cache.k_scale.shape == (1, 2, 2)

    def refused(text, **kw):
        a = dict(k=k, v=v, off=off, st=st, cache=cache, sh=sh, status=None)
        a.update(kw)
        with pytest.raises(moelib.MoeError, match=text) as e:
            moelib.kv8_write(a["sh"], a["k"], a["v"], a["off"], a["st"], a["cache"], a["status"], stream=0)
        assert e.value.status == moelib.MOE_ERR_INVALID_ARG

    refused("k_new is torch.float32", k=k.float())
    refused("k_new has shape", k=k[:2])
    refused("v_new has strides", v=v.contiguous())
    refused("v_new has strides", v=v.transpose(1, 2).contiguous().transpose(1, 2))
    refused("offsets is torch.int64", off=off.long())
    refused("offsets has shape", off=off[:1])
    refused("starts has shape", st=torch.zeros(2, dtype=torch.int32))
    refused("status is torch.int64", status=torch.zeros(1, dtype=torch.int64))
    for text, c in [("k is torch.int8", (cache.k.to(torch.int8), cache.v, cache.k_scale, cache.v_scale)),
                    ("v has shape", (cache.k, cache.v[:, :, :19], cache.k_scale, cache.v_scale)),
                    ("v is torch.int8", (cache.k, cache.v.to(torch.int8), cache.k_scale, cache.v_scale)),
                    ("k has strides", (cache.k.transpose(1, 2), cache.v, cache.k_scale, cache.v_scale)),
                    ("k_scale is torch.float64", (cache.k, cache.v, cache.k_scale.double(), cache.v_scale)),
                    ("v_scale has shape", (cache.k, cache.v, cache.k_scale, cache.v_scale[:, :, :1])),
                    ("scales", (cache.k, cache.v, cache.k_scale[0], cache.v_scale))]:
        with pytest.raises(moelib.MoeError, match=text):
            moelib.Kv8Cache(*c)
    c = moelib.Kv8Cache(cache.k, cache.v, cache.k_scale[:, :, :1].contiguous(), cache.v_scale[:, :, :1].contiguous())
    refused("the cache holds", cache=c)
    refused("the cache holds", sh=moelib.kv8_shape(B=1, T=3, Hq=4, Hkv=2, D=64, L_max=33, block=16, kv_stride=256))
    fp8 = moelib.kv8_alloc_cache(moelib.kv8_shape(B=1, T=3, Hq=4, Hkv=2, D=64, L_max=20, block=16, format=1), "cpu")
    refused("the cache holds", cache=fp8)
    q, ws = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(1 << 16, dtype=torch.uint8)
    for text, kw in [("q is torch.float16", dict(q=q.half())), ("o has shape", dict(o=q[:1])),
                     ("lens is torch.int64", dict(st=st.long())), ("workspace is torch.float32", dict(ws=ws.float()))]:
        a = {**dict(q=q, o=q, st=st, ws=ws), **kw}
        with pytest.raises(moelib.MoeError, match=text):
            moelib.kv8_attn(sh, a["q"], cache, off, a["st"], a["o"], a["ws"], stream=0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    refused("not on the current device")
