"""The size of the 8-bit KV cache attention's workspace: one for the largest call
serves the smaller ones."""
import ctypes

import pytest
import torch

SHAPES = [(1, 16, 2, 256), (16, 16, 4, 128), (64, 16, 2, 256), (128, 40, 8, 128), (256, 40, 8, 128), (300, 8, 8, 64),
          (4096, 16, 16, 128), (7, 64, 1, 64), (33, 20, 4, 128)]


def _bytes(m, B, T, Hq, Hkv, D):
    n = ctypes.c_size_t()
    assert m.lib().moe_kv8_workspace_bytes(ctypes.byref(m.kv8_shape(B, T, Hq, Hkv, D, 4096)), ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("B,Hq,Hkv,D", SHAPES)
def test_more_tokens_need_no_less(moelib, B, Hq, Hkv, D):
    """Around every change of kernels and of rows per tile, and far beyond."""
    last = (36 * B * Hkv + 192) // Hq
    r = Hq // Hkv
    marks = {0, 1, last, B * (8 // r), B * (16 // r), 2 * last, 1 << 20}
    ts = sorted({max(t + d, 0) for t in marks for d in range(-3, 4)} | {last * i // 50 for i in range(120)})
    sizes = [_bytes(moelib, B, t, Hq, Hkv, D) for t in ts]
    assert sizes == sorted(sizes), [(t, a, b) for t, a, b in zip(ts, sizes, sizes[1:]) if b < a]


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,D", [(128, 40, 8, 128), (256, 8, 8, 64)])
def test_one_workspace_for_all_steps(moelib, cuda_dev, B, Hq, Hkv, D):
    """A workspace sized at the largest step, whose kernels need less of it than
    a smaller step's: every step runs in it, and as in one of its own."""
    m, dev, L = moelib, cuda_dev, 40
    gen = torch.Generator(device=dev).manual_seed(3)
    i32 = dict(dtype=torch.int32, device=dev)
    cache = m.kv8_alloc_cache(m.kv8_shape(B, 0, Hq, Hkv, D, L, 16), dev)
    sizes = [31, 1, 3, 6, 8, 12]
    ws = m.kv8_alloc_workspace(m.kv8_shape(B, B * max(sizes), Hq, Hkv, D, L, 16), dev)
    for i, n in enumerate(sizes):
        sh = m.kv8_shape(B, B * n, Hq, Hkv, D, L, 16)
        q, k, v = (torch.randn(B * n, h, D, generator=gen, device=dev).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
        off, lens = torch.arange(B + 1, **i32) * n, torch.full((B,), max(n, 31), **i32)
        m.kv8_write(sh, k, v, off, lens - n, cache)
        o, want = torch.zeros_like(q), torch.ones_like(q)
        m.kv8_attn(sh, q, cache, off, lens, o, ws)
        assert m.status_read(ws[:4].view(torch.int32)) == 0
        m.kv8_attn(sh, q, cache, off, lens, want, m.kv8_alloc_workspace(sh, dev))
        assert torch.equal(o, want)
