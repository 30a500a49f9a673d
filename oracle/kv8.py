"""fp64 CPU oracle of the 8-bit KV cache (test infrastructure only): writing
new tokens into it, reading it back, and causal attention over it, as their
plain definitions.

The cache keeps one byte per value and one scale per (sequence, KV head, block
of positions). A stored value is code * scale:
  int8  code in -127..127, stored as code + 128; scale = fp32(a / 127) for a
        block whose largest magnitude is a;
  e4m3  4 exponent bits of bias 7, 3 mantissa bits, largest value 448; scale
        = the smallest power of two with a / scale <= 448; at 2^120, the
        largest there is, codes stop at 240 (256 would be 2^128, past bf16).
Bytes that a write never stores count as what their bits say without special
cases: 0 in int8 is -128, 0x7F and 0xFF (the NaNs of e4m3) are +-480.
A scale is at least 2^-60, and 0 for a block of zeros. The stored scale is an
fp32 number and the code is x * fp32(1 / scale) rounded to nearest even; the
product is taken in fp32 (one rounding), as everything is that decides a code.

Parity status: pinned by tests/test_kv8_oracle.py (hand-worked codes, the e4m3
value table, round trips within half a step, growth of an open block, and
torch's scaled_dot_product_attention on the dequantised cache).
"""
from __future__ import annotations

import math

import numpy as np

from .moe import bf16_bits_to_f64

FLOOR = np.float32(2.0 ** -60)


def e4m3_value(code) -> np.ndarray:
    """The value of e4m3 bytes (fp64; +-480 for the two NaN codes)."""
    c = np.asarray(code, dtype=np.int64)
    e, m = (c >> 3) & 15, c & 7
    mag = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where(c & 128, -mag, mag)


_E4M3 = e4m3_value(np.arange(127))  # 0 .. 448, increasing


def e4m3_code(y) -> np.ndarray:
    """The byte of the e4m3 number nearest to y (ties to the even code),
    saturating: by search in the table of all values."""
    y = np.asarray(y, dtype=np.float64)
    mag = np.minimum(np.abs(y), 448.0)
    hi = np.clip(np.searchsorted(_E4M3, mag), 1, 126)
    lo = hi - 1
    dl, dh = mag - _E4M3[lo], _E4M3[hi] - mag
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(mag == 0, 0, code)
    return np.where(np.signbit(y), code | 128, code).astype(np.uint8)


def scale_of(a, fmt):
    """The fp32 scale of a block with largest magnitude a (fp32)."""
    a = np.float32(a)
    if a == 0:
        return np.float32(0)
    if fmt == "int8":
        s = np.float32(a / np.float32(127))
    else:
        e = -200
        while float(a) > 448.0 * 2.0 ** e:
            e += 1
        s = np.float32(2.0 ** e)
    return max(s, FLOOR)


def value_of(code, scale, fmt) -> np.ndarray:
    c = np.asarray(code, dtype=np.float64) - 128.0 if fmt == "int8" else e4m3_value(code)
    return c * np.float64(scale)


def code_of(x, scale, fmt) -> np.ndarray:
    """Codes of fp32 values x at an fp32 scale."""
    inv = np.float32(1) / scale if scale > 0 else np.float32(0)
    y = np.asarray(x, dtype=np.float32) * inv
    if fmt == "int8":
        return (np.clip(np.rint(y), -127, 127) + 128).astype(np.uint8)
    return e4m3_code(np.clip(y, -240, 240) if scale == np.float32(2.0 ** 120) else y)


def write(x_bits, offsets, starts, codes, scales, block, fmt):
    """New tokens x_bits uint16 [T, H, D] into codes uint8 [B, H, L, D] and
    scales fp32 [B, H, nblk] (one of K and V), in place. Returns whether an
    input was not finite (a NaN then counts as 0, an infinity as its sign
    times the largest finite magnitude of the block's new values)."""
    x = bf16_bits_to_f64(x_bits).astype(np.float32)
    odd = False
    for b in range(len(starts)):
        lo, n, p = int(offsets[b]), int(offsets[b + 1] - offsets[b]), int(starts[b])
        done = 0
        while done < n:
            blk = (p + done) // block
            take = min(n - done, (blk + 1) * block - (p + done))
            r0 = p + done - blk * block
            for h in range(x.shape[1]):
                new = x[lo + done:lo + done + take, h].copy()
                fin = np.isfinite(new)
                a = np.abs(new[fin]).max() if fin.any() else np.float32(0)
                odd |= not fin.all()
                new[np.isnan(new)] = 0
                new = np.clip(new, -a, a)
                s_old = scales[b, h, blk] if r0 > 0 else np.float32(0)
                s = max(s_old, scale_of(a, fmt))
                rows = codes[b, h, blk * block:blk * block + r0]
                if r0 > 0 and s > s_old:
                    rows[:] = code_of((value_of(rows, 1.0, fmt).astype(np.float32) * s_old), s, fmt)
                codes[b, h, p + done:p + done + take] = code_of(new, s, fmt)
                scales[b, h, blk] = s
            done += take
    return odd


def read(offsets, starts, codes, scales, block, fmt) -> np.ndarray:
    """The stored values of the ranges, fp64 [T, H, D]."""
    out = []
    for b in range(len(starts)):
        for j in range(int(offsets[b + 1] - offsets[b])):
            p = int(starts[b]) + j
            out.append(value_of(codes[b, :, p], scales[b, :, p // block][:, None].astype(np.float64), fmt))
    return np.stack(out) if out else np.zeros((0,) + codes.shape[1::2])


def attention(q_bits, k_codes, v_codes, k_scales, v_scales, offsets, lens, block, fmt, scale=None):
    """Causal attention of every sequence's last tokens over its cache.
    Returns o and the same sums over |V| (what rounding errors scale with),
    fp64 [T, Hq, D]."""
    q = bf16_bits_to_f64(q_bits)
    T, Hq, D = q.shape
    H = k_codes.shape[1]
    r = Hq // H
    s = 1.0 / math.sqrt(D) if scale is None else float(scale)
    o, o_abs = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    for b in range(len(lens)):
        lo, n, L = int(offsets[b]), int(offsets[b + 1] - offsets[b]), int(lens[b])
        if n == 0 or L == 0:
            continue
        at = np.arange(L) // block
        for g in range(H):
            K = value_of(k_codes[b, g, :L], k_scales[b, g][at][:, None], fmt)
            V = value_of(v_codes[b, g, :L], v_scales[b, g][at][:, None], fmt)
            for i in range(n):
                see = L - n + i + 1
                if see <= 0:
                    continue
                for h in range(g * r, (g + 1) * r):
                    z = s * (K[:see] @ q[lo + i, h])
                    w = np.exp(z - z.max())
                    w /= w.sum()
                    o[lo + i, h] = w @ V[:see]
                    o_abs[lo + i, h] = w @ np.abs(V[:see])
    return o, o_abs
