"""fp64 CPU oracle of rotary positions and of the paged KV cache (test
infrastructure only): the frequencies of the scalings, heads normed and
rotated, tokens appended, attention (causal and for trees of drafts), and the
accepted drafts kept, as their plain definitions.

Arrays hold bf16 bit patterns (uint16) where the library holds bf16. Position p
of sequence b is row p % page of page tables[b][p // page].

Parity status: pinned by tests/test_paged_oracle.py (hand-worked rotations,
rotation as a complex product, the difference of positions alone deciding a
score, scalings at their ends, torch's scaled_dot_product_attention on
gathered pages with the tree's mask, moves of hand-made paths).
"""
from __future__ import annotations

import math

import numpy as np

from .moe import bf16_bits_to_f64


def frequencies(rot, base=1e4, scaling="plain", factor=1.0, original=0, low=1.0, high=None):
    """Radians per position of the rot / 2 pairs and the magnitude."""
    high = (32.0 if scaling == "ramp" else 4.0) if high is None else high
    out = []
    for i in range(rot // 2):
        w = base ** (-2.0 * i / rot)
        if scaling == "linear":
            w = w / factor
        elif scaling == "bands":
            t = original * w / (2 * math.pi)
            if t <= low:
                w = w / factor
            elif t < high:
                w = w / factor + (w - w / factor) * (t - low) / (high - low)
        elif scaling == "ramp":
            lo, hi = (rot * math.log(original / (2 * math.pi * t)) / (2 * math.log(base)) for t in (high, low))
            lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
            u = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            w = w * (1 - u) + w / factor * u
        out.append(w)
    return np.array(out), 0.1 * math.log(factor) + 1.0 if scaling == "ramp" else 1.0


def normed(x, gain=None, eps=1e-6, offset=0.0):
    """Heads x fp64 [..., D] over their root mean square, times offset + gain (1 without a gain)."""
    y = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return y if gain is None else y * (offset + gain)


def rotated(x, positions, w, pairs=False, magnitude=1.0):
    """Heads x fp64 [T, H, D]: the first 2 len(w) values of each turned by its token's position. Angles are
    reduced in integers: positions up to 2^31 times w in plain fp64 would lose 2^-22."""
    rot = 2 * len(w)
    a = np.asarray(positions, dtype=object)[:, None] * np.array([_fraction(v) for v in w], dtype=object)[None]
    turn = np.array([[float(int(v) % (1 << 120)) / float(1 << 120) for v in row] for row in a]).reshape(len(a), len(w))
    c, s = (magnitude * f(2 * math.pi * turn)[:, None, :] for f in (np.cos, np.sin))
    y = x.copy()
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., two] * c + x[..., one] * s
    return y


def _fraction(w) -> int:
    """w / 2 pi in units of 2^-120, by integers (2 pi to 200 bits)."""
    from fractions import Fraction
    return int(Fraction(float(w)) / _TWO_PI * (1 << 120))


def _two_pi():
    """2 pi by Machin's formula, pi = 16 atan(1/5) - 4 atan(1/239), in integers."""
    from fractions import Fraction
    one = 1 << 260

    def atan_inv(n):
        total, term, k = 0, one // n, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total
    return Fraction(2 * (16 * atan_inv(5) - 4 * atan_inv(239)), one)


_TWO_PI = _two_pi()


def rows_of(pages, table, n, page):
    """Positions 0 .. n - 1 of a sequence: [Hkv, n, D]."""
    H, D = pages.shape[1], pages.shape[3]
    out = np.empty((H, n, D), dtype=pages.dtype)
    for p in range(n):
        out[:, p] = pages[table[p // page], :, p % page]
    return out


def append(new_bits, offsets, starts, pages, tables, page):
    """New rows (bits, [T, Hkv, D]) to their places, in place."""
    for b in range(len(starts)):
        for i in range(int(offsets[b + 1] - offsets[b])):
            p = int(starts[b]) + i
            pages[tables[b][p // page], :, p % page] = new_bits[int(offsets[b]) + i]


def visible(n, length, words=None):
    """[n, length] truth values: what each of a sequence's last n tokens sees; words: ints of each draft's bits."""
    see = np.zeros((n, length), dtype=bool)
    for i in range(n):
        for j in range(min(length, max(0, length - n + i + 1))):
            d = j - (length - n)
            see[i, j] = words is None or d < 0 or (words[i] >> d) & 1
    return see


def attention(q_bits, k_pages, v_pages, tables, page, offsets, lens, words=None, scale=None):
    """Attention of every sequence's last tokens over its pages; words: per
    token of the call an int of its draft's bits. Returns o and the same sums
    over |V|, fp64 [T, Hq, D]. Values that a query does not see are not touched."""
    q = bf16_bits_to_f64(q_bits)
    T, Hq, D = q.shape
    r = Hq // k_pages.shape[1]
    s = 1.0 / math.sqrt(D) if scale is None else float(scale)
    o, o_abs = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    for b in range(len(lens)):
        lo, n, L = int(offsets[b]), int(offsets[b + 1] - offsets[b]), int(lens[b])
        if n == 0 or L == 0:
            continue
        K, V = (bf16_bits_to_f64(rows_of(x, tables[b], L, page)) for x in (k_pages, v_pages))
        see = visible(n, L, None if words is None else words[lo:lo + n])
        for i in range(n):
            at = np.flatnonzero(see[i])
            if len(at) == 0:
                continue
            for h in range(Hq):
                z = s * (K[h // r][at] @ q[lo + i, h])
                w = np.exp(z - z.max())
                w /= w.sum()
                o[lo + i, h] = w @ V[h // r][at]
                o_abs[lo + i, h] = w @ np.abs(V[h // r][at])
    return o, o_abs


def keep(pages, tables, page, starts, path, kept):
    """The accepted drafts' rows behind the context, in place."""
    for b in range(len(starts)):
        rows = [pages[tables[b][(starts[b] + j) // page], :, (starts[b] + j) % page].copy() for j in path[b][:kept[b]]]
        for k, row in enumerate(rows):
            p = starts[b] + k
            pages[tables[b][p // page], :, p % page] = row
