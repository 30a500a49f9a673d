"""The 8-bit KV cache through the binding on the GPU against the fp64 oracle.

Writing and reading have no tolerance: codes, scales and read-back values are
the oracle's, bit for bit (every step that decides one is a single fp32
operation, the same on both sides; the read-back rounds once to bf16).

Attention, per element, from the arithmetic (u = 2^-24):
  * o is rounded to bf16: 2^-8 |o| (half a step of bf16);
  * every probability is rounded to fp16: 2^-11 * sum_j w_j |v_j|, and as much
    again for a denominator that sums rounded ones;
  * a score is a sum of D products of up to `amp` in all, with
    amp = scale * sum_d |q_d| * (largest stored magnitude: 255 code steps of
    int8, whose codes enter the product as code + 128, or the largest e4m3
    value) * the largest K scale; each of the D + 8 operations of its chain
    is off by at most 2 u of that, so the score by ds = (D + 8) 2 u amp, and
    the weights by a factor of up to e^(2 ds): 2 ds * sum_j w_j |v_j| for the
    ds here (below 0.05; a further 5 % covers the square term);
  * the sum over positions runs in chains of at most L / 16 + 64 additions,
    each off by 2 u of at most the largest stored V magnitude.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import kv8
from oracle.moe import bf16_bits_to_f64
from tests._util import bits16

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
FMTS = ["int8", "e4m3"]


def _fmt(m, fmt):
    return m.KV8_INT8 if fmt == "int8" else m.KV8_E4M3


def _i32(v):
    return torch.tensor([int(x) for x in v], dtype=torch.int32, device=DEV)


def _packed(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(int)


def _rand(gen, *shape):
    return torch.randn(shape, generator=gen, dtype=torch.float32)


class Pair:
    """A cache on the GPU beside the oracle's arrays, the same bytes in both.
    Positions that hold nothing yet hold arbitrary bytes and scales."""

    def __init__(self, m, B, Hkv, D, L, block, fmt, seed=0):
        rng = np.random.default_rng(seed)
        self.m, self.dims, self.block, self.fmt = m, (B, Hkv, D, L), block, fmt
        nblk = -(-L // block)
        self.codes = [rng.integers(0, 256, (B, Hkv, L, D)).astype(np.uint8) for _ in range(2)]
        self.scales = [np.where(rng.random((B, Hkv, nblk)) < 0.3, np.nan, rng.random((B, Hkv, nblk)) * 1e30)
                       .astype(np.float32) for _ in range(2)]
        t = [torch.from_numpy(c.copy()).to(DEV) for c in self.codes]
        if fmt == "e4m3":
            t = [x.view(torch.float8_e4m3fn) for x in t]
        self.gpu = m.Kv8Cache(*t, *[torch.from_numpy(s.copy()).to(DEV) for s in self.scales])

    def shape(self, T, Hq=None, **kw):
        B, Hkv, D, L = self.dims
        return self.m.kv8_shape(B, T, Hq or Hkv, Hkv, D, L, self.block, _fmt(self.m, self.fmt), **kw)

    def write(self, x, counts, starts, stream=None, expect=0, oracle=True):
        """x: K and V bf16 [T, Hkv, D] on the CPU."""
        off = _packed(counts)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.m.kv8_write(self.shape(int(off[-1])), x[0].to(DEV), x[1].to(DEV), _i32(off), _i32(starts), self.gpu,
                         status=st, stream=stream)
        assert self.m.status_read(st) == expect
        if oracle:
            for i in range(2):
                kv8.write(bits16(x[i]), off, starts, self.codes[i], self.scales[i], self.block, self.fmt)

    def bytes(self):
        return [x.view(torch.uint8).cpu().numpy() for x in (self.gpu.k, self.gpu.v)]

    def check(self):
        for got, want in zip(self.bytes(), self.codes):
            assert np.array_equal(got, want), np.argwhere(got != want)[:5]
        for got, want in zip((self.gpu.k_scale, self.gpu.v_scale), self.scales):
            assert np.array_equal(got.cpu().numpy(), want, equal_nan=True)

    def read(self, counts, starts):
        B, Hkv, D, _ = self.dims
        off = _packed(counts)
        T = int(off[-1])
        out = [torch.full((T, Hkv, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.m.kv8_read(self.shape(T), self.gpu, _i32(off), _i32(starts), *out, status=st)
        assert self.m.status_read(st) == 0
        for i in range(2):
            want = kv8.read(off, starts, self.codes[i], self.scales[i], self.block, self.fmt)
            want = torch.from_numpy(want).to(torch.float32).to(torch.bfloat16)
            assert torch.equal(out[i].cpu(), want)

    def fill(self, lens, seed=1, k_std=1.0, v_std=1.0):
        gen = torch.Generator().manual_seed(seed)
        _, Hkv, D, _ = self.dims
        T = sum(lens)
        gain = torch.exp(0.5 * _rand(gen, 1, Hkv, D))
        x = [(_rand(gen, T, Hkv, D) * gain * k_std).to(torch.bfloat16),
             (_rand(gen, T, Hkv, D) * v_std).to(torch.bfloat16)]
        self.write(x, lens, [0] * len(lens))
        return gen

    def attend(self, q, news, lens, scale=None, o=None, ws=None, stream=None):
        off = _packed(news)
        T, Hq, D = q.shape
        q = q if q.is_cuda else q.to(DEV)
        sh = self.shape(T, Hq, q_stride=0 if T < 2 else q.stride(0))
        o = torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16, device=DEV) if o is None else o
        ws = self.m.kv8_alloc_workspace(sh, DEV) if ws is None else ws
        self.m.kv8_attn(sh, q, self.gpu, _i32(off), _i32(lens), o, ws, scale=scale, stream=stream)
        assert self.m.status_read(ws[:4].view(torch.int32)) == 0
        return o

    def check_attention(self, q, news, lens, scale=None, rows=None):
        got = self.attend(q, news, lens, scale).double().cpu().numpy()
        off = _packed(news)
        want, o_abs = kv8.attention(bits16(q), *self.codes, *self.scales, off, lens, self.block, self.fmt, scale)
        self.compare(got, want, o_abs, q, lens, scale)

    def compare(self, got, want, o_abs, q, lens, scale=None):
        D = q.shape[2]
        s = D ** -0.5 if scale is None else scale
        top = [0.0, 0.0]
        for b, n in enumerate(lens):
            nb = -(-n // self.block)
            for i in range(2):
                sc = self.scales[i][b, :, :nb]
                step = 255.0 if self.fmt == "int8" else 448.0
                top[i] = max(top[i], step * float(sc.max()) if nb else 0.0)
        u2 = 2.0 ** -23
        amp = s * np.abs(bf16_bits_to_f64(bits16(q))).sum(2, keepdims=True) * top[0]
        ds = (D + 8) * u2 * amp
        assert ds.max(initial=0) < 0.05
        tol = 2.0 ** -8 * np.abs(want) + (2 * 2.0 ** -11 + 2.1 * ds) * o_abs + (max(lens) / 16 + 64) * u2 * top[1]
        err = np.abs(got - want)
        assert np.isfinite(got).all()
        assert (err <= tol).all(), (float((err / np.maximum(tol, 1e-300)).max()), np.argwhere(err > tol)[:4])


# ------------------------------------------------------------ write, read ---

WRITES = [  # B, Hkv, D, L, block, counts and starts of each call in turn
    (1, 2, 256, 200, 64, [([1], [0]), ([1], [1]), ([62], [2]), ([1], [64]), ([135], [65])]),
    (3, 1, 64, 77, 16, [([5, 0, 17], [0, 9, 60]), ([1, 1, 0], [5, 15, 77]), ([60, 33, 0], [6, 16, 0])]),
    (2, 3, 128, 70, 32, [([31, 70], [0, 0]), ([2, 1], [31, 69]), ([1, 5], [33, 3])]),
    (4, 8, 128, 33, 32, [([33, 1, 0, 32], [0, 32, 33, 1])]),
    (1, 1, 64, 1, 16, [([1], [0])]),
    (70, 2, 64, 20, 16, [([i % 4 for i in range(70)], [i % 17 for i in range(70)])]),
    (300, 1, 64, 40, 16, [([i % 3 for i in range(300)], [i % 37 for i in range(300)])]),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", range(len(WRITES)))
def test_write_and_read_are_the_oracles(moelib, cuda_dev, case, fmt):
    B, Hkv, D, L, block, calls = WRITES[case]
    p = Pair(moelib, B, Hkv, D, L, block, fmt, seed=case)
    # where a call starts inside a block, the block holds earlier tokens: give it a scale
    first = calls[0]
    for b, (n, s) in enumerate(zip(*first)):
        if s % block:
            for i, t in enumerate((p.gpu.k_scale, p.gpu.v_scale)):
                p.scales[i][b, :, s // block] = np.float32(2.0 ** -7)
                t[b, :, s // block] = 2.0 ** -7
    gen = torch.Generator().manual_seed(100 + case)
    for k, (counts, starts) in enumerate(calls):
        T = sum(counts)
        size = torch.exp(1.5 * _rand(gen, T, Hkv, 1))  # magnitudes that grow and shrink from token to token
        x = [(_rand(gen, T, Hkv, D) * size).to(torch.bfloat16) for _ in range(2)]
        p.write(x, counts, starts)
        p.check()
        before = p.bytes()
        p.write(x, counts, starts, oracle=False)  # the same again changes nothing
        assert all(np.array_equal(a, b) for a, b in zip(before, p.bytes()))
        p.check()
    p.read(calls[-1][0], calls[-1][1])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,lens", [(64, [7001, 0, 1, 3333]), (128, [2500, 2777]), (256, [5003, 64, 1])])
def test_write_and_read_of_many_tokens(moelib, cuda_dev, D, lens, fmt):
    """More tiles than the read kernel's blocks, of the larger kind."""
    p = Pair(moelib, len(lens), 8, D, max(lens), 32, fmt, seed=5)
    p.fill(lens, seed=6)
    p.check()
    p.read(lens, [0] * len(lens))
    p.read([max(n - 17, 0) for n in lens], [min(n, 17) for n in lens])


@pytest.mark.parametrize("fmt", FMTS)
def test_write_of_strided_tokens(moelib, cuda_dev, fmt):
    """Keys and values as column ranges of one projection output."""
    p = Pair(moelib, 2, 2, 128, 100, 32, fmt)
    gen = torch.Generator().manual_seed(3)
    T, Hq = 57, 6
    x = _rand(gen, T, (Hq + 4) * 128).to(torch.bfloat16)
    k, v = x[:, Hq * 128:(Hq + 2) * 128].view(T, 2, 128), x[:, (Hq + 2) * 128:].view(T, 2, 128)
    xg = x.to(DEV)
    kg, vg = xg[:, Hq * 128:(Hq + 2) * 128].view(T, 2, 128), xg[:, (Hq + 2) * 128:].view(T, 2, 128)
    off = _packed([40, 17])
    moelib.kv8_write(p.shape(T, Hq, kv_stride=x.shape[1]), kg, vg, _i32(off), _i32([0, 64]), p.gpu)
    for i, t in enumerate((k, v)):
        kv8.write(bits16(t), off, [0, 64], p.codes[i], p.scales[i], 32, fmt)
    p.check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("kind", ["zeros", "tiny", "huge", "subnormal", "edges"])
def test_write_of_extreme_values(moelib, cuda_dev, kind, fmt):
    p = Pair(moelib, 1, 2, 64, 96, 32, fmt)
    gen = torch.Generator().manual_seed(11)
    x = _rand(gen, 80, 2, 64)
    x = {"zeros": x * 0, "tiny": x * 2.0 ** -66, "huge": x.clamp(-3, 3) * 2.0 ** 126, "subnormal": x * 2.0 ** -130,
         "edges": torch.sign(x) * torch.tensor([448.0, 450.0, 1.0, 127.0, 63.5, 0.5])
          .repeat(80 * 2 * 64 // 6 + 1)[:80 * 2 * 64].view(80, 2, 64)}[kind]
    x = x.to(torch.bfloat16)
    p.write([x, -x], [80], [0])
    p.check()
    p.read([80], [0])
    y = _rand(gen, 5, 2, 64).to(torch.bfloat16)  # ordinary values join the open block
    p.write([y, y], [5], [80])
    p.check()
    p.read([60], [25])


@pytest.mark.parametrize("fmt", FMTS)
def test_write_reports_values_that_are_not_finite(moelib, cuda_dev, fmt):
    p = Pair(moelib, 2, 2, 64, 64, 16, fmt)
    gen = torch.Generator().manual_seed(12)
    x = [_rand(gen, 50, 2, 64).to(torch.bfloat16) for _ in range(2)]
    x[0][3, 0, 5], x[0][3, 1, 6], x[1][20, 0, :] = float("nan"), float("inf"), float("-inf")
    x[1][33:50] = float("nan")
    p.write(x, [33, 17], [0, 0], expect=moelib.MOE_ERR_RANGE)
    p.check()
    p.read([33, 17], [0, 0])


@pytest.mark.parametrize("entry", ["write", "read", "attn"])
@pytest.mark.parametrize("off,tab", [
    ([0, 3, 2, 6], [0, 0, 0]), ([1, 3, 4, 6], [0, 0, 0]), ([0, 3, 4, 5], [0, 0, 0]), ([0, 3, 4, 7], [0, 0, 0]),
    ([0, -1, 4, 6], [0, 0, 0]), ([0, 3, 4, 6], [-1, 0, 0]), ([0, 3, 4, 6], [0, 0, 41]),
    ([0, 3, 4, 6], [0, 2 ** 31 - 1, 0]), ([0, 3, 4, 6], [0, -2 ** 31, 0]), ([0, 2 ** 31 - 1, -2 ** 31, 6], [0, 0, 0])])
def test_bad_tables_write_nothing(moelib, cuda_dev, entry, off, tab):
    p = Pair(moelib, 3, 2, 64, 40, 16, "int8")
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = [torch.full((6, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    x = torch.ones(6, 2, 64, dtype=torch.bfloat16, device=DEV)
    if entry == "write":
        moelib.kv8_write(p.shape(6), x, x, _i32(off), _i32(tab), p.gpu, status=st)
    elif entry == "read":
        moelib.kv8_read(p.shape(6), p.gpu, _i32(off), _i32(tab), *out, status=st)
    else:
        ws = moelib.kv8_alloc_workspace(p.shape(6), DEV)
        moelib.kv8_attn(p.shape(6), x, p.gpu, _i32(off), _i32(tab), out[0], ws)
        st = ws[:4].view(torch.int32)
    assert moelib.status_read(st) == moelib.MOE_ERR_INVALID_ARG
    p.check()
    assert all((o == 7).all() for o in out)


# -------------------------------------------------------------- attention ---

ATTN = [  # Hq, Hkv, D, block, lens, news
    (16, 2, 256, 64, [1], [1]),
    (16, 2, 256, 64, [300], [1]),
    (16, 2, 256, 64, [63, 64, 65, 0, 1000], [1, 1, 1, 1, 1]),
    (8, 8, 128, 32, [77, 300], [1, 1]),
    (4, 1, 64, 16, [200, 5, 16, 17], [1, 1, 1, 1]),
    (6, 3, 256, 32, [513, 64, 9], [1, 0, 1]),
    (16, 2, 256, 64, [700, 90, 5], [3, 2, 5]),
    (16, 4, 128, 32, [333, 64, 700, 3], [4, 0, 1, 7]),       # more queries than positions: empty rows
    (64, 1, 128, 16, [150, 31], [1, 2]),                     # 64 query heads a KV head
    (20, 4, 64, 16, [260], [9]),                             # 5 query heads a KV head
    (16, 2, 256, 64, [130], [130]),                          # a whole prompt
    (16, 2, 256, 64, [400, 129, 33], [150, 129, 1]),         # chunks and a decode together
    (8, 8, 128, 16, [200], [200]),
    (4, 1, 64, 16, [600], [513]),
    (14, 2, 64, 32, [257], [200]),                           # 7 query heads a KV head
    (8, 1, 128, 64, [100, 40], [100, 60]),                   # 20 empty rows
    (3, 3, 64, 16, [40] * 40, [i % 3 for i in range(40)]),
    (2, 1, 64, 16, [1], [300]),                              # all rows but the last empty
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attention_matches_oracle(moelib, cuda_dev, case, fmt):
    Hq, Hkv, D, block, lens, news = ATTN[case]
    p = Pair(moelib, len(lens), Hkv, D, max(lens), block, fmt, seed=case)
    gen = p.fill(lens, seed=200 + case)
    p.check_attention(_rand(gen, sum(news), Hq, D).to(torch.bfloat16), news, lens)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("news", [1, 40])
@pytest.mark.parametrize("q_std,k_std,v_std", [(6.0, 1.0, 1.0), (1.0, 1e-3, 1e4), (2.0 ** 70, 2.0 ** -72, 1e-9),
                                               (2.0 ** -70, 2.0 ** 71, 2.0 ** 60), (0.0, 1.0, 1.0)])
def test_attention_at_other_magnitudes(moelib, cuda_dev, q_std, k_std, v_std, news, fmt):
    if k_std < 2.0 ** -60:
        k_std = 2.0 ** -45  # scales stay above their floor
        q_std = 2.0 ** 43
    p = Pair(moelib, 1, 2, 128, 500, 32, fmt)
    gen = p.fill([500], seed=17, k_std=k_std, v_std=v_std)
    p.check_attention((_rand(gen, news, 8, 128) * q_std).to(torch.bfloat16), [news], [500])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("news", [1, 70])
def test_attention_with_blocks_of_very_different_size(moelib, cuda_dev, news, fmt):
    """Scales that differ by up to 2^40 from block to block, and blocks of zeros."""
    p = Pair(moelib, 1, 2, 64, 400, 16, fmt)
    gen = torch.Generator().manual_seed(23)
    size = torch.exp2(torch.randint(-20, 20, (25, 1, 1, 1), generator=gen).float())
    x = (_rand(gen, 25, 16, 2, 64) * size)
    x[[3, 11, 24]] = 0
    x = x.view(400, 2, 64)
    k = _rand(gen, 400, 2, 64)
    k[64:80] = 0
    p.write([k.to(torch.bfloat16), x.to(torch.bfloat16)], [400], [0])
    p.check_attention(_rand(gen, news, 8, 64).to(torch.bfloat16), [news], [400])
    # values of zeros only
    z = torch.zeros(400, 2, 64, dtype=torch.bfloat16)
    p.write([k.to(torch.bfloat16), z], [400], [0])
    o = p.attend(_rand(gen, news, 8, 64).to(torch.bfloat16), [news], [400])
    assert (o == 0).all()


@pytest.mark.parametrize("news", [1, 50, 90])
def test_attention_of_queries_that_are_not_finite(moelib, cuda_dev, news):
    """A NaN or an infinity in one query row stays in that row."""
    p = Pair(moelib, 1, 2, 128, 300, 32, "int8")
    gen = p.fill([300], seed=29)
    q = _rand(gen, news, 4, 128).to(torch.bfloat16)
    good = p.attend(q, [news], [300]).cpu()
    q[0, 1, 7], q[0, 3, 9] = float("nan"), float("inf")
    got = p.attend(q, [news], [300]).cpu()
    bad = torch.zeros(news, 4, dtype=torch.bool)
    bad[0, 1] = bad[0, 3] = True
    assert got[bad].isnan().all() and torch.equal(got[~bad], good[~bad])


@pytest.mark.parametrize("fmt", FMTS)
def test_attention_explicit_scale_and_strided_queries(moelib, cuda_dev, fmt):
    p = Pair(moelib, 2, 2, 128, 300, 32, fmt)
    gen = p.fill([300, 111], seed=31)
    for news in ([1, 1], [4, 3], [90, 60]):
        T = sum(news)
        x = _rand(gen, T, 12 * 128).to(torch.bfloat16)
        q = x[:, 128:9 * 128].view(T, 8, 128)
        want, o_abs = kv8.attention(bits16(q), *p.codes, *p.scales, _packed(news), [300, 111], 32, fmt, 0.2)
        xg = x.to(DEV)
        got = p.attend(xg[:, 128:9 * 128].view(T, 8, 128), news, [300, 111], scale=0.2)
        p.compare(got.double().cpu().numpy(), want, o_abs, q, [300, 111], 0.2)


@pytest.mark.parametrize("fmt", FMTS)
def test_a_run_of_them_together(moelib, cuda_dev, fmt):
    """Serving: ragged prompts in, then chunks, then decode steps; every step
    writes its tokens and attends from them, and the context is read back."""
    B, Hq, Hkv, D, L, block = 3, 8, 2, 128, 240, 32
    p = Pair(moelib, B, Hkv, D, L, block, fmt)
    gen = torch.Generator().manual_seed(41)
    lens = [0] * B
    for news in ([70, 3, 150], [40, 0, 33], [1, 1, 1], [1, 1, 1], [4, 4, 4], [1, 0, 1]):
        T = sum(news)
        x = _rand(gen, T, (Hq + 2 * Hkv) * D).to(torch.bfloat16)
        q, k, v = (t.view(T, -1, D) for t in x.split([Hq * D, Hkv * D, Hkv * D], 1))
        p.write([k.contiguous(), v.contiguous()], news, lens)
        lens = [a + b for a, b in zip(lens, news)]
        p.check_attention(q.contiguous(), news, lens)
    p.check()
    p.read(lens, [0] * B)


@pytest.mark.parametrize("news", [1, 4, 80])
def test_attention_repeats_bit_for_bit_and_in_a_graph(moelib, cuda_dev, news):
    """The same bits from call to call, from another stream, and from a
    captured graph replayed on new data in the same buffers; two graphs share
    one workspace, replayed in turn on one stream."""
    p = Pair(moelib, 2, 2, 256, 3000, 64, "int8")
    gen = p.fill([3000, 1234], seed=43)
    q1, q2 = (_rand(gen, 2 * news, 16, 256).to(torch.bfloat16).to(DEV) for _ in range(2))
    counts, lens = [news, news], [3000, 1234]
    a1, a2 = p.attend(q1, counts, lens), p.attend(q2, counts, lens)
    assert torch.equal(a1, p.attend(q1, counts, lens))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sh = p.shape(2 * news, 16)
    ws, off, ln = moelib.kv8_alloc_workspace(sh, DEV), _i32(_packed(counts)), _i32(lens)
    q, outs, graphs = q1.clone(), [torch.empty_like(q1) for _ in range(2)], []
    torch.cuda.synchronize()
    moelib.kv8_attn(sh, q, p.gpu, off, ln, outs[0], ws, stream=s)
    s.synchronize()
    assert torch.equal(outs[0], a1)
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            moelib.kv8_attn(sh, q, p.gpu, off, ln, outs[i], ws)
        graphs.append(g)
    for want, data in ((a2, q2), (a1, q1)):
        q.copy_(data)
        for o in outs:
            o.zero_()
        for _ in range(3):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)


def test_write_and_read_in_a_graph(moelib, cuda_dev):
    p = Pair(moelib, 2, 2, 64, 50, 16, "int8")
    gen = torch.Generator().manual_seed(47)
    x = [_rand(gen, 6, 2, 64).to(torch.bfloat16) for _ in range(4)]
    k, v, off, st = x[0].to(DEV), x[1].to(DEV), _i32([0, 2, 6]), _i32([0, 0])
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    moelib.kv8_write(p.shape(6), k, v, off, st, p.gpu)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moelib.kv8_write(p.shape(6), k, v, off, st, p.gpu)
        moelib.kv8_read(p.shape(6), p.gpu, off, st, ko, vo)
    for i in range(2):
        kv8.write(bits16(x[i]), [0, 2, 6], [0, 0], p.codes[i], p.scales[i], 16, "int8")
    k.copy_(x[2]), v.copy_(x[3]), st.copy_(_i32([2, 4]))
    g.replay()
    for i in range(2):
        kv8.write(bits16(x[2 + i]), [0, 2, 6], [2, 4], p.codes[i], p.scales[i], 16, "int8")
    p.check()
    p.read([2, 4], [2, 4])


def test_no_tokens_is_a_no_op(moelib, cuda_dev):
    p = Pair(moelib, 2, 1, 64, 20, 16, "int8")
    e = torch.empty(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    off, tab = _i32([0, 0, 0]), _i32([3, 4])
    moelib.kv8_write(p.shape(0), e, e, off, tab, p.gpu)
    moelib.kv8_read(p.shape(0), p.gpu, off, tab, e, e)
    ws = torch.full((moelib.kv8_workspace_bytes(p.shape(0)),), 255, dtype=torch.uint8, device=DEV)
    moelib.kv8_attn(p.shape(0), e, p.gpu, off, tab, e, ws)
    assert moelib.status_read(ws[:4].view(torch.int32)) == 0
    p.check()


@pytest.mark.parametrize("news", [1, 33])
def test_attention_leaves_its_surroundings_alone(moelib, cuda_dev, news):
    """Rows around o and bytes past the workspace's stated size keep their
    values."""
    p = Pair(moelib, 1, 2, 256, 333, 64, "e4m3")
    gen = p.fill([333], seed=53)
    q = _rand(gen, news, 16, 256).to(torch.bfloat16)
    big = torch.full((news + 2, 16, 256), 3.0, dtype=torch.bfloat16, device=DEV)
    n = moelib.kv8_workspace_bytes(p.shape(news, 16))
    ws = torch.full((n + 4096,), 171, dtype=torch.uint8, device=DEV)
    p.attend(q, [news], [333], o=big[1:-1], ws=ws[:n])
    assert (big[0] == 3).all() and (big[-1] == 3).all() and (ws[n:] == 171).all()
    assert torch.equal(big[1:-1], p.attend(q, [news], [333]))


@pytest.mark.parametrize("fmt", FMTS)
def test_long_decode_against_the_oracle(moelib, cuda_dev, fmt):
    lens = [20000, 777]
    p = Pair(moelib, 2, 2, 256, 20000, 64, fmt)
    gen = p.fill(lens, seed=59)
    p.check_attention((_rand(gen, 2, 16, 256) * 2).to(torch.bfloat16), [1, 1], lens)


def test_cache_offsets_past_32_bits(moelib, cuda_dev):
    """A cache of more than 2^32 bytes per array: the last sequence's rows lie
    past every 32-bit offset."""
    B, Hkv, D, L, block = 9, 8, 128, 1 << 19, 64
    codes = [torch.empty(B, Hkv, L, D, dtype=torch.uint8, device=DEV) for _ in range(2)]
    assert codes[0].numel() > 1 << 32
    scales = [torch.zeros(B, Hkv, L // block, device=DEV) for _ in range(2)]
    big = moelib.Kv8Cache(*codes, *scales)
    small = Pair(moelib, 1, Hkv, D, 300, block, "int8")
    gen = small.fill([300], seed=61)
    x = [_rand(gen, 20, Hkv, D).to(torch.bfloat16) for _ in range(2)]
    start = L - 320
    for i in range(2):  # the last 300 positions before the new ones
        codes[i][8, :, start:start + 300] = torch.from_numpy(small.codes[i][0]).to(DEV)
        scales[i][8, :, start // block:start // block + 5] = torch.from_numpy(small.scales[i][0]).to(DEV)
    sh = moelib.kv8_shape(B, 20, 8, Hkv, D, L, block)
    off, st = _i32([0] * 9 + [20]), _i32([0] * 8 + [L - 20])
    moelib.kv8_write(sh, x[0].to(DEV), x[1].to(DEV), off, st, big)
    ko, vo = (torch.empty(20, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    moelib.kv8_read(sh, big, off, st, ko, vo)
    ref = Pair(moelib, 1, Hkv, D, 320, block, "int8")
    for i in range(2):
        ref.codes[i][:, :, :300], ref.scales[i][:] = small.codes[i], small.scales[i]
        kv8.write(bits16(x[i]), [0, 20], [300], ref.codes[i], ref.scales[i], block, "int8")
        want = torch.from_numpy(kv8.read([0, 20], [300], ref.codes[i], ref.scales[i], block, "int8")).float()
        assert torch.equal((ko, vo)[i].cpu(), want.to(torch.bfloat16))
    # every value before those 320 positions zero
    for i in range(2):
        codes[i][8, :, :start] = 128
    scales[0][8, :, :start // block] = 0
    q = torch.zeros(20, 8, D, dtype=torch.bfloat16)
    o = torch.empty(20, 8, D, dtype=torch.bfloat16, device=DEV)
    ws = moelib.kv8_alloc_workspace(sh, DEV)
    moelib.kv8_attn(sh, q.to(DEV), big, off, _i32([0] * 8 + [L]), o, ws)
    assert moelib.status_read(ws[:4].view(torch.int32)) == 0
    # q = 0: o is the mean of the visible values, those before the tail zero
    scale = ref.scales[1][0][:, np.arange(320) // block][:, :, None].astype(np.float64)
    V = kv8.value_of(ref.codes[1][0], scale, "int8")
    # the weights are equal and the sums of codes exact, so what is off is the
    # rounding of o and of the probabilities
    n = (start + 301 + np.arange(20))[:, None, None]
    want, o_abs = (np.stack([x[:, :301 + i].sum(1) for i in range(20)]) / n for x in (V, np.abs(V)))
    assert (np.abs(o.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.1 * 2.0 ** -11 * o_abs).all()


def _plain_attention_gpu(p, q, news, lens):
    """fp64 attention on the GPU from the oracle's arrays, for sizes the numpy
    oracle is too slow for. Returns o and the same sums over |V|."""
    B, Hkv, D, L = p.dims
    r = q.shape[1] // Hkv
    out, out_abs = [], []
    at = np.arange(L) // p.block
    off = _packed(news)
    for b, (n, ln) in enumerate(zip(news, lens)):
        K, V = (kv8.value_of(p.codes[i][b, :, :ln], p.scales[i][b][:, at[:ln]][:, :, None], p.fmt) for i in range(2))
        K, V = torch.from_numpy(K).to(DEV), torch.from_numpy(V).to(DEV)
        x = q[off[b]:off[b + 1]].to(DEV).double().view(n, Hkv, r, D)
        o, oa = (torch.zeros(n, Hkv, r, D, dtype=torch.float64, device=DEV) for _ in range(2))
        for g in range(Hkv):
            s = torch.einsum("nrd,jd->nrj", x[:, g], K[g]) * D ** -0.5
            hide = torch.arange(ln, device=DEV) > ln - n + torch.arange(n, device=DEV)[:, None]
            w = torch.softmax(s.masked_fill(hide[:, None], -torch.inf), -1)
            o[:, g], oa[:, g] = w @ V[g], w @ V[g].abs()
        out.append(o.view(n, Hkv * r, D)), out_abs.append(oa.view(n, Hkv * r, D))
    return torch.cat(out).cpu().numpy(), torch.cat(out_abs).cpu().numpy()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("Hq,Hkv,D,block,lens,news", [
    (16, 4, 128, 32, [700 + 491 * i for i in range(16)], [1 + i % 5 for i in range(16)]),
    (16, 2, 256, 64, [4000 - 333 * i for i in range(11)], [1 + i % 3 for i in range(11)]),
    (32, 2, 256, 64, [1500, 77, 3000], [1, 1, 1]),
    (12, 3, 64, 16, [3000 - 100 * i for i in range(24)], [i % 9 for i in range(24)]),
])
def test_attention_of_many_drafts(moelib, cuda_dev, Hq, Hkv, D, block, lens, news, fmt):
    """Several row tiles in every block's run, some of one unit, over long
    rings, against fp64, and the same bits every time."""
    p = Pair(moelib, len(lens), Hkv, D, max(lens), block, fmt, seed=73)
    gen = p.fill(lens, seed=74)
    q = (_rand(gen, sum(news), Hq, D) * 1.5).to(torch.bfloat16)
    got = p.attend(q, news, lens)
    want, o_abs = _plain_attention_gpu(p, q, news, lens)
    p.compare(got.double().cpu().numpy(), want, o_abs, q, lens)
    for _ in range(50):
        assert torch.equal(got, p.attend(q, news, lens))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("Hq,Hkv,D,block,lens,news", [
    (16, 2, 256, 64, [2500], [2500]),             # several tiles per run, of 1 to 20 units
    (16, 2, 256, 32, [7000, 900], [700, 900]),    # tiles longer than a run
    (16, 4, 128, 16, [3000, 2000], [1500, 2000]),
    (8, 2, 64, 64, [5000], [3000]),
    (10, 2, 64, 64, [2000, 1, 800], [1600, 1, 900]),
])
def test_attention_of_long_prompts(moelib, cuda_dev, Hq, Hkv, D, block, lens, news, fmt):
    """Runs of many units and tiles per block, against fp64, and the same bits
    every time."""
    p = Pair(moelib, len(lens), Hkv, D, max(lens), block, fmt, seed=71)
    gen = p.fill(lens, seed=72)
    q = (_rand(gen, sum(news), Hq, D) * 1.5).to(torch.bfloat16)
    got = p.attend(q, news, lens)
    seen = torch.cat([torch.arange(n) >= n - ln for n, ln in zip(news, lens)]).numpy()
    assert (got.cpu()[~seen] == 0).all()
    want, o_abs = _plain_attention_gpu(p, q, news, lens)
    want[~seen], o_abs[~seen] = 0, 0
    p.compare(got.double().cpu().numpy(), want, o_abs, q, lens)
    for _ in range(20):
        assert torch.equal(got, p.attend(q, news, lens))


@pytest.mark.parametrize("Hq,Hkv,D,lens,news,block", [
    (16, 2, 256, [20000], [1], 3),       # the split-context kernel
    (16, 2, 256, [3000], [600], 0),      # the tiles: the first block of a pair, which issues the products,
    (16, 2, 256, [3000], [600], 1),      # the second,
    (8, 2, 64, [3000], [900], 2),        # a block on its own
])
def test_timeout_is_reported_not_hung(moelib, cuda_dev, Hq, Hkv, D, lens, news, block):
    """One grid block never brings its operands: the waits run out after 20 ms,
    the call reports it, and the next one on the same workspace is as before."""
    p = Pair(moelib, 1, Hkv, D, max(lens), 64, "int8", seed=81)
    gen = p.fill(lens, seed=82)
    q = _rand(gen, sum(news), Hq, D).to(torch.bfloat16)
    want = p.attend(q, news, lens)
    sh = moelib.kv8_shape(1, sum(news), Hq, Hkv, D, max(lens), 64)
    ws, x, o = moelib.kv8_alloc_workspace(sh, DEV), q.to(DEV), torch.empty_like(want)
    off, ln = _i32(_packed(news)), _i32(lens)
    moelib.kv8_attn_test_stall(sh, x, p.gpu, off, ln, o, ws, block, 20_000_000)
    assert moelib.status_read(ws[:4].view(torch.int32)) == moelib.MOE_ERR_DEVICE_TIMEOUT
    moelib.kv8_attn(sh, x, p.gpu, off, ln, o, ws)
    assert moelib.status_read(ws[:4].view(torch.int32)) == moelib.MOE_OK
    assert torch.equal(o, want)


FIRST_CALL = """
import torch
import bit_grouped_expert_moe_gb300 as m
i32 = dict(dtype=torch.int32, device="cuda")
for n in (1, 200):
    sh = m.kv8_shape(1, n, 8, 2, 128, 256, 32)
    cache, off, st = m.kv8_alloc_cache(sh, "cuda"), torch.tensor([0, n], **i32), torch.zeros(1, **i32)
    x = torch.ones(n, 2, 128, dtype=torch.bfloat16, device="cuda")
    q, ws, ln = torch.zeros(n, 8, 128, dtype=torch.bfloat16, device="cuda"), m.kv8_alloc_workspace(sh, "cuda"), st + n
    o, y, z = torch.zeros_like(q), torch.zeros_like(x), torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.kv8_write(sh, x, x, off, st, cache)
        m.kv8_read(sh, cache, off, st, y, z)
        m.kv8_attn(sh, q, cache, off, ln, o, ws)
    g.replay()
    torch.cuda.synchronize()
    assert m.status_read(ws[:4].view(torch.int32)) == 0
    assert (y == 1).all() and (z == 1).all() and (o == 1).all()
"""


def test_first_calls_may_be_captured(moelib, cuda_dev):
    """In a process of its own, whose first calls are made during a capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
