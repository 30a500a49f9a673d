"""The paged KV cache on the GPU against the fp64 oracle.

Append: keys and queries as in tests/test_gpu_rope.py, values and everything
else in the pools bit for bit. Keep has no tolerance.

Attention, per element, from the arithmetic (u = 2^-24):
  * o is rounded to bf16: 2^-8 |o|;
  * every weight is rounded to bf16 for its product with V: 2^-8 sum_j w_j |v_j|
    (their sum takes them before that rounding);
  * a score is a sum of D products of up to `amp` in all, amp = scale sum_d |q_d| max |k|; each of the D + 8
    operations of its chain is off by at most 2 u of that, so the score by ds = (D + 8) 2 u amp, and the weights
    by a factor of up to e^(2 ds): 2.1 ds sum_j w_j |v_j| for the ds here (below 0.05);
  * the sum over positions runs in chains of at most L / 16 + 64 additions, each
    off by 2 u of at most the largest |v|.
"""
import math
import os
import random
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import paged
from oracle.moe import bf16_bits_to_f64
from tests._util import bits16
from tests.test_gpu_rope import check as check_rope, make_spec

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NAN = float("nan")


def _i32(v):
    return torch.tensor(np.asarray(v, dtype=np.int64).tolist(), dtype=torch.int32, device=DEV)


def _packed(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(int)


def _rand(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen) * std).to(torch.bfloat16)


def parents(rng, n, reach=6):
    return [-1] + [rng.randint(max(-1, i - reach), i - 1) for i in range(1, n)] if n else []


def words_of(par):
    out = []
    for i, p in enumerate(par):
        out.append((out[p] if p >= 0 else 0) | 1 << i)
    return out


def tree_tensor(words, W):
    a = np.array([[(w >> (64 * k)) & (2 ** 64 - 1) for k in range(W)] for w in words], dtype=np.uint64).reshape(len(words), W)
    return torch.from_numpy(a.view(np.int64)).to(DEV)


class Paged:
    """A cache whose every unused row, page and table entry is poison: NaN in the pages, pages far out of the pools
    in the table."""

    def __init__(self, m, lens, Hkv, D, page, seed=0, spare=2, max_pages=None, std=(1.0, 1.0)):
        self.m, self.Hkv, self.D, self.page, self.lens = m, Hkv, D, page, list(lens)
        gen = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lens]
        self.P = max_pages or max(max(need), 1)
        self.n = sum(need) + spare
        where, at = torch.randperm(self.n, generator=gen).tolist(), 0
        self.tables = np.full((len(lens), self.P), 1 << 30, dtype=np.int64)
        pools = [torch.full((self.n, Hkv, page, D), NAN, dtype=torch.bfloat16) for _ in range(2)]
        gain = torch.exp(0.5 * torch.randn(1, Hkv, 1, D, generator=gen))
        for b, k in enumerate(need):
            self.tables[b, :k] = where[at:at + k]
            for j in range(k):
                rows = min(page, lens[b] - j * page)
                x, y = _rand(gen, Hkv, rows, D, std=std[0]), _rand(gen, Hkv, rows, D, std=std[1])
                pools[0][where[at + j], :, :rows] = (x * gain[0]).to(torch.bfloat16)
                pools[1][where[at + j], :, :rows] = y
            at += k
        self.k, self.v = (bits16(x) for x in pools)
        self.gpu = m.PagedCache(*[x.to(DEV) for x in pools], _i32(self.tables))

    def shape(self, T, Hq, B=None, **kw):
        return self.m.paged_shape(B or len(self.lens), T, Hq, self.Hkv, self.D, self.page, self.n, self.P, **kw)

    def attend(self, q, news, lens=None, words=None, scale=None, o=None, ws=None, stream=None, expect=0):
        lens = self.lens if lens is None else lens
        T, Hq, D = q.shape
        q = q if q.is_cuda else q.to(DEV)
        W = 0 if words is None else max(1, -(-max(news) // 64))
        sh = self.shape(T, Hq, q_stride=0 if T < 2 else q.stride(0), tree_words=W)
        o = torch.full((T, Hq, D), NAN, dtype=torch.bfloat16, device=DEV) if o is None else o
        ws = self.m.paged_alloc_workspace(sh, DEV) if ws is None else ws
        self.m.paged_attn(sh, q, self.gpu, _i32(_packed(news)), _i32(lens), o, ws,
                          tree=None if words is None else tree_tensor(words, W), scale=scale, stream=stream)
        assert self.m.status_read(ws[:4].view(torch.int32)) == expect
        return o

    def exact(self, q, news, lens=None, words=None, scale=None):
        """fp64 on the GPU: o and the same sums over |V|."""
        lens = self.lens if lens is None else lens
        T, Hq, D = q.shape
        r = Hq // self.Hkv
        s = D ** -0.5 if scale is None else scale
        o, oa = torch.zeros(2, T, Hq, D, dtype=torch.float64, device=DEV)
        at = 0
        for b, (n, L) in enumerate(zip(news, lens)):
            if n and L:
                pages = torch.tensor(self.tables[b, :-(-L // self.page)], device=DEV)
                K, V = (x[pages].transpose(1, 2).reshape(-1, self.Hkv, D)[:L].double() for x in (self.gpu.k, self.gpu.v))
                i, j = torch.arange(n, device=DEV)[:, None], torch.arange(L, device=DEV)[None]
                see = j <= L - n + i
                if words is not None:
                    a = np.zeros((n, L), dtype=bool)
                    for t in range(n):
                        for d in range(max(0, n - L), n):
                            a[t, L - n + d] = words[at + t] >> d & 1
                    see = see & ((j < L - n) | torch.from_numpy(a).to(DEV))
                x = q[at:at + n].to(DEV).double().view(n, self.Hkv, r, D)
                for g in range(self.Hkv):
                    z = torch.einsum("nrd,jd->nrj", x[:, g], K[:, g]) * s
                    w = torch.softmax(z.masked_fill(~see[:, None], -torch.inf), -1).nan_to_num(0.0)
                    w = torch.where(see[:, None], w, 0.0)
                    o[at:at + n, g * r:(g + 1) * r] = w @ V[:, g]
                    oa[at:at + n, g * r:(g + 1) * r] = w @ V[:, g].abs()
            at += n
        return o.cpu().numpy(), oa.cpu().numpy()

    def compare(self, got, want, o_abs, q, scale=None, rows=None):
        D = q.shape[2]
        s = D ** -0.5 if scale is None else scale
        top = [np.nanmax(np.abs(np.where(np.isfinite(f), f, 0))) for f in (bf16_bits_to_f64(self.k), bf16_bits_to_f64(self.v))]
        u2 = 2.0 ** -23
        ds = (D + 8) * u2 * s * np.abs(bf16_bits_to_f64(bits16(q))).sum(2, keepdims=True) * top[0]
        assert ds.max(initial=0) < 0.05
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.1 * ds) * o_abs + (max(self.lens) / 16 + 64) * u2 * top[1]
        got = got.double().cpu().numpy()
        err = np.abs(got - want)
        if rows is not None:
            got, err, tol = got[rows], err[rows], tol[rows]
        assert np.isfinite(got).all(), np.argwhere(~np.isfinite(got))[:4]
        assert (err <= tol).all(), (float((err / np.maximum(tol, 1e-300)).max()), np.argwhere(err > tol)[:4])

    def check(self, q, news, lens=None, words=None, scale=None):
        got = self.attend(q, news, lens, words, scale)
        self.compare(got, *self.exact(q, news, lens, words, scale), q, scale)
        return got


# ---------------------------------------------------------------- append ---

@pytest.mark.parametrize("Hq,Hkv,D,page,starts,counts,rot,norm,positions", [
    (16, 2, 256, 64, [0], [1], 64, 3, False), (16, 2, 256, 64, [63, 64, 100], [1, 1, 1], 64, 3, False),
    (8, 8, 128, 16, [5, 0, 33, 16], [60, 0, 1, 47], 128, 0, True), (4, 1, 64, 256, [255, 0], [2, 300], 32, 2, False),
    (6, 3, 64, 32, [7 * i for i in range(70)], [i % 3 for i in range(70)], 64, 1, True),
    (5, 5, 128, 128, [1000], [700], 0, 3, False)])
@pytest.mark.parametrize("fused", [False, True])
def test_append_is_the_oracles(moelib, cuda_dev, Hq, Hkv, D, page, starts, counts, rot, norm, positions, fused):
    m = moelib
    lens = [s + n for s, n in zip(starts, counts)]
    p = Paged(m, lens, Hkv, D, page, seed=3)
    spec, oracle = make_spec(m, D, rot, page == 16, norm)
    gen = torch.Generator().manual_seed(4)
    T, off, w = sum(counts), _packed(counts), (Hq + 2 * Hkv) * D
    x = _rand(gen, T, w)
    y = x.to(DEV)
    cols = [slice(0, Hq * D), slice(Hq * D, (Hq + Hkv) * D), slice((Hq + Hkv) * D, w)]
    parts = [x[:, c].reshape(T, -1, D) for c in cols]
    ins = [y[:, c].view(T, -1, D) if fused else y[:, c].reshape(T, -1, D).contiguous() for c in cols]
    at = [s + i for s, n in zip(starts, counts) for i in range(n)]
    pos = [int(v) for v in torch.randint(0, 1 << 20, (T,), generator=gen)] if positions else at
    q_out = torch.full((T, Hq, D), NAN, dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    stride = w if fused and T > 1 else 0
    m.paged_append(p.shape(T, Hq, q_stride=stride, kv_stride=stride), spec, *ins, _i32(off), _i32(starts), p.gpu, q_out,
                   positions=_i32(pos) if positions else None, status=st)
    assert m.status_read(st) == 0
    check_rope(q_out, *oracle(parts[0], pos))
    # values, and every row that no new token took, bit for bit
    want_v, want_k = p.v.copy(), p.k.copy()
    paged.append(bits16(parts[2]), off, starts, want_v, p.tables, page)
    assert np.array_equal(bits16(p.gpu.v), want_v)
    marks = np.zeros(p.k.shape, dtype=np.uint16)
    paged.append(np.ones((T, Hkv, D), np.uint16), off, starts, marks, p.tables, page)
    got_k = bits16(p.gpu.k)
    assert np.array_equal(got_k[marks == 0], want_k[marks == 0])
    rows = np.stack([got_k[p.tables[b][q // page], :, q % page] for b, (s, n) in enumerate(zip(starts, counts))
                     for q in range(s, s + n)])
    check_rope(torch.from_numpy(bf16_bits_to_f64(rows)), *oracle(parts[1], pos, True))
    # without queries, and with keys as they are
    m.paged_append(p.shape(T, Hq, q_stride=stride, kv_stride=stride), None, None, *ins[1:], _i32(off), _i32(starts), p.gpu)
    paged.append(bits16(parts[1]), off, starts, want_k, p.tables, page)
    assert np.array_equal(bits16(p.gpu.k), want_k) and np.array_equal(bits16(p.gpu.v), want_v)


def test_append_of_tokens_with_bad_tables_writes_nothing_for_them(moelib, cuda_dev):
    """A page out of the pools, a start below zero, positions past the table, offsets that run backwards: reported, the
    tokens concerned are not written, the others are."""
    m = moelib
    good = dict(offsets=[0, 2, 4, 6], starts=[3, 0, 10], table=None)
    for kw, lost in [(dict(), []), (dict(table=(0, 0, 99)), [0, 1]), (dict(table=(0, 0, -1)), [0, 1]),
                     (dict(starts=[3, -1, 10]), [2, 3]), (dict(starts=[3, 0, 47]), [5]), (dict(starts=[3, 2 ** 31 - 1, 10]), [2, 3]),
                     (dict(offsets=[0, 2, 4, 5]), [5]), (dict(offsets=[1, 2, 4, 6]), [0])]:
        a = {**good, **kw}
        p = Paged(m, [48, 48, 48], 2, 64, 16, seed=5)
        if a["table"]:
            b, j, v = a["table"]
            p.gpu.tables[b, j] = v
        x = _rand(torch.Generator().manual_seed(6), 6, 2, 64)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        q, q_out = x.to(DEV), torch.full((6, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        m.paged_append(p.shape(6, 2), None, q, q, q, _i32(a["offsets"]), _i32(a["starts"]), p.gpu, q_out, status=st)
        assert m.status_read(st) == (m.MOE_ERR_INVALID_ARG if lost else 0), kw
        kept = [t for t in range(6) if t not in lost]
        assert torch.equal(q_out.cpu()[kept], x[kept]) and (q_out.cpu()[lost] == 7).all(), kw
        want, changed = p.k.copy(), p.v.copy()
        for t in kept:
            b = max(i for i in range(3) if a["offsets"][i] <= t)
            pos = a["starts"][b] + t - a["offsets"][b]
            want[p.tables[b][pos // 16], :, pos % 16] = changed[p.tables[b][pos // 16], :, pos % 16] = bits16(x)[t]
        assert np.array_equal(bits16(p.gpu.k), want) and np.array_equal(bits16(p.gpu.v), changed), kw


# ------------------------------------------------------------- attention ---

@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("Hq,Hkv,D,lens,news", [
    (16, 2, 256, [1], [1]), (16, 2, 256, [300], [1]), (16, 2, 256, [128, 129, 127, 0, 1], [1, 1, 1, 0, 1]),
    (8, 8, 128, [200, 1, 513], [1, 1, 1]), (64, 1, 64, [333], [1]), (6, 3, 64, [50, 700], [3, 5]),
    (5, 5, 128, [260, 300], [130, 20]), (16, 4, 128, [129, 70, 3], [129, 33, 3]), (16, 2, 256, [400, 33], [100, 33]),
    (3, 1, 256, [600], [90]), (64, 1, 128, [100], [9])])
def test_causal_attention_is_the_oracles(moelib, cuda_dev, Hq, Hkv, D, lens, news, page):
    p = Paged(moelib, lens, Hkv, D, page, seed=11)
    q = _rand(torch.Generator().manual_seed(12), sum(news), Hq, D, std=1.5)
    got = p.check(q, news)
    small = [b for b, (n, ln) in enumerate(zip(news, lens)) if n * ln < 4000]
    if len(small) == len(lens):  # the numpy statement, too
        want, o_abs = paged.attention(bits16(q), p.k, p.v, p.tables, page, _packed(news), lens)
        p.compare(got, want, o_abs, q)


@pytest.mark.parametrize("Hq,Hkv,D,page,lens,news", [
    (16, 2, 256, 64, [1], [1]), (16, 2, 256, 64, [300, 64, 65], [20, 64, 63]), (8, 8, 128, 16, [90, 500, 3], [65, 7, 3]),
    (16, 4, 128, 32, [700, 1300], [40, 0]), (4, 1, 64, 128, [600, 200, 129], [500, 200, 128]),
    (16, 2, 256, 32, [2000], [200]), (6, 3, 64, 16, [333] * 5, [1, 2, 64, 65, 129]), (64, 1, 128, 256, [512], [512])])
def test_attention_of_trees_is_the_oracles(moelib, cuda_dev, Hq, Hkv, D, page, lens, news):
    rng = random.Random(13)
    p = Paged(moelib, lens, Hkv, D, page, seed=14)
    words = [w for n in news for w in words_of(parents(rng, n))]
    q = _rand(torch.Generator().manual_seed(15), sum(news), Hq, D, std=1.5)
    got = p.check(q, news, words=words)
    if sum(n * ln for n, ln in zip(news, lens)) < 9000:
        want, o_abs = paged.attention(bits16(q), p.k, p.v, p.tables, page, _packed(news), lens, words)
        p.compare(got, want, o_abs, q)
    # bits of later drafts, and past the sequence's own, count for nothing
    loud = [w | -(2 << i) & (1 << 64 * max(1, -(-max(news) // 64))) - 1 for n, s in zip(news, _packed(news))
            for i, w in enumerate(words[s:s + n])]
    assert torch.equal(got, p.attend(q, news, words=loud))
    # a chain is causal attention (in another order of nothing: the same units, the same bits)
    chain = [(2 << i) - 1 for n in news for i in range(n)]
    assert torch.equal(p.attend(q, news, words=chain), p.attend(q, news))


@pytest.mark.parametrize("D,r,news,lens", [(256, 8, [5, 40], [3, 40]), (64, 4, [70, 9], [200, 0]), (128, 1, [300], [50]),
                                           (128, 2, [130, 1], [130, 1])])
def test_rows_that_see_nothing_are_zero(moelib, cuda_dev, D, r, news, lens):
    """More queries than positions, and drafts without a bit over no context."""
    p = Paged(moelib, lens, 2, D, 16, seed=16)
    q = _rand(torch.Generator().manual_seed(17), sum(news), 2 * r, D)
    got = p.check(q, news).cpu()
    at = 0
    for n, ln in zip(news, lens):
        assert (got[at:at + max(0, n - ln)] == 0).all()
        at += n
    rng = random.Random(18)
    words = [0 if rng.random() < 0.3 else w & rng.getrandbits(512) for n in news for w in words_of(parents(rng, n))]
    got = p.check(q, news, words=words).cpu()
    at = 0
    for n, ln in zip(news, lens):
        for i in range(n):
            if n >= ln and (words[at + i] & ((2 << i) - 1)) >> (n - ln) == 0:
                assert (got[at + i] == 0).all()
        at += n


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,page,L,n", [(16, 2, 256, 64, 700, 300), (16, 2, 256, 16, 300, 10), (8, 8, 128, 32, 400, 200),
                                               (8, 4, 128, 32, 1000, 500), (4, 1, 64, 128, 260, 250)])
def test_what_a_query_does_not_see_has_no_part_in_it(moelib, cuda_dev, Hq, Hkv, D, page, L, n, tree):
    """Keys and values of new tokens that are NaN or infinite leave every row that does not see them as it was, bit
    for bit, and make every row that does not finite."""
    rng = random.Random(19)
    p = Paged(moelib, [L, 90], Hkv, D, page, seed=20)
    news = [n, 1]
    words = [w for k in news for w in words_of(parents(rng, k))] if tree else None
    q = _rand(torch.Generator().manual_seed(21), n + 1, Hq, D)
    before = p.attend(q, news, words=words).cpu()
    bad = sorted(rng.sample(range(n), 3)) + [n - 1]
    see = paged.visible(n, L, words[:n] if tree else None)
    for pool, value in ((1, NAN), (1, float("inf")), (0, NAN)):
        x = (p.gpu.k, p.gpu.v)[pool]
        old = x.clone()
        for i, d in enumerate(bad):
            pos = L - n + d
            x[int(p.tables[0][pos // page]), i % Hkv, pos % page, (37 * i) % D] = value if i % 2 else -value
        after = p.attend(q, news, words=words).cpu()
        x.copy_(old)
        r = Hq // Hkv
        for g in range(Hkv):
            hit = np.zeros(n + 1, dtype=bool)
            for i, d in enumerate(bad):
                if i % Hkv == g:
                    hit[:n] |= see[:, L - n + d]
            a, b = after[:, g * r:(g + 1) * r], before[:, g * r:(g + 1) * r]
            assert torch.equal(a[~hit], b[~hit])
            assert (~torch.isfinite(a[hit].float())).any(-1).all()


@pytest.mark.parametrize("news", [1, 100])
def test_a_value_that_every_row_sees_and_is_not_finite(moelib, cuda_dev, news):
    p = Paged(moelib, [900], 2, 256, 64, seed=22)
    q = _rand(torch.Generator().manual_seed(23), news, 16, 256)
    before = p.attend(q, [news]).cpu()
    p.gpu.v[int(p.tables[0][3]), 1, 5, 77] = float("inf")
    after = p.attend(q, [news]).cpu()
    assert torch.equal(after[:, :8], before[:, :8])
    assert (~torch.isfinite(after[:, 8:, 77].float())).all()


@pytest.mark.parametrize("scale,std", [(100.0, 30.0), (1e5, 100.0), (1e-30, 1.0)])
@pytest.mark.parametrize("D,L,n", [(256, 900, 1), (128, 700, 300), (64, 500, 40)])
def test_scores_of_any_size(moelib, cuda_dev, D, L, n, scale, std):
    """Scores so far apart that one position takes a row whole (o is its value), or so small that all weigh the same."""
    p = Paged(moelib, [L], 2, D, 32, seed=24)
    q = _rand(torch.Generator().manual_seed(25), n, 4, D, std=std)
    got = p.attend(q, [n], scale=scale)
    want, o_abs = p.exact(q, [n], scale=scale)
    K = bf16_bits_to_f64(paged.rows_of(p.k, p.tables[0], L, 32))
    V = bf16_bits_to_f64(paged.rows_of(p.v, p.tables[0], L, 32))
    qs, got = bf16_bits_to_f64(bits16(q)), got.double().cpu().numpy()
    assert np.isfinite(got).all()
    for t in range(0, n, 7):
        for h in range(4):
            z = scale * (K[h // 2][:L - n + t + 1] @ qs[t, h])
            # scores are off by ds at most: positions further than that below the largest stay below it
            ds = (D + 8) * 2.0 ** -23 * scale * np.abs(qs[t, h]) @ np.abs(K[h // 2]).max(0)
            near = np.flatnonzero(z >= z.max() - 2 * ds - 40.0)
            if scale < 1:
                tol = 2.0 ** -8 * np.abs(want[t, h]) + (2.0 ** -8 + 1e-5) * o_abs[t, h] + 1e-4
                assert (np.abs(got[t, h] - want[t, h]) <= tol).all()
            elif len(near) == 1:
                assert (np.abs(got[t, h] - V[h // 2][near[0]]) <= 2.0 ** -7 * np.abs(V[h // 2][near[0]]) + 1e-15).all()
            else:
                lo, hi = V[h // 2][near].min(0), V[h // 2][near].max(0)
                slack = 2.0 ** -7 * np.maximum(np.abs(lo), np.abs(hi)) + 1e-12
                assert (got[t, h] >= lo - slack).all() and (got[t, h] <= hi + slack).all()


@pytest.mark.parametrize("D,L,n,r", [(256, 777, 1, 16), (256, 600, 100, 8), (128, 700, 1, 16), (128, 500, 90, 4), (64, 900, 1, 16), (64, 700, 200, 2)])
def test_a_position_that_has_most_of_a_row(moelib, cuda_dev, D, L, n, r):
    """Scores that one position leads by much. Weights are off by 2^-8 of each at most; in calls of few rows (n r <= 16
    here) the largest is 1, and exact."""
    p = Paged(moelib, [L], 2, D, 32, seed=71)
    rng = np.random.default_rng(72)
    K = bf16_bits_to_f64(paged.rows_of(p.k, p.tables[0], L, 32))
    V = bf16_bits_to_f64(paged.rows_of(p.v, p.tables[0], L, 32))
    to = rng.integers(0, L - n + 1, size=(n, 2 * r))
    q = np.empty((n, 2 * r, D))
    for h in range(2 * r):
        k = K[h // r][to[:, h]]
        # the score of `to` some 9 to 14 above 0
        q[:, h] = k * (rng.uniform(9.0, 14.0, size=n) * math.sqrt(D) / (k * k).sum(1))[:, None]
    q = torch.from_numpy(q).to(torch.bfloat16)
    got, qs = p.attend(q, [n]).double().cpu().numpy(), bf16_bits_to_f64(bits16(q))
    for t in range(n):
        for h in range(2 * r):
            k, v = K[h // r][:L - n + t + 1], V[h // r][:L - n + t + 1]
            z = k @ qs[t, h] / math.sqrt(D)
            w = np.exp(z - z.max())
            w /= w.sum()
            o, m, all_of = w @ v, int(z.argmax()), w @ np.abs(v)
            rounded = all_of - w[m] * np.abs(v[m]) if n * r <= 16 else all_of
            # (1.01: second order; 1e-4: fp32's errors of scores up to 14, and of their sums)
            tol = 2.0 ** -8 * 1.01 * (np.abs(o) + rounded) + 1e-4 * all_of
            assert (np.abs(got[t, h] - o) <= tol).all(), (t, h, w[m], float((np.abs(got[t, h] - o) / tol).max()))


@pytest.mark.parametrize("Hq,Hkv,D,page,lens,news,tree", [
    (16, 2, 256, 64, [20000, 777], [1, 1], False), (16, 4, 128, 16, [700 + 491 * i for i in range(16)], [1 + i % 5 for i in range(16)], False),
    (16, 2, 256, 64, [4000 - 333 * i for i in range(11)], [1 + 7 * i % 30 for i in range(11)], True),
    (12, 3, 64, 16, [3000 - 100 * i for i in range(24)], [i % 9 for i in range(24)], True),
    (16, 2, 256, 64, [2500], [2500], False), (16, 2, 256, 32, [7000, 900], [700, 900], False),
    (16, 4, 128, 16, [3000, 2000], [1500, 2000], False), (8, 2, 64, 64, [5000], [3000], False),
    (10, 2, 64, 64, [2000, 1, 800], [1600, 1, 900], False), (16, 2, 256, 128, [9000, 5000], [200, 300], True),
    (8, 8, 128, 256, [3000] * 40, [1] * 40, False)])
def test_long_runs_and_many_tiles_the_same_every_time(moelib, cuda_dev, Hq, Hkv, D, page, lens, news, tree):
    """Runs of many units and tiles, over long rings, against fp64, and the same bits every time."""
    rng = random.Random(26)
    p = Paged(moelib, lens, Hkv, D, page, seed=27)
    words = [w for n in news for w in words_of(parents(rng, n, 12))] if tree else None
    q = _rand(torch.Generator().manual_seed(28), sum(news), Hq, D, std=1.5)
    got = p.check(q, news, words=words)
    for _ in range(20):
        assert torch.equal(got, p.attend(q, news, words=words))


@pytest.mark.parametrize("Hq,Hkv,D,lens,news,tree", [
    (4, 2, 64, [1 + 7 * i % 200 for i in range(300)], [i % 2 for i in range(300)], False),      # more sequences than tables
    (4, 2, 64, [1 + 7 * i % 200 for i in range(256)], [1] * 256, False),                        # the most that they hold
    (16, 2, 256, [100 + 3 * i for i in range(70)], [1 + i % 40 for i in range(70)], True),       # of one and several tiles
    (6, 2, 128, [90 * (i % 5) for i in range(33)], [60 * (i % 4) for i in range(33)], False),
    (64, 1, 64, [4500], [4200], False),                                                          # more tiles than are counted
    (1, 1, 128, [900, 3, 400], [900, 1, 399], False)])
def test_every_search_for_a_runs_start(moelib, cuda_dev, Hq, Hkv, D, lens, news, tree):
    rng = random.Random(64)
    p = Paged(moelib, lens, Hkv, D, 32, seed=65)
    words = [w for n in news for w in words_of(parents(rng, n))] if tree else None
    q = _rand(torch.Generator().manual_seed(66), sum(news), Hq, D)
    p.check(q, news, words=words)


def test_a_run_of_random_calls(moelib, cuda_dev):
    rng = random.Random(29)
    for i in range(40):
        Hkv, r, D = rng.choice([1, 2, 5]), rng.choice([1, 3, 8, 17]), rng.choice([64, 128, 256])
        B, page = rng.randint(1, 6), rng.choice([16, 32, 64, 128, 256])
        lens = [rng.choice([0, 1, 127, 128, 129, rng.randint(1, 1500)]) for _ in range(B)]
        tree = rng.random() < 0.5
        news = [min(n, rng.choice([0, 1, 2, rng.randint(0, 200)])) for n in lens]
        if sum(news) == 0:
            lens[0], news[0] = max(lens[0], 1), 1
        p = Paged(moelib, lens, Hkv, D, page, seed=i)
        words = [w for n in news for w in words_of(parents(rng, n))] if tree else None
        q = _rand(torch.Generator().manual_seed(i), sum(news), Hkv * r, D, std=rng.choice([0.1, 1.0, 2.0]))
        p.check(q, news, words=words)


def test_strided_queries_and_surroundings(moelib, cuda_dev):
    """q as columns of a projection; rows around o and bytes past the workspace's stated size keep their values."""
    p = Paged(moelib, [333, 50], 2, 128, 64, seed=30)
    gen = torch.Generator().manual_seed(31)
    for news in ([1, 1], [150, 40]):
        T = sum(news)
        x = _rand(gen, T, 12 * 128).to(DEV)
        q = x[:, 256:256 + 8 * 128].view(T, 8, 128)
        big = torch.full((T + 2, 8, 128), 3.0, dtype=torch.bfloat16, device=DEV)
        n = moelib.paged_workspace_bytes(p.shape(T, 8))
        ws = torch.full((n + 4096,), 171, dtype=torch.uint8, device=DEV)
        p.attend(q, news, o=big[1:-1], ws=ws[:n])
        assert (big[0] == 3).all() and (big[-1] == 3).all() and (ws[n:] == 171).all()
        assert torch.equal(big[1:-1], p.attend(q.contiguous(), news))


def test_sequences_may_share_pages(moelib, cuda_dev):
    """Two sequences with the same first pages, as with a common prompt."""
    p = Paged(moelib, [300, 300], 2, 128, 64, seed=32)
    p.tables[1, :3] = p.tables[0, :3]
    p.gpu.tables.copy_(_i32(p.tables))
    q = _rand(torch.Generator().manual_seed(33), 40, 4, 128)
    p.check(q, [39, 1])


def test_bad_tables_are_reported(moelib, cuda_dev):
    """Offsets, lengths, drafts past the words' bits: nothing is written. A page out of the pools: reported, read as
    nothing, and the other sequence's rows are right."""
    m = moelib
    p = Paged(m, [300, 200], 2, 128, 64, seed=34)
    q = _rand(torch.Generator().manual_seed(35), 80, 4, 128).to(DEV)
    sh, ws = p.shape(80, 4), m.paged_alloc_workspace(p.shape(80, 4), DEV)
    limit = p.P * 64
    for off, lens in [([0, 40, 79], [300, 200]), ([1, 40, 80], [300, 200]), ([0, 81, 80], [300, 200]), ([0, -1, 80], [300, 200]),
                      ([0, 40, 80], [-1, 200]), ([0, 40, 80], [300, limit + 1])]:
        o = torch.full((80, 4, 128), 5.0, dtype=torch.bfloat16, device=DEV)
        m.paged_attn(sh, q, p.gpu, _i32(off), _i32(lens), o, ws)
        assert m.status_read(ws[:4].view(torch.int32)) == m.MOE_ERR_INVALID_ARG and (o == 5).all()
    tree = tree_tensor([1] * 80, 1)
    o = torch.full((80, 4, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    m.paged_attn(p.shape(80, 4, tree_words=1), q, p.gpu, _i32([0, 65, 80]), _i32([300, 200]), o, ws, tree=tree)
    assert m.status_read(ws[:4].view(torch.int32)) == m.MOE_ERR_INVALID_ARG and (o == 5).all()
    for news in ([1, 1], [40, 40]):
        T = sum(news)
        good = p.attend(q[:T], news)
        for bad in (-1, p.n, 2 ** 31 - 1, -2 ** 31):
            old = p.gpu.tables[0, 1].clone()
            p.gpu.tables[0, 1] = bad
            o = torch.empty(T, 4, 128, dtype=torch.bfloat16, device=DEV)
            m.paged_attn(p.shape(T, 4), q[:T], p.gpu, _i32(_packed(news)), _i32(p.lens), o, ws)
            assert m.status_read(ws[:4].view(torch.int32)) == m.MOE_ERR_INVALID_ARG
            p.gpu.tables[0, 1] = old
        assert torch.equal(good, p.attend(q[:T], news, ws=ws))


@pytest.mark.parametrize("Hq,Hkv,D,lens,news,block", [
    (16, 2, 256, [20000], [1], 3),   # a block on its own
    (16, 2, 256, [3000], [600], 0),  # the first block of a pair, which issues the products,
    (16, 2, 256, [3000], [600], 1),  # the second
    (16, 4, 128, [20000], [1], 3), (16, 4, 128, [3000], [600], 0), (16, 4, 128, [3000], [600], 1),
    (8, 2, 64, [3000], [900], 2)])
def test_timeout_is_reported_not_hung(moelib, cuda_dev, Hq, Hkv, D, lens, news, block):
    """One grid block never brings its keys: the waits run out after 20 ms, the call reports it, and the next one on
    the same workspace is as before."""
    m, p = moelib, Paged(moelib, lens, Hkv, D, 64, seed=36)
    q = _rand(torch.Generator().manual_seed(37), sum(news), Hq, D).to(DEV)
    want = p.attend(q, news)
    sh = p.shape(sum(news), Hq)
    ws, o, off, ln = m.paged_alloc_workspace(sh, DEV), torch.empty_like(want), _i32(_packed(news)), _i32(lens)
    m.paged_attn_test_stall(sh, q, p.gpu, off, ln, o, ws, block, 20_000_000)
    assert m.status_read(ws[:4].view(torch.int32)) == m.MOE_ERR_DEVICE_TIMEOUT
    m.paged_attn(sh, q, p.gpu, off, ln, o, ws)
    assert m.status_read(ws[:4].view(torch.int32)) == m.MOE_OK
    assert torch.equal(o, want)


def test_cache_offsets_past_32_bits(moelib, cuda_dev):
    """Pools of more than 2^32 values: the last pages lie past every 32-bit offset."""
    m, Hkv, D, page = moelib, 2, 256, 64
    n = (1 << 32) // (Hkv * D * page) + 8
    k, v = (torch.empty(n, Hkv, page, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    assert k.numel() > 1 << 32
    table = [n - 1, 0, n - 3, n - 2]
    cache = m.PagedCache(k, v, _i32([table]))
    small = Paged(m, [250], Hkv, D, page, seed=38)
    gen = torch.Generator().manual_seed(39)
    rows = [_rand(gen, 250, Hkv, D) for _ in range(2)]
    sh = m.paged_shape(1, 250, 16, Hkv, D, page, n, 4)
    off, st = _i32([0, 250]), _i32([0])
    m.paged_append(sh, None, None, rows[0].to(DEV), rows[1].to(DEV), off, st, cache)
    m.paged_append(small.shape(250, 16), None, None, rows[0].to(DEV), rows[1].to(DEV), off, st, small.gpu)
    for j, pg in enumerate(table):
        c = min(page, 250 - j * page)
        for a, b in ((k, small.gpu.k), (v, small.gpu.v)):
            assert torch.equal(a[pg, :, :c], b[int(small.tables[0][j]), :, :c])
    for T in (1, 40):
        q = _rand(gen, T, 16, D)
        o, ws = torch.empty(T, 16, D, dtype=torch.bfloat16, device=DEV), m.paged_alloc_workspace(sh, DEV)
        m.paged_attn(m.paged_shape(1, T, 16, Hkv, D, page, n, 4), q.to(DEV), cache, _i32([0, T]), _i32([250]), o, ws)
        assert m.status_read(ws[:4].view(torch.int32)) == 0
        assert torch.equal(o, small.attend(q, [T]))
    keep = (_i32([200]), _i32([3]), _i32([[1, 5, 40]]))
    m.paged_keep(sh, cache, *keep)
    m.paged_keep(small.shape(0, 16), small.gpu, *keep)
    assert torch.equal(k[n - 2, :, :58], small.gpu.k[int(small.tables[0][3]), :, :58])


# ------------------------------------------------------------------ keep ---

@pytest.mark.parametrize("Hkv,D,page", [(2, 256, 64), (1, 64, 16), (8, 128, 32), (5, 64, 256)])
def test_keep_is_the_oracles(moelib, cuda_dev, Hkv, D, page):
    m, rng = moelib, random.Random(40)
    lens = [600, 64, 700, 100, 512, 530]
    p = Paged(m, lens, Hkv, D, page, seed=41)
    news = [300, 64, 40, 1, 512, 530]
    kept = [200, 0, 39, 1, 512, 17]
    starts = [n - k for n, k in zip(lens, news)]
    path = [sorted(rng.sample(range(n), k)) for n, k in zip(news, kept)]
    width = 512
    arr = np.full((6, width), -7)
    for b, q in enumerate(path):
        arr[b, :len(q)] = q
    out, st = torch.empty(6, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    m.paged_keep(p.shape(0, Hkv), p.gpu, _i32(starts), _i32(kept), _i32(arr), lens_out=out, status=st)
    assert m.status_read(st) == 0 and out.tolist() == [s + k for s, k in zip(starts, kept)]
    for bits, gpu in ((p.k, p.gpu.k), (p.v, p.gpu.v)):
        paged.keep(bits, p.tables, page, starts, path, kept)
        assert np.array_equal(bits16(gpu), bits)
    m.paged_keep(p.shape(0, Hkv), p.gpu, _i32(starts), _i32([0] * 6), _i32(arr[:, :0].reshape(6, 0)))  # nothing to keep
    assert np.array_equal(bits16(p.gpu.v), p.v)


def test_keep_leaves_sequences_with_bad_entries_alone(moelib, cuda_dev):
    m = moelib
    good = dict(starts=[10, 20], kept=[2, 3], path=[[1, 4, 0], [0, 2, 7]], page=None)
    for kw in (dict(starts=[-1, 20]), dict(kept=[-1, 3]), dict(kept=[4, 3]), dict(path=[[1, 1, 0], [0, 2, 7]]),
               dict(path=[[4, 1, 0], [0, 2, 7]]), dict(path=[[-1, 1, 0], [0, 2, 7]]), dict(path=[[1, 2 ** 31 - 1, 0], [0, 2, 7]]),
               dict(starts=[2 ** 31 - 1, 20]), dict(path=[[1, 100, 0], [0, 2, 7]]), dict(page=99), dict(page=-1)):
        a = {**good, **kw}
        p = Paged(m, [32, 32], 2, 64, 16, seed=42)
        if a["page"] is not None:
            p.gpu.tables[0, 0] = a["page"]
        out, st = _i32([-5, -5]), torch.zeros(1, dtype=torch.int32, device=DEV)
        m.paged_keep(p.shape(0, 2), p.gpu, _i32(a["starts"]), _i32(a["kept"]), _i32(a["path"]), lens_out=out, status=st)
        assert m.status_read(st) == m.MOE_ERR_INVALID_ARG and out.tolist() == [-5, 23], kw
        for bits, gpu in ((p.k, p.gpu.k), (p.v, p.gpu.v)):
            paged.keep(bits, p.tables, 16, [10, 20], [[], [0, 2, 7]], [0, 3])
            assert np.array_equal(bits16(gpu), bits), kw


# ---------------------------------------------------- a run of them together ---

def _serve(m, mode, steps=4, fast=False):
    """Prompts, then steps that each draft a tree, verify it and keep a path: everything on the device. Returns the
    outputs and the rows held in the end."""
    rng, gen = random.Random(50), torch.Generator(device=DEV).manual_seed(51)
    B, Hq, Hkv, D, page, n = 3, 8, 2, 128, 32, 24
    prompt = [70, 1, 130]
    P = -(-(max(prompt) + steps * n + n) // page)
    n_pages = B * P
    i32 = dict(dtype=torch.int32, device=DEV)
    table = m.rope_table(64, 1e6, device=DEV)
    g = [torch.randn(D, generator=gen, device=DEV).to(torch.bfloat16) for _ in range(2)]
    spec = m.rope_spec(table, norm=m.ROPE_NORM_QK, q_gain=g[0], k_gain=g[1])
    pages = [torch.zeros(n_pages, Hkv, page, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    tables = torch.tensor(rng.sample(range(n_pages), n_pages), **i32).view(B, P)
    cache = m.PagedCache(*pages, tables)

    def tokens(T):
        x = torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen, device=DEV).to(torch.bfloat16)
        return x

    T0, T1, w = sum(prompt), B * n, (Hq + 2 * Hkv) * D
    sh0 = m.paged_shape(B, T0, Hq, Hkv, D, page, n_pages, P, q_stride=w, kv_stride=w)
    sh1 = m.paged_shape(B, T1, Hq, Hkv, D, page, n_pages, P, tree_words=1, q_stride=w, kv_stride=w)
    at1 = m.paged_shape(B, T1, Hq, Hkv, D, page, n_pages, P, tree_words=1)
    at0 = m.paged_shape(B, T0, Hq, Hkv, D, page, n_pages, P)
    ws = m.paged_alloc_workspace(at1, DEV)
    off0, off1 = torch.tensor(_packed(prompt).tolist(), **i32), torch.tensor(_packed([n] * B).tolist(), **i32)
    x0 = tokens(T0)
    xs = [tokens(T1) for _ in range(steps)]
    trees, depths, paths, kepts = [], [], [], []
    for _ in range(steps):
        ws_, ds, ps, ks = [], [], [], []
        for b in range(B):
            par = parents(rng, n, 5)
            wd = words_of(par)
            ds += [bin(v).count("1") - 1 for v in wd]
            ws_ += wd
            leaf = rng.randrange(n)
            ps.append([i for i in range(n) if wd[leaf] >> i & 1])
            ks.append(len(ps[-1]))
        trees.append(tree_tensor(ws_, 1)), depths.append(torch.tensor(ds, **i32)), kepts.append(torch.tensor(ks, **i32))
        paths.append(torch.tensor([p + [0] * (n - len(p)) for p in ps], **i32))
    seq = torch.arange(B, device=DEV).repeat_interleave(n)
    starts, lens, kept, pos = (torch.zeros(k, **i32) for k in (B, B, B, T1))
    zero, prompt_t = torch.zeros(B, **i32), torch.tensor(prompt, **i32)
    x, q0, q1 = torch.zeros_like(xs[0]), torch.empty(T0, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(T1, Hq, D, dtype=torch.bfloat16, device=DEV)
    tree, path = torch.zeros_like(trees[0]), torch.zeros_like(paths[0])
    o0, o1 = torch.empty_like(q0), torch.empty(steps, *q1.shape, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, **i32)
    pause = torch.cuda.synchronize if mode == "sync" else lambda: None

    def split(y, T):
        return y[:, :Hq * D].view(T, Hq, D), y[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D), y[:, (Hq + Hkv) * D:].view(T, Hkv, D)

    def go():
        m.paged_append(sh0, spec, *split(x0, T0), off0, zero, cache, q0, status=status)
        pause()
        m.paged_attn(at0, q0, cache, off0, prompt_t, o0, ws)
        pause()
        starts.copy_(prompt_t)
        for i in range(steps):
            x.copy_(xs[i]), tree.copy_(trees[i]), path.copy_(paths[i]), kept.copy_(kepts[i])
            torch.add(starts, n, out=lens)
            torch.add(starts[seq], depths[i], out=pos)
            pause()
            m.paged_append(sh1, spec, *split(x, T1), off1, starts, cache, q1, positions=pos, status=status)
            pause()
            m.paged_attn(at1, q1, cache, off1, lens, o1[i], ws, tree=tree)
            pause()
            m.paged_keep(at1, cache, starts, kept, path, lens_out=lens, status=status)
            pause()
            starts.copy_(lens)
            pause()

    if mode == "graph":
        go()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            go()
        o0.zero_(), o1.zero_()
        for t in pages:
            t.zero_()
        graph.replay()
    else:
        if mode == "queue":
            torch.cuda.synchronize()
            torch.cuda._sleep(20_000_000)  # the host gets ahead
        go()
    torch.cuda.synchronize()
    assert m.status_read(ws[:4].view(torch.int32)) == 0 and m.status_read(status) == 0
    ends = starts.tolist()
    held = [t[tables[b].long()].transpose(1, 2).reshape(-1, Hkv, D)[:e].clone() for t in pages for b, e in enumerate(ends)]
    return [o0, o1] + held, (x0, xs, paths, kepts, prompt, split, spec, sh0, ends)


def test_a_tree_that_is_kept_is_the_chain_that_was_drafted(moelib, cuda_dev):
    """Drafting trees, verifying and keeping paths leaves the cache and gives the outputs of a run that had the
    accepted tokens, one after the other, from the start."""
    m = moelib
    outs, (x0, xs, paths, kepts, prompt, split, spec, sh0, ends) = _serve(m, "sync")
    B, Hq, Hkv, D, page = 3, 8, 2, 128, 32
    n = 24
    for b in range(B):
        at = sum(prompt[:b])
        tok, rows = [x0[at:at + prompt[b]]], [outs[0][at:at + prompt[b]]]
        for i in range(len(xs)):
            k = int(kepts[i][b])
            idx = (paths[i][b, :k] + b * n).long()
            tok.append(xs[i][idx]), rows.append(outs[1][i][idx])
        x, want = torch.cat(tok).contiguous(), torch.cat(rows)
        T = x.shape[0]
        assert T == ends[b]
        P = -(-T // page)
        sh = m.paged_shape(1, T, Hq, Hkv, D, page, P, P, q_stride=x.shape[1], kv_stride=x.shape[1])
        cache = m.paged_alloc_cache(sh, DEV)
        cache.tables.copy_(torch.arange(P, device=DEV).view(1, P))
        q, o, ws = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV), m.paged_alloc_workspace(sh, DEV)
        m.paged_append(sh, spec, *split(x, T), _i32([0, T]), _i32([0]), cache, q)
        for pool, held in ((cache.k, outs[2 + b]), (cache.v, outs[2 + B + b])):
            assert torch.equal(pool.transpose(1, 2).reshape(-1, Hkv, D)[:T], held)
        m.paged_attn(m.paged_shape(1, T, Hq, Hkv, D, page, P, P), q, cache, _i32([0, T]), _i32([T]), o, ws)
        # other units and weights: each side within its rounding of the formula, 2 (2^-8 |o| + 2^-8 sum w |v|)
        V = cache.v.transpose(1, 2).reshape(-1, Hkv, D)[:T].double().abs().amax()
        assert ((o.double() - want.double()).abs() <= 2.0 ** -6 * V).all()
        assert (o.double() - want.double()).norm() <= 2.0 ** -7 * want.double().norm()


@pytest.mark.parametrize("mode", ["queue", "graph"])
def test_a_queue_of_calls_is_the_synchronised_run(moelib, cuda_dev, mode):
    """Calls that follow one another without the host between them (every kernel may be set up while the one before
    it still writes what it reads), eager and in a graph that is replayed: the bits of the synchronised run."""
    want, _ = _serve(moelib, "sync")
    assert all(torch.isfinite(t.float()).all() for t in want)
    for _ in range(3):
        got, _ = _serve(moelib, mode)
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_replays_with_other_lengths_and_two_graphs_at_once(moelib, cuda_dev):
    """A captured call follows its tables; two with workspaces of their own may run at the same time."""
    m = moelib
    p = Paged(m, [900, 700], 2, 256, 64, seed=60)
    gen = torch.Generator().manual_seed(61)
    q = _rand(gen, 2, 16, 256).to(DEV)
    sh, off, ln = p.shape(2, 16), _i32([0, 1, 2]), _i32([900, 700])
    streams, ws, outs, graphs = [torch.cuda.Stream() for _ in range(2)], [m.paged_alloc_workspace(sh, DEV) for _ in range(2)], [torch.empty_like(q) for _ in range(2)], []
    torch.cuda.synchronize()
    for i in range(2):
        m.paged_attn(sh, q, p.gpu, off, ln, outs[i], ws[i], stream=streams[i])
        streams[i].synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            m.paged_attn(sh, q, p.gpu, off, ln, outs[i], ws[i])
        graphs.append(g)
    for lens in ([900, 700], [1, 699], [0, 128], [513, 2]):
        ln.copy_(_i32(lens))
        torch.cuda.synchronize()
        for _ in range(5):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        want = p.attend(q, [1, 1], lens)
        assert all(torch.equal(o, want) for o in outs)


def test_no_tokens_and_refusals_of_the_binding(moelib, cuda_dev):
    m = moelib
    p = Paged(m, [20, 30], 1, 64, 16, seed=62)
    e = torch.empty(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    off, tab = _i32([0, 0, 0]), _i32([3, 4])
    m.paged_append(p.shape(0, 1), None, e, e, e, off, tab, p.gpu, e)
    ws = torch.full((m.paged_workspace_bytes(p.shape(0, 1)),), 255, dtype=torch.uint8, device=DEV)
    m.paged_attn(p.shape(0, 1), e, p.gpu, off, tab, e, ws)
    assert m.status_read(ws[:4].view(torch.int32)) == 0
    x = torch.zeros(3, 1, 64, dtype=torch.bfloat16, device=DEV)
    off, sh = _i32([0, 1, 3]), p.shape(3, 1)

    def append(**kw):
        a = dict(q=x, k=x, v=x, off=off, st=tab, c=p.gpu, o=x.clone(), pos=None, sh=sh, spec=None)
        a.update(kw)
        m.paged_append(a["sh"], a["spec"], a["q"], a["k"], a["v"], a["off"], a["st"], a["c"], a["o"], positions=a["pos"])

    wide = torch.zeros(3, 1, 128, dtype=torch.bfloat16, device=DEV)
    for text, kw in [("q is torch.float16", dict(q=x.half())), ("k_new has shape", dict(k=x[:2])), ("v_new has strides", dict(v=wide[..., :64])),
                     ("offsets is torch.int64", dict(off=off.long())), ("starts has shape", dict(st=off)), ("starts is on cpu", dict(st=tab.cpu())),
                     ("q without q_out", dict(o=None)), ("positions has shape", dict(pos=tab)), ("q_out is torch.float32", dict(o=x.float())),
                     ("the cache holds", dict(sh=m.paged_shape(2, 3, 1, 1, 64, 32, p.n, p.P))),
                     ("the spec's tensors", dict(spec=m.rope_spec(None, norm=1, q_gain=wide[0, 0].clone())))]:
        with pytest.raises(m.MoeError, match=text) as err:
            append(**kw)
        assert err.value.status == m.MOE_ERR_INVALID_ARG
    tsh = p.shape(3, 1, tree_words=2)
    for text, call in [("tree has shape", lambda: m.paged_attn(tsh, x, p.gpu, off, tab, x, ws, tree=tree_tensor([1] * 3, 1))),
                       ("tree is torch.int32", lambda: m.paged_attn(tsh, x, p.gpu, off, tab, x, ws, tree=tree_tensor([1] * 3, 2).int())),
                       ("invalid argument", lambda: m.paged_attn(tsh, x, p.gpu, off, tab, x, ws)),
                       ("tree has shape", lambda: m.paged_attn(sh, x, p.gpu, off, tab, x, ws, tree=tree_tensor([1] * 3, 1))),
                       ("workspace is torch.float32", lambda: m.paged_attn(sh, x, p.gpu, off, tab, x, ws.float())),
                       ("workspace too small", lambda: m.paged_attn(sh, x, p.gpu, off, tab, x, ws[:1024])),
                       ("lens has shape", lambda: m.paged_attn(sh, x, p.gpu, off, off, x, ws)),
                       ("o has shape", lambda: m.paged_attn(sh, x, p.gpu, off, tab, x[:2], ws)),
                       ("kept has shape", lambda: m.paged_keep(sh, p.gpu, tab, off, _i32([[0], [1]]))),
                       ("path has shape", lambda: m.paged_keep(sh, p.gpu, tab, tab, _i32([[0]]))),
                       ("lens_out is torch.int64", lambda: m.paged_keep(sh, p.gpu, tab, tab, _i32([[0], [1]]), lens_out=tab.long())),
                       ("unsupported shape", lambda: m.paged_keep(sh, p.gpu, tab, tab, torch.zeros(2, 513, dtype=torch.int32, device=DEV)))]:
        with pytest.raises(m.MoeError, match=text):
            call()
    assert np.array_equal(bits16(p.gpu.k), p.k)


FIRST_CALL = """
import torch
import bit_grouped_expert_moe_gb300 as m
i32 = dict(dtype=torch.int32, device="cuda")
table = m.rope_table(64)
spec = m.rope_spec(table)
for n in (1, 200):
    sh = m.paged_shape(1, n, 8, 2, 128, 32, 9, 8)
    cache, off, st = m.paged_alloc_cache(sh, "cuda"), torch.tensor([0, n], **i32), torch.zeros(1, **i32)
    cache.tables.copy_(torch.arange(8, 0, -1, **i32).view(1, 8))
    x = torch.ones(n, 2, 128, dtype=torch.bfloat16, device="cuda")
    q, ws, ln = torch.zeros(n, 8, 128, dtype=torch.bfloat16, device="cuda"), m.paged_alloc_workspace(sh, "cuda"), st + n
    o, pos = torch.zeros_like(q), torch.arange(n, **i32)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.rope(m.rope_shape(n, 8, 0, 128), spec, q, None, pos, q, None)
        m.paged_append(sh, spec, q, x, x, off, st, cache, q)
        m.paged_attn(sh, q, cache, off, ln, o, ws)
        m.paged_keep(sh, cache, st, st + 1, st.view(1, 1))
    g.replay()
    torch.cuda.synchronize()
    assert m.status_read(ws[:4].view(torch.int32)) == 0
    assert (o == 1).all()
"""


def test_first_calls_may_be_captured(moelib, cuda_dev):
    """In a process of its own, whose first calls are made during a capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
