"""Attention over the paged cache where its numbers are far from the usual ones. Against fp64."""
import numpy as np
import pytest
import torch

from oracle import paged
from tests.test_gpu_paged import Paged, _packed, _rand, words_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("top", [1 << 9, 1 << 14, 1 << 18, 700_000])
@pytest.mark.parametrize("D,Hkv,r,lens,news", [
    (64, 1, 8, [2000], [1]), (128, 1, 8, [2000], [1]), (256, 1, 8, [2000], [1]),     # a unit per run: partial states
    (64, 8, 2, [700] * 8, [1] * 8), (128, 8, 2, [700] * 8, [1] * 8), (256, 8, 2, [700] * 8, [1] * 8),  # units of one run
    (64, 2, 4, [1500], [300]), (128, 2, 4, [1500], [300]), (256, 2, 4, [1500], [300])])  # many rows
def test_large_scores_that_are_exact(moelib, cuda_dev, D, Hkv, r, lens, news, top):
    """Scores are whole numbers near `top` (at scale 1; every product and sum is below 2^24), level + 0, 1, 2 or 3 by
    halves of units, and V is 1 in the quarter of the head dims that belongs to its level: o is the levels' shares of
    the weight, of which no error of a score takes anything. Every weight and o are rounded to bf16, 2^-8 of each; the
    exponents (below 2^3 from the largest) are off by 2^-16 at most and a factor of 1 + 2^-22, so a share by 2^-15,
    and a sum of up to 2000 positions in chains of 200 additions by 200 2^-24 < 2^-16 of it."""
    p = Paged(moelib, lens, Hkv, D, 32, seed=81)
    rng = np.random.default_rng(82)
    K, V = torch.zeros_like(p.gpu.k), torch.zeros_like(p.gpu.v)
    for b, n in enumerate(lens):
        level = rng.integers(0, 4, size=-(-n // 64)).repeat(64)[:n]
        for j in range(n):
            page, row = int(p.tables[b][j // 32]), j % 32
            K[page, :, row, 0], K[page, :, row, 1] = 64.0, float(level[j])
            V[page, :, row, int(level[j])::4] = 1.0
    p.gpu.k.copy_(K), p.gpu.v.copy_(V)
    T, Hq = sum(news), Hkv * r
    q = torch.zeros(T, Hq, D)
    q[..., 0] = torch.from_numpy(rng.uniform(0.8, 1.0, size=(T, Hq)) * top / 64)
    q[..., 1] = 1.0
    q = q.to(torch.bfloat16)  # 64 times a value of 4 or more that has 8 bits is whole
    want, o_abs = p.exact(q, news, scale=1.0)
    got = p.attend(q, news, scale=1.0).double().cpu().numpy()
    tol = 2.0 ** -8 * want + (2.0 ** -8 + 2.0 ** -14) * o_abs
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / np.maximum(tol, 1e-30)).max())


@pytest.mark.parametrize("scale,std", [(2.0 ** -120, 7e17), (1e-39, 1.5e18), (1e30, 7e-16)])
@pytest.mark.parametrize("D,lens,news", [(64, [900], [1]), (256, [2000], [1]), (128, [700], [200]), (256, [600, 40], [100, 40])])
def test_scales_near_the_ends_of_fp32(moelib, cuda_dev, D, lens, news, scale, std):
    """Scores far from 1 that the scale brings back there, in single tiles and joined from partial states."""
    p = Paged(moelib, lens, 2, D, 32, seed=83, std=(std, 1.0))
    q = _rand(torch.Generator().manual_seed(84), sum(news), 8, D, std=std * (64 / D) ** 0.5)
    p.check(q, news, scale=scale)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,page,lens,news", [
    (4, 2, 64, 16, [90, 40], [1, 1]), (16, 2, 256, 64, [2000, 300], [1, 1]), (8, 2, 128, 32, [1000, 70], [40, 70]),
    (4, 2, 64, 32, [900, 200], [150, 60]), (16, 2, 256, 64, [700, 50], [200, 50])])
def test_a_row_whose_scores_are_all_minus_infinity(moelib, cuda_dev, Hq, Hkv, D, page, lens, news, tree):
    """It is NaN, as its softmax is. Beside a finite score one of minus infinity weighs nothing, and a row that sees
    nothing is zero, whatever the keys hold."""
    p = Paged(moelib, lens, Hkv, D, page, seed=85)
    q = _rand(torch.Generator().manual_seed(86), sum(news), Hq, D)
    q[..., 0] = q[..., 0].abs() + 0.125
    words = [w for n in news for w in words_of([i - 1 if i % 5 else -1 for i in range(n)])] if tree else None
    if tree:  # rows without a bit; over no context they see nothing
        for t in range(0, len(words), 7):
            words[t] = 0
    r, off = Hq // Hkv, _packed(news)

    def at(b, j):
        return int(p.tables[b][j // page]), j % page

    # sequence 0, head 1: all keys; sequence 1, head 0: all but one that everybody sees, or the first draft
    for j in range(lens[0]):
        pg, row = at(0, j)
        p.gpu.k[pg, 1, row, 0] = -torch.inf
    one = 0
    for j in range(lens[1]):
        if j != one:
            pg, row = at(1, j)
            p.gpu.k[pg, 0, row, 0] = -torch.inf
    got = p.attend(q, news, words=words).float().cpu()
    K1, V1 = p.gpu.k[at(1, one)[0], 0, at(1, one)[1]], p.gpu.v[at(1, one)[0], 0, at(1, one)[1]].float().cpu()
    assert torch.isfinite(K1.float()).all()
    for b, (n, ln) in enumerate(zip(news, lens)):
        see = paged.visible(n, ln, words[off[b]:off[b + 1]] if tree else None)
        for i in range(n):
            o = got[off[b] + i]
            if not see[i].any():
                assert (o == 0).all(), (b, i)
            elif b == 0:
                assert torch.isnan(o[r:2 * r]).all() and torch.isfinite(o[:r]).all(), (b, i)
            elif see[i, one]:
                assert (o[:r] == V1).all() and torch.isfinite(o[r:]).all(), (b, i)
            else:
                assert torch.isnan(o[:r]).all() and torch.isfinite(o[r:]).all(), (b, i)
