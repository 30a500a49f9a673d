"""The 8-bit KV cache over the range of values that its header allows, on the GPU
against the fp64 oracle: blocks whose V scales lie far apart, scores far from
zero, magnitudes up to bf16's largest.

Tolerance of attention per element, from the arithmetic (u = 2^-24, codes c,
softmax weights p, V scales s, sums over the row's visible positions):
  * o is rounded to bf16: 2^-8 of the value before;
  * a weight goes to fp16: 2^-11 of it, and as much again for the sums and the
    exponentials below; or 2^-25 where that is more, with the row's largest
    p_j s(j) at 2^7 at least: 2^-32 max_j(p_j s(j)) sum_j |c_j|;
  * q goes to fp16 with its row's largest magnitude in [1, 2): nothing is lost
    above 2^-14, and below at most 2^-25: of a score,
    scale * 2 max|q| * 2^-25 * sum_d |K_d|;
  * a score: D + 8 operations, each off by at most 2 u of
    amp = scale * sum_d |q_d| * (255 code steps of int8, or 448) * K scale;
    on the base-2 scale, with log2 s added and m taken off, three roundings of
    at most u (|score| + 128) each, twice (a weight, and their sum);
  * a row's scores off by ds change its weights by a factor within e^(2 ds), and
    o by e^(2 ds) - 1 of the sum of magnitudes;
  * sums of at most L / 16 + 64 terms in fp32, each addition off by 2 u of at
    most the sum of magnitudes.
Every figure is the row's own: a block that other sequences hold has no part."""
import numpy as np
import pytest
import torch

from oracle import kv8
from oracle.moe import bf16_bits_to_f64
from tests._util import bits16
from tests.test_gpu_kv8 import FMTS, Pair, _packed, _rand

pytestmark = pytest.mark.gpu


def _bf16(x):
    return torch.as_tensor(x).to(torch.bfloat16)


def _tolerance(p, q, news, lens):
    """o of the formula and what the kernels may be off by, fp64 [T, Hq, D]."""
    off = _packed(news)
    T, Hq, D = q.shape
    r = Hq // p.dims[1]
    x = bf16_bits_to_f64(bits16(q))
    scale, u = D ** -0.5, 2.0 ** -24
    o, tol = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    for b, (n, ln) in enumerate(zip(news, lens)):
        at = np.arange(ln) // p.block
        for g in range(p.dims[1]):
            sk, sv = (p.scales[i][b, g][at].astype(np.float64) for i in range(2))
            K = kv8.value_of(p.codes[0][b, g, :ln], sk[:, None], p.fmt)
            c = kv8.value_of(p.codes[1][b, g, :ln], 1.0, p.fmt)
            step = 255.0 if p.fmt == "int8" else 448.0
            for i in range(n):
                see = ln - n + i + 1
                if see <= 0:
                    continue
                for h in range(g * r, (g + 1) * r):
                    y = x[off[b] + i, h]
                    z = scale * (K[:see] @ y)
                    w = np.exp(z - z.max())
                    w /= w.sum()
                    amp = scale * np.abs(y).sum() * step * sk[:see].max()
                    ds = (D + 8) * 2 * u * amp
                    ds += scale * 2 * np.abs(y).max() * 2.0 ** -25 * np.abs(K[:see]).sum(1).max()
                    ds += 6 * u * (np.abs(z).max() * np.log2(np.e) + 128) * np.log(2)
                    assert ds < 0.5
                    weighed = (w * sv[:see])
                    absolute = weighed @ np.abs(c[:see])
                    e = (2.1 * 2.0 ** -11 + np.expm1(2 * ds) + (see / 16 + 64) * 2 * u) * absolute
                    e += 2.0 ** -32 * weighed.max() * np.abs(c[:see]).sum(0)
                    o[off[b] + i, h] = weighed @ c[:see]
                    tol[off[b] + i, h] = e + 2.0 ** -8 * (np.abs(o[off[b] + i, h]) + e)
    return o, tol


def _check(p, q, news, lens):
    got = p.attend(q, news, lens).double().cpu().numpy()
    want, tol = _tolerance(p, q, news, lens)
    assert np.isfinite(got).all()
    err = np.abs(got - want)
    assert (err <= tol).all(), (float((err / np.maximum(tol, 1e-300)).max()), np.argwhere(err > tol)[:4],
                                got[err > tol][:4], want[err > tol][:4])


# the few-query kernels with 8, 16 and (at 128 head dims) 32 rows a tile, and the tiles
FORMS = [(64, 2, 1), (64, 4, 70), (128, 2, 1), (128, 8, 3), (128, 16, 3), (128, 4, 70), (256, 2, 1), (256, 8, 2),
         (256, 4, 70)]


def _blocks(gen, exponents, rows, D, Hkv=1):
    """Values whose block i is about 2^exponents[i] in size (None: zeros)."""
    out = []
    for e in exponents:
        v = _rand(gen, rows, Hkv, D).clamp(-3, 3)
        out.append(v * 0 if e is None else v * 2.0 ** e)
    return torch.cat(out)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("exponents", [
    [None, 100, None], [118, None, None, 118, None], [None, 74, 0], [60, None, -58, None, 60], [-50, 118, -50, 118],
    [118, -58, None, -58], [-58, -58, None, None, -58], [80, -40, 80, 0, None], [118, 118, 118]])
@pytest.mark.parametrize("D,r,news", FORMS)
def test_v_blocks_far_apart(moelib, cuda_dev, D, r, news, exponents, fmt):
    """Every position counts in a row's sum of weights, however small its V
    scale is beside another's, zeros among them."""
    block = 64 if D == 256 else 16
    L = block * len(exponents)
    p = Pair(moelib, 1, 1, D, L, block, fmt)
    gen = torch.Generator().manual_seed(7)
    v = _blocks(gen, exponents, block, D)
    p.write([_bf16(_rand(gen, L, 1, D)), _bf16(v)], [L], [0])
    p.check()
    for size in (0.0, 1.0):  # equal weights, then others
        _check(p, _bf16(_rand(gen, news, r, D) * size), [news], [L])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,r,news", FORMS)
def test_v_blocks_far_apart_across_runs(moelib, cuda_dev, D, r, news, fmt):
    """The same where many blocks of the grid share a sequence and their states
    are merged, and where a warp sees many units."""
    block, count = 64, 90
    L = block * count
    p = Pair(moelib, 1, 1, D, L, block, fmt)
    gen = torch.Generator().manual_seed(8)
    exponents = [[None, 110, -55, 3][int(i)] for i in torch.randint(0, 4, (count,), generator=gen)]
    v = _blocks(gen, exponents, block, D)
    p.write([_bf16(_rand(gen, L, 1, D)), _bf16(v)], [L], [0])
    _check(p, _bf16(_rand(gen, news, r, D)), [news], [L])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,r,news", FORMS)
def test_a_peaked_row_whose_top_value_is_zero(moelib, cuda_dev, D, r, news, fmt):
    """One position has nearly all the weight and zeros in some head dims: what
    the others add there is within the bound's term for weights that fp16 holds
    as subnormals or not at all."""
    L = 300
    p = Pair(moelib, 1, 1, D, L, 32, fmt)
    gen = torch.Generator().manual_seed(9)
    k, v, q = _rand(gen, L, 1, D) * 0.05, _rand(gen, L, 1, D), _rand(gen, news, r, D) * 0.05
    k[10, :, :8] = 4.0
    v[10, :, ::3] = 0
    for peak in (4.0, 8.0, 16.0, 24.0):  # of the score
        q[:, :, :8] = peak * D ** 0.5 / 32
        p.write([_bf16(k), _bf16(v)], [L], [0])
        _check(p, _bf16(q), [news], [L])


# ---------------------------------------------------------------- scores ---

def _top(p, q, news, ln):
    """What a row does whose scores are more than 1000 from the top one or as near
    to it as fp32 tells apart. A score is rounded to fp32 after log2 of its block's
    V scale is added, so that equal scores come out up to 2^-23 of their size apart
    and the tops share the weight in some way: o lies between their values. With
    one V scale they stay equal. Returns the least and largest of the tops' values,
    and the largest magnitude."""
    T, Hq, D = q.shape
    x = bf16_bits_to_f64(bits16(q))
    sk, sv = (p.scales[i][0, 0][np.arange(ln) // p.block].astype(np.float64)[:, None] for i in range(2))
    K, V = kv8.value_of(p.codes[0][0, 0, :ln], sk, p.fmt), kv8.value_of(p.codes[1][0, 0, :ln], sv, p.fmt)
    lo, hi = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    for i in range(news):
        for h in range(Hq):
            see = ln - news + i + 1
            z = (K[:see] @ x[i, h]) * D ** -0.5
            top = z == z.max()
            assert top.all() or z.max() - z[~top].max() > 1000 + 2.0 ** -20 * np.abs(z.max())
            one = (sv[:see][top] == sv[:see][top][0]).all()
            tops = V[:see][top].mean(0, keepdims=True) if one else V[:see][top]
            lo[i, h], hi[i, h] = tops.min(0), tops.max(0)
            total = np.abs(V[:see][top]).max(0)
            lo[i, h] -= 2.0 ** -8 * np.abs(lo[i, h]) + 2.2 * 2.0 ** -11 * total
            hi[i, h] += 2.0 ** -8 * np.abs(hi[i, h]) + 2.2 * 2.0 ** -11 * total
    return lo, hi


def _check_top(p, q, news, ln):
    got = p.attend(q, [news], [ln]).double().cpu().numpy()
    lo, hi = _top(p, q, news, ln)
    assert np.isfinite(got).all()
    bad = (got < lo) | (got > hi)
    assert not bad.any(), (bad.mean(), got[bad][:4], lo[bad][:4], hi[bad][:4])


SCORES = [(12, 11), (12, 14), (13, 16), (20, 20), (50, 52), (60, 61)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("a,b", SCORES)
@pytest.mark.parametrize("D,r,news", FORMS)
def test_scores_far_from_zero(moelib, cuda_dev, D, r, news, a, b, fmt):
    """Scores of both signs up to 2^121 and more, each more than 1000 from the
    next or equal to it. (The products are whole multiples of a power of two, so
    equal scores are equal in fp32; every block has the same K scale.)"""
    L, block = 200, 16
    p = Pair(moelib, 1, 1, D, L, block, fmt)
    gen = torch.Generator().manual_seed(10)
    k = (1 + torch.randint(0, 8, (L, 1, 1), generator=gen) / 8.0).expand(L, 1, D).clone()
    k[::block] = 1.875
    p.write([_bf16(k * 2.0 ** b), _bf16(_rand(gen, L, 1, D))], [L], [0])
    sign = torch.where(torch.arange(r) % 2 == 1, -1.0, 1.0)[None, :, None]
    q = _bf16((sign * 2.0 ** a).expand(news, r, D).clone())
    _check_top(p, q, news, L)
    k[5], k[37] = 2.0, 0.5  # one largest and one smallest, which every row sees
    p.write([_bf16(k * 2.0 ** b), _bf16(_rand(gen, L, 1, D))], [L], [0])
    _check_top(p, q, news, L)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("a,b", [(50, 52), (56, 57), (60, 61)])
@pytest.mark.parametrize("D,r,news", FORMS)
def test_all_scores_far_below_zero(moelib, cuda_dev, D, r, news, a, b, fmt):
    """Every visible score lies below -1e30 and all are equal; the first query of
    a prompt sees one position only and returns its value."""
    p = Pair(moelib, 1, 1, D, max(news, 2), 16, fmt)
    L = news
    gen = torch.Generator().manual_seed(11)
    v = _rand(gen, L, 1, D)
    q = _bf16(torch.full((news, r, D), 2.0 ** a))
    for values in (v, torch.cat([v[:1].sign(), v[1:].clamp(-1, 1)])):
        if values is not v:
            values[::16] = values[::16].sign()  # every block's largest is 1: one V scale
        p.write([_bf16(torch.full((L, 1, D), -2.0 ** b)), _bf16(values)], [L], [0])
        _check_top(p, q, news, L)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("a,b", [(4, 3), (10, 9), (12, 14), (20, 20), (60, 61)])
@pytest.mark.parametrize("D,r,news", FORMS)
def test_large_scores_over_v_blocks_far_apart(moelib, cuda_dev, D, r, news, a, b, fmt):
    """Both at once, over several units and runs: the tops share the weight, and
    their values lie up to 2^176 apart."""
    block, count = 16, 100
    L = block * count
    p = Pair(moelib, 1, 1, D, L, block, fmt)
    gen = torch.Generator().manual_seed(17)
    exponents = [[None, 115, -58, 3][int(i)] for i in torch.randint(0, 4, (count,), generator=gen)]
    k = (1 + torch.randint(0, 8, (L, 1, 1), generator=gen) / 8.0).expand(L, 1, D).clone()
    k[::block] = 1.875
    p.write([_bf16(k * 2.0 ** b), _bf16(_blocks(gen, exponents, block, D))], [L], [0])
    sign = torch.where(torch.arange(r) % 2 == 1, -1.0, 1.0)[None, :, None]
    q = _bf16((sign * 2.0 ** a).expand(news, r, D).clone())
    if (a, b) == (4, 3):  # scores below 2^13: fp32 tells them from their neighbours
        got = p.attend(q, [news], [L]).double().cpu().numpy()
        want, tol = _tolerance(p, q, [news], [L])
        assert np.isfinite(got).all() and (np.abs(got - want) <= tol).all()
    else:
        _check_top(p, q, news, L)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("size", [2.0 ** 21, 2.0 ** 24.5, 2.0 ** 25.2, 2.0 ** 26.1, 2.0 ** 28])
@pytest.mark.parametrize("D,r,news", FORMS)
def test_scores_that_rise_by_a_little(moelib, cuda_dev, D, r, news, size, fmt):
    """Each block's scores lie 4 to 16 (on the base-2 scale) above the last one's,
    next to a maximum of up to 2^28, where that is an fp32 step or less: o lies
    between the visible values. K's scales are set by hand."""
    block, count = 16, 80
    L = block * count
    p = Pair(moelib, 1, 1, D, L, block, fmt)
    gen = torch.Generator().manual_seed(14)
    p.write([_bf16(torch.ones(L, 1, D)), _bf16(_rand(gen, L, 1, D))], [L], [0])
    code = 127.0 if fmt == "int8" else 256.0  # of 1.0
    for step in (4.0, 8.0, 16.0):
        base2 = size + step * np.arange(count)
        p.scales[0][0, 0] = (base2 / (code * D * D ** -0.5 * np.log2(np.e))).astype(np.float32)
        p.gpu.k_scale.copy_(torch.from_numpy(p.scales[0]))
        got = p.attend(_bf16(torch.ones(news, r, D)), [news], [L]).double().cpu().numpy()
        V = kv8.value_of(p.codes[1][0, 0], p.scales[1][0, 0][np.arange(L) // block].astype(np.float64)[:, None], fmt)
        edge = 2.0 ** -7 * np.abs(V).max(0)
        assert np.isfinite(got).all()
        assert (got >= V.min(0) - edge).all() and (got <= V.max(0) + edge).all()
        # no more than 256 fp32 steps below the top takes part
        near = base2 > base2[(L - news) // block] - 40 - 256 * 2.0 ** -23 * size
        V = V[np.repeat(near, block)]
        assert (got >= V.min(0) - edge).all() and (got <= V.max(0) + edge).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("size", [0, 14])
@pytest.mark.parametrize("D,r,news", FORMS)
def test_queries_that_are_not_finite(moelib, cuda_dev, D, r, news, size, fmt):
    """A row with a NaN or an infinity is NaN; the rows beside it, whose scores are
    ordinary or large, are what they are without it but for the last rounding."""
    L = 300
    p = Pair(moelib, 1, 1, D, L, 32, fmt)
    gen = torch.Generator().manual_seed(18)
    p.write([_bf16(_rand(gen, L, 1, D) * 2.0 ** size), _bf16(_rand(gen, L, 1, D))], [L], [0])
    q = _bf16(_rand(gen, news, r, D) * 2.0 ** size)
    good = p.attend(q, [news], [L]).double().cpu()
    assert good.isfinite().all()
    for k, value in enumerate((float("nan"), float("inf"), float("-inf"))):
        x = q.clone()
        x[news // 2, 1, 5 + k] = value
        got = p.attend(x, [news], [L]).double().cpu()
        assert got[news // 2, 1].isnan().all()
        got[news // 2, 1] = good[news // 2, 1]
        assert ((got - good).abs() <= 2.0 ** -7 * good.abs() + 2.0 ** -10 * 4).all()


# ------------------------------------------------------- largest magnitudes ---

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,block", [(64, 16), (128, 32), (256, 64)])
def test_values_up_to_the_largest_of_bf16(moelib, cuda_dev, D, block, fmt):
    """Everything finite that is written reads back finite, within half a step:
    of a code (a / 254, and what the fp32 scale and product round) for int8,
    2^-4 relative for e4m3."""
    L = 5 * block + 3
    p = Pair(moelib, 1, 2, D, L, block, fmt)
    gen = torch.Generator().manual_seed(12)
    big = torch.finfo(torch.bfloat16).max
    x = _bf16((1 - 0.06 * torch.rand(L, 2, D, generator=gen)) * big * torch.sign(_rand(gen, L, 2, D)))
    x[0, 0, 0], x[0, 1, 1] = big, -big
    x[block:block + 5] = _bf16(torch.tensor(1.9375 * 2.0 ** 127))  # between two codes
    x[2 * block:3 * block] *= 2.0 ** -9
    y = x.clone()
    y[3, 0, 2:4], y[3, 1, 5] = float("inf"), float("nan")  # an infinity is as large as its block's largest
    first = 2 * block + 3  # the second call starts inside a block and makes its scale grow
    for v, status in ((x, moelib.MOE_OK), (y, moelib.MOE_ERR_RANGE)):
        p.write([v[:first], -v[:first]], [first], [0], expect=status)
        p.write([v[first:], -v[first:]], [L - first], [first])
        p.check()
        p.read([L], [0])
        for codes, scales, sign in zip((p.gpu.k, p.gpu.v), p.scales, (1, -1)):
            s = scales[0][:, np.arange(L) // block][:, :, None].astype(np.float64)
            stored = kv8.value_of(codes.view(torch.uint8).cpu().numpy()[0], s, fmt).transpose(1, 0, 2)
            assert (np.abs(stored) < 2.0 ** 128 * (1 - 2.0 ** -9)).all()  # rounds to a finite bf16
            want = sign * x.double().numpy()
            keep = np.isfinite(v.double().numpy())
            err = np.abs(stored - want)[keep]
            half = big / 254 * (1 + 2.0 ** -20) if fmt == "int8" else np.abs(want[keep]) * 2.0 ** -4
            grown = (np.arange(L)[:, None, None] >= 2 * block) & (np.arange(L)[:, None, None] < first)
            half = np.where(np.broadcast_to(grown, want.shape)[keep], big / 64, half)  # quantised twice
            assert (err <= half).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,r,news", FORMS)
def test_attention_over_the_largest_of_bf16(moelib, cuda_dev, D, r, news, fmt):
    L, block = 130, 16
    p = Pair(moelib, 1, 1, D, L, block, fmt)
    gen = torch.Generator().manual_seed(13)
    big = torch.finfo(torch.bfloat16).max
    v = _bf16((1 - 0.06 * torch.rand(L, 1, D, generator=gen)) * big)
    v[5:9] = big
    p.write([_bf16(_rand(gen, L, 1, D)), v], [L], [0])
    p.check()
    _check(p, _bf16(_rand(gen, news, r, D)), [news], [L])


# ------------------------------------------------------- words of the header ---

@pytest.mark.parametrize("D", [64, 128, 256])
def test_read_rounds_the_fp32_product(moelib, cuda_dev, D):
    """INT8 codes times scales whose product lies next to the middle of two bf16:
    fp32 rounds it to the middle, and that goes to the even one."""
    block, L = 16, 16 * 200
    p = Pair(moelib, 1, 1, D, L, block, "int8")
    rng = np.random.default_rng(15)
    code = rng.integers(64, 128, L // block)
    middle = (rng.integers(128, 256, L // block) + 0.5) * 2.0 ** -7
    scale = np.float32(middle / code)
    product = scale * code.astype(np.float32)
    exact = scale.astype(np.float64) * code
    assert ((product == middle) & (exact != middle)).sum() > 50
    p.codes = [np.repeat(128 + code, block).astype(np.uint8)[None, None, :, None] * np.ones((1, 1, 1, D), np.uint8)] * 2
    p.scales = [scale[None, None]] * 2
    p.gpu.k.copy_(torch.from_numpy(p.codes[0])), p.gpu.v.copy_(torch.from_numpy(p.codes[1]))
    p.gpu.k_scale.copy_(torch.from_numpy(p.scales[0])), p.gpu.v_scale.copy_(torch.from_numpy(p.scales[1]))
    p.read([L], [0])
    out = torch.empty(L, 1, D, dtype=torch.bfloat16, device="cuda:0")
    off, st = (torch.tensor(v, dtype=torch.int32, device="cuda:0") for v in ([0, L], [0]))
    moelib.kv8_read(p.shape(L), p.gpu, off, st, out, torch.empty_like(out))
    want = torch.from_numpy(product).to(torch.bfloat16).repeat_interleave(block)
    assert torch.equal(out[:, 0].cpu(), want[:, None].expand(L, D))


@pytest.mark.parametrize("fmt", FMTS)
def test_writing_over_earlier_positions(moelib, cuda_dev, fmt):
    """A write at a block's start takes the scale of its own values: what follows
    in the block keeps its bytes and is written again, as the header says."""
    p = Pair(moelib, 1, 2, 64, 48, 16, fmt)
    gen = torch.Generator().manual_seed(16)
    a, b = (_bf16(_rand(gen, n, 2, 64) * s) for n, s in ((5, 1.0), (14, 9.0)))
    p.write([a, -a], [5], [0])
    p.write([b, -b], [14], [5])
    p.write([b, -b], [14], [5])  # the last write repeated
    p.check()
    before = p.bytes()
    p.write([a, -a], [5], [0])
    p.check()
    assert all(np.array_equal(x[:, :, 5:], y[:, :, 5:]) for x, y in zip(before, p.bytes()))
    p.write([b, -b], [14], [5])
    p.check()
    p.read([19], [0])
