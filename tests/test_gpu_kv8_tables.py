"""The tables of the 8-bit KV cache's calls on the tensor-core tiles: bad entries,
and ragged batches of more sequences than a warp looks at together."""
import numpy as np
import pytest
import torch

from tests.test_gpu_kv8 import FMTS, Pair, _i32, _packed, _plain_attention_gpu, _rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 1, 64), (16, 2, 256)])
@pytest.mark.parametrize("off,lens", [
    ([0, 300, 200, 600], [40, 40, 40]), ([1, 300, 400, 600], [40, 40, 40]), ([0, 300, 400, 599], [40, 40, 40]),
    ([0, 300, 400, 601], [40, 40, 40]), ([0, -1, 400, 600], [40, 40, 40]), ([0, 300, 400, 600], [-1, 40, 40]),
    ([0, 300, 400, 600], [40, 40, 41]), ([0, 300, 400, 600], [40, 2 ** 31 - 1, 40]),
    ([0, 300, 400, 600], [40, -2 ** 31, 40]), ([0, 2 ** 31 - 1, -2 ** 31, 600], [40, 40, 40])])
def test_bad_tables_write_nothing(moelib, cuda_dev, Hq, Hkv, D, off, lens):
    """600 tokens, which the tiles take; the next call on the workspace is good."""
    p = Pair(moelib, 3, Hkv, D, 40, 16, "int8")
    gen = p.fill([40, 40, 40], seed=3)
    sh = p.shape(600, Hq)
    q = _rand(gen, 600, Hq, D).to(torch.bfloat16).to("cuda:0")
    o = torch.full_like(q, 7.0)
    ws = moelib.kv8_alloc_workspace(sh, "cuda:0")
    moelib.kv8_attn(sh, q, p.gpu, _i32(off), _i32(lens), o, ws)
    assert moelib.status_read(ws[:4].view(torch.int32)) == moelib.MOE_ERR_INVALID_ARG
    assert (o == 7).all()
    p.check()
    news = [300, 100, 200]
    assert torch.equal(p.attend(q, news, [40, 40, 40], o=o, ws=ws), p.attend(q, news, [40, 40, 40]))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("Hq,Hkv,D,B", [(4, 1, 64, 40), (16, 4, 128, 70), (16, 2, 256, 33)])
def test_many_ragged_sequences(moelib, cuda_dev, Hq, Hkv, D, B, fmt):
    """Sequences without tokens, without positions, with more tokens than positions
    and with one of each, among longer ones, past the first 32 and at both ends."""
    rng = np.random.default_rng(B)
    news = rng.integers(0, 120, B)
    lens = news + rng.integers(0, 400, B)
    news[[0, 5, 31, 32, B - 1]] = [0, 0, 90, 0, 77]
    lens[[0, 5, 31, 32, B - 1]] = [50, 0, 0, 33, 80]
    news[7], lens[7] = 100, 60
    news[33 % B], lens[33 % B] = 70, 1
    news[9], lens[9] = 1, 1
    news, lens = [int(v) for v in news], [int(v) for v in lens]
    p = Pair(moelib, B, Hkv, D, max(lens), 32, fmt, seed=B)
    gen = p.fill(lens, seed=B + 1)
    q = _rand(gen, sum(news), Hq, D).to(torch.bfloat16)
    assert sum(news) * Hq > 36 * B * Hkv + 192  # the tiles
    got = p.attend(q, news, lens)
    seen = torch.cat([torch.arange(n) >= n - ln for n, ln in zip(news, lens)]).numpy()
    assert (got.cpu()[~seen] == 0).all()
    want, o_abs = _plain_attention_gpu(p, q, news, lens)
    want[~seen], o_abs[~seen] = 0, 0
    assert len(want) == _packed(news)[-1]
    p.compare(got.double().cpu().numpy(), want, o_abs, q, lens)
    for _ in range(5):
        assert torch.equal(got, p.attend(q, news, lens))


@pytest.mark.parametrize("fmt", FMTS)
def test_a_long_chunk_among_single_tokens(moelib, cuda_dev, fmt):
    """In one call, and as two on ranges of the same cache."""
    B, Hq, Hkv, D, L = 20, 8, 2, 128, 700
    lens, news = [100 + 7 * i for i in range(B - 1)] + [L], [1] * (B - 1) + [300]
    p = Pair(moelib, B, Hkv, D, L, 32, fmt, seed=5)
    gen = p.fill(lens, seed=6)
    q = _rand(gen, sum(news), Hq, D).to(torch.bfloat16)
    want, o_abs = _plain_attention_gpu(p, q, news, lens)
    p.compare(p.attend(q, news, lens).double().cpu().numpy(), want, o_abs, q, lens)
    c, x = p.gpu, q.to("cuda:0")
    o = torch.empty_like(x)
    for at, rows in ((slice(0, B - 1), slice(0, B - 1)), (slice(B - 1, B), slice(B - 1, None))):
        part = moelib.Kv8Cache(c.k[at], c.v[at], c.k_scale[at], c.v_scale[at])
        counts = news[at]
        sh = moelib.kv8_shape(len(counts), sum(counts), Hq, Hkv, D, L, 32, p.shape(1).format)
        ws = moelib.kv8_alloc_workspace(sh, "cuda:0")
        moelib.kv8_attn(sh, x[rows], part, _i32(_packed(counts)), _i32(lens[at]), o[rows], ws)
        assert moelib.status_read(ws[:4].view(torch.int32)) == 0
    p.compare(o.double().cpu().numpy(), want, o_abs, q, lens)
