"""Pins of the fp64 oracle of rotary positions and the paged KV cache
(oracle/paged.py), without a GPU."""
import math

import numpy as np
import pytest
import torch

from oracle import paged
from oracle.moe import bf16_bits_to_f64
from tests._util import bits16


def _bits(v):
    return bits16(torch.as_tensor(np.asarray(v, dtype=np.float32)).to(torch.bfloat16))


def test_two_pi():
    assert abs(float(paged._TWO_PI) - 2 * math.pi) < 1e-15
    assert float(paged._TWO_PI - paged._TWO_PI.__class__(2 * math.pi)) == pytest.approx(2.449293598294706e-16, rel=1e-10)


def test_hand_worked_rotations():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0, 6.0]]])
    quarter = np.array([math.pi / 2, math.pi])
    assert np.allclose(paged.rotated(x, [1], quarter, pairs=True), [[[-2, 1, -3, -4, 5, 6]]])
    assert np.allclose(paged.rotated(x, [1], quarter), [[[-3, -2, 1, -4, 5, 6]]])
    assert np.allclose(paged.rotated(x, [-1], quarter, pairs=True, magnitude=2.0), [[[4, -2, -6, -8, 5, 6]]])
    assert np.array_equal(paged.rotated(x, [0], quarter), x)


@pytest.mark.parametrize("pairs", [False, True])
def test_rotation_is_a_complex_product_and_scores_go_by_the_distance(pairs):
    rng = np.random.default_rng(1)
    w, _ = paged.frequencies(32, 1e4)
    x, y = rng.normal(size=(2, 1, 1, 40))
    z = paged.rotated(x, [77], w, pairs)
    c = (lambda v: v[0, 0, 0:32:2] + 1j * v[0, 0, 1:32:2]) if pairs else (lambda v: v[0, 0, :16] + 1j * v[0, 0, 16:32])
    assert np.allclose(c(z), c(x) * np.exp(1j * 77 * w)) and np.array_equal(z[..., 32:], x[..., 32:])
    far = 2 ** 31 - 1
    a = (paged.rotated(x, [far], w, pairs) * paged.rotated(y, [far - 100], w, pairs)).sum()
    b = (paged.rotated(x, [100], w, pairs) * paged.rotated(y, [0], w, pairs)).sum()
    assert a == pytest.approx(b, abs=1e-9)


def test_norm():
    x = np.array([[3.0, 4.0, 0.0, 0.0]])
    assert np.allclose(paged.normed(x, eps=0.0), [[1.2, 1.6, 0, 0]])
    assert np.allclose(paged.normed(x, np.array([0.5, 1, 2, 3]), 0.0, 1.0), [[1.8, 3.2, 0, 0]])
    assert (paged.normed(np.zeros((1, 4)), eps=1e-6) == 0).all()


def test_scalings_at_their_ends():
    plain, one = paged.frequencies(64, 1e4)
    assert one == 1.0 and plain[0] == 1.0 and plain[31] == pytest.approx(1e4 ** (-62 / 64))
    assert np.allclose(paged.frequencies(64, 1e4, "linear", 4.0)[0], plain / 4)
    bands, _ = paged.frequencies(64, 1e4, "bands", 8.0, 8192)
    t = 8192 * plain / (2 * math.pi)
    assert np.allclose(bands[t >= 4], plain[t >= 4]) and np.allclose(bands[t <= 1], plain[t <= 1] / 8)
    mid = (t > 1) & (t < 4)
    assert mid.any() and (bands[mid] < plain[mid]).all() and (bands[mid] > plain[mid] / 8).all()
    ramp, m = paged.frequencies(64, 1e4, "ramp", 16.0, 4096)
    assert m == pytest.approx(0.1 * math.log(16) + 1) and ramp[0] == plain[0] and ramp[31] == pytest.approx(plain[31] / 16)
    assert (np.diff(ramp / plain) <= 1e-12).all()


def _pool(rng, n_pages, H, page, D):
    return [_bits(rng.normal(0, 1, (n_pages, H, page, D))) for _ in range(2)]


def test_attention_is_torchs_on_the_gathered_pages_with_the_trees_mask():
    rng = np.random.default_rng(2)
    H, r, D, page, L, n = 2, 3, 16, 4, 23, 7
    k, v = _pool(rng, 9, H, page, D)
    table = rng.permutation(9)[:6]
    words = [1, 3, 5, 11, 21, 37, 0b1000101]  # parents -, 0, 0, 1, 2, 2, 2
    q = _bits(rng.normal(0, 1, (n, H * r, D)))
    o, o_abs = paged.attention(q, k, v, [table], page, [0, n], [L], words)
    mask = torch.ones(n, L, dtype=torch.bool)
    for i, w in enumerate(words):
        for d in range(n):
            mask[i, L - n + d] = bool(w >> d & 1) and d <= i
    K, V = (torch.from_numpy(bf16_bits_to_f64(x[table].transpose(1, 0, 2, 3).reshape(H, -1, D)[:, :L]))
            .repeat_interleave(r, 0) for x in (k, v))
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(bf16_bits_to_f64(q)).transpose(0, 1), K, V, attn_mask=mask).transpose(0, 1)
    assert np.allclose(o, want.numpy(), rtol=1e-12, atol=1e-14) and (o_abs >= np.abs(o) - 1e-15).all()
    # a chain of drafts is causal attention
    chain, _ = paged.attention(q, k, v, [table], page, [0, n], [L], [(2 << i) - 1 for i in range(n)])
    assert np.array_equal(chain, paged.attention(q, k, v, [table], page, [0, n], [L])[0])


def test_rows_without_a_visible_position_are_zero():
    rng = np.random.default_rng(3)
    k, v = _pool(rng, 3, 1, 4, 8)
    q = _bits(rng.normal(0, 1, (4, 1, 8)))
    o, _ = paged.attention(q, k, v, [[2, 0]], 4, [0, 4], [2])
    assert (o[:2] == 0).all() and (np.abs(o[2:]).max(-1) > 0).all()
    o, _ = paged.attention(q, k, v, [[2, 0]], 4, [0, 4], [4], [0, 2, 4, 0])
    assert (o[[0, 3]] == 0).all() and np.allclose(o[1, 0], bf16_bits_to_f64(v)[2, 0, 1])


def test_append_and_keep():
    pages = np.zeros((3, 1, 2, 1), np.uint16)
    paged.append(np.array([5, 6, 7], np.uint16).reshape(3, 1, 1), [0, 3], [1], pages, [[2, 0]], 2)
    assert pages[:, 0, :, 0].tolist() == [[6, 7], [0, 0], [0, 5]]
    paged.keep(pages, [[2, 0]], 2, [1], [[0, 2]], [2])  # drafts 0 and 2 of those at 1 ..
    assert pages[:, 0, :, 0].tolist() == [[7, 7], [0, 0], [0, 5]]
