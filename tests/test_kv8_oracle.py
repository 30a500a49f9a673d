"""Pins of the 8-bit KV cache's fp64 oracle (oracle/kv8.py), without a GPU."""
import math

import numpy as np
import pytest
import torch

from oracle import kv8
from tests._util import bits16


def _bits(v):
    return bits16(torch.as_tensor(np.asarray(v, dtype=np.float32)).to(torch.bfloat16))


def test_e4m3_table_is_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    got = kv8.e4m3_value(codes.numpy())
    assert got[127] == 480 and got[255] == -480 and np.isnan(want[[127, 255]]).all()
    rest = np.arange(256) % 128 != 127
    assert np.array_equal(got[rest], want[rest])


def test_e4m3_rounding_is_to_nearest_even():
    rng = np.random.default_rng(1)
    y = np.concatenate([rng.normal(0, 3, 2000), rng.normal(0, 200, 2000), 2.0 ** rng.uniform(-12, 8.7, 2000),
                        kv8._E4M3[:-1] / 2 + kv8._E4M3[1:] / 2, [0.0, 448.0, 460.0, 1e9]]).astype(np.float32)
    y = np.concatenate([y, -y])
    want = torch.from_numpy(np.clip(y, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kv8.e4m3_code(y), want)


@pytest.mark.parametrize("a,int8,e4m3", [
    (0.0, 0.0, 0.0), (127.0, 1.0, 0.5), (448.0, np.float32(448) / np.float32(127), 1.0),
    (450.0, np.float32(450) / np.float32(127), 2.0), (1.0, np.float32(1) / np.float32(127), 2.0 ** -8),
    (1e-30, 2.0 ** -60, 2.0 ** -60), (2.0 ** 127, np.float32(2.0 ** 127) / np.float32(127), 2.0 ** 119)])
def test_scales(a, int8, e4m3):
    assert kv8.scale_of(a, "int8") == np.float32(int8) and kv8.scale_of(a, "e4m3") == np.float32(e4m3)


def test_hand_worked_block():
    # one head, two values per token, blocks of two positions
    x = _bits([[[127.0, -1.0]], [[63.5, 0.25]], [[0.0, 0.0]]])
    codes, scales = np.zeros((1, 1, 4, 2), np.uint8), np.zeros((1, 1, 2), np.float32)
    assert not kv8.write(x, [0, 3], [0], codes, scales, 2, "int8")
    assert scales.tolist() == [[[1.0, 0.0]]]
    # 63.5 is a tie and goes to 64; 0.25 to 0
    assert codes[0, 0].tolist() == [[255, 127], [192, 128], [128, 128], [0, 0]]
    # position 3 joins the block of zeros: its scale becomes that of the new value
    kv8.write(_bits([[[254.0, 2.0]]]), [0, 1], [3], codes, scales, 2, "int8")
    assert scales[0, 0, 1] == 2.0 and codes[0, 0, 3].tolist() == [255, 129] and codes[0, 0, 2].tolist() == [128, 128]


def test_growth_requantises_earlier_codes_only():
    codes, scales = np.full((1, 1, 16, 2), 7, np.uint8), np.full((1, 1, 1), 99.0, np.float32)
    kv8.write(_bits([[[1.27, -0.64]]]), [0, 1], [0], codes, scales, 16, "int8")
    s0 = scales[0, 0, 0]
    kv8.write(_bits([[[5.08, 0.0]]]), [0, 1], [1], codes, scales, 16, "int8")
    s1 = scales[0, 0, 0]
    assert s1 > s0 and codes[0, 0, 0, 0] - 128 == round(127 * s0 / s1) and codes[0, 0, 1].tolist() == [255, 128]
    assert (codes[0, 0, 2:] == 7).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_round_trip_is_within_half_a_step(fmt):
    rng = np.random.default_rng(5)
    x = _bits(rng.normal(0, 2, (50, 2, 64)))
    codes, scales = np.zeros((1, 2, 64, 64), np.uint8), np.zeros((1, 2, 4), np.float32)
    kv8.write(x, [0, 50], [0], codes, scales, 16, fmt)
    from oracle.moe import bf16_bits_to_f64
    v, got = bf16_bits_to_f64(x), kv8.read([0, 50], [0], codes, scales, 16, fmt)
    s = scales[0][:, np.arange(50) // 16].T[:, :, None].astype(np.float64)
    step = s if fmt == "int8" else np.maximum(2.0 ** np.floor(np.log2(np.abs(v / s) + 1e-300)), 2.0 ** -6) * s / 8
    assert (np.abs(got - v) <= step * (0.5 + 1e-5)).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_values_that_are_not_finite(fmt):
    x = _bits([[[1.0, math.nan, math.inf, -math.inf]], [[-2.0, 0.5, 1.0, 0.0]]])
    codes, scales = np.zeros((1, 1, 2, 4), np.uint8), np.zeros((1, 1, 1), np.float32)
    assert kv8.write(x, [0, 2], [0], codes, scales, 16, fmt)
    assert np.allclose(kv8.read([0, 2], [0], codes, scales, 16, fmt)[:, 0],
                       [[1.0, 0.0, 2.0, -2.0], [-2.0, 0.5, 1.0, 0.0]], atol=2 / 254)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_attention_is_torchs_on_the_dequantised_cache(fmt):
    rng = np.random.default_rng(6)
    L, n, H, r, D = 40, 7, 2, 3, 64
    codes = [rng.integers(1, 127 if fmt == "e4m3" else 256, (1, H, L, D)).astype(np.uint8) for _ in range(2)]
    scales = [rng.uniform(0.001, 0.004, (1, H, 3)).astype(np.float32) for _ in range(2)]
    q = _bits(rng.normal(0, 1, (n, H * r, D)))
    o, o_abs = kv8.attention(q, *codes, *scales, [0, n], [L], 16, fmt)
    from oracle.moe import bf16_bits_to_f64
    at = np.arange(L) // 16
    K, V = (torch.from_numpy(kv8.value_of(c[0], s[0][:, at][:, :, None], fmt)).repeat_interleave(r, 0)
            for c, s in zip(codes, scales))
    mask = torch.arange(L)[None] <= (L - n + torch.arange(n))[:, None]
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(bf16_bits_to_f64(q)).transpose(0, 1), K, V, attn_mask=mask).transpose(0, 1)
    assert np.allclose(o, want.numpy(), rtol=1e-12, atol=1e-14) and (o_abs >= np.abs(o) - 1e-15).all()


def test_attention_rows_without_a_visible_position_are_zero():
    rng = np.random.default_rng(7)
    codes = [rng.integers(0, 256, (2, 1, 8, 64)).astype(np.uint8) for _ in range(2)]
    scales = [np.full((2, 1, 1), 0.01, np.float32)] * 2
    q = _bits(rng.normal(0, 1, (5, 1, 64)))
    o, _ = kv8.attention(q, *codes, *scales, [0, 4, 5], [2, 0], 16, "int8")
    assert (o[[0, 1, 4]] == 0).all() and (np.abs(o[2:4]).max(-1) > 0).all()
