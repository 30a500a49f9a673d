"""The 8-bit KV cache's oracle at the ends of bf16's range, without a GPU."""
import numpy as np
import pytest

from oracle import kv8


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_every_large_bf16_is_stored_finite_and_near(fmt):
    """All bf16 of the two top binades as a block of their own and beside the
    largest, both signs: the stored value rounds to a finite bf16 and is within
    half a step (of the code for int8, 2^-4 of the value for e4m3)."""
    bits = np.arange(0x7E80, 0x7F80, dtype=np.uint16)
    for sign in (0, 0x8000):
        for with_top in (False, True):
            for b in bits[::1 if not with_top else 3]:
                x = np.array([b | sign, 0x7F7F if with_top else b], dtype=np.uint16).reshape(1, 1, 2)
                codes, scales = np.zeros((1, 1, 16, 2), np.uint8), np.zeros((1, 1, 1), np.float32)
                assert not kv8.write(x, [0, 1], [0], codes, scales, 16, fmt)
                got = kv8.value_of(codes[0, 0, 0], scales[0, 0, 0], fmt)
                want = kv8.bf16_bits_to_f64(x)[0, 0]
                assert (np.abs(got) < 2.0 ** 128 * (1 - 2.0 ** -9)).all()
                half = np.abs(want).max() / 254 * (1 + 2.0 ** -20) if fmt == "int8" else np.abs(want) * 2.0 ** -4
                assert (np.abs(got - want) <= half).all()


@pytest.mark.parametrize("fmt,top", [("int8", 1.9921875 * 2.0 ** 127), ("e4m3", 1.875 * 2.0 ** 127)])
def test_infinities_are_as_large_as_the_largest(fmt, top):
    x = np.array([0x7F80, 0xFF80, 0x7F7F, 0x7FC0], dtype=np.uint16).reshape(1, 1, 4)
    codes, scales = np.zeros((1, 1, 16, 4), np.uint8), np.zeros((1, 1, 1), np.float32)
    assert kv8.write(x, [0, 1], [0], codes, scales, 16, fmt)
    got = kv8.value_of(codes[0, 0, 0], scales[0, 0, 0], fmt)
    assert np.allclose(got, [top, -top, top, 0], rtol=2.0 ** -22, atol=0)
