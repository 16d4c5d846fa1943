"""The 4-bit weights' and the rotary plain definitions, pinned by brute force."""
import math

import numpy as np
import pytest

from oracle import q4, rope


def test_pack_round_trip():
    c = np.random.default_rng(1).integers(0, 16, (5, 24)).astype(np.uint8)
    p = q4.pack(c)
    assert p[2, 3] == c[2, 6] + 16 * c[2, 7]
    assert np.array_equal(q4.unpack(p), c)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_quantise_is_near(zeros, dtype):
    g = np.random.default_rng(2)
    W = q4.ROUND[dtype](g.standard_normal((6, 72)).astype(np.float32))
    c, s, z = q4.quantise(W, dtype, 32, zeros)
    assert s.shape == (6, 3) and c.max() <= 15
    back = q4.dense(c, s, z, 32)
    step = np.repeat(s, 32, 1)[:, :72]
    # half a step to the nearest code; with zero points the range's ends may
    # miss by another half (the zero point is rounded), and the scale's own
    # rounding moves them by up to 15 half-steps of the type
    slack = 0.5 + (0.5 if zeros else 0) + 15 * q4.HALF_STEP[dtype]
    assert np.all(np.abs(back - W) <= slack * step)


def test_quantise_edges():
    W = np.zeros((4, 32), np.float32)
    W[1, 3], W[2, 5], W[3, 0], W[3, 1] = np.nan, np.inf, -7.0, 3.5
    c, s, z = q4.quantise(W, "float16", 32, False)
    assert np.all(c[0] == 8) and s[0, 0] == 0 and np.all(c[1] == 8) and np.all(c[2] == 8)
    assert s[3, 0] == 1 and c[3, 0] == 1 and c[3, 1] == 12  # 3.5 to even: 4
    c, s, z = q4.quantise(np.array([[1.0] * 16 + [15.0] * 16], np.float32), "float16", 32, True)
    assert z[0, 0] == 0 and s[0, 0] == 1 and c[0, 0] == 1 and c[0, 31] == 15


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotate_by_hand(interleaved, inverse):
    g = np.random.default_rng(3)
    x, pos = g.standard_normal((3, 2, 12)), np.array([[5, 1000000, -1], [7, 3, 2]])
    freqs, axis = [1.0, 0.1, 0.01, 0.3], [0, 1, 0, 1]
    y = rope.rotate(x, pos, freqs, axis, interleaved, scale=1.5, inverse=inverse)
    assert np.array_equal(y[2], x[2]) and np.array_equal(y[..., 8:], x[..., 8:])
    for r in range(2):
        for i in range(4):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 4)
            p = pos[axis[i]][r] * freqs[i] * (-1 if inverse else 1)
            z = complex(x[r, 1, a], x[r, 1, b]) * 1.5 * complex(math.cos(p), math.sin(p))
            assert abs(y[r, 1, a] - z.real) < 1e-9 and abs(y[r, 1, b] - z.imag) < 1e-9
