"""Angles of rotary positions: small ones keep their relative accuracy, far ones their place in the turn."""
from decimal import Decimal, getcontext

import numpy as np
import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from oracle import q4
from test_gpu_rope import dev

pytestmark = pytest.mark.gpu

TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")


def turned(r, positions, interleaved):
    """What (a, b) = (0, 1) and (1, 0) become at each position: (-sin p, cos p), (cos p, sin p), pair by pair."""
    import torch
    half = r.rot // 2
    x = torch.zeros((len(positions), 2, r.dim), dtype=torch.bfloat16, device="cuda")
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    x[:, 0, second], x[:, 1, first] = 1, 1
    y = r.apply(x, None, dev(np.asarray(positions, np.int32))).double().cpu().numpy()
    return -y[:, 0, first], y[:, 0, second], y[:, 1, first], y[:, 1, second]


def angles(freqs, positions):
    """Radians within half a turn of zero, from 60 digits."""
    getcontext().prec = 60
    out = np.empty((len(positions), len(freqs)))
    for i, p in enumerate(positions):
        for j, f in enumerate(freqs):
            t = Decimal(p) * Decimal(f) / TWO_PI
            out[i, j] = float((t - t.to_integral_value()) * TWO_PI)
    return out


POSITIONS = [1, 2, 3, 7, 1000, 65535, 1 << 20, 10 ** 9 + 7, 2 ** 31 - 1]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("base", [1e4, 5e5, 1e7, 1e9])
def test_sines_and_cosines(base, interleaved):
    """Sine and cosine within the frequency's fixed point (position 2^-65 turns, and as much again for the frequency's own last
    bit), 2^-22 of themselves (the angle's rounding to fp32, and the functions', a few units of 2^-24) and half a step of the type."""
    r = bsp.Rotary(128, base=base, interleaved=interleaved)
    p = angles(r.freqs, POSITIONS)
    sin0, cos0, cos1, sin1 = turned(r, POSITIONS, interleaved)
    fixed = 2 * np.pi * np.asarray(POSITIONS, np.float64)[:, None] * 2.0 ** -64
    for got, want in ((sin0, np.sin(p)), (sin1, np.sin(p)), (cos0, np.cos(p)), (cos1, np.cos(p))):
        before = fixed + np.abs(want) * 2.0 ** -22 + np.abs(p) * 2.0 ** -24
        assert np.all(np.abs(got - want) <= before + (np.abs(want) + before) * q4.HALF_STEP["bfloat16"] + q4.TINY["bfloat16"])
    r.close()


def test_a_frequency_of_any_size():
    """Frequencies next to the ends of their range, and negative ones: all is one turn after another."""
    freqs = [65536.0, -65536.0, 65535.99999999, 3.0, -1e-12, 6.283185307179586, 1e-300, 0.0]
    r = bsp.Rotary(16, freqs=freqs)
    p = angles(freqs, POSITIONS)
    sin0, cos0, cos1, sin1 = turned(r, POSITIONS, False)
    fixed = 2 * np.pi * np.asarray(POSITIONS, np.float64)[:, None] * 2.0 ** -64
    for got, want in ((sin0, np.sin(p)), (sin1, np.sin(p)), (cos0, np.cos(p)), (cos1, np.cos(p))):
        before = fixed + np.abs(want) * 2.0 ** -22 + np.abs(p) * 2.0 ** -24
        assert np.all(np.abs(got - want) <= before + (np.abs(want) + before) * q4.HALF_STEP["bfloat16"] + q4.TINY["bfloat16"])
    r.close()
