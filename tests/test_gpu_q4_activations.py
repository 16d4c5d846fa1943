"""Activations of the gated form over the whole range of their gate, against the definition in 64 bits."""
import numpy as np
import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from oracle import q4
from test_gpu_q4 import dev

pytestmark = pytest.mark.gpu

# what the gate's sum is, one row of W each: bf16 values times +-1, ascending
GATES = np.unique(q4.to_bf16(np.concatenate([np.linspace(-100, 100, 801), np.geomspace(1e-6, 200, 200), -np.geomspace(1e-6, 200, 200)]).astype(np.float32)))


def exactly(g, name):
    """act(g) in 64 bits without cancellation."""
    if name == "silu":
        return g * np.exp(np.minimum(g, 0)) / (1 + np.exp(-np.abs(g)))
    if name == "gelu_tanh":
        y = 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
        return g * np.exp(np.minimum(y, 0)) / (1 + np.exp(-np.abs(y)))
    return q4.act(g, name)


@pytest.mark.parametrize("name", sorted(bsp.ACTIVATIONS))
@pytest.mark.parametrize("N", [1, 12, 30, 70])
@pytest.mark.parametrize("size", [0, 100])
def test_range(size, N, name):
    """act(g) times 2^size.  Before its last rounding: the exponential's argument, up to 2^7.5 here, rounds to 2^-24 of itself twice (its
    polynomial, and the factor log2 e), and the exponential, quotient and products add 2^-20: 2^-14 of act(g); results
    below the normal range of fp32 lose 2^-149 for each 2^size more."""
    M, K = len(GATES), 32
    codes = np.full((M, K), 8, np.uint8)
    codes[:, 0] = np.where(GATES < 0, 7, 9)
    up = np.full((M, K), 8, np.uint8)
    up[:, 0] = 9
    one = np.full((M, 1), np.ldexp(1.0, size), np.float32)
    g = bsp.Int4Matrix.from_arrays(dev(q4.pack(codes)), dev(np.abs(GATES)[:, None], "bfloat16"), group=32)
    u = bsp.Int4Matrix.from_arrays(dev(q4.pack(up)), dev(one, "bfloat16"), group=32)
    x = np.zeros((N, K), np.float32)
    x[:, 0] = 1
    y = g.gated(u, dev(x, "bfloat16"), activation=name).double().cpu().numpy()
    want = np.ldexp(exactly(GATES.astype(np.float64), name), size)
    lim = np.abs(want) * (2.0 ** -14 + q4.HALF_STEP["bfloat16"] * (1 + 2.0 ** -14)) + np.ldexp(4 * 100 * 2.0 ** -149, size) + q4.TINY["bfloat16"]
    off = np.abs(y - want)
    worst = np.argmax((off / lim).max(0))
    assert np.all(off <= lim), (GATES[worst], y[0, worst], want[worst], (off / lim).max())
    g.close()
    u.close()
