"""Products of 4-bit weights at the ends of the types' ranges."""
import numpy as np
import pytest

from oracle import q4
from test_gpu_q4 import close, dev, matrix, rows, weight

pytestmark = pytest.mark.gpu


def scaled(N, K, M, group, zeros, up, down):
    """bfloat16 activations times 2^up and scales times 2^down."""
    return np.ldexp(rows(N, K, "bfloat16", 2), up), smaller(weight(M, K, group, zeros, "bfloat16", 1), down)


def smaller(w, down):
    """The same weight with scales times 2^down (the smallest are subnormal)."""
    return w[0], q4.ROUND["bfloat16"](np.ldexp(w[1], down)), w[2]


@pytest.mark.parametrize("up,down", [(110, -110), (120, -100), (120, -120), (-90, 60), (-120, 110), (60, -118)])
@pytest.mark.parametrize("N", [1, 9, 20, 40, 300])
@pytest.mark.parametrize("group,zeros", [(32, False), (64, True), (128, False)])
def test_activations_of_any_size(group, zeros, N, up, down):
    """Sums of a group before its scale stay finite wherever the activations are: up to 20 x 2^122 x 15 x 128 is far past
    fp32 as it stands.  Tolerances are those of any product: powers of two change none of them."""
    K, M = 520, 150
    x, w = scaled(N, K, M, group, zeros, up, down)
    assert np.isfinite(x).all() and np.isfinite(w[1]).all()
    m = matrix(w, group, "bfloat16")
    with np.errstate(all="ignore"):
        close(m.mm(dev(x, "bfloat16")), q4.product(x, *w, group), q4.error_bound(x, *w, group), "bfloat16")
    m.check()
    m.close()


def test_gated_of_any_size():
    import torch
    K, M, N = 264, 100, 50
    for n in (2, N):
        x, w = scaled(n, K, M, 64, True, 118, -118)
        u = smaller(weight(M, K, 64, False, "bfloat16", 7), -118)
        a, b = matrix(w, 64, "bfloat16"), matrix(u, 64, "bfloat16")
        gs, us = q4.product(x, *w, 64), q4.product(x, *u, 64)
        eg, eu = q4.error_bound(x, *w, 64), q4.error_bound(x, *u, 64)
        y = a.gated(b, dev(x, "bfloat16"), activation="gelu")
        assert torch.isfinite(y).all()
        close(y, q4.act(gs, "gelu") * us, q4.gated_bound(gs, us, eg, eu, "gelu"), "bfloat16")
        a.close()
        b.close()
