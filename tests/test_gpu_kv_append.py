"""The append's corners, bit for bit against the definition."""
import numpy as np
import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from oracle import kv_cache as kv
from test_gpu_kv_cache import dev, make_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("dim,page,n", [(16, 16, 1), (128, 64, 3), (256, 32, 40), (80, 256, 300)])
def test_scales_that_stay_zero(dim, page, n, dtype):
    """Earlier codes under a scale of 0, then rows of zeros and NaN: all codes
    are 0 while the scale is."""
    import torch
    g = np.random.default_rng(n)
    heads, at = 3, page // 2 + 1
    k, v, ks, vs = make_cache(4, heads, page, dim, g)
    ks[:], vs[:, 1] = 0, 0
    table = np.array([[2, 0, 3]], np.int32)
    x = np.zeros((n, heads, dim), np.float32)
    x[0, 1] = np.nan
    y = x.copy()
    y[:, 0] = g.standard_normal((n, dim))
    t = [dev(a) for a in (k, v, ks, vs)]
    cache = bsp.KvCache(*t)
    xd, yd = dev(x).to(getattr(torch, dtype)), dev(y).to(getattr(torch, dtype))
    seq, start = np.array([at + n], np.int32), np.array([0, n], np.int32)
    cache.append(bsp.KvStep(dev(table), dev(seq), dev(start), n), xd, yd)
    for codes, scale, rows, got_c, got_s in ((k, ks, xd, t[0], t[2]), (v, vs, yd, t[1], t[3])):
        c, s = kv.append(codes, scale, rows.float().cpu().numpy(), table, seq, start, page)
        assert np.array_equal(got_c.cpu().numpy(), c) and np.array_equal(got_s.cpu().numpy(), s)
    cache.close()
