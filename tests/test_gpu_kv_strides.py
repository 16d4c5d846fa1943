"""Layouts of the paged 8-bit KV cache's tensors beyond the contiguous ones."""
import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from test_gpu_kv_attention import case, run
from test_gpu_kv_cache import dev

pytestmark = pytest.mark.gpu


def step_of(c):
    return bsp.KvStep(dev(c["table"]), dev(c["seq"]), dev(c["start"]), c["max_new"])


@pytest.mark.parametrize("lens,heads,kvh", [([(70, 1)], 4, 2), ([(70, 5), (30, 1)], 1, 1), ([(90, 700)], 2, 1), ([(0, 1)], 1, 1)])
def test_strides_that_are_not_used(lens, heads, kvh):
    """One row, one head or one page: what their strides say does not matter."""
    import torch
    c = case(lens, heads, kvh, 64, 16, torch.float16, 80)
    want, wl = run(c)
    rows = c["q"].shape[0]

    def odd(t):
        s = [3 if n == 1 else k for n, k in zip(t.shape, t.stride())]
        return t.as_strided(t.shape, s)
    one = [odd(dev(c[n])) for n in ("k", "v", "ks", "vs")]
    cache, step = bsp.KvCache(*one), step_of(c)
    out = torch.empty((rows, heads, 64), dtype=torch.float16, device="cuda")
    got, gl = cache.attention(step, odd(c["q"]), out=odd(out), with_lse=True)
    assert torch.equal(got, want) and torch.equal(gl, wl)
    x = torch.randn((rows, kvh, 64), device="cuda").half()
    cache.append(step, odd(x), odd(x))
    plain = bsp.KvCache(*[dev(c[n]) for n in ("k", "v", "ks", "vs")])
    plain.append(step, x, x)
    assert torch.equal(cache.k, plain.k) and torch.equal(cache.v_scale, plain.v_scale)
    cache.close()
    plain.close()


def test_one_page_cache_with_any_page_stride():
    import torch
    k = torch.zeros((1, 1, 16, 32), dtype=torch.int8, device="cuda").as_strided((1, 1, 16, 32), (5, 7, 32, 1))
    s = torch.ones((1, 1), device="cuda").as_strided((1, 1), (0, 9))
    cache = bsp.KvCache(k, k.clone().as_strided(k.shape, k.stride()), s, s.clone().as_strided((1, 1), (0, 9)))
    a, b = cache.read(torch.arange(16, device="cuda"))
    assert a.shape == (16, 1, 32) and (a == 0).all() and (b == 0).all()
    cache.close()
