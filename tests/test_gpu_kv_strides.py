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


def tokens_first(c, pad):
    """The case's cache as the two halves of one tensor, tokens before heads,
    rows and pages with room between them."""
    import torch
    pages, heads, page, dim = c["k"].shape
    both = torch.full((pages, 2, page, heads, dim + pad), 77, dtype=torch.int8, device="cuda")
    sc = torch.full((2, pages, heads + 3), float("nan"), device="cuda")
    got = [both[:, i, :, :, :dim].transpose(1, 2) for i in range(2)] + [sc[i, :, 2:2 + heads] for i in range(2)]
    for t, n in zip(got, ("k", "v", "ks", "vs")):
        t.copy_(dev(c[n]))
    return got


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("heads,kvh,dim,page,pad", [(4, 4, 64, 16, 0), (16, 2, 128, 64, 16), (6, 2, 80, 32, 0),
                                                    (6, 3, 256, 128, 32), (40, 8, 128, 16, 0), (1, 1, 96, 16, 16)])
@pytest.mark.parametrize("lens", [[(70, 1), (0, 1), (700, 1)], [(64, 5), (3, 2)], [(100, 200), (50, 1), (0, 129)],
                                  [(900, 400)]])
def test_attention_and_read_of_a_strided_cache(heads, kvh, dim, page, pad, lens, dtype):
    import torch
    c = case(lens, heads, kvh, dim, page, getattr(torch, dtype), 81)
    want, wl = run(c)
    t = tokens_first(c, pad)
    got, gl = run(c, tensors=t)
    assert torch.equal(got, want) and torch.equal(gl, wl)
    cache, plain = bsp.KvCache(*t), bsp.KvCache(*[dev(c[n]) for n in ("k", "v", "ks", "vs")])
    slots = torch.arange(-2, c["k"].shape[0] * page + 3, device="cuda")
    for a, b in zip(cache.read(slots, dtype=c["q"].dtype), plain.read(slots, dtype=c["q"].dtype)):
        assert torch.equal(a, b)
    cache.close()
    plain.close()
