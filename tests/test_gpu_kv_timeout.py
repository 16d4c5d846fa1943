"""Waits of the KV attention kernels that run out, in the test build of the
library: the kernel drains its copies and returns, the error word says so once,
and the next call on the same handle is right."""
import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from test_gpu_kv_attention import case, check, run
from test_gpu_kv_cache import dev

pytestmark = pytest.mark.gpu


def time_out(lens, heads, kvh, dim, page, dtype):
    import torch
    c = case(lens, heads, kvh, dim, page, getattr(torch, dtype), 17 + dim)
    want = run(c)
    with bsp.test_library() as T:
        cache = bsp.KvCache(*[dev(c[n]) for n in ("k", "v", "ks", "vs")])
        step = bsp.KvStep(dev(c["table"]), dev(c["seq"]), dev(c["start"]), c["max_new"])
        for _ in range(2):
            try:
                assert T.bsp_testing_set_stall(1) == 0 and T.bsp_testing_set_spin_cap(2000) == 0
                cache.attention(step, c["q"])
                with pytest.raises(bsp.BspError) as e:
                    cache.check()
                assert e.value.status == 7
            finally:
                T.bsp_testing_set_stall(0)
                T.bsp_testing_set_spin_cap(0)
            cache.check()  # cleared
            out, lse = cache.attention(step, c["q"], with_lse=True)
            cache.check()
            check(c, out, lse)
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        cache.close()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("lens,heads,kvh,dim,page", [
    ([(516, 1)], 40, 40, 128, 16),                       # one stream
    ([(900, 1), (0, 1), (31, 1), (5000, 1)], 8, 2, 64, 32),
    ([(3000, 5), (1, 5)], 8, 2, 128, 64),                # queries in shared memory
    ([(700, 3), (60, 20)], 4, 2, 256, 16)])
def test_few_queries(lens, heads, kvh, dim, page, dtype):
    time_out(lens, heads, kvh, dim, page, dtype)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("lens,heads,kvh,dim,page", [
    ([(0, 40), (0, 100)], 16, 4, 64, 16),                # one or two row tiles, one tile of codes
    ([(0, 900)], 8, 2, 128, 64),                         # cached rows split, and joined
    ([(300, 200), (64, 1), (0, 90)], 64, 8, 128, 32)])   # beside single tokens
def test_prompts(lens, heads, kvh, dim, page, dtype):
    time_out(lens, heads, kvh, dim, page, dtype)
