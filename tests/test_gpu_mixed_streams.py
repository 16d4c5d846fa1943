"""The tensor-memory kernels of all formats at once, each on a stream of its own: what they share is the SMs alone."""
import pytest

import bitmap_encoded_unstructured_gb300 as bsp

pytestmark = pytest.mark.gpu


def cached(new, heads, kv, dim):
    """A cache with one step of `new` rows a request appended, its step and queries."""
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    cache = bsp.KvCache.empty(64, kv, dim, 64)
    table = torch.full((len(new), 40), -1, **i32)
    step = cache.plan(torch.zeros(len(new), **i32), torch.tensor(new, **i32), table, torch.arange(64, **i32),
                      torch.tensor([64], **i32), tokens=sum(new), max_new=max(new))
    k, v = (torch.randn((sum(new), kv, dim), device="cuda", generator=g).half() for _ in range(2))
    cache.append(step, k, v)
    return cache, step, torch.randn((sum(new), heads, dim), device="cuda", generator=g).half()


def test_products_and_attention_at_once():
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)

    def rand(*shape):
        return torch.randn(shape, device="cuda", generator=g).half()

    W = torch.where(torch.rand((4096, 2048), device="cuda", generator=g) < 0.5, rand(4096, 2048), 0).half()
    A = bsp.BitmapMatrix(W)
    A.set_deterministic()
    # one matrix a stream where a handle has a workspace (the pruned ones)
    B = bsp.BitmapMatrix(W)
    B.set_deterministic()
    m, u = bsp.Int4Matrix(rand(4096, 2048), group=64, zeros=True), bsp.Int4Matrix(rand(4096, 2048), group=64)
    cache, step, q = cached([900, 300], 16, 4, 128)
    r, pos = bsp.Rotary(128), torch.arange(2000, dtype=torch.int32, device="cuda")
    x, few, some, t = rand(700, 2048), rand(8, 2048), rand(60, 2048), rand(2000, 8, 128)
    work = [lambda: [m.mm(x), m.gated(u, some), m.mm(few)],
            lambda: [A.spmm(x), A.spmm(some)],
            lambda: [B.spmm(few), B.spmm(few)],
            lambda: [cache.attention(step, q)],
            lambda: [u.mm(some), u.gated(m, x), r.apply(t, None, pos)]]
    want = [f() for f in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(15):
        got = [[] for _ in work]
        for _ in range(4):
            for i, f in enumerate(work):
                with torch.cuda.stream(streams[i]):
                    got[i].append(f())
        torch.cuda.synchronize()
        for i, (calls, right) in enumerate(zip(got, want)):
            for outs in calls:
                assert all(torch.equal(a, b) for a, b in zip(outs, right)), i
    for h in (A, B, m, u, cache):
        h.check()
        h.close()
    r.close()
