"""Outputs that a call given a stream of its own allocates: not in memory that the current stream still uses."""
import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from test_gpu_explicit_streams import busy

pytestmark = pytest.mark.gpu


def outputs(y):
    import torch
    return [y] if torch.is_tensor(y) else [t for t in y if t is not None]


def apart(call):
    """call(stream): what was freed on the current stream is still read there, late, while the call writes on another."""
    import torch
    want = [t.clone() for t in outputs(call(None))]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    old = [torch.full_like(t, 1) for t in want for _ in range(3)]
    seen = [torch.zeros_like(t) for t in old]
    torch.cuda.synchronize()
    work = busy()
    for a, b in zip(seen, old):
        a.copy_(b)          # queued behind the work
    del a, b, old           # their memory goes back to the current stream's pool
    got = outputs(call(s))
    got += outputs(call(s.cuda_stream))
    torch.cuda.synchronize()
    for t in seen:
        assert torch.all(t == 1)
    for t, w in zip(got, want + want):
        assert torch.equal(t, w)
    del work


def rand(shape, dtype, seed=1):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    if dtype is torch.int8:
        return torch.randint(-7, 8, shape, device="cuda", generator=g, dtype=torch.int8)
    return torch.randn(shape, device="cuda", generator=g).to(dtype)


def test_int4():
    import torch
    m = bsp.Int4Matrix(rand((2048, 1024), torch.float16), group=64, zeros=True)
    u = bsp.Int4Matrix(rand((2048, 1024), torch.float16, 2), group=64)
    for n in (600, 16):
        x = rand((n, 1024), torch.float16, 3)
        apart(lambda s: m.mm(x, stream=s))
        apart(lambda s: m.gated(u, x, stream=s))
    apart(lambda s: m.decode(stream=s))
    apart(lambda s: m.arrays(stream=s))
    m.close()
    u.close()


def test_rotary():
    import torch
    r = bsp.Rotary(128)
    q, k = rand((3000, 8, 128), torch.bfloat16), rand((3000, 2, 128), torch.bfloat16, 2)
    p = torch.arange(3000, dtype=torch.int32, device="cuda")
    apart(lambda s: r.apply(q, k, p, stream=s))
    r.close()


def test_pruned_formats():
    import torch
    W = torch.where(rand((2048, 2048), torch.float16) > 0, rand((2048, 2048), torch.float16, 2), 0).half()
    A, B = bsp.BitmapMatrix(W), bsp.BitmapMatrix((W * 3).clamp(-7, 7).to(torch.int8))
    A.set_deterministic(True)
    x, v = rand((700, 2048), torch.float16, 3), rand((2048,), torch.float16, 4)
    apart(lambda s: A.spmm(x, stream=s))
    apart(lambda s: A.spmm(x[:8].contiguous(), stream=s))
    apart(lambda s: A.spmspv(v, stream=s))
    apart(lambda s: A.spmspv_threshold(v, 0.1, stream=s))
    apart(lambda s: A.decode(stream=s))
    apart(lambda s: A.arrays(stream=s))
    x8, scale = rand((16, 2048), torch.int8, 5), rand((2048,), torch.float32, 6)
    apart(lambda s: B.spmm(x8, stream=s))
    apart(lambda s: B.spmm_scaled(x8, scale, stream=s))
    A.build_column_index()
    apart(lambda s: A.column_index_arrays(stream=s))
    U = bsp.UnionMatrix(rand((1024, 1024), torch.int8, 7), 4, reorder=True)
    xu = rand((16, 1024), torch.int8, 8)
    apart(lambda s: U.spmm(xu, stream=s))
    apart(lambda s: U.decode(stream=s))
    apart(lambda s: U.arrays(stream=s))
    apart(lambda s: U.perms(stream=s))
    for m in (A, B, U):
        m.close()


def test_cache():
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = bsp.KvCache.empty(64, 2, 128, 64)
    table, new = torch.full((2, 16), -1, **i32), torch.tensor([700, 300], **i32)
    ctx, free, count = torch.zeros(2, **i32), torch.arange(64, **i32), torch.tensor([64], **i32)

    tables = iter([torch.full_like(table, -1) for _ in range(3)])  # a plan writes into its own

    def plan(s):
        step = cache.plan(ctx, new, next(tables), free, count, tokens=1000, max_new=700, stream=s)
        return step.slots, step.positions, step.seq_len, step.q_start, step.granted, step.free_count

    apart(plan)
    step = cache.plan(ctx, new, table, free, count, tokens=1000, max_new=700)
    k, v, q = rand((1000, 2, 128), torch.float16, 1), rand((1000, 2, 128), torch.float16, 2), rand((1000, 8, 128), torch.float16, 3)
    cache.append(step, k, v)
    torch.cuda.synchronize()
    apart(lambda s: cache.attention(step, q, with_lse=True, stream=s))
    apart(lambda s: cache.read(step.slots, stream=s))
    cache.check()
    cache.close()

