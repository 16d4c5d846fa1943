"""The paged 8-bit KV cache on the GPU: plan, append and read against the
plain definitions bit for bit."""
import numpy as np
import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from oracle import kv_cache as kv

pytestmark = pytest.mark.gpu


def dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def table_of(counts, spare, g, width=None):
    """Block table of scattered pages and the pages left over."""
    pool = g.permutation(int(sum(counts)) + spare)
    width = width or max(1, max(counts, default=1))
    table, at = np.full((len(counts), width), -1, np.int32), 0
    for b, n in enumerate(counts):
        table[b, :n] = pool[at:at + n]
        at += n
    return table, pool[at:].astype(np.int32), len(pool)


# ---------------------------------------------------------------------- plan

def run_plan(ctx, new, table, free, capacity, tokens, page, in_place=False):
    import torch
    cache = bsp.KvCache.empty(4, 1, 16, page)
    stack = np.full(capacity, -7, np.int32)
    stack[:len(free)] = free
    t, f = dev(table), dev(stack)
    count = torch.tensor([len(free)], dtype=torch.int32, device="cuda")
    step = bsp.KvStep.empty(len(ctx), tokens, free_count=count if in_place else None)
    cache.plan(dev(np.array(ctx, np.int32)), dev(np.array(new, np.int32)), t, f, count, tokens, out=step)
    torch.cuda.synchronize()
    want = kv.plan(ctx, new, table, stack, len(free), tokens, page)
    for name in ("granted", "seq_len", "q_start", "slots", "positions"):
        assert np.array_equal(getattr(step, name).cpu().numpy(), want[name]), name
    assert np.array_equal(t.cpu().numpy(), want["block_table"])
    assert np.array_equal(f.cpu().numpy(), want["free_list"])
    assert int(step.free_count) == want["free_count"]
    if not in_place:
        assert int(count) == len(free)
    cache.close()
    return want


@pytest.mark.parametrize("batch,page,spare,slack", [
    (1, 16, 3, 0), (2, 64, 0, 0), (31, 16, 40, 5), (33, 128, 9, 0), (513, 32, 300, 17), (1500, 16, 4000, 0),
    (1500, 16, 700, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_random(batch, page, spare, slack, in_place):
    g = np.random.default_rng(batch * 31 + spare)
    ctx = g.integers(0, 12 * page, batch)
    new = np.where(g.random(batch) < 0.3, g.integers(0, 3 * page, batch), 1)
    new[g.random(batch) < 0.15] = -1
    new[g.random(batch) < 0.1] = 0
    table, free, total = table_of([kv.pages_of(c, page) for c in ctx], spare, g, width=13)
    run_plan(ctx, new, table, free, total, int(np.maximum(new, 0).sum()) + slack, page, in_place)


def test_plan_edges():
    g = np.random.default_rng(5)
    table, free, total = table_of([2, 1, 3], 2, g, width=4)
    run_plan([20, 16, 40], [-1, -1, -1], table, free, total, 0, 16)          # everything ends, no rows
    run_plan([20, 16, 40], [0, 0, 0], table, free, total, 5, 16)             # nothing asked
    run_plan([20, 16, 40], [1, 1, 25], table, free, total, 27, 16)           # outgrows its row
    run_plan([20, 16, 40], [12, 1, 1], table, free, total, 13, 16)           # the row capacity ends it
    run_plan([20, 16, 40], [-1, 40, 1], table, free[:0], total, 41, 16)      # only what comes back, in the same step
    run_plan([0], [5], np.full((1, 1), -1, np.int32), [0], 1, 5, 16)
    w = run_plan([0], [17], np.full((1, 2), -1, np.int32), [0], 1, 17, 16)   # one page short
    assert w["granted"].tolist() == [0]


def test_plan_stack_smaller_than_what_comes_back():
    # a stack that cannot hold every returned page keeps what fits
    table = np.array([[3, 4, 5], [6, 7, -1]], np.int32)
    run_plan([48, 20], [-1, -1], table, [1], 3, 1, 16)


def test_plan_empty_batch():
    import torch
    cache = bsp.KvCache.empty(2, 1, 16, 16)
    table = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    stack = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    count = torch.tensor([2], dtype=torch.int32, device="cuda")
    step = cache.plan(none, none, table, stack, count, tokens=3)
    assert step.q_start.tolist() == [0] and step.slots.tolist() == [-1] * 3 and step.free_count.tolist() == [2]
    cache.close()


# -------------------------------------------------------------- append, read

def make_cache(pages, heads, page, dim, g, scale=0.02):
    k = g.integers(-127, 128, (pages, heads, page, dim)).astype(np.int8)
    v = g.integers(-127, 128, (pages, heads, page, dim)).astype(np.int8)
    ks = (scale * np.exp(0.5 * g.standard_normal((pages, heads)))).astype(np.float32)
    vs = (scale * np.exp(0.5 * g.standard_normal((pages, heads)))).astype(np.float32)
    return k, v, ks, vs


def check_append(lens, heads, dim, page, dtype, g, strided=False, drop=False, size=1.0, touch=None, spread=False):
    import torch
    ctx, new = [c for c, _ in lens], [n for _, n in lens]
    table, _, total = table_of([kv.pages_of(c + n, page) for c, n in lens], 2, g)
    if drop:
        table[g.random(table.shape) < 0.3] = -1
        table[0, 0] = total + 5
    k, v, ks, vs = make_cache(total, heads, page, dim, g)
    rows = sum(new)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    seq = np.array(ctx, np.int32) + np.array(new, np.int32)
    if strided:  # K and V as views of one projection output with rows to spare
        buf = torch.from_numpy((size * g.standard_normal((rows + 3, 4, heads, dim))).astype(np.float32)).cuda().to(dtype)
        kn, vn = buf[:, 1], buf[:, 3]
    else:
        kn = dev((size * g.standard_normal((rows, heads, dim))).astype(np.float32), dtype)
        vn = dev((0.3 * size * g.standard_normal((rows, heads, dim))).astype(np.float32), dtype)
    if spread:
        kn *= torch.exp(3 * torch.randn(kn.shape[0], 1, 1, device="cuda")).to(dtype)
    if touch:
        touch(kn)
    tensors = [dev(a) for a in (k, v, ks, vs)]
    cache = bsp.KvCache(*tensors)
    step = bsp.KvStep(dev(table), dev(seq), dev(start), max_new=max(new))
    cache.append(step, kn, vn)
    torch.cuda.synchronize()
    for codes, scale, x, got_c, got_s in ((k, ks, kn, tensors[0], tensors[2]), (v, vs, vn, tensors[1], tensors[3])):
        want_c, want_s = kv.append(codes, scale, x.float().cpu().numpy(), table, seq, start, page)
        assert np.array_equal(got_s.cpu().numpy(), want_s)
        assert np.array_equal(got_c.cpu().numpy(), want_c)
    cache.close()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("heads,dim,page", [(1, 16, 16), (3, 64, 16), (40, 128, 16), (8, 128, 64), (2, 80, 32),
                                            (5, 96, 128), (2, 256, 256), (1, 240, 64)])
def test_append_matches_definition(heads, dim, page, dtype):
    import torch
    g = np.random.default_rng(heads * dim + page)
    lens = [(0, 1), (page - 1, 2), (5, 0), (page, page), (3 * page + 7, 1), (1, 2 * page + 3), (0, page - 1)]
    check_append(lens, heads, dim, page, getattr(torch, dtype), g)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_append_strided_rows_and_spare_rows(dtype):
    import torch
    g = np.random.default_rng(8)
    check_append([(3, 9), (0, 40), (31, 1)], 3, 48, 16, getattr(torch, dtype), g, strided=True)


def test_append_drops_rows_without_a_page():
    import torch
    check_append([(3, 90), (0, 40), (31, 1), (5, 5)], 2, 64, 16, torch.float16, np.random.default_rng(9), drop=True)


def test_append_more_rows_than_length():
    import torch
    g = np.random.default_rng(13)
    k, v, ks, vs = make_cache(6, 2, 16, 32, g)
    table = np.array([[0, 4], [5, 2], [1, 3]], np.int32)
    seq, start = np.array([0, 3, 20], np.int32), np.array([0, 2, 9, 20], np.int32)
    x = dev(g.standard_normal((20, 2, 32)).astype(np.float16))
    t = [dev(a) for a in (k, v, ks, vs)]
    cache = bsp.KvCache(*t)
    cache.append(bsp.KvStep(dev(table), dev(seq), dev(start)), x, x)
    c, s = kv.append(k, ks, x.float().cpu().numpy(), table, seq, start, 16)
    assert np.array_equal(t[0].cpu().numpy(), c) and np.array_equal(t[2].cpu().numpy(), s)
    cache.close()


def test_append_scales_that_differ_widely():
    import torch
    g = np.random.default_rng(10)
    check_append([(7, 30), (60, 1), (61, 1), (62, 2)], 4, 64, 64, torch.float16, g, spread=True)
    check_append([(7, 30), (60, 1)], 4, 64, 64, torch.float16, g, size=1e-6)  # subnormal rows


def test_append_non_finite_and_zero_rows():
    import torch

    def touch(x):
        x[0] = float("nan")
        x[1, 0, 3] = float("inf")
        x[1, 1] = float("-inf")
        x[2] = 0
        x[3:20, 1] = 0
    check_append([(5, 1), (7, 1), (16, 3), (0, 16), (40, 2)], 2, 32, 16, torch.float16, np.random.default_rng(11),
                 touch=touch)


def test_append_empty_calls():
    import torch
    cache = bsp.KvCache.empty(2, 2, 32, 16)
    z = torch.zeros((0, 2, 32), dtype=torch.float16, device="cuda")
    step = bsp.KvStep(torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                      torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"))
    cache.append(step, z, z)
    out, lse = cache.attention(step, z, with_lse=True)
    assert out.shape == (0, 2, 32) and lse.shape == (0, 2)
    k, v = cache.read(torch.zeros(0, dtype=torch.int64, device="cuda"))
    assert k.shape == (0, 2, 32)
    cache.close()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("heads,dim,page,n", [(1, 16, 16, 1), (3, 80, 32, 77), (40, 128, 16, 1000), (2, 256, 256, 515)])
def test_read_matches_definition(heads, dim, page, n, dtype):
    import torch
    g = np.random.default_rng(n)
    pages = 9
    k, v, ks, vs = make_cache(pages, heads, page, dim, g)
    slots = g.integers(-3, pages * page + 5, n)
    cache = bsp.KvCache(dev(k), dev(v), dev(ks), dev(vs))
    dt = getattr(torch, dtype)
    got = cache.read(dev(slots), dtype=dt)
    for codes, scale, x in ((k, ks, got[0]), (v, vs, got[1])):
        # fp32 product rounded once: the definition in fp32, bit for bit
        p, off = np.clip(slots // page, 0, pages - 1), slots % page
        w = codes[p, :, off].astype(np.float32) * scale[p][:, :, None]
        w[(slots < 0) | (slots >= pages * page)] = 0
        assert torch.equal(x, dev(w, dt))
        ref = kv.read(codes, scale, slots, page)
        assert np.allclose(x.float().cpu().numpy(), ref, rtol=2 ** -7 if dtype == "bfloat16" else 2 ** -10, atol=1e-6)
    cache.close()


def test_strided_cache():
    """K and V as the two halves of one tensor, tokens before heads."""
    import torch
    g = np.random.default_rng(12)
    pages, heads, page, dim = 7, 3, 16, 32
    both = torch.zeros((pages, 2, page, heads, dim), dtype=torch.int8, device="cuda")
    sc = torch.zeros((2, pages, 5), dtype=torch.float32, device="cuda")
    cache = bsp.KvCache(both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2), sc[0, :, :heads], sc[1, :, :heads])
    x = g.standard_normal((2, 50, heads, dim)).astype(np.float16)
    table = np.array([[4, 0, 6, 2]], np.int32)
    step = bsp.KvStep(dev(table), dev(np.array([50], np.int32)), dev(np.array([0, 50], np.int32)))
    cache.append(step, dev(x[0]), dev(x[1]))
    z = np.zeros((pages, heads, page, dim), np.int8), np.zeros((pages, heads), np.float32)
    for i, got in ((0, cache.k), (1, cache.v)):
        c, s = kv.append(*z, x[i].astype(np.float32), table, [50], [0, 50], page)
        assert np.array_equal(got.cpu().numpy(), c)
        assert np.array_equal(sc[i, :, :heads].cpu().numpy(), s)
    assert (sc[:, :, heads:] == 0).all()
    cache.close()


# ------------------------------------------------------------------ refusals

def test_refusals():
    import torch
    L = bsp.lib()
    cache = bsp.KvCache.empty(8, 2, 64, 16)
    i32 = dict(dtype=torch.int32, device="cuda")
    table, seq, start = torch.zeros((1, 4), **i32), torch.tensor([5], **i32), torch.tensor([0, 5], **i32)
    step = bsp.KvStep(table, seq, start)
    x = torch.zeros((5, 2, 64), dtype=torch.float16, device="cuda")
    with pytest.raises(TypeError):
        cache.append(step, x.float(), x.float())
    with pytest.raises(ValueError):
        cache.append(step, x, x.bfloat16())
    with pytest.raises(ValueError):
        cache.append(step, x[:, :1], x[:, :1])
    with pytest.raises(ValueError):
        cache.attention(step, x[..., :32])
    with pytest.raises(ValueError):
        cache.read(torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        bsp.KvStep(table, seq, start[:1])
    with pytest.raises(ValueError):
        bsp.KvStep(table.long(), seq, start)
    for bad in (dict(window=-1), dict(scale=float("nan")), dict(scale=-1.0)):
        with pytest.raises(bsp.BspError) as e:
            cache.attention(step, x, **bad)
        assert e.value.status == 1
    with pytest.raises(bsp.BspError) as e:  # 3 heads over 2 KV heads
        cache.attention(step, torch.zeros((5, 3, 64), dtype=torch.float16, device="cuda"))
    assert e.value.status == 2
    wide = torch.zeros((5, 2, 68), dtype=torch.float16, device="cuda")
    with pytest.raises(bsp.BspError) as e:  # rows that do not start on 16 bytes
        cache.append(step, wide[..., :64], wide[..., :64])
    assert e.value.status == 2
    flat = torch.zeros(5 * 128 + 4, dtype=torch.float16, device="cuda")[4:].view(5, 2, 64)
    with pytest.raises(bsp.BspError) as e:
        cache.attention(step, flat)
    assert e.value.status == 4
    p = x.data_ptr()
    assert L.bsp_kv_attention(cache.h, step._ref, p, 1, 5, 2, 128, 64, 1.0, 0, p, 128, 64, None, None) == 3  # int8
    assert L.bsp_kv_attention(cache.h, None, p, 0, 5, 2, 128, 64, 1.0, 0, p, 128, 64, None, None) == 1
    assert L.bsp_kv_attention(cache.h, step._ref, None, 0, 5, 2, 128, 64, 1.0, 0, p, 128, 64, None, None) == 1
    assert L.bsp_kv_read(cache.h, p, -1, p, p, 0, None) == 1
    narrow = bsp.bsp_kv_step_t(1, 4, 3, table.data_ptr(), seq.data_ptr(), start.data_ptr(), 0)
    import ctypes
    assert L.bsp_kv_append(cache.h, ctypes.addressof(narrow), p, p, 0, 5, 128, 64, 128, 64, None) == 2
    big = bsp.bsp_kv_step_t(bsp.BSP_KV_MAX_BATCH + 1, 4, 4, table.data_ptr(), seq.data_ptr(), start.data_ptr(), 0)
    assert L.bsp_kv_append(cache.h, ctypes.addressof(big), p, p, 0, 5, 128, 64, 128, 64, None) == 1
    cache.check()
    cache.close()
    with pytest.raises(bsp.BspError):
        cache.read(torch.zeros(1, dtype=torch.int64, device="cuda"))
