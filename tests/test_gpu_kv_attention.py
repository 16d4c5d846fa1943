"""Attention over the paged 8-bit KV cache against the 64-bit definition.

The bound of an output element, from the arithmetic that include/bsp.h
states (u = 2^-11 for float16 and 2^-8 for bfloat16 outputs):
* a logit is an fp32 sum of dim exact products, off by at most
  d = dim 2^-23 scale sum |q k| (one truncation per addition) plus a few ulp
  of its own scaling, so p is off by a relative 2 d + 2^-20 against the sum;
* p times its V scale is rounded to fp16: 2^-11 relative, or 2^-24 of the
  largest V where it is subnormal;
* the output is rounded once: u relative.
"""
import numpy as np
import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from oracle import kv_cache as kv
from test_gpu_kv_cache import dev, make_cache, table_of

pytestmark = pytest.mark.gpu

U = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}


def case(lens, heads, kv_heads, dim, page, dtype, seed, q_size=1.5):
    """Numpy arrays of a step: [(cached, new)] lengths."""
    g = np.random.default_rng(seed)
    table, _, total = table_of([kv.pages_of(c + n, page) for c, n in lens], 1, g)
    k, v, ks, vs = make_cache(total, kv_heads, page, dim, g)
    new = [n for _, n in lens]
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    seq = np.array([c + n for c, n in lens], np.int32)
    q = dev((q_size * g.standard_normal((sum(new), heads, dim))).astype(np.float32)).to(dtype)
    return dict(q=q, k=k, v=v, ks=ks, vs=vs, table=table, seq=seq, start=start, page=page, max_new=max(new))


def check(c, out, lse, window=0, scale=None, what=""):
    dim = c["q"].shape[2]
    scale = dim ** -0.5 if scale is None else scale
    q = c["q"].float().cpu().numpy()
    n = int(c["start"][-1])
    ref, rl, weight, spread, seen = kv.attention(q, c["k"], c["v"], c["ks"], c["vs"], c["table"], c["seq"], c["start"],
                                                 c["page"], scale, window)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    empty = np.isneginf(rl)
    assert (np.isneginf(gl) == empty).all(), what
    assert (got[empty] == 0).all(), what
    vmax = 127 * np.nanmax(np.where(np.isfinite(c["vs"]), c["vs"], 0))
    d = dim * 2.0 ** -23 * spread[..., None] + 2.0 ** -20
    u = U[str(c["q"].dtype).split(".")[1]]
    bound = u * np.abs(ref) + (2 * d + 2.0 ** -11) * weight + seen[..., None] * 2.0 ** -24 * vmax + 1e-7
    off = np.abs(got - ref)
    assert np.isfinite(got).all(), what
    assert (off <= bound).all(), f"{what}: {(off / bound).max():.3g} of the bound at {np.argmax((off / bound))}"
    dl = np.abs(np.where(empty, 0, gl) - np.where(empty, 0, rl))
    bl = d[..., 0] + 2.0 ** -20 * (1 + np.where(empty, 0, np.abs(rl)))
    assert (dl <= bl).all(), f"{what}: lse {(dl / bl).max():.3g} of the bound"
    assert (got[n:] == 0).all()


def run(c, window=0, scale=None, max_new=None, tensors=None):
    t = tensors or [dev(c[n]) for n in ("k", "v", "ks", "vs")]
    cache = bsp.KvCache(*t)
    step = bsp.KvStep(dev(c["table"]), dev(c["seq"]), dev(c["start"]), c["max_new"] if max_new is None else max_new)
    out, lse = cache.attention(step, c["q"], scale=scale, window=window, with_lse=True)
    cache.check()
    cache.close()
    return out, lse


SHAPES = [  # heads, KV heads, dim, page
    (1, 1, 16, 16), (4, 4, 64, 16), (40, 40, 128, 16), (8, 1, 128, 64), (16, 2, 128, 128), (6, 2, 80, 32),
    (5, 1, 96, 16), (4, 2, 256, 64), (2, 2, 240, 256), (12, 4, 112, 32), (33, 1, 64, 64), (64, 4, 128, 32)]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_single_tokens(shape, dtype):
    import torch
    heads, kvh, dim, page = shape
    lens = [(0, 1), (1, 1), (15, 1), (16, 1), (63, 1), (64, 1), (65, 1), (200, 1), (page * 5 - 1, 1), (777, 1)]
    c = case(lens, heads, kvh, dim, page, getattr(torch, dtype), heads + dim)
    check(c, *run(c))


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_several_tokens(shape, dtype):
    import torch
    heads, kvh, dim, page = shape
    lens = [(0, 3), (7, 2), (100, 5), (64, 4), (130, 1), (3, 0)]
    c = case(lens, heads, kvh, dim, page, getattr(torch, dtype), heads + dim + 1)
    check(c, *run(c))


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_prompts(shape, dtype):
    import torch
    heads, kvh, dim, page = shape
    lens = [(0, 131), (50, 70), (0, 1), (300, 17), (9, 0), (127, 129)]
    c = case(lens, heads, kvh, dim, page, getattr(torch, dtype), heads + dim + 2)
    check(c, *run(c))


@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 128, 5000])
@pytest.mark.parametrize("new", [1, 6, 150])
def test_window(window, new):
    import torch
    c = case([(0, new), (40, new), (333, new), (1000, 1)], 8, 2, 64, 16, torch.float16, window + new)
    check(c, *run(c, window=window), window=window)


@pytest.mark.parametrize("new", [1, 5, 90])
def test_long_context(new):
    """Work split along the cached rows and joined."""
    import torch
    c = case([(9001, new), (17, new), (4093, 1)], 4, 2, 128, 64, torch.bfloat16, new)
    check(c, *run(c))


def test_mixed_lengths_in_one_step():
    import torch
    lens = [(500, 1)] * 3 + [(100, 200)] + [(37, 1), (0, 40), (900, 2)]
    c = case(lens, 8, 4, 128, 32, torch.float16, 77)
    check(c, *run(c))
    check(c, *run(c, max_new=0), what="bound not known")


@pytest.mark.parametrize("new", [1, 4, 70])
def test_missing_pages_leave_rows_empty(new):
    import torch
    c = case([(60, new), (0, new), (200, new), (31, new)], 4, 2, 64, 16, torch.float16, 5 + new)
    g = np.random.default_rng(new)
    c["table"][0, :] = -1                                  # nothing left
    c["table"][2, g.random(c["table"].shape[1]) < 0.5] = -1
    c["table"][3, 0] = 1 << 30                             # not a page
    check(c, *run(c))


@pytest.mark.parametrize("new", [1, 4, 70, 90])
def test_more_rows_than_length(new):
    """Idle requests of a padded batch: rows whose position is negative see nothing."""
    import torch
    c = case([(60, new), (0, new), (0, new), (9, new)], 4, 2, 64, 16, torch.float16, 6 + new)
    c["seq"][1] = 0
    c["seq"][2] = new // 2
    out, lse = run(c)
    check(c, out, lse)
    assert torch.isneginf(lse[new:2 * new]).all()


@pytest.mark.parametrize("new", [1, 4, 70, 120])
def test_unseen_rows_do_not_matter(new):
    """Garbage in rows and scales that no query sees changes nothing, bit for bit."""
    import torch
    c = case([(60, new), (9, new), (400, new)], 4, 2, 64, 16, torch.float16, 9 + new)
    window = 40
    out, lse = run(c, window=window)
    check(c, out, lse, window=window)
    for b in range(3):
        n = int(c["start"][b + 1] - c["start"][b])
        first = max(0, int(c["seq"][b]) - n - window + 1)
        for j in range(kv.pages_of(int(c["seq"][b]), 16)):
            p = c["table"][b, j]
            if (j + 1) * 16 <= first:                      # a page wholly outside
                c["ks"][p], c["vs"][p] = np.nan, np.inf
                c["k"][p], c["v"][p] = 127, -128
            for i in range(16):
                if j * 16 + i < first or j * 16 + i >= c["seq"][b]:
                    c["k"][p, :, i], c["v"][p, :, i] = 127, -127
    spare = set(range(len(c["ks"]))) - set(int(p) for p in c["table"].ravel())
    for p in spare:
        c["ks"][p] = c["vs"][p] = np.nan
    out2, lse2 = run(c, window=window)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("new", [1, 40, 200])
def test_extreme_scales(new):
    """Sharp and flat rows, V scales that span many powers of two, zero scales."""
    import torch
    c = case([(300, new), (70, new)], 4, 2, 64, 16, torch.float16, 21, q_size=20.0)
    g = np.random.default_rng(3)
    c["vs"][:] = np.exp2(g.integers(-12, 6, c["vs"].shape)).astype(np.float32)
    c["ks"][::3] = 0
    check(c, *run(c), what="wide")
    c["vs"][:] = 0
    out, lse = run(c)
    assert (out == 0).all()
    c["vs"][:] = 1e-30
    out, lse = run(c)
    assert torch.isfinite(out).all() and (out == 0).all()


@pytest.mark.parametrize("new", [1, 40, 600])
def test_queries_beyond_fp16_range(new):
    """bfloat16 queries whose values fp16 does not hold."""
    import torch
    c = case([(100, new)], 2, 1, 64, 16, torch.bfloat16, 22)
    for f in (2.0 ** 40, 2.0 ** -40):
        d = dict(c, q=c["q"] * f)
        check(d, *run(d, scale=0.125 / f), scale=0.125 / f)


@pytest.mark.parametrize("new", [1, 3, 64, 200])
def test_strided_queries_and_outputs(new):
    import torch
    c = case([(100, new), (20, new)], 6, 2, 64, 16, torch.float16, 30 + new)
    rows = c["q"].shape[0]
    want, wl = run(c)
    wide = torch.full((rows + 2, 10, 96), 7.0, dtype=torch.float16, device="cuda")
    wide[:rows, 2:8, 16:80] = c["q"]
    to = torch.full((rows + 2, 8, 72), 5.0, dtype=torch.float16, device="cuda")
    cache = bsp.KvCache(*[dev(c[n]) for n in ("k", "v", "ks", "vs")])
    step = bsp.KvStep(dev(c["table"]), dev(c["seq"]), dev(c["start"]), new)
    out, lse = cache.attention(step, wide[:, 2:8, 16:80], out=to[:, 1:7, 8:72], with_lse=True)
    assert torch.equal(out[:rows], want) and torch.equal(lse[:rows], wl)
    assert (out[rows:] == 0).all() and torch.isneginf(lse[rows:]).all()  # rows past the step's
    to[:, 1:7, 8:72] = 5.0
    assert (to == 5.0).all()                                             # nothing written beside them
    cache.close()


@pytest.mark.parametrize("new", [1, 5, 80])
def test_same_answer_every_time(new):
    import torch
    c = case([(3000, new), (100, new), (800, new)], 8, 2, 128, 32, torch.float16, 40)
    t = [dev(c[n]) for n in ("k", "v", "ks", "vs")]
    first = run(c, tensors=t)
    for _ in range(5):
        again = run(c, tensors=t)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("lens,heads,kvh,window", [
    ([(0, 1100)], 4, 4, 0), ([(5000, 300)], 8, 1, 0), ([(3000, 140), (2, 150)], 8, 2, 100), ([(64, 1), (1000, 260)], 8, 2, 0)])
def test_prompts_shared_by_several_blocks(lens, heads, kvh, window):
    """Few row tiles: their cached rows are split and joined."""
    import torch
    c = case(lens, heads, kvh, 128, 64, torch.bfloat16, 90)
    check(c, *run(c, window=window), window=window)


@pytest.mark.parametrize("batch", [129, 700])
def test_many_requests(batch):
    """More requests than a block has threads, some without rows."""
    import torch
    g = np.random.default_rng(batch)
    lens = [(int(g.integers(0, 90)), int(g.integers(0, 3))) for _ in range(batch)]
    c = case(lens, 4, 2, 64, 16, torch.float16, 91)
    check(c, *run(c))
    lens[3] = (10, 150)
    c = case(lens, 4, 2, 64, 16, torch.float16, 92)
    check(c, *run(c))


def test_few_streams_of_many_rows():
    """Segments cut into more parts than one warp joins."""
    import torch
    c = case([(40000, 1), (12000, 2)], 16, 1, 128, 16, torch.float16, 93)
    check(c, *run(c))


def test_other_stream_and_graph_replay_on_new_lengths():
    """A step captured once and replayed after the lengths on the device changed."""
    import torch
    g = np.random.default_rng(50)
    page, heads, kvh, dim, batch = 16, 8, 2, 64, 3
    pages = 40
    cache = bsp.KvCache.empty(pages, kvh, dim, page)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.full((batch, 12), -1, **i32)
    free = torch.arange(pages, **i32)
    count, ctx, new = torch.tensor([pages], **i32), torch.zeros(batch, **i32), torch.ones(batch, **i32)
    step = bsp.KvStep.empty(batch, 8, free_count=count)
    x = torch.zeros((3, 8, kvh, dim), dtype=torch.float16, device="cuda")
    q = torch.zeros((8, heads, dim), dtype=torch.float16, device="cuda")
    out = torch.empty_like(q)
    side = torch.cuda.Stream()

    def go():
        cache.plan(ctx, new, table, free, count, tokens=8, out=step)
        cache.append(step, x[0], x[1])
        cache.attention(step, q, out=out)
        ctx.copy_(step.seq_len)

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()  # a first call outside the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    zero = np.zeros((pages, kvh, page, dim), np.int8), np.zeros((pages, kvh), np.float32)
    ctx.zero_()
    count.fill_(pages)
    table.fill_(-1)
    free.copy_(torch.arange(pages, **i32))
    kc, ks = zero[0].copy(), zero[1].copy()
    vc, vs = zero[0].copy(), zero[1].copy()
    lens = [0] * batch
    for news in ([4, 1, 3], [1, 1, 1], [1, 5, 1], [1, 0, 1], [2, 1, 4]):
        kn, vn = (g.standard_normal((8, kvh, dim)).astype(np.float16) for _ in range(2))
        qn = g.standard_normal((8, heads, dim)).astype(np.float16)
        x[0].copy_(dev(kn)), x[1].copy_(dev(vn)), q.copy_(dev(qn))
        new.copy_(torch.tensor(news, **i32))
        graph.replay()
        torch.cuda.synchronize()
        lens = [c + n for c, n in zip(lens, news)]
        start = np.concatenate([[0], np.cumsum(news)])
        assert step.seq_len.tolist() == lens and step.q_start.tolist() == start.tolist()
        t = table.cpu().numpy()
        kc, ks = kv.append(kc, ks, kn.astype(np.float32), t, lens, start, page)
        vc, vs = kv.append(vc, vs, vn.astype(np.float32), t, lens, start, page)
        used = np.unique(t[t >= 0])
        assert np.array_equal(cache.k_scale.cpu().numpy()[used], ks[used])
        ref, _, weight, _, _ = kv.attention(qn.astype(np.float32), kc, vc, ks, vs, t, lens, start, page, dim ** -0.5)
        n = start[-1]
        off = np.abs(out.double().cpu().numpy() - ref)[:n]
        assert (off <= 2.0 ** -9 * weight[:n] + 1e-3).all()
        assert (out[n:] == 0).all()
    cache.check()
    cache.close()


def test_cache_past_32_bit_offsets():
    """Pages whose codes lie beyond 2^31 bytes (and scales in their places)."""
    import torch
    page, kvh, dim = 256, 8, 128
    pages = 2 ** 33 // (page * kvh * dim) + 9
    k = torch.zeros((pages, kvh, page, dim), dtype=torch.int8, device="cuda")
    v = torch.zeros((pages, kvh, page, dim), dtype=torch.int8, device="cuda")
    ks = torch.full((pages, kvh), 0.02, dtype=torch.float32, device="cuda")
    vs = torch.full((pages, kvh), 0.02, dtype=torch.float32, device="cuda")
    small = case([(700, 1), (300, 40)], 16, kvh, dim, page, torch.float16, 60)
    far = {}
    used = sorted(int(p) for p in set(small["table"].ravel()) if p >= 0)
    for i, p in enumerate(used):
        to = pages - 1 - i if i % 2 else 3 + i
        far[p] = to
        k[to], v[to] = dev(small["k"][p]), dev(small["v"][p])
        ks[to], vs[to] = dev(small["ks"][p]), dev(small["vs"][p])
    want = run(small)
    moved = dict(small, table=np.vectorize(lambda p: far.get(int(p), -1))(small["table"]).astype(np.int32))
    got = run(moved, tensors=[k, v, ks, vs])
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    cache = bsp.KvCache(k, v, ks, vs)
    slots = torch.tensor([(pages - 2) * page + 17, 4 * page + 3], device="cuda")
    a, b = cache.read(slots)
    assert torch.equal(a[0], (k[pages - 2, :, 17].float() * ks[pages - 2][:, None]).half())
    cache.close()
