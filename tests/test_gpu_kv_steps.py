"""Steps of the paged 8-bit KV cache one behind the other, with nothing in
between that waits for the device."""
import numpy as np
import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from oracle import kv_cache as kv
from test_gpu_kv_cache import dev

pytestmark = pytest.mark.gpu


def test_two_steps_take_turns():
    """A step's lengths are the next plan's, without a copy; the lengths and
    offsets stand beside the block table's rows, in one buffer."""
    import torch
    page, pages, batch, width = 16, 200, 7, 12
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = bsp.KvCache.empty(pages, 1, 16, page)
    buf = torch.full((batch, width + 20), -1, **i32)
    table, count = buf[:, :width], torch.tensor([pages], **i32)
    free = torch.arange(pages, **i32)
    steps = [bsp.KvStep.empty(batch, 64, free_count=count) for _ in range(2)]
    for i, s in enumerate(steps):
        s.seq_len, s.granted = buf[2 * i, width:width + batch], buf[2 * i + 1, width:width + batch]
        s._out = tuple(t.data_ptr() for t in (s.seq_len, s.q_start, s.granted, s.slots, s.positions, s.free_count))
    ctx = torch.zeros(batch, **i32)
    t, f, n, c = np.full((batch, width), -1, np.int32), np.arange(pages, dtype=np.int32), pages, [0] * batch
    g = np.random.default_rng(4)
    for i in range(9):
        new = g.integers(0, 9, batch)
        new[g.random(batch) < 0.1] = -1
        step = cache.plan(ctx, dev(new.astype(np.int32)), table, free, count, tokens=64, out=steps[i % 2])
        ctx = step.seq_len
        want = kv.plan(c, new, t, f, n, 64, page)
        t, f, n, c = want["block_table"], want["free_list"], want["free_count"], want["seq_len"]
        for name in ("granted", "seq_len", "q_start", "slots", "positions"):
            assert np.array_equal(getattr(step, name).cpu().numpy(), want[name]), name
        assert np.array_equal(table.cpu().numpy(), t) and int(count) == n
    with pytest.raises(bsp.BspError) as e:  # in place
        cache.plan(ctx, dev(new.astype(np.int32)), table, free, count, tokens=64, out=step)
    assert e.value.status == 1
    cache.close()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("heads,kvh", [(32, 8), (8, 2)])  # prompt and decode kernel side by side; one behind the other
def test_attention_sees_the_append_before_it(heads, kvh, dtype):
    """A chunk of a prompt and single tokens, step after step, into pages that
    hold earlier rows and whose scales grow: the same bits whether or not the
    host waits between the calls."""
    import torch
    dtype, page, dim, steps, chunk, streams = getattr(torch, dtype), 64, 64, 40, 130, 16
    batch = streams + 1
    counts = [kv.pages_of(chunk * steps, page)] + [kv.pages_of(200 + steps, page)] * streams
    pages = sum(counts)
    table = torch.full((batch, max(counts)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    table = table.cuda()
    g = torch.Generator(device="cuda").manual_seed(6)
    new = torch.tensor([chunk] + [1] * streams)
    start = torch.cat([torch.zeros(1, dtype=torch.long), new.cumsum(0)]).int().cuda()
    first = torch.tensor([0] + [200 - 7 * b for b in range(streams)])
    rows = int(new.sum())
    x = [[torch.randn(rows, h, dim, device="cuda", generator=g).mul_(1.15 ** i if j else 1.0).to(dtype)
          for j, h in enumerate((heads, kvh, kvh))] for i in range(steps)]
    seq = [(first + new * (i + 1)).int().cuda() for i in range(steps)]

    def go(wait):
        cache = bsp.KvCache.empty(pages, kvh, dim, page)
        cache.k_scale.fill_(0.01)
        cache.v_scale.fill_(0.01)
        got = []
        torch.cuda.synchronize()
        for (q, k, v), s in zip(x, seq):
            step = bsp.KvStep(table, s, start, max_new=chunk)
            cache.append(step, k, v)
            if wait:
                torch.cuda.synchronize()
            got.append(cache.attention(step, q, with_lse=True))
            if wait:
                torch.cuda.synchronize()
        cache.check()
        got.append((cache.k_scale, cache.v_scale))
        cache.close()
        return got

    want = go(True)
    for _ in range(4):
        for (a, b), (c, d) in zip(want, go(False)):
            assert torch.equal(a, c) and torch.equal(b, d)


def test_products_behind_prompts():
    """The product kernel, which takes tensor memory before it waits for the
    kernels ahead of it, close behind prompts of many and of few blocks."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(9)
    page, kvh, heads, dim, pages = 32, 8, 32, 128, 300
    cache = bsp.KvCache.empty(pages, kvh, dim, page)
    cache.k.copy_(torch.randint(-127, 128, cache.k.shape, device="cuda", generator=g))
    cache.v.copy_(torch.randint(-127, 128, cache.v.shape, device="cuda", generator=g))
    cache.k_scale.fill_(0.01)
    cache.v_scale.fill_(0.01)
    i32 = dict(dtype=torch.int32, device="cuda")
    steps = []
    for lens in ([(0, 500)] + [(70, 1)] * 12, [(1000, 130), (64, 1)], [(300, 90)] * 6):
        n = [kv.pages_of(a + b, page) for a, b in lens]
        table = torch.zeros((len(lens), max(n)), **i32)
        for b in range(len(lens)):
            table[b, :n[b]] = torch.randperm(pages, device="cuda", generator=g)[:n[b]]
        new = [b for _, b in lens]
        start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), **i32)
        step = bsp.KvStep(table, torch.tensor([a + b for a, b in lens], **i32), start, max(new))
        steps.append((step, torch.randn(sum(new), heads, dim, device="cuda", generator=g).half()))
    w = torch.randn(1024, heads * dim, device="cuda", generator=g)
    w = torch.where(w.abs() < 0.7, 0, w).half()
    m = bsp.BitmapMatrix(w)
    m.set_deterministic(True)

    def go(wait):
        got = []
        for i in range(60):
            y = cache.attention(*steps[i % 3])
            if wait:
                torch.cuda.synchronize()
            got += [y, m.spmm(y[:8].reshape(8, -1))]
            if wait:
                torch.cuda.synchronize()
        cache.check()
        m.check()
        return got

    for a, b in zip(go(True), go(False)):
        assert torch.equal(a, b)
    m.close()
    cache.close()


@pytest.mark.parametrize("heads,kvh", [(32, 8), (8, 2)])
def test_graph_of_a_mixed_step(heads, kvh):
    """Prompt and decode kernel side by side (or behind a joining kernel),
    captured once and replayed on other rows, lengths and pages."""
    import torch
    page, dim, pages, width = 32, 64, 400, 24
    g = torch.Generator(device="cuda").manual_seed(12)
    i32 = dict(dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 150, 151, 152, 160, 161], **i32)
    rows = 170                                              # 9 rows to spare
    table, seq = torch.zeros((5, width), **i32), torch.zeros(5, **i32)
    q, k, v = (torch.zeros((rows, h, dim), dtype=torch.bfloat16, device="cuda") for h in (heads, kvh, kvh))
    cache, plain = (bsp.KvCache.empty(pages, kvh, dim, page) for _ in range(2))
    step = bsp.KvStep(table, seq, start, 150)
    out = torch.empty_like(q)

    def go(c):
        c.append(step, k, v)
        return c.attention(step, q, out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        seq.copy_(start[1:] - start[:-1])
        table.copy_(torch.arange(5 * width, **i32).view(5, width))
        go(cache)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(cache)
    for i in range(12):
        table.copy_(torch.randperm(pages, device="cuda", generator=g)[:5 * width].view(5, width))
        n = start[1:] - start[:-1]
        seq.copy_(n + torch.randint(0, width * page - 150, (5,), device="cuda", generator=g).int())
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, device="cuda", generator=g))
        for a, b in zip((plain.k, plain.v, plain.k_scale, plain.v_scale), (cache.k, cache.v, cache.k_scale, cache.v_scale)):
            a.copy_(b)
        graph.replay()
        got = out.clone()
        out.fill_(7)
        torch.cuda.synchronize()
        go(plain)
        assert torch.equal(got, out)
        assert torch.equal(cache.k, plain.k) and torch.equal(cache.v_scale, plain.v_scale)
    cache.check()
    cache.close()
    plain.close()
