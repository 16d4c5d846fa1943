"""The paged 8-bit KV cache's operators: their cases, plain forms and definitions.

A decoder layer multiplies its activations by pruned weights and, between the
QKV and the output projection, attends over what it has cached.  The cache
holds K and V as int8 codes in pages of ``page`` tokens, with one fp32 scale
for each page and KV head (K and V apart): value = code * scale.  Four
operators work on it:

* ``plan``       request lengths -> pages granted from a free list, block
                 table, ragged offsets, slot and position of every new token;
* ``append``     new K / V rows quantised into their pages (a page's scale
                 grows with its largest value, and what it held is rounded to
                 the new scale); its cases read the touched pages back too;
* ``read``       cached rows back by slot, as the values the codes stand for;
* ``attention``  new queries against the cached rows of their requests,
                 causal, with an optional sliding window.

``run`` computes them with elementary torch operations in 32 bits where
``own`` is false, and by the framework's entry points where it is true.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one scheduling step of a small server: every request decodes one token
        dict(name="plan-step-64", op="plan", batch=64, page=16, ctx_min=1, ctx_max=2048, new_min=1,
             new_max=1, chunks=0, release=4, spare=64, lens=1),
        # a large server's step: prompts and decodes mixed, requests ending, too few pages for all
        dict(name="plan-mixed-1024", op="plan", batch=1024, page=64, ctx_min=0, ctx_max=16384, new_min=1,
             new_max=700, chunks=128, release=8, spare=300, lens=2),
        # a single stream's next token in an OPT-13B-shaped layer (40 heads of 128)
        dict(name="append-step-1", op="append", batch=1, kv_heads=40, dim=128, page=16, ctx_min=700,
             ctx_max=700, new_min=1, new_max=1, chunks=0, type="fp16", lens=3),
        # the same layer with 64 streams, each with one token to store
        dict(name="append-step-64", op="append", batch=64, kv_heads=40, dim=128, page=16, ctx_min=1,
             ctx_max=2048, new_min=1, new_max=1, chunks=0, type="fp16", lens=4),
        # prompts of a Llama-2-70B-shaped layer (8 KV heads of 128), stored in large pages, some of
        # them continuing a page that an earlier chunk began
        dict(name="append-prompts", op="append", batch=11, kv_heads=8, dim=128, page=64, ctx_min=0,
             ctx_max=1000, new_min=1, new_max=2500, chunks=11, type="bf16", lens=5),
        # one request's whole context read back, to move it elsewhere
        dict(name="read-request", op="read", batch=1, kv_heads=8, dim=128, page=64, ctx_min=30011,
             ctx_max=30011, new_min=0, new_max=0, chunks=0, type="fp16", lens=6),
        # short prefixes of many requests read back
        dict(name="read-prefixes", op="read", batch=48, kv_heads=40, dim=64, page=16, ctx_min=1,
             ctx_max=96, new_min=0, new_max=0, chunks=0, type="bf16", lens=7),
        # latency: one stream, one token, a short context (OPT-13B-shaped heads)
        dict(name="decode-1", op="attention", batch=1, heads=40, kv_heads=40, dim=128, page=16, ctx_min=516,
             ctx_max=516, new_min=1, new_max=1, chunks=0, window=0, type="fp16", lens=8),
        # serving: 64 streams of ragged length, grouped heads (Llama-2-70B-shaped)
        dict(name="decode-64", op="attention", batch=64, heads=64, kv_heads=8, dim=128, page=64, ctx_min=200,
             ctx_max=16384, new_min=1, new_max=1, chunks=0, window=0, type="fp16", lens=9),
        # few streams of long context, several draft tokens each to verify
        dict(name="verify-long", op="attention", batch=3, heads=32, kv_heads=8, dim=128, page=32, ctx_min=60000,
             ctx_max=120000, new_min=5, new_max=5, chunks=0, window=0, type="bf16", lens=10),
        # a step that mixes one chunk of a prompt with decoding streams, under a sliding window
        dict(name="mixed-window", op="attention", batch=17, heads=40, kv_heads=40, dim=128, page=16, ctx_min=30,
             ctx_max=4000, new_min=1, new_max=513, chunks=1, window=1024, type="fp16", lens=11),
        # a long prompt at once (Llama-2-70B-shaped)
        dict(name="prompt-8k", op="attention", batch=1, heads=64, kv_heads=8, dim=128, page=64, ctx_min=0,
             ctx_max=0, new_min=8101, new_max=8101, chunks=1, window=0, type="bf16", lens=12),
    ]


def _log_int(r, lo, hi):
    """A whole number in lo..hi, spread over its logarithm."""
    return min(hi, max(lo, int(math.exp(r.uniform(math.log(max(lo, 1) * 1.0), math.log(hi + 1.0))))))


def draw(rng):
    r = rng
    kind = r.choice(["plan", "append", "read", "attention", "attention", "attention"])
    page = r.choice([16, 32, 64, 128])
    lens = r.randrange(1 << 30)
    if kind == "plan":
        batch = _log_int(r, 1, 1500)
        chunks = r.choice([0, 1, batch // 8])
        return dict(op="plan", batch=batch, page=page, ctx_min=r.choice([0, 1]), ctx_max=_log_int(r, 1, 16384),
                    new_min=r.choice([0, 1, 3]), new_max=max(3, _log_int(r, 3, 60000 // max(chunks, 60))),
                    chunks=chunks, release=batch // 16, spare=_log_int(r, 1, 4000), lens=lens)
    kv_heads, group = r.choice([(40, 1), (8, 8), (32, 1), (8, 4), (4, 7), (1, 16), (2, 5), (12, 1)])
    dim = r.choice([64, 128, 128, 128, 80, 96, 256])
    kind_of = r.choice(["fp16", "bf16"])
    if kind in ("append", "read"):
        rows = _log_int(r, 1, 24_000_000 // (kv_heads * dim))  # rows of the step, at most
        batch = _log_int(r, 1, min(256, rows))
        if kind == "read":
            return dict(op="read", batch=batch, kv_heads=kv_heads, dim=dim, page=page, ctx_min=1,
                        ctx_max=max(1, rows // batch), new_min=0, new_max=0, chunks=0, type=kind_of, lens=lens)
        one = r.random() < 0.4
        return dict(op="append", batch=batch, kv_heads=kv_heads, dim=dim, page=page, ctx_min=0,
                    ctx_max=_log_int(r, 1, 2000), new_min=1, new_max=1 if one else max(1, rows // batch),
                    chunks=0 if one else batch, type=kind_of, lens=lens)
    heads = kv_heads * group
    shape = r.choice(["decode", "decode", "verify", "prompt", "mixed"])
    window = r.choice([0, 0, 0, 128, 1000])
    if shape in ("decode", "verify"):
        new = 1 if shape == "decode" else r.randrange(2, 9)
        total = _log_int(r, 64, 900_000_000 // (kv_heads * dim))  # cached rows, at most
        batch = _log_int(r, 1, min(256, max(1, total // 16)))
        longest = max(1, min(131072, total // batch))
        return dict(op="attention", batch=batch, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                    ctx_min=max(0, longest // r.choice([1, 4, 64])), ctx_max=longest, new_min=new, new_max=new,
                    chunks=0, window=window, type=kind_of, lens=lens)
    # logits of the padded batch stay under 2.5e9 and the products under a
    # third of the largest listed case's
    batch = r.randrange(1, 9) if shape == "prompt" else r.randrange(2, 24)
    new = _log_int(r, 9, 3000)
    ctx = _log_int(r, 1, 8000)
    while batch * heads * new * (ctx + new) > 2_500_000_000 or batch * heads * new * (ctx + new) * dim > 1.2e11:
        new, ctx, batch = max(9, new * 3 // 4), max(1, ctx * 3 // 4), max(1 if shape == "prompt" else 2, batch * 7 // 8)
        if batch <= 2 and new <= 9 and ctx <= 1:
            break
    return dict(op="attention", batch=batch, heads=heads, kv_heads=kv_heads, dim=dim, page=page, ctx_min=0,
                ctx_max=ctx, new_min=1, new_max=new, chunks=batch if shape == "prompt" else 1, window=window,
                type=kind_of, lens=lens)


def lengths(case):
    """[(cached tokens, new tokens)] of the requests: the first is the longest;
    the first ``chunks`` bring up to ``new_max`` tokens, the others ``new_min``."""
    r = random.Random(case["lens"])
    got = []
    for b in range(case["batch"]):
        lo, hi = case["ctx_min"], case["ctx_max"]
        ctx = hi if b == 0 or lo >= hi else _log_int(r, lo, hi) - (1 if lo == 0 else 0)
        new = case["new_min"]
        if b < case["chunks"]:
            new = case["new_max"] if b == 0 else _log_int(r, max(1, case["new_max"] // 6), case["new_max"])
        got.append((max(0, ctx), new))
    return got


def _pages(tokens, page):
    return -(-tokens // page)


# ------------------------------------------------------------------ inputs

def _codes(shape, gen):
    """int8 codes as a page with its own scale holds them: a bell over +-127."""
    return torch.randn(shape, dtype=torch.float16, device="cuda", generator=gen).mul_(38).round_().clamp_(-127, 127).to(
        torch.int8)


def _table(counts, spare, gen):
    """Block table [B][width] of pages scattered over a pool, -1 beyond each
    request's own, and the pool's size."""
    counts = torch.tensor(counts, dtype=torch.int64)
    total, width = int(counts.sum()) + spare, max(1, int(counts.max()))
    pool = torch.randperm(total, device="cuda", generator=gen)
    start = (torch.cumsum(counts, 0) - counts).cuda()
    col = torch.arange(width, device="cuda")
    at = (start[:, None] + col).clamp(max=total - 1)
    table = torch.where(col < counts.cuda()[:, None], pool[at], -1)
    return table.to(torch.int32), total, pool[int(counts.sum()):].to(torch.int32)


def _prepare_plan(case, gen):
    batch, page = case["batch"], case["page"]
    lens = lengths(case)
    width = max(_pages(c + n, page) for c, n in lens)
    counts = [_pages(c, page) for c, n in lens]
    every = max(1, batch // max(1, case["release"]))
    new = [-1 if case["release"] and b % every == every - 1 else n for b, (c, n) in enumerate(lens)]
    table, total, free = _table(counts, case["spare"], gen)
    full = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    full[:, :min(width, table.shape[1])] = table[:, :width]
    stack = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    stack[:free.numel()] = free
    s = dict(ctx_len=torch.tensor([c for c, n in lens], dtype=torch.int32, device="cuda"),
             new_len=torch.tensor(new, dtype=torch.int32, device="cuda"), block_table=full, free_list=stack,
             free_count=torch.tensor([free.numel()], dtype=torch.int32, device="cuda"), page=page,
             tokens=max(1, sum(max(0, n) for n in new)))
    if own:  # the server's cache (the plan deals in page numbers: one small head stands for all)
        import bitmap_encoded_unstructured_gb300 as bsp
        pool = torch.zeros((total, 1, page, 16), dtype=torch.int8, device="cuda")
        scale = torch.zeros((total, 1), dtype=torch.float32, device="cuda")
        s["cache"] = bsp.KvCache(pool, pool.clone(), scale, scale.clone())
        s["step"] = bsp.KvStep.empty(batch, s["tokens"])
    return s


def _prepare_cache(case, gen):
    """The cache with what is in it: pool, scales, block table, lengths."""
    page, hkv, dim = case["page"], case["kv_heads"], case["dim"]
    lens = lengths(case)
    table, total, _ = _table([_pages(c + n, page) for c, n in lens], 3, gen)
    s = dict(k=_codes((total, hkv, page, dim), gen), v=_codes((total, hkv, page, dim), gen), block_table=table, page=page)
    for name, size in (("k_scale", 1.0 / 38), ("v_scale", 0.4 / 38)):
        s[name] = torch.randn((total, hkv), device="cuda", generator=gen).mul_(0.3).exp_().mul_(size)
    starts = [0]
    for c, n in lens:
        starts.append(starts[-1] + n)
    s["seq_len"] = torch.tensor([c + n for c, n in lens], dtype=torch.int32, device="cuda")
    s["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["rows"], s["max_new"] = starts[-1], max(1, max(n for c, n in lens))
    if own:  # the handles a server keeps over these arrays
        import bitmap_encoded_unstructured_gb300 as bsp
        s["cache"] = bsp.KvCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["step"] = bsp.KvStep(s["block_table"], s["seq_len"], s["q_start"], max_new=s["max_new"])
    return s


def _slots_of(s, case, first):
    """Slots of the cached rows from first[b] on, of every request in turn."""
    rows, page = [], case["page"]
    table = s["block_table"].to(torch.int64)
    for b, (c, n) in enumerate(lengths(case)):
        at = torch.arange(first[b], c + n, device="cuda")
        rows.append(table[b, at // page] * page + at % page)
    return torch.cat(rows)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    if case["op"] == "plan":
        return dict(_prepare_plan(case, gen), op="plan")
    s = dict(_prepare_cache(case, gen), op=case["op"])
    dtype = DTYPES[case["type"]]
    if case["op"] == "attention":
        # logits of a few units: some rows attend broadly, some to a handful of tokens
        q = torch.randn((s["rows"], case["heads"], case["dim"]), device="cuda", generator=gen)
        s["q"] = q.mul_(1.7).to(dtype)
        s["window"] = case["window"]
    elif case["op"] == "append":
        for name, size in (("k_new", 1.0), ("v_new", 0.4)):
            x = torch.randn((s["rows"], case["kv_heads"], case["dim"]), device="cuda", generator=gen)
            s[name] = x.mul_(size).to(dtype)
        s["slots"] = _slots_of(s, case, [c // case["page"] * case["page"] for c, n in lengths(case)])
    else:
        s["slots"], s["dtype"] = _slots_of(s, case, [0] * case["batch"]), dtype
    return s


# ------------------------------------------------------------- plain forms

def _plain_plan(s):
    """Releases first, then pages in request order to those that fit, first come first served."""
    page, table, stack = s["page"], s["block_table"].long(), s["free_list"].long()
    ctx, new, count = s["ctx_len"].long(), s["new_len"].long(), s["free_count"].long()
    batch, width = table.shape
    ends = new < 0
    ask = new.clamp(min=0)
    ask = torch.where(ctx + ask > width * page, 0, ask)
    have = (ctx + page - 1) // page
    need = torch.where(ends, 0, (ctx + ask + page - 1) // page - have)
    back = torch.where(ends, have, 0)
    back_end = torch.cumsum(back, 0)
    avail = count + back_end[-1]
    fits = (torch.cumsum(need, 0) <= avail) & (torch.cumsum(ask, 0) <= s["tokens"])
    granted, need = torch.where(fits, ask, 0), torch.where(fits, need, 0)
    seq_len = torch.where(ends, 0, ctx + granted)
    q_end, need_end = torch.cumsum(granted, 0), torch.cumsum(need, 0)
    left = avail - need_end[-1]
    # the stack with what was released on top; its last place takes what is not stored
    col = torch.arange(width, device=table.device)
    to = torch.where(col < back[:, None], count + (back_end - back)[:, None] + col, stack.numel())
    full = torch.cat([stack, stack[:1]]).scatter(0, to.reshape(-1), table.reshape(-1))[:-1]
    nth = (need_end - need)[:, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None])
    table = torch.where(fresh, full[(avail - 1 - nth).clamp(0, stack.numel() - 1)], table)
    row = torch.arange(stack.numel(), device=table.device)
    stack = torch.where(row < left, full, stack)
    t = torch.arange(s["tokens"], device=table.device)
    req = torch.searchsorted(q_end, t, right=True).clamp(max=batch - 1)
    pos = ctx[req] + t - (q_end - granted)[req]
    slot = table[req, (pos // page).clamp(max=width - 1)] * page + pos % page
    live = t < q_end[-1]
    i32 = torch.int32
    return dict(block_table=table.to(i32), seq_len=seq_len.to(i32),
                q_start=torch.cat([q_end.new_zeros(1), q_end]).to(i32), granted=granted.to(i32),
                slots=torch.where(live, slot, -1), positions=torch.where(live, pos, -1).to(i32),
                free_list=stack.to(i32), free_count=left.to(i32).reshape(1))


def _rows_to_slots(s):
    """Slot of every new row, from the block table."""
    t = torch.arange(s["rows"], device=s["q_start"].device)
    start = s["q_start"].long()
    req = torch.searchsorted(start[1:], t, right=True)
    pos = s["seq_len"].long()[req] - start[req + 1] + t
    return s["block_table"].long()[req, pos // s["page"]] * s["page"] + pos % s["page"]


def _plain_append_one(codes, scale, x, slot, page):
    total, hkv = scale.shape
    x = x.float()
    peak = torch.where(x.isfinite(), x.abs(), 0).amax(-1)
    home, off = slot // page, slot % page
    top = torch.zeros_like(scale).index_reduce_(0, home, peak, "amax")
    first = torch.full((total,), page, device=slot.device).index_reduce_(0, home, off, "amin")
    kept = ((first > 0) & (first < page))[:, None]      # pages that hold earlier rows
    touched = (first < page)[:, None]
    grown = torch.maximum(torch.where(kept, scale, 0), top / 127)
    ratio = torch.where(grown > 0, scale / grown, 0)
    old = torch.round(codes.float() * ratio[..., None, None])
    codes.copy_(torch.where(kept[..., None, None], old.to(torch.int8), codes))
    scale.copy_(torch.where(touched, grown, scale))
    by = scale[home][..., None]
    q = torch.where(by > 0, x / by, 0)
    q = torch.round(torch.where(q.isnan(), 0, q).clamp(-127, 127))
    codes[home, :, off] = q.to(torch.int8)


def _plain_read(s, dtype):
    slot, page = s["slots"], s["page"]
    home, off = (slot // page).clamp(min=0), slot % page
    got = []
    for codes, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
        x = codes[home, :, off].float() * scale[home][..., None]
        got.append(torch.where(slot[:, None, None] >= 0, x, 0).to(dtype))
    return got


def _plain_attention(s):
    q, page, table = s["q"], s["page"], s["block_table"].long()
    hkv, dim = s["k"].shape[1], s["k"].shape[3]
    rows, heads, _ = q.shape
    batch, width = table.shape
    group, most, span = heads // hkv, s["max_new"], width * page
    home = table.clamp(min=0)

    def cached(codes, scale):  # [B][Hkv][span][D]
        x = codes[home].float() * scale[home][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(batch, hkv, span, dim)

    start, seq = s["q_start"].long(), s["seq_len"].long()
    new = start[1:] - start[:-1]
    i = torch.arange(most, device=q.device)
    at = (start[:-1, None] + i).clamp(max=rows - 1)     # [B][most] row of q
    x = q[at.reshape(-1)].float().reshape(batch, most, hkv, group, dim)
    x = x.permute(0, 2, 1, 3, 4).reshape(batch, hkv, most * group, dim)
    logits = torch.matmul(x, cached(s["k"], s["k_scale"]).transpose(-1, -2)) * (1 / math.sqrt(dim))
    logits = logits.reshape(batch, hkv, most, group, span)
    pos = (seq - new)[:, None] + i                      # [B][most]
    j = torch.arange(span, device=q.device)
    seen = (j <= pos[..., None]) & (j < seq[:, None, None]) & (table >= 0).repeat_interleave(page, 1)[:, None]
    if s["window"]:
        seen &= j > pos[..., None] - s["window"]
    logits.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits.sub_(torch.where(top.isinf(), 0, top)))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.reshape(batch, hkv, most * group, span), cached(s["v"], s["v_scale"]))
    out = out.reshape(batch, hkv, most, group, dim) / torch.where(total > 0, total, 1)
    lse = (top + torch.log(total))[..., 0]
    t = torch.arange(rows, device=q.device)             # back to the ragged rows
    req = torch.searchsorted(start[1:], t, right=True)
    out = out.permute(0, 2, 1, 3, 4)[req, t - start[req]].reshape(rows, heads, dim)
    lse = lse.permute(0, 2, 1, 3)[req, t - start[req]].reshape(rows, heads)
    return dict(out=out.to(q.dtype), lse=lse)


def run(state):
    s = state
    if s["op"] == "plan":
        if own:
            p = s["cache"].plan(s["ctx_len"], s["new_len"], s["block_table"], s["free_list"], s["free_count"],
                                tokens=s["tokens"], out=s["step"])
            return dict(block_table=p.block_table, seq_len=p.seq_len, q_start=p.q_start, granted=p.granted,
                        slots=p.slots, positions=p.positions, free_list=s["free_list"], free_count=p.free_count)
        return _plain_plan(s)
    if s["op"] == "append":
        if own:
            s["cache"].append(s["step"], s["k_new"], s["v_new"])
            k, v = s["cache"].read(s["slots"], dtype=s["k_new"].dtype)
        else:
            slot = _rows_to_slots(s)
            _plain_append_one(s["k"], s["k_scale"], s["k_new"], slot, s["page"])
            _plain_append_one(s["v"], s["v_scale"], s["v_new"], slot, s["page"])
            k, v = _plain_read(s, s["k_new"].dtype)
        return dict(k=k, v=v, k_scale=s["k_scale"], v_scale=s["v_scale"])
    if s["op"] == "read":
        k, v = s["cache"].read(s["slots"], dtype=s["dtype"]) if own else _plain_read(s, s["dtype"])
        return dict(k=k, v=v)
    if own:
        out, lse = s["cache"].attention(s["step"], s["q"], window=s["window"], with_lse=True)
        return dict(out=out, lse=lse)
    return _plain_attention(s)


# -------------------------------------------------------- what a pass needs

def work(case):
    page, lens = case["page"], lengths(case)
    if case["op"] == "plan":
        pages = sum(_pages(c + n, page) - c // page for c, n in lens)
        new = sum(n for c, n in lens)
        # lengths in; table entries of the new rows; offsets, slots and positions out
        return {"bytes": 20 * case["batch"] + 8 * pages + 12 * new, "flops": 0}
    row = case["kv_heads"] * case["dim"]                 # values of one K (or V) row
    if case["op"] == "append":
        new = sum(n for c, n in lens)
        touched = sum(_pages(c + n, page) - c // page for c, n in lens)
        back = sum(c + n - c // page * page for c, n in lens)
        # rows in and codes out, both scales of the touched pages, and the pages read back as 16-bit rows
        return {"bytes": 2 * row * (new * 3 + back * 3) + 16 * touched * case["kv_heads"] + 8 * back, "flops": 4 * row * new}
    if case["op"] == "read":
        rows = sum(c + n for c, n in lens)
        pages = sum(_pages(c + n, page) for c, n in lens)
        return {"bytes": 2 * row * rows * 3 + 8 * pages * case["kv_heads"] + 8 * rows, "flops": 2 * row * rows}
    w, pairs, cached, pages, new = case["window"], 0, 0, 0, 0
    for c, n in lens:
        first = max(0, c + 1 - w) if w else 0            # the first row that any query sees
        cached += c + n - first if n else 0
        pages += _pages(c + n, page) - first // page if n else 0
        new += n
        if w:
            pairs += sum(min(c + i + 1, w) for i in range(n))
        else:
            pairs += n * c + n * (n + 1) // 2
    codes = 2 * row * cached + 8 * pages * case["kv_heads"] + 4 * pages
    return {"bytes": codes + case["heads"] * new * (4 * case["dim"] + 4), "flops": 4 * case["heads"] * case["dim"] * pairs}


# ------------------------------------------------------ definitions, 64 bits

def _exact_plan(s):
    """The scheduler's rule, request by request."""
    page, table, stack = s["page"], s["block_table"].tolist(), s["free_list"].tolist()
    ctx, new, count = s["ctx_len"].tolist(), s["new_len"].tolist(), int(s["free_count"])
    kept, batch, width = stack[:], len(ctx), len(table[0])
    for b in range(batch):
        if new[b] < 0:
            for j in range(_pages(ctx[b], page)):
                stack[count] = table[b][j]
                count += 1
    granted, seq_len, slots, positions, q_start, room, asked, blocked = [], [], [], [], [0], count, 0, False
    for b in range(batch):
        n = max(0, new[b])
        n = 0 if ctx[b] + n > width * page else n
        have, want = _pages(ctx[b], page), _pages(ctx[b] + n, page)
        room, asked = room - (want - have if new[b] >= 0 else 0), asked + n
        blocked = blocked or room < 0 or asked > s["tokens"]
        n = 0 if blocked else n
        if n:
            for j in range(have, want):
                count -= 1
                table[b][j] = stack[count]
        for p in range(ctx[b], ctx[b] + n):
            slots.append(table[b][p // page] * page + p % page)
            positions.append(p)
        granted.append(n)
        seq_len.append(0 if new[b] < 0 else ctx[b] + n)
        q_start.append(q_start[-1] + n)
    rest = s["tokens"] - len(slots)
    i32 = torch.int32
    return dict(block_table=torch.tensor(table, dtype=i32), seq_len=torch.tensor(seq_len, dtype=i32),
                q_start=torch.tensor(q_start, dtype=i32), granted=torch.tensor(granted, dtype=i32),
                slots=torch.tensor(slots + [-1] * rest), positions=torch.tensor(positions + [-1] * rest, dtype=i32),
                free_list=torch.tensor(stack[:count] + kept[count:], dtype=i32),
                free_count=torch.tensor([count], dtype=i32))


def _exact_read(codes, scale, slots, page):
    return torch.stack([codes[i // page, :, i % page].double() * scale[i // page].double()[:, None]
                        for i in slots.tolist()]) if len(slots) < 4000 else (
        codes[slots // page, :, slots % page].double() * scale[slots // page].double()[..., None])


def _exact_append(s, case):
    out = {}
    table = s["block_table"].tolist()
    for name in ("k", "v"):
        codes, scale, x = s[name].clone(), s[name + "_scale"].double(), s[name + "_new"].double()
        at = 0
        for b, (c, n) in enumerate(lengths(case)):
            done = 0
            while done < n:                              # page by page
                p, o = table[b][(c + done) // case["page"]], (c + done) % case["page"]
                m = min(n - done, case["page"] - o)
                rows = x[at + done:at + done + m]
                top = rows.abs().amax(dim=(0, 2)) / 127
                now = torch.maximum(scale[p], top) if o else top
                if o:
                    codes[p, :, :o] = torch.round(codes[p, :, :o].double() * (scale[p] / now)[:, None, None]).to(torch.int8)
                scale[p] = now
                codes[p, :, o:o + m] = torch.round(rows / now[:, None]).transpose(0, 1).to(torch.int8)
                done += m
            at += n
        out[name] = _exact_read(codes, scale, s["slots"], case["page"])
        out[name + "_scale"] = scale
    return out


def _exact_attention(s, case):
    page, hkv, dim, heads = case["page"], case["kv_heads"], case["dim"], case["heads"]
    group, out, lse, at = heads // hkv, [], [], 0
    for b, (c, n) in enumerate(lengths(case)):
        length = c + n
        low = max(0, c + 1 - s["window"]) // page if s["window"] else 0   # first page that any query sees
        home = s["block_table"][b, low:_pages(length, page)].long()
        cols = torch.arange(low * page, low * page + home.numel() * page, device="cuda")
        outs, lses = [], []
        for h in range(hkv):
            k = (s["k"][home, h].double() * s["k_scale"][home, h].double()[:, None, None]).reshape(-1, dim)
            v = (s["v"][home, h].double() * s["v_scale"][home, h].double()[:, None, None]).reshape(-1, dim)
            rows_o, rows_l = [], []
            for lo in range(0, n, 1024):
                m = min(1024, n - lo)
                q = s["q"][at + lo:at + lo + m, h * group:(h + 1) * group].double()
                pos = torch.arange(c + lo, c + lo + m, device="cuda")[:, None, None]
                x = torch.einsum("mgd,sd->mgs", q, k) / math.sqrt(dim)
                gone = (cols > pos) | ((cols <= pos - s["window"]) if s["window"] else (cols < 0))
                x = x.masked_fill(gone, -math.inf)
                rows_l.append(torch.logsumexp(x, -1))
                rows_o.append(torch.einsum("mgs,sd->mgd", torch.exp(x - rows_l[-1][..., None]), v))
            outs.append(torch.cat(rows_o) if rows_o else torch.zeros((0, group, dim), dtype=torch.double, device="cuda"))
            lses.append(torch.cat(rows_l) if rows_l else torch.zeros((0, group), dtype=torch.double, device="cuda"))
        out.append(torch.cat(outs, 1))
        lse.append(torch.cat(lses, 1))
        at += n
    return dict(out=torch.cat(out), lse=torch.cat(lse))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(s)
    if case["op"] == "append":
        return _exact_append(s, case)
    if case["op"] == "read":
        return dict(k=_exact_read(s["k"], s["k_scale"], s["slots"], s["page"]),
                    v=_exact_read(s["v"], s["v_scale"], s["slots"], s["page"]))
    if work(case)["flops"] > 4e12:  # over 20 s in 64 bits
        return None
    return _exact_attention(s, case)
