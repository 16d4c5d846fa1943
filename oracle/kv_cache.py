"""Plain definitions of the paged 8-bit KV cache's operators (numpy, CPU).

Request by request and page by page, in 64 bits where values are computed;
the quantisation is also given in fp32 with the operations that include/bsp.h
names (maximum, division, product, round to nearest even), so that codes and
scales can be compared bit for bit.  Test infrastructure only.
"""
from __future__ import annotations

import numpy as np


def pages_of(tokens: int, page: int) -> int:
    return -(-tokens // page)


def plan(ctx, new, table, free, count, tokens, page):
    """The scheduler's rule: returns a dict of the outputs (table and free
    list are copies)."""
    table, free = np.array(table), np.array(free)
    batch, width = table.shape
    ctx = [min(max(int(c), 0), width * page) for c in ctx]
    live = min(max(int(count), 0), len(free))
    stack = list(free[:live])
    for b in range(batch):
        if new[b] < 0:
            stack += list(table[b, :pages_of(ctx[b], page)])
    granted, seq, q_start, slots, positions = [], [], [0], [], []
    room, asked, closed = len(stack), 0, False
    for b in range(batch):
        n = max(int(new[b]), 0)
        if ctx[b] + n > width * page:
            n = 0
        have, want = pages_of(ctx[b], page), pages_of(ctx[b] + n, page)
        if new[b] >= 0:
            room -= want - have
        asked += n
        closed = closed or room < 0 or asked > tokens
        if closed:
            n, want = 0, have
        for j in range(have, want if new[b] >= 0 else have):
            table[b, j] = stack.pop()
        for p in range(ctx[b], ctx[b] + n):
            slots.append(int(table[b, p // page]) * page + p % page)
            positions.append(p)
        granted.append(n)
        seq.append(0 if new[b] < 0 else ctx[b] + n)
        q_start.append(q_start[-1] + n)
    rest = tokens - len(slots)
    left = min(len(stack), len(free))
    free[:left] = stack[:left]
    return dict(block_table=table, granted=np.array(granted, np.int32), seq_len=np.array(seq, np.int32),
                q_start=np.array(q_start, np.int32), slots=np.array(slots + [-1] * rest, np.int64),
                positions=np.array(positions + [-1] * rest, np.int32), free_list=free, free_count=left)


def append(codes, scale, x, table, seq, q_start, page):
    """Quantise rows x [rows][heads][dim] (float32) into copies of codes
    [pages][heads][page][dim] and scale [pages][heads]; fp32 arithmetic."""
    codes, scale = codes.copy(), scale.copy()
    f = np.float32
    for b in range(len(seq)):
        lo, n = int(q_start[b]), int(q_start[b + 1] - q_start[b])
        start = int(seq[b]) - n
        done = max(0, -start)  # rows at negative positions are not stored
        while done < n:
            j, off = (start + done) // page, (start + done) % page
            m = min(n - done, page - off)
            p = int(table[b, j])
            rows = x[lo + done:lo + done + m]
            done += m
            if not 0 <= p < codes.shape[0]:
                continue
            for h in range(codes.shape[1]):
                r = rows[:, h].astype(f)
                fine = np.abs(r[np.isfinite(r)])
                top = fine.max() if fine.size else f(0)
                old = scale[p, h] if off else f(0)
                now = max(old, f(top) / f(127))
                if off:
                    ratio = old / now if now > 0 else f(0)
                    codes[p, h, :off] = np.rint(codes[p, h, :off].astype(f) * ratio).astype(np.int8)
                with np.errstate(invalid="ignore"):
                    q = r / now if now > 0 else np.zeros_like(r)
                q = np.where(np.isnan(q), 0, np.clip(q, -127, 127))
                codes[p, h, off:off + m] = np.rint(q).astype(np.int8)
                scale[p, h] = now
    return codes, scale


def read(codes, scale, slots, page):
    """Rows [n][heads][dim] in 64 bits; zeros outside the cache."""
    out = np.zeros((len(slots), codes.shape[1], codes.shape[3]))
    for i, s in enumerate(slots):
        p = int(s) // page
        if s >= 0 and p < codes.shape[0]:
            out[i] = codes[p, :, int(s) % page].astype(np.float64) * scale[p].astype(np.float64)[:, None]
    return out


def attention(q, k, v, k_scale, v_scale, table, seq, q_start, page, scale, window=0):
    """(out, lse, weight, spread, seen) in 64 bits for q [rows][heads][dim]:
    weight[row][head][dim] = sum p |v| / sum p, spread[row][head] = the
    largest scale * sum |q k| of a seen row, seen = how many rows are seen;
    the last three carry the error bounds of the tests."""
    rows, heads, dim = q.shape
    group = heads // k.shape[1]
    out, lse = np.zeros((rows, heads, dim)), np.full((rows, heads), -np.inf)
    weight, spread, seen = np.zeros_like(out), np.zeros((rows, heads)), np.zeros((rows, heads))
    for b in range(len(seq)):
        n = int(q_start[b + 1] - q_start[b])
        length = int(seq[b])
        home = np.array([table[b, j] for j in range(pages_of(length, page))], dtype=np.int64)
        there = (home >= 0) & (home < k.shape[0])
        there_rows = np.repeat(there, page)[:length]
        for h in range(k.shape[1]):
            kk, vv = np.zeros((len(home) * page, dim)), np.zeros((len(home) * page, dim))
            for j in np.nonzero(there)[0]:
                kk[j * page:(j + 1) * page] = k[home[j], h].astype(np.float64) * np.float64(k_scale[home[j], h])
                vv[j * page:(j + 1) * page] = v[home[j], h].astype(np.float64) * np.float64(v_scale[home[j], h])
            kk, vv = kk[:length], vv[:length]
            for i in range(n):
                row, pos = int(q_start[b]) + i, length - n + i
                see = there_rows & (np.arange(length) <= pos)
                if window:
                    see &= np.arange(length) > pos - window
                if not see.any():
                    continue
                for a in range(h * group, (h + 1) * group):
                    x = kk[see] @ q[row, a].astype(np.float64) * scale
                    p = np.exp(x - x.max())
                    out[row, a] = p @ vv[see] / p.sum()
                    lse[row, a] = x.max() + np.log(p.sum())
                    weight[row, a] = p @ np.abs(vv[see]) / p.sum()
                    spread[row, a] = (np.abs(kk[see]) @ np.abs(q[row, a].astype(np.float64))).max() * scale
                    seen[row, a] = see.sum()
    return out, lse, weight, spread, seen
