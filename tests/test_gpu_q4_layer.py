"""A gated decoder layer of the framework's operators alone: 4-bit QKV, rotary
positions, paged 8-bit cache, attention, 4-bit output, gated block, down."""
import numpy as np
import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from oracle import kv_cache as kv
from oracle import q4, rope

pytestmark = pytest.mark.gpu


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def near(got, want, before, what):
    """Within `before` of the definition (of the same, already rounded, inputs) and one rounding to fp16."""
    off = np.abs(got.double().cpu().numpy() - want)
    lim = before + (np.abs(want) + before) * 2.0 ** -11 + 2.0 ** -25
    assert np.all(off <= lim), (what, (off / lim).max())


@pytest.mark.parametrize("hidden,heads,kvh,inner,group", [(512, 8, 2, 1376, 64), (256, 2, 2, 600, 128)])
def test_layer(hidden, heads, kvh, inner, group):
    import torch
    dim, page = hidden // heads, 16
    g = np.random.default_rng(hidden)
    i32 = dict(dtype=torch.int32, device="cuda")

    def weight(rows, cols):
        W = dev((g.standard_normal((rows, cols)) * cols ** -0.5).astype(np.float16))
        m = bsp.Int4Matrix(W, group=group, zeros=bool(rows % 3 == 0))
        c, s, z = m.arrays()
        return m, (q4.unpack(c.cpu().numpy()), s.float().cpu().numpy(), None if z is None else z.cpu().numpy())

    qkv, out, gate, up, down = (weight(r, c) for r, c in (
        ((heads + 2 * kvh) * dim, hidden), (hidden, hidden), (inner, hidden), (inner, hidden), (hidden, inner)))
    turn = bsp.Rotary(dim, sections=[dim // 8, dim // 8, dim // 4])
    cache = bsp.KvCache.empty(40, kvh, dim, page)
    table, free, count = torch.full((3, 20), -1, **i32), torch.arange(40, **i32), torch.tensor([40], **i32)
    ctx = torch.zeros(3, **i32)
    k8, ks = np.zeros((40, kvh, page, dim), np.int8), np.zeros((40, kvh), np.float32)
    v8, vs = k8.copy(), ks.copy()

    def mm(w, x, want_of=q4.product):
        m, arrays = w
        y = m.mm(x)
        xs = x.float().cpu().numpy()
        near(y, q4.product(xs, *arrays, group), q4.error_bound(xs, *arrays, group, "float16"), "mm")
        return y

    for new in ([200, 3, 40], [1, 1, 1], [0, 5, 1]):
        n, room = sum(new), sum(new) + 2                     # a step with two rows to spare
        step = cache.plan(ctx, torch.tensor(new, **i32), table, free, count, tokens=room, max_new=max(new))
        count, ctx = step.free_count, step.seq_len
        x = dev(g.standard_normal((room, hidden)).astype(np.float16))
        a = mm(qkv, x).view(room, heads + 2 * kvh, dim)
        q, k, v = a[:, :heads], a[:, heads:heads + kvh], a[:, heads + kvh:]
        pos = torch.stack([step.positions, torch.where(step.positions < 0, -1, step.positions % 7),
                           torch.where(step.positions < 0, -1, step.positions // 7)])
        before = a.clone()
        turn.apply(q, k, pos, out=(q, k))                    # where they are
        for y, b in ((q, before[:, :heads]), (k, before[:, heads:heads + kvh])):
            b, p = b.float().cpu().numpy(), pos.cpu().numpy()
            want = rope.rotate(b, p, turn.freqs, turn.axis, False)
            lim = rope.bound(b, want, dim, "float16")
            live = (p >= 0).all(0)
            assert live.sum() == n
            assert np.all(np.abs(y.double().cpu().numpy() - want)[live] <= lim[live])
            assert np.array_equal(y.float().cpu().numpy()[~live], b[~live])
        cache.append(step, k, v)
        y = cache.attention(step, q)
        t, seq, start = table.cpu().numpy(), step.seq_len.tolist(), step.q_start.tolist()
        k8, ks = kv.append(k8, ks, k.float().cpu().numpy(), t, seq, start, page)
        v8, vs = kv.append(v8, vs, v.float().cpu().numpy(), t, seq, start, page)
        assert np.array_equal(cache.k.cpu().numpy(), k8) and np.array_equal(cache.v_scale.cpu().numpy(), vs)
        want, _, w, _, _ = kv.attention(q.float().cpu().numpy(), k8, v8, ks, vs, t, seq, start, page, dim ** -0.5)
        assert np.all(np.abs(y.double().cpu().numpy() - want) <= 2.0 ** -9 * w + 1e-4)
        h = x + mm(out, y.view(room, hidden))
        m = gate[0].gated(up[0], h)
        hs = h.float().cpu().numpy()
        gs, us = q4.product(hs, *gate[1], group), q4.product(hs, *up[1], group)
        eg, eu = (q4.error_bound(hs, *w_, group, "float16") for w_ in (gate[1], up[1]))
        near(m, q4.act(gs, "silu") * us, q4.gated_bound(gs, us, eg, eu, "silu"), "gated")
        mm(down, m)
    for w in (qkv, out, gate, up, down):
        w[0].check()
        w[0].close()
    cache.check()
    cache.close()
    turn.close()
