"""Rotary positions against their plain definition in 64 bits."""
import numpy as np
import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from oracle import q4, rope

pytestmark = pytest.mark.gpu

DT = ["float16", "bfloat16"]


def dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(getattr(torch, dtype))


def data(rows, heads, dim, dtype, seed):
    return q4.ROUND[dtype](np.random.default_rng(seed).standard_normal((rows, heads, dim)).astype(np.float32))


def places(axes, rows, far, seed):
    return np.random.default_rng(seed).integers(0, far, (axes, rows)).astype(np.int32)


def close(y, x, pos, r, dtype, inverse=False):
    want = rope.rotate(x, pos, r.freqs, r.axis, r.interleaved, r.scale, inverse)
    lim = rope.bound(x, want, r.rot, dtype, r.scale, r.interleaved)
    live = (pos >= 0).all(0)
    off = np.abs(y.double().cpu().numpy() - want)[live]
    assert np.all(off <= lim[live]), (off / lim[live]).max()


CASES = [  # dim, rot, sections, cyclic, own frequencies
    (128, 128, None, False, False), (64, 64, [16, 8, 8], False, False), (128, 128, [24, 20, 20], True, False),
    (80, 32, None, False, False), (96, 24, [4, 8], False, True), (8, 8, [1, 1, 1, 1], False, False),
    (256, 64, [32], False, False), (1024, 1024, [100, 400, 12], True, False), (1016, 8, None, False, False),
    (112, 104, [20, 16, 16], True, True)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_apply(case, interleaved, dtype):
    import torch
    dim, rot, sections, cyclic, own = CASES[case]
    r = bsp.Rotary(dim, rot=rot, sections=sections, cyclic=cyclic, own_freqs=own, interleaved=interleaved,
                   scale=1.0 if case % 2 else 1.25)
    for rows, heads, kv, far in ((1, 1, 1, 10), (1, 40, 8, 5000), (7, 5, 1, 1 << 20), (130, 3, 3, 2**31 - 1), (2500, 2, 1, 32768)):
        q, k = data(rows, heads, dim, dtype, rows), data(rows, kv, dim, dtype, rows + 1)
        pos = places(r.axes, rows, far, 3)
        p = dev(pos if r.axes > 1 else pos[0])
        for inverse in (False, True):
            yq, yk = r.apply(dev(q, dtype), dev(k, dtype), p, inverse=inverse)
            close(yq, q, pos, r, dtype, inverse)
            close(yk, k, pos, r, dtype, inverse)
        assert torch.equal(r.apply(dev(q, dtype), None, p, inverse=True), yq)
    r.close()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_in_a_qkv_tensor(interleaved, dtype):
    """Queries and keys turned where they are; values, and rows that are not there, stay."""
    import torch
    rows, heads, kv, dim = 50, 6, 2, 96
    r = bsp.Rotary(dim, rot=48, sections=[12, 6, 6], interleaved=interleaved)
    x = data(rows, heads + 2 * kv, dim, dtype, 5)
    pos = places(3, rows, 4000, 6)
    pos[0, 7], pos[2, 20], pos[:, 44:] = -1, -5, -1
    t = dev(x, dtype)
    before = t.clone()
    q, k = t[:, :heads], t[:, heads:heads + kv]
    a, b = r.apply(q, k, dev(pos), out=(q, k))
    assert a is q and b is k
    close(t[:, :heads], x[:, :heads], pos, r, dtype)
    close(t[:, heads:heads + kv], x[:, heads:heads + kv], pos, r, dtype)
    gone = dev((pos < 0).any(0))
    assert torch.equal(t[gone], before[gone]) and torch.equal(t[:, heads + kv:], before[:, heads + kv:])
    assert torch.equal(t[..., 48:], before[..., 48:])
    # the same into new tensors, whose rows that are not there stay as they were
    new = torch.full((rows, heads, dim), 3.0, dtype=t.dtype, device="cuda")
    r.apply(before[:, :heads], None, dev(pos), out=(new, None))
    assert torch.equal(new[~gone], t[:, :heads][~gone]) and torch.all(new[gone] == 3)
    r.close()


def test_strides_and_layouts():
    """Heads before rows, padded rows, a broadcast input head, positions a slice."""
    import torch
    rows, heads, dim, dtype = 33, 4, 64, "float16"
    r = bsp.Rotary(dim, sections=[16, 16])
    x, pos = data(rows, heads, dim, dtype, 1), places(2, rows, 999, 2)
    wide = torch.zeros((2, rows + 5), dtype=torch.int32, device="cuda")
    wide[:, :rows] = dev(pos)
    p = wide[:, :rows]
    want = r.apply(dev(x, dtype), None, p)
    close(want, x, pos, r, dtype)
    by_head = torch.zeros((heads, rows + 2, dim + 8), dtype=torch.float16, device="cuda")
    v = by_head[:, :rows, :dim].transpose(0, 1)
    v.copy_(dev(x, dtype))
    out = torch.full((heads, rows, dim + 8), 9.0, dtype=torch.float16, device="cuda")
    r.apply(v, None, p, out=(out[..., :dim].transpose(0, 1), None))
    assert torch.equal(out[..., :dim].transpose(0, 1), want) and torch.all(out[..., dim:] == 9)
    one = dev(x, dtype)[:, :1].expand(rows, heads, dim)
    assert torch.equal(r.apply(one, None, p), r.apply(one.contiguous(), None, p))
    r.close()


def test_empty_and_refused():
    import torch
    r = bsp.Rotary(64)
    q = torch.zeros((0, 3, 64), dtype=torch.float16, device="cuda")
    assert r.apply(q, None, torch.zeros(0, dtype=torch.int32, device="cuda")).shape == q.shape
    x, p = torch.zeros((4, 3, 64), dtype=torch.float16, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    assert r.apply(x, x[:, :0], p)[1].shape == (4, 0, 64)
    for args in ((x.float(), None, p), (x, x.bfloat16(), p), (x, x[:3], p), (x[..., :32], None, p), (x, None, p[:3]), (x, None, p.long()),
                 (x, None, p.cpu()), (x, None, torch.zeros(8, dtype=torch.int32, device="cuda")[::2])):
        with pytest.raises((ValueError, TypeError)):
            r.apply(*args)
    with pytest.raises(bsp.BspError):  # one row's output over the next row's input
        r.apply(x[:3], None, p[:3], out=(x[1:], None))
    r.close()


def test_no_turn_is_a_copy_and_turning_back():
    import torch
    x = dev(data(40, 5, 128, "bfloat16", 3), "bfloat16")
    r = bsp.Rotary(128)
    assert torch.equal(r.apply(x, None, torch.zeros(40, dtype=torch.int32, device="cuda")), x)
    pos = torch.arange(40, dtype=torch.int32, device="cuda") * 1000
    back = r.apply(r.apply(x, None, pos), None, pos, inverse=True)
    # two roundings to the type (2^-8 of a value of at most |a| + |b| each) turned into either half
    lim = 4 * 2.0 ** -8 * (x.float().abs() + x.float().roll(64, -1).abs())
    assert torch.all((back.float() - x.float()).abs() <= lim + 1e-30)
    r.close()


@pytest.mark.parametrize("dtype", DT)
def test_inverse_is_the_gradient(dtype):
    """sum(w . rotate(x)) changes with x by what the inverse makes of w: against the formula's differences in 64 bits."""
    g = np.random.default_rng(4)
    r = bsp.Rotary(32, rot=24, sections=[6, 6])
    x, w, pos = g.standard_normal((5, 2, 32)), data(5, 2, 32, dtype, 5), places(2, 5, 500, 6)
    grad = r.apply(dev(w, dtype), None, dev(pos), inverse=True).double().cpu().numpy()
    lim = rope.bound(w, np.abs(w) + 1, 24, dtype) + 1e-6
    for at in ((0, 0, 0), (1, 1, 5), (2, 0, 13), (4, 1, 23), (3, 0, 30)):
        e = np.zeros_like(x)
        e[at] = 1e-4
        d = [(w * rope.rotate(x + s * e, pos, r.freqs, r.axis, False)).sum() for s in (1, -1)]
        assert abs((d[0] - d[1]) / 2e-4 - grad[at]) <= lim[at] * 2
    r.close()


def test_streams_and_graphs():
    import torch
    r = bsp.Rotary(128, sections=[16, 24, 24], cyclic=True)
    q, k = dev(data(300, 8, 128, "float16", 1), "float16"), dev(data(300, 2, 128, "float16", 2), "float16")
    pos = dev(places(3, 300, 10000, 3))
    want = r.apply(q, k, pos)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            got.append(r.apply(q, k, pos))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want[0]) and torch.equal(b, want[1]) for a, b in got)
    graph, x = torch.cuda.CUDAGraph(), q.clone()
    with torch.cuda.graph(graph):
        y, z = r.apply(x, k, pos)
    pos[:, 100:] = -1
    x.copy_(q.flip(0))
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y[:100], r.apply(q.flip(0)[:100].contiguous(), None, pos[:, :100])) and torch.all(y[100:] == 0)
    r.close()
