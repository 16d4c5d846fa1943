"""Rotary positions of prompts long enough that a block turns three to eight rows, against the definition in 64 bits."""
import pytest

import bitmap_encoded_unstructured_gb300 as bsp

pytestmark = pytest.mark.gpu


def defined(x, pos, r, inverse):
    """The turned rows in 64 bits, on the GPU, and the bound of oracle.rope.bound before its last rounding."""
    import torch
    half = r.rot // 2
    at = pos.double()[torch.tensor(r.axis, device="cuda")].t() * torch.tensor(r.freqs, dtype=torch.float64, device="cuda")
    c, s = (f(-at if inverse else at)[:, None] * r.scale for f in (torch.cos, torch.sin))
    y = x.double()
    first = (..., slice(0, r.rot, 2) if r.interleaved else slice(0, half))
    second = (..., slice(1, r.rot, 2) if r.interleaved else slice(half, r.rot))
    a, b = y[first], y[second]
    want, before = y.clone(), torch.zeros_like(y)
    want[first], want[second] = a * c - b * s, b * c + a * s
    both = (a.abs() + b.abs()) * abs(r.scale) * (torch.pi * 2.0 ** -24 + 2.0 ** -21 + 2 * torch.pi * 2.0 ** -31)
    before[first] = before[second] = both
    return want, before


def near(y, want, before):
    import torch
    step, tiny = {torch.float16: (2.0 ** -11, 2.0 ** -25), torch.bfloat16: (2.0 ** -8, 2.0 ** -134)}[y.dtype]
    off = (y.double() - want).abs() - (before + (want.abs() + before) * step + tiny)
    assert bool((off <= 0).all()), (float(off.max()), int((off > 0).sum()))


# rows / (8 blocks x 152 SMs) rows a block, 1 to 8
ROWS = [1216 * 3 + 5, 1216 * 4, 1216 * 5 + 1, 1216 * 6 + 700, 1216 * 7 + 3, 1216 * 8, 1216 * 9 + 7, 30001]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot,sections,heads,kv", [(128, 128, [16, 24, 24], 5, 1), (80, 24, [12], 3, 2), (64, 64, [20, 12], 1, 0),
                                                       (96, 8, None, 2, 2)])
def test_prompts(dim, rot, sections, heads, kv, interleaved, dtype):
    import torch
    r = bsp.Rotary(dim, rot=rot, sections=sections, cyclic=True, interleaved=interleaved, scale=1.25)
    g = torch.Generator(device="cuda").manual_seed(dim)
    for i, rows in enumerate(ROWS):
        qkv = torch.randn((rows, heads + 2 * kv, dim), device="cuda", generator=g).to(getattr(torch, dtype))
        pos = torch.randint(0, 2 ** 31 - 1 if i % 2 else 40000, (r.axes, rows), device="cuda", generator=g, dtype=torch.int32)
        pos[0, 3::11], pos[-1, -4:] = -1, -7
        live = (pos >= 0).all(0)
        q, k = qkv[:, :heads], qkv[:, heads:heads + kv]
        before = qkv.clone()
        for inverse in (False, True):
            new = torch.full((rows, heads, dim), 3.0, dtype=qkv.dtype, device="cuda")
            y, z = r.apply(q, k, pos, out=(new, torch.full((rows, kv, dim), 3.0, dtype=qkv.dtype, device="cuda")), inverse=inverse)
            for got, x in ((y, q), (z, k)):
                want, lim = defined(x, pos, r, inverse)
                near(got[live], want[live], lim[live])
                assert bool((got[~live] == 3).all())
        r.apply(q, k, pos, out=(q, k), inverse=True)  # where they are
        assert torch.equal(q[live], y[live]) and torch.equal(k[live], z[live])
        assert torch.equal(qkv[~live], before[~live]) and torch.equal(qkv[:, heads + kv:], before[:, heads + kv:])
    r.close()
