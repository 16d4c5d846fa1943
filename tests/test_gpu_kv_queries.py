"""Attention over the paged 8-bit KV cache for queries out of the ordinary."""
import numpy as np
import pytest

from oracle import kv_cache as kv
from test_gpu_kv_attention import case, check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("lens,heads,kvh,dim", [
    ([(300, 1), (0, 1), (40, 1), (2000, 1)], 8, 2, 64),         # single tokens, segments cut between warps
    ([(500, 5), (9, 3)], 4, 1, 128), ([(70, 2), (3, 40)], 4, 2, 256),
    ([(0, 700), (64, 1)], 8, 2, 128),                           # a prompt beside a single token
    ([(3000, 140)], 8, 1, 128)])                                # its cached rows split
def test_nan_queries(lens, heads, kvh, dim, dtype):
    """A NaN in a query gives a NaN row and lse, an infinite one too, as the
    formula does; rows that see nothing stay zeros, other rows what they are."""
    import torch
    c = case(lens, heads, kvh, dim, 16, getattr(torch, dtype), 70 + dim)
    clean = run(c)
    rows = c["q"].shape[0]
    g = np.random.default_rng(71)
    bad = torch.zeros((rows, heads), dtype=torch.bool, device="cuda")
    for i, (r, h) in enumerate({(0, 0), (rows - 1, heads - 1), (int(g.integers(rows)), int(g.integers(heads)))}):
        bad[r, h] = True
        # an infinite query times codes of both signs (and zeros): infinity less infinity
        c["q"][r, h, int(g.integers(dim))] = float("nan")
        if i == 1:
            c["q"][r, h] = float("inf")
    out, lse = run(c)
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    c["q"][bad] = 0
    reference = run(c)
    out[bad], lse[bad] = reference[0][bad], reference[1][bad]
    check(c, out, lse)
    assert torch.isfinite(clean[0]).all()


@pytest.mark.parametrize("new", [1, 4, 300])
def test_nan_queries_that_see_nothing(new):
    import torch
    c = case([(0, new), (30, new)], 8, 2, 64, 16, torch.float16, 75)
    c["table"][0, :] = -1
    c["q"][:new] = float("nan")
    out, lse = run(c)
    assert (out[:new] == 0).all() and torch.isneginf(lse[:new]).all()
    assert torch.isfinite(out[new:]).all()


@pytest.mark.parametrize("down", [8, 16, 18])
@pytest.mark.parametrize("new", [1, 6, 300])
def test_bfloat16_queries_of_wide_range(new, down):
    """One value of each query is 2^down times the others and meets codes of 0,
    so the logits are the small values' alone.  Scaled by their row's power of
    two, bfloat16 values are exact in fp16 down to 2^-17 of it; below, each is
    off by at most 2^-25 of it, so a logit by scale 2^-25 sum |k| more."""
    import torch
    heads, dim, page = 4, 64, 16
    c = case([(200, new), (17, new)], heads, 2, dim, page, torch.bfloat16, 90 + down)
    c["q"] *= 2.0 ** -down
    c["q"][:, :, 5] = 1.0                                   # the row's power of two is 1 (or 2^-down |q|)
    c["q"].clamp_(-1, 1)
    c["k"][:, :, :, 5] = 0
    scale = dim ** -0.5 * 2.0 ** down
    out, lse = run(c, scale=scale)
    q = c["q"].float().cpu().numpy()
    ref, rl, weight, spread, seen = kv.attention(q, c["k"], c["v"], c["ks"], c["vs"], c["table"], c["seq"], c["start"],
                                                 page, scale)
    k = np.abs(c["k"].astype(np.float64)).sum(-1).max(2) * c["ks"]     # largest sum |k| of a page and head
    d = dim * 2.0 ** -23 * spread[..., None] + 2.0 ** -20 + scale * 2.0 ** -25 * k.max()
    vmax = 127 * c["vs"].max()
    bound = 2.0 ** -8 * np.abs(ref) + (2 * d + 2.0 ** -11) * weight + seen[..., None] * 2.0 ** -24 * vmax + 1e-7
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()
    assert (np.abs(lse.double().cpu().numpy() - rl) <= d[..., 0] + 2.0 ** -20 * (1 + np.abs(rl))).all()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("heads,kvh,dim", [(2, 2, 64), (8, 2, 128), (6, 2, 256)])
@pytest.mark.parametrize("new", [1, 4, 40, 700])
def test_v_scales_of_zero_beside_large_ones(heads, kvh, dim, new, dtype):
    """Rows that have seen V scales of 0 only, where a page that they do not see
    (or whose weights vanish) has a large one."""
    import torch
    page = 16
    c = case([(3 * page - 1, new), (300, new)], heads, kvh, dim, page, getattr(torch, dtype), 60 + dim)
    for b in range(2):
        zero = c["table"][b][:kv.pages_of(int(c["seq"][b]), page) // 2 + 1]
        c["vs"][:] = 8.0
        c["vs"][zero[zero >= 0]] = 0
        check(c, *run(c), what="unseen")
        check(c, *run(c, window=20), window=20, what="window")
    # weights that vanish: the second request's rows see logits thousands
    # apart; its largest are where V is 0
    d = dict(c, k=c["k"].copy(), ks=c["ks"].copy(), q=torch.ones_like(c["q"]))
    d["vs"] = np.full_like(c["vs"], 100.0)
    d["ks"][:] = 1.0
    for j, p in enumerate(d["table"][1][:kv.pages_of(int(d["seq"][1]), page)]):
        d["k"][p] = 100 if j % 3 == 0 else -100
        d["vs"][p] = 0 if j % 3 == 0 else 100.0
    out, lse = run(d, scale=1.0)
    n = int(d["start"][1])
    assert (out[n:] == 0).all() and torch.isfinite(lse[n:]).all()


@pytest.mark.parametrize("power", [-110, -122, -126])
@pytest.mark.parametrize("lens,heads,kvh,dim", [([(300, 1), (40, 1)], 8, 2, 64), ([(500, 5)], 4, 1, 128),
                                                ([(70, 30)], 4, 2, 256), ([(0, 700), (64, 1)], 8, 2, 128)])
def test_v_scales_near_the_smallest_number(lens, heads, kvh, dim, power):
    """Outputs scale with V down to the smallest bfloat16 numbers: the same
    calls with V scales of 1 and of 2^power, where a weight keeps at least 2^-9
    of itself in fp16 (rows of equal logits) and an output is rounded to 2^-8."""
    import torch
    c = case(lens, heads, kvh, dim, 16, torch.bfloat16, 95)
    c["ks"][:] = 0
    c["v"] = np.abs(c["v"])
    c["vs"][:] = 1
    want, wl = run(c)
    c["vs"][:] = 2.0 ** power
    out, lse = run(c)
    assert torch.equal(lse, wl)
    off = (out.double() * 2.0 ** -power - want.double()).abs()
    assert (off <= 2.0 ** -7 * want.double()).all()
