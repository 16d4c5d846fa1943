"""Attention over the paged 8-bit KV cache for queries out of the ordinary."""
import numpy as np
import pytest

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
