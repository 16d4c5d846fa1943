"""Outputs that the rotary makes itself hold no stale bits: rows that are not there are zeros."""
import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from test_gpu_rope import close, data, dev, places

pytestmark = pytest.mark.gpu


def litter(n, dtype):
    """Leaves NaN in the memory that the next allocations take."""
    import torch
    for _ in range(4):
        torch.full((n,), float("nan"), dtype=dtype, device="cuda")
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows", [1, 50, 4000])
@pytest.mark.parametrize("dim,rot", [(96, 48), (64, 64), (80, 24), (24, 8)])
def test_rows_that_are_not_there(dim, rot, rows, interleaved, dtype):
    import torch
    r = bsp.Rotary(dim, rot=rot, sections=[rot // 2 - 2, 1, 1], interleaved=interleaved)
    q, k = data(rows, 5, dim, dtype, 1), data(rows, 2, dim, dtype, 2)
    pos = places(3, rows, 4000, 3)
    pos[0, ::3], pos[2, 1::7], pos[:, -1] = -1, -2 ** 31, -1
    gone = (pos < 0).any(0)
    a, b = dev(q, dtype), dev(k, dtype)
    for n in (a.numel(), b.numel()):
        litter(n, a.dtype)
    y, z = r.apply(a, b, dev(pos))
    close(y, q, pos, r, dtype)
    close(z, k, pos, r, dtype)
    assert torch.all(y[dev(gone)] == 0) and torch.all(z[dev(gone)] == 0)
    # one output given, one made: the given one's rows are left
    mine = torch.full_like(b, 3.0)
    litter(a.numel(), a.dtype)
    y2, z2 = r.apply(a, b, dev(pos), out=(None, mine))
    assert z2 is mine and torch.equal(y2, y) and torch.all(mine[dev(gone)] == 3)
    assert torch.equal(mine[dev(~gone)], z[dev(~gone)])
    r.close()


@pytest.mark.parametrize("clear", [0, 1])
def test_in_place(clear):
    """The C entry point on its own input: rows that are not there are left, or become zeros if asked for."""
    import torch
    r = bsp.Rotary(64, rot=32)
    x = data(30, 3, 64, "float16", 1)
    pos = places(1, 30, 500, 2)
    pos[0, 4:9] = -1
    t, p = dev(x, "float16"), dev(pos[0])
    q = bsp._ROPE_ROWS(t.data_ptr(), t.data_ptr(), 3, clear, 192, 64, 192, 64)
    assert bsp.lib().bsp_rope_apply(r.h, q, None, bsp.BSP_FP16, 30, p.data_ptr(), 30, 0,
                                    torch.cuda.current_stream().cuda_stream) == 0
    close(t, x, pos, r, "float16")
    assert torch.equal(t[4:9], torch.zeros_like(t[4:9]) if clear else dev(x, "float16")[4:9])
    r.close()
