"""A refused allocation is that call's own: the next calls are not refused for it."""
import ctypes as C

import numpy as np
import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from test_gpu_q4 import dev, matrix, weight

pytestmark = pytest.mark.gpu

OOM = 5
M, K = 2 ** 31 - 1, 128  # 137 GB of codes


def too_large(L):
    """A call that asks for more memory than there is before it does anything else."""
    h = C.c_void_p(7)
    st = L.bsp_q4_import(0x1000, 0x1000, None, 0, M, K, 32, None, C.byref(h))
    assert not h.value
    return st


def test_after_a_refused_allocation():
    import torch
    room = torch.cuda.mem_get_info()[0] - (60 << 30)
    held = torch.empty(max(room, 0), dtype=torch.uint8, device="cuda")  # never touched
    try:
        assert torch.cuda.mem_get_info()[0] < M * K // 2 - (1 << 30)        # the call below cannot get its memory
        L = bsp.lib()
        w = weight(70, 136, 32, True, "float16", 3)
        m = matrix(w, 32, "float16")
        assert too_large(L) == OOM
        n = matrix(w, 32, "float16")
        assert too_large(L) == OOM
        assert all(torch.equal(a, b) for a, b in zip(m.arrays(), n.arrays()))
        assert too_large(L) == OOM
        want = m.decode()
        assert too_large(L) == OOM
        e = bsp.Int4Matrix(want, group=32)
        assert too_large(L) == OOM
        b = bsp.BitmapMatrix(dev(np.eye(128, dtype=np.float16)))
        for h in (m, n, e, b):
            h.close()
    finally:
        del held
        torch.cuda.empty_cache()  # to the library's own allocations
