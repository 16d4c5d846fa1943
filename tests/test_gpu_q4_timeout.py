"""Waits of the wide 4-bit products that run out, in the test build of the
library: the kernel drains what is in flight and returns, the error word says so
once, and the next call on the same matrix is right."""
import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from test_gpu_q4 import dev, matrix, rows, weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("M,K,N,group", [(300, 1024, 33, 64), (256, 512, 60, 128), (130, 4096, 100, 32), (512, 1024, 200, 128)])
def test_wait_that_runs_out(M, K, N, group, dtype):
    import torch
    w, u = weight(M, K, group, True, dtype, 1), weight(M, K, group, False, dtype, 2)
    x = dev(rows(N, K, dtype, 3), dtype)
    m, up = matrix(w, group, dtype), matrix(u, group, dtype)
    want = m.mm(x), m.gated(up, x)
    m.check()
    m.close()
    up.close()
    with bsp.test_library() as T:
        m, up = matrix(w, group, dtype), matrix(u, group, dtype)
        for call, right in ((lambda: m.mm(x), want[0]), (lambda: m.gated(up, x), want[1])):
            try:
                assert T.bsp_testing_set_stall(1) == 0 and T.bsp_testing_set_spin_cap(2000) == 0
                call()
                with pytest.raises(bsp.BspError) as e:
                    m.check()
                assert e.value.status == 7
            finally:
                T.bsp_testing_set_stall(0)
                T.bsp_testing_set_spin_cap(0)
            m.check()  # cleared
            assert torch.equal(call(), right)
            m.check()
        m.close()
        up.close()
