"""The narrow tcgen05 kernel, started while the kernel before it still runs: that kernel's time does not count against the
limit of its waits."""
import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from test_gpu_q4_prior import POLLS, before  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [4, 16])
@pytest.mark.parametrize("M,K", [(2000, 64), (11008, 64), (9000, 192), (128, 256),    # a tile ends in a decoder group's first step
                                 (20000, 2048), (11008, 4096)])                       # dense: as few stages as there may be
def test_products(before, M, K, N):  # noqa: F811
    import torch
    T, long, first = before
    g = torch.Generator(device="cuda").manual_seed(M)
    W = torch.randint(1, 4, (M, K), device="cuda", generator=g).half()  # no zeros
    x = torch.randint(-2, 3, (N, K), device="cuda", generator=g).half()
    want = (x.double() @ W.double().T).half()                           # sums of small integers: exact in any order
    A = bsp.BitmapMatrix(W)
    try:
        assert torch.equal(A.spmm(x), want)
        A.check()
        assert T.bsp_testing_set_spin_cap(POLLS) == 0
        for _ in range(3):
            long()
            y = A.spmm(x)
            first.check()
            A.check()
            assert torch.equal(y, want)
    finally:
        T.bsp_testing_set_spin_cap(0)
        A.close()
