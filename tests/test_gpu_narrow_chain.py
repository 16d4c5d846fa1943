"""Products of the narrow tcgen05 kernel one behind the other through the same buffers, atomic and deterministic: each
starts while the one before it, and the kernel that adds up its parts, still run."""
import pytest

import bitmap_encoded_unstructured_gb300 as bsp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("N", [3, 16])
@pytest.mark.parametrize("M,K", [(1024, 4096), (256, 20480), (5120, 5120)])
def test_through_the_same_buffers(M, K, N, deterministic):
    import torch
    g = torch.Generator(device="cuda").manual_seed(M)
    A, W = [], []
    for _ in range(2):
        W.append(torch.randint(-1, 2, (M, K), device="cuda", generator=g).half())
        A.append(bsp.BitmapMatrix(W[-1]))
        A[-1].set_deterministic(deterministic)
    xs = [torch.randint(-2, 3, (N, K), device="cuda", generator=g).half() for _ in range(5)]
    want = [[(x.double() @ w.double().T).half() for x in xs] for w in W]  # small integers: exact in any order
    x, y = torch.empty_like(xs[0]), torch.empty((N, M), dtype=torch.float16, device="cuda")
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for rep in range(200):
        i, j = rep % 5, rep % 2
        x.copy_(xs[i])
        A[j].spmm(x, out=y)
        A[j].spmm(x, out=y)
        bad += (y != want[j][i]).any()
    assert int(bad) == 0
    for a in A:
        a.check()
        a.close()
