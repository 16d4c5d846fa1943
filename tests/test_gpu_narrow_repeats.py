"""The narrow tcgen05 kernel gives the same sums however its CTAs' segments fall:
products repeated behind other work, where segments are a step or two long
(spans of 18 steps over tiles of 64 in runs of 16; tiles of one step)."""
import pytest

import bitmap_encoded_unstructured_gb300 as bsp

pytestmark = pytest.mark.gpu


def repeated(A, x, want, times):
    import torch
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for rep in range(times):
        if rep % 3 == 0:
            torch.randn(1 << (10 + rep % 12), device="cuda").sort()
        bad += (A.spmm(x) != want).any()
    A.check()
    return int(bad)


@pytest.mark.parametrize("M,K", [(11008, 4096), (4096, 11008), (11008, 64), (9000, 128)])
def test_int8(M, K):
    import torch
    g = torch.Generator(device="cuda").manual_seed(M)
    W = torch.randint(-127, 128, (M, K), device="cuda", generator=g, dtype=torch.int8)
    W = torch.where(torch.rand((M, K), device="cuda", generator=g) < 0.5, 0, W).to(torch.int8)
    A = bsp.BitmapMatrix(W)
    for N in (8, 16):
        x = torch.randint(-127, 128, (N, K), device="cuda", generator=g, dtype=torch.int8)
        want = (x.double() @ W.double().T).to(torch.int32)  # exact: below 2^53
        assert repeated(A, x, want, 600) == 0
    A.close()


@pytest.mark.parametrize("M,K", [(11008, 64), (20000, 128), (11008, 192)])
def test_fp16_small_k(M, K):
    """Every tile a segment of K / 64 steps: the sums of few products of small integers are exact."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(M)
    W = torch.randint(-3, 4, (M, K), device="cuda", generator=g).half()
    A = bsp.BitmapMatrix(W)
    for N in (4, 16):
        x = torch.randint(-2, 3, (N, K), device="cuda", generator=g).half()
        want = (x.double() @ W.double().T).half()  # integers up to 6 K = 1152: exact in fp16
        assert repeated(A, x, want, 600) == 0
    A.close()
