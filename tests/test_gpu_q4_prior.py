"""Kernels that start while the one before them still runs: what they wait for then
does not count against the limit of their own waits.

In the test build of the library, with a limit far below the run of the kernel before: a
product of a few CTAs and very many columns, which lets the next kernel start at
once, on the SMs that it leaves idle."""
import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from test_gpu_q4 import dev, matrix, rows, weight

pytestmark = pytest.mark.gpu

POLLS = 200  # a poll waits for two to four microseconds
COLUMNS = 1 << 22


def took(call):
    import torch
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    call()
    b.record()
    b.synchronize()
    return a.elapsed_time(b)


@pytest.fixture(scope="module")
def before():
    """(the test library, a call that runs some milliseconds on eight SMs, its matrix)"""
    import torch
    with bsp.test_library() as T:
        g = torch.Generator(device="cuda").manual_seed(1)
        codes = torch.randint(0, 256, (100, COLUMNS // 2), device="cuda", generator=g, dtype=torch.uint8)
        scales = torch.full((100, COLUMNS // 128), 2.0 ** -6, dtype=torch.float16, device="cuda")
        long = bsp.Int4Matrix.from_arrays(codes, scales)
        x = torch.randn((40, COLUMNS), device="cuda", generator=g).half()
        y = torch.empty((40, 100), dtype=torch.float16, device="cuda")
        long.mm(x, out=y)
        yield T, lambda: long.mm(x, out=y), long
        long.close()


def behind(before, make, call, right):
    """`call(m)` of `make()` behind the long call and under the short limit: no wait runs out, and the outputs are `right`."""
    import torch
    T, long, first = before
    m = make()
    ms = min(took(long) for _ in range(3))
    try:
        assert T.bsp_testing_set_spin_cap(POLLS) == 0 and T.bsp_testing_set_stall(1) == 0
        given_up = took(lambda: call(m))     # how long the limit is
        with pytest.raises(bsp.BspError) as e:
            m.check()
        assert e.value.status == 7
        T.bsp_testing_set_stall(0)
        print(f"the call before takes {ms:.2f} ms, a wait that runs out {given_up:.2f}")
        assert ms > 2 * given_up
        for _ in range(3):
            long()
            y = call(m)
            first.check()
            m.check()
            assert torch.equal(y, right)
    finally:
        T.bsp_testing_set_stall(0)
        T.bsp_testing_set_spin_cap(0)
        m.close()


def product(before, M, K, N, group, dtype):
    w, x = weight(M, K, group, True, dtype, 1), dev(rows(N, K, dtype, 3), dtype)
    m = matrix(w, group, dtype)
    right = m.mm(x)
    m.check()
    m.close()
    behind(before, lambda: matrix(w, group, dtype), lambda m: m.mm(x), right)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("M,K,N,group", [(300, 2048, 40, 64), (256, 1024, 60, 32), (512, 4096, 33, 128)])
def test_wide_product(before, M, K, N, group, dtype):
    """Tiles of 64 columns: both CTAs of a pair start, and free their tensor memory, behind the long call."""
    product(before, M, K, N, group, dtype)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("M,K,N,group", [(1000, 1024, 1300, 64), (2600, 1032, 900, 128), (2600, 2056, 400, 64), (3300, 520, 2000, 32)])
def test_large_tiles(before, M, K, N, group, dtype):
    """Tiles of 128 and 256 columns: a ring of codes no longer than that of the tiles they become."""
    product(before, M, K, N, group, dtype)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("N", [5, 50, 700])
def test_gated(before, N, dtype):
    import torch
    M, K, group = 2600, 1032, 64
    x = dev(rows(N, K, dtype, 3), dtype)

    class Pair:
        def __init__(self):
            self.a, self.b = (matrix(weight(M, K, group, z, dtype, 4), group, dtype) for z in (True, False))

        def check(self):
            self.a.check()

        def close(self):
            self.a.close()
            self.b.close()

    p = Pair()
    right = p.a.gated(p.b, x)
    p.close()
    if N > 32:
        behind(before, Pair, lambda p: p.a.gated(p.b, x), right)
        return
    T, long, first = before  # the narrow kernel has no bounded wait
    p = Pair()
    for _ in range(3):
        long()
        assert torch.equal(p.a.gated(p.b, x), right)
    p.close()
