"""Products of 4-bit weights one behind the other through buffers that are used again: each reads what the kernel
before it has just written, and starts while that one still runs."""
import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from test_gpu_q4 import dev, matrix, rows, weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("N", [1, 7, 16, 30, 90, 600])
@pytest.mark.parametrize("size", [256, 2048, 5120])
def test_through_one_pair_of_buffers(size, N, dtype):
    import torch
    w, u = weight(size, size, 128, True, dtype, 1), weight(size, size, 128, False, dtype, 2)
    w, u = ((c, s / size ** 0.5 / 4, z) for c, s, z in (w, u))  # outputs about as large as inputs
    a, b = matrix(w, 128, dtype), matrix(u, 128, dtype)
    start = [dev(rows(N, size, dtype, 3 + i), dtype) for i in range(6)]
    x, y = torch.empty_like(start[0]), torch.empty_like(start[0])

    def steps(i, between):
        """Six layers, each into the other buffer."""
        x.copy_(start[i])
        between()
        for k in range(3):
            (a.mm(x, out=y) if k != 1 else a.gated(b, x, out=y))
            between()
            b.mm(y, out=x)
            between()
        return x

    want = []
    for i in range(6):
        want.append(steps(i, torch.cuda.synchronize).clone())
    torch.cuda.synchronize()
    got = []
    for rep in range(20):
        for i in range(6):
            got.append((i, steps(i, lambda: None).clone()))
    torch.cuda.synchronize()
    assert all(torch.isfinite(t).all() for t in want)
    assert all(torch.equal(t, want[i]) for i, t in got)
    graph, first = torch.cuda.CUDAGraph(), start[0].clone()
    with torch.cuda.graph(graph):
        x.copy_(first)
        for k in range(3):
            (a.mm(x, out=y) if k != 1 else a.gated(b, x, out=y))
            b.mm(y, out=x)
    for i in (3, 1, 5):
        first.copy_(start[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want[i])
    for m in (a, b):
        m.check()
        m.close()
