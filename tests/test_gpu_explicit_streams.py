"""Calls given a stream of their own, while the current stream is still busy: what a
call makes for itself (a contiguous copy of a strided tensor, an output that it allocates) is
ordered with the stream it was given.  The caller orders only what it hands over."""
import pytest

import bitmap_encoded_unstructured_gb300 as bsp

pytestmark = pytest.mark.gpu


def busy():
    """Some ten milliseconds of work on the current stream."""
    import torch
    a = torch.randn((8192, 8192), device="cuda")
    for _ in range(8):
        a = torch.sin(a @ a)
    return a


def litter(*tensors):
    """Leaves wrong values in the memory that copies of these tensors will take."""
    import torch
    kept = [torch.full(t.shape, 3, dtype=t.dtype, device="cuda") for t in tensors for _ in range(8)]
    del kept
    torch.cuda.synchronize()


def transposed(shape, dtype, seed):
    """A matrix whose rows are not contiguous, there for every stream."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    if dtype is torch.int8:
        t = torch.randint(-7, 8, shape[::-1], device="cuda", generator=g, dtype=torch.int8)
    elif dtype is torch.uint8:
        t = torch.randint(0, 256, shape[::-1], device="cuda", generator=g, dtype=torch.uint8)
    else:
        t = torch.randn(shape[::-1], device="cuda", generator=g).to(dtype)
    torch.cuda.synchronize()
    return t.t()


def by_handle(s):
    return s.cuda_stream


FORMS = [lambda s: s, by_handle]


@pytest.mark.parametrize("form", FORMS, ids=["stream", "handle"])
def test_int4_from_a_strided_weight(form):
    import torch
    W = transposed((640, 1024), torch.bfloat16, 1)
    right = bsp.Int4Matrix(W.contiguous(), group=64, zeros=True)
    litter(W)
    s = torch.cuda.Stream()
    work = busy()
    m = bsp.Int4Matrix(W, group=64, zeros=True, stream=form(s))
    assert all(torch.equal(a, b) for a, b in zip(m.arrays(), right.arrays()))
    del work
    m.close()
    right.close()


@pytest.mark.parametrize("form", FORMS, ids=["stream", "handle"])
def test_int4_from_strided_arrays(form):
    import torch
    codes, zeros = transposed((512, 640), torch.uint8, 2), transposed((512, 20), torch.uint8, 3) % 16
    zeros = zeros.t().contiguous().t()
    scales = transposed((512, 20), torch.float16, 4)
    bsp.Int4Matrix.from_arrays(codes.contiguous(), scales.contiguous(), zeros.contiguous(), group=64).close()  # kernels loaded
    litter(codes, scales, zeros)
    s = torch.cuda.Stream()
    work = busy()
    m = bsp.Int4Matrix.from_arrays(codes, scales, zeros, group=64, stream=form(s))
    for got, want in zip(m.arrays(), (codes, scales, zeros)):
        assert torch.equal(got, want)
    del work
    m.close()


@pytest.mark.parametrize("kind", ["fp16", "int8", "union", "union reordered"])
def test_pruned_formats_from_a_strided_weight(kind):
    import torch
    W = transposed((512, 768), torch.float16 if kind == "fp16" else torch.int8, 5)
    make = {"fp16": bsp.BitmapMatrix, "int8": bsp.BitmapMatrix,
            "union": lambda W, stream: bsp.UnionMatrix(W, 4, stream=stream),
            "union reordered": lambda W, stream: bsp.UnionMatrix(W, 4, stream=stream, reorder=True)}[kind]
    make(W.contiguous(), stream=None).close()  # kernels loaded: no waits for that
    litter(W)
    s = torch.cuda.Stream()
    work = busy()
    m = make(W, stream=s)
    assert torch.equal(m.decode(), W)
    del work
    m.close()


def test_bitmap_from_strided_arrays():
    import torch
    W = transposed((512, 768), torch.float16, 6).contiguous()
    m = bsp.BitmapMatrix(W)
    arrays = [torch.stack((a, a), 1)[:, 0] for a in m.arrays()]  # every second element
    bsp.BitmapMatrix.from_arrays(*[a.contiguous() for a in arrays], 512, 768).close()
    litter(*arrays)
    s = torch.cuda.Stream()
    work = busy()
    n = bsp.BitmapMatrix.from_arrays(*arrays, 512, 768, stream=s)
    assert torch.equal(n.decode(), W)
    del work
    m.close()
    n.close()
