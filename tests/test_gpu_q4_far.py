"""4-bit weights, outputs and rotary rows whose offsets pass 32 bits, on sampled rows against the definition in 64 bits."""
import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from test_gpu_q4_tiles import defined, near, rows

pytestmark = pytest.mark.gpu


def sampled(codes, scales, zeros, group, at):
    """(None, scales, W) of the rows `at`, in 64 bits, as test_gpu_q4_tiles' helpers take them."""
    import torch
    c = codes[at]
    K = 2 * c.shape[1]
    W = torch.stack((c & 15, c >> 4), -1).reshape(len(at), K).double()
    W -= zeros[at].double().repeat_interleave(group, 1)[:, :K]
    W *= scales[at].double().repeat_interleave(group, 1)[:, :K]
    return None, scales[at].double(), W


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_weights_past_4_gb(dtype):
    import torch
    M, K, group = 9000, 1 << 20, 128                     # 4.7 GB of codes
    t = getattr(torch, dtype)
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 256, (M, K // 2), device="cuda", generator=g, dtype=torch.uint8)
    scales = torch.rand((M, K // group), device="cuda", generator=g).mul_(1e-4).add_(1e-5).to(t)
    zeros = torch.randint(0, 16, (M, K // group), device="cuda", generator=g, dtype=torch.uint8)
    m = bsp.Int4Matrix.from_arrays(codes, scales, zeros, group=group)
    at = torch.tensor([0, 1, 127, 4095, 4096, 8191, 8192, 8959, 8960, M - 1], device="cuda")
    w = sampled(codes, scales, zeros, group, at)
    for N in (1, 12, 32, 40, 300):
        x = rows(N, K, t, N)
        want, before = defined(x, w, group)
        near(m.mm(x)[:, at].contiguous(), want, before, N)
    m.check()
    back = m.arrays()
    assert torch.equal(back[0], codes) and torch.equal(back[1], scales) and torch.equal(back[2], zeros)
    del back
    assert torch.equal(m.decode()[at], w[2].to(t))
    m.close()


def test_outputs_past_32_bits():
    import torch
    M, K, N, group = 40000, 64, 60001, 32                # 2.4e9 outputs
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 256, (M, K // 2), device="cuda", generator=g, dtype=torch.uint8)
    scales = torch.rand((M, K // group), device="cuda", generator=g).half()
    zeros = torch.full((M, K // group), 8, device="cuda", dtype=torch.uint8)
    m = bsp.Int4Matrix.from_arrays(codes, scales, None, group=group)
    x = rows(N, K, torch.float16, 2)
    at, n = torch.tensor([0, 130, 39999], device="cuda"), torch.tensor([0, 1, 53686, 53687, 53688, 60000], device="cuda")
    want, before = defined(x[n], sampled(codes, scales, zeros, group, at), group)
    near(m.mm(x)[n][:, at], want, before, "mm")
    y = m.gated(m, x, activation="relu")[n][:, at]
    near(y, want.clamp(min=0) * want, 2 * before * want.abs() + before * before, "gated")
    m.check()
    m.close()


def test_rotary_rows_past_32_bits():
    import torch
    rows_, heads, dim = 40000, 64, 1024                  # 2.6e9 values, in place
    r = bsp.Rotary(dim, rot=64)
    t = torch.full((rows_, heads, dim), 1.0, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(rows_, dtype=torch.int32, device="cuda")
    r.apply(t, None, pos, out=(t, None))
    one = torch.ones((1, heads, dim), dtype=torch.bfloat16, device="cuda")
    for p in (0, 1, 32767, 32768, 39999):
        assert torch.equal(t[p:p + 1], r.apply(one, None, pos[p:p + 1]))
    assert bool((t[:, :, 64:] == 1).all())
    r.close()
