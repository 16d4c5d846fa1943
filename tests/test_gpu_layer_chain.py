"""Steps of a decoder layer with nothing waited for between its operators: each starts while the one before it still runs, through
buffers that are used again, and gives what it gives when every call is waited for."""
import pytest

import bitmap_encoded_unstructured_gb300 as bsp

pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV, DIM, INNER = 1024, 16, 4, 64, 2816


class Layer:
    def __init__(self, dtype, pruned):
        import torch
        g = torch.Generator(device="cuda").manual_seed(1)

        def weight(rows, cols):
            W = (torch.randn((rows, cols), device="cuda", generator=g) * cols ** -0.5).to(dtype)
            if not pruned:
                return bsp.Int4Matrix(W, group=64)
            m = bsp.BitmapMatrix(torch.where(torch.rand((rows, cols), device="cuda", generator=g) < 0.5, W, 0).half())
            m.set_deterministic()
            return m

        self.dtype, self.pruned = dtype, pruned
        self.qkv, self.out, self.down = (weight(*s) for s in (((HEADS + 2 * KV) * DIM, HIDDEN), (HIDDEN, HIDDEN), (HIDDEN, INNER)))
        W = [(torch.randn((INNER, HIDDEN), device="cuda", generator=g) * HIDDEN ** -0.5).to(dtype) for _ in range(2)]
        self.gate, self.up = (bsp.Int4Matrix(w, group=128) for w in W)
        self.turn = bsp.Rotary(DIM)

    def close(self):
        for m in (self.qkv, self.out, self.down, self.gate, self.up):
            m.check()
            m.close()
        self.turn.close()

    def mm(self, m, x, out):
        return m.spmm(x, out=out) if self.pruned else m.mm(x, out=out)

    def run(self, new, steps, between):
        """`steps` steps of requests with new[b] rows each (their own rows fed back as the next step's input), from an empty cache."""
        import torch
        rows = sum(new)
        i32 = dict(dtype=torch.int32, device="cuda")
        cache = bsp.KvCache.empty(256, KV, DIM, 64)
        table, free, count = torch.full((len(new), 64), -1, **i32), torch.arange(256, **i32), torch.tensor([256], **i32)
        ctx, asked = torch.zeros(len(new), **i32), torch.tensor(new, **i32)
        a = torch.zeros((rows, HEADS + 2 * KV, DIM), dtype=self.dtype, device="cuda")
        y, h, m = (torch.zeros((rows, n), dtype=self.dtype, device="cuda") for n in (HIDDEN, HIDDEN, INNER))
        x = torch.randn((rows, HIDDEN), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).to(self.dtype)
        kept = []
        for _ in range(steps):
            step = cache.plan(ctx, asked, table, free, count, tokens=rows, max_new=max(new))
            ctx, count = step.seq_len, step.free_count
            between()
            self.mm(self.qkv, x, a.view(rows, -1))
            between()
            q, k, v = a[:, :HEADS], a[:, HEADS:HEADS + KV], a[:, HEADS + KV:]
            self.turn.apply(q, k, step.positions, out=(q, k))
            between()
            cache.append(step, k, v)
            between()
            cache.attention(step, q, out=y.view(rows, HEADS, DIM))
            between()
            self.mm(self.out, y, h)
            between()
            self.gate.gated(self.up, h, out=m)
            between()
            self.mm(self.down, m, x)
            between()
            kept += [x.clone(), a.clone(), y.clone()]
            x.copy_(x / (x.float().square().mean(1, keepdim=True) + 1e-6).sqrt())  # a norm: sizes stay
            between()
        torch.cuda.synchronize()
        cache.check()
        kept += [cache.k.clone(), cache.v_scale.clone()]
        cache.close()
        return kept


@pytest.mark.parametrize("pruned", [False, True])
@pytest.mark.parametrize("new", [[1], [1] * 12, [1] * 25, [7, 1, 20], [50, 1, 3], [300, 130]])
def test_steps(new, pruned):
    import torch
    for dtype in (torch.float16,) if pruned else (torch.float16, torch.bfloat16):
        layer = Layer(dtype, pruned)
        want = layer.run(new, 6, torch.cuda.synchronize)
        assert all(torch.isfinite(t.float()).all() for t in want)
        for _ in range(6):
            got = layer.run(new, 6, lambda: None)
            bad = [i for i, (a, b) in enumerate(zip(got, want)) if not torch.equal(a, b)]
            assert not bad, (dtype, bad)
        layer.close()
