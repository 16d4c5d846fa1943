"""The attention block of a decoder layer, pruned weights and 8-bit KV cache together.

    python examples/kv_decoder_layer.py [hidden] [heads]

The QKV and output projections are bitmap-encoded pruned weights
(``BitmapMatrix``); between them a step's pages are planned from request
lengths, the new K and V rows are quantised into the paged cache and the
queries attend over it (``KvCache``).  Prompts and single tokens go the same
way: the rows of a step are the concatenated new rows of its requests.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bitmap_encoded_unstructured_gb300 as bsp  # noqa: E402


class AttentionBlock:
    """y = x + W_out attention(W_qkv x), over one layer's cache."""

    def __init__(self, w_qkv, w_out, heads: int, cache: bsp.KvCache):
        self.qkv, self.out = bsp.BitmapMatrix(w_qkv), bsp.BitmapMatrix(w_out)
        self.heads, self.cache = heads, cache

    def __call__(self, x, step: bsp.KvStep):
        rows, hidden = x.shape
        qkv = self.qkv.spmm(x).view(rows, 3, self.heads, hidden // self.heads)
        self.cache.append(step, qkv[:, 1], qkv[:, 2])           # strided views: nothing is copied
        y = self.cache.attention(step, qkv[:, 0])
        return x + self.out.spmm(y.view(rows, hidden))

    def close(self):
        self.qkv.close()
        self.out.close()


class Server:
    """Block table, free list and lengths of a batch of request slots, all on
    the GPU: a step needs no length on the host but its row count."""

    def __init__(self, cache: bsp.KvCache, batch: int, width: int):
        i32 = dict(dtype=torch.int32, device=cache.device)
        self.cache = cache
        self.table = torch.full((batch, width), -1, **i32)
        self.free = torch.arange(cache.pages - 1, -1, -1, **i32)  # page 0 comes off the top first
        self.count = torch.tensor([cache.pages], **i32)
        self.length = torch.zeros(batch, **i32)

    def step(self, new, tokens: int, max_new: int) -> bsp.KvStep:
        """Plan a step: ``new`` rows for each slot (-1 ends its request)."""
        out = bsp.KvStep.empty(self.table.shape[0], tokens, self.cache.device, free_count=self.count)
        plan = self.cache.plan(self.length, new, self.table, self.free, self.count, tokens, out=out, max_new=max_new)
        self.length = plan.seq_len
        return plan


def run(hidden=512, heads=8, prompts=(37, 5, 120), tokens=6, page=16, seed=0):
    """Three prompts, then ``tokens`` decoding steps; returns what a check needs."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def pruned(rows):
        w = torch.randn(rows, hidden, device="cuda", generator=g) * hidden ** -0.5
        return torch.where(w.abs() < 0.67 * hidden ** -0.5, 0, w).half()  # about half of them zeros

    w_qkv, w_out = pruned(3 * hidden), pruned(hidden)
    pages = sum(-(-(n + tokens) // page) for n in prompts) + 1
    cache = bsp.KvCache.empty(pages, heads, hidden // heads, page)
    block, server = AttentionBlock(w_qkv, w_out, heads, cache), Server(cache, len(prompts), 64)
    inputs, outputs = [], []
    for new in [prompts] + [(1,) * len(prompts)] * tokens:
        x = torch.randn(sum(new), hidden, device="cuda", generator=g).half()
        step = server.step(torch.tensor(new, dtype=torch.int32, device="cuda"), sum(new), max(new))
        inputs.append(x)
        outputs.append(block(x, step))
    last = server.step(torch.full((len(prompts),), -1, dtype=torch.int32, device="cuda"), 1, 1)
    cache.check()
    freed = int(last.free_count)
    block.close()
    cache.close()
    return dict(w_qkv=w_qkv, w_out=w_out, prompts=prompts, inputs=inputs, outputs=outputs, freed=freed, pages=pages)


if __name__ == "__main__":
    hidden, heads = (int(v) for v in (sys.argv[1:] + ["5120", "40"])[:2]) if len(sys.argv) != 2 else (int(sys.argv[1]), 8)
    r = run(hidden, heads)
    print(f"{len(r['inputs'])} steps of {len(r['prompts'])} requests, hidden {hidden}, {heads} heads: "
          f"outputs {tuple(r['outputs'][0].shape)} and {tuple(r['outputs'][-1].shape)}, "
          f"{r['freed']} of {r['pages']} pages free at the end")
