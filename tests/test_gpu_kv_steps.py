"""Steps of the paged 8-bit KV cache one behind the other, with nothing in
between that waits for the device."""
import numpy as np
import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from oracle import kv_cache as kv
from test_gpu_kv_cache import dev

pytestmark = pytest.mark.gpu


def test_two_steps_take_turns():
    """A step's lengths are the next plan's, without a copy; the lengths and
    offsets stand beside the block table's rows, in one buffer."""
    import torch
    page, pages, batch, width = 16, 200, 7, 12
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = bsp.KvCache.empty(pages, 1, 16, page)
    buf = torch.full((batch, width + 20), -1, **i32)
    table, count = buf[:, :width], torch.tensor([pages], **i32)
    free = torch.arange(pages, **i32)
    steps = [bsp.KvStep.empty(batch, 64, free_count=count) for _ in range(2)]
    for i, s in enumerate(steps):
        s.seq_len, s.granted = buf[2 * i, width:width + batch], buf[2 * i + 1, width:width + batch]
        s._out = tuple(t.data_ptr() for t in (s.seq_len, s.q_start, s.granted, s.slots, s.positions, s.free_count))
    ctx = torch.zeros(batch, **i32)
    t, f, n, c = np.full((batch, width), -1, np.int32), np.arange(pages, dtype=np.int32), pages, [0] * batch
    g = np.random.default_rng(4)
    for i in range(9):
        new = g.integers(0, 9, batch)
        new[g.random(batch) < 0.1] = -1
        step = cache.plan(ctx, dev(new.astype(np.int32)), table, free, count, tokens=64, out=steps[i % 2])
        ctx = step.seq_len
        want = kv.plan(c, new, t, f, n, 64, page)
        t, f, n, c = want["block_table"], want["free_list"], want["free_count"], want["seq_len"]
        for name in ("granted", "seq_len", "q_start", "slots", "positions"):
            assert np.array_equal(getattr(step, name).cpu().numpy(), want[name]), name
        assert np.array_equal(table.cpu().numpy(), t) and int(count) == n
    with pytest.raises(bsp.BspError) as e:  # in place
        cache.plan(ctx, dev(new.astype(np.int32)), table, free, count, tokens=64, out=step)
    assert e.value.status == 1
    cache.close()
