"""The binding refuses a step, or a free count, of another device before its
pointers reach the library (stand-ins for what needs two devices)."""
import types

import pytest
import torch

import bitmap_encoded_unstructured_gb300 as bsp


def cache_of(calls):
    """A cache of 2 heads of 16 on the device that CPU tensors report (-1)."""
    c = bsp.KvCache.__new__(bsp.KvCache)
    c.heads, c.dim, c.device, c._index, c._scale, c.h = 2, 16, "here", -1, 0.25, None
    c._append = c._attention = lambda *a: calls.append(a) or 0
    c._current, c._empty, c._float32 = lambda index: 0, torch.empty, torch.float32
    return c


def step_on(index):
    s = bsp.KvStep.__new__(bsp.KvStep)
    s._index, s._ref = index, 0
    return s


@pytest.mark.parametrize("index", [0, 1, None])
def test_step_of_another_device(index):
    calls = []
    c, x = cache_of(calls), torch.zeros((3, 2, 16), dtype=torch.float16)
    with pytest.raises(ValueError):
        c.append(step_on(index), x, x)
    with pytest.raises(ValueError):
        c.attention(step_on(index), x, out=x)
    assert not calls
    c.append(step_on(-1), x, x)
    c.attention(step_on(-1), x, out=x)
    assert len(calls) == 2


def test_free_count_of_another_device():
    def count(index):
        return types.SimpleNamespace(dtype=torch.int32, shape=(1,), get_device=lambda: index, is_contiguous=lambda: True,
                                     data_ptr=lambda: 64)
    with pytest.raises(ValueError):
        bsp.KvStep.empty(2, 5, device="cpu", free_count=count(0))
    assert bsp.KvStep.empty(2, 5, device="cpu", free_count=count(-1)).free_count is not None
