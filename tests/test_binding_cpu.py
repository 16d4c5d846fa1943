"""What the binding hands to the library, without a device: the library's entry is replaced by one that looks at it."""
import contextlib
import ctypes as C
import types

import numpy as np
import pytest
import torch

import bitmap_encoded_unstructured_gb300 as bsp


def test_bitmap_from_strided_numpy_arrays(monkeypatch):
    """The copies that the pointers point to live until the call returns."""
    g = np.random.default_rng(1)
    arrays = [g.integers(0, 1 << 30, (n, 2)).astype(t)[:, 0] for n, t in ((900, np.uint64), (900, np.uint64), (3600, np.uint16))]

    def look(bitmaps, offsets, values, *rest):
        for a, p in zip(arrays, (bitmaps, offsets, values)):
            assert C.string_at(p, a.nbytes) == a.tobytes()
        return 0

    monkeypatch.setattr(bsp, "bsp_import", look)
    bsp.BitmapMatrix.from_arrays(*arrays, 64, 64, device="cuda:0", stream=0)


def test_int4_from_arrays_refuses_another_kind_of_device():
    """(It went to the current GPU.)"""
    with pytest.raises(ValueError, match="GPU"):
        bsp.Int4Matrix.from_arrays(torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.float16), group=32,
                                   device="cpu")


def test_rotary_sections(monkeypatch):
    """Any iterable; the number of axes is that of sections; no negative ones."""
    seen = []

    def create(d, stream, out):
        seen.append(bsp.bsp_rope_desc_t.from_address(d).axes)
        return 0

    monkeypatch.setattr(bsp, "lib", lambda: types.SimpleNamespace(bsp_rope_create=create, bsp_rope_apply=None, bsp_rope_destroy=lambda h: 0))
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for sections in ([2, 1, 1], (2, 1, 1), iter([2, 1, 1]), np.array([2, 1, 1])):
        r = bsp.Rotary(8, sections=sections, device="cuda:0", stream=0)
        assert r.axes == 3 and r.axis == [0, 0, 1, 2]
    assert bsp.Rotary(8, sections=[4, 0], device="cuda:0", stream=0).axes == 2
    assert seen == [3, 3, 3, 3, 2]
    with pytest.raises(ValueError):
        bsp.Rotary(8, sections=[5, -1], device="cuda:0", stream=0)
