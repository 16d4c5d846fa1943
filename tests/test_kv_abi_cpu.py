"""Refusals of the KV cache's entry points that need no device."""
import ctypes

import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from bitmap_encoded_unstructured_gb300.build import build_library

OK, INVALID, SHAPE, DTYPE, ALIGN = 0, 1, 2, 3, 4
P = 0x1000  # an aligned address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    build_library()
    return bsp.lib()


def desc(**kw):
    d = dict(k=P, v=P, k_scale=P, v_scale=P, pages=4, heads=2, page=16, dim=64, page_stride=2048, head_stride=1024,
             row_stride=64, scale_stride=2)
    d.update(kw)
    return bsp.bsp_kv_desc_t(*[d[n] for n, _ in bsp.bsp_kv_desc_t._fields_])


@pytest.mark.parametrize("change,status", [
    (dict(k=None), INVALID), (dict(v_scale=None), INVALID), (dict(page=24), SHAPE), (dict(page=8), SHAPE),
    (dict(page=512), SHAPE), (dict(dim=8), SHAPE), (dict(dim=72), SHAPE), (dict(dim=272), SHAPE), (dict(pages=0), SHAPE),
    (dict(pages=1 << 31), SHAPE), (dict(heads=0), SHAPE), (dict(heads=32768), SHAPE), (dict(row_stride=48), SHAPE),
    (dict(row_stride=72), SHAPE), (dict(head_stride=8), SHAPE), (dict(page_stride=2056), SHAPE),
    (dict(page_stride=-2048), SHAPE), (dict(scale_stride=1), SHAPE), (dict(k=P + 8), ALIGN), (dict(v=P + 1), ALIGN),
    (dict(k_scale=P + 2), ALIGN)])
def test_create_refuses(lib, change, status):
    h = ctypes.c_void_p(7)
    d = desc(**change)
    assert lib.bsp_kv_create(ctypes.addressof(d), None, ctypes.byref(h)) == status
    assert not h.value


def test_null_handles(lib):
    h = ctypes.c_void_p()
    assert lib.bsp_kv_create(None, None, ctypes.byref(h)) == INVALID
    assert lib.bsp_kv_create(ctypes.addressof(desc()), None, None) == INVALID
    step = bsp.bsp_kv_step_t(1, 1, 1, P, P, P, 0)
    ref = ctypes.addressof(step)
    assert lib.bsp_kv_destroy(None) == INVALID
    assert lib.bsp_kv_check(None, None) == INVALID
    assert lib.bsp_kv_plan(None, P, P, 1, P, 1, 1, P, 1, P, 1, P, P, P, P, P, P, None) == INVALID
    assert lib.bsp_kv_append(None, ref, P, P, 0, 1, 64, 64, 64, 64, None) == INVALID
    assert lib.bsp_kv_read(None, P, 1, P, P, 0, None) == INVALID
    assert lib.bsp_kv_attention(None, ref, P, 0, 1, 1, 64, 64, 1.0, 0, P, 64, 64, None, None) == INVALID


def test_rows_are_16_bit_types(lib):
    """Only the cache's rows take BSP_BF16: the weights' entry points refuse it."""
    h = ctypes.c_void_p()
    assert lib.bsp_encode(P, bsp.BSP_BF16, 64, 64, None, ctypes.byref(h)) == DTYPE
    assert lib.bsp_import(P, P, P, bsp.BSP_BF16, 64, 64, 1, None, ctypes.byref(h)) == DTYPE
