"""Attention refuses an output whose rows or heads share memory, before any
device call."""
import ctypes as C

import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from bitmap_encoded_unstructured_gb300.build import build_library

SHAPE, P = 2, 0x1000  # an aligned address, never dereferenced: the calls below are refused


class Handle(C.Structure):  # what the checks see of a handle: 2 KV heads of 64
    _fields_ = [("magic", C.c_uint32), ("device", C.c_int), ("num_sms", C.c_int), ("pad", C.c_int),
                ("at", C.c_void_p * 4), ("pages", C.c_int32), ("heads", C.c_int32), ("page_shift", C.c_int32),
                ("dim", C.c_int32), ("rest", C.c_char * 4096)]


@pytest.fixture(scope="module")
def lib():
    build_library()
    return bsp.lib()


@pytest.mark.parametrize("rows,heads,row,head", [
    (2, 4, 0, 64), (9, 2, 0, 64), (9, 4, 64, 64), (9, 4, 192, 64), (9, 4, 248, 64), (9, 4, 64, 568), (9, 4, 64, 512),
    (2, 4, 64, 64), (1 << 30, 2, 64, 1 << 35)])
def test_outputs_that_overlap(lib, rows, heads, row, head):
    h = Handle(magic=0xB5B1CAC8, pages=4, heads=2, page_shift=4, dim=64)
    step = bsp.bsp_kv_step_t(1, 1, 1, P, P, P, 0)
    assert lib.bsp_kv_attention(C.addressof(h), C.addressof(step), P, 0, rows, heads, heads * 64, 64, 1.0, 0, P, row,
                                head, None, None) == SHAPE
