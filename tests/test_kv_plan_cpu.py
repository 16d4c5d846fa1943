"""The plan refuses arrays that share memory, before any device call: other
blocks still read the lengths and the stack while one writes its outputs."""
import ctypes

import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from bitmap_encoded_unstructured_gb300.build import build_library

INVALID = 1
BATCH, WIDTH, STRIDE, CAPACITY, TOKENS = 6, 5, 9, 40, 16
# addresses far apart, never dereferenced: the calls below are refused
NAMES = ("ctx_len", "new_len", "block_table", "free_list", "free_count", "seq_len", "q_start", "granted", "slots",
         "positions", "free_count_out")
AT = {n: 0x100000 * (i + 1) for i, n in enumerate(NAMES)}
BYTES = dict(ctx_len=4 * BATCH, new_len=4 * BATCH, free_list=4 * CAPACITY, free_count=4, seq_len=4 * BATCH,
             q_start=4 * BATCH + 4, granted=4 * BATCH, slots=8 * TOKENS, positions=4 * TOKENS, free_count_out=4)
WRITTEN = ("seq_len", "q_start", "granted", "slots", "positions", "free_list", "free_count_out")


@pytest.fixture(scope="module")
def lib():
    build_library()
    return bsp.lib()


def plan(lib, **at):
    handle = (ctypes.c_uint32 * 1024)(0xB5B1CAC8)  # what the checks see of a handle
    p = dict(AT, **at)
    return lib.bsp_kv_plan(ctypes.addressof(handle), p["ctx_len"], p["new_len"], BATCH, p["block_table"], WIDTH, STRIDE,
                           p["free_list"], CAPACITY, p["free_count"], TOKENS, p["seq_len"], p["q_start"], p["granted"],
                           p["slots"], p["positions"], p["free_count_out"], None)


@pytest.mark.parametrize("one", WRITTEN)
@pytest.mark.parametrize("other", [n for n in NAMES if n != "block_table"])
def test_written_array_that_meets_another(lib, one, other):
    if one == other:
        return
    if {one, other} != {"free_count", "free_count_out"}:  # the count alone may be updated in place
        assert plan(lib, **{one: AT[other]}) == INVALID
    if BYTES[other] > 4:
        assert plan(lib, **{one: AT[other] + BYTES[other] - 4}) == INVALID   # its last word
    if BYTES[one] > 4:
        assert plan(lib, **{one: AT[other] - BYTES[one] + 4}) == INVALID     # its first word


@pytest.mark.parametrize("name", [n for n in NAMES if n != "block_table"])
def test_array_that_meets_a_table_row(lib, name):
    for row in range(BATCH):
        at = AT["block_table"] + 4 * STRIDE * row
        assert plan(lib, **{name: at}) == INVALID
        assert plan(lib, **{name: at + 4 * (WIDTH - 1)}) == INVALID
        assert plan(lib, **{name: at - BYTES[name] + 4}) == INVALID
