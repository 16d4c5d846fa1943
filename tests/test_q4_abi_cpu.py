"""Refusals of the 4-bit weights' and the rotary entry points, before any device call."""
import ctypes as C
import types

import pytest
import torch

import bitmap_encoded_unstructured_gb300 as bsp
from bitmap_encoded_unstructured_gb300.build import build_library

OK, INVALID, SHAPE, DTYPE, ALIGN = 0, 1, 2, 3, 4
P = 0x100000  # an aligned address; never dereferenced
FAR = P + (1 << 40)


@pytest.fixture(scope="module")
def lib():
    build_library()
    return bsp.lib()


class Q4(C.Structure):  # what the checks see of a handle
    _fields_ = [("magic", C.c_uint32), ("device", C.c_int), ("num_sms", C.c_int), ("dtype", C.c_int), ("M", C.c_int64),
                ("K", C.c_int64), ("group", C.c_int32), ("pad", C.c_int32), ("strips", C.c_int64),
                ("k_tiles", C.c_int64), ("at", C.c_void_p * 4)]


def q4(**kw):
    d = dict(magic=0xB5B14B17, device=0, num_sms=152, dtype=0, M=40, K=64, group=32, strips=1, k_tiles=2)
    d.update(kw)
    return Q4(**d)


class Rope(C.Structure):
    _fields_ = [("magic", C.c_uint32), ("device", C.c_int), ("num_sms", C.c_int), ("dim", C.c_int32),
                ("rot", C.c_int32), ("axes", C.c_int32), ("interleaved", C.c_int32), ("scale", C.c_float),
                ("at", C.c_void_p * 2)]


@pytest.mark.parametrize("change,status", [
    (dict(W=None), INVALID), (dict(zeros=2), INVALID), (dict(dtype=1), DTYPE), (dict(dtype=7), DTYPE), (dict(M=0), SHAPE),
    (dict(K=0), SHAPE), (dict(K=60), SHAPE), (dict(group=16), SHAPE), (dict(group=256), SHAPE), (dict(group=0), SHAPE),
    (dict(M=1 << 31), SHAPE), (dict(M=1 << 30, K=1 << 20), SHAPE), (dict(W=P + 8), ALIGN)])
def test_encode_refuses(lib, change, status):
    d = dict(W=P, dtype=0, M=40, K=64, group=32, zeros=0)
    d.update(change)
    h = C.c_void_p(7)
    assert lib.bsp_q4_encode(d["W"], d["dtype"], d["M"], d["K"], d["group"], d["zeros"], None, C.byref(h)) == status
    assert not h.value
    if "W" not in change and "zeros" not in change:
        h = C.c_void_p(7)
        assert lib.bsp_q4_import(P, P, None, d["dtype"], d["M"], d["K"], d["group"], None, C.byref(h)) == status
        assert not h.value


def test_null_handles(lib):
    h, u = C.c_void_p(), C.c_uint64()
    assert lib.bsp_q4_encode(P, 0, 40, 64, 32, 0, None, None) == INVALID
    assert lib.bsp_q4_import(None, P, None, 0, 40, 64, 32, None, C.byref(h)) == INVALID
    assert lib.bsp_q4_import(P, None, None, 0, 40, 64, 32, None, C.byref(h)) == INVALID
    assert lib.bsp_q4_import(P, P, None, 0, 40, 64, 32, None, None) == INVALID
    good = C.addressof(q4())
    for bad in (None, C.addressof(q4(magic=1))):
        assert lib.bsp_q4_export(bad, P, P, P, None) == INVALID
        assert lib.bsp_q4_decode(bad, P, None) == INVALID
        assert lib.bsp_q4_info(bad, P) == INVALID
        assert lib.bsp_q4_storage_bytes(bad, C.byref(u)) == INVALID
        assert lib.bsp_q4_check(bad, None) == INVALID
        assert lib.bsp_q4_destroy(bad) == INVALID
        assert lib.bsp_q4_mm(bad, P, 64, 1, FAR, 40, None) == INVALID
        assert lib.bsp_q4_gated(bad, bad, P, 64, 1, 0, FAR, 40, None) == INVALID
        assert lib.bsp_rope_destroy(bad) == INVALID
        assert lib.bsp_rope_apply(bad, None, None, 0, 1, P, 1, 0, None) == INVALID
    g = q4()
    good = C.addressof(g)
    assert lib.bsp_q4_gated(good, None, P, 64, 1, 0, FAR, 40, None) == INVALID
    assert lib.bsp_q4_info(good, None) == INVALID and lib.bsp_q4_storage_bytes(good, None) == INVALID
    assert lib.bsp_q4_decode(good, None, None) == INVALID and lib.bsp_q4_decode(good, P + 2, None) == ALIGN
    assert lib.bsp_q4_export(good, P + 2, P, P, None) == ALIGN and lib.bsp_q4_export(good, P, P + 1, P, None) == ALIGN


def test_info_and_bytes(lib):
    g, i, u = q4(M=41, K=72), bsp.bsp_q4_info_t(), C.c_uint64()
    assert lib.bsp_q4_info(C.addressof(g), C.addressof(i)) == OK
    assert (i.M, i.K, i.group, i.groups, i.zeros) == (41, 72, 32, 3, 0)
    assert lib.bsp_q4_storage_bytes(C.addressof(g), C.byref(u)) == OK and u.value == 41 * 36 + 2 * 41 * 3
    g.at[2] = P
    assert lib.bsp_q4_storage_bytes(C.addressof(g), C.byref(u)) == OK and u.value == 41 * 36 + 2 * 41 * 3 + 62


ROWS = [
    (dict(N=-1), INVALID), (dict(N=1 << 31), INVALID), (dict(X=None), INVALID), (dict(Y=None), INVALID),
    (dict(xs=56), SHAPE), (dict(xs=68), SHAPE), (dict(xs=-64), SHAPE), (dict(ys=39), SHAPE), (dict(xs=1 << 62), SHAPE),
    (dict(ys=1 << 62), SHAPE), (dict(X=P + 8), ALIGN), (dict(Y=FAR + 2), ALIGN),
    (dict(Y=P), INVALID),                           # Y is X
    (dict(Y=P + 2 * 64 * 4), INVALID),              # Y begins inside X
    (dict(Y=P + 2 * 64, xs=96, ys=96), INVALID),    # a slice beside X that runs into its next row
    (dict(N=1, Y=P + 16), INVALID),
    (dict(N=0, X=None, Y=None), OK), (dict(N=0), OK)]


@pytest.mark.parametrize("change,status", ROWS)
def test_products_refuse(lib, change, status):
    d = dict(X=P, xs=64, N=5, Y=FAR, ys=40)
    d.update(change)
    a, b = q4(), q4()
    assert lib.bsp_q4_mm(C.addressof(a), d["X"], d["xs"], d["N"], d["Y"], d["ys"], None) == status
    assert lib.bsp_q4_gated(C.addressof(a), C.addressof(b), d["X"], d["xs"], d["N"], 0, d["Y"], d["ys"], None) == status


@pytest.mark.parametrize("change,act,status", [
    (dict(M=41), 0, SHAPE), (dict(K=72), 0, SHAPE), (dict(group=64), 0, SHAPE), (dict(dtype=2), 0, DTYPE),
    (dict(device=1), 0, INVALID), (dict(), -1, INVALID), (dict(), 4, INVALID)])
def test_gated_refuses_pairs(lib, change, act, status):
    a, b = q4(), q4(**change)
    assert lib.bsp_q4_gated(C.addressof(a), C.addressof(b), P, 64, 2, act, FAR, 40, None) == status


def desc(**kw):
    d = dict(dim=16, rot=8, axes=2, interleaved=0, freq=[1.0, 0.5, 0.25, 0.1], axis=[0, 1, 0, 1], scale=1.0)
    d.update(kw)
    f = None if d["freq"] is None else (C.c_double * 512)(*d["freq"])
    a = None if d["axis"] is None else (C.c_uint8 * 512)(*d["axis"])
    s = bsp.bsp_rope_desc_t(d["dim"], d["rot"], d["axes"], d["interleaved"], f and C.addressof(f), a and C.addressof(a),
                            d["scale"])
    return s, f, a


@pytest.mark.parametrize("change,status", [
    (dict(freq=None), INVALID), (dict(dim=12), SHAPE), (dict(dim=0), SHAPE), (dict(dim=1032), SHAPE), (dict(rot=0), SHAPE),
    (dict(rot=12), SHAPE), (dict(rot=24), SHAPE), (dict(axes=0), SHAPE), (dict(axes=9), SHAPE), (dict(interleaved=2), INVALID),
    (dict(axis=[0, 2, 0, 0]), INVALID), (dict(freq=[1.0, float("nan"), 0, 0]), INVALID),
    (dict(freq=[1.0, float("-inf"), 0, 0]), INVALID), (dict(freq=[65537.0, 0, 0, 0]), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID)])
def test_rope_create_refuses(lib, change, status):
    d, f, a = desc(**change)
    h = C.c_void_p(7)
    assert lib.bsp_rope_create(C.addressof(d), None, C.byref(h)) == status
    assert not h.value
    assert lib.bsp_rope_create(None, None, C.byref(h)) == INVALID and lib.bsp_rope_create(C.addressof(d), None, None) == INVALID


def rows(**kw):
    d = dict(in_=P, out=FAR, heads=3, in_row=48, in_head=16, out_row=48, out_head=16)
    d.update(kw)
    return bsp.bsp_rope_rows_t(*[d[n] for n, _ in bsp.bsp_rope_rows_t._fields_])


POS = FAR + (1 << 40)


@pytest.mark.parametrize("q,k,call,status", [
    (dict(heads=-1), {}, {}, SHAPE), (dict(in_=None), {}, {}, INVALID), (dict(out=None), {}, {}, INVALID),
    (dict(in_row=44), {}, {}, SHAPE), (dict(in_head=12), {}, {}, SHAPE), (dict(in_row=-48), {}, {}, SHAPE),
    (dict(out_row=8), {}, {}, SHAPE), (dict(out_head=8), {}, {}, SHAPE), (dict(out_row=32), {}, {}, SHAPE),
    (dict(out_head=0), {}, {}, SHAPE), (dict(in_=P + 8), {}, {}, ALIGN), (dict(out=FAR + 4), {}, {}, ALIGN),
    (dict(in_row=1 << 61), {}, {}, SHAPE), (dict(out_head=1 << 61), {}, {}, SHAPE),
    ({}, {}, dict(dtype=1), DTYPE), ({}, {}, dict(rows=-1), INVALID), ({}, {}, dict(rows=1 << 31), INVALID),
    ({}, {}, dict(pos=None), INVALID), ({}, {}, dict(pos=POS + 2), ALIGN), ({}, {}, dict(stride=4), SHAPE),
    ({}, {}, dict(inverse=2), INVALID),
    (dict(out=P + 32), {}, {}, INVALID),                                  # shifted over its own input
    (dict(out=P, out_row=64), {}, {}, INVALID),                           # its input's address, another stride
    (dict(out=POS), {}, {}, INVALID),                                     # over the positions
    (dict(), dict(in_=FAR), {}, INVALID),                                 # q's output over k's input
    (dict(), dict(in_=P + (1 << 30)), {}, INVALID),                       # both outputs in one place
    (dict(out=P, in_row=96, out_row=96), dict(in_=P + 64, out=P + 64, in_row=96, out_row=96), {}, INVALID),  # slices that meet
    (dict(heads=0), dict(heads=0), {}, OK), ({}, {}, dict(rows=0, pos=None), OK)])
def test_rope_apply_refuses(lib, q, k, call, status):
    h = Rope(magic=0xB5B10709, dim=16, rot=8, axes=2, scale=1.0)
    c = dict(dtype=0, rows=5, pos=POS, stride=5, inverse=0)
    c.update(call)
    a, b = rows(**q), rows(**k) if k else None
    st = lib.bsp_rope_apply(C.addressof(h), C.addressof(a), C.addressof(b) if b else None, c["dtype"], c["rows"], c["pos"],
                            c["stride"], c["inverse"], None)
    assert st == status


def stand_in(**kw):
    """A matrix of 16 x 64 on the device that CPU tensors report (-1)."""
    m = bsp.Int4Matrix.__new__(bsp.Int4Matrix)
    m.h, m.device, m._index, m.torch_dtype, m.M, m.K = None, "here", -1, torch.float16, 16, 64
    m.calls = []
    m._mm = m._gated = lambda *a: m.calls.append(a) or 0
    m._current, m._empty = lambda index: 0, lambda shape, dtype, device: torch.empty(shape, dtype=dtype)
    return m


def test_binding_refuses():
    m, x = stand_in(), torch.zeros((3, 64), dtype=torch.float16)
    bad = [x.bfloat16(), x[:, :56], x[0], torch.zeros((3, 128), dtype=torch.float16)[:, ::2]]
    for b in bad:
        with pytest.raises(ValueError):
            m.mm(b)
    for o in (torch.zeros((3, 15), dtype=torch.float16), torch.zeros((3, 16)), torch.zeros((3, 32), dtype=torch.float16)[:, ::2]):
        with pytest.raises(ValueError):
            m.mm(x, out=o)
    with pytest.raises(ValueError):
        m.gated(types.SimpleNamespace(h=0), x, activation="tanh")
    far = types.SimpleNamespace(shape=(3, 64), dtype=torch.float16, get_device=lambda: 1, stride=lambda: (64, 1))
    with pytest.raises(ValueError):
        m.mm(far)
    assert not m.calls
    m.mm(x)
    m.gated(types.SimpleNamespace(h=0), x, activation="relu", out=torch.zeros((3, 16), dtype=torch.float16))
    assert len(m.calls) == 2


def test_from_arrays_refuses():
    u8, h = torch.uint8, torch.float16
    with pytest.raises(TypeError):
        bsp.Int4Matrix.from_arrays(torch.zeros((4, 32)), torch.zeros((4, 2), dtype=h), group=32)
    with pytest.raises(TypeError):
        bsp.Int4Matrix.from_arrays(torch.zeros((4, 32), dtype=u8), torch.zeros((4, 2)), group=32)
    with pytest.raises(ValueError):
        bsp.Int4Matrix.from_arrays(torch.zeros((4, 32), dtype=u8), torch.zeros((4, 3), dtype=h), group=32)
    with pytest.raises(ValueError):
        bsp.Int4Matrix.from_arrays(torch.zeros((4, 32), dtype=u8), torch.zeros((4, 2), dtype=h),
                                   torch.zeros((4, 2), dtype=torch.int8), group=32)


def test_rotary_axes():
    assert bsp.Rotary._axes_of([2, 1, 1], False) == [0, 0, 1, 2]
    assert bsp.Rotary._axes_of([3, 1, 2], True) == [0, 1, 2, 0, 2, 0]
    for kw in (dict(sections=[2, 1]), dict(axis=[0, 0, 0, 8]), dict(axis=[0] * 4, sections=[4]), dict(freqs=[1.0] * 3)):
        with pytest.raises(ValueError):
            bsp.Rotary(8, **kw)
