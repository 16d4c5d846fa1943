"""4-bit weights against their plain definitions in 64 bits."""
import numpy as np
import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from oracle import q4

pytestmark = pytest.mark.gpu

DT = ["float16", "bfloat16"]


def dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(getattr(torch, dtype))


def weight(M, K, group, zeros, dtype, seed):
    """(codes, scales fp32 of the type's values, zero points or None)"""
    g = np.random.default_rng(seed)
    groups = -(-K // group)
    z = g.integers(0, 16, (M, groups)).astype(np.uint8) if zeros else None
    c = g.integers(0, 16, (M, K)).astype(np.uint8)
    s = q4.ROUND[dtype]((0.01 * np.exp(g.standard_normal((M, groups)))).astype(np.float32))
    return c, s, z


def matrix(w, group, dtype):
    c, s, z = w
    return bsp.Int4Matrix.from_arrays(dev(q4.pack(c)), dev(s, dtype), None if z is None else dev(z), group=group)


def rows(N, K, dtype, seed):
    x = np.random.default_rng(seed).standard_normal((N, K)).astype(np.float32)
    x[:, ::37] *= 20
    return q4.ROUND[dtype](x)


def close(y, want, before, dtype):
    """y (tensor) within `before` of want, and then one rounding."""
    got = y.double().cpu().numpy()
    lim = before + (np.abs(want) + before) * q4.HALF_STEP[dtype] + q4.TINY[dtype]
    if dtype == "float16":  # past the type's range it is infinite
        over = np.abs(want) + before >= 65504
        assert np.all(np.isinf(got[over & (np.abs(want) - before >= 65520)]))
        got, want, lim = np.where(over, 0, got), np.where(over, 0, want), np.where(over, 1, lim)
    off = np.abs(got - want)
    worst = np.argmax(off / lim)
    assert np.all(off <= lim), (np.unravel_index(worst, off.shape), got.flat[worst], want.flat[worst], lim.flat[worst])


SHAPES = [(1, 8, 128), (16, 64, 64), (17, 72, 32), (128, 128, 128), (130, 1000, 32), (200, 136, 128), (1000, 512, 64),
          (37, 4104, 128), (300, 2048, 32), (2056, 264, 64), (24, 11008, 128)]
TOKENS = [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 100, 129, 200, 257]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_mm(shape, zeros, dtype):
    M, K, group = SHAPES[shape]
    w = weight(M, K, group, zeros, dtype, 10 + shape)
    m = matrix(w, group, dtype)
    for i, N in enumerate(TOKENS):
        x = rows(N, K, dtype, 100 * shape + i)
        y = m.mm(dev(x, dtype))
        close(y, q4.product(x, *w, group), q4.error_bound(x, *w, group, dtype), dtype)
    m.check()
    m.close()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_mm_larger(group, dtype):
    """Enough rows and columns for every split of the work."""
    for M, K, zeros in ((5120, 1280, True), (136, 8192, False), (1024, 4096, True)):
        w = weight(M, K, group, zeros, dtype, group + M)
        m = matrix(w, group, dtype)
        for N in (1, 5, 12, 16, 20, 48, 130, 300, 600):
            x = rows(N, K, dtype, N)
            y = m.mm(dev(x, dtype))
            close(y, q4.product(x, *w, group), q4.error_bound(x, *w, group, dtype), dtype)
        m.check()
        m.close()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("act", sorted(bsp.ACTIVATIONS))
@pytest.mark.parametrize("M,K,group,zg,zu", [(1, 8, 32, False, False), (129, 136, 64, True, False), (500, 1032, 32, False, True),
                                             (2048, 640, 128, True, True)])
def test_gated(M, K, group, zg, zu, act, dtype):
    wg, wu = weight(M, K, group, zg, dtype, M), weight(M, K, group, zu, dtype, M + 1)
    a, b = matrix(wg, group, dtype), matrix(wu, group, dtype)
    for N in (1, 3, 8, 11, 16, 17, 40, 130, 280):
        x = rows(N, K, dtype, N)
        g, u = q4.product(x, *wg, group), q4.product(x, *wu, group)
        eg, eu = q4.error_bound(x, *wg, group, dtype), q4.error_bound(x, *wu, group, dtype)
        y = a.gated(b, dev(x, dtype), activation=act)
        close(y, q4.act(g, act) * u, q4.gated_bound(g, u, eg, eu, act), dtype)
    # the same matrix twice
    x = rows(2, K, dtype, 5)
    g, eg = q4.product(x, *wg, group), q4.error_bound(x, *wg, group, dtype)
    close(a.gated(a, dev(x, dtype), activation=act), q4.act(g, act) * g, q4.gated_bound(g, g, eg, eg, act), dtype)
    a.check()
    a.close()
    b.close()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_encode(zeros, group, dtype):
    """Codes, scales and zero points bit for bit, special values among them; export and decode."""
    import torch
    g = np.random.default_rng(group)
    for M, K in ((1, 8), (50, 72), (130, 1000), (33, 264)):
        W = (g.standard_normal((M, K)) * np.exp(3 * g.standard_normal((M, 1)))).astype(np.float32)
        W = q4.ROUND[dtype](W)
        W[0, :8] = 0
        W.reshape(-1)[3::97] = np.nan
        W.reshape(-1)[5::101] = np.inf
        W.reshape(-1)[6::103] = -np.inf
        W[M // 2] = q4.ROUND[dtype](np.float32(3e-7))  # scales that round to little or nothing
        c, s, z = q4.quantise(W, dtype, group, zeros)
        m = bsp.Int4Matrix(dev(W, dtype), group=group, zeros=zeros)
        codes, scales, zp = m.arrays()
        assert np.array_equal(q4.unpack(codes.cpu().numpy()), c)
        assert np.array_equal(scales.float().cpu().numpy(), s)
        assert (zp is None) == (not zeros) and (zp is None or np.array_equal(zp.cpu().numpy(), z))
        want = torch.from_numpy(q4.dense(c, s, z, group).astype(np.float32)).to(getattr(torch, dtype))
        assert torch.equal(m.decode().cpu(), want)
        assert m.storage_bytes() == (M * K + 1) // 2 + 2 * s.size + ((s.size + 1) // 2 if zeros else 0)
        m.close()


def test_import_from_host_and_round_trip():
    import torch
    w = weight(70, 136, 32, True, "bfloat16", 3)
    c, s, z = torch.from_numpy(q4.pack(w[0])), torch.from_numpy(w[1]).bfloat16(), torch.from_numpy(w[2])
    m = bsp.Int4Matrix.from_arrays(c, s, z, group=32)
    codes, scales, zp = m.arrays()
    assert torch.equal(codes.cpu(), c) and torch.equal(scales.cpu(), s) and torch.equal(zp.cpu(), z)
    bad = z.clone()
    bad[69, 4] = 16
    with pytest.raises(bsp.BspError) as e:
        bsp.Int4Matrix.from_arrays(c, s, bad, group=32)
    assert e.value.status == 1
    m.close()


@pytest.mark.parametrize("N", [1, 6, 14, 40, 300])
@pytest.mark.parametrize("dtype", DT)
def test_strides(N, dtype):
    """Slices of wider tensors; what lies around the output stays."""
    import torch
    M, K, group = 200, 264, 64
    w = weight(M, K, group, True, dtype, 8)
    m = matrix(w, group, dtype)
    x = rows(N, K, dtype, 9)
    t = getattr(torch, dtype)
    wide = torch.full((N + 2, K + 24 + M + 8), 7.0, dtype=t, device="cuda")
    wide[:N, 16:16 + K] = dev(x, dtype)
    at = K + 24                                   # input and output in one tensor's rows
    y = m.mm(wide[:N, 16:16 + K], out=wide[:N, at:at + M])
    close(y, q4.product(x, *w, group), q4.error_bound(x, *w, group, dtype), dtype)
    assert torch.equal(y, m.mm(dev(x, dtype)))
    wide[:N, 16:16 + K] = 7
    wide[:N, at:at + M] = 7
    assert torch.all(wide == 7)
    assert m.mm(wide[:0, 16:16 + K]).shape == (0, M)
    m.check()
    m.close()


@pytest.mark.parametrize("N", [2, 12, 33, 280])
def test_non_finite_rows_stay_their_own(N):
    import torch
    M, K = 136, 512
    w = weight(M, K, 128, False, "float16", 4)
    m = matrix(w, 128, "float16")
    x = rows(N, K, "float16", 5)
    want = m.mm(dev(x, "float16"))
    x[1, 300], x[N - 1, 7] = np.inf, np.nan
    y = m.mm(dev(x, "float16"))
    bad = [1, N - 1]
    good = [i for i in range(N) if i not in bad]
    assert torch.equal(y[good], want[good])
    assert not torch.isfinite(y[N - 1]).any()
    # codes of 8 meet the infinity with a weight of 0
    assert not torch.isfinite(y[1][dev(w[0][:, 300] != 8)]).any()
    m.close()


@pytest.mark.parametrize("dtype", DT)
def test_same_bits_on_any_stream_and_in_graphs(dtype):
    """Two streams at once, captured and replayed on other inputs, two graphs of one matrix."""
    import torch
    M, K = 1024, 2048
    w, u = weight(M, K, 128, True, dtype, 1), weight(M, K, 128, False, dtype, 2)
    m, up = matrix(w, 128, dtype), matrix(u, 128, dtype)
    for N in (1, 10, 24, 150):
        xs = [dev(rows(N, K, dtype, 20 + i), dtype) for i in range(4)]
        want = [(m.mm(x), m.gated(up, x)) for x in xs]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = [None] * 4
        for r in range(3):
            for i, x in enumerate(xs):
                with torch.cuda.stream(streams[i % 2]):
                    got[i] = (m.mm(x), m.gated(up, x))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        graphs, x = [], xs[0].clone()
        for s in streams:
            with torch.cuda.stream(s):
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=s):
                    y = m.mm(x)
                    z = m.gated(up, x)
                    v = up.mm(x)
                graphs.append((g, y, z, v))
        for i in (1, 2):
            x.copy_(xs[i])
            torch.cuda.synchronize()
            for s, (g, *_) in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
                    g.replay()
            torch.cuda.synchronize()
            for _, y, z, v in graphs:
                assert torch.equal(y, want[i][0]) and torch.equal(z, want[i][1]) and torch.equal(v, up.mm(xs[i]))
    m.check()
    m.close()
    up.close()


@pytest.mark.parametrize("group", [32, 64, 128])
def test_repeats_give_the_same_bits(group):
    """Rings that hand a slot on too early show here: one block in some thousands."""
    import torch
    M, K = 2048, 2560
    m = matrix(weight(M, K, group, True, "float16", 1), group, "float16")
    for N in (1, 16, 30, 50, 100, 300, 600):
        x = dev(rows(N, K, "float16", N), "float16")
        want = m.mm(x)
        bad = torch.zeros((), dtype=torch.int64, device="cuda")
        for _ in range(150):
            bad += (m.mm(x) != want).any()
        assert int(bad) == 0, N
    m.check()
    m.close()


FRESH = """
import sys, threading
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import bitmap_encoded_unstructured_gb300 as bsp
from test_gpu_q4 import dev, matrix, rows, weight
m, u = (matrix(weight(300, 520, 64, z, "bfloat16", 3), 64, "bfloat16") for z in (True, False))
xs = [dev(rows(n, 520, "bfloat16", n), "bfloat16") for n in (1, 12, 30, 70, 200)]
torch.cuda.synchronize()
{body}
for x, (y, z) in zip(xs, got):
    assert torch.equal(m.mm(x), y) and torch.equal(m.gated(u, x), z)
m.check()
print("fine")
"""
CAPTURED = """
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = [(m.mm(x), m.gated(u, x)) for x in xs]
g.replay()
torch.cuda.synchronize()
"""
THREADS = """
res = [None] * 4
def work(i):
    with torch.cuda.stream(torch.cuda.Stream()):
        res[i] = [(m.mm(x), m.gated(u, x)) for x in xs]
        torch.cuda.current_stream().synchronize()
ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
[t.start() for t in ts]
[t.join() for t in ts]
got = res[0]
assert all(torch.equal(a, c) and torch.equal(b, d) for r in res for (a, b), (c, d) in zip(r, got))
"""


@pytest.mark.parametrize("body", [CAPTURED, THREADS], ids=["captured", "threads"])
def test_first_calls_of_a_process(body):
    """The first calls: captured in a graph, or from four threads at once."""
    import os
    import subprocess
    import sys
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FRESH.format(root=os.path.dirname(tests), tests=tests, body=body)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("fine"), r.stderr[-2000:]


def test_device_by_name():
    import torch
    w = weight(16, 64, 32, False, "float16", 1)
    m = bsp.Int4Matrix.from_arrays(dev(q4.pack(w[0])), dev(w[1], "float16"), group=32, device="cuda")
    assert m.device == torch.device("cuda", torch.cuda.current_device())
    x = rows(3, 64, "float16", 2)
    close(m.mm(dev(x, "float16")), q4.product(x, *w, 32), q4.error_bound(x, *w, 32), "float16")
    m.close()


def test_binding_errors():
    import torch
    m = matrix(weight(16, 64, 32, False, "float16", 1), 32, "float16")
    other = matrix(weight(24, 64, 32, False, "float16", 1), 32, "float16")
    x = torch.zeros((3, 64), dtype=torch.float16, device="cuda")
    with pytest.raises(bsp.BspError) as e:
        m.gated(other, x)
    assert e.value.status == 2
    with pytest.raises(bsp.BspError) as e:  # an odd slice: its rows are not 16-byte aligned
        m.mm(torch.zeros((3, 72), dtype=torch.float16, device="cuda")[:, 4:68])
    assert e.value.status == 4
    with pytest.raises(ValueError):
        m.mm(x.cpu())
    with pytest.raises(TypeError):
        bsp.Int4Matrix(torch.zeros((4, 64), device="cuda"))
    m.close()
    with pytest.raises(bsp.BspError):
        m.mm(x)
    other.close()
