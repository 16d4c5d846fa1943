"""4-bit products on every tile of the wide kernel, and at the size of whole layers, against the definition in 64 bits
(computed on the GPU: elementary double-precision operations)."""
import pytest

import bitmap_encoded_unstructured_gb300 as bsp
from oracle import q4

pytestmark = pytest.mark.gpu


def weight(M, K, group, zeros, dtype, seed):
    """(matrix, |scale| [M][groups], W [M][K]), the last two in 64 bits."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    groups = -(-K // group)
    codes = torch.randint(0, 256, (M, K // 2), device="cuda", generator=g, dtype=torch.uint8)
    scales = torch.randn((M, groups), device="cuda", generator=g).exp_().mul_(0.01).to(dtype)
    zp = torch.randint(0, 16, (M, groups), device="cuda", generator=g, dtype=torch.uint8) if zeros else None
    W = torch.stack((codes & 15, codes >> 4), -1).reshape(M, K).double()
    W -= 8 if zp is None else zp.double().repeat_interleave(group, 1)[:, :K]
    W *= scales.double().repeat_interleave(group, 1)[:, :K]
    return bsp.Int4Matrix.from_arrays(codes, scales, zp, group=group), scales.double(), W


def rows(N, K, dtype, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((N, K), device="cuda", generator=g)
    x[:, ::37] *= 20
    return x.to(dtype)


def defined(x, w, group):
    """The product and the bound of its error before the last rounding (oracle.q4.error_bound's terms)."""
    import torch
    _, scales, W = w
    x, groups = x.double(), scales.shape[1]
    sums = torch.nn.functional.pad(x.abs(), (0, groups * group - x.shape[1])).view(x.shape[0], groups, group).sum(2)
    inner = 15 * (sums @ scales.t()) * ((group / 16 + 2) * 2.0 ** -22)
    return x @ W.t(), inner + (x.abs() @ W.abs().t()) * (groups + 64) * 2.0 ** -24


def act(g, name):
    import torch
    if name == "silu":
        return g / (1 + torch.exp(-g))
    if name == "gelu":
        return 0.5 * g * torch.special.erfc(-g * 0.5 ** 0.5)
    return g.clamp(min=0)


def near(y, want, before, what):
    import torch
    dtype = {torch.float16: "float16", torch.bfloat16: "bfloat16"}[y.dtype]
    lim = before + (want.abs() + before) * q4.HALF_STEP[dtype] + q4.TINY[dtype]
    if y.dtype is torch.float16:  # past the type's range it is infinite
        big = want.abs() + before >= 65504
        assert bool(y[big & (want.abs() - before >= 65520)].isinf().all()), what
        y, want = y.masked_fill(big, 0), want.masked_fill(big, 0)
    off = (y.double() - want).abs() / lim
    assert bool((off <= 1).all()), (what, float(off.nan_to_num(nan=9e9).max()), int((~(off <= 1)).sum()))


def check(M, K, N, group, gated, dtype, activation="silu", seed=1):
    import torch
    dtype = getattr(torch, dtype)
    w, u = weight(M, K, group, True, dtype, seed), weight(M, K, group, False, dtype, seed + 1) if gated else None
    for n in (N,) if isinstance(N, int) else N:
        x = rows(n, K, dtype, seed + 2)
        want, before = defined(x, w, group)
        if not gated:
            near(w[0].mm(x), want, before, (n, "mm"))
            continue
        v, ev = defined(x, u, group)
        a = act(want, activation)  # the terms of oracle.q4.gated_bound
        da = 1.13 * before + 2.0 ** -18 * a.abs() + 2.0 ** -17 * want.abs() * torch.exp(-want.abs()) + 1e-37
        near(w[0].gated(u[0], x, activation=activation), a * v, da * (v.abs() + ev) + a.abs() * ev, (n, "gated"))
    for m in (w, u):
        if m:
            m[0].check()
            m[0].close()


# Sizes by the tile that the cost rule gives them on 152 SMs: (columns of Y a
# tile takes, pairs of CTAs that share its columns of W).
PRODUCTS = {
    32: [(64, 1, 300, 264, 900), (64, 2, 300, 520, 900), (64, 3, 100, 264, 40), (64, 4, 100, 2056, 40),
         (128, 1, 2600, 264, 400), (128, 2, 2600, 4104, 280), (128, 3, 300, 2056, 1300), (128, 4, 300, 4104, 900),
         (256, 1, 2600, 264, 900), (256, 2, 3300, 4104, 400), (256, 3, 2600, 1032, 400), (256, 4, 3300, 4104, 150)],
    64: [(64, 1, 100, 264, 40), (64, 2, 300, 1032, 900), (64, 3, 100, 520, 40), (64, 4, 100, 2056, 40),
         (128, 1, 2600, 264, 400), (128, 2, 3300, 2056, 150), (128, 3, 300, 2056, 1300), (128, 4, 300, 4104, 900),
         (256, 1, 2600, 264, 900), (256, 2, 3300, 8200, 400), (256, 3, 2600, 2056, 400), (256, 4, 3300, 8200, 150)],
    128: [(64, 1, 100, 264, 40), (64, 2, 300, 1032, 900), (64, 3, 100, 520, 40), (64, 4, 100, 2056, 40),
          (128, 1, 2600, 264, 400), (128, 2, 3300, 2056, 150), (128, 3, 300, 2056, 1300), (128, 4, 300, 4104, 900),
          (256, 1, 2600, 264, 900), (256, 2, 3300, 4104, 400), (256, 3, 2600, 2056, 400), (256, 4, 3300, 4104, 150)]}
GATED = {
    32: [(64, 1, 200, 264, 900), (64, 2, 200, 520, 900), (64, 3, 100, 264, 40), (64, 4, 100, 2056, 40),
         (128, 1, 3300, 264, 150), (128, 2, 3300, 4104, 100), (128, 3, 200, 2056, 1300), (128, 4, 200, 4104, 900),
         (256, 1, 3300, 264, 280), (256, 2, 3300, 4104, 150), (256, 3, 2600, 1032, 200), (256, 4, 2000, 4104, 150)],
    64: [(64, 1, 100, 264, 40), (64, 2, 200, 1032, 900), (64, 3, 100, 520, 40), (64, 4, 100, 2056, 40),
         (128, 1, 3300, 264, 150), (128, 2, 2000, 2056, 150), (128, 3, 200, 2056, 1300), (128, 4, 200, 4104, 900),
         (256, 1, 3300, 264, 280), (256, 2, 3300, 8200, 150), (256, 3, 2600, 2056, 200), (256, 4, 2000, 8200, 150)],
    128: [(64, 1, 100, 264, 40), (64, 2, 200, 1032, 900), (64, 3, 100, 520, 40), (64, 4, 100, 2056, 40),
          (128, 1, 3300, 264, 150), (128, 2, 2000, 2056, 150), (128, 3, 200, 2056, 1300), (128, 4, 200, 4104, 900),
          (256, 1, 3300, 264, 280), (256, 2, 3300, 4104, 150), (256, 3, 2600, 2056, 200), (256, 4, 2000, 4104, 150)]}
DT = ["float16", "bfloat16"]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("case", range(12))
@pytest.mark.parametrize("group", [32, 64, 128])
def test_products(group, case, dtype):
    _, _, M, K, N = PRODUCTS[group][case]
    check(M, K, N, group, False, dtype, seed=10 * case)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("case", range(12))
@pytest.mark.parametrize("group", [32, 64, 128])
def test_gated(group, case, dtype):
    _, _, M, K, N = GATED[group][case]
    check(M, K, N, group, True, dtype, ("silu", "gelu", "relu")[case % 3], seed=10 * case)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("M,K,group,N", [(28672, 8192, 128, (1, 16, 24, 70, 700)), (8192, 28672, 64, (2, 9, 30, 400)),
                                         (11008, 4096, 32, (1, 12, 33, 203, 2048))])
def test_layers(M, K, group, N, dtype):
    check(M, K, N, group, False, dtype)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("M,K,group,N", [(28672, 8192, 128, (1, 12, 40, 520)), (11008, 4096, 64, (3, 20, 203, 1500))])
def test_gated_layers(M, K, group, N, dtype):
    check(M, K, N, group, True, dtype)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_repeats_give_the_same_bits(group):
    """Products of large tiles, shared and not, again and again behind other work."""
    import torch
    for gated, cases in ((False, PRODUCTS[group]), (True, GATED[group])):
        for bn, shares, M, K, N in cases[4:]:
            w, u = weight(M, K, group, True, torch.bfloat16, 1)[0], weight(M, K, group, False, torch.bfloat16, 2)[0]
            x = rows(N, K, torch.bfloat16, 3)
            call = (lambda: w.gated(u, x)) if gated else (lambda: w.mm(x))
            want, bad = call(), torch.zeros((), dtype=torch.int64, device="cuda")
            for rep in range(100):
                if rep % 5 == 0:
                    torch.randn(1 << (10 + rep % 11), device="cuda").sort()
                bad += (call() != want).any()
            assert int(bad) == 0, (bn, shares)
            for m in (w, u):
                m.check()
                m.close()
