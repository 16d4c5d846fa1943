"""4-bit weights and rotary positions: their cases, plain forms and definitions.

What a gated decoder layer computes beside its pruned products and its KV
cache:

* ``mm``      activations times a weight held as 4-bit codes with a scale (and
              optionally a zero point) for each group of a row:
              Y[n][m] = sum_k s[m][k / G] (c[m][k] - z[m][k / G]) X[n][k];
* ``gated``   the first half of a gated feed-forward block over two such
              weights, act(W_gate X) * (W_up X), rounded once;
* ``rotary``  query and key rows rotated by their positions on one or several
              axes (time, height, width), before keys are cached.

``run`` computes them with elementary torch operations in 32 bits (the angles
in 64) where ``own`` is false, and by the framework's entry points where it is
true.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # latency: one token through an OPT-13B-shaped output projection
        dict(name="mm-out-1", op="mm", rows=5120, cols=5120, tokens=1, group=128, zeros=False, wide=0, type="fp16"),
        # one token through a Llama-2-70B-shaped up projection, zero points
        dict(name="mm-up-1", op="mm", rows=28672, cols=8192, tokens=1, group=128, zeros=True, wide=0, type="bf16"),
        # sixteen streams through an OPT-13B-shaped first feed-forward layer
        dict(name="mm-fc1-16", op="mm", rows=20480, cols=5120, tokens=16, group=64, zeros=False, wide=0, type="fp16"),
        # drafts of a few streams, a slice of a wider activation, fine groups, the last one short
        dict(name="mm-drafts-37", op="mm", rows=4096, cols=11000, tokens=37, group=32, zeros=True, wide=64, type="bf16"),
        # a prompt through a Llama-2-70B-shaped down projection
        dict(name="mm-down-1501", op="mm", rows=8192, cols=28672, tokens=1501, group=128, zeros=False, wide=0, type="fp16"),
        # one token through a 4096 x 11008 gated block
        dict(name="gated-1", op="gated", rows=11008, cols=4096, tokens=1, group=128, zeros=False, wide=0, act="silu",
             type="fp16"),
        # a small batch through a Llama-2-70B-shaped gated block
        dict(name="gated-12", op="gated", rows=28672, cols=8192, tokens=12, group=128, zeros=False, wide=0, act="silu",
             type="bf16"),
        # short prompts, another activation, ragged sizes
        dict(name="gated-203", op="gated", rows=11001, cols=4096, tokens=203, group=64, zeros=True, wide=0, act="gelu",
             type="fp16"),
        # a prompt through the Llama-2-70B-shaped gated block
        dict(name="gated-2048", op="gated", rows=28672, cols=8192, tokens=2048, group=128, zeros=False, wide=0,
             act="silu", type="bf16"),
        # one token's heads of an OPT-13B-shaped layer
        dict(name="rotary-1", op="rotary", tokens=1, heads=40, kv_heads=40, dim=128, rot=128, axes=1, cyclic=False,
             pairs="half", far=4096, inverse=False, type="fp16"),
        # a batch of streams far into their contexts, part of each head rotated
        dict(name="rotary-256", op="rotary", tokens=256, heads=32, kv_heads=4, dim=80, rot=32, axes=1, cyclic=False,
             pairs="interleaved", far=1000000, inverse=False, type="fp16"),
        # a prompt with images: three axes taking turns, grouped heads
        dict(name="rotary-8101", op="rotary", tokens=8101, heads=64, kv_heads=8, dim=128, rot=128, axes=3, cyclic=True,
             pairs="half", far=32768, inverse=False, type="bf16"),
    ]


def _log_int(r, lo, hi):
    """A whole number in lo..hi, spread over its logarithm."""
    return min(hi, max(lo, int(math.exp(r.uniform(math.log(lo), math.log(hi + 1.0))))))


def draw(rng):
    r = rng
    op = r.choice(["mm", "mm", "gated", "rotary"])
    kind = r.choice(["fp16", "bf16"])
    if op == "rotary":
        heads, kv_heads = r.choice([(40, 40), (64, 8), (32, 4), (28, 4), (16, 1), (12, 12), (5, 1)])
        dim = r.choice([64, 80, 96, 128, 128, 128, 256])
        rot = r.choice([dim, dim, dim // 16 * 8])
        return dict(op="rotary", tokens=_log_int(r, 1, 74_000_000 // ((heads + kv_heads) * dim)), heads=heads,
                    kv_heads=kv_heads, dim=dim, rot=rot, axes=r.choice([1, 1, 2, 3]), cyclic=r.random() < 0.5,
                    pairs=r.choice(["half", "half", "interleaved"]), far=_log_int(r, 64, 4_000_000),
                    inverse=r.random() < 0.25, type=kind)
    if r.random() < 0.5:  # shapes of the benchmark's layers
        rows, cols = r.choice([(5120, 5120), (15360, 5120), (20480, 5120), (5120, 20480), (8192, 8192), (28672, 8192),
                               (8192, 28672), (11008, 4096), (4096, 11008), (1024, 8192)])
    else:
        rows, cols = _log_int(r, 16, 28672), _log_int(r, 8, 2500) * 8
        while rows * cols > 28672 * 8192:
            rows //= 2
    most = 2048 * 28672 * 8192 // (rows * cols) if op == "gated" else 4096 * 28672 * 8192 // (rows * cols)
    case = dict(op=op, rows=rows, cols=cols, tokens=_log_int(r, 1, min(4096, most)), group=r.choice([32, 64, 128, 128]),
                zeros=r.random() < 0.5, wide=r.choice([0, 0, 8, 200]), type=kind)
    if op == "gated":
        case["act"] = r.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"])
    return case


# ------------------------------------------------------------------ inputs

def _weight(case, gen):
    """Codes [rows][cols / 2] (two a byte, the even column in the low half), scales and zero points [rows][groups]."""
    rows, cols, groups = case["rows"], case["cols"], -(-case["cols"] // case["group"])
    zeros = None
    if case["zeros"]:
        zeros = torch.randint(5, 12, (rows, groups), device="cuda", generator=gen, dtype=torch.uint8)
    # a group's codes are a bell around its zero point
    c = torch.randn((rows, cols), device="cuda", generator=gen, dtype=torch.float16).mul_(2.6)
    if zeros is None:
        c += 8
    else:
        c += zeros.half().repeat_interleave(case["group"], 1)[:, :cols]
    c = c.round_().clamp_(0, 15).to(torch.uint8)
    packed = (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous()
    s = torch.randn((rows, groups), device="cuda", generator=gen).mul_(0.3).exp_().mul_(0.4 / math.sqrt(cols))
    return packed, s.to(DTYPES[case["type"]]), zeros


def _prepare_product(case, gen):
    s = dict(op=case["op"], group=case["group"], cols=case["cols"], act=case.get("act"))
    names = ["gate", "up"] if case["op"] == "gated" else ["weight"]
    for name in names:
        s[name] = _weight(case, gen)
    # activations behind a norm: a bell, a few channels many times as large
    cols = case["cols"]
    x = torch.randn((case["tokens"], cols + case["wide"]), device="cuda", generator=gen)
    loud = torch.rand(cols + case["wide"], device="cuda", generator=gen) < 0.002
    x = torch.where(loud, x * 15, x).to(DTYPES[case["type"]])
    s["x"] = x[:, :cols]
    if own:  # the handles that a server keeps
        import bitmap_encoded_unstructured_gb300 as bsp
        for name in names:
            codes, scales, zeros = s[name]
            s[name + "_matrix"] = bsp.Int4Matrix.from_arrays(codes, scales, zeros, group=case["group"])
    return s


def _frequencies(case):
    """Angle a step of each pair, and the pair's axis: equal runs of pairs, or the axes in turn."""
    half, axes = case["rot"] // 2, case["axes"]
    freq = [10000.0 ** (-i / half) for i in range(half)]
    axis = [i % axes if case["cyclic"] else i * axes // half for i in range(half)]
    return freq, axis


def _prepare_rotary(case, gen):
    rows, dtype = case["tokens"], DTYPES[case["type"]]
    heads = case["heads"] + 2 * case["kv_heads"]
    # the output of a QKV projection, of which queries and keys are views
    qkv = torch.randn((rows, heads, case["dim"]), device="cuda", generator=gen, dtype=torch.float32).to(dtype)
    # rows that follow one another in time; places in an image
    start = torch.randint(0, case["far"], (1,), device="cuda", generator=gen)
    pos = [(start + torch.arange(rows, device="cuda")) % case["far"]]
    for _ in range(1, case["axes"]):
        pos.append(torch.randint(0, min(case["far"], 1024), (rows,), device="cuda", generator=gen))
    freq, axis = _frequencies(case)
    s = dict(op="rotary", q=qkv[:, :case["heads"]], k=qkv[:, case["heads"]:case["heads"] + case["kv_heads"]],
             positions=torch.stack(pos).to(torch.int32), rot=case["rot"], pairs=case["pairs"], inverse=case["inverse"],
             freq=torch.tensor(freq, dtype=torch.float64, device="cuda"), axis=torch.tensor(axis, device="cuda"))
    if own:
        import bitmap_encoded_unstructured_gb300 as bsp
        s["rotary"] = bsp.Rotary(case["dim"], rot=case["rot"], freqs=freq, axis=axis,
                                 interleaved=case["pairs"] == "interleaved")
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    return _prepare_rotary(case, gen) if case["op"] == "rotary" else _prepare_product(case, gen)


# ------------------------------------------------------------- plain forms

def _plain_product(weight, x, group, cols):
    codes, scales, zeros = weight
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], cols).float()
    z = torch.full_like(scales, 8.0, dtype=torch.float32) if zeros is None else zeros.float()
    w = (c - z.repeat_interleave(group, 1)[:, :cols]) * scales.float().repeat_interleave(group, 1)[:, :cols]
    return torch.matmul(x.float(), w.transpose(0, 1))


def _plain_act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "gelu":
        return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))
    return torch.clamp(g, min=0)


def _plain_rotate(x, cos, sin, rot, pairs):
    y = x.float()
    if pairs == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((turned, y[..., rot:]), -1).to(x.dtype)


def _plain_rotary(s):
    angle = s["positions"][s["axis"]].double().transpose(0, 1) * s["freq"]  # [rows][rot / 2]
    if s["inverse"]:
        angle = -angle
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    return dict(q=_plain_rotate(s["q"], cos, sin, s["rot"], s["pairs"]),
                k=_plain_rotate(s["k"], cos, sin, s["rot"], s["pairs"]))


def run(state):
    s = state
    if s["op"] == "mm":
        if own:
            return s["weight_matrix"].mm(s["x"])
        return _plain_product(s["weight"], s["x"], s["group"], s["cols"]).to(s["x"].dtype)
    if s["op"] == "gated":
        if own:
            return s["gate_matrix"].gated(s["up_matrix"], s["x"], activation=s["act"])
        g = _plain_product(s["gate"], s["x"], s["group"], s["cols"])
        u = _plain_product(s["up"], s["x"], s["group"], s["cols"])
        return (_plain_act(g, s["act"]) * u).to(s["x"].dtype)
    if own:
        q, k = s["rotary"].apply(s["q"], s["k"], s["positions"], inverse=s["inverse"])
        return dict(q=q, k=k)
    return _plain_rotary(s)


# -------------------------------------------------------- what a pass needs

def work(case):
    n = case["tokens"]
    if case["op"] == "rotary":
        values = n * (case["heads"] + case["kv_heads"]) * case["dim"]
        turned = n * (case["heads"] + case["kv_heads"]) * case["rot"]
        return {"bytes": 4 * values + 4 * n * case["axes"], "flops": 3 * turned}
    rows, cols, groups = case["rows"], case["cols"], -(-case["cols"] // case["group"])
    weight = rows * cols / 2 + rows * groups * (2.5 if case["zeros"] else 2)
    two = 2 if case["op"] == "gated" else 1
    return {"bytes": two * weight + 2 * n * cols + 2 * n * rows, "flops": 2 * two * rows * cols * n}


# ------------------------------------------------------ definitions, 64 bits

def _exact_product(weight, x, group):
    codes, scales, zeros = weight
    x, out = x.double(), []
    for lo in range(0, codes.shape[0], 4096):  # some rows of the weight at a time
        byte = codes[lo:lo + 4096].to(torch.int32)
        w = torch.empty((byte.shape[0], 2 * byte.shape[1]), dtype=torch.float64, device=byte.device)
        w[:, 0::2], w[:, 1::2] = byte.remainder(16), byte.div(16, rounding_mode="floor")
        for g in range(scales.shape[1]):
            part = w[:, g * group:(g + 1) * group]
            part -= 8 if zeros is None else zeros[lo:lo + 4096, g, None].double()
            part *= scales[lo:lo + 4096, g, None].double()
        out.append(torch.einsum("nk,mk->nm", x, w))
    return torch.cat(out, 1)


def _exact_rotate(x, turn, rot, pairs):
    y = x.double()
    half = rot // 2
    z = torch.complex(y[..., :half].contiguous(), y[..., half:rot].contiguous()) if pairs == "half" else \
        torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], half, 2).contiguous())
    z = z * turn[:, None]
    out = y.clone()
    if pairs == "half":
        out[..., :half], out[..., half:rot] = z.real, z.imag
    else:
        out[..., 0:rot:2], out[..., 1:rot:2] = z.real, z.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        freq, axis = _frequencies(case)
        sign = -1.0 if case["inverse"] else 1.0
        at = torch.stack([s["positions"][a].double() * f for f, a in zip(freq, axis)], 1) * sign
        turn = torch.polar(torch.ones_like(at), at)
        return dict(q=_exact_rotate(s["q"], turn, case["rot"], case["pairs"]),
                    k=_exact_rotate(s["k"], turn, case["rot"], case["pairs"]))
    if case["op"] == "mm":
        return _exact_product(s["weight"], s["x"], case["group"])
    g, u = (_exact_product(s[name], s["x"], case["group"]) for name in ("gate", "up"))
    if case["act"] == "silu":
        g = torch.where(g >= 0, g / (1 + torch.exp(-g.abs())), g * torch.exp(-g.abs()) / (1 + torch.exp(-g.abs())))
    elif case["act"] == "gelu":
        g = 0.5 * g * torch.special.erfc(-g / math.sqrt(2.0))
    elif case["act"] == "gelu_tanh":
        g = g / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    else:
        g = g.relu()
    return g * u
