"""The operators of a layer's dense path, as a serving program calls them: cases, inputs, plain forms and 64-bit values.

    norm     h = x + residual; RMS norm of h; its rows in int8 with one scale each
    qmatmul  product of int8 rows with int8 weights, a scale for each token and one for each output channel
    silu     silu(gate) * up; its rows in int8 with one scale each
    rope     rotary positions of queries and keys

``own`` False: elementary torch operations in 32 bits (the angles in 64).  True: the library's calls.
Rows in int8 come back as the values they stand for (integer times scale, in bf16), next to their scales.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5  # of every norm here

# The limits of drawn cases: the largest listed ones.
MOST_NORM = 8192 * 6144
MOST_PRODUCT = 8192 * 12288 * 6144
MOST_WEIGHTS = 12288 * 6144
MOST_SILU = 4096 * 12288
MOST_ROPE = 8192 * 72 * 128


def listed():
    return [
        # one token of a decode step ahead of its layer: latency
        {"name": "norm 1 token", "op": "norm", "S": 1, "H": 6144, "dtype": "bf16", "residual": True, "y": "bf16", "pad": 0},
        # fp32 activations of odd width cut out of a wider buffer, no residual: a small model's tail chunk
        {"name": "norm 500x2047 f32", "op": "norm", "S": 500, "H": 2047, "dtype": "f32", "residual": False, "y": "f32", "pad": 3},
        # a long prompt's hidden states
        {"name": "norm 8192x6144", "op": "norm", "S": 8192, "H": 6144, "dtype": "bf16", "residual": True, "y": "bf16", "pad": 0},
        # one token through the gate and up projections of a 2048-wide FFN: streams the weights
        {"name": "qmatmul 1 token", "op": "qmatmul", "S": 1, "N": 4096, "K": 6144, "out": "bf16", "pad": 0},
        # sizes that fit no tile, rows that start at any byte
        {"name": "qmatmul 77 odd f32", "op": "qmatmul", "S": 77, "N": 577, "K": 1111, "out": "f32", "pad": 0},
        # a batch of decoding sequences, or a short prompt
        {"name": "qmatmul 256", "op": "qmatmul", "S": 256, "N": 6144, "K": 6144, "out": "bf16", "pad": 0},
        # a long prompt through a dense layer's FFN
        {"name": "qmatmul 8192", "op": "qmatmul", "S": 8192, "N": 12288, "K": 6144, "out": "bf16", "pad": 0},
        # a verify batch of four tokens between the FFN's two products
        {"name": "silu 4 tokens", "op": "silu", "S": 4, "I": 2048, "dtype": "f32", "pad": 0},
        # a prompt chunk between a dense layer's two products
        {"name": "silu 4096x12288", "op": "silu", "S": 4096, "I": 12288, "dtype": "bf16", "pad": 0},
        # decoding sequences at far positions, rotary part split off the heads, one shared key
        {"name": "rope 8 tokens", "op": "rope", "S": 8, "heads": 64, "kheads": 1, "D": 64, "rot": 64, "offset": 0,
         "inter": True, "dtype": "bf16", "scaling": "none", "far": 200000},
        # fp32, the last 64 of 192 dimensions, odd counts
        {"name": "rope 999 part f32", "op": "rope", "S": 999, "heads": 24, "kheads": 3, "D": 192, "rot": 64, "offset": 128,
         "inter": True, "dtype": "f32", "scaling": "linear", "far": 32768},
        # a long prompt with grouped keys, half layout, frequencies blended for four times the trained context
        {"name": "rope 8192", "op": "rope", "S": 8192, "heads": 64, "kheads": 8, "D": 128, "rot": 128, "offset": 0,
         "inter": False, "dtype": "bf16", "scaling": "blend", "far": 131072},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _size(rng, low, high):
    """A width: half of them multiples of 64, the others any number."""
    n = _log(rng, low, high)
    return max(64, n // 64 * 64) if rng.random() < 0.5 and high >= 64 else n


def draw(rng):
    op = rng.choice(["norm", "qmatmul", "qmatmul", "silu", "rope"])
    pad = rng.choice([0, 0, 8, 5])  # elements between the rows of the input's buffer
    if op == "norm":
        H = _size(rng, 64, 16384)
        return {"op": op, "S": _log(rng, 1, min(16384, MOST_NORM // H)), "H": H, "dtype": rng.choice(["f32", "bf16", "bf16"]),
                "residual": rng.random() < 0.6, "y": rng.choice(["none", "f32", "bf16"]), "pad": pad}
    if op == "qmatmul":
        K = _size(rng, 64, 16384)
        N = _size(rng, 64, min(16384, MOST_WEIGHTS // K))
        return {"op": op, "S": _log(rng, 1, min(8192, MOST_PRODUCT // (N * K))), "N": N, "K": K,
                "out": rng.choice(["f32", "bf16", "bf16"]), "pad": pad * 2}
    if op == "silu":
        I = _size(rng, 64, 16384)
        return {"op": op, "S": _log(rng, 1, min(16384, MOST_SILU // I)), "I": I, "dtype": rng.choice(["f32", "bf16", "bf16"]), "pad": pad}
    D = 2 * _log(rng, 16, 128)
    rot = D if rng.random() < 0.5 else 2 * rng.randint(8, D // 2)
    heads, kheads = _log(rng, 1, 64), _log(rng, 1, 8)
    return {"op": op, "S": _log(rng, 1, min(16384, MOST_ROPE // ((heads + kheads) * D))), "heads": heads, "kheads": kheads, "D": D,
            "rot": rot, "offset": rng.choice([0, D - rot]), "inter": rng.random() < 0.5, "dtype": rng.choice(["f32", "bf16", "bf16"]),
            "scaling": rng.choice(["none", "linear", "blend"]), "far": _log(rng, 512, 1000000)}


# ---- inputs ---------------------------------------------------------------------------------------------------------

def _rows(g, S, width, pad, dtype):
    """Hidden states: N(0, 1) with a few channels twenty times as wide, rows `pad` elements apart."""
    wide = 1.0 + 19.0 * (torch.rand(width + pad, generator=g, device="cuda") < 0.002)
    return (torch.randn(S, width + pad, generator=g, device="cuda") * wide).to(dtype)[:, :width]


def _codes(g, rows, width, pad):
    """Quantised rows: N(0, 1) in steps of a thirty-second, as rows whose largest value is four deviations have it."""
    n = torch.randn(rows, width + pad, generator=g, device="cuda").mul_(32).round_().clamp_(-127, 127)
    return n.to(torch.int8)[:, :width]


def _frequencies(case):
    """(float64 [rot / 2], factor of the sines and cosines): 10000^(-2i/rot), divided by 4 for "linear"; "blend" divides the
    slow ones only, with a ramp between those that turn 32 times and once in 32768 tokens, and raises the factor."""
    R = case["rot"]
    f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    if case["scaling"] == "linear":
        return f / 4.0, 1.0
    if case["scaling"] == "blend":
        turns = 32768 * f / (2 * math.pi)
        slow = ((math.log(32.0) - turns.log()) / math.log(32.0)).clamp(0, 1)
        return f / 4.0 * slow + f * (1 - slow), 0.1 * math.log(4.0) + 1.0
    return f, 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op == "norm":
        dt = DTYPES[case["dtype"]]
        s["x"] = _rows(g, case["S"], case["H"], case["pad"], dt)
        s["residual"] = _rows(g, case["S"], case["H"], 0, dt) if case["residual"] else None
        s["gamma"] = (1.0 + 0.1 * torch.randn(case["H"], generator=g, device="cuda")).to(dt)
    elif op == "qmatmul":
        s["q"] = _codes(g, case["S"], case["K"], case["pad"])
        s["d"] = 0.01 + 0.04 * torch.rand(case["S"], generator=g, device="cuda")
        s["w"] = _codes(g, case["N"], case["K"], 0)
        s["dw"] = (0.02 / 32) * torch.randn(case["N"], generator=g, device="cuda").abs()
    elif op == "silu":
        s["gu"] = _rows(g, case["S"], 2 * case["I"], case["pad"], DTYPES[case["dtype"]])
    else:
        dt = DTYPES[case["dtype"]]
        # queries and keys as a projection leaves them: side by side in each token's row
        both = torch.randn(case["S"], case["heads"] + case["kheads"], case["D"], generator=g, device="cuda").to(dt)
        s["qk"] = both[:, :case["heads"]], both[:, case["heads"]:]
        s["pos"] = torch.randint(0, case["far"], (case["S"],), generator=g, device="cuda")
        f, s["factor"] = _frequencies(case)
        s["freqs"] = f.cuda()
    return s


# ---- the plain forms ------------------------------------------------------------------------------------------------

def _values(q, d):
    """What int8 rows stand for, in bf16."""
    return torch.mul(q, d[:, None], out=torch.empty(q.shape, dtype=torch.bfloat16, device=q.device))


def _plain_quant(v):
    """Rows in int8: d = max|v| / 127, q = v / d rounded to the nearest integer (all of them 0 in a row of zeros)."""
    d = v.abs().amax(1) / 127.0
    q = torch.where(d[:, None] > 0, v / d[:, None], 0.0).round().clamp(-127, 127)
    return _values(q.to(torch.int8), d), d


def _plain_norm(x, residual, gamma, y):
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    f = h.float()
    n = f / (f.square().mean(1, keepdim=True) + EPS).sqrt() * gamma.float()
    return (None if residual is None else h, None if y is None else n.to(y), *_plain_quant(n))


def _plain_qmatmul(q, d, w, dw, out):
    return (q.float() @ w.float().t() * d[:, None] * dw).to(out)


def _plain_silu(gu):
    g, u = gu.float().chunk(2, 1)
    return _plain_quant(g / (1.0 + torch.exp(-g)) * u)


def _plain_rope(x, cos, sin, case):
    o, R = case["offset"], case["rot"]
    f = x[..., o:o + R].float()
    a, b = (f[..., 0::2], f[..., 1::2]) if case["inter"] else (f[..., :R // 2], f[..., R // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    y = x.clone()
    y[..., o:o + R] = (torch.stack((a, b), -1).flatten(-2) if case["inter"] else torch.cat((a, b), -1)).to(x.dtype)
    return y


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        return _plain_norm(s["x"], s["residual"], s["gamma"], DTYPES.get(case["y"]))
    if op == "qmatmul":
        return _plain_qmatmul(s["q"], s["d"], s["w"], s["dw"], DTYPES[case["out"]])
    if op == "silu":
        return _plain_silu(s["gu"])
    angle = s["pos"].double()[:, None, None] * s["freqs"]
    cos, sin = (angle.cos() * s["factor"]).float(), (angle.sin() * s["factor"]).float()
    return tuple(_plain_rope(x, cos, sin, case) for x in s["qk"])


# ---- the library's calls --------------------------------------------------------------------------------------------

def _calls(s):
    from int4_routed_expert_amd import moe as M
    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        h, y, q, d = M.norm_quant(s["x"], s["gamma"], EPS, residual=s["residual"], y_dtype=DTYPES.get(case["y"]))
        return h, y, _values(q, d), d
    if op == "qmatmul":
        return M.qmatmul(s["q"], s["d"], s["w"], s["dw"], out_dtype=DTYPES[case["out"]])
    if op == "silu":
        _, q, d = M.silu_quant(s["gu"])
        return _values(q, d), d
    return M.rope(*s["qk"], s["pos"], s["freqs"], offset=case["offset"], interleaved=case["inter"], factor=s["factor"])


def run(state):
    return _calls(state) if own else _plain(state)


# ---- what a pass cannot do without ------------------------------------------------------------------------------------

def work(case):
    op, S = case["op"], case["S"]
    size = {"none": 0, "f32": 4, "bf16": 2}
    if op == "norm":
        t = size[case["dtype"]]
        each = t + (2 * t if case["residual"] else 0) + size[case["y"]] + 2  # the values of the int8 rows in bf16
        return {"bytes": S * case["H"] * each + case["H"] * t + 4 * S, "flops": 8 * S * case["H"]}
    if op == "qmatmul":
        N, K = case["N"], case["K"]
        return {"bytes": S * K + N * K + 4 * (S + N) + S * N * size[case["out"]], "flops": 2 * S * N * K}
    if op == "silu":
        return {"bytes": S * case["I"] * (2 * size[case["dtype"]] + 2) + 4 * S, "flops": 8 * S * case["I"]}
    n = S * (case["heads"] + case["kheads"]) * case["D"]
    return {"bytes": 2 * n * size[case["dtype"]] + 8 * S + 4 * case["rot"], "flops": 3 * n * case["rot"] // case["D"]}


# ---- 64-bit values ----------------------------------------------------------------------------------------------------

def _exact_rows(v):
    step = v.abs().max(dim=1).values / 127
    safe = torch.where(step == 0, torch.ones_like(step), step).unsqueeze(1)
    return torch.round(v / safe) * step.unsqueeze(1), step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"].double()
        if s["residual"] is not None:  # the norm is that of the stored sum, rounded to its type
            h = (h + s["residual"].double()).to(s["x"].dtype).double()
        n = h * torch.rsqrt((h * h).sum(1, keepdim=True) / case["H"] + EPS) * s["gamma"].double()
        return (h if s["residual"] is not None else None, n if case["y"] != "none" else None, *_exact_rows(n))
    if op == "qmatmul":
        return torch.mm(s["q"].double() * s["d"].double().unsqueeze(1), s["w"].double().t().contiguous() * s["dw"].double())
    if op == "silu":
        I = case["I"]
        g, u = s["gu"][:, :I].double(), s["gu"][:, I:].double()
        return _exact_rows(g * torch.sigmoid(g) * u)
    a = s["pos"].double().unsqueeze(1) * s["freqs"].unsqueeze(0)
    turn = torch.polar(torch.full_like(a, s["factor"]), a).unsqueeze(1)  # [S, 1, rot / 2], complex
    o, half, got = case["offset"], case["rot"] // 2, []
    for x in s["qk"]:
        y = x.double().clone()
        part = y[..., o:o + 2 * half].clone()
        pair = part.reshape(*part.shape[:2], half, 2) if case["inter"] else part.reshape(*part.shape[:2], 2, half).transpose(2, 3)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        y[..., o:o + 2 * half] = (z if case["inter"] else z.transpose(2, 3)).reshape(part.shape)
        got.append(y)
    return tuple(got)
