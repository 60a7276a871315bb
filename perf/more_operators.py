"""The operators of experts in other formats, as a serving program calls them: cases, inputs, plain forms and 64-bit values.

    quant     rows, or the SwiGLU of rows, in microscaled 4-bit floating point (e2m1 codes, one power of two per 32 of them)
    mx        product of such rows with such weights
    grouped   product of bf16 rows grouped by expert with each group's own weights, groups of any size
    mxgroup   the same of microscaled rows and weights
    dispatch  the grouping of tokens by their experts, and the weighted return of the experts' rows to the tokens

``own`` False: elementary torch operations in 32 bits (quotients by powers of two in 64).  True: the library's calls.
Microscaled rows come back as the values they stand for (exact in bf16), next to their scales.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}

# The limits of drawn cases: the largest listed ones.
MOST_QUANT = 8192 * 6144
MOST_PRODUCT = 8192 * 12288 * 6144
MOST_WEIGHTS = 12288 * 6144
MOST_EXPERTS = 256 * 4096 * 6144   # weights of all experts
MOST_GROUPED = 16384 * 4096 * 6144  # rows times weights of an expert
MOST_RETURN = 65536 * 6144


def listed():
    return [
        # a verify batch of four tokens between an expert's two products
        {"name": "quant 4 tokens", "op": "quant", "S": 4, "H": 2048, "silu": True, "up": False, "dtype": "f32", "pad": 0},
        # a long prompt's hidden states ahead of a product
        {"name": "quant 8192x6144", "op": "quant", "S": 8192, "H": 6144, "silu": False, "up": False, "dtype": "bf16", "pad": 0},
        # one token through the gate and up projections of a 2048-wide FFN: streams the weights
        {"name": "mx 1 token", "op": "mx", "S": 1, "N": 4096, "blocks": 192, "out": "bf16", "pad": 0},
        # sizes that fit no tile, rows cut out of a wider buffer
        {"name": "mx 77 odd f32", "op": "mx", "S": 77, "N": 577, "blocks": 35, "out": "f32", "pad": 3},
        # a long prompt through a dense layer's FFN
        {"name": "mx 8192", "op": "mx", "S": 8192, "N": 12288, "blocks": 192, "out": "bf16", "pad": 0},
        # a verify batch's gate and up projections: 32 rows over 256 experts
        {"name": "grouped 4 tokens", "op": "grouped", "S": 4, "k": 8, "E": 256, "N": 4096, "K": 6144, "gather": True, "out": "bf16"},
        # a small model's down projection, no size a multiple of a tile
        {"name": "grouped 700 tokens f32", "op": "grouped", "S": 700, "k": 3, "E": 24, "N": 1411, "K": 1000, "gather": False, "out": "f32"},
        # a long prompt's down projection: 256 rows an expert
        {"name": "grouped 8192 tokens", "op": "grouped", "S": 8192, "k": 8, "E": 256, "N": 6144, "K": 2048, "gather": False, "out": "bf16"},
        # one token of a decode step: eight experts' gate and up projections
        {"name": "mxgroup 1 token", "op": "mxgroup", "S": 1, "k": 8, "E": 256, "N": 4096, "K": 6144, "gather": True, "out": "bf16"},
        # a prompt chunk's gate and up projections: 64 rows an expert, every expert's weights read
        {"name": "mxgroup 2048 tokens", "op": "mxgroup", "S": 2048, "k": 8, "E": 256, "N": 4096, "K": 6144, "gather": True, "out": "bf16"},
        # one token of a decode step: latency
        {"name": "dispatch 1 token", "op": "dispatch", "S": 1, "k": 8, "E": 256, "H": 6144, "dropped": False, "add": True, "dtype": "bf16", "out": "f32"},
        # a long prompt's rows back from their experts, on top of the shared expert's
        {"name": "dispatch 8192 tokens", "op": "dispatch", "S": 8192, "k": 8, "E": 256, "H": 6144, "dropped": False, "add": True, "dtype": "bf16", "out": "bf16"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _size(rng, low, high):
    """A width: half of them multiples of 64, the others any number."""
    n = _log(rng, low, high)
    return max(64, n // 64 * 64) if rng.random() < 0.5 and high >= 64 else n


def draw(rng):
    op = rng.choice(["quant", "mx", "mx", "grouped", "grouped", "mxgroup", "mxgroup", "dispatch"])
    if op == "quant":
        H = _size(rng, 32, 16384)
        silu = rng.random() < 0.5
        return {"op": op, "S": _log(rng, 1, min(16384, MOST_QUANT // (2 * H if silu else H))), "H": H, "silu": silu,
                "up": rng.random() < 0.5, "dtype": rng.choice(["f32", "bf16", "bf16"]) if silu else "bf16", "pad": rng.choice([0, 0, 8, 5])}
    if op == "mx":
        blocks = _log(rng, 2, 512)
        N = _size(rng, 64, min(16384, MOST_WEIGHTS // (32 * blocks)))
        return {"op": op, "S": _log(rng, 1, min(8192, MOST_PRODUCT // (N * 32 * blocks))), "N": N, "blocks": blocks,
                "out": rng.choice(["f32", "bf16", "bf16"]) if N * 32 * blocks < MOST_WEIGHTS // 8 else "bf16", "pad": rng.choice([0, 0, 1, 5])}
    E = _log(rng, 4, 256)
    k = rng.randint(1, min(8, E))
    if op == "dispatch":
        H = _size(rng, 64, 8192)
        return {"op": op, "S": _log(rng, 1, min(8192, MOST_RETURN // (k * H))), "k": k, "E": E, "H": H, "dropped": rng.random() < 0.3,
                "add": rng.random() < 0.5, "dtype": "bf16", "out": rng.choice(["f32", "bf16"]) if k > 2 else "bf16"}
    K = _size(rng, 64, 8192)
    if K % 64 and rng.random() < 0.7:
        K = (K + 7) // 8 * 8  # most rows start at a multiple of 16 bytes
    N = _size(rng, 64, min(8192, MOST_EXPERTS // (4 * E * K)))
    return {"op": op, "S": _log(rng, 1, min(8192, max(1, MOST_GROUPED // (2 * k * N * K)))), "k": k, "E": E, "N": N, "K": K,
            "gather": rng.random() < 0.5, "out": rng.choice(["f32", "bf16", "bf16"])}


# ---- inputs ---------------------------------------------------------------------------------------------------------

def _rows(g, S, width, pad, dtype):
    """Hidden states: N(0, 1) with a few channels twenty times as wide, rows `pad` elements apart."""
    wide = 1.0 + 19.0 * (torch.rand(width + pad, generator=g, device="cuda") < 0.002)
    return (torch.randn(S, width + pad, generator=g, device="cuda") * wide).to(dtype)[:, :width]


def _microscaled(g, rows, blocks, pad, size):
    """(codes [rows, 16 blocks], scales [rows, blocks]): blocks drawn from 65536 of N(0, size^2) each with a spread of its own."""
    v = torch.randn(65536, 32, generator=g, device="cuda") * (size * torch.exp(0.3 * torch.randn(65536, 1, generator=g, device="cuda")))
    c, e = _plain_codes(v, False)
    pick = torch.randint(0, 65536, (rows, blocks + pad), generator=g, device="cuda")
    q = c[pick].flatten(1)
    return q[:, :16 * blocks], e.view(-1)[pick][:, :blocks]


def _routing(g, case):
    """The experts of each token, some of them busier than others: [S, k] int32, no expert twice in a row."""
    busy = 0.7 * torch.randn(case["E"], generator=g, device="cuda")
    score = busy + torch.randn(case["S"], case["E"], generator=g, device="cuda")
    return score.topk(case["k"], dim=1).indices.to(torch.int32)


def _plan(idx, E):
    """(first row of each expert and the end, pairs in the experts' order, place of each pair in it or -1); -1 goes last."""
    flat = torch.where(idx.flatten() < 0, E, idx.flatten()).long()
    order = torch.sort(flat, stable=True).indices
    first = torch.zeros(E + 1, dtype=torch.int32, device=idx.device)
    first[1:] = torch.bincount(flat, minlength=E + 1)[:E].cumsum(0)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=idx.device)
    place = torch.where(flat < E, place, -1)
    return first, order.to(torch.int32), place.to(torch.int32).view(idx.shape)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op == "quant":
        s["x"] = _rows(g, case["S"], case["H"] * (2 if case["silu"] else 1), case["pad"], DTYPES[case["dtype"]])
        return s
    if op == "mx":
        s["q"], s["e"] = _microscaled(g, case["S"], case["blocks"], case["pad"], 1.0)
        s["w"], s["ew"] = _microscaled(g, case["N"], case["blocks"], 0, 0.02)
        return s
    S, k, E = case["S"], case["k"], case["E"]
    idx = _routing(g, case)
    if op == "dispatch":
        if case["dropped"]:  # pairs that found no room
            idx = torch.where(torch.rand(S, k, generator=g, device="cuda") < 0.1, -1, idx)
        s["idx"] = idx
        w = torch.rand(S, k, generator=g, device="cuda") + 0.1
        s["w"] = 2.5 * w / w.sum(1, keepdim=True)
        s["z"] = torch.randn(S * k, case["H"], generator=g, device="cuda", dtype=DTYPES[case["dtype"]])
        s["add"] = torch.randn(S, case["H"], generator=g, device="cuda", dtype=DTYPES[case["dtype"]]) if case["add"] else None
        return s
    s["first"], s["order"], _ = _plan(idx, E)
    s["ends"] = s["first"].tolist()  # for the plain form, which launches expert by expert
    rows = S if case["gather"] else S * k
    if op == "grouped":
        s["x"] = torch.randn(rows, case["K"], generator=g, device="cuda", dtype=torch.bfloat16)
        s["w"] = torch.randn(E, case["N"], case["K"], generator=g, device="cuda", dtype=torch.bfloat16) * 0.02
    else:
        blocks = (case["K"] + 31) // 32
        s["q"], s["e"] = _microscaled(g, rows, blocks, 0, 1.0)
        s["w"] = torch.empty(E, case["N"], 16 * blocks, dtype=torch.uint8, device="cuda")
        s["ew"] = torch.empty(E, case["N"], blocks, dtype=torch.uint8, device="cuda")
        for i in range(0, E, 32):
            n = min(32, E - i)
            w, ew = _microscaled(g, n * case["N"], blocks, 0, 0.02)
            s["w"][i:i + n], s["ew"][i:i + n] = w.view(n, case["N"], -1), ew.view(n, case["N"], -1)
    return s


# ---- the plain forms ------------------------------------------------------------------------------------------------

def _plain_codes(v, up):
    """Blocks v [..., 32] as (codes [..., 16], two to a byte, scales [..., 1]): the scale is the power of two a quarter of that
    of the largest magnitude, or twice it where `up` and a value would exceed 6; codes the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6."""
    m, p = torch.frexp(v.abs().amax(-1, keepdim=True))
    e = p - 3 + (m > 0.75) if up else p - 3
    e = torch.where(m > 0, (e + 127).clamp(0, 254), 0)
    a = v.abs().double() / _scales(e)
    c = torch.where(a < 2, (2 * a).round(), torch.where(a < 4, 2 + a.round(), 4 + (a / 2).round())).clamp(max=7).to(torch.uint8)
    c = c + 8 * torch.signbit(v)
    return c[..., 0::2] + 16 * c[..., 1::2], e.to(torch.uint8)


def _plain_values(q, e):
    """The numbers that codes [..., 16 blocks] with scales [..., blocks] stand for, in fp32."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=q.device)
    grid = torch.cat((grid, -grid))
    c = torch.stack((q & 15, q >> 4), -1).flatten(-2)
    v = grid[c.int()].unflatten(-1, (-1, 32))
    return (v * _scales(e)[..., None].float()).flatten(-2)


def _scales(e):
    """2^(e - 127) in fp64, by its bits."""
    return ((e.long() + 896) << 52).view(torch.float64)


def _plain_quant(s):
    case, v = s["case"], s["x"].float()
    if case["silu"]:
        g, u = v.chunk(2, 1)
        v = g / (1.0 + torch.exp(-g)) * u
    H = case["H"]
    padded = torch.nn.functional.pad(v, (0, -H % 32))
    q, e = _plain_codes(padded.unflatten(1, (-1, 32)), case["up"])
    q, e = q.flatten(1), e.squeeze(-1)
    return _plain_values(q, e)[:, :H].to(torch.bfloat16), _scales(e)


def _plain_grouped(s, values):
    case, ends = s["case"], s["ends"]
    y = torch.empty(case["S"] * case["k"], case["N"], dtype=DTYPES[case["out"]], device="cuda")
    for i in range(case["E"]):
        lo, hi = ends[i], ends[i + 1]
        if lo < hi:
            rows = s["order"][lo:hi].long() // case["k"] if case["gather"] else slice(lo, hi)
            a, w = values(i, rows)
            y[lo:hi] = (a @ w.t()).to(y.dtype)
    return y


def _plain_dispatch(s):
    case = s["case"]
    first, order, place = _plan(s["idx"], case["E"])
    w = torch.where(place < 0, 0.0, s["w"])
    y = (s["z"][place.clamp(min=0).long()].float() * w[..., None]).sum(1)
    if s["add"] is not None:
        y = y + s["add"].float()
    return first, order, place, y.to(DTYPES[case["out"]])


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "quant":
        return _plain_quant(s)
    if op == "mx":
        return (_plain_values(s["q"], s["e"]) @ _plain_values(s["w"], s["ew"]).t()).to(DTYPES[case["out"]])
    if op == "grouped":
        return _plain_grouped(s, lambda i, rows: (s["x"][rows].float(), s["w"][i].float()))
    if op == "mxgroup":
        return _plain_grouped(s, lambda i, rows: (_plain_values(s["q"][rows], s["e"][rows]), _plain_values(s["w"][i], s["ew"][i])))
    return _plain_dispatch(s)


# ---- the library's calls --------------------------------------------------------------------------------------------

def _calls(s):
    from int4_routed_expert_amd import moe as M
    case, op = s["case"], s["case"]["op"]
    if op == "quant":
        q, e = (M.mx_silu_quant if case["silu"] else M.mx_quant)(s["x"], round_up=case["up"])
        return M.mx_values(q, e, width=case["H"]), _scales(e)
    if op == "mx":
        # the state's codes are wider integers than the bytes that the call takes
        return M.mx_matmul(s["q"].to(torch.uint8), s["e"], s["w"].to(torch.uint8), s["ew"], out_dtype=DTYPES[case["out"]])
    if op == "dispatch":
        first, order, place = M.group(s["idx"], case["E"])
        return first, order, place, M.combine(s["z"], s["w"], place, add=s["add"], out_dtype=DTYPES[case["out"]])
    # gathered: row i is that of the token of pair order[i]
    plan = {"order": s["order"], "top_k": case["k"]} if case["gather"] else {}
    if op == "grouped":
        return M.grouped_matmul(s["x"], s["w"], s["first"], out_dtype=DTYPES[case["out"]], **plan)
    return M.mx_grouped_matmul(s["q"].to(torch.uint8), s["e"], s["w"], s["ew"], s["first"], out_dtype=DTYPES[case["out"]], **plan)


def run(state):
    return _calls(state) if own else _plain(state)


# ---- what a pass cannot do without ------------------------------------------------------------------------------------

def _busy(case):
    """How many experts have rows, as far as the sizes say: each pair finds one, most often another one."""
    E, T = case["E"], case["S"] * case["k"]
    return min(E, max(case["k"], round(E * (1 - (1 - 1 / E) ** T))))


def work(case):
    op, S = case["op"], case["S"]
    size = {"f32": 4, "bf16": 2}
    if op == "quant":
        n = S * case["H"]
        blocks = S * ((case["H"] + 31) // 32)
        return {"bytes": n * size[case["dtype"]] * (2 if case["silu"] else 1) + 2 * n + 8 * blocks, "flops": (8 if case["silu"] else 3) * n}
    if op == "mx":
        N, blocks = case["N"], case["blocks"]
        return {"bytes": 17 * blocks * (S + N) + S * N * size[case["out"]], "flops": 64 * S * N * blocks}
    T, E = S * case["k"], case["E"]
    if op == "dispatch":
        H = case["H"]
        rows = (T + (S if case["add"] else 0)) * H * size[case["dtype"]]
        return {"bytes": rows + S * H * size[case["out"]] + 16 * T + 4 * (E + 1), "flops": 2 * T * H}
    N, K = case["N"], case["K"]
    row = 2 * K if op == "grouped" else 17 * ((K + 31) // 32)
    return {"bytes": (S if case["gather"] else T) * row + _busy(case) * N * row + T * N * size[case["out"]] + 4 * (E + 1) + (4 * T if case["gather"] else 0),
            "flops": 2 * T * N * K}


# ---- 64-bit values ----------------------------------------------------------------------------------------------------

def _numbers(q, e):
    """Codes and scales as fp64, from the fields of e2m1: sign, two bits of exponent (bias 1), one of mantissa."""
    c = torch.empty(*q.shape[:-1], 2 * q.shape[-1], dtype=torch.int64, device=q.device)
    c[..., 0::2], c[..., 1::2] = q % 16, q // 16
    power, half = c // 2 % 4, (c % 2).double() / 2
    v = torch.where(power == 0, half, (1 + half) * 2.0 ** (power - 1).double()) * (1 - 2 * (c // 8)).double()
    return v * (2.0 ** (e.double() - 127)).repeat_interleave(32, dim=-1)


def _exact_quant(s):
    case, v = s["case"], s["x"].double()
    H = case["H"]
    if case["silu"]:
        v = v[:, :H] * torch.sigmoid(v[:, :H]) * v[:, H:]
    blocks = (H + 31) // 32
    b = torch.zeros(case["S"], blocks * 32, dtype=torch.float64, device="cuda")
    b[:, :H] = v
    b = b.view(case["S"], blocks, 32)
    top = b.abs().amax(2)
    power = torch.floor(torch.log2(top))
    power = power + (2.0 ** (power + 1) <= top).double() - (2.0 ** power > top).double()
    step = 2.0 ** (power - 2)
    if case["up"]:
        step = torch.where(top > 6 * step, 2 * step, step)
    step = torch.where(top == 0, 2.0 ** -127, step.clamp(2.0 ** -127, 2.0 ** 127))
    a = (b / step[..., None]).abs()
    unit = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))  # between neighbours
    near = (torch.round(a / unit) * unit).clamp(max=6) * torch.sign(b)
    return (near * step[..., None]).view(case["S"], -1)[:, :H], step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        return _exact_quant(s)
    if op == "mx":
        return torch.mm(_numbers(s["q"], s["e"]), _numbers(s["w"], s["ew"]).t().contiguous())
    if op == "dispatch":
        S, k, E = case["S"], case["k"], case["E"]
        flat = s["idx"].flatten().long()
        flat = torch.where(flat < 0, E, flat)
        # a pair's place: the pairs of lower experts, and those of its own ahead of it
        order = torch.argsort(flat * (S * k) + torch.arange(S * k, device="cuda"))
        first = torch.searchsorted(flat[order], torch.arange(E + 1, device="cuda")).to(torch.int32)
        place = torch.argsort(order)
        kept = flat < E
        pairs = s["w"].double().flatten() * kept
        y = torch.zeros(S, case["H"], dtype=torch.float64, device="cuda")
        at = place.view(S, k)
        for j in range(k):
            y += pairs.view(S, k)[:, j, None] * s["z"][at[:, j]].double()
        if s["add"] is not None:
            y += s["add"].double()
        return first, order.to(torch.int32), torch.where(kept, place, -1).to(torch.int32).view(S, k), y
    T, k = case["S"] * case["k"], case["k"]
    group = torch.bucketize(torch.arange(T, device="cuda"), s["first"].long(), right=True) - 1
    source = torch.div(s["order"].long(), k, rounding_mode="floor") if case["gather"] else torch.arange(T, device="cuda")
    y = torch.zeros(T, case["N"], dtype=torch.float64, device="cuda")
    for i in torch.unique(group).tolist():
        mine = torch.nonzero(group == i).flatten()
        if op == "grouped":
            y[mine] = torch.mm(s["x"][source[mine]].double(), s["w"][i].double().t().contiguous())
        else:
            y[mine] = torch.mm(_numbers(s["q"][source[mine]], s["e"][source[mine]]), _numbers(s["w"][i], s["ew"][i]).t().contiguous())
    return y
