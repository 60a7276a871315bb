"""Microscaled rows and products grouped by expert in 64 bits, on whichever device the inputs are on."""
import torch

GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def quantise(v, up=False):
    """(q [S, 16 B], e [S, B]) of the rows v [S, H], by comparing each magnitude with the midpoints of the grid."""
    S, H = v.shape
    B = (H + 31) // 32
    full = torch.zeros(S, 32 * B, dtype=torch.float64, device=v.device)
    full[:, :H] = v.double()
    b = full.view(S, B, 32)
    poison = ~torch.isfinite(b).all(2)
    b = torch.where(poison[..., None], 0.0, b)
    m, p = torch.frexp(b.abs().amax(2))  # m in [0.5, 1)
    e = p - 3
    if up:
        e = e + (m > 0.75)
    e = torch.where(m > 0, (e + 127).clamp(min=0), 0)
    a = b.abs() * torch.exp2((127 - e).double())[..., None]
    grid = torch.tensor(GRID, dtype=torch.float64, device=v.device)
    mid = (grid[1:] + grid[:-1]) / 2
    low, high = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)  # differ at a midpoint: the even code
    c = torch.where(low % 2 == 0, low, high)
    c = c + 8 * torch.signbit(b)
    c = torch.where(poison[..., None], 0, c)
    e = torch.where(poison, 255, e)
    q = c[..., 0::2] + 16 * c[..., 1::2]
    return q.flatten(1).to(torch.uint8), e.to(torch.uint8)


def values(q, e):
    """What codes [..., 16 B] with scales [..., B] stand for, in fp64."""
    grid = torch.tensor(GRID + [-g for g in GRID], dtype=torch.float64, device=q.device)
    c = torch.stack((q & 15, q >> 4), -1).flatten(-2).long()
    scale = torch.where(e == 255, torch.nan, torch.exp2(e.double() - 127))
    return grid[c] * scale.repeat_interleave(32, -1)


def group(idx, E):
    """(first, order, place) of moe_group, by Python's stable sort."""
    flat = idx.flatten().tolist()
    key = [x if 0 <= x < E else E for x in flat]
    order = sorted(range(len(key)), key=lambda p: key[p])
    place = [-1] * len(key)
    for at, p in enumerate(order):
        if key[p] < E:
            place[p] = at
    first = [sum(k < e for k in key) for e in range(E + 1)]
    as32 = lambda v: torch.tensor(v, dtype=torch.int32)
    return as32(first), as32(order), as32(place).view(idx.shape)


def product(x, w, first, y, order=None, top_k=1):
    """y (fp64) with the rows of each expert written over: fp64 x [rows, K], w [E, N, K]."""
    for e in range(w.shape[0]):
        for_rows = range(int(first[e]), int(first[e + 1]))
        if len(for_rows) == 0:
            continue
        at = torch.tensor(list(for_rows), device=x.device)
        src = at if order is None else torch.div(order[at].long(), top_k, rounding_mode="floor")
        y[at] = x[src] @ w[e].t().contiguous()
    return y
