"""Microscaled rows, products grouped by expert, grouping and return, on the GPU against plain forms in 64 bits.

Tolerances, derived before the first run, in units of U = 2^-24 (half a step of fp32, relative).
  quant    the codes and scales are the formula's, bit for bit (powers of two scale exactly; one rounding).  Of a SwiGLU:
           those of the fp32 SwiGLU that moe_silu_quant writes, bit for bit.
  values   exact in fp32, one rounding in bf16.
  products of small whole numbers (and their halves): every partial sum is a multiple of a quarter below 2^22, so the sum
           in fp32 is exact in any order: equal.  Of other numbers: a product of two values is exact and is added up within
           one matrix instruction of at most 128 values and then over the instructions of at least 16 (bf16) or 64 values;
           each addition is off by at most 2 U (it may cut off) of a partial sum, at most sum |x w|: (128 + K / 16 + 16) 2 U
           sum |x w|, and 2^-8 of the result more where that is bf16 (half a step is 2^-9 of the next power of two).
  group    equal.
  combine  k products and sums of fp32 and the last one: (k + 1) 2 U (sum |w z| + |add|), and the output's rounding.
"""
import pytest
import torch

import mxref as R

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def M():
    from int4_routed_expert_amd import moe
    return moe


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def near(got, want, bound):
    """got within bound of want, in its type; NaN where want has them."""
    extra = 2.0 ** -8 if got.dtype == BF else 0.0
    g, w = got.double(), want.double()
    assert torch.equal(torch.isnan(g), torch.isnan(w))
    bad = (g - w).abs() > bound + extra * w.abs()
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, first {g[bad][:4].tolist()} for {w[bad][:4].tolist()}"


def padded(t, pad, fill=0):
    """t with its rows `pad` elements further apart."""
    buf = torch.full((*t.shape[:-1], t.shape[-1] + pad), fill, dtype=t.dtype, device=t.device)
    buf[..., :t.shape[-1]] = t
    return buf[..., :t.shape[-1]]


# ---- microscaled rows -------------------------------------------------------------------------------------------------

def hard_rows(S, H, dtype, seed):
    """Rows whose blocks lie at all magnitudes, with zeros, ties, values next to ties and to powers of two."""
    g = torch.Generator().manual_seed(seed)
    grid = torch.tensor(R.GRID)
    ties = torch.cat((grid, (grid[1:] + grid[:-1]) / 2, torch.tensor([7.0, 7.5, 6.5])))
    v = torch.randn(S, H, generator=g)
    t = ties[torch.randint(0, len(ties), (S, H), generator=g)] * (torch.randint(0, 2, (S, H), generator=g) * 2 - 1)
    v = torch.where(torch.rand(S, 1, generator=g) < 0.5, t, v)
    v = torch.where(torch.rand(S, H, generator=g) < 0.2, torch.nextafter(v, torch.randn(S, H, generator=g).sign() * 100), v)
    scale = torch.exp2(torch.randint(-20, 20, (S, (H + 31) // 32), generator=g).float()).repeat_interleave(32, 1)[:, :H]
    v = (v * scale).double()
    v[torch.rand(S, H, generator=g) < 0.1] = 0
    return v.to(dtype).cuda()


@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("S,H,dtype,pad", [(1, 1, F32, 0), (1, 31, BF, 0), (3, 32, BF, 1), (5, 33, F32, 0), (2, 64, BF, 0),
                                           (7, 1000, F32, 3), (40, 2047, BF, 1), (300, 256, BF, 8), (64, 6144, BF, 0),
                                           (2000, 1024, F32, 0), (900, 3001, BF, 0)])
def test_quant(M, S, H, dtype, pad, up):
    x = padded(hard_rows(S, H, dtype, S + H), pad, fill=9e9)
    q, e = M.mx_quant(x, round_up=up)
    wq, we = R.quantise(x, up)
    assert torch.equal(e, we) and torch.equal(q, wq)
    if up:  # nothing is cut off: within half a step of the grid at most 6
        v = R.values(q, e)[:, :H]
        assert ((v - x.double()).abs() <= torch.exp2(e.double() - 127).repeat_interleave(32, 1)[:, :H]).all()


def test_quant_every_bf16(M):
    """Each finite bf16 number as the largest of its block, with smaller ones beside it."""
    bits = torch.arange(0, 0x7F80, dtype=torch.int32)
    m = bits.to(torch.int16).view(BF)
    g = torch.Generator().manual_seed(1)
    small = (torch.rand(len(m), 32, generator=g) * 2 - 1).double() * m.double()[:, None]
    x = small.to(BF)
    x = torch.where(x.double().abs() > m.double()[:, None], 0.0, x).to(BF)
    x[:, 5] = -m
    x = x.cuda()
    for up in (False, True):
        q, e = M.mx_quant(x, round_up=up)
        wq, we = R.quantise(x, up)
        assert torch.equal(e, we) and torch.equal(q, wq)


def test_quant_far_fp32(M):
    """fp32's ends: the largest numbers, denormals and zeros."""
    x = torch.zeros(6, 64, device="cuda")
    x[0, 0], x[0, 33] = 3.4028234e38, -3e38
    x[1, 1], x[1, 2], x[1, 40] = 2.0 ** -149, -2.0 ** -130, 2.0 ** -126
    x[2, 3], x[2, 4] = 2.0 ** -125, 1.9 * 2.0 ** -125
    x[3, 0] = 2.0 ** -124
    x[4, 0] = -0.0
    for up in (False, True):
        q, e = M.mx_quant(x, round_up=up)
        wq, we = R.quantise(x.cpu(), up)
        assert torch.equal(e.cpu(), we) and torch.equal(q.cpu(), wq)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_quant_poison_stays_in_its_block(M, dtype):
    x = torch.randn(4, 100, generator=rng(0), device="cuda").to(dtype)
    x[0, 3], x[1, 40], x[2, 99] = float("inf"), float("nan"), -float("inf")
    q, e = M.mx_quant(x)
    wq, we = R.quantise(x)
    assert torch.equal(e, we) and torch.equal(q, wq)
    assert (e == 255).sum() == 3
    v = M.mx_values(q, e, width=100, dtype=F32)
    assert torch.isnan(v[0, :32]).all() and torch.isfinite(v[0, 32:]).all() and torch.isnan(v[2, 96:]).all()


@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("S,I,dtype,pad,two", [(1, 32, F32, 0, False), (4, 2048, F32, 0, False), (9, 333, BF, 1, False),
                                               (600, 2048, BF, 0, False), (33, 100, F32, 4, True), (5, 65, BF, 3, True)])
def test_silu_quant(M, S, I, dtype, pad, two, up):
    gu = padded((3 * torch.randn(S, 2 * I, generator=rng(I), device="cuda")).to(dtype), pad)
    args = (gu[:, :I], gu[:, I:]) if two else (gu,)
    y, _, _ = M.silu_quant(*args, y_dtype=F32)
    q, e = M.mx_silu_quant(*args, round_up=up)
    wq, we = R.quantise(y, up)
    assert torch.equal(e, we) and torch.equal(q, wq)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_values_of_every_code_and_scale(M, dtype):
    e = torch.arange(256, dtype=torch.uint8, device="cuda").repeat_interleave(2).view(64, 8)
    q = torch.randint(0, 256, (64, 128), generator=rng(2), device="cuda", dtype=torch.uint8)
    q[:, :8] = torch.tensor([0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE], dtype=torch.uint8)
    got = M.mx_values(q, e, dtype=dtype)
    want = R.values(q.cpu(), e.cpu()).to(dtype)  # rounded once (over the type's range: infinity)
    assert torch.equal(torch.nan_to_num(got.cpu(), nan=-1.0), torch.nan_to_num(want, nan=-1.0))


@pytest.mark.parametrize("S,H,pad", [(1, 1, 0), (3, 31, 2), (700, 1000, 0), (5, 4097, 1), (2000, 2048, 0)])
def test_values_sizes(M, S, H, pad):
    q, e = M.mx_quant(torch.randn(S, H, generator=rng(H), device="cuda"))
    q, e = padded(q, 16 * pad, 255), padded(e, pad, 255)
    for dtype in (F32, BF):
        assert torch.equal(M.mx_values(q, e, width=H, dtype=dtype).double(), R.values(q, e)[:, :H])


# ---- products ---------------------------------------------------------------------------------------------------------

def whole(g, *shape, dtype=torch.uint8):
    """Codes whose values are 0, +-0.5, +-1, +-1.5, +-2 (mostly), and scales of 2^-1 .. 2^1, as q [.., 16 B], e [.., B]."""
    *lead, B = shape
    c = torch.randint(0, 5, (*lead, 32 * B), generator=g, device="cuda") + 8 * torch.randint(0, 2, (*lead, 32 * B), generator=g,
                                                                                           device="cuda")
    c = torch.where(torch.rand(*lead, 32 * B, generator=g, device="cuda") < 0.02, 7, c)
    q = (c[..., 0::2] + 16 * c[..., 1::2]).to(torch.uint8)
    return q, torch.randint(126, 129, (*lead, B), generator=g, device="cuda").to(torch.uint8)


# S, N, B, blocks between rows
MX = [(1, 1, 1, 0), (1, 16, 2, 0), (1, 33, 64, 0), (1, 100, 191, 0), (2, 17, 5, 1), (3, 64, 4, 0), (4, 577, 35, 3), (5, 31, 3, 0),
      (8, 130, 67, 1), (9, 48, 16, 0), (16, 16, 8, 0), (17, 65, 9, 2), (33, 100, 7, 0), (77, 577, 35, 3), (64, 256, 32, 0),
      (130, 257, 16, 0), (129, 300, 33, 0), (256, 640, 48, 0), (300, 520, 33, 1), (515, 384, 17, 0)]


@pytest.mark.parametrize("S,N,B,pad", MX)
def test_mx_matmul_whole_numbers(M, S, N, B, pad):
    g = rng(S * 7 + N)
    q, e = whole(g, S, B)
    w, ew = whole(g, N, B)
    want = R.values(q, e) @ R.values(w, ew).t().contiguous()
    q, e = padded(q, 16 * pad, 0x77), padded(e, pad, 255)
    w, ew = padded(w, 16 * pad, 0x77), padded(ew, pad, 255)
    assert torch.equal(M.mx_matmul(q, e, w, ew, out_dtype=F32).double(), want)
    assert torch.equal(M.mx_matmul(q, e, w, ew), want.to(BF))


@pytest.mark.parametrize("S,N,B", [(1, 300, 70), (6, 100, 200), (40, 77, 65), (200, 300, 40)])
def test_mx_matmul_any_numbers(M, S, N, B):
    x = torch.randn(S, 32 * B, generator=rng(S), device="cuda") * torch.exp2(torch.randint(-30, 30, (S, 1), device="cuda").float())
    q, e = M.mx_quant(x)
    w, ew = M.mx_quant(torch.randn(N, 32 * B, generator=rng(N), device="cuda") * 0.02)
    X, W = R.values(q, e), R.values(w, ew).t().contiguous()
    bound = (128 + 32 * B / 16 + 16) * 2 * U * (X.abs() @ W.abs())
    for dtype in (F32, BF):
        near(M.mx_matmul(q, e, w, ew, out_dtype=dtype), X @ W, bound)


@pytest.mark.parametrize("S", [1, 3, 20, 150])
def test_mx_matmul_poison_stays_in_its_rows(M, S):
    g = rng(S)
    q, e = whole(g, S, 20)
    w, ew = whole(g, 200, 20)
    want = R.values(q, e) @ R.values(w, ew).t().contiguous()
    e[S // 2, 13], ew[77, 3], ew[199, 19] = 255, 255, 255
    q[S // 2, 13 * 16:14 * 16] = 0
    want[S // 2], want[:, 77], want[:, 199] = float("nan"), float("nan"), float("nan")
    got = M.mx_matmul(q, e, w, ew, out_dtype=F32).double()
    assert torch.equal(torch.nan_to_num(got, nan=1e30), torch.nan_to_num(want, nan=1e30))


def counts_of(kind, E, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "few":
        return torch.randint(0, 3, (E,), generator=g)
    if kind == "one":  # all with one expert
        c = torch.zeros(E, dtype=torch.long)
        c[E // 2] = 45
        return c
    if kind == "many":
        return torch.randint(0, 80, (E,), generator=g) * torch.randint(0, 2, (E,), generator=g) + 1
    if kind == "none":
        return torch.zeros(E, dtype=torch.long)
    c = torch.randint(0, 30, (E,), generator=g)  # ragged, one far larger than the others
    c[E - 1] = 333
    return c


GROUPED = [  # counts, E, N, K, rows ahead of the first expert's, behind the last one's
    ("few", 6, 33, 64, 0, 0), ("few", 300, 40, 96, 2, 3), ("one", 9, 100, 128, 0, 0), ("many", 5, 65, 256, 1, 7),
    ("ragged", 7, 130, 160, 3, 70), ("none", 4, 20, 32, 2, 3), ("few", 1, 16, 32, 0, 1), ("many", 65, 48, 64, 0, 0),
    ("ragged", 3, 300, 512, 0, 0), ("few", 1024, 17, 32, 0, 0), ("few", 40, 600, 1024, 0, 0), ("many", 12, 272, 800, 5, 1)]


def plan(counts, ahead, behind):
    first = torch.zeros(len(counts) + 1, dtype=torch.int32)
    first[1:] = counts.cumsum(0)
    first = first + ahead
    return first.cuda(), int(first[-1]) + behind


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("kind,E,N,K,ahead,behind", GROUPED)
def test_mx_grouped(M, kind, E, N, K, ahead, behind, gather):
    g = rng(E + N)
    first, T = plan(counts_of(kind, E, N), ahead, behind)
    top_k = 3
    rows = T if not gather else T // top_k + 2
    order = torch.randint(0, rows * top_k, (T,), generator=g, device="cuda").to(torch.int32) if gather else None
    q, e = whole(g, rows, K // 32)
    w, ew = whole(g, E, N, K // 32)
    for dtype in (F32, BF):
        y = torch.full((T, N + 5), 7.0, dtype=dtype, device="cuda")[:, :N]
        want = R.product(R.values(q, e), R.values(w, ew), first.tolist(), y.double(), order, top_k).to(dtype)
        got = M.mx_grouped_matmul(q, e, w, ew, first, order, top_k if gather else None, out=y)
        assert got is y and torch.equal(got, want)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("kind,E,N,K,ahead,behind", GROUPED + [
    ("few", 6, 33, 1, 0, 0), ("few", 30, 40, 97, 0, 3), ("many", 5, 65, 255, 1, 7), ("ragged", 7, 130, 1003, 3, 70),
    ("ragged", 4, 257, 130, 0, 0), ("one", 3, 100, 1001, 0, 0), ("ragged", 5, 64, 72, 0, 0)])
def test_grouped(M, kind, E, N, K, ahead, behind, gather):
    g = rng(E + N)
    first, T = plan(counts_of(kind, E, N), ahead, behind)
    top_k = 2
    rows = T if not gather else T // top_k + 2
    order = torch.randint(0, rows * top_k, (T,), generator=g, device="cuda").to(torch.int32) if gather else None
    x = torch.randint(-4, 5, (rows, K), generator=g, device="cuda").to(BF)
    w = torch.randint(-4, 5, (E, N, K), generator=g, device="cuda").to(BF)
    for dtype in (F32, BF):
        y = torch.full((T, N + 3), 7.0, dtype=dtype, device="cuda")[:, :N]
        want = R.product(x.double(), w.double(), first.tolist(), y.double(), order, top_k).to(dtype)
        got = M.grouped_matmul(x, w, first, order, top_k if gather else None, out=y)
        assert got is y and torch.equal(got, want)


@pytest.mark.parametrize("xpad,wpad,epad", [(0, 8, 0), (8, 0, 16), (1, 0, 0), (0, 1, 0), (3, 5, 7)])
@pytest.mark.parametrize("kind", ["few", "many"])
def test_grouped_strides(M, kind, xpad, wpad, epad):
    E, N, K = 7, 70, 136
    g = rng(xpad + wpad)
    first, T = plan(counts_of(kind, E, N), 0, 0)
    x = padded(torch.randint(-4, 5, (T, K), generator=g, device="cuda").to(BF), xpad, 1e30)
    W = torch.randint(-4, 5, (E, N, K), generator=g, device="cuda").to(BF)
    buf = torch.full((E * (N * (K + wpad) + epad),), float("nan"), dtype=BF, device="cuda")
    w = buf.as_strided((E, N, K), (N * (K + wpad) + epad, K + wpad, 1))
    w.copy_(W)
    want = R.product(x.double(), W.double(), first.tolist(), torch.zeros(T, N, dtype=torch.float64, device="cuda"))
    assert torch.equal(M.grouped_matmul(x, w, first, out_dtype=F32).double(), want)


@pytest.mark.parametrize("kind", ["few", "ragged"])
def test_grouped_any_numbers(M, kind):
    E, N, K = 8, 200, 2000
    first, T = plan(counts_of(kind, E, 5), 0, 0)
    x = torch.randn(T, K, generator=rng(1), device="cuda").to(BF)
    w = torch.randn(E, N, K, generator=rng(2), device="cuda").to(BF)
    zeros = lambda: torch.zeros(T, N, dtype=torch.float64, device="cuda")
    want = R.product(x.double(), w.double(), first.tolist(), zeros())
    bound = (128 + K / 16 + 16) * 2 * U * R.product(x.double().abs(), w.double().abs(), first.tolist(), zeros())
    for dtype in (F32, BF):
        near(M.grouped_matmul(x, w, first, out_dtype=dtype), want, bound)


@pytest.mark.parametrize("kind", ["few", "ragged"])
def test_grouped_rows_outside_x_are_nan(M, kind):
    E, N, K, top_k = 5, 48, 64, 2
    g = rng(3)
    first, T = plan(counts_of(kind, E, 5), 0, 0)
    rows = 20
    order = torch.randint(0, rows * top_k, (T,), generator=g, device="cuda").to(torch.int32)
    order[0], order[T // 2], order[T - 1] = -1, rows * top_k, 2 ** 31 - 1
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[0] = bad[T // 2] = bad[T - 1] = True
    safe = torch.where(bad, 0, order)
    x = torch.randint(-4, 5, (rows, K), generator=g, device="cuda").to(BF)
    w = torch.randint(-4, 5, (E, N, K), generator=g, device="cuda").to(BF)
    want = R.product(x.double(), w.double(), first.tolist(), torch.zeros(T, N, dtype=torch.float64, device="cuda"), safe, top_k)
    got = M.grouped_matmul(x, w, first, order, top_k, out_dtype=F32).double()
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])
    q, e = M.mx_quant(x)
    v, ve = M.mx_quant(w.view(E * N, K))
    want = R.product(R.values(q, e), R.values(v, ve).view(E, N, K), first.tolist(), want, safe, top_k)
    got = M.mx_grouped_matmul(q, e, v.view(E, N, -1), ve.view(E, N, -1), first, order, top_k, out_dtype=F32).double()
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("bad", [[0, 500, 10, 20], [-7, 5, 10, 20], [0, 10, 4, 20], [30, 20, 10, 0]])
def test_grouped_bad_first_stays_in_range(M, bad):
    """first beyond T, below 0 or decreasing: rows of experts it does describe are right, and nothing else is touched."""
    E, N, K, T = 3, 40, 64, 20
    g = rng(4)
    x = torch.randint(-4, 5, (T, K), generator=g, device="cuda").to(BF)
    w = torch.randint(-4, 5, (E, N, K), generator=g, device="cuda").to(BF)
    buf = torch.full((T + 20, N), 7.0, device="cuda")
    M.grouped_matmul(x, w, torch.tensor(bad, dtype=torch.int32, device="cuda"), out=buf[10:10 + T])
    assert (buf[:10] == 7).all() and (buf[10 + T:] == 7).all()


# ---- grouping and return ----------------------------------------------------------------------------------------------

@pytest.mark.parametrize("S,k,E", [(0, 4, 7), (1, 1, 1), (1, 8, 256), (5, 3, 1024), (64, 1, 2), (100, 8, 16), (1000, 8, 256),
                                   (1024, 8, 1024), (1025, 8, 64), (9000, 1, 3), (8192, 8, 256), (30001, 3, 1023)])
def test_group(M, S, k, E):
    g = torch.Generator().manual_seed(S + E)
    idx = torch.randint(-1, E + 1, (S, k), generator=g, dtype=torch.int32)
    if S * k > 5:
        idx.view(-1)[3], idx.view(-1)[4] = -2 ** 31, 2 ** 31 - 1
    first, order, place = M.group(idx.cuda(), E)
    key = torch.where((idx < 0) | (idx >= E), E, idx).flatten().long()
    worder = torch.sort(key, stable=True).indices
    wplace = torch.empty_like(worder)
    wplace[worder] = torch.arange(S * k)
    wplace = torch.where(key < E, wplace, -1)
    wfirst = torch.zeros(E + 1, dtype=torch.long)
    wfirst[1:] = torch.bincount(key, minlength=E + 1)[:E].cumsum(0)
    assert torch.equal(first.cpu().long(), wfirst)
    assert torch.equal(order.cpu().long(), worder)
    assert torch.equal(place.cpu().long(), wplace.view(S, k))


@pytest.mark.parametrize("dropped", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("S,k,H,dtype,out,add,pad", [
    (1, 1, 1, F32, F32, False, 0), (1, 8, 6144, BF, F32, True, 0), (7, 3, 333, BF, BF, True, 1), (30, 8, 2048, F32, BF, False, 0),
    (5, 9, 2049, F32, F32, True, 3), (300, 16, 64, BF, BF, True, 8), (2000, 8, 4096, BF, BF, True, 0), (3, 20, 100, BF, F32, False, 0)])
def test_combine(M, S, k, H, dtype, out, add, pad, dropped):
    g = rng(S + H)
    T = S * k
    z = padded(torch.randn(T, H, generator=g, device="cuda").to(dtype), pad)
    w = torch.randn(S, k, generator=g, device="cuda")
    place = torch.randperm(T, generator=g, device="cuda").to(torch.int32).view(S, k)
    gone = torch.rand(S, k, generator=g, device="cuda") < dropped
    z[place[gone].long()] = float("nan")  # rows that no pair has are not read
    w[gone] = float("inf")
    place[gone] = -1
    if dropped and T > 3:
        place[gone.nonzero()[0, 0], gone.nonzero()[0, 1]] = T
    a = padded(torch.randn(S, H, generator=g, device="cuda").to(dtype), pad) if add else None
    picked = torch.where(gone[..., None], 0.0, z[torch.where(gone, 0, place).long()].double()) * torch.where(gone, 0.0, w.double())[..., None]
    want, size = picked.sum(1), picked.abs().sum(1)
    if add:
        want, size = want + a.double(), size + a.double().abs()
    near(M.combine(z, w, place, add=a, out_dtype=out), want, (k + 1) * 2 * U * size)
