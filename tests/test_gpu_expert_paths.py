"""Every kernel of the products by name, at sizes where its tiles, stages and row blocks end in all ways; the operators
together, captured, on other streams, and at sizes beyond 32-bit offsets.

Whole numbers: every partial sum is a multiple of a quarter below 2^22 and so exact in fp32 in any order.
"""
import os
import sys

import pytest
import torch

import mxref as R
from tests.test_gpu_experts import U, near, rng, whole

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def M():
    from int4_routed_expert_amd import moe
    return moe


def kernels_of(M, call):
    """(result, names of the kernels that ran)."""
    M.moe_profile_enable(True)
    try:
        y = call()
        torch.cuda.synchronize()
        return y, set(M.moe_profile_report())
    finally:
        M.moe_profile_enable(False)


RAGGED = (256, 257, 1, 64, 65, 128, 129, 192, 193, 0, 200, 15)  # row blocks of the widest tiles: none to all


def counts(T, E):
    """T rows over E experts, as raggedly as RAGGED."""
    c = torch.tensor([RAGGED[i % len(RAGGED)] for i in range(E)], dtype=torch.float64)
    c = (c * T / c.sum()).floor().long()
    c[0] += T - c.sum()
    return c


def first_of(c):
    f = torch.zeros(len(c) + 1, dtype=torch.int32)
    f[1:] = c.cumsum(0)
    return f.cuda()


GROUPED = [  # kernel (of the microscaled product / of the bf16 one), T, E, N, K of each (None: not among these)
    ("vec2", 1, 4, 100, 1024, 512), ("vec8", 8, 40, 4000, 4096, 2048), ("few16/vec2", 20, 10, 500, 512, 512),
    ("few16", 20, 40, 1000, 256, None), ("tile32", 60, 40, 1500, 1536, None), ("tile32", 300, 10, 1000, 6144, 512),
    ("tile64", 300, 12, 2000, 544, 264), ("tile64", 500, 10, 2000, 1024, 1024), ("tile64", 330, 12, 2050, 2080, 1000),
    ("tile64", 900, 20, 4000, 2080, 2081), ("tile128", 2000, 20, 2000, 512, 512), ("tile128", 2000, 20, 2001, 96, 40),
    ("tile128/tile256x128", 600, 12, 4000, 1056, 1050), ("tile256x128", 600, 12, 4000, 4096, 1024),
    ("tile256x128", 601, 12, 4011, 4192, 1032), ("tile256x128", 1500, 12, 6000, 2080, 1050), ("tile128/tile256", 1500, 12, 4000, 256, 512),
    ("tile128/tile256", 1500, 12, 4100, 288, 264), ("tile256", 1500, 12, 4000, 1056, 512), ("tile256", 3000, 12, 6000, 544, 1055)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("kernel,T,E,N,K,mx", [(name.split("/")[0 if mx else -1], T, E, N, K, mx) for name, T, E, N, *both in GROUPED
                                               for mx, K in zip((True, False), both) if K])
def test_grouped_kernels(M, kernel, T, E, N, K, gather, mx):
    g = rng(T + N)
    first = first_of(counts(T, E))
    top_k = 3
    rows = T // top_k + 2 if gather else T
    order = torch.randint(0, rows * top_k, (T,), generator=g, device="cuda").to(torch.int32) if gather else None
    plan = (order, top_k) if gather else (None, None)
    zeros = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    if mx:
        q, e = whole(g, rows, (K + 31) // 32)
        w, ew = whole(g, E, N, (K + 31) // 32)
        want = R.product(R.values(q, e), R.values(w, ew), first.tolist(), zeros, order, top_k)
        call = lambda dtype: M.mx_grouped_matmul(q, e, w, ew, first, *plan, out_dtype=dtype)
    else:
        x = torch.randint(-4, 5, (rows, K), generator=g, device="cuda").to(BF)
        w = torch.randint(-4, 5, (E, N, K), generator=g, device="cuda").to(BF)
        want = R.product(x.double(), w.double(), first.tolist(), zeros, order, top_k)
        call = lambda dtype: M.grouped_matmul(x, w, first, *plan, out_dtype=dtype)
    got, names = kernels_of(M, lambda: call(F32))
    assert torch.equal(got.double(), want)
    assert torch.equal(call(BF), want.to(BF))
    if not gather:
        assert f"product_{kernel}" in names, names


MX = [("vec2", 1, 333, 70), ("vec2", 5, 500, 20), ("few16", 70, 600, 20), ("tile32", 90, 5000, 32), ("tile32", 300, 2000, 64), ("tile64", 600, 3000, 17),
      ("tile64", 100, 12000, 8), ("tile64", 600, 3000, 16), ("tile128", 2000, 6000, 16), ("tile128", 200, 16000, 33),
      ("tile128", 300, 9000, 67), ("tile128", 2500, 4001, 9), ("tile256x128", 600, 7000, 128), ("tile256x128", 600, 7000, 131),
      ("tile256", 1500, 20000, 16), ("tile256", 1000, 12001, 17), ("tile256", 700, 12000, 67)]


@pytest.mark.parametrize("kernel,S,N,B", MX)
def test_mx_kernels(M, kernel, S, N, B):
    g = rng(S + N)
    q, e = whole(g, S, B)
    w, ew = whole(g, N, B)
    want = R.values(q, e) @ R.values(w, ew).t().contiguous()
    got, names = kernels_of(M, lambda: M.mx_matmul(q, e, w, ew, out_dtype=F32))
    assert torch.equal(got.double(), want)
    assert torch.equal(M.mx_matmul(q, e, w, ew), want.to(BF))
    assert f"product_{kernel}" in names, names


@pytest.mark.parametrize("K", [509, 510, 511, 1001])
def test_grouped_rows_copied_first(M, K):
    """Rows off 16-byte boundaries through the tiles: both operands, and only one, copied to the workspace."""
    g = rng(K)
    T, E, N = 1500, 12, 4000
    first = first_of(counts(T, E))
    x = torch.randint(-4, 5, (T, K), generator=g, device="cuda").to(BF)
    w = torch.randint(-4, 5, (E, N, K), generator=g, device="cuda").to(BF)
    want = R.product(x.double(), w.double(), first.tolist(), torch.zeros(T, N, dtype=torch.float64, device="cuda"))
    got, names = kernels_of(M, lambda: M.grouped_matmul(x, w, first, out_dtype=F32))
    assert "product_align" in names and torch.equal(got.double(), want)
    # the caller's own workspace, with the memory behind it left as it was
    from int4_routed_expert_amd.moe import _GROUPS
    plan = _GROUPS.pack(first.data_ptr(), 0, E, 0)
    need = M.lib().moe_grouped_matmul_workspace_bytes(x.data_ptr(), K, T, w.data_ptr(), K, N * K, plan, T, N, K)
    ws = torch.full((need + 64,), 7, dtype=torch.uint8, device="cuda")
    assert torch.equal(M.grouped_matmul(x, w, first, out_dtype=F32, ws=ws[:need]).double(), want) and (ws[need:] == 7).all()
    with pytest.raises(M.MoeError) as err:
        M.grouped_matmul(x, w, first, ws=ws[:need - 1])
    assert err.value.status == M.MOE_EWORKSPACE
    if K % 8 == 0 or K == 1001:
        return
    even = torch.zeros(T, 512, dtype=BF, device="cuda")[:, :K // 8 * 8]
    even.copy_(x[:, :K // 8 * 8])
    odd = w[:, :, :K // 8 * 8]  # rows K apart
    want = R.product(even.double(), odd.double(), first.tolist(), torch.zeros(T, N, dtype=torch.float64, device="cuda"))
    assert torch.equal(M.grouped_matmul(even, odd, first, out_dtype=F32).double(), want)


@pytest.mark.parametrize("mx", [True, False])
@pytest.mark.parametrize("T,E,N,K", [(60, 40, 600, 512), (600, 12, 4000, 4096), (1500, 12, 4000, 512)])
def test_rows_of_no_expert_are_left_alone(M, T, E, N, K, mx):
    """Rows ahead of the first expert's and behind the last one's, columns beyond N, memory around the output."""
    g = rng(T)
    c = counts(T, E)
    first = first_of(c) + 5
    rows = T + 5 + 40
    y = torch.full((rows + 20, N + 8), 7.0, device="cuda")
    out = y[10:10 + rows, :N]
    if mx:
        q, e = whole(g, rows, K // 32)
        w, ew = whole(g, E, N, K // 32)
        want = R.product(R.values(q, e), R.values(w, ew), first.tolist(), out.double())
        M.mx_grouped_matmul(q, e, w, ew, first, out=out)
    else:
        x = torch.randint(-4, 5, (rows, K), generator=g, device="cuda").to(BF)
        w = torch.randint(-4, 5, (E, N, K), generator=g, device="cuda").to(BF)
        want = R.product(x.double(), w.double(), first.tolist(), out.double())
        M.grouped_matmul(x, w, first, out=out)
    assert torch.equal(out.double(), want)
    assert (y[:10] == 7).all() and (y[10 + rows:] == 7).all() and (y[:, N:] == 7).all()


@pytest.mark.parametrize("T,E,N,K", [(60, 40, 600, 512), (600, 12, 4000, 4096), (1500, 12, 4000, 512)])
def test_poison_stays_in_its_rows(M, T, E, N, K):
    """A NaN in a row of x, in a weight row, and an input that does not exist: those outputs only."""
    g = rng(T)
    first = first_of(counts(T, E))
    x = torch.randint(-4, 5, (T, K), generator=g, device="cuda").to(BF)
    w = torch.randint(-4, 5, (E, N, K), generator=g, device="cuda").to(BF)
    order = torch.arange(T, device="cuda", dtype=torch.int32)
    want = R.product(x.double(), w.double(), first.tolist(), torch.zeros(T, N, dtype=torch.float64, device="cuda"))
    bad = (3, T // 2, T - 2)
    x[bad[0], K - 1] = float("nan")
    order[bad[1]] = T
    w[0, N - 1, 0] = float("nan")
    want[bad[0]] = want[bad[1]] = float("nan")
    want[int(first[0]):int(first[1]), N - 1] = float("nan")
    got = M.grouped_matmul(x, w, first, order, 1, out_dtype=F32).double()
    assert torch.equal(torch.nan_to_num(got, nan=1e30), torch.nan_to_num(want, nan=1e30))


@pytest.mark.parametrize("T,E,N,K", [(8, 40, 4000, 4096), (20, 10, 500, 512), (60, 40, 600, 512), (600, 12, 4000, 4096),
                                     (1500, 12, 4000, 512)])
@pytest.mark.parametrize("short", [1, 7])
def test_rows_beyond_x_are_nan(M, T, E, N, K, short):
    """A call without order whose x has fewer rows than y."""
    g = rng(T)
    first = first_of(counts(T, E))
    rows = T - short
    x = torch.full((T, K), 3.0, device="cuda").to(BF)
    x[:rows] = torch.randint(-4, 5, (rows, K), generator=g, device="cuda").to(BF)
    w = torch.randint(-4, 5, (E, N, K), generator=g, device="cuda").to(BF)
    want = R.product(x.double(), w.double(), first.tolist(), torch.zeros(T, N, dtype=torch.float64, device="cuda"))
    plan = M.moe_groups(first.data_ptr(), None, E, 0)
    y = torch.zeros(T, N, device="cuda")
    M.moe_grouped_matmul(x, K, rows, w, K, N * K, plan, T, N, K, y, M.MOE_F32, N, None, 0)
    assert torch.equal(y[:rows].double(), want[:rows]) and torch.isnan(y[rows:]).all()
    q, e = M.mx_quant(x)
    v, ve = M.mx_quant(w.view(E * N, K))
    want = R.product(R.values(q, e), R.values(v, ve).view(E, N, K), first.tolist(), want)
    y = torch.zeros(T, N, device="cuda")
    a = M.moe_mx_rows(q.data_ptr(), e.data_ptr(), K // 2, K // 32, 0, 0)
    b = M.moe_mx_rows(v.data_ptr(), ve.data_ptr(), K // 2, K // 32, N * K // 2, N * K // 32)
    M.moe_mx_grouped_matmul(a, rows, b, plan, T, N, K // 32, y, M.MOE_F32, N, None, 0)
    assert torch.equal(y[:rows].double(), want[:rows]) and torch.isnan(y[rows:]).all()


@pytest.mark.parametrize("E", [1, 63, 65, 1000, 1024])
def test_many_experts(M, E):
    """One lane of the search has up to sixteen experts; most have no rows."""
    g = rng(E)
    c = torch.where(torch.rand(E, generator=torch.Generator().manual_seed(E)) < 0.05, 37, 0)
    c[-1] = 3
    first = first_of(c)
    T, N, K = int(first[-1]), 70, 64
    x = torch.randint(-4, 5, (T, K), generator=g, device="cuda").to(BF)
    w = torch.randint(-4, 5, (E, N, K), generator=g, device="cuda").to(BF)
    want = R.product(x.double(), w.double(), first.tolist(), torch.zeros(T, N, dtype=torch.float64, device="cuda"))
    assert torch.equal(M.grouped_matmul(x, w, first, out_dtype=F32).double(), want)


def test_far_operands(M):
    """Weights and outputs beyond 4 GB from their start, and gathered rows 4 GB apart."""
    g = rng(1)
    E, N, K, T = 3, 4096, 512, 700
    buf = torch.zeros(2 * ((5 << 30) // 2) + N * K, dtype=BF, device="cuda")  # experts 5 GB apart
    w = buf.as_strided((E, N, K), ((5 << 30) // 2, K, 1))
    w.copy_(torch.randint(-4, 5, (E, N, K), generator=g, device="cuda").to(BF))
    first = first_of(torch.tensor([300, 1, 399]))
    x = torch.randint(-4, 5, (T, K), generator=g, device="cuda").to(BF)
    want = R.product(x.double(), w.double(), first.tolist(), torch.zeros(T, N, dtype=torch.float64, device="cuda"))
    assert torch.equal(M.grouped_matmul(x, w, first, out_dtype=F32).double(), want)
    del buf, w
    w = torch.randint(-4, 5, (E, N, K), generator=g, device="cuda").to(BF)
    far = torch.zeros(699 * (8 << 20) + K, dtype=BF, device="cuda").as_strided((T, K), (8 << 20, 1))  # 16 MB apart
    far.copy_(x)
    want = R.product(x.double(), w.double(), first.tolist(), torch.zeros(T, N, dtype=torch.float64, device="cuda"))
    order = torch.arange(T, device="cuda", dtype=torch.int32).flip(0)
    wanted = R.product(x.double(), w.double(), first.tolist(), torch.zeros(T, N, dtype=torch.float64, device="cuda"), order, 1)
    assert torch.equal(M.grouped_matmul(far, w, first, out_dtype=F32).double(), want)
    assert torch.equal(M.grouped_matmul(far, w, first, order, 1, out_dtype=F32).double(), wanted)


# ---- together ---------------------------------------------------------------------------------------------------------

def experts(M, mx, E, H, I, seed):
    g = rng(seed)
    mats = [(torch.randn(E, n, k, generator=g, device="cuda") / k ** 0.5).to(BF) for n, k in ((2 * I, H), (H, I))]
    if not mx:
        return [(m,) for m in mats]
    out = []
    for m in mats:
        q, e = M.mx_quant(m.flatten(0, 1))
        out.append((q.view(E, m.shape[1], -1), e.view(E, m.shape[1], -1)))
    return out


def inputs(S, k, E, H, seed):
    g = rng(seed)
    idx = torch.rand(S, E, generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
    idx[torch.rand(S, k, generator=g, device="cuda") < 0.1] = -1  # pairs that found no room
    return (torch.randn(S, H, generator=g, device="cuda").to(BF), idx, torch.rand(S, k, generator=g, device="cuda"),
            torch.randn(S, H, generator=g, device="cuda").to(BF))


def layer(M, mx, w, x, idx, weights, add, E, stream=None):
    """Every stage's output, of tokens that go through their experts."""
    k = idx.shape[1]
    first, order, place = M.group(idx, E, stream=stream)
    if mx:
        rows = M.mx_quant(x, stream=stream)
        gu = M.mx_grouped_matmul(*rows, *w[0], first, order, k, stream=stream)
        act = M.mx_silu_quant(gu, stream=stream)
        z = M.mx_grouped_matmul(*act, *w[1], first, stream=stream)
    else:
        rows = (x,)
        gu = M.grouped_matmul(x, *w[0], first, order, k, stream=stream)
        act = M.silu_quant(gu, y_dtype=BF, quant=False, stream=stream)[:1]
        z = M.grouped_matmul(*act, *w[1], first, stream=stream)
    return first, order, place, rows, gu, act, z, M.combine(z, weights, place, add=add, out_dtype=F32, stream=stream)


def kept(outs, n):
    """The rows that belong to an expert: the others were never written."""
    first, order, place, rows, gu, act, z, y = outs
    return [first, order, place, *rows, gu[:n], *(t[:n] for t in act), z[:n], y]


SIZES = [(1, 8, 64, 512, 256), (5, 3, 9, 333 * 8, 320), (300, 4, 16, 1024, 512), (2000, 2, 8, 512, 1024)]  # S, k, E, H, I


@pytest.mark.parametrize("mx", [True, False])
@pytest.mark.parametrize("S,k,E,H,I", SIZES)
def test_layer_stage_by_stage(M, S, k, E, H, I, mx):
    """A layer's stages as they are used together, each against 64 bits of its own inputs."""
    w = experts(M, mx, E, H, I, S)
    x, idx, weights, add = inputs(S, k, E, H, S)
    outs = layer(M, mx, w, x, idx, weights, add, E)
    first, order, place, rows, gu, act, z, y = outs
    wf, wo, wp = R.group(idx.cpu(), E)
    assert torch.equal(first.cpu(), wf) and torch.equal(order.cpu(), wo) and torch.equal(place.cpu(), wp)
    n, bound = int(wf[-1]), wf.tolist()
    num = R.values if mx else (lambda t: t.double())
    blank = lambda width: torch.zeros(S * k, width, dtype=torch.float64, device="cuda")

    def product(got, a, b, plan):
        a, b = num(*a), num(*b)
        K = a.shape[1]
        want = R.product(a, b, bound, blank(b.shape[1]), *plan)
        size = R.product(a.abs(), b.abs(), bound, blank(b.shape[1]), *plan)
        near(got[:n], want[:n], ((128 + K / 16 + 16) * 2 * U * size)[:n])

    if mx:
        assert all(torch.equal(a, b) for a, b in zip(rows, R.quantise(x)))
    product(gu, rows, w[0], (order, k))
    silu = M.silu_quant(gu[:n], y_dtype=F32, quant=False)[0]
    want = R.quantise(silu) if mx else (silu.to(BF),)
    assert all(torch.equal(a[:n], b) for a, b in zip(act, want))
    product(z, act, w[1], (None, 1))
    at = place.clamp(min=0).long()
    terms = torch.where(place[..., None] >= 0, z[at].double() * weights.double()[..., None], 0.0)
    near(y, terms.sum(1) + add.double(), (k + 1) * 2 * U * (terms.abs().sum(1) + add.double().abs()))


@pytest.mark.parametrize("mx", [True, False])
@pytest.mark.parametrize("S,k,E,H,I", SIZES)
def test_layer_graph_replays(M, S, k, E, H, I, mx):
    """Captured once, replayed with new inputs between eager work: every replay equals the eager result."""
    w = experts(M, mx, E, H, I, 1)
    static = inputs(S, k, E, H, 1)
    layer(M, mx, w, *static, E)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = layer(M, mx, w, *static, E)
    for i in range(4):
        new = inputs(S, k, E, H, 10 + i)
        want = layer(M, mx, w, *new, E)
        n = int(want[0][-1])
        for a, b in zip(static, new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(kept(want, n), kept(outs, n)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("mx", [True, False])
@pytest.mark.parametrize("S,k,E,H,I", SIZES)
def test_layer_on_another_stream(M, S, k, E, H, I, mx):
    """Outputs and workspaces belong to the stream given, inputs may be freed at once, and two streams do not meet."""
    w = experts(M, mx, E, H, I, 2)
    args = [inputs(S, k, E, H, 20 + i) for i in range(2)]
    want = [layer(M, mx, w, *a, E) for a in args]
    n = [int(o[0][-1]) for o in want]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for st, a in zip(streams, args):
            fresh = [t.clone() for t in a]
            st.wait_stream(torch.cuda.current_stream())
            got.append(layer(M, mx, w, *fresh, E, stream=st))
            del fresh
        junk = [torch.full_like(t, 1) for a in args for t in a]
        for st in streams:
            st.synchronize()
        for o, v, m in zip(want, got, n):
            for a, b in zip(kept(o, m), kept(v, m)):
                assert torch.equal(a, b)
        del got, junk


def test_written_over_outputs_raise_their_version(M):
    x, w = torch.ones(3, 8, device="cuda").to(BF), torch.ones(1, 4, 8, device="cuda").to(BF)
    out = torch.zeros(3, 4, device="cuda")
    before = out._version
    M.grouped_matmul(x, w, first_of(torch.tensor([3])), out=out)
    assert out._version > before and (out == 8).all()
    with pytest.raises(ValueError):
        M.grouped_matmul(x, w, first_of(torch.tensor([3])), out=out, out_dtype=BF)


@pytest.mark.parametrize("tokens", [1, 16, 200])
def test_example_runs(M, tokens):
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import expert_layer as X
    for mx in (False, True):
        layer = X.Layer(mx)
        x = torch.randn(tokens, layer.c.hidden, generator=rng(tokens), device="cuda").to(BF)
        y = layer.forward(x)
        assert y.shape == x.shape and y.dtype == F32 and torch.isfinite(y).all()
