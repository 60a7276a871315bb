"""Paths of the dense operators that only certain sizes and places take, each named by the test that takes it:
workgroups that go on to a second row, launches in several pieces, copies of one operand, several tokens a workgroup,
and the layer's own int8 activations next to the dense operators'."""
import numpy as np
import pytest
import torch

from tests.test_gpu_dense import check_rope, operands

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
GRID = 1 << 20  # workgroups of a row kernel's launch at most, and of one piece of the rotary kernel's


@pytest.fixture(scope="module")
def M():
    from int4_routed_expert_amd import moe
    return moe


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("H,step", [(1040, 8), (1041, 9), (2056, 8), (4104, 8), (4105, 9), (6152, 8), (8200, 8), (8201, 9),
                                    (12296, 8), (12297, 9), (16392, 8)])
def test_rows_of_a_second_turn(M, H, step):
    """More rows than workgroups, at one row a workgroup: rows of the second turn, and their neighbours, equal the same
    rows in a small call.  The rows overlap in memory, `step` elements apart, so that they differ and fit."""
    S = GRID + 300
    g = rng(H)
    buf = torch.randn(S * step + H, generator=g, device="cuda").bfloat16()
    other = torch.randn(S * step + H, generator=g, device="cuda").bfloat16()
    x, r = (b.as_strided((S, H), (step, 1)) for b in (buf, other))
    gamma = torch.rand(H, generator=g, device="cuda")
    parts = [slice(0, 40), slice(290, 310), slice(GRID - 40, GRID + 40), slice(S - 40, S)]

    def small(call):
        return [[t for t in call(p) if t is not None] for p in parts]

    def same(many, few):
        many = [t for t in many if t is not None]
        for p, want in zip(parts, few):
            assert len(many) == len(want) and all(torch.equal(a[p], b) for a, b in zip(many, want))
    # two barriers a row
    same(M.norm_quant(x, gamma, 1e-5), small(lambda p: M.norm_quant(x[p], gamma, 1e-5)))
    same(M.silu_quant(x, r), small(lambda p: M.silu_quant(x[p], r[p])))
    if H < 2000:  # one barrier a row, and all outputs
        same(M.norm_quant(x, gamma, 1e-5, residual=r, y_dtype=BF, quant=False),
             small(lambda p: M.norm_quant(x[p], gamma, 1e-5, residual=r[p], y_dtype=BF, quant=False)))
        same(M.norm_quant(x, gamma, 1e-5, residual=r, y_dtype=BF),
             small(lambda p: M.norm_quant(x[p], gamma, 1e-5, residual=r[p], y_dtype=BF)))


def test_second_turns_after_far_rows(M):
    """A row that is summed twice (its squares leave the range of fp32) between rows of other turns of its workgroup."""
    S, H = GRID + 300, 1040
    buf = torch.randn(S * 8 + H, generator=rng(1), device="cuda")
    far = torch.full((1,), 3e19, device="cuda")
    for at in (0, 290, 299, GRID - 1, GRID, GRID + 200, S - 1):
        buf[at * 8 + 7] = far  # in up to 130 rows around each
    x = buf.as_strided((S, H), (8, 1))
    one = torch.ones(H, device="cuda")
    _, _, q, d = M.norm_quant(x, one, 0.0)
    for p in (slice(0, 300), slice(GRID - 150, S)):
        v = x[p].double()
        v = v / torch.sqrt((v * v).mean(1, keepdim=True))
        step = v.abs().amax(1, keepdim=True) / 127
        assert ((d[p, None].double() - step).abs() <= 2.0 ** -19 * step).all()
        assert ((q[p].double() - v / step).abs() <= 0.5 + 127 * 2.0 ** -18).all()


def pieces(S, heads, units):
    """(tokens of a workgroup, workgroups) of the rotary kernel, from the rule in csrc/rope.hip for its widest units."""
    tokens = max(1, min(256 // (heads * units), S // 1024))
    return tokens, -(-S // tokens)


@pytest.mark.parametrize("S,heads,D,units,tokens", [(GRID + 5, 2, 130, 65, 1), (2 * GRID + 7, 2, 1024, 64, 2)])
@pytest.mark.parametrize("wide", [torch.int32, torch.int64])
def test_rope_in_several_launches(M, S, heads, D, units, tokens, wide):
    """The second launch goes on where the first ended, with its positions, inputs and outputs."""
    assert pieces(S, heads, units)[0] == tokens and pieces(S, heads, units)[1] > GRID
    g = rng(D)
    # rows that overlap, 16 elements apart
    x = torch.randn(S * 16 + heads * D, generator=g, device="cuda").bfloat16().as_strided((S, heads, D), (16, D, 1))
    pos = torch.randint(0, 5000, (S,), generator=g, device="cuda", dtype=wide)
    freqs, _ = M.rope_freqs(D)
    y, _ = M.rope(x, None, pos, freqs)
    cut = GRID * tokens
    for p in (slice(0, 3), slice(cut - 5, cut + 9), slice(S - 3, S)):
        check_rope(y[p], x[p], pos[p], freqs, 0, False, 1.0)
        assert torch.equal(y[p], M.rope(x[p], None, pos[p], freqs)[0])


@pytest.mark.parametrize("S,heads,kheads,D,rot,offset", [
    (2049, 1, 1, 36, 36, 0), (5003, 2, 1, 64, 32, 32), (16383, 1, 1, 20, 12, 3), (4097, 1, 0, 24, 16, 8),
    (3001, 3, 2, 32, 30, 2), (2051, 1, 1, 512, 512, 0), (20001, 1, 0, 2, 2, 0)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rope_of_several_tokens_a_workgroup(M, S, heads, kheads, D, rot, offset, inter, dtype):
    """Few elements a token: a workgroup takes several, the last one fewer."""
    g = rng(S + D)
    both = torch.randn(S, heads + kheads, D, generator=g, device="cuda").to(dtype)
    q, k = both[:, :heads], both[:, heads:] if kheads else None
    pos = torch.randint(0, 100000, (S,), generator=g, device="cuda")
    freqs, factor = M.rope_freqs(rot, 10000.0, "yarn", 4.0, 4096)
    qo, ko = M.rope(q, k, pos, freqs, offset=offset, interleaved=inter, factor=factor)
    check_rope(qo, q, pos, freqs, offset, inter, factor)
    if kheads:
        check_rope(ko, k, pos, freqs, offset, inter, factor)
    # the same bits one token a workgroup
    few, _ = M.rope(q[:700], None, pos[:700], freqs, offset=offset, interleaved=inter, factor=factor)
    assert torch.equal(qo[:700], few)


COPIES = [  # kernel, S, N, K, whether q and w lie on 16-byte boundaries
    ("few", 17, 40, 528, 0, 1), ("few", 40, 40, 272, 1, 0), ("few32", 200, 500, 272, 0, 1), ("few32", 200, 500, 272, 1, 0),
    ("tile32", 17, 6200, 4112, 0, 1), ("tile32", 700, 300, 4112, 1, 0), ("tile32", 500, 500, 4112, 0, 0),
    ("tile32x64", 130, 2100, 2064, 0, 1), ("tile32x64", 500, 900, 1552, 1, 0), ("tile32x64", 1540, 300, 1552, 0, 0),
    ("tile64", 130, 4100, 1040, 0, 1), ("tile64", 500, 1500, 1040, 1, 0), ("tile64", 1540, 500, 1040, 0, 0),
    ("tile64x128", 1030, 1500, 1552, 0, 1), ("tile64x128", 1030, 1500, 1552, 1, 0), ("tile64x128", 200, 6200, 1552, 0, 0),
    ("tile128", 500, 6200, 528, 0, 1), ("tile128", 1030, 3000, 528, 1, 0), ("tile128", 2050, 1500, 528, 0, 0),
    ("tile128x2", 2050, 3000, 272, 0, 1), ("tile128x2", 3000, 2100, 272, 1, 0), ("tile128x2", 700, 8200, 272, 0, 0),
    ("tile256", 2050, 6200, 1040, 0, 1), ("tile256", 3000, 4100, 1040, 1, 0), ("tile256", 3000, 4100, 1040, 0, 0),
]


@pytest.mark.parametrize("kernel,S,N,K,q16,w16", COPIES)
def test_product_copies_the_operand_that_needs_it(M, kernel, S, N, K, q16, w16):
    """Tokens, weights or both away from 16-byte boundaries: the tile kernels run behind a copy of just those."""
    g = rng(S + N + K)
    q, d, _, _ = operands(g, S, 1, K, *((0, 0) if q16 else (5, 3)))
    _, _, w, dw = operands(g, 1, N, K, *((0, 0) if w16 else (7, 1)))
    rows = (0 if q16 else S) + (0 if w16 else N)
    need = M.moe_qmatmul_workspace_bytes(q, q.stride(0), w, w.stride(0), S, N, K)
    assert need == (rows * K if kernel.startswith("tile") else 0)
    ws = torch.full((need + 64,), 99, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    M.moe_profile_enable(True)
    try:
        y = M.qmatmul(q, d, w, dw, out_dtype=F32, ws=ws[:need] if need else None)
        ran = set(M.moe_profile_report())
    finally:
        M.moe_profile_enable(False)
    assert ran == {"qmatmul_" + kernel} | ({"qmatmul_align"} if need else set())
    assert (ws[need:] == 99).all()
    want = (q.double() @ w.double().t().contiguous()).round().float() * (d[:, None] * dw)  # exact sums under 2^53
    assert torch.equal(y, want)


def test_the_layers_int8_activations(M):
    """moe_ffn with act_int8 and int8 weights, next to the same experts put together from the dense operators: it
    quantises the norm's fp32 rows to the norm's own int8 rows.  All sums of integers are exact; the scales' products may
    be rounded in another order, which moves an element of h that lies on a rounding border by one step (a few 1e-3 of
    the output at most: the bars of the layer's own int8 tests, 5e-3 at most and 1e-5 for the median token)."""
    from gen import inputs as gen
    from tests.devlayer import DeviceLayer
    w = gen.WORKLOADS["tiny"]
    w = w.with_(cfg=gen.LayerConfig(**{**w.cfg.__dict__, "weight_format": 2}))
    dl = DeviceLayer(w, host_experts=True, mfma_min_tokens=0, act_int8=1)
    c, S = dl.c, 37
    x0 = torch.randn(S, c.hidden, generator=rng(3), device="cuda") * 3
    _, x, q, d = M.norm_quant(x0, 1 + 0.2 * torch.rand(c.hidden, generator=rng(4), device="cuda"), 1e-5, y_dtype=F32)
    idx, wt = dl.route(x, M.MOE_F32)
    got = dl.ffn(x, M.MOE_F32, idx, wt)

    def expert(e):
        i8 = lambda a: torch.from_numpy(np.ascontiguousarray(a).view(np.int8)).cuda()  # noqa: E731
        h = dl.host_expert(e)
        qg, sg, qu, su, qd, sd = h.parts()
        gate, up = (M.qmatmul(q, d, i8(a).view(h.inter, c.hidden), torch.from_numpy(b).cuda().float().view(-1), out_dtype=F32)
                    for a, b in ((qg, sg), (qu, su)))
        _, hq, hd = M.silu_quant(gate, up)
        return M.qmatmul(hq, hd, i8(qd).view(c.hidden, h.inter), torch.from_numpy(sd).cuda().float().view(-1), out_dtype=F32)
    want = expert(c.n_experts).double() if c.shared_inter > 0 else torch.zeros(S, c.hidden, dtype=torch.float64, device="cuda")
    for e in range(c.n_experts):
        share = (wt * (idx == e)).sum(1)
        if share.any():
            want += share[:, None].double() * expert(e).double()
    errs = (got.double() - want).abs().amax(1) / want.abs().amax(1)
    assert errs.max() <= 5e-3 and errs.median() <= 1e-5
