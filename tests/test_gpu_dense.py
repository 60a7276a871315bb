"""Dense operators on the GPU against plain forms in 64 bits.

Tolerances, derived before the first run, in units of U = 2^-24 (half a step of fp32 at most, relative); a result stored
in bf16 may be off by 2^-8 more.
  norm   a sum of squares is added up by threads of at most 32 elements (or every 256th) and a tree: at most
         max(32, H / 256) + 16 roundings, halved by the square root; then the mean, eps, root, reciprocal and the two
         products: relative error (max(32, H / 256) / 2 + 14) U.
  SwiGLU exp within 4 U; 1 + exp, the reciprocal (2 U) or division and two products: 10 U, plus values under 1e-35
         that may vanish.
  codes  |q - v / d| <= 1/2 + 127 times twice the value's relative error (v and d both carry it); and the fp32 output
         of the same call determines them exactly: d = max|y| / 127, q = y / d rounded.
  product exact sums: the result is the formula's fp32 value, bit for bit.
  rope   the reduced angle is within 2^-25, sine and cosine within 2 U of it, times factor; two products and their sum:
         (|x1| + |x2|) factor 7 U.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def M():
    from int4_routed_expert_amd import moe
    return moe


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows(g, S, H, dtype, pad=0, start=0):
    """[S, H] of N(0, 1) with some wide channels, its rows pad elements apart and `start` elements into its buffer."""
    wide = 1 + 30.0 * (torch.rand(H, generator=g, device="cuda") < 0.01)
    buf = torch.zeros(start + S * (H + pad), dtype=dtype, device="cuda")
    x = buf[start:].view(S, H + pad)[:, :H]
    x.copy_(torch.randn(S, H, generator=g, device="cuda") * wide)
    return x


def close(got, want, rel, floor=0.0):
    rel = rel + (2.0 ** -8 if got.dtype == BF else 0)
    got, want = got.double(), want.double()
    bad = (got - want).abs() > rel * want.abs() + floor
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, first {got[bad][:4].tolist()} for {want[bad][:4].tolist()}"


def check_codes(q, d, v, rel):
    """int8 rows q, d against 64-bit values v known to a relative error of rel."""
    d64 = v.abs().amax(1) / 127
    close(d, d64, rel + U, floor=1e-37)
    ratio = torch.where(d64[:, None] > 0, v / d64[:, None].clamp_min(1e-300), 0.0)
    assert (q.double() - ratio).abs().max() <= 0.5 + 127 * 2 * (rel + U)
    assert int(q.min()) >= -127


def check_own_codes(q, d, y):
    """int8 rows of a call against its own fp32 output."""
    y = y.cpu()
    step = y.abs().amax(1) / torch.tensor(127.0)
    assert torch.equal(d.cpu(), step)
    usable = (step > 0) & torch.isfinite(step)
    want = torch.where(usable[:, None], torch.round(y / step[:, None]), torch.zeros(())).clamp(-127, 127)
    assert torch.equal(q.cpu().float(), want)


def norm64(x, res, gamma, eps):
    h = x.double() if res is None else (x.float() + res.float()).to(x.dtype).double()
    return h, h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * gamma.double()


NORM = [  # S, H, dtype, residual, pad, start
    (1, 1, F32, True, 0, 0), (1, 7, BF, False, 0, 0), (3, 64, BF, True, 0, 0), (5, 65, F32, True, 3, 1),
    (2, 511, BF, True, 1, 1), (4, 512, BF, True, 0, 0), (1, 513, F32, False, 0, 0), (700, 1000, BF, True, 8, 0),
    (9, 1536, F32, True, 0, 0), (6, 2047, F32, False, 3, 0), (700, 2048, F32, True, 0, 0), (700, 2049, BF, True, 7, 0),
    (1, 6144, BF, True, 0, 0), (2, 6144, F32, True, 0, 2), (600, 6144, BF, True, 0, 0), (600, 4104, F32, True, 0, 0),
    (3, 8192, BF, True, 0, 0), (600, 8192, F32, False, 0, 0), (3, 8200, F32, True, 0, 0), (5, 16384, BF, True, 0, 0),
    (300, 12296, BF, True, 8, 0), (2, 32768, F32, True, 0, 0), (2, 32769, BF, True, 0, 0), (2, 50001, F32, True, 1, 0),
]


@pytest.mark.parametrize("S,H,dtype,res,pad,start", NORM)
def test_norm(M, S, H, dtype, res, pad, start):
    g = rng(S * 131 + H)
    x = rows(g, S, H, dtype, pad, start)
    r = rows(g, S, H, dtype) if res else None
    rel = (max(32, H / 256) / 2 + 14) * U
    for gd in (F32, BF):
        gamma = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(gd)
        h64, v64 = norm64(x, r, gamma, 1e-5)
        for yd in (F32, BF, None):
            h, y, q, d = M.norm_quant(x, gamma, 1e-5, residual=r, y_dtype=yd)
            if res:
                assert torch.equal(h.double(), h64)
            else:
                assert h is None
            if yd is None:
                assert y is None
            else:
                close(y, v64, rel)
            check_codes(q, d, v64, rel)
            if yd == F32:
                check_own_codes(q, d, y)
        h, y, q, d = M.norm_quant(x, gamma, 1e-5, residual=r, y_dtype=BF, quant=False)
        assert q is None and d is None
        close(y, v64, rel)
        if res:
            assert torch.equal(h.double(), h64)


@pytest.mark.parametrize("H", [100, 6144, 20000, 40000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_in_place(M, H, dtype):
    """The sum over the residual, and the norm over x, give what separate outputs give."""
    g = rng(H)
    x, r = rows(g, 5, H, dtype), rows(g, 5, H, dtype)
    gamma = torch.rand(H, generator=g, device="cuda")
    h, y, q, d = M.norm_quant(x, gamma, 1e-6, residual=r, y_dtype=dtype)
    r2 = r.clone()
    h2, y2, q2, d2 = M.norm_quant(x, gamma, 1e-6, residual=r2, h=r2, y_dtype=dtype)
    assert h2 is r2
    for a, b in ((h, h2), (y, y2), (q, q2), (d, d2)):
        assert torch.equal(a, b)
    x2, code = x.clone(), M._code(dtype, "x")
    M.moe_norm_quant(x2, code, H, r, H, gamma, M.MOE_F32, 1e-6, 5, H, None, 0, x2, code, H, q2, H, d2)
    assert torch.equal(x2, y) and torch.equal(q2, q) and torch.equal(d2, d)
    x3 = x.clone()
    M.moe_norm_quant(x3, code, H, r, H, gamma, M.MOE_F32, 1e-6, 5, H, x3, H, y2, code, H, q2, H, d2)
    assert torch.equal(x3, h) and torch.equal(y2, y) and torch.equal(q2, q)


SPECIAL = [float("nan"), float("inf"), float("-inf")]


@pytest.mark.parametrize("H", [33, 6144, 40000])
@pytest.mark.parametrize("S", [6, 1200])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_special_rows(M, S, H, dtype):
    """Rows of zeros, and rows holding an infinity or a NaN, keep to themselves."""
    if S * H > 10 ** 7:
        S = 60
    g = rng(H + S)
    x = rows(g, S, H, dtype)
    x[1] = 0
    for i, v in enumerate(SPECIAL):
        x[2 + i, H // 2 + i] = v
    gamma = torch.ones(H, device="cuda")
    _, y, q, d = M.norm_quant(x, gamma, 1e-5, y_dtype=F32)
    assert (y[1] == 0).all() and (q[1] == 0).all() and d[1] == 0
    for i in range(3):
        assert not torch.isfinite(y[2 + i]).all() and (q[2 + i] == 0).all() and not torch.isfinite(d[2 + i])
    rest = [0] + list(range(5, S))
    assert torch.isfinite(y[rest]).all()
    check_own_codes(q[rest], d[rest], y[rest])
    if H % 2 == 0:
        y, q, d = M.silu_quant(x, y_dtype=F32)
        assert (y[1] == 0).all() and (q[1] == 0).all() and d[1] == 0
        for i in range(3):
            assert (q[2 + i] == 0).all() and (not torch.isfinite(d[2 + i]) or torch.isfinite(y[2 + i]).all())
        check_own_codes(q[rest], d[rest], y[rest])


@pytest.mark.parametrize("scale", [1e-45, 3e-43, 1e-40, 1e-37, 1e-31, 1e-29, 1.0, 1e29, 1e31, 1e37])
def test_codes_at_extreme_scales(M, scale):
    """Values from denormals to beyond the largest (whose rows have d = inf) keep to the rule."""
    g = torch.full((4, 1000), 30.0, device="cuda")
    u = torch.randn(4, 1000, generator=rng(3), device="cuda") * scale
    y, q, d = M.silu_quant(g, u, y_dtype=F32)
    check_own_codes(q, d, y)


def test_scale_is_ieee_division(M):
    """Ties and near-ties of v / d over many scales round as IEEE division and rint do."""
    g = rng(9)
    u = torch.randint(-254, 255, (3000, 512), generator=g, device="cuda").float() / 2
    u[:, 0] = 127.0
    u *= torch.exp2(torch.rand(3000, 1, generator=g, device="cuda") * 20 - 10)
    y, q, d = M.silu_quant(torch.full_like(u, 40.0), u, y_dtype=F32)
    check_own_codes(q, d, y)


SILU = [(1, 1, F32, 0), (3, 63, BF, 1), (4, 64, BF, 0), (4, 2048, F32, 0), (700, 500, BF, 4), (5, 513, F32, 3),
        (600, 2048, BF, 0), (600, 2056, F32, 0), (3, 6144, BF, 0), (600, 6152, BF, 8), (3, 12288, BF, 0),
        (300, 12288, F32, 0), (2, 32768, BF, 0), (2, 33000, F32, 0), (3, 40001, BF, 1)]


@pytest.mark.parametrize("S,I,dtype,pad", SILU)
def test_silu(M, S, I, dtype, pad):
    g = rng(S + I)
    gu = rows(g, S, 2 * I, dtype, pad)
    gu[:, :I] *= torch.rand(S, I, generator=g, device="cuda").to(dtype) * 4
    a, u = gu[:, :I].double(), gu[:, I:].double()
    v64 = a / (1 + torch.exp(-a)) * u
    for yd in (F32, BF, None):
        y, q, d = M.silu_quant(gu, y_dtype=yd)
        if yd is None:
            assert y is None
        else:
            close(y, v64, 10 * U, floor=1e-33)
        check_codes(q, d, v64, 10 * U)
        if yd == F32:
            check_own_codes(q, d, y)
    y2, q2, d2 = M.silu_quant(gu[:, :I], gu[:, I:], y_dtype=F32)
    y, q, d = M.silu_quant(gu, y_dtype=F32)
    assert torch.equal(y2, y) and torch.equal(q2, q) and torch.equal(d2, d)
    y3, q3, d3 = M.silu_quant(gu, y_dtype=F32, quant=False)
    assert torch.equal(y3, y) and q3 is None and d3 is None


def test_silu_gate_range(M):
    """Gates from far below to far above the range of exp, and infinities."""
    g = torch.cat((torch.linspace(-120, 120, 4001), torch.tensor([-1e30, 1e30, float("inf"), -0.0, 0.0]))).cuda()
    u = torch.ones_like(g)
    y, _, _ = M.silu_quant(g[None], u[None], y_dtype=F32, quant=False)
    a = g.double()
    close(y[0], a / (1 + torch.exp(-a)), 10 * U, floor=1e-33)


def product64(q, d, w, dw, dtype):
    """The formula in fp32 from exact sums (on the CPU, where every step is IEEE)."""
    q, d, w, dw = (v.cpu() for v in (q, d, w, dw))
    sums = (q.double() @ w.double().t()).round()  # integers under 2^53: exact
    return (sums.float() * (d[:, None] * dw)).to(dtype)


def operands(g, S, N, K, pad=0, start=0):
    def mat(R):
        buf = torch.zeros(start + R * (K + pad), dtype=torch.int8, device="cuda")
        m = buf[start:].view(R, K + pad)[:, :K]
        m.copy_(torch.randint(-128, 128, (R, K), generator=g, device="cuda", dtype=torch.int8))
        return m
    q, w = mat(S), mat(N)
    d = 0.01 + torch.rand(S, generator=g, device="cuda")
    dw = torch.randn(N, generator=g, device="cuda")
    return q, d, w, dw


PRODUCT = [  # S, N, K, pad, start
    (1, 1, 1, 0, 0), (1, 17, 5, 0, 0), (2, 64, 64, 0, 0), (1, 4096, 6144, 0, 0), (1, 33, 8192, 0, 0), (1, 100, 1111, 1, 1),
    (3, 576, 6144, 0, 0), (4, 6144, 2048, 0, 0), (5, 257, 1000, 24, 0), (8, 96, 16384, 0, 0), (15, 16, 130, 0, 0),
    (16, 2048, 512, 0, 0), (17, 2048, 512, 0, 0), (31, 100, 300, 3, 5), (32, 1000, 4096, 0, 0), (33, 65, 4112, 0, 16),
    (48, 576, 2048, 0, 0), (64, 64, 64, 0, 0), (65, 4096, 1024, 0, 0), (77, 577, 1111, 0, 0), (100, 1200, 128, 16, 0),
    (128, 128, 128, 0, 0), (129, 255, 127, 1, 0), (200, 3000, 1008, 0, 0), (256, 1024, 2048, 0, 0), (257, 513, 2064, 0, 0),
    (300, 257, 80, 0, 0), (511, 512, 192, 0, 0), (512, 2048, 256, 0, 0), (1000, 1000, 1000, 0, 0), (1024, 4096, 512, 0, 0),
    (2049, 2100, 320, 16, 16), (4096, 512, 144, 0, 0), (1, 7, 131071, 0, 0), (70, 9, 131071, 0, 0),
]


@pytest.mark.parametrize("S,N,K,pad,start", PRODUCT)
def test_product(M, S, N, K, pad, start):
    g = rng(S * 7 + N * 3 + K)
    q, d, w, dw = operands(g, S, N, K, pad, start)
    for dtype in (F32, BF):
        y = M.qmatmul(q, d, w, dw, out_dtype=dtype)
        assert torch.equal(y.cpu(), product64(q, d, w, dw, dtype))


@pytest.mark.parametrize("S,N,K,kernel", [
    (1, 500, 300, "vec"), (3, 20000, 64, "vec"), (6, 576, 6144, "vec"), (8, 1000, 2064, "vec"), (5, 1024, 9008, "vec"),
    (2, 900, 8208, "vec"), (4, 700, 16400, "vec"), (1, 600, 8256, "vec"), (2, 2500, 1040, "vec"), (8, 1000, 2049, "vec"), (4, 4000, 1040, "vec"), (9, 300, 1030, "few"), (64, 700, 512, "few"),
    (130, 700, 272, "few32"), (17, 4100, 272, "few32"), (17, 4096, 4112, "tile32"), (130, 1024, 2064, "tile32"),
    (30, 700, 16400, "tile32"), (260, 1024, 528, "tile32x64"), (1540, 300, 272, "tile32x64"),
    (770, 1024, 272, "tile64"), (48, 8208, 528, "tile64"), (200, 6160, 2064, "tile64x128"), (770, 4096, 272, "tile128"),
    (200, 12304, 272, "tile128"), (1540, 4096, 272, "tile128x2"), (2050, 6160, 1040, "tile256"), (1030, 12300, 1056, "tile256")])
def test_every_product_kernel(M, S, N, K, kernel):
    """Each kernel runs where its estimate is least; results exact, on 16-byte boundaries and at other places."""
    g = rng(S + N)
    for pad, start in ((0, 0), (5, 3)):
        q, d, w, dw = operands(g, S, N, K, pad, start)
        torch.cuda.synchronize()
        M.moe_profile_enable(True)
        try:
            y = M.qmatmul(q, d, w, dw, out_dtype=F32)
            ran = M.moe_profile_report()
        finally:
            M.moe_profile_enable(False)
        if pad == 0 and K % 16 == 0:
            assert set(ran) - {"qmatmul_align"} == {"qmatmul_" + kernel}
        want = ((q.double() @ w.double().t().contiguous()).round().float() * (d[:, None] * dw))  # exact sums under 2^53
        assert torch.equal(y, want)


@pytest.mark.parametrize("S", [1, 20, 300])
def test_product_extreme_sum(M, S):
    """All -128: the largest sum that int32 has to hold."""
    K = 131071
    q = torch.full((S, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((20, K), -128, dtype=torch.int8, device="cuda")
    w[3] = 127
    one = torch.ones(max(S, 20), device="cuda")
    y = M.qmatmul(q, one[:S], w, one[:20], out_dtype=F32)
    want = torch.full((S, 20), float(16384 * K), device="cuda")
    want[:, 3] = -128.0 * 127 * K
    assert torch.equal(y, want)


@pytest.mark.parametrize("S", [2, 40, 400])
def test_product_special_scales(M, S):
    """A NaN or infinite scale poisons its own row or column; one token's result does not depend on the others."""
    g = rng(S)
    q, d, w, dw = operands(g, S, 300, 256)
    clean = M.qmatmul(q, d, w, dw, out_dtype=F32)
    d2, dw2 = d.clone(), dw.clone()
    d2[1], dw2[7] = float("nan"), float("inf")
    y = M.qmatmul(q, d2, w, dw2, out_dtype=F32)
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[:, 7]).any()
    keep = [c for c in range(300) if c != 7]
    assert torch.equal(y[0, keep], clean[0, keep]) and torch.equal(y[2:][:, keep], clean[2:][:, keep])
    assert torch.equal(M.qmatmul(q[1:2], d[1:2], w, dw, out_dtype=F32)[0], clean[1])


def test_product_into_wider_rows(M):
    """Output rows further apart than N leave what lies between them alone."""
    g = rng(4)
    for S, N, K in ((3, 100, 256), (150, 1001, 272)):
        q, d, w, dw = operands(g, S, N, K)
        for dtype in (F32, BF):
            y = torch.full((S, N + 9), 5.0, dtype=dtype, device="cuda")
            ws = torch.empty(max(16, M.moe_qmatmul_workspace_bytes(q, K, w, K, S, N, K)), dtype=torch.uint8, device="cuda")
            M.moe_qmatmul(q, K, d, w, K, dw, S, N, K, y, M._code(dtype, "y"), N + 9, ws, ws.numel())
            assert torch.equal(y[:, :N].cpu(), product64(q, d, w, dw, dtype)) and (y[:, N:] == 5).all()


ROPE = [  # S, heads, kheads, D, rot, offset
    (1, 1, 0, 2, 2, 0), (1, 64, 1, 64, 64, 0), (8, 64, 8, 128, 128, 0), (3, 5, 2, 20, 12, 3), (7, 24, 3, 192, 64, 128),
    (33, 3, 1, 80, 32, 0), (130, 1, 1, 64, 64, 0), (130, 1, 0, 64, 16, 48), (9, 2, 2, 1024, 1024, 0), (5, 9, 4, 96, 48, 24),
    (300, 16, 4, 128, 128, 0), (50, 7, 3, 72, 40, 4), (50, 6, 2, 68, 68, 0), (21, 3, 1, 44, 20, 24), (4, 1000, 1, 64, 32, 32), (1000, 2, 1, 36, 36, 0), (1500, 1, 1, 256, 64, 64),
]


def rope64(x, pos, freqs, offset, inter, factor):
    x = x.double()
    a = pos.double()[:, None, None] * freqs
    c, s, n = a.cos() * factor, a.sin() * factor, freqs.numel()
    y, size = x.clone(), torch.zeros_like(x)
    i1 = offset + (2 * torch.arange(n) if inter else torch.arange(n))
    i2 = i1 + (1 if inter else n)
    x1, x2 = x[..., i1], x[..., i2]
    y[..., i1], y[..., i2] = x1 * c - x2 * s, x2 * c + x1 * s
    size[..., i1] = size[..., i2] = (x1.abs() + x2.abs()) * factor
    return y, size


def check_rope(got, x, pos, freqs, offset, inter, factor):
    y, size = rope64(x, pos, freqs, offset, inter, factor)
    tol = 7 * U * size + (2.0 ** -8 * y.abs() if got.dtype == BF else 0)
    outside = size == 0
    assert torch.equal(got.double()[outside], y[outside])
    bad = (got.double() - y).abs() > tol
    assert not bad.any(), f"{int(bad.sum())}: {got[bad][:4].tolist()} for {y[bad][:4].tolist()}"


@pytest.mark.parametrize("S,heads,kheads,D,rot,offset", ROPE)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rope(M, S, heads, kheads, D, rot, offset, inter, dtype):
    g = rng(S + heads * 3 + D)
    for wide, far, pad in ((torch.int64, 1 << 20, 0), (torch.int32, 4096, 5)):
        # queries and keys cut out of one projection's rows
        both = torch.randn(S, heads + kheads, D + pad, generator=g, device="cuda").to(dtype)[..., :D]
        q, k = both[:, :heads], both[:, heads:] if kheads else None
        pos = torch.randint(-far // 8, far, (S,), generator=g, device="cuda", dtype=wide)
        pos[0] = 0
        freqs, factor = M.rope_freqs(rot, 10000.0, "linear" if pad else "none", 2.0 if pad else 1.0)
        factor = 1.25 if pad else 1.0
        qo, ko = M.rope(q, k, pos, freqs, offset=offset, interleaved=inter, factor=factor)
        check_rope(qo, q, pos, freqs, offset, inter, factor)
        assert (ko is None) == (k is None)
        if k is not None:
            check_rope(ko, k, pos, freqs, offset, inter, factor)
        if factor == 1.0:  # position 0 turns by nothing
            assert torch.equal(qo[0], q[0])
        buf = both.clone()
        q2, k2 = M.rope(buf[:, :heads], buf[:, heads:] if kheads else None, pos, freqs, offset=offset, interleaved=inter,
                        factor=factor, inplace=True)
        assert q2.data_ptr() == buf.data_ptr() and torch.equal(q2, qo) and (k is None or torch.equal(k2, ko))


def test_rope_head_major_and_shared_rows(M):
    """[heads, S, D] storage, and one key row that every token shares (stride 0)."""
    g = rng(2)
    q = torch.randn(12, 50, 64, generator=g, device="cuda").transpose(0, 1)
    k = torch.randn(1, 1, 64, generator=g, device="cuda").expand(50, 1, 64)
    pos = torch.arange(50, device="cuda")
    freqs, _ = M.rope_freqs(64)
    qo, ko = M.rope(q, k, pos, freqs)
    check_rope(qo, q, pos, freqs, 0, False, 1.0)
    check_rope(ko, k, pos, freqs, 0, False, 1.0)


def test_rope_far_positions(M):
    """Positions up to 2^40 keep their angles (fp64 products and reduction: 2^-12 of a turn lost at most there)."""
    pos = torch.tensor([0, 1, 2 ** 20 + 1, 2 ** 31 + 5, 2 ** 40 + 3], device="cuda")
    x = torch.randn(5, 4, 64, generator=rng(1), device="cuda")
    freqs, _ = M.rope_freqs(64)
    y, _ = M.rope(x, None, pos, freqs)
    want, size = rope64(x, pos, freqs, 0, False, 1.0)
    tol = size * (7 * U + pos.double()[:, None, None] * 2.0 ** -51)
    assert ((y.double() - want).abs() <= tol).all()


def test_no_rows(M):
    e = torch.empty
    h, y, q, d = M.norm_quant(e(0, 64, device="cuda"), e(64, device="cuda"), 1e-5, residual=e(0, 64, device="cuda"), y_dtype=F32)
    assert h.shape == y.shape == q.shape == (0, 64) and d.shape == (0,)
    y, q, d = M.silu_quant(e(0, 64, device="cuda"), y_dtype=BF)
    assert y.shape == q.shape == (0, 32) and d.shape == (0,)
    assert M.qmatmul(q, d, e(8, 32, dtype=torch.int8, device="cuda"), e(8, device="cuda")).shape == (0, 8)
    q, k = M.rope(e(0, 4, 64, device="cuda"), e(0, 1, 64, device="cuda"), e(0, dtype=torch.int64, device="cuda"), M.rope_freqs(64)[0])
    assert q.shape == (0, 4, 64) and k.shape == (0, 1, 64)


def test_offsets_beyond_32_bits(M):
    """Rows whose offsets pass 2^32 elements, in inputs and outputs."""
    far = (1 << 32) // 2 + 16
    buf = torch.empty(2 * far + 4096, dtype=torch.int8, device="cuda")
    g = rng(7)
    q, d, w, dw = operands(g, 3, 40, 512)
    qf = buf.as_strided((3, 512), (far, 1))
    qf.copy_(q)
    assert torch.equal(M.qmatmul(qf, d, w, dw, out_dtype=F32), M.qmatmul(q, d, w, dw, out_dtype=F32))
    wf = buf.as_strided((3, 512), (far, 1), 1024)
    wf.copy_(w[:3])
    assert torch.equal(M.qmatmul(q, d, wf, dw[:3], out_dtype=F32), M.qmatmul(q, d, w[:3].contiguous(), dw[:3], out_dtype=F32))
    yf = buf.view(BF).as_strided((3, 40), (far // 2, 1), 1024)  # 2^31 elements and their bytes beyond 2^32
    ws = torch.empty(max(16, M.moe_qmatmul_workspace_bytes(q, 512, w, 512, 3, 40, 512)), dtype=torch.uint8, device="cuda")
    M.moe_qmatmul(q, 512, d, w, 512, dw, 3, 40, 512, yf, M.MOE_BF16, far // 2, ws, ws.numel())
    assert torch.equal(yf, M.qmatmul(q, d, w, dw))
    x = rows(g, 3, 1024, BF)
    xf = buf.view(BF).as_strided((3, 1024), (far // 2, 1))
    xf.copy_(x)
    gamma = torch.rand(1024, generator=g, device="cuda")
    want = M.norm_quant(x, gamma, 1e-5, y_dtype=BF)
    got = M.norm_quant(xf, gamma, 1e-5, y_dtype=BF)
    assert all(torch.equal(a, b) for a, b in zip(want[1:], got[1:]))
    assert all(torch.equal(a, b) for a, b in zip(M.silu_quant(x)[1:], M.silu_quant(xf)[1:]))
    pos = torch.tensor([5, 6, 7], device="cuda")
    freqs, _ = M.rope_freqs(64)
    heads = buf.view(BF).as_strided((3, 16, 64), (far // 2, 64, 1))
    assert torch.equal(M.rope(heads, None, pos, freqs)[0], M.rope(x.view(3, 16, 64), None, pos, freqs)[0])


def chain(M, x, r, gamma, w1, dw1, w2, dw2, pos, freqs, stream=None):
    h, y, q, d = M.norm_quant(x, gamma, 1e-5, residual=r, y_dtype=BF, stream=stream)
    gu = M.qmatmul(q, d, w1, dw1, stream=stream)
    _, q2, d2 = M.silu_quant(gu, stream=stream)
    out = M.qmatmul(q2, d2, w2, dw2, stream=stream)
    turned, _ = M.rope(out.view(out.shape[0], -1, 64), None, pos, freqs, stream=stream)
    return h, y, q, d, gu, q2, d2, out, turned


def chain_inputs(M, S, seed):
    g = rng(seed)
    H, I = 512, 384
    _, _, w1, dw1 = operands(g, 1, 2 * I, H)
    _, _, w2, dw2 = operands(g, 1, H, I)
    return [rows(g, S, H, BF), rows(g, S, H, BF), torch.rand(H, generator=g, device="cuda"), w1, dw1 * 1e-3, w2, dw2 * 1e-3,
            torch.randint(0, 9999, (S,), generator=g, device="cuda"), M.rope_freqs(64)[0]]


@pytest.mark.parametrize("S", [1, 4, 30, 700])
def test_streams(M, S):
    """On a stream of their own the calls give the same bits, and their memory is not reused under them."""
    args = chain_inputs(M, S, S)
    want = chain(M, *args)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for _ in range(5):
        fresh = [a.clone() for a in args]
        st.wait_stream(torch.cuda.current_stream())
        got = chain(M, *fresh, stream=st)
        del fresh
        junk = [torch.full_like(a, 1) for a in args]  # would take the inputs' memory if it were free
        st.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
        del got, junk


@pytest.mark.parametrize("S", [1, 4, 30, 700])
def test_graph_replays(M, S):
    """Captured once, replayed with new inputs between eager work: every replay equals the eager result."""
    static = chain_inputs(M, S, 50 + S)
    chain(M, *static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = chain(M, *static)
    for k in range(4):
        new = chain_inputs(M, S, 100 + k)
        want = chain(M, *new)
        for a, b in zip(static, new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert torch.equal(a, b)


@pytest.mark.parametrize("H", [500, 1000, 2048, 4104, 6144, 8192, 12288, 16384, 20000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_do_not_depend_on_the_batch(M, H, dtype):
    """A row's bits are the same alone, in a small batch and in a large one."""
    g = rng(H)
    x, r = rows(g, 1030, H, dtype), rows(g, 1030, H, dtype)
    gamma = torch.rand(H, generator=g, device="cuda")
    many = M.norm_quant(x, gamma, 1e-5, residual=r, y_dtype=BF) + M.silu_quant(x, r, y_dtype=BF)
    for lo, hi in ((0, 1), (7, 8), (100, 109), (1000, 1030)):
        few = M.norm_quant(x[lo:hi], gamma, 1e-5, residual=r[lo:hi], y_dtype=BF) + M.silu_quant(x[lo:hi], r[lo:hi], y_dtype=BF)
        for a, b in zip(many, few):
            assert torch.equal(a[lo:hi], b)


@pytest.mark.parametrize("H", [77, 1000, 6144])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_do_not_depend_on_where_they_lie(M, H, dtype):
    """The same rows at other offsets and distances give the same bits."""
    x = rows(rng(H), 9, H, dtype)
    gamma = torch.rand(H, device="cuda", generator=rng(1))
    want = M.norm_quant(x, gamma, 1e-5, residual=x, y_dtype=dtype) + M.silu_quant(x, x, y_dtype=dtype)
    for pad, start in ((1, 0), (0, 1), (3, 5), (8, 2), (16, 8)):
        buf = torch.full((start + 9 * (H + pad),), float("nan"), dtype=dtype, device="cuda")
        z = buf[start:].view(9, H + pad)[:, :H]
        z.copy_(x)
        got = M.norm_quant(z, gamma, 1e-5, residual=z, y_dtype=dtype) + M.silu_quant(z, z, y_dtype=dtype)
        for a, b in zip(want, got):
            assert torch.equal(a, b)


def test_same_rule_as_the_layers_int8_activations(M):
    """The norm's int8 rows are what moe_cfg.act_int8 makes of the same fp32 rows: d = max|v| / 127, q = rint(v / d)."""
    x = rows(rng(1), 50, 1024, F32)
    _, y, q, d = M.norm_quant(x, torch.ones(1024, device="cuda"), 1e-5, y_dtype=F32)
    check_own_codes(q, d, y)


def test_profile_names(M):
    M.moe_profile_enable(True)
    try:
        args = chain_inputs(M, 4, 1)
        chain(M, *args)
        seen = M.moe_profile_report()
    finally:
        M.moe_profile_enable(False)
    assert {"norm_quant", "silu_quant", "rope"} <= set(seen) and any(n.startswith("qmatmul") for n in seen)


@pytest.mark.parametrize("S", [1, 5, 130])
def test_example_layer(M, S):
    """The example's dense layer and MoE layer against float64.  An int8 row's values are off by at most half a step each,
    uniformly: d / sqrt(12) = max|v| / 440 on average, at most 5 / 440 of a row's root mean square for its maxima here
    (rows of 256 to 768), so 1.2% for each of three products, and weights are exact; bf16 adds 0.2% in eight places.
    Each reaches the residual stream once and does not grow on the way: under 5% together."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import dense_layer as E
    layer = E.Layer()
    h, x, pos = E.inputs(layer, S)
    want_h, want_y = E.reference(layer, h, x, pos)
    before = h.clone()
    got_h, got_y, moe = layer.forward(h, x, pos)
    assert got_h is h and not torch.equal(h, before)
    for got, want in ((got_h, want_h), (got_y, want_y)):
        assert (got.double() - want).norm() <= 0.05 * want.norm()
    assert moe.shape == (S, layer.c.hidden) and torch.isfinite(moe).all()


def test_more_rows_than_one_launch(M):
    """Numbers of rows, weights and tokens beyond what one launch or one pass of its workgroups takes."""
    g = rng(5)
    for S, H in (((1 << 22) + 9, 8), ((1 << 20) + 5, 520)):  # four rows and one row a workgroup
        x = torch.randn(S, H, generator=g, device="cuda").bfloat16()
        gamma = torch.rand(H, generator=g, device="cuda")
        _, y, q, d = M.norm_quant(x, gamma, 1e-5, y_dtype=BF)
        at = torch.tensor([0, 1, S // 2, (1 << 20) - 1, 1 << 20, (1 << 20) + 1, S - 2, S - 1], device="cuda")
        want = M.norm_quant(x[at], gamma, 1e-5, y_dtype=BF)
        assert all(torch.equal(a[at], b) for a, b in zip((y, q, d), want[1:]))
        z, zq, zd = M.silu_quant(x, x, y_dtype=BF)
        assert all(torch.equal(a[at], b) for a, b in zip((z, zq, zd), M.silu_quant(x[at], x[at], y_dtype=BF)))
        del x, y, q, z, zq
    many = (1 << 18) + 7
    for S, N, K in ((many, 5, 16), (3, many, 16), (many, 3, 13), (70, many, 33)):
        q, d, w, dw = operands(g, S, N, K)
        y = M.qmatmul(q, d, w, dw, out_dtype=F32)
        want = (q.double() @ w.double().t().contiguous()).round().float() * (d[:, None] * dw)
        assert torch.equal(y, want)
        del y, want
    S = (1 << 20) + 3
    x = torch.randn(1, 2, 1024, generator=g, device="cuda").bfloat16().expand(S, 2, 1024)
    pos = torch.randint(0, 5000, (S,), generator=g, device="cuda")
    freqs, _ = M.rope_freqs(1024)
    y, _ = M.rope(x, None, pos, freqs)
    at = torch.tensor([0, 5, 1 << 19, (1 << 20) - 1, 1 << 20, S - 1], device="cuda")
    assert torch.equal(y[at], M.rope(x[at], None, pos[at], freqs)[0])
