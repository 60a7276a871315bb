"""Dense operators on the GPU at the edges of their ranges, against 64-bit values.

Tolerances, derived before the first run, in units of U = 2^-24 (half a step of fp32, relative); a result stored in bf16
may be off by 2^-8 more.
  norm   a lane's eight squares are added up in eight roundings, all later sums are fp64; half of that through the root;
         the mean, eps, root, quotient (2) and the product with gamma one each: (8 / 2 + 6) U.  Far from 1 a row's
         statistics are fp64 and its values scaled by a power of two: nothing more, except values that leave the range of
         normal fp32 on the way, which are below 2^-60 of the largest.
  codes  |q - v / d| <= 1/2 + 127 times twice the value's relative error (v and d both carry it).
"""
import math

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


def check_rows(y, q, d, v, rel):
    """y, and the int8 rows q, d, against 64-bit values v."""
    more = 2.0 ** -8 if y.dtype == BF else 0.0
    top = v.abs().amax(1, keepdim=True)
    assert ((y.double() - v).abs() <= (rel + more) * v.abs() + top * 2.0 ** -60).all()
    step = top[:, 0] / 127
    assert ((d.double() - step).abs() <= (rel + U) * step).all()
    assert ((q.double() - v / step[:, None]).abs() <= 0.5 + 127 * 2 * (rel + U)).all()


# widths of every way to split a row over waves, for few rows and for many
WIDTHS = [5, 500, 1000, 1001, 2048, 4096, 4099, 6144, 8192, 12288, 16384, 16385, 20000]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("S", [3, 70])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_of_far_magnitudes(M, H, S, dtype):
    """Rows whose squares leave the range of fp32 have the norm that the formula gives them, also beside ordinary rows."""
    g = rng(H + S)
    gamma = 1 + 0.2 * torch.randn(H, generator=g, device="cuda")
    base = torch.randn(S, H, generator=g, device="cuda").clamp(-3, 3)
    for scale in (1e19, 7e18, 1e25, 1e37, 1e-15, 1e-19, 1e-23, 1e-30, 1e-38):
        x = (base * scale).to(dtype)
        x[1] = base[1].to(dtype)
        for eps in (0.0, 1e-40) if scale < 1 else (0.0, 1e-5):
            for yd in (F32, BF):
                _, y, q, d = M.norm_quant(x, gamma, eps, y_dtype=yd)
                f, e = x.double(), torch.tensor(eps, dtype=F32).item()
                check_rows(y, q, d, f / torch.sqrt((f * f).mean(1, keepdim=True) + e) * gamma.double(), (8 / 2 + 6) * U)


@pytest.mark.parametrize("H", [700, 6144, 20000])
def test_norm_of_one_large_value(M, H):
    """One value whose square alone is beyond fp32, while the mean is not; zeros with eps = 0 stay NaN in their row."""
    x = torch.randn(6, H, generator=rng(H), device="cuda")
    x[2, H // 2] = 2e19
    x[4] = 0
    one = torch.ones(H, device="cuda")
    _, y, q, d = M.norm_quant(x, one, 0.0, y_dtype=F32)
    keep = [0, 1, 2, 3, 5]
    f = x[keep].double()
    check_rows(y[keep], q[keep], d[keep], f / torch.sqrt((f * f).mean(1, keepdim=True)), (8 / 2 + 6) * U)
    assert torch.isnan(y[4]).all() and (q[4] == 0).all() and torch.isnan(d[4])


def exact_turns(pos, freqs):
    """(cos, sin) of pos * f as float64 tensors [S, n], the product exact and reduced by pi to 90 digits (Machin's sum)."""
    from fractions import Fraction
    one = 10 ** 90

    def arctan_of_inverse(k):
        total, term, n = 0, one // k, 1
        while term:
            total += term // n if n % 4 == 1 else -(term // n)
            term //= k * k
            n += 2
        return total
    two_pi = Fraction(8 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239)), one)
    c, s = [], []
    for p in pos:
        for f in freqs:
            a = Fraction(p) * Fraction(f)
            a -= round(a / two_pi) * two_pi
            c.append(math.cos(a))
            s.append(math.sin(a))
    shape = len(pos), len(freqs)
    return (torch.tensor(v, dtype=torch.float64, device="cuda").view(shape) for v in (c, s))


FAR = [0, 1, 7, 100003, (1 << 24) + 1, (1 << 28) + 3, (1 << 31) - 1, -(1 << 31), (1 << 36) + 11, (1 << 40) + 3, -(1 << 44) - 5]
FARTHEST = [(1 << 49) + 1, -(1 << 50) - 3, (1 << 53) - 1, 5 << 52, -(7 << 56), (1 << 61) + (1 << 20), -(1 << 62) + (1 << 30)]


@pytest.mark.parametrize("inter", [False, True])
def test_rope_keeps_the_angles_of_far_positions(M, inter):
    """The angle is the exact product of position and frequency, whatever its size.  A pair (1, 0) gives cosine and sine:
    each within 2 U of the true value (the zero beside them adds nothing)."""
    freqs, _ = M.rope_freqs(64)
    freqs[1] = 0.7364182
    pos = torch.tensor(FAR, device="cuda")
    x = torch.zeros(len(FAR), 3, 64, device="cuda")
    (x[..., 0::2] if inter else x[..., :32]).fill_(1)
    y, _ = M.rope(x, None, pos, freqs, interleaved=inter)
    c, s = exact_turns(FAR, freqs.tolist())
    got_c, got_s = (y[..., 0::2], y[..., 1::2]) if inter else (y[..., :32], y[..., 32:])
    for got, want in ((got_c, c), (got_s, s)):
        assert ((got.double() - want[:, None]).abs() <= 2 * U).all()
    far = torch.tensor(FARTHEST, device="cuda")  # all of them fp64 values
    y2, _ = M.rope(x[:len(FARTHEST)], None, far, freqs[:2].contiguous(), interleaved=inter)
    c, s = exact_turns(FARTHEST, freqs[:2].tolist())
    got_c, got_s = (y2[..., 0:4:2], y2[..., 1:4:2]) if inter else (y2[..., :2], y2[..., 2:4])
    x1, x2 = (x[0, 0, 0:4:2], x[0, 0, 1:4:2]) if inter else (x[0, 0, :2], x[0, 0, 2:4])
    for got, want in ((got_c, c * x1 - s * x2), (got_s, c * x2 + s * x1)):
        assert ((got.double() - want[:, None]).abs() <= 4 * U).all()
    k = 7  # the positions that int32 holds
    y32, _ = M.rope(x[:k], None, pos[:k].int(), freqs, interleaved=inter)
    assert torch.equal(y32, y[:k])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("far", [1, 1 << 10, 1 << 16])
def test_rope_coefficients_are_rounded_once(M, far, inter):
    """A pair (1, 0) gives factor * (cos a, sin a): rounded to fp32 once, from a value within 2^-35 of the formula's (an fp64
    series whose first term left out is below 2^-36 up to pi / 4; the angle itself is rounded at 2^-38 here)."""
    S, n = 4096, 32
    for factor in (1.0, 0.1 * math.log(4.0) + 1.0, 1.25):
        freqs, _ = M.rope_freqs(2 * n)
        pos = torch.randint(-far, far + 1, (S,), generator=rng(far), device="cuda")
        x = torch.zeros(S, 1, 2 * n, device="cuda")
        (x[..., 0::2] if inter else x[..., :n]).fill_(1)
        y, _ = M.rope(x, None, pos, freqs, interleaved=inter, factor=factor)
        a = pos.double()[:, None] * freqs
        got_c, got_s = (y[..., 0::2], y[..., 1::2]) if inter else (y[..., :n], y[..., n:])
        for got, want in ((got_c, a.cos() * factor), (got_s, a.sin() * factor)):
            want = want[:, None]
            assert ((got.double() - want).abs() <= U * want.abs() + factor * 2.0 ** -35).all()


def test_yarn_factor_keeps_its_bits(M):
    """The frequencies' factor comes as the fp64 value of its formula, and goes into the call as such."""
    _, factor = M.rope_freqs(64, 10000.0, "yarn", 4.0, 4096)
    assert abs(factor - (0.1 * math.log(4.0) + 1.0)) <= 2.0 ** -52
