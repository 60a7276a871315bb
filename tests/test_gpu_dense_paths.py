"""Paths of the dense operators that only certain sizes and places take, each named by the test that takes it:
workgroups that go on to a second row, launches in several pieces, copies of one operand, several tokens a workgroup,
and the layer's own int8 activations next to the dense operators'."""
import pytest
import torch

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
