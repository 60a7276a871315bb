"""Calls of the dense operators that have to be refused, or to leave a mark, before anything runs (no GPU needed)."""
import pytest
import torch

from int4_routed_expert_amd import moe as M

A = 1 << 20  # an address that is never read: every call here is refused
BIG = [1 << 31, (1 << 32) + 2]  # the second one's low 32 bits are an ordinary size


def wide(n, m, dtype=torch.float32):
    """[n, m] of one element's memory along n, or along m where m is large (contiguous rows, which need real ones)."""
    return torch.zeros((1, m), dtype=dtype).expand(n, m)


def i8(*shape):
    return torch.zeros(shape, dtype=torch.int8)


@pytest.mark.parametrize("n", BIG)
@pytest.mark.parametrize("call", [
    lambda n: M.norm_quant(wide(n, 8), torch.zeros(8), 1e-5),
    lambda n: M.silu_quant(wide(n, 8)),
    lambda n: M.silu_quant(wide(n, 8), wide(n, 8)),
    lambda n: M.qmatmul(wide(n, 16, torch.int8), torch.zeros(()).expand(n), i8(4, 16), torch.zeros(4)),
    lambda n: M.qmatmul(i8(2, 16), torch.zeros(2), wide(n, 16, torch.int8), torch.zeros(()).expand(n)),
    lambda n: M.rope(torch.zeros(1, 2, 8).expand(n, 2, 8), None, torch.zeros((), dtype=torch.int64).expand(n),
                     torch.zeros(4, dtype=torch.float64)),
    lambda n: M.rope(torch.zeros(2, 1, 8).expand(2, n, 8), None, torch.zeros(2, dtype=torch.int64),
                     torch.zeros(4, dtype=torch.float64)),
    lambda n: M.rope(torch.zeros(2, 1, 8), torch.zeros(2, 1, 8).expand(2, n, 8), torch.zeros(2, dtype=torch.int64),
                     torch.zeros(4, dtype=torch.float64)),
    lambda n: M.rope(torch.zeros(2, 1, 8), None, torch.zeros(2, dtype=torch.int64), torch.zeros(2, dtype=torch.float64),
                     offset=n),
    lambda n: M.rope_freqs(n, device="cpu"),
    lambda n: M.rope_freqs(64, 10000.0, "yarn", 4.0, n, device="cpu"),
    lambda n: M.moe_norm_quant(A, 0, 64, None, 0, A, 0, 1e-5, n, 64, None, 0, A, 0, 64, None, 0, None, 0),
    lambda n: M.moe_norm_quant(A, 0, n, None, 0, A, 0, 1e-5, 1, n, None, 0, A, 0, n, None, 0, None, 0),
    lambda n: M.moe_silu_quant(A, A, 0, 64, n, 64, A, 0, 64, None, 0, None, 0),
    lambda n: M.moe_silu_quant(A, A, 0, n, 1, n, A, 0, n, None, 0, None, 0),
    lambda n: M.moe_qmatmul(A, 64, A, A, 64, A, n, 4, 64, A, 0, 4, None, 0, 0),
    lambda n: M.moe_qmatmul(A, 64, A, A, 64, A, 1, n, 64, A, 0, n, None, 0, 0),
    lambda n: M.moe_qmatmul(A, n, A, A, n, A, 1, 4, n, A, 0, 4, None, 0, 0),
    lambda n: M.moe_rope(M.moe_rope_tensor(A, A, 8, 8, 8, 8, 1), None, 0, n, 8, 8, 0, 0, A, 1, A, 1.0, 0),
    lambda n: M.moe_rope(M.moe_rope_tensor(A, A, 8, 8, 8, 8, 1), None, 0, 1, n, 8, 0, 0, A, 1, A, 1.0, 0),
    lambda n: M.moe_rope(M.moe_rope_tensor(A, A, 8, 8, 8, 8, 1), None, 0, 1, 8, n, 0, 0, A, 1, A, 1.0, 0),
    lambda n: M.moe_rope(M.moe_rope_tensor(A, A, 8, 8, 8, 8, 1), None, 0, 1, 8, 2, n, 0, A, 1, A, 1.0, 0),
])
def test_sizes_beyond_the_abi(call, n, monkeypatch):
    """Sizes that the ABI's 32 bits do not hold are refused as a size out of range, not cut to their low bits."""
    def never(*args):
        raise AssertionError("the C entry was called")
    for name in ("moe_norm_quant", "moe_silu_quant", "moe_qmatmul", "moe_rope", "moe_rope_freqs"):
        monkeypatch.setattr(M._lib, name, never)
    monkeypatch.setattr(M, "_vector", lambda *args: None)  # the vectors of such sizes are stand-ins of one element
    with pytest.raises(M.MoeError) as e:
        call(n)
    assert e.value.status == M.MOE_EINVAL


@pytest.mark.parametrize("n", BIG)
def test_workspace_of_sizes_beyond_the_abi(n):
    for S, N, K in ((n, 4, 64), (4, n, 64), (4, 4, n)):
        assert M.moe_qmatmul_workspace_bytes(A, 64, A, 64, S, N, K) == M.MOE_EINVAL


@pytest.mark.parametrize("rot", [-2, -(1 << 31) + 2])
def test_negative_sizes_reach_the_check(rot):
    with pytest.raises(M.MoeError) as e:
        M.rope_freqs(rot, device="cpu")
    assert e.value.status == M.MOE_EINVAL


@pytest.mark.parametrize("ws", [torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(1 << 20, dtype=torch.uint8)[::2]])
def test_workspace_has_to_be_one_piece(ws):
    """A tensor whose elements do not lie one after another has less memory, or other memory, than its size says."""
    with pytest.raises(ValueError, match="ws"):
        M.qmatmul(i8(70, 33), torch.zeros(70), i8(9, 33), torch.zeros(9), ws=ws)


F, B = M.MOE_F32, M.MOE_BF16
X, R, Y, Q = (A + (i << 24) for i in range(4))


def norm(x=X, xd=B, ldx=64, res=None, ldr=0, h=None, ldh=0, y=None, yd=B, ldy=0, q=None, S=2):
    return M._lib.moe_norm_quant(x, xd, ldx, res, ldr, A, F, 1e-5, S, 64, h, ldh, y, yd, ldy, q, 64, q, None)


def silu(y, yd=B, ldy=64, ldx=64, S=2):
    return M._lib.moe_silu_quant(X, R, B, ldx, S, 64, y, yd, ldy, None, 0, None, None)


@pytest.mark.parametrize("call", [
    lambda: norm(y=X, yd=F, ldy=64), lambda: norm(xd=F, ldx=64, y=X, yd=B, ldy=64), lambda: norm(y=X, ldy=72),
    lambda: norm(res=R, ldr=64, h=R, ldh=72), lambda: norm(res=R, ldr=64, h=X, ldh=72), lambda: norm(y=X, yd=F, ldy=64, S=1),
    lambda: silu(X, yd=F), lambda: silu(R, yd=F), lambda: silu(X, ldy=72), lambda: silu(R, ldy=72, ldx=80)])
def test_in_place_at_another_type_or_stride(call):
    """An output over its input has to have its type and stride: rows would be written over rows not read yet."""
    assert call() == M.MOE_EINVAL


def grad(*shape):
    return torch.zeros(shape, requires_grad=True)


POS, FREQS = torch.zeros(2, dtype=torch.int64), torch.zeros(4, dtype=torch.float64)
WITH_GRAD = [
    lambda: M.norm_quant(grad(2, 8), torch.zeros(8), 1e-5),
    lambda: M.norm_quant(torch.zeros(2, 8), grad(8), 1e-5),
    lambda: M.norm_quant(torch.zeros(2, 8), torch.zeros(8), 1e-5, residual=grad(2, 8)),
    lambda: M.silu_quant(grad(2, 8)),
    lambda: M.silu_quant(torch.zeros(2, 8), grad(2, 8)),
    lambda: M.qmatmul(i8(2, 8), grad(2), i8(4, 8), torch.zeros(4)),
    lambda: M.qmatmul(i8(2, 8), torch.zeros(2), i8(4, 8), grad(4)),
    lambda: M.rope(grad(2, 4, 8), None, POS, FREQS),
    lambda: M.rope(torch.zeros(2, 4, 8), grad(2, 1, 8), POS, FREQS),
]


@pytest.mark.parametrize("call", WITH_GRAD)
def test_no_gradient_is_lost_silently(call):
    """There is no backward pass: an input that asks for gradients is refused where torch would record the call."""
    with pytest.raises(ValueError, match="no_grad"):
        call()
    for off in (torch.no_grad(), torch.inference_mode()):
        with off, pytest.raises(ValueError, match="on a GPU"):  # past that check, refused for the CPU tensors
            call()


@pytest.fixture
def on_cpu(monkeypatch):
    """The binding's calls on CPU tensors, up to the C entries, which do nothing."""
    monkeypatch.setattr(M, "_gpu", lambda *tensors: 0)
    monkeypatch.setattr(M, "_current_gpu", lambda: 0)
    monkeypatch.setattr(M, "_stream_of", lambda gpu: None)
    for name in ("moe_norm_quant", "moe_rope"):
        monkeypatch.setattr(M._lib, name, lambda *args: 0)


def test_in_place_writes_raise_the_version(on_cpu):
    """A tensor that a call writes over counts as changed, so that torch refuses a backward pass through its old values."""
    x, r, g = torch.zeros(2, 8), torch.zeros(2, 8), torch.zeros(8)
    versions = lambda *ts: [t._version for t in ts]  # noqa: E731
    before = versions(x, r, g)
    h = M.norm_quant(x, g, 1e-5, residual=r, h=r)[0]
    assert h is r and versions(x, r, g) == [before[0], before[1] + 1, before[2]]
    M.norm_quant(x, g, 1e-5, residual=r, h=x)
    assert versions(x, r) == [before[0] + 1, before[1] + 1]
    M.norm_quant(x, g, 1e-5, residual=r)
    assert versions(x, r) == [before[0] + 1, before[1] + 1]
    both = torch.zeros(2, 5, 8)
    q, k = both[:, :4], both[:, 4:]
    M.rope(q, k, POS, FREQS)
    assert both._version == 0
    M.rope(q, k, POS, FREQS, inplace=True)
    assert both._version > 0
    k = torch.zeros(2, 1, 8)
    M.rope(torch.zeros(2, 4, 8), k, POS, FREQS, inplace=True)
    assert k._version == 1
    leaf = torch.ones(2, 8, requires_grad=True)
    saved = torch.ones(2, 8)
    loss = (leaf * saved).sum()
    M.norm_quant(x, g, 1e-5, residual=saved, h=saved)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        M.norm_quant(torch.zeros(2, 8), g, 1e-5, residual=r, h=torch.zeros(2, 8))


class OtherGpusStream:
    cuda_stream, device_index = 64, 1


def test_stream_of_another_gpu():
    """A stream belongs to one GPU: the call would run on the tensors' own current stream instead, unordered with it."""
    with pytest.raises(ValueError, match="stream"):
        M._elsewhere(0, OtherGpusStream(), lambda: None, ())


def test_header_names():
    """moe.HEADER is include/moe.h, as it was before there were two headers."""
    assert M.HEADER == M.HEADERS[0] and M.HEADER.endswith("moe.h")
    assert "int moe_layer(" in open(M.HEADER).read()
