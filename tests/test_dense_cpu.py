"""Dense operators without a GPU: refusals at the C entries and in the binding, sizes, rotary frequencies."""
import ctypes
import math

import numpy as np
import pytest
import torch

from int4_routed_expert_amd import moe as M

L = M.lib()
A = 1 << 20  # an address that is never read: every call here is refused, or has no rows


def norm(x=A, xd=0, ldx=64, res=A, ldr=64, g=A, gd=0, eps=1e-5, S=2, H=64, h=A, ldh=64, y=A, yd=0, ldy=64, q=A, ldq=64,
         d=A):
    return L.moe_norm_quant(x, xd, ldx, res, ldr, g, gd, eps, S, H, h, ldh, y, yd, ldy, q, ldq, d, None)


@pytest.mark.parametrize("bad,status", [
    (dict(S=-1), M.MOE_EINVAL), (dict(H=0), M.MOE_EINVAL), (dict(eps=-1.0), M.MOE_EINVAL),
    (dict(eps=float("nan")), M.MOE_EINVAL), (dict(eps=float("inf")), M.MOE_EINVAL), (dict(xd=7), M.MOE_EDTYPE),
    (dict(gd=-1), M.MOE_EDTYPE), (dict(yd=2), M.MOE_EDTYPE), (dict(x=None), M.MOE_ENULL), (dict(g=None), M.MOE_ENULL),
    (dict(h=None, y=None, q=None, d=None), M.MOE_ENULL), (dict(res=None), M.MOE_ENULL), (dict(q=None), M.MOE_ENULL),
    (dict(d=None), M.MOE_ENULL), (dict(x=A + 2), M.MOE_EINVAL), (dict(x=A + 1, xd=1), M.MOE_EINVAL),
    (dict(g=A + 2), M.MOE_EINVAL), (dict(y=A + 2), M.MOE_EINVAL), (dict(d=A + 2), M.MOE_EINVAL),
    (dict(ldx=-1), M.MOE_EINVAL), (dict(ldr=-64), M.MOE_EINVAL), (dict(ldh=63), M.MOE_EINVAL),
    (dict(ldy=63), M.MOE_EINVAL), (dict(ldq=63), M.MOE_EINVAL)])
def test_norm_refusals(bad, status):
    assert norm(**bad) == status


def silu(g=A, u=A, xd=0, ldx=64, S=2, I=64, y=A, yd=0, ldy=64, q=A, ldq=64, d=A):
    return L.moe_silu_quant(g, u, xd, ldx, S, I, y, yd, ldy, q, ldq, d, None)


@pytest.mark.parametrize("bad,status", [
    (dict(S=-1), M.MOE_EINVAL), (dict(I=0), M.MOE_EINVAL), (dict(xd=3), M.MOE_EDTYPE), (dict(yd=3), M.MOE_EDTYPE),
    (dict(g=None), M.MOE_ENULL), (dict(u=None), M.MOE_ENULL), (dict(y=None, q=None, d=None), M.MOE_ENULL),
    (dict(d=None), M.MOE_ENULL), (dict(u=A + 2), M.MOE_EINVAL), (dict(ldx=-1), M.MOE_EINVAL),
    (dict(ldy=1), M.MOE_EINVAL), (dict(ldq=1), M.MOE_EINVAL)])
def test_silu_refusals(bad, status):
    assert silu(**bad) == status


def product(q=A, ldq=64, d=A, w=A, ldw=64, dw=A, S=2, N=64, K=64, y=A, yd=0, ldy=64, ws=A, wb=1 << 30):
    return L.moe_qmatmul(q, ldq, d, w, ldw, dw, S, N, K, y, yd, ldy, ws, wb, None)


@pytest.mark.parametrize("bad,status", [
    (dict(S=-1), M.MOE_EINVAL), (dict(N=0), M.MOE_EINVAL), (dict(K=0), M.MOE_EINVAL), (dict(K=131072), M.MOE_EINVAL),
    (dict(yd=9), M.MOE_EDTYPE), (dict(q=None), M.MOE_ENULL), (dict(d=None), M.MOE_ENULL), (dict(w=None), M.MOE_ENULL),
    (dict(dw=None), M.MOE_ENULL), (dict(y=None), M.MOE_ENULL), (dict(ldq=-1), M.MOE_EINVAL), (dict(ldw=-1), M.MOE_EINVAL),
    (dict(ldy=63), M.MOE_EINVAL), (dict(d=A + 1), M.MOE_EINVAL), (dict(dw=A + 2), M.MOE_EINVAL),
    (dict(y=A + 2), M.MOE_EINVAL), (dict(y=A + 1, yd=1), M.MOE_EINVAL)])
def test_product_refusals(bad, status):
    assert product(**bad) == status


def test_product_workspace():
    """Operands on 16-byte boundaries need none; for others the size is the copies' and a workspace is required exactly
    where it is not 0."""
    sizes = [(1, 1, 1), (1, 4096, 6144), (16, 576, 16384), (64, 576, 16384), (256, 6144, 6144), (8192, 12288, 6144),
             (77, 577, 1111), (600, 4097, 6143), (1, 1, 131071), (500, 300, 131071)]
    seen = 0
    for S, N, K in sizes:
        for off, ld in ((0, K), (0, K + 5), (1, K + 16)):
            args = dict(q=A + off, ldq=ld, w=A + off, ldw=ld, S=S, N=N, K=K)
            need = M.moe_qmatmul_workspace_bytes(args["q"], ld, args["w"], ld, S, N, K)
            assert 0 <= need <= (S + N) * (K + 15)
            if off == 0 and ld % 16 == 0 and K % 16 == 0:
                assert need == 0
            if need:
                seen += 1
                assert product(**args, ldy=N, ws=None) == M.MOE_ENULL
                assert product(**args, ldy=N, ws=A + 4) == M.MOE_EINVAL
                assert product(**args, ldy=N, wb=need - 1) == M.MOE_EWORKSPACE
    assert seen
    assert M.moe_qmatmul_workspace_bytes(None, 64, None, 64, 0, 64, 64) == 0
    for S, N, K in [(-1, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, 131072)]:
        assert M.moe_qmatmul_workspace_bytes(A, 64, A, 64, S, N, K) == M.MOE_EINVAL


def turn(q=(A, A, 256, 64, 256, 64, 4), k=(A, A, 64, 64, 64, 64, 1), xd=0, S=2, D=64, rot=64, offset=0, layout=0, pos=A,
         wide=1, freqs=A):
    t = [None if v is None else ctypes.byref(M.moe_rope_tensor(*v)) for v in (q, k)]
    return L.moe_rope(*t, xd, S, D, rot, offset, layout, pos, wide, freqs, 1.0, None)


@pytest.mark.parametrize("bad,status", [
    (dict(S=-1), M.MOE_EINVAL), (dict(D=1), M.MOE_EINVAL), (dict(D=1026), M.MOE_EINVAL), (dict(rot=63), M.MOE_EINVAL),
    (dict(rot=0), M.MOE_EINVAL), (dict(rot=66), M.MOE_EINVAL), (dict(offset=2), M.MOE_EINVAL),
    (dict(offset=-2, rot=32), M.MOE_EINVAL), (dict(layout=2), M.MOE_EINVAL), (dict(wide=2), M.MOE_EINVAL),
    (dict(xd=5), M.MOE_EDTYPE), (dict(q=None), M.MOE_ENULL), (dict(pos=None), M.MOE_ENULL), (dict(freqs=None), M.MOE_ENULL),
    (dict(pos=A + 4), M.MOE_EINVAL), (dict(freqs=A + 4), M.MOE_EINVAL), (dict(q=(None, A, 256, 64, 256, 64, 4)), M.MOE_ENULL),
    (dict(k=(A, None, 64, 64, 64, 64, 1)), M.MOE_ENULL), (dict(q=(A, A, 256, 64, 256, 64, 0)), M.MOE_EINVAL),
    (dict(k=(A, A, 64, 64, 64, 64, -1)), M.MOE_EINVAL), (dict(q=(A, A + 4096, 256, 64, 63, 64, 4)), M.MOE_EINVAL),
    (dict(q=(A, A + 4096, 256, 64, 256, 63, 4)), M.MOE_EINVAL), (dict(q=(A, A, 512, 64, 256, 64, 4)), M.MOE_EINVAL),
    (dict(q=(A, A, -256, 64, 256, 64, 4)), M.MOE_EINVAL), (dict(q=(A + 2, A, 256, 64, 256, 64, 4)), M.MOE_EINVAL),
    (dict(q=(A, A, 1 << 21, 64, 1 << 21, 64, 16384)), M.MOE_EINVAL)])
def test_rope_refusals(bad, status):
    assert turn(**bad) == status


def test_no_rows_is_no_work():
    """S = 0 returns before any pointer or launch; the binding's forms need a GPU to allocate on and are tested there."""
    assert norm(S=0, x=None) == silu(S=0, g=None) == product(S=0, q=None, ws=None) == turn(S=0, pos=None) == M.MOE_OK


def test_rope_frequencies():
    """Each scaling against its formula, written here once more."""
    R, theta = 64, 10000.0
    plain = np.array([theta ** (-2 * i / R) for i in range(R // 2)])
    f, m = M.moe_rope_freqs(R, theta, M.MOE_ROPE_PLAIN, 1.0, 0, 0, 0)
    assert np.allclose(f, plain, rtol=1e-14, atol=0) and m == 1.0
    f, m = M.moe_rope_freqs(R, theta, M.MOE_ROPE_LINEAR, 4.0, 0, 0, 0)
    assert np.allclose(f, plain / 4, rtol=1e-14, atol=0) and m == 1.0
    f, m = M.moe_rope_freqs(R, theta, M.MOE_ROPE_NTK, 4.0, 0, 0, 0)
    assert f[0] == 1.0 and abs(f[-1] / (plain[-1] / 4) - 1) < 1e-12 and m == 1.0  # fastest kept, slowest over scale
    f, m = M.moe_rope_freqs(R, theta, M.MOE_ROPE_YARN, 8.0, 4096, 32.0, 1.0)
    assert abs(m - (0.1 * math.log(8.0) + 1)) < 1e-7
    turns = 4096 * plain / (2 * math.pi)
    ratio = f / plain
    assert np.allclose(ratio[turns > 32 * theta ** (2 / R)], 1.0, rtol=1e-14)  # one index beyond the rounded ends
    assert np.allclose(ratio[turns < theta ** (-2 / R)], 1 / 8, rtol=1e-14)
    assert np.all(np.diff(ratio) <= 1e-15) and np.all(np.abs(np.diff(ratio, 2))[(ratio[1:-1] < 1) & (ratio[1:-1] > 1 / 8)][1:-1] < 1e-12)
    f, m = M.moe_rope_freqs(R, theta, M.MOE_ROPE_YARN, 1.0, 4096, 32.0, 1.0)  # no stretch: nothing changes
    assert np.allclose(f, plain, rtol=1e-14) and m == 1.0
    for bad in [(63, theta, 0, 1.0, 0, 0, 0), (0, theta, 0, 1.0, 0, 0, 0), (R, 1.0, 0, 1.0, 0, 0, 0),
                (R, theta, 4, 1.0, 0, 0, 0), (R, theta, 1, 0.5, 0, 0, 0), (2, theta, 2, 2.0, 0, 0, 0),
                (R, theta, 3, 2.0, 0, 32, 1), (R, theta, 3, 2.0, 4096, 1, 1), (R, theta, 3, 2.0, 4096, 1, 0),
                (R, float("nan"), 0, 1.0, 0, 0, 0)]:
        with pytest.raises(M.MoeError):
            M.moe_rope_freqs(*bad)


def t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("call", [
    lambda: M.norm_quant(t(2, 8, dtype=torch.float16), t(8), 1e-5),
    lambda: M.norm_quant(t(2, 8), t(8, dtype=torch.int8), 1e-5),
    lambda: M.norm_quant(t(8, 2).t(), t(8), 1e-5),
    lambda: M.norm_quant(t(2, 8), t(7), 1e-5),
    lambda: M.norm_quant(t(2, 8), t(8), 1e-5, residual=t(2, 9)),
    lambda: M.norm_quant(t(2, 8), t(8), 1e-5, residual=t(2, 8, dtype=torch.bfloat16)),
    lambda: M.norm_quant(t(2, 8), t(8), 1e-5, h=t(2, 8)),
    lambda: M.norm_quant(t(2, 8), t(8), 1e-5, residual=t(2, 8), h=t(2, 8, dtype=torch.bfloat16)),
    lambda: M.norm_quant(t(2, 8), t(8), 1e-5, y_dtype=torch.float16),
    lambda: M.norm_quant(t(2, 8), t(8), 1e-5, quant=False),
    lambda: M.norm_quant(t(2, 8), t(8), 1e-5),  # not on a GPU
    lambda: M.silu_quant(t(2, 7)),
    lambda: M.silu_quant(t(2, 8), t(2, 7)),
    lambda: M.silu_quant(t(2, 8), t(2, 16)[:, :8]),
    lambda: M.silu_quant(t(2, 8), t(2, 8, dtype=torch.bfloat16)),
    lambda: M.silu_quant(t(2, 8), quant=False),
    lambda: M.silu_quant(t(2, 8)),
    lambda: M.qmatmul(t(2, 8), t(2), t(4, 8, dtype=torch.int8), t(4)),
    lambda: M.qmatmul(t(2, 8, dtype=torch.int8), t(3), t(4, 8, dtype=torch.int8), t(4)),
    lambda: M.qmatmul(t(2, 8, dtype=torch.int8), t(2), t(4, 9, dtype=torch.int8), t(4)),
    lambda: M.qmatmul(t(2, 8, dtype=torch.int8), t(2), t(4, 8, dtype=torch.int8), t(5)),
    lambda: M.qmatmul(t(2, 8, dtype=torch.int8), t(2), t(8, 4, dtype=torch.int8).t(), t(4)),
    lambda: M.qmatmul(t(2, 8, dtype=torch.int8), t(2), t(4, 8, dtype=torch.int8), t(4), out_dtype=torch.float16),
    lambda: M.qmatmul(t(2, 8, dtype=torch.int8), t(2), t(4, 8, dtype=torch.int8), t(4)),
    lambda: M.rope(t(2, 4, 8), t(3, 1, 8), t(2, dtype=torch.int64), t(4, dtype=torch.float64)),
    lambda: M.rope(t(2, 4, 8), t(2, 1, 6), t(2, dtype=torch.int64), t(4, dtype=torch.float64)),
    lambda: M.rope(t(2, 4, 8), t(2, 1, 8, dtype=torch.bfloat16), t(2, dtype=torch.int64), t(4, dtype=torch.float64)),
    lambda: M.rope(t(2, 4, 8), None, t(2, dtype=torch.int16), t(4, dtype=torch.float64)),
    lambda: M.rope(t(2, 4, 8), None, t(3, dtype=torch.int64), t(4, dtype=torch.float64)),
    lambda: M.rope(t(2, 4, 8), None, t(2, dtype=torch.int64), t(4)),
    lambda: M.rope(t(2, 8, 4).transpose(1, 2), None, t(2, dtype=torch.int64), t(4, dtype=torch.float64)),
    lambda: M.rope(t(2, 4, 8), None, t(2, dtype=torch.int64), t(4, dtype=torch.float64)),
    lambda: M.rope_freqs(64, scaling="other", device="cpu"),
])
def test_binding_refusals(call):
    with pytest.raises(ValueError):
        call()


def test_header_is_plain_c(tmp_path):
    """include/moe_dense.h compiles by itself as strict C11, and its functions are exported and bound."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "t.c"
    src.write_text('#include "moe_dense.h"\nint main(void) { moe_rope_tensor t = {0}; return t.heads + MOE_ROPE_YARN - 3; }\n')
    subprocess.check_call(["gcc", "-std=c11", "-pedantic-errors", "-Wall", "-Wextra", "-Werror", "-I",
                           os.path.join(root, "include"), "-c", str(src), "-o", str(tmp_path / "t.o")])
    names = {"moe_norm_quant", "moe_silu_quant", "moe_qmatmul", "moe_qmatmul_workspace_bytes", "moe_rope", "moe_rope_freqs"}
    assert names <= set(M.header_functions())
    for n in names:
        assert hasattr(L, n) and callable(getattr(M, n))
