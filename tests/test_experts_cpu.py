"""Microscaled rows, grouped products, grouping and return without a GPU: refusals at the C entries and in the binding."""
import ctypes

import pytest
import torch

import mxref as R
from int4_routed_expert_amd import moe as M

L = M.lib()
A = 1 << 20  # an address that is never read: every call here is refused, or has no rows


def quant(x=A, xd=0, ldx=64, S=2, H=64, r=0, q=A, ldq=32, e=A, lde=2):
    return L.moe_mx_quant(x, xd, ldx, S, H, r, q, ldq, e, lde, None)


@pytest.mark.parametrize("bad,status", [
    (dict(S=-1), M.MOE_EINVAL), (dict(H=0), M.MOE_EINVAL), (dict(H=2 ** 25 + 1), M.MOE_EINVAL), (dict(r=2), M.MOE_EINVAL),
    (dict(xd=2), M.MOE_EDTYPE), (dict(x=None), M.MOE_ENULL), (dict(q=None), M.MOE_ENULL), (dict(e=None), M.MOE_ENULL),
    (dict(x=A + 2), M.MOE_EINVAL), (dict(x=A + 1, xd=1), M.MOE_EINVAL), (dict(ldx=-1), M.MOE_EINVAL), (dict(q=A + 8), M.MOE_EINVAL),
    (dict(ldq=40), M.MOE_EINVAL), (dict(ldq=16), M.MOE_EINVAL), (dict(lde=1), M.MOE_EINVAL), (dict(lde=-2), M.MOE_EINVAL),
    (dict(S=0, x=None, q=None, e=None), M.MOE_OK)])
def test_quant_refusals(bad, status):
    assert quant(**bad) == status


def silu(g=A, u=A, xd=0, ldx=64, S=2, I=64, r=0, q=A, ldq=32, e=A, lde=2):
    return L.moe_mx_silu_quant(g, u, xd, ldx, S, I, r, q, ldq, e, lde, None)


@pytest.mark.parametrize("bad,status", [
    (dict(S=-1), M.MOE_EINVAL), (dict(I=0), M.MOE_EINVAL), (dict(r=-1), M.MOE_EINVAL), (dict(xd=9), M.MOE_EDTYPE),
    (dict(g=None), M.MOE_ENULL), (dict(u=None), M.MOE_ENULL), (dict(u=A + 2), M.MOE_EINVAL), (dict(e=None), M.MOE_ENULL),
    (dict(q=A + 1), M.MOE_EINVAL), (dict(S=0), M.MOE_OK)])
def test_silu_refusals(bad, status):
    assert silu(**bad) == status


def values(q=A, ldq=32, e=A, lde=2, S=2, H=64, y=A, yd=0, ldy=64):
    return L.moe_mx_values(q, ldq, e, lde, S, H, y, yd, ldy, None)


@pytest.mark.parametrize("bad,status", [
    (dict(S=-1), M.MOE_EINVAL), (dict(H=0), M.MOE_EINVAL), (dict(yd=-1), M.MOE_EDTYPE), (dict(y=None), M.MOE_ENULL),
    (dict(q=None), M.MOE_ENULL), (dict(e=None), M.MOE_ENULL), (dict(y=A + 2), M.MOE_EINVAL), (dict(ldy=63), M.MOE_EINVAL),
    (dict(q=A + 4), M.MOE_EINVAL), (dict(ldq=17), M.MOE_EINVAL), (dict(lde=-1), M.MOE_EINVAL), (dict(S=0), M.MOE_OK)])
def test_values_refusals(bad, status):
    assert values(**bad) == status


def rows(q=A, e=A, ldq=64, lde=4, expert_q=0, expert_e=0):
    return M.moe_mx_rows(q, e, ldq, lde, expert_q, expert_e)


def matmul(x=rows(), w=rows(), S=2, N=3, B=4, y=A, yd=0, ldy=3, ws=A, wb=1 << 40):
    r = lambda t: None if t is None else ctypes.byref(t)
    return L.moe_mx_matmul(r(x), r(w), S, N, B, y, yd, ldy, ws, wb, None), L.moe_mx_matmul_workspace_bytes(r(x), r(w), S, N, B)


@pytest.mark.parametrize("bad,status", [
    (dict(S=-1), M.MOE_EINVAL), (dict(S=2 ** 24 + 1), M.MOE_EINVAL), (dict(N=0), M.MOE_EINVAL), (dict(N=2 ** 24 + 1), M.MOE_EINVAL),
    (dict(B=0), M.MOE_EINVAL), (dict(B=2 ** 20 + 1), M.MOE_EINVAL), (dict(x=None), M.MOE_ENULL), (dict(w=None), M.MOE_ENULL),
    (dict(x=rows(q=None)), M.MOE_ENULL), (dict(w=rows(e=None)), M.MOE_ENULL), (dict(x=rows(q=A + 8)), M.MOE_EINVAL),
    (dict(w=rows(ldq=72)), M.MOE_EINVAL), (dict(x=rows(lde=-4)), M.MOE_EINVAL), (dict(S=0), M.MOE_OK)])
def test_mx_matmul_refusals(bad, status):
    rc, need = matmul(**bad)
    assert rc == status and (need == status if status else need == 0)


@pytest.mark.parametrize("bad,status", [
    (dict(yd=5), M.MOE_EDTYPE), (dict(y=None), M.MOE_ENULL), (dict(ldy=2), M.MOE_EINVAL), (dict(y=A + 2), M.MOE_EINVAL)])
def test_mx_matmul_output_refusals(bad, status):
    assert matmul(**bad)[0] == status


def groups(first=A, order=None, n=5, top_k=0):
    return M.moe_groups(first, order, n, top_k)


def grouped(x=A, ldx=64, rows=9, w=A, ldw=64, expert=64 * 3, g=groups(), T=2, N=3, K=64, y=A, yd=0, ldy=3, ws=A, wb=1 << 40):
    r = None if g is None else ctypes.byref(g)
    return L.moe_grouped_matmul(x, ldx, rows, w, ldw, expert, r, T, N, K, y, yd, ldy, ws, wb, None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), M.MOE_EINVAL), (dict(T=2 ** 24 + 1), M.MOE_EINVAL), (dict(N=0), M.MOE_EINVAL), (dict(K=0), M.MOE_EINVAL),
    (dict(K=2 ** 24 + 1), M.MOE_EINVAL), (dict(rows=0), M.MOE_EINVAL), (dict(rows=-1), M.MOE_EINVAL), (dict(g=None), M.MOE_ENULL),
    (dict(g=groups(first=None)), M.MOE_ENULL), (dict(g=groups(n=0)), M.MOE_EINVAL), (dict(g=groups(n=1025)), M.MOE_EINVAL),
    (dict(g=groups(first=A + 2)), M.MOE_EINVAL), (dict(g=groups(order=A)), M.MOE_EINVAL),
    (dict(g=groups(order=A + 1, top_k=2)), M.MOE_EINVAL), (dict(x=None), M.MOE_ENULL), (dict(w=None), M.MOE_ENULL),
    (dict(x=A + 1), M.MOE_EINVAL), (dict(w=A + 1), M.MOE_EINVAL), (dict(ldx=-1), M.MOE_EINVAL), (dict(ldw=-1), M.MOE_EINVAL),
    (dict(expert=-1), M.MOE_EINVAL), (dict(y=None), M.MOE_ENULL), (dict(yd=2), M.MOE_EDTYPE), (dict(ldy=2), M.MOE_EINVAL),
    (dict(y=A + 2), M.MOE_EINVAL), (dict(T=0), M.MOE_OK)])
def test_grouped_refusals(bad, status):
    assert grouped(**bad) == status


def mx_grouped(x=rows(), n=9, w=rows(expert_q=192, expert_e=12), g=groups(), T=2, N=3, B=4, y=A, yd=0, ldy=3, ws=A, wb=1 << 40):
    r = lambda t: None if t is None else ctypes.byref(t)
    return L.moe_mx_grouped_matmul(r(x), n, r(w), r(g), T, N, B, y, yd, ldy, ws, wb, None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), M.MOE_EINVAL), (dict(N=0), M.MOE_EINVAL), (dict(B=0), M.MOE_EINVAL), (dict(n=0), M.MOE_EINVAL),
    (dict(g=None), M.MOE_ENULL), (dict(g=groups(n=2000)), M.MOE_EINVAL), (dict(x=None), M.MOE_ENULL), (dict(w=None), M.MOE_ENULL),
    (dict(w=rows(expert_q=8)), M.MOE_EINVAL), (dict(w=rows(expert_e=-1)), M.MOE_EINVAL), (dict(x=rows(ldq=8)), M.MOE_EINVAL),
    (dict(y=None), M.MOE_ENULL), (dict(yd=2), M.MOE_EDTYPE), (dict(ldy=2), M.MOE_EINVAL), (dict(T=0), M.MOE_OK)])
def test_mx_grouped_refusals(bad, status):
    assert mx_grouped(**bad) == status


def group(idx=A, S=2, k=3, E=5, first=A, order=A, place=A, ws=A, wb=1 << 30):
    return L.moe_group(idx, S, k, E, first, order, place, ws, wb, None)


@pytest.mark.parametrize("bad,status", [
    (dict(S=-1), M.MOE_EINVAL), (dict(k=0), M.MOE_EINVAL), (dict(E=0), M.MOE_EINVAL), (dict(E=1025), M.MOE_EINVAL),
    (dict(S=2 ** 23, k=3), M.MOE_EINVAL), (dict(S=2 ** 30, k=2 ** 30), M.MOE_EINVAL), (dict(idx=None), M.MOE_ENULL),
    (dict(first=None), M.MOE_ENULL), (dict(order=None), M.MOE_ENULL), (dict(place=None), M.MOE_ENULL), (dict(idx=A + 2), M.MOE_EINVAL),
    (dict(first=A + 2), M.MOE_EINVAL), (dict(order=A + 1), M.MOE_EINVAL), (dict(place=A + 2), M.MOE_EINVAL),
    (dict(S=2 ** 20, ws=None), M.MOE_ENULL), (dict(S=2 ** 20, ws=A + 2), M.MOE_EINVAL), (dict(S=2 ** 20, wb=100), M.MOE_EWORKSPACE)])
def test_group_refusals(bad, status):
    assert group(**bad) == status


def combine(z=A, zd=0, ldz=64, T=6, w=A, place=A, S=2, k=3, H=64, add=A, lda=64, y=A, yd=0, ldy=64):
    return L.moe_combine(z, zd, ldz, T, w, place, S, k, H, add, lda, y, yd, ldy, None)


@pytest.mark.parametrize("bad,status", [
    (dict(S=-1), M.MOE_EINVAL), (dict(k=0), M.MOE_EINVAL), (dict(H=0), M.MOE_EINVAL), (dict(T=-1), M.MOE_EINVAL),
    (dict(S=2 ** 23, k=3), M.MOE_EINVAL), (dict(zd=2), M.MOE_EDTYPE), (dict(yd=2), M.MOE_EDTYPE), (dict(z=None), M.MOE_ENULL),
    (dict(w=None), M.MOE_ENULL), (dict(place=None), M.MOE_ENULL), (dict(y=None), M.MOE_ENULL), (dict(z=A + 2), M.MOE_EINVAL),
    (dict(add=A + 2), M.MOE_EINVAL), (dict(y=A + 2), M.MOE_EINVAL), (dict(w=A + 2), M.MOE_EINVAL), (dict(place=A + 2), M.MOE_EINVAL),
    (dict(ldz=-1), M.MOE_EINVAL), (dict(lda=-1), M.MOE_EINVAL), (dict(ldy=63), M.MOE_EINVAL), (dict(S=0), M.MOE_OK),
    (dict(H=2 ** 30 + 1, ldy=2 ** 30 + 1), M.MOE_EINVAL)])  # columns are counted in 31 bits, whole workgroups of them
def test_combine_refusals(bad, status):
    assert combine(**bad) == status


def test_sizes_beyond_int32():
    big = 1 << 31
    for f in (lambda: M.moe_mx_quant(A, 0, 64, big, 64, 0, A, 32, A, 2, stream=0),
              lambda: M.moe_mx_values(A, 32, A, 2, 2, big, A, 0, 64, stream=0),
              lambda: M.moe_mx_matmul(rows(), rows(), 2, big, 4, A, 0, 3, None, 0, stream=0),
              lambda: M.moe_group(A, big, 3, 5, A, A, A, None, 0, stream=0),
              lambda: M.moe_grouped_matmul(A, 64, big, A, 64, 64, groups(), 2, 3, 64, A, 0, 3, None, 0, stream=0),
              lambda: M.moe_combine(A, 0, 64, big, A, A, 2, 3, 64, None, 0, A, 0, 64, stream=0)):
        with pytest.raises(M.MoeError) as err:
            f()
        assert err.value.status == M.MOE_EINVAL


u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)


@pytest.mark.parametrize("call", [
    lambda: M.mx_quant(torch.zeros(3, 4, dtype=torch.float16)), lambda: M.mx_quant(torch.zeros(4)),
    lambda: M.mx_quant(torch.zeros(4, 3).t()), lambda: M.mx_quant(torch.zeros(3, 4)),  # on the CPU
    lambda: M.mx_silu_quant(torch.zeros(3, 5)), lambda: M.mx_silu_quant(torch.zeros(3, 4), torch.zeros(3, 5)),
    lambda: M.mx_silu_quant(torch.zeros(3, 4), torch.zeros(3, 4).bfloat16()),
    lambda: M.mx_values(u8(3, 32), u8(3, 3)), lambda: M.mx_values(u8(3, 32), u8(3, 2), width=65),
    lambda: M.mx_values(u8(3, 32), u8(3, 2), width=32), lambda: M.mx_values(u8(3, 32).to(torch.int8), u8(3, 2)),
    lambda: M.mx_values(u8(3, 32), u8(3, 2), dtype=torch.float16), lambda: M.mx_values(u8(3, 32), u8(6)),
    lambda: M.mx_matmul(u8(3, 32), u8(3, 2), u8(5, 48), u8(5, 3)), lambda: M.mx_matmul(u8(3, 32), u8(3, 2), u8(5, 32), u8(4, 2)),
    lambda: M.mx_matmul(u8(3, 32), u8(3, 2), u8(5, 32), u8(5, 2), out_dtype=torch.float64),
    lambda: M.mx_matmul(u8(3, 32), u8(3, 2), u8(5, 32), u8(5, 2), ws=u8(64, 2)[:, 0]),
    lambda: M.group(i32(6), 4), lambda: M.group(i32(3, 4).long(), 4), lambda: M.group(i32(4, 3).t(), 4),
    lambda: M.grouped_matmul(bf(4, 8), bf(2, 5, 8).float(), i32(3)), lambda: M.grouped_matmul(bf(4, 8), bf(2, 5, 9), i32(3)),
    lambda: M.grouped_matmul(bf(4, 8), bf(5, 8), i32(3)), lambda: M.grouped_matmul(bf(4, 8), bf(2, 5, 8), i32(2)),
    lambda: M.grouped_matmul(bf(4, 8), bf(2, 5, 8), i32(3), order=i32(6)), lambda: M.grouped_matmul(bf(4, 8), bf(2, 5, 8), i32(3), top_k=2),
    lambda: M.grouped_matmul(bf(4, 8), bf(2, 5, 8), i32(3), order=i32(6), top_k=0),
    lambda: M.grouped_matmul(bf(4, 8), bf(2, 5, 8), i32(3), order=i32(3, 2), top_k=2),
    lambda: M.grouped_matmul(bf(4, 8), bf(2, 5, 8), i32(3).long()), lambda: M.grouped_matmul(bf(4, 8), bf(2, 8, 5).transpose(1, 2), i32(3)),
    lambda: M.grouped_matmul(bf(4, 8).requires_grad_(), bf(2, 5, 8), i32(3)),
    lambda: M.mx_grouped_matmul(u8(4, 32), u8(4, 2), u8(2, 5, 32), u8(2, 5, 3), i32(3)),
    lambda: M.mx_grouped_matmul(u8(4, 32), u8(4, 2), u8(2, 5, 16), u8(2, 5, 2), i32(3)),
    lambda: M.mx_grouped_matmul(u8(4, 32), u8(4, 2), u8(5, 32), u8(5, 2), i32(3)),
    lambda: M.combine(bf(6, 8), torch.zeros(2, 3), i32(2, 2)), lambda: M.combine(bf(6, 8), torch.zeros(2, 3).double(), i32(2, 3)),
    lambda: M.combine(bf(6, 8), torch.zeros(2, 3), i32(2, 3), add=torch.zeros(2, 8)),
    lambda: M.combine(bf(6, 8), torch.zeros(2, 3), i32(2, 3), add=bf(3, 8)), lambda: M.combine(bf(6, 8), torch.zeros(2, 3), i32(6)),
    lambda: M.combine(bf(6, 8), torch.zeros(2, 3), i32(2, 3), out_dtype=torch.float16)])
def test_binding_refusals(call):
    with pytest.raises(ValueError):
        call()


def test_reference_of_the_tests():
    """The 64-bit quantiser of the GPU tests, by hand: ties go to the even code, 6.5 is cut off, zeros have scale 0."""
    v = torch.zeros(1, 70)
    v[0, :8] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5])
    v[0, 8] = -0.3
    q, e = R.quantise(v)
    assert e.tolist() == [[127, 0, 0]]
    assert q[0, :5].tolist() == [0x20, 0x42, 0x64, 0x76, 0x09]
    q, e = R.quantise(v, up=True)
    assert e.tolist() == [[128, 0, 0]] and R.values(q, e)[0, 7] == 6.0 and R.values(q, e)[0, 6] == 4.0
    first, order, place = R.group(torch.tensor([[1, 0], [5, 1]]), 3)
    assert first.tolist() == [0, 1, 3, 3] and order.tolist() == [1, 0, 3, 2] and place.tolist() == [[1, 0], [-1, 2]]
