"""perf/more_operators.py: what its library form hands to the calls, and that both forms compute the same on small cases.

Bound of floating outputs, in the 2-norm and relative to that of the 64-bit values: a bf16 output is rounded by at most
2^-8 of itself; sums of K <= 256 products are off by at most (144 + K / 16) 2^-23 sum |x w| (test_gpu_experts.py), and the
norm of sum |x w| is below sqrt(K) = 16 times that of the sums of such numbers: 3.1e-4.  Together below 2^-7, and without
the rounding below 2^-11.
"""
import importlib.util
import os

import pytest
import torch

from int4_routed_expert_amd import moe as M

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def cases():
    spec = importlib.util.spec_from_file_location("more_operators", os.path.join(ROOT, "perf", "more_operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def codes(cases, *shape):
    """Codes and scales as a state has them."""
    g = torch.Generator().manual_seed(len(shape))
    c, e = cases._plain_codes(torch.randn(*shape, 32, generator=g), False)
    return c.flatten(-2), e.squeeze(-1)


@pytest.mark.parametrize("op", ["mx", "mxgroup"])
def test_calls_take_bytes(cases, monkeypatch, op):
    """The calls are made with the codes' values as the bytes that the library takes."""
    q, e = codes(cases, 4, 3)
    w, ew = codes(cases, 5, 3) if op == "mx" else codes(cases, 2, 5, 3)
    state = {"case": {"op": op, "out": "bf16", "gather": False}, "q": q, "e": e, "w": w if op == "mx" else w.to(torch.uint8), "ew": ew,
             "first": torch.zeros(3, dtype=torch.int32)}
    seen = []
    monkeypatch.setattr(M, "mx_matmul", lambda *a, **kw: seen.append(a))
    monkeypatch.setattr(M, "mx_grouped_matmul", lambda *a, **kw: seen.append(a))
    cases.own = True
    cases.run(state)
    for got, given in zip(seen[0][:4], (q, e, w, ew)):
        assert got.dtype == torch.uint8 and torch.equal(got.long(), given.long())
    assert M._codes(*seen[0][:2], "q")[:2] == (4, 3)


SMALL = [
    {"op": "quant", "S": 5, "H": 70, "silu": False, "up": True, "dtype": "bf16", "pad": 3},
    {"op": "quant", "S": 4, "H": 64, "silu": True, "up": False, "dtype": "f32", "pad": 0},
    {"op": "mx", "S": 1, "N": 33, "blocks": 8, "out": "bf16", "pad": 0},
    {"op": "mx", "S": 70, "N": 65, "blocks": 5, "out": "f32", "pad": 3},
    {"op": "grouped", "S": 40, "k": 3, "E": 7, "N": 50, "K": 200, "gather": True, "out": "bf16"},
    {"op": "grouped", "S": 9, "k": 2, "E": 4, "N": 64, "K": 64, "gather": False, "out": "f32"},
    {"op": "mxgroup", "S": 40, "k": 3, "E": 7, "N": 50, "K": 200, "gather": False, "out": "f32"},
    {"op": "mxgroup", "S": 1, "k": 4, "E": 9, "N": 64, "K": 128, "gather": True, "out": "bf16"},
    {"op": "dispatch", "S": 30, "k": 3, "E": 7, "H": 100, "dropped": True, "add": True, "dtype": "bf16", "out": "f32"}]


@pytest.mark.gpu
@pytest.mark.parametrize("case", SMALL, ids=lambda c: f"{c['op']}-{c['S']}")
def test_both_forms_agree(cases, case):
    as_list = lambda v: list(v) if isinstance(v, (tuple, list)) else [v]
    want = as_list(cases.exact(case, 3))
    for own in (False, True):
        cases.own = own
        got = as_list(cases.run(cases.prepare(case, 3)))
        assert len(got) == len(want)
        for a, b in zip(got, want):
            assert a.shape == b.shape
            if not a.is_floating_point():
                assert torch.equal(a.long(), b.long())
            else:
                off = ((a.double() - b.double()).norm() / b.double().norm()).item()
                assert off <= (2.0 ** -7 if a.dtype == torch.bfloat16 else 2.0 ** -11), (own, off)
