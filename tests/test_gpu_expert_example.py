"""examples/expert_layer.py: every product of the layer is one of the library's."""
import os
import sys

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

PRODUCTS = {"mm", "addmm", "bmm", "baddbmm", "mv", "addmv", "dot", "linear", "_scaled_mm", "_grouped_mm"}


class Names(TorchDispatchMode):
    """The torch operations that run inside."""

    def __init__(self):
        super().__init__()
        self.seen = set()

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.seen.add(func.overloadpacket.__name__)
        return func(*args, **(kwargs or {}))


@pytest.mark.parametrize("mx", [False, True])
def test_products_are_the_library_s(mx):
    import expert_layer as X
    layer = X.Layer(mx)
    x = torch.randn(5, layer.c.hidden, generator=torch.Generator(device="cuda").manual_seed(0), device="cuda").to(torch.bfloat16)
    with Names() as names:
        layer.forward(x)
    assert names.seen and not names.seen & PRODUCTS


def test_a_product_of_torch_s_is_seen():
    a = torch.ones(3, 4, device="cuda")
    with Names() as names:
        a @ a.t()
    assert names.seen & PRODUCTS
