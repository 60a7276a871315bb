"""Products whose plan is not as moe_group makes it, and gathered rows, by every kernel.

Whole numbers: bf16 products are whole, their sums below 16 K < 2^24; microscaled ones (halves times powers from 2^-1 to 2,
at most 12) are multiples of 1/16 with sums below 144 K < 2^20 up to K = 7281.  Both are exact in fp32 in any order.
"""
import pytest
import torch

import mxref as R
from int4_routed_expert_amd import moe as M
from tests.test_gpu_expert_paths import GROUPED, counts, first_of, kernels_of
from tests.test_gpu_experts import rng, whole

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


class Operands:
    """Rows and experts' weights of either kind, with their values in 64 bits."""

    def __init__(self, mx, rows, E, N, K):
        g = rng(rows + N + K)
        self.mx = mx
        if mx:
            self.x, self.w = whole(g, rows, K // 32), whole(g, E, N, K // 32)
            self.values = R.values(*self.x), R.values(*self.w)
        else:
            self.x = (torch.randint(-4, 5, (rows, K), generator=g, device="cuda").to(BF),)
            self.w = (torch.randint(-4, 5, (E, N, K), generator=g, device="cuda").to(BF),)
            self.values = self.x[0].double(), self.w[0].double()

    def call(self, first, order=None, top_k=None, **kw):
        return (M.mx_grouped_matmul if self.mx else M.grouped_matmul)(*self.x, *self.w, first, order, top_k, **kw)


# kernel, T, E, N, K, microscaled
PLANS = [("vec2", 20, 10, 1000, 1024, False), ("few16", 20, 40, 1000, 256, True), ("few16", 64, 8, 1024, 1024, False),
         ("tile32", 60, 40, 1500, 1536, True), ("tile32", 300, 10, 1000, 512, False), ("tile64", 500, 10, 2000, 1024, True),
         ("tile64", 500, 10, 2000, 1024, False), ("tile128", 2000, 20, 2000, 512, True), ("tile128", 1500, 20, 8000, 1024, True),
         ("tile128", 2000, 20, 2000, 512, False), ("tile256x128", 600, 12, 4000, 4096, True), ("tile256x128", 600, 12, 4000, 1024, False),
         ("tile256", 1500, 12, 4000, 1056, True), ("tile256", 1500, 12, 4000, 512, False)]


def through(names, kernel):
    return f"product_{kernel}" in names and names <= {f"product_{kernel}", "product_align"}


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("how", ["beyond", "below", "both", "far"])
@pytest.mark.parametrize("kernel,T,E,N,K,mx", PLANS)
def test_first_outside_the_rows(kernel, T, E, N, K, mx, how, gather):
    """first beyond T or below 0, not decreasing: taken within [0, T]; rows of no expert and memory around y as they were."""
    first = first_of(counts(T, E)).cpu()
    shift = {"beyond": T // 3, "below": -(T // 3), "both": 0, "far": 0}[how]
    first = first + shift
    if how == "both":
        first = (first - T // 2) * 2
    if how == "far":
        first[0], first[-1] = -2 ** 31, 2 ** 31 - 1
    p = Operands(mx, T, E, N, K)
    plan = (torch.randperm(2 * T, generator=rng(T), device="cuda")[:T].to(torch.int32), 2) if gather else (None, None)
    buf = torch.full((T + 40, N), 7.0, device="cuda")
    y = buf[20:20 + T]
    want = R.product(*p.values, first.clamp(0, T).tolist(), y.double(), *(plan if gather else ()))
    _, names = kernels_of(M, lambda: p.call(first.cuda(), *plan, out=y))
    assert through(names, kernel), names
    assert torch.equal(y.double(), want)
    assert (buf[:20] == 7).all() and (buf[20 + T:] == 7).all()


@pytest.mark.parametrize("how", ["swapped", "reversed", "high and low", "random"])
@pytest.mark.parametrize("kernel,T,E,N,K,mx", PLANS)
def test_first_that_decreases(kernel, T, E, N, K, mx, how):
    """Rows may belong to several experts or to none: those of none and the memory around y are as they were."""
    first = first_of(counts(T, E)).cpu()
    if how == "swapped":
        first[E // 2], first[E // 2 + 1] = int(first[E // 2 + 1]), int(first[E // 2])
    elif how == "reversed":
        first = first.flip(0)
    elif how == "high and low":
        first[0::2], first[1::2] = T // 4, T + 1000
    else:
        first = torch.randint(-T, 2 * T, (E + 1,), generator=torch.Generator().manual_seed(T), dtype=torch.int32)
    bound = first.clamp(0, T).tolist()
    of_some = torch.zeros(T, dtype=torch.bool)
    for lo, hi in zip(bound, bound[1:]):
        of_some[lo:max(lo, hi)] = True
    p = Operands(mx, T, E, N, K)
    buf = torch.full((T + 40, N), 7.0, device="cuda")
    y = buf[20:20 + T]
    _, names = kernels_of(M, lambda: p.call(first.cuda(), out=y))
    assert through(names, kernel), names
    assert (y[~of_some.cuda()] == 7).all()
    assert (buf[:20] == 7).all() and (buf[20 + T:] == 7).all()


@pytest.mark.parametrize("kernel,T,E,N,K,mx", [(name.split("/")[0 if mx else -1], T, E, N, K, mx) for name, T, E, N, *both in GROUPED
                                               for mx, K in zip((True, False), both) if K and K % (512 if mx else 8) == 0])
def test_gathered_rows_take_the_same_kernel(kernel, T, E, N, K, mx):
    """Where nothing is copied, rows that are gathered go through the kernel of rows that lie in order."""
    first = first_of(counts(T, E))
    rows = T // 3 + 2
    p = Operands(mx, rows, E, N, K)
    order = torch.randint(0, rows * 3, (T,), generator=rng(T), device="cuda").to(torch.int32)
    want = R.product(*p.values, first.tolist(), torch.zeros(T, N, dtype=torch.float64, device="cuda"), order, 3)
    got, names = kernels_of(M, lambda: p.call(first, order, 3, out_dtype=F32))
    assert names == {f"product_{kernel}"}
    assert torch.equal(got.double(), want)
