"""Products at the limits of one launch: more workgroups than it holds, so that the weight rows go in pieces."""
import pytest
import torch

import mxref as R
from tests.test_gpu_experts import rng, whole
from int4_routed_expert_amd import moe as M

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


# S x N outputs of one block of K each: tiles of 16 x 16 by 512 threads are 2^32 threads in all, or just below and above it
@pytest.mark.parametrize("S,N,launches", [(512, 1 << 22, 2), (128, 1 << 24, 2), (100, (1 << 24) - 3, 1), (520, (1 << 22) + 7, 2)])
def test_weight_rows_in_pieces(S, N, launches):
    g = rng(N)
    q, e = whole(g, S, 1)
    w, ew = whole(g, N, 1)
    M.moe_profile_enable(True)
    try:
        y = M.mx_matmul(q, e, w, ew)
        torch.cuda.synchronize()
        ran = M.moe_profile_report()
    finally:
        M.moe_profile_enable(False)
    assert ran["product_few16"][1] == launches and len(ran) == 1
    a = R.values(q, e)
    step = 1 << 20
    for n in range(0, N, step):  # products are multiples of 1/16, their sums below 2^20: exact in any order
        want = a @ R.values(w[n:n + step], ew[n:n + step]).t().contiguous()
        assert torch.equal(y[:, n:n + step], want.to(BF))
        del want
