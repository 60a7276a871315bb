"""Rotary frequencies whose blend lies at an end of the pairs."""
import math

import numpy as np
import pytest

from int4_routed_expert_amd import moe as M


@pytest.mark.parametrize("R,theta", [(8, 10000.0), (64, 10000.0), (128, 500000.0), (2, 100.0)])
@pytest.mark.parametrize("L,fast,slow", [(1, 32.0, 1.0), (4, 32.0, 1.0), (6, 32.0, 1.0), (7, 32.0, 1.0), (100, 32.0, 1.0),
                                         (100, 500.0, 20.0), (1 << 30, 32.0, 1.0), (1 << 30, 2.0, 1e-9), (1 << 30, 1e9, 2e8)])
def test_blend_at_the_ends(R, theta, L, fast, slow):
    """A pair that turns at least `fast` times in L keeps its frequency, one that turns at most `slow` times has it divided,
    also where that is every pair or none.  (Pairs within an index of the rounded ends aside, unless they lie beyond the
    first pair or the last.)"""
    scale = 4.0
    f, m = M.moe_rope_freqs(R, theta, M.MOE_ROPE_YARN, scale, L, fast, slow)
    plain = np.array([theta ** (-2 * i / R) for i in range(R // 2)])
    turns = L * plain / (2 * math.pi)
    ratio = f / plain
    assert abs(m - (0.1 * math.log(scale) + 1)) < 1e-7
    assert np.all((ratio <= 1 + 1e-14) & (ratio >= 1 / scale - 1e-14)) and np.all(np.diff(ratio) <= 1e-14)
    index = theta ** (2 / R)
    keeps, divided = turns >= fast * index, turns <= slow / index
    if turns[0] <= slow:
        divided[:] = True
    if turns[-1] >= fast:
        keeps[:] = True
    assert np.allclose(ratio[keeps], 1.0, rtol=1e-14) and np.allclose(ratio[divided], 1 / scale, rtol=1e-14)
