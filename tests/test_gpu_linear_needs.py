"""linear_backward with only the operands that the wanted gradients need."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pts():
    import persistent_tile_scheduling_amd as mod
    return mod


@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("m,n,k", [(40, 96, 72), (300, 64, 2200), (700, 2104, 200), (1, 8, 8), (0, 8, 8), (300, 8, 0)])
def test_only_what_is_needed(pts, m, n, k, act):
    g = torch.Generator(device="cuda").manual_seed(1)
    dy, x, w, z = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((m, n), (m, k), (n, k), (m, n)))
    whole = pts.linear_backward(dy, x, w, z if act else None, activation=act)
    for need in ((a, b, c) for a in (True, False) for b in (True, False) for c in (True, False)):
        # what is not needed is None, or anything else
        for other in (None, torch.zeros(3)):
            part = pts.linear_backward(dy, x if need[1] else other, w if need[0] else other, z if act else other, activation=act,
                                       need_dx=need[0], need_dw=need[1], need_dbias=need[2])
            for one, all_, wanted in zip(part, whole, need):
                assert (one is None) != wanted and (not wanted or torch.equal(one, all_))
