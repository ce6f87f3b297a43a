"""The activations' slopes relative to their own size, in the tails too."""
from __future__ import annotations

import math

import pytest
import torch

from tests import linear_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def pts():
    import persistent_tile_scheduling_amd as mod
    return mod


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_slopes_are_good_to_steps_of_their_terms(pts, act):
    """m = 1 and dy = 1: dbias is the slope. It is p + z p' with p from an exponential of u. Of u's relative error at most three
    roundings stay, |u| 2^-24 of the exponential each; the rest, reciprocals, polynomial and sums, is 16 steps."""
    z = torch.arange(65536, device=DEV, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    z = z[torch.isfinite(z)][None]
    z = torch.nn.functional.pad(z, (0, -z.shape[1] % 8))
    got = pts.linear_backward(torch.ones_like(z), None, None, z, activation=act, need_dx=False, need_dw=False).dbias.double()
    z = z[0].double()
    if act == "gelu":
        u, p, slope = z * z / 2, 0.5 * torch.special.erfc(-z / math.sqrt(2)), torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    else:
        c, d = (1.0, 0.0) if act == "silu" else (2 * math.sqrt(2 / math.pi), 0.044715)
        u = c * (z + d * z ** 3)
        p, slope = torch.sigmoid(u), torch.sigmoid(u) * torch.sigmoid(-u) * c * (1 + 3 * d * z * z)
    terms = p + (z * slope).abs()
    far = (got - R.slope(z, act)).abs()
    seen = terms > 2.0 ** -119
    steps = (far[seen] / terms[seen]) * 2.0 ** 24
    worst = (steps / (16 + 3 * u[seen].abs())).max()
    assert worst <= 1, f"{worst:.3g} times the bound"
    assert (far[~seen] <= 2.0 ** -119).all()
    assert seen.sum() > 20000
