"""Short sides' Newton-Schulz steps as chains of the Gram matrix, on the CPU: what a chain in 64 bits may do, and that one in
32 bits, or one that never ends, is seen."""
from __future__ import annotations

import pytest
import torch

from tests import steps_reference as S


@pytest.mark.parametrize("steps", [1, 5, 8, 10, 20, 64])
@pytest.mark.parametrize("kind", S.MATRICES)
@pytest.mark.parametrize("coefficients,per", [(S.QUINTIC, 8), (S.CUBIC, 16)])
def test_chains_in_64_bits_are_as_near_as_steps(kind, coefficients, per, steps):
    """A chain does not see X's own rounding, which is below 2^-6 at its end: its square is missing in A, where it counts by
    |q'| top <= 4.775 1.21 < 2^2.6. So it is 2^-9.4 off at most, a third of a rounding to bf16."""
    x = S.matrix(kind)
    S.check(x, S.follow(x, steps, coefficients, per, torch.float64), steps, coefficients, 2.0 ** -10.4)


@pytest.mark.parametrize("kind,coefficients,steps,per,gram", [
    ("rank 5", S.QUINTIC, 10, 64, torch.float32), ("rank 5", S.CUBIC, 64, 64, torch.float32),
    ("condition 1e4", S.QUINTIC, 8, 64, torch.float32), ("condition 1e4", S.CUBIC, 40, 64, torch.float32),
    ("rank 5", S.QUINTIC, 40, 64, torch.float64),
])
def test_chains_that_run_away_are_seen(kind, coefficients, steps, per, gram):
    x = S.matrix(kind)
    with pytest.raises(AssertionError):
        S.check(x, S.follow(x, steps, coefficients, per, gram), steps, coefficients, S.HALF_BF16)
