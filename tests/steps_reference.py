"""Newton-Schulz steps of matrices with a short side: in 64 bits, in 32 bits with a Gram matrix made from X at every step,
and as chains of a Gram matrix that follows several steps by itself.

The last is how the library takes short sides; the second is what it is measured by. Two fp32 forms of the same steps
make rounding errors of the same size in each step, and these pass through the same steps that remain, so their distances
from the exact result are alike; a factor of 8 leaves room for chance.
"""
from __future__ import annotations

import torch

QUINTIC = (3.4445, -4.7750, 2.0315)
CUBIC = (1.5, -0.5, 0.0)
MATRICES = ["wide", "square", "rank 5", "rows sum to 0", "condition 1e4", "tall"]
HALF_BF16 = 2.0 ** -8


def matrix(kind):
    g = torch.Generator().manual_seed(1)

    def normal(*shape):
        return torch.randn(shape, generator=g)
    if kind == "wide":
        return normal(20, 300)
    if kind == "square":
        return normal(64, 64)
    if kind == "tall":
        return normal(700, 33)
    if kind == "rank 5":
        return normal(40, 5) @ normal(5, 400)
    if kind == "rows sum to 0":             # the gradient of a softmax's weight
        x = normal(10, 512)
        return x - x.mean(0, keepdim=True)
    u, v = torch.linalg.qr(normal(30, 30))[0], torch.linalg.qr(normal(200, 30))[0]
    return u @ torch.diag(torch.logspace(0, -4, 30)) @ v.t()


def start(x):
    x = x.float().cpu()
    x = x if x.shape[0] <= x.shape[1] else x.t()
    x = x.double()
    return (x / (x.norm() + 1e-7)).float()


def follow(x, steps, coefficients, per=1, gram=torch.float32):
    """The steps on the short side's left, X in fp32 and a Gram matrix of type `gram` made anew every `per` steps."""
    a, b, c = coefficients
    x = start(x)
    if gram is None:                        # the definition: everything in 64 bits
        x, gram = x.double(), torch.float64
    one = torch.eye(x.shape[0], dtype=gram)
    for i in range(0, steps, per):
        y = x.to(gram)
        m = y @ y.t()
        for _ in range(min(per, steps - i)):
            poly = b * m + c * (m @ m)
            x = a * x + poly.to(x.dtype) @ x
            q = poly + a * one
            m = q @ (q @ m)
    return x


def distances(x, y, steps, coefficients):
    """Of a result y (short side first) from the exact one, relative: altogether, and in the directions that x has."""
    exact = follow(x, steps, coefficients, gram=None)
    off = y.double().cpu() - exact
    u, s, _ = torch.linalg.svd(start(x).double(), full_matrices=False)
    u = u[:, s > 1e-6]
    return off.norm() / exact.norm(), (u.t() @ off).norm() / exact.norm()


def check(x, y, steps, coefficients, rounding):
    """y is finite, within the map's reach, and as near to the exact steps as fp32 steps that make A from X each time."""
    assert torch.isfinite(y).all(), "not finite"
    top = 1.21 if coefficients == QUINTIC else 1.0      # p on [0, 1.21] and on [0, 1]
    largest = torch.linalg.matrix_norm(y.double().cpu(), ord=2)
    assert largest <= top * (1 + 1e-4) + rounding * y.double().norm(), f"a singular value of {largest:.4g}"
    near = follow(x, steps, coefficients)
    for have, allowed in zip(distances(x, y, steps, coefficients), distances(x, near, steps, coefficients)):
        assert have <= 8 * allowed + 2 * rounding, f"{have:.3g} off, where fp32 steps are {allowed:.3g}"
