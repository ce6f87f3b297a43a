"""The linear layer's operators in 64 bits, and bounds on how far a kernel may be off.

A sum of k products in fp32, in any order, is within k 2^-24 times the sum of the
products' magnitudes; a rounding is off by at most half a step of its type.
"""
from __future__ import annotations

import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
ACTIVATIONS = [None, "relu", "gelu", "gelu_tanh", "silu"]
QUINTIC = (3.4445, -4.7750, 2.0315)


def activation(z, kind):
    if kind is None:
        return z
    if kind == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if kind == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if kind == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z)


def slope(z, kind):
    if kind is None:
        return torch.ones_like(z)
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        p = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        q = torch.sigmoid(-c * (z + 0.044715 * z ** 3))
        return p + z * p * q * c * (1 + 3 * 0.044715 * z * z)
    return torch.sigmoid(z) * (1 + z * torch.sigmoid(-z))


def linear(x, w, bias=None, act=None, residual=None):
    """(y, z, bound of y's sums, bound of z's): 64 bits; the bounds are for fp32 results, before their rounding.

    An activation's slope is at most 1.13. Its own error is 16 steps of its value and, from its exponential's argument u
    (z, 1.6 z + 0.0714 z^3, z^2 / 2), whose at most three roundings stay in the result, 3 |u| more; left of -88 it is 0."""
    x, w = x.double(), w.double()
    z = x @ w.t()
    mass = x.abs() @ w.abs().t()
    if bias is not None:
        z, mass = z + bias.double(), mass + bias.double().abs()
    y = activation(z, act)
    bound_z = (x.shape[1] + 1) * HALF[torch.float32] * mass
    u = {None: 0 * z, "relu": 0 * z, "silu": z, "gelu": z * z / 2, "gelu_tanh": 1.6 * z + 0.0714 * z ** 3}[act].abs()
    u = torch.where(y.abs() > 2.0 ** -119, u, torch.zeros_like(u)).clamp(max=128)
    bound_y = 1.13 * bound_z + (16 + 3 * u) * HALF[torch.float32] * y.abs() + 2.0 ** -119
    if residual is not None:
        y = y + residual.double()
        bound_y = bound_y + HALF[torch.float32] * y.abs()
    return y, z, bound_y, bound_z


def slope_bound(dy, z, act):
    """dz = dy act'(z), and how far its fp32 value may be off: a slope is good to 64 steps of one, and with gelu_tanh to
    2^-24 of its logistic's argument u, which the logistic (its slope with 2 sqrt(2 / pi) (|z| + 3 0.044715 |z|^3)) carries."""
    dy = dy.double()
    if act is None:
        return dy, torch.zeros_like(dy)
    z = z.double()
    steps = torch.full_like(z, 64.0)
    if act == "gelu_tanh":
        a = z.abs().clamp(max=16)
        u = 1.6 * (a + 0.045 * a ** 3)
        p = torch.sigmoid(-u)
        steps = steps + 4 * u * (p + p * 1.6 * (a + 0.135 * a ** 3))
    s = slope(z, act)
    return dy * s, dy.abs() * steps * HALF[torch.float32] * torch.ones_like(s)


def gradients(dy, x, w, z=None, act=None):
    """(dx, dw, dbias, bound of each in fp32): dz's own rounding to bf16, with an activation, is part of the first two."""
    x, w = x.double(), w.double()
    m, n = dy.shape
    fp32 = HALF[torch.float32]
    dz, off = slope_bound(dy, z, act)
    mass = dz.abs() + off
    rounded = off if act is None else off + HALF[torch.bfloat16] * mass
    dx, dw = dz @ w, dz.t() @ x
    bound_dx = rounded @ w.abs() + (n + 1) * fp32 * (mass @ w.abs())
    bound_dw = rounded.t() @ x.abs() + (m + 1) * fp32 * (mass.t() @ x.abs())
    return dx, dw, dz.sum(0), bound_dx, bound_dw, off.sum(0) + (m + 1) * fp32 * mass.sum(0)


def check(got, want, bound, what=""):
    """Every element within its bound, and half a step of its type's rounding."""
    assert got.shape == want.shape, f"{what}: {tuple(got.shape)} != {tuple(want.shape)}"
    if not got.numel():
        return
    far = (got.double() - want).abs()
    allowed = bound + HALF[got.dtype] * (want.abs() + bound) + 1e-40
    assert torch.isfinite(got).all(), f"{what}: not finite"
    worst = (far / allowed).max().item()
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound at {(far / allowed).argmax().item()} of {tuple(got.shape)}"


def orthogonalize(x, steps=5, coefficients=QUINTIC, eps=1e-7, rounded=False):
    """The steps in 64 bits; rounded: with the kernel's roundings, of the products' operands to fp16 and of the matrix to
    fp16 and what that is short of it in e4m3 (to fp16 alone before the last step)."""
    a, b, c = coefficients
    x = x.double()
    x = x / (x.square().sum((-1, -2), keepdim=True).sqrt() + eps)
    tall = x.shape[-2] > x.shape[-1]
    rounded = rounded and min(x.shape[-2:]) > 64    # shorter sides are fp32 throughout

    def half(v, scale):
        return (v * scale).half().double() / scale if rounded else v

    for i in range(steps):
        h = half(x, 1024.0)
        gram = half(h.transpose(-1, -2) @ h if tall else h @ h.transpose(-1, -2), 256.0)
        poly = half(b * gram + c * (gram @ gram), 256.0)
        x = a * x + (h @ poly if tall else poly @ h)
        if rounded and i + 1 < steps:
            whole = half(x, 1024.0)
            rest = ((x - whole) * 2.0 ** 19).clamp(-448, 448).to(torch.float8_e4m3fn).double() / 2.0 ** 19
            x = whole + rest if i + 2 < steps else whole
    return x
