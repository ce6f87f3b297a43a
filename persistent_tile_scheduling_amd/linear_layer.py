"""Python binding of the linear layer's operators (``include/pts_linear.h``).

Argument marshalling only, like the package's GEMM binding: the ``pts_*``
functions carry the C ABI's names and take pointers (or tensors) and sizes; the
others take torch tensors, check them (``ValueError``) and allocate their
results and workspaces.

Tensors must be on the current GPU. Work is enqueued on the current stream and
nothing is kept between calls; every call may be recorded into a HIP graph.
There is no autograd here: gradients are functions of their own.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch

from . import GEMM_DTYPE_BF16, GEMM_DTYPE_F32, _check, _lib, _ptr, _stream_handle
from .experts import _device, _expect

PTS_ACTIVATION_NONE = 0
PTS_ACTIVATION_RELU = 1
PTS_ACTIVATION_GELU = 2
PTS_ACTIVATION_GELU_TANH = 3
PTS_ACTIVATION_SILU = 4

_P, _I, _L, _F, _D, _Z = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double,
                          ctypes.c_size_t)
_SIGNATURES = {
    "pts_linear_workspace": (_L, [_L, _L, _L]),
    "pts_linear": (ctypes.c_int, [_P, _L, _P, _L, _P, _I, _I, _P, _L, _P, _L, _I, _P, _L, _L, _L, _L, _P, _Z, _P]),
    "pts_linear_backward_workspace": (_L, [_L, _L, _L, _I]),
    "pts_linear_backward": (ctypes.c_int, [_P, _L, _P, _L, _I, _P, _L, _P, _L, _P, _L, _P, _L, _I, _P, _L, _L, _L, _P,
                                           _Z, _P]),
    "pts_orthogonalize_workspace": (_L, [_L, _L, _L, _I]),
    "pts_orthogonalize": (ctypes.c_int, [_P, _I, _L, _L, _L, _L, _L, _I, _F, _F, _F, _D, _P, _L, _L, _P, _Z, _P]),
}
for _name, (_res, _args) in _SIGNATURES.items():
    getattr(_lib, _name).restype = _res
    getattr(_lib, _name).argtypes = _args


# ---------------------------------------------------------------------------
# C ABI, same names (the stream, last, defaults to the current one)
# ---------------------------------------------------------------------------

def _call(name, args, stream):
    _check(getattr(_lib, name)(*[_ptr(a) if isinstance(a, torch.Tensor) else a for a in args], _stream_handle(stream)))


def pts_linear_workspace(m: int, n: int, k: int) -> int:
    return _lib.pts_linear_workspace(m, n, k)


def pts_linear(*args, stream=None) -> None:
    _call("pts_linear", args, stream)


def pts_linear_backward_workspace(m: int, n: int, k: int, activation: int) -> int:
    return _lib.pts_linear_backward_workspace(m, n, k, activation)


def pts_linear_backward(*args, stream=None) -> None:
    _call("pts_linear_backward", args, stream)


def pts_orthogonalize_workspace(count: int, rows: int, cols: int, steps: int) -> int:
    return _lib.pts_orthogonalize_workspace(count, rows, cols, steps)


def pts_orthogonalize(*args, stream=None) -> None:
    _call("pts_orthogonalize", args, stream)


# ---------------------------------------------------------------------------
# Tensors
# ---------------------------------------------------------------------------

_BF16, _F32 = torch.bfloat16, torch.float32
_DTYPES = {_BF16: GEMM_DTYPE_BF16, _F32: GEMM_DTYPE_F32}
_VALUES = tuple(_DTYPES)
_ACTIVATIONS = {None: PTS_ACTIVATION_NONE, "relu": PTS_ACTIVATION_RELU, "gelu": PTS_ACTIVATION_GELU,
                "gelu_tanh": PTS_ACTIVATION_GELU_TANH, "silu": PTS_ACTIVATION_SILU}
_raw_stream = torch._C._cuda_getCurrentRawStream
_empty = torch.empty_strided
_linear, _backward, _orthogonalize = _lib.pts_linear, _lib.pts_linear_backward, _lib.pts_orthogonalize
# Sizes alone decide a workspace's bytes: the call into the library is made once for each.
_linear_workspace = functools.lru_cache(1024)(_lib.pts_linear_workspace)
_backward_workspace = functools.lru_cache(1024)(_lib.pts_linear_backward_workspace)
_orthogonalize_workspace = functools.lru_cache(1024)(_lib.pts_orthogonalize_workspace)


def _operand(name, t) -> int:
    """Row stride of a bf16 matrix that a product reads."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _BF16 or t.dim() != 2:
        _expect(name, t, (_BF16,), (None, None))
    rows, width = t.shape
    if not rows or not width:
        return (width + 7) // 8 * 8
    row, col = t.stride()
    if (col != 1 and width > 1) or (rows > 1 and (row < width or row % 8)) or t.data_ptr() % 16:
        raise ValueError(f"{name} must have unit stride along its rows, a row stride that is a multiple of 8 and at "
                         f"least its width, and start 16-byte aligned, not strides {t.stride()} at {t.data_ptr():#x}")
    return row if rows > 1 else (width + 7) // 8 * 8


def _pitch(name, t) -> int:
    """Row stride of a matrix that is added or written."""
    rows, width = t.shape[-2:]
    if not rows or not width:
        return width
    row, col = t.stride(-2), t.stride(-1)
    if (col != 1 and width > 1) or (rows > 1 and row < width):
        raise ValueError(f"{name} must have unit stride along its rows and rows that do not overlap, not strides "
                         f"{t.stride()}")
    return row if rows > 1 else width


def _padded(m, n, dtype, device):
    """An (m, n) result whose rows start at whole 16 bytes, and its row stride. What the last row lacks to a whole piece,
    up to the next 16 bytes, belongs to the allocation, whose size is a multiple of more."""
    ld = (n + 7) // 8 * 8
    return _empty((m, n), (ld, 1), dtype=dtype, device=device), ld


def _work(need, device):
    return _empty((need,), (1,), dtype=torch.uint8, device=device) if need else None


def _activation(name) -> int:
    try:
        return _ACTIVATIONS[name]
    except (KeyError, TypeError):
        raise ValueError(f"activation must be one of {list(_ACTIVATIONS)}, not {name!r}") from None


def linear(x: torch.Tensor, w: torch.Tensor, bias: torch.Tensor | None = None, activation: str | None = None,
           residual: torch.Tensor | None = None, out_dtype=torch.bfloat16, preactivation: bool = False,
           out: torch.Tensor | None = None):
    """``y = activation(x w^T + bias) + residual``, or ``(y, z)`` with
    ``z = x w^T + bias`` in bf16 if ``preactivation`` (what
    :func:`linear_backward` takes).

    ``x``: (m, k) and ``w``: (n, k) bf16, as for :func:`gemm` (row strides multiples
    of 8, first elements 16-byte aligned). ``bias``: (n) bf16 or fp32.
    ``activation``: None, "relu", "gelu", "gelu_tanh" or "silu". ``residual``:
    (m, n) of ``y``'s dtype. ``y``: (m, n) bf16 or fp32 (``out_dtype``), rounded once
    from fp32; ``out`` is written in place when given (it may be ``residual``, and
    must not share memory with another operand, not checked). New results have
    rows of whole 16 bytes, so that they can be operands again.
    """
    ldx, ldw = _operand("x", x), _operand("w", w)
    m, k = x.shape
    n = w.shape[0]
    if w.shape[1] != k:
        raise ValueError(f"x and w have {k} and {w.shape[1]} columns")
    act = _activation(activation)
    if bias is not None and (not isinstance(bias, torch.Tensor) or bias.dtype not in _DTYPES or bias.shape != (n,)
                             or (n > 1 and bias.stride(0) != 1)):
        _expect("bias", bias, _VALUES, (n,))
        raise ValueError("bias must be contiguous")
    if out is not None:
        _expect("out", out, _VALUES, (m, n))
        dtype = out.dtype
    elif out_dtype not in _DTYPES:
        raise ValueError(f"out_dtype must be float32 or bfloat16, not {out_dtype}")
    else:
        dtype = out_dtype
    if residual is not None and (not isinstance(residual, torch.Tensor) or residual.dtype is not dtype or residual.shape != (m, n)):
        _expect("residual", residual, (dtype,), (m, n))
    dev = _device(x, w, bias, residual, out)
    y, ldy = _padded(m, n, dtype, x.device) if out is None else (out, _pitch("out", out))
    r = ldr = 0
    if residual is not None:
        r, ldr = residual.data_ptr(), _pitch("residual", residual)
    z, zp, ldz = None, None, 0
    if preactivation:
        z, ldz = _padded(m, n, _BF16, x.device)
        zp = z.data_ptr()
    need = _linear_workspace(m, n, k)
    work = _work(need, x.device)
    status = _linear(x.data_ptr(), ldx, w.data_ptr(), ldw, None if bias is None else bias.data_ptr(),
                     0 if bias is None else _DTYPES[bias.dtype], act, r or None, ldr, y.data_ptr(), ldy, _DTYPES[dtype],
                     zp, ldz, m, n, k, None if work is None else work.data_ptr(), need, _raw_stream(dev))
    if status:
        _check(status)
    return (y, z) if preactivation else y


class LinearGradients(NamedTuple):
    """What :func:`linear_backward` returns; None where a gradient was not asked for."""
    dx: torch.Tensor | None     # (m, k) bf16
    dw: torch.Tensor | None     # (n, k)
    dbias: torch.Tensor | None  # (n) fp32


def linear_backward(dy: torch.Tensor, x: torch.Tensor | None, w: torch.Tensor | None, z: torch.Tensor | None = None,
                    activation: str | None = None, dw_dtype=torch.bfloat16, need_dx: bool = True,
                    need_dw: bool = True, need_dbias: bool = True) -> LinearGradients:
    """The gradients of :func:`linear` from ``dy`` (m, n), bf16:
    ``dz = dy activation'(z)``, ``dx = dz w``, ``dw = dz^T x`` and ``dbias``, the sum of
    dz's rows. The residual's gradient is ``dy`` itself.

    ``x``, ``w``, ``activation``: as in the forward call; ``z``: (m, n) bf16, its
    preactivation. ``x`` is for dw only, ``w`` for dx, ``z`` for an activation; they
    are not looked at otherwise and may be None. All have row strides that are
    multiples of 8 and start 16-byte aligned, as :func:`linear` leaves its results.
    ``dw_dtype``: bf16 or fp32. The products take dz rounded to bf16; dbias (fp32)
    is summed from the unrounded one. A gradient that is not needed is not computed.
    """
    ld_dy, xp, wp, ldx, ldw, k = _operand("dy", dy), None, None, 0, 0, 0
    m, n = dy.shape
    if need_dw:
        ldx, xp, k = _operand("x", x), x.data_ptr(), x.shape[1]
    if need_dx:
        ldw, wp, k = _operand("w", w), w.data_ptr(), w.shape[1]
    if (need_dw and x.shape != (m, k)) or (need_dx and w.shape[0] != n):
        raise ValueError("dy {}, x {} and w {} do not fit together".format(
            tuple(dy.shape), *(tuple(t.shape) if need else None for t, need in ((x, need_dw), (w, need_dx)))))
    act, zp, ldz = _activation(activation), None, 0
    if act:
        ldz = _operand("z", z)
        if z.shape != (m, n):
            _expect("z", z, (_BF16,), (m, n))
        zp = z.data_ptr()
    if dw_dtype not in _DTYPES:
        raise ValueError(f"dw_dtype must be float32 or bfloat16, not {dw_dtype}")
    dev, device = _device(dy, x if need_dw else None, w if need_dx else None, z if act else None), dy.device
    dx = dw = dbias = None
    ld_dx = ld_dw = 0
    if need_dx:
        dx, ld_dx = _padded(m, k, _BF16, device)
    if need_dw:
        dw, ld_dw = _padded(n, k, dw_dtype, device)
    if need_dbias:
        dbias = _empty((n,), (1,), dtype=_F32, device=device)
    need = _backward_workspace(m, n, k, act if need_dx or need_dw else PTS_ACTIVATION_NONE)
    work = _work(need, device)
    status = _backward(dy.data_ptr(), ld_dy, zp, ldz, act, xp, ldx, wp, ldw,
                       dx.data_ptr() if need_dx else None, ld_dx, dw.data_ptr() if need_dw else None, ld_dw,
                       _DTYPES[dw_dtype], dbias.data_ptr() if need_dbias else None, m, n, k,
                       None if work is None else work.data_ptr(), need, _raw_stream(dev))
    if status:
        _check(status)
    return LinearGradients(dx, dw, dbias)


def _turned(t) -> bool:
    """Whether a matrix (each of a stack) has contiguous columns and not rows; a single strided row counts as columns."""
    return t.shape[-1] > 1 and t.stride(-1) != 1 and (t.stride(-2) == 1 or t.shape[-2] == 1)


def _apart(t) -> bool:
    """Whether no two matrices of a stack share an element (one after the other, or between each other's rows)."""
    if t.dim() < 3 or t.shape[0] < 2 or not t.numel():
        return True
    (rows, row), (width, _) = sorted(zip(t.shape[-2:], t.stride()[-2:]), key=lambda d: -d[1])
    step = t.stride(0)
    return step >= (rows - 1) * row + width or (step >= width and row >= (t.shape[0] - 1) * step + width)


def orthogonalize(x: torch.Tensor, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), eps: float = 1e-7,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """``steps`` Newton-Schulz steps from ``x / (|x|_F + eps)`` towards its orthogonal
    factor (the update of a weight that the Muon optimiser takes), in bf16: each
    maps the singular values s to ``a s + b s^3 + c s^5``, the ``coefficients``.

    ``x``: (rows, cols), or (count, rows, cols): a stack of matrices, each by
    itself; bf16 or fp32, rows or columns contiguous. ``out``: bf16, of ``x``'s shape,
    rows or columns contiguous (where not the same as ``x``'s, it takes a copy),
    written in place when given, must not share memory with ``x`` (not checked).
    Up to 64 rows or columns all is fp32 or more; beyond, the products are of fp16
    operands and the matrix itself has eight bits more. The coefficients must keep
    the singular values of [0, 1], with the steps' roundings, below 8 (the defaults: 1.2).
    """
    if not isinstance(x, torch.Tensor) or x.dtype not in _DTYPES or x.dim() not in (2, 3):
        _expect("x", x, _VALUES, (None, None))
    if out is not None:
        _expect("out", out, (_BF16,), x.shape)
    if steps not in range(1, 65):     # 5.0 and other types' whole numbers are in it
        raise ValueError(f"steps must be a whole number in [1, 64], not {steps!r}")
    steps = int(steps)
    dev = _device(x, out)
    rows, cols = x.shape[-2:]
    if out is not None and _turned(x) != _turned(out) and rows > 1:
        _pitch("out", out.transpose(-1, -2) if _turned(out) else out)
        if not _apart(out):
            raise ValueError(f"out's matrices overlap (strides {out.stride()})")
        return out.copy_(orthogonalize(x, steps, coefficients, eps))
    if _turned(x) or (out is not None and _turned(out)):    # the factor of a transpose is the transpose of the factor
        y = orthogonalize(x.transpose(-1, -2), steps, coefficients, eps, None if out is None else out.transpose(-1, -2))
        return y.transpose(-1, -2) if out is None else out
    if out is None:
        out = torch.empty(x.shape, dtype=_BF16, device=x.device)
    ldx, ldo = _pitch("x", x), _pitch("out", out)
    count = x.shape[0] if x.dim() == 3 else 1
    a, b, c = map(float, coefficients)
    need = _orthogonalize_workspace(count, rows, cols, steps)
    work = _work(need, x.device)
    status = _orthogonalize(x.data_ptr(), _DTYPES[x.dtype], ldx, x.stride(0) if count > 1 else 0, count, rows, cols,
                            steps, a, b, c, float(eps), out.data_ptr(), ldo, out.stride(0) if count > 1 else 0,
                            None if work is None else work.data_ptr(), need, _raw_stream(dev))
    if status:
        _check(status)
    return out
