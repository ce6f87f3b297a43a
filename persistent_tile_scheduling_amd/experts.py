"""Python binding of the routed-experts operators (``include/pts_experts.h``).

Argument marshalling only, like the package's GEMM binding: the ``pts_*``
functions carry the C ABI's names and take pointers (or tensors) and sizes; the
others take torch tensors, check them (``ValueError``) and allocate their
results.

Tensors must be on the current GPU. Work is enqueued on the current stream and
nothing is kept between calls; every call may be recorded into a HIP graph.
There is no autograd here: gradients are functions of their own.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import (GEMM_COL_MAJOR, GEMM_DTYPE_BF16, GEMM_DTYPE_F32, GEMM_ROW_MAJOR, _check, _lib, _ptr,
               _stream_handle)

PTS_FP8_BLOCK = 128
PTS_MOE_MAX_EXPERTS = 1024
PTS_MOE_MAX_TOP = 32
PTS_MOE_MAX_GROUPS = 64
PTS_SCORE_SOFTMAX = 0
PTS_SCORE_SIGMOID = 1

_P, _I, _L, _F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_SIGNATURES = {
    "pts_quantize_fp8": (ctypes.c_int, [_P, _I, _I, _L, _L, _L, _I, _I, _P, _L, _P, _L, _L, _P]),
    "pts_gemm_fp8": (ctypes.c_int, [_P, _L, _P, _L, _L, _P, _L, _P, _L, _L, _I, _P, _L, _I, _L, _L, _L, _P]),
    "pts_gemm_fp8_experts": (ctypes.c_int, [_P, _L, _L, _P, _L, _L, _P, _L, _L, _P, _L, _L, _L, _I, _P, _P, _P, _L, _I,
                                            _L, _L, _L, _P]),
    "pts_moe_route_workspace": (_L, [_L, _I, _I]),
    "pts_moe_route": (ctypes.c_int, [_P, _I, _L, _P, _L, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _P, _P, _P,
                                     ctypes.c_size_t, _P]),
    "pts_moe_route_backward": (ctypes.c_int, [_P, _P, _I, _L, _P, _L, _I, _I, _I, _I, _F, _P, _L, _P]),
    "pts_moe_combine": (ctypes.c_int, [_P, _I, _L, _L, _P, _P, _L, _L, _I, _P, _L, _P]),
    "pts_moe_combine_backward": (ctypes.c_int, [_P, _L, _P, _I, _L, _L, _P, _P, _L, _L, _I, _P, _L, _P, _P]),
}
for _name, (_res, _args) in _SIGNATURES.items():
    getattr(_lib, _name).restype = _res
    getattr(_lib, _name).argtypes = _args


# ---------------------------------------------------------------------------
# C ABI, same names (the stream, last, defaults to the current one)
# ---------------------------------------------------------------------------

def _call(name, args, stream):
    _check(getattr(_lib, name)(*[_ptr(a) if isinstance(a, torch.Tensor) else a for a in args], _stream_handle(stream)))


def pts_quantize_fp8(*args, stream=None) -> None:
    _call("pts_quantize_fp8", args, stream)


def pts_gemm_fp8(*args, stream=None) -> None:
    _call("pts_gemm_fp8", args, stream)


def pts_gemm_fp8_experts(*args, stream=None) -> None:
    _call("pts_gemm_fp8_experts", args, stream)


def pts_moe_route_workspace(m: int, experts: int, top: int) -> int:
    return _lib.pts_moe_route_workspace(m, experts, top)


def pts_moe_route(*args, stream=None) -> None:
    _call("pts_moe_route", args, stream)


def pts_moe_route_backward(*args, stream=None) -> None:
    _call("pts_moe_route_backward", args, stream)


def pts_moe_combine(*args, stream=None) -> None:
    _call("pts_moe_combine", args, stream)


def pts_moe_combine_backward(*args, stream=None) -> None:
    _call("pts_moe_combine_backward", args, stream)


# ---------------------------------------------------------------------------
# Tensors
# ---------------------------------------------------------------------------

# The checks below stand in the way of kernels of a few microseconds: each call
# tests its arguments inline and only then asks the functions here to say what is
# wrong.

_DTYPES = {torch.bfloat16: GEMM_DTYPE_BF16, torch.float32: GEMM_DTYPE_F32}
_E4M3, _F32, _I32 = torch.float8_e4m3fn, torch.float32, torch.int32
_VALUES = tuple(_DTYPES)
_raw_stream = torch._C._cuda_getCurrentRawStream
_current = torch._C._cuda_getDevice
_empty = torch.empty_strided


def _expect(name, t, dtypes, shape) -> None:
    """Refuse a tensor that has not one of the dtypes and the shape (None: any extent)."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.dim() != len(shape) or any(
            want is not None and have != want for have, want in zip(t.shape, shape)):
        have = f"{t.dtype} {tuple(t.shape)}" if isinstance(t, torch.Tensor) else type(t).__name__
        kinds = " or ".join(str(d).replace("torch.", "") for d in dtypes)
        raise ValueError(f"{name} must be {kinds} of shape ({', '.join('*' if w is None else str(w) for w in shape)}), "
                         f"not {have}")


def _matrix(name, t, dtypes) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.dim() != 2:
        _expect(name, t, dtypes, (None, None))


def _exactly(name, t, dtype, shape) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape:
        _expect(name, t, (dtype,), shape)


def _index(name, t, shape) -> None:
    """A contiguous int32 tensor."""
    _exactly(name, t, _I32, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _weights(name, t, shape) -> None:
    """A contiguous fp32 tensor."""
    _exactly(name, t, _F32, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _device(first, *others) -> int:
    """The current device's index; every tensor must be on it."""
    dev = first.get_device()
    if dev < 0 or dev != _current():
        raise ValueError(f"tensors are on {first.device}, not on the current GPU")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"a tensor is on {t.device}, not on the current GPU ({first.device})")
    return dev


def _leading(name, t, of: int = 1) -> int:
    """Row stride of a row-major matrix (the last two dimensions); for a single row its width, rounded up to `of`."""
    rows, width = t.shape[-2], t.shape[-1]
    if rows > 1 and width > 1:
        row, col = t.stride(-2), t.stride(-1)
        if col != 1 or row < width:
            raise ValueError(f"{name} must have unit stride along its rows and rows that do not overlap, "
                             f"not strides {t.stride()}")
        return row
    if width > 1 and rows and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit stride along its rows")
    if rows > 1 and width:
        if t.stride(-2) < 1:
            raise ValueError(f"{name}'s rows overlap")
        return t.stride(-2)
    return (width + of - 1) // of * of


_BLOCKS = {(1, 128): 1, (128, 128): 128}
_quantize, _gemm, _gemm_experts = _lib.pts_quantize_fp8, _lib.pts_gemm_fp8, _lib.pts_gemm_fp8_experts
_route_workspace, _route, _route_backward = (_lib.pts_moe_route_workspace, _lib.pts_moe_route,
                                             _lib.pts_moe_route_backward)
_combine, _combine_backward = _lib.pts_moe_combine, _lib.pts_moe_combine_backward


def quantize_fp8(x: torch.Tensor, block=(1, 128), swiglu: bool = False) -> tuple[torch.Tensor, torch.Tensor]:
    """e4m3 codes of ``x`` and their fp32 scales: ``(q, scale)`` with
    ``x ~ q * scale`` over blocks of 128 along the rows, or of 128 x 128.

    ``x``: bf16 or fp32, (m, k), either dimension contiguous (``w.t()`` quantises
    a transpose without a copy). ``block``: (1, 128) or (128, 128). ``swiglu``:
    quantise ``silu(x[:, :k]) * x[:, k:]`` of an (m, 2 k) ``x`` instead.
    ``q``: float8_e4m3fn (m, k), its row stride a multiple of 16; ``scale``:
    (m, ceil(k / 128)), stored with the rows next to each other, or
    (ceil(m / 128), ceil(k / 128)). scale = max(max |x| / 448, 2^-126); a block
    with an infinity or a NaN comes out NaN.
    """
    _matrix("x", x, _VALUES)
    tall = _BLOCKS.get(block if type(block) is tuple else tuple(block))
    if tall is None:
        raise ValueError(f"block must be (1, 128) or (128, 128), not {block}")
    dev, device = _device(x), x.device
    m, k = x.shape
    row, col = x.stride()
    if col == 1 or k <= 1 or m == 0:
        layout, ld = GEMM_ROW_MAJOR, row if m > 1 and k else k
    elif row == 1 or m == 1:
        layout, ld = GEMM_COL_MAJOR, col
    else:
        raise ValueError(f"x must be contiguous along one of its dimensions, not strides {x.stride()}")
    if ld < (k if layout == GEMM_ROW_MAJOR else m):
        raise ValueError(f"x's rows overlap (strides {x.stride()})")
    if swiglu:
        if k % 2:
            raise ValueError(f"the gated form takes an even width, not {k}")
        k //= 2
    kb, wide = (k + 127) // 128, (k + 15) // 16 * 16
    q = _empty((m, k), (wide, 1), dtype=_E4M3, device=device) if wide == k else \
        torch.empty((m, wide), dtype=_E4M3, device=device)[:, :k]
    if tall == 1:
        scale, sm, sk = _empty((m, kb), (1, m), dtype=_F32, device=device), 1, m or 1
    else:
        mb = (m + 127) // 128
        scale, sm, sk = _empty((mb, kb), (kb, 1), dtype=_F32, device=device), kb or 1, 1
    status = _quantize(x.data_ptr(), _DTYPES[x.dtype], layout, m, k, ld, tall, 1 if swiglu else 0, q.data_ptr(), wide,
                       scale.data_ptr(), sm, sk, _raw_stream(dev))
    if status:
        _check(status)
    return q, scale


def _output(out, m, n, out_dtype, device):
    """The result's tensor and row stride."""
    if out is None:
        if out_dtype not in _DTYPES:
            raise ValueError(f"out_dtype must be float32 or bfloat16, not {out_dtype}")
        return _empty((m, n), (n, 1), dtype=out_dtype, device=device), n
    _expect("out", out, _VALUES, (m, n))
    return out, _leading("out", out)


def gemm_fp8(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor, out_dtype=torch.float32,
             out: torch.Tensor | None = None) -> torch.Tensor:
    """D = A . B for block-scaled e4m3 ``a`` (m, k) and ``b`` (n, k: B's transpose,
    as for :func:`gemm`).

    ``a_scale``: (m, ceil(k / 128)) fp32, any strides. ``b_scale``: one per row
    and block, (n, ceil(k / 128)), or one per 128 x 128 block,
    (ceil(n / 128), ceil(k / 128)). Row strides of ``a`` and ``b`` must be
    multiples of 16 and their first elements 16-byte aligned, as
    :func:`quantize_fp8` leaves them. ``out`` (fp32 or bf16) is written in place
    when given and must not share memory with an operand (not checked).

    The product's gradients are products too: dA = dD . B^T is
    ``gemm_fp8(*quantize_fp8(dd), *quantize_fp8(b_t, (128, 128)))`` and
    dB^T = dD^T . A is ``gemm_fp8(*quantize_fp8(dd.t()), *quantize_fp8(a.t()))``.
    """
    _matrix("a", a, (_E4M3,))
    _matrix("b", b, (_E4M3,))
    m, k = a.shape
    n, kb = b.shape[0], (k + 127) // 128
    if b.shape[1] != k:
        raise ValueError(f"a and b have {k} and {b.shape[1]} columns")
    _exactly("a_scale", a_scale, _F32, (m, kb))
    blocks = isinstance(b_scale, torch.Tensor) and b_scale.shape == ((n + 127) // 128, kb)
    _exactly("b_scale", b_scale, _F32, b_scale.shape if blocks else (n, kb))
    dev = _device(a, a_scale, b, b_scale, out)
    d, ldd = _output(out, m, n, out_dtype, a.device)
    sam, sak = a_scale.stride()
    sbn, sbk = b_scale.stride()
    status = _gemm(a.data_ptr(), _leading("a", a, 16), a_scale.data_ptr(), sam if m > 1 else 0, sak if kb > 1 else 0,
                   b.data_ptr(), _leading("b", b, 16), b_scale.data_ptr(), sbn if b_scale.shape[0] > 1 else 0,
                   sbk if kb > 1 else 0, 128 if blocks else 1, d.data_ptr(), ldd, _DTYPES[d.dtype], m, n, k,
                   _raw_stream(dev))
    if status:
        _check(status)
    return d


def gemm_fp8_experts(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
                     offsets: torch.Tensor, rows: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    """The product of :func:`gemm_fp8` for each expert over its own rows: rows
    ``offsets[e]`` to ``offsets[e + 1]`` of the result are (rows of A) . B_e.

    ``b``: (experts, n, k), ``b_scale``: (experts, ceil(n / 128), ceil(k / 128)).
    ``offsets``: int32 (experts + 1), on the GPU, non-decreasing; ``rows``: int32
    (m), the row of ``a`` that each row of the result reads (as
    :func:`moe_route` returns both), or None: row i reads row i. Rows in no
    expert's range are left as they were (in a new result: not set).
    """
    _matrix("a", a, (_E4M3,))
    have, k = a.shape
    if not isinstance(b, torch.Tensor) or b.dtype is not _E4M3 or b.dim() != 3 or b.shape[2] != k:
        _expect("b", b, (_E4M3,), (None, None, k))
    experts, n, kb = b.shape[0], b.shape[1], (k + 127) // 128
    _exactly("a_scale", a_scale, _F32, (have, kb))
    _exactly("b_scale", b_scale, _F32, (experts, (n + 127) // 128, kb))
    _index("offsets", offsets, (experts + 1,))
    m, index = have, None
    if rows is not None:
        _expect("rows", rows, (_I32,), (None,))
        _index("rows", rows, rows.shape)
        m, index = rows.shape[0], rows.data_ptr()
    dev = _device(a, a_scale, b, b_scale, offsets, rows, out)
    d, ldd = _output(out, m, n, out_dtype, a.device)
    sam, sak = a_scale.stride()
    sbe, sbn, sbk = b_scale.stride()
    status = _gemm_experts(a.data_ptr(), have, _leading("a", a, 16), a_scale.data_ptr(), sam if have > 1 else 0,
                           sak if kb > 1 else 0, b.data_ptr(), _leading("b", b, 16), b.stride(0) if experts > 1 else 0,
                           b_scale.data_ptr(), sbe if experts > 1 else 0, sbn if n > 128 else 0, sbk if kb > 1 else 0,
                           experts, offsets.data_ptr(), index, d.data_ptr(), ldd, _DTYPES[d.dtype], m, n, k,
                           _raw_stream(dev))
    if status:
        _check(status)
    return d


class MoeRouting(NamedTuple):
    """What :func:`moe_route` returns (int32, weights fp32)."""
    ids: torch.Tensor        # (tokens, k): experts, best first; -1: none
    weights: torch.Tensor    # (tokens, k)
    offsets: torch.Tensor    # (experts + 1): first row of each expert
    rows: torch.Tensor       # (tokens * k): the token of each row
    positions: torch.Tensor  # (tokens, k): the row of each slot; -2 - row where its id is -1


_SCORES = {"softmax": PTS_SCORE_SOFTMAX, "sigmoid": PTS_SCORE_SIGMOID}
_GROUP_SCORES = {"max": 0, "top2_sum": 1}


def moe_route(logits: torch.Tensor, k: int, *, score: str = "softmax", bias: torch.Tensor | None = None,
              groups: int = 1, topk_groups: int = 1, group_score: str = "max", renormalize: bool = True,
              scale: float = 1.0) -> MoeRouting:
    """Choose ``k`` experts for each token and order the (token, expert) rows by
    expert.

    ``logits``: (tokens, experts) bf16 or fp32. ``score``: "softmax" or
    "sigmoid". ``bias`` (fp32, experts) is added to the scores for the choice
    only. ``groups`` > 1: only the experts of the ``topk_groups`` best groups of
    consecutive experts are chosen from, a group's score being its largest
    ("max") or the sum of its two largest ("top2_sum"). ``weights`` are the
    chosen scores, divided by their sum + 1e-20 if ``renormalize``, times
    ``scale``. Ties go to the lowest index. A logit of -inf (or NaN) closes an
    expert to a token; a row of them (a padded token) gets ids -1, weights 0 and
    rows behind ``offsets[-1]``.
    """
    _matrix("logits", logits, _VALUES)
    m, experts = logits.shape
    if score not in _SCORES or group_score not in _GROUP_SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, group_score one of {sorted(_GROUP_SCORES)}")
    if bias is not None:
        _weights("bias", bias, (experts,))
    top = int(k)
    if not 1 <= top <= experts:
        raise ValueError(f"k must be in [1, {experts}], not {k}")
    dev, device, ld = _device(logits, bias), logits.device, _leading("logits", logits)
    ids = _empty((m, top), (top, 1), dtype=_I32, device=device)
    weights = _empty((m, top), (top, 1), dtype=_F32, device=device)
    offsets = _empty((experts + 1,), (1,), dtype=_I32, device=device)
    rows = _empty((m * top,), (1,), dtype=_I32, device=device)
    positions = _empty((m, top), (top, 1), dtype=_I32, device=device)
    need, work = _route_workspace(m, experts, top), None
    if need:
        work = _empty((need,), (1,), dtype=torch.uint8, device=device)
    status = _route(logits.data_ptr(), _DTYPES[logits.dtype], ld, None if bias is None else bias.data_ptr(), m, experts, top,
                    _SCORES[score], groups, topk_groups, _GROUP_SCORES[group_score], 1 if renormalize else 0, scale,
                    ids.data_ptr(), weights.data_ptr(), offsets.data_ptr(), rows.data_ptr(), positions.data_ptr(),
                    None if work is None else work.data_ptr(), need, _raw_stream(dev))
    if status:
        _check(status)
    return MoeRouting(ids, weights, offsets, rows, positions)


def moe_route_backward(dweights: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor, *, score: str = "softmax",
                       renormalize: bool = True, scale: float = 1.0) -> torch.Tensor:
    """The gradient of the logits (their dtype and shape) from that of
    :func:`moe_route`'s weights; ``ids``, ``score``, ``renormalize`` and ``scale``
    as in the forward call. The choice, and with it the bias, has no gradient."""
    _matrix("logits", logits, _VALUES)
    m, experts = logits.shape
    _matrix("ids", ids, (_I32,))
    top = ids.shape[1]
    _index("ids", ids, (m, top))
    _weights("dweights", dweights, (m, top))
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}")
    dev, ld = _device(logits, dweights, ids), _leading("logits", logits)
    out = _empty((m, experts), (experts, 1), dtype=logits.dtype, device=logits.device)
    status = _route_backward(dweights.data_ptr(), logits.data_ptr(), _DTYPES[logits.dtype], ld, ids.data_ptr(), m, experts,
                             top, _SCORES[score], 1 if renormalize else 0, scale, out.data_ptr(), experts, _raw_stream(dev))
    if status:
        _check(status)
    return out


def moe_combine(y: torch.Tensor, weights: torch.Tensor, positions: torch.Tensor) -> torch.Tensor:
    """out[t] = sum over j of ``weights[t, j] * y[positions[t, j]]``, in fp32, in
    ``y``'s dtype (bf16 or fp32). A position outside ``y`` adds nothing."""
    _matrix("y", y, _VALUES)
    _matrix("positions", positions, (_I32,))
    m, top = positions.shape
    _index("positions", positions, (m, top))
    _weights("weights", weights, (m, top))
    rows, n = y.shape
    dev, ld = _device(y, weights, positions), _leading("y", y)
    out = _empty((m, n), (n, 1), dtype=y.dtype, device=y.device)
    status = _combine(y.data_ptr(), _DTYPES[y.dtype], ld, rows, weights.data_ptr(), positions.data_ptr(), m, n, top,
                      out.data_ptr(), n, _raw_stream(dev))
    if status:
        _check(status)
    return out


def moe_combine_backward(dout: torch.Tensor, y: torch.Tensor, weights: torch.Tensor,
                         positions: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """``(dy, dweights)`` of :func:`moe_combine`. Every row of ``y`` should be some
    slot's (as :func:`moe_route` numbers them: the rows of slots without an
    expert get a gradient of 0); a row that no position names is not set. No two
    slots may name the same row."""
    _matrix("y", y, _VALUES)
    _matrix("positions", positions, (_I32,))
    m, top = positions.shape
    rows, n = y.shape
    _index("positions", positions, (m, top))
    _weights("weights", weights, (m, top))
    _exactly("dout", dout, y.dtype, (m, n))
    dev, ld, ld_d = _device(y, dout, weights, positions), _leading("y", y), _leading("dout", dout)
    dy = _empty((rows, n), (n, 1), dtype=y.dtype, device=y.device)
    dweights = _empty((m, top), (top, 1), dtype=_F32, device=y.device)
    status = _combine_backward(dout.data_ptr(), ld_d, y.data_ptr(), _DTYPES[y.dtype], ld, rows, weights.data_ptr(),
                               positions.data_ptr(), m, n, top, dy.data_ptr(), n, dweights.data_ptr(), _raw_stream(dev))
    if status:
        _check(status)
    return dy, dweights


def moe_fp8(x: torch.Tensor, logits: torch.Tensor, k: int, gate_up: torch.Tensor, gate_up_scale: torch.Tensor,
            down: torch.Tensor, down_scale: torch.Tensor, **routing) -> torch.Tensor:
    """A layer of routed experts: each token's ``k`` experts' outputs
    ``down_e . (silu(gate_e x) * (up_e x))``, weighted and added.

    ``x``: (tokens, hidden) bf16 or fp32 (the result is bf16); ``gate_up``: (experts, 2 inner, hidden) and
    ``down``: (experts, hidden, inner), e4m3 with 128 x 128 scales; ``routing``:
    keywords of :func:`moe_route`. Eight launches at most and no host
    synchronisation.
    """
    _matrix("x", x, _VALUES)
    _expect("logits", logits, _VALUES, (x.shape[0], None))
    r = moe_route(logits, k, **routing)
    h = gemm_fp8_experts(*quantize_fp8(x), gate_up, gate_up_scale, r.offsets, r.rows)
    y = gemm_fp8_experts(*quantize_fp8(h, swiglu=True), down, down_scale, r.offsets)
    return moe_combine(y, r.weights, r.positions)
