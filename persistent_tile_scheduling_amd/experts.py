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

_DTYPES = {torch.bfloat16: GEMM_DTYPE_BF16, torch.float32: GEMM_DTYPE_F32}
_E4M3 = torch.float8_e4m3fn
_raw_stream = torch._C._cuda_getCurrentRawStream


def _device(**tensors) -> int:
    """The current device's index; every tensor must be on it."""
    dev = torch.cuda.current_device() if torch.cuda.is_available() else -1
    for name, t in tensors.items():
        if t is not None and (not isinstance(t, torch.Tensor) or t.get_device() != dev or dev < 0):
            where = t.device if isinstance(t, torch.Tensor) else type(t).__name__
            raise ValueError(f"{name} is on {where}, not on the current GPU")
    return dev


def _expect(name, t, dtypes, shape) -> None:
    """dtype and shape (None: any extent) of a tensor."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.dim() != len(shape) or any(
            want is not None and have != want for have, want in zip(t.shape, shape)):
        have = f"{t.dtype} {tuple(t.shape)}" if isinstance(t, torch.Tensor) else type(t).__name__
        kinds = " or ".join(str(d).replace("torch.", "") for d in dtypes)
        raise ValueError(f"{name} must be {kinds} of shape ({', '.join('*' if w is None else str(w) for w in shape)}), "
                         f"not {have}")


def _leading(name, t, of: int = 1) -> int:
    """Row stride of a row-major matrix (the last two dimensions); for a single row its width, rounded up to `of`."""
    rows, width = t.shape[-2], t.shape[-1]
    if t.numel() and width > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit stride along its rows")
    if rows <= 1 or not t.numel():
        return (width + of - 1) // of * of
    if t.stride(-2) < width:
        raise ValueError(f"{name}'s row stride {t.stride(-2)} is below its width {width}")
    return t.stride(-2)


def _contiguous(name, t) -> None:
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


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
    _expect("x", x, (torch.bfloat16, torch.float32), (None, None))
    block = tuple(block)
    if block not in ((1, 128), (128, 128)):
        raise ValueError(f"block must be (1, 128) or (128, 128), not {block}")
    dev = _device(x=x)
    m, k = x.shape
    row, col = x.stride()
    layout = GEMM_ROW_MAJOR
    if k > 1 and col != 1 and x.numel():
        if m > 1 and row != 1:
            raise ValueError("x must be contiguous along one of its dimensions")
        layout = GEMM_COL_MAJOR
    ld = (col if layout == GEMM_COL_MAJOR else row) if m > 1 and x.numel() else max(k, 1)
    if layout == GEMM_COL_MAJOR:
        ld = col
    if x.numel() and ld < (m if layout == GEMM_COL_MAJOR else k):
        raise ValueError("x's rows overlap")
    if swiglu:
        if k % 2:
            raise ValueError(f"the gated form takes an even width, not {k}")
        k //= 2
    kb = (k + 127) // 128
    wide = (k + 15) // 16 * 16
    q = torch.empty((m, wide), dtype=_E4M3, device=x.device)
    if block[0] == 1:
        scale = torch.empty((kb, m), dtype=torch.float32, device=x.device).t()
    else:
        scale = torch.empty(((m + 127) // 128, kb), dtype=torch.float32, device=x.device)
    _check(_lib.pts_quantize_fp8(x.data_ptr(), _DTYPES[x.dtype], layout, m, k, ld, block[0], 1 if swiglu else 0,
                                 q.data_ptr(), wide, scale.data_ptr(), max(scale.stride(0), 1), max(scale.stride(1), 1),
                                 _raw_stream(dev)))
    return (q if wide == k else q[:, :k]), scale


def _scale_strides(t) -> tuple[int, int]:
    return t.stride(-2) if t.shape[-2] > 1 else 0, t.stride(-1) if t.shape[-1] > 1 else 0


def _output(out, m, n, out_dtype, device):
    if out is None:
        if out_dtype not in _DTYPES:
            raise ValueError(f"out_dtype must be float32 or bfloat16, not {out_dtype}")
        out = torch.empty((m, n), dtype=out_dtype, device=device)
    else:
        _expect("out", out, tuple(_DTYPES), (m, n))
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
    _expect("a", a, (_E4M3,), (None, None))
    m, k = a.shape
    _expect("b", b, (_E4M3,), (None, k))
    n, kb = b.shape[0], (k + 127) // 128
    _expect("a_scale", a_scale, (torch.float32,), (m, kb))
    blocks = b_scale.dim() == 2 and b_scale.shape[0] == (n + 127) // 128
    _expect("b_scale", b_scale, (torch.float32,), ((n + 127) // 128 if blocks else n, kb))
    dev = _device(a=a, a_scale=a_scale, b=b, b_scale=b_scale, out=out)
    out, ldd = _output(out, m, n, out_dtype, a.device)
    _check(_lib.pts_gemm_fp8(a.data_ptr(), _leading("a", a, 16), a_scale.data_ptr(), *_scale_strides(a_scale),
                             b.data_ptr(), _leading("b", b, 16), b_scale.data_ptr(), *_scale_strides(b_scale),
                             128 if blocks else 1, out.data_ptr(), ldd, _DTYPES[out.dtype], m, n, k, _raw_stream(dev)))
    return out


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
    _expect("a", a, (_E4M3,), (None, None))
    have, k = a.shape
    _expect("b", b, (_E4M3,), (None, None, k))
    experts, n = b.shape[:2]
    kb = (k + 127) // 128
    _expect("a_scale", a_scale, (torch.float32,), (have, kb))
    _expect("b_scale", b_scale, (torch.float32,), (experts, (n + 127) // 128, kb))
    _expect("offsets", offsets, (torch.int32,), (experts + 1,))
    _contiguous("offsets", offsets)
    m, index = have, None
    if rows is not None:
        _expect("rows", rows, (torch.int32,), (None,))
        _contiguous("rows", rows)
        m, index = rows.shape[0], rows.data_ptr()
    dev = _device(a=a, a_scale=a_scale, b=b, b_scale=b_scale, offsets=offsets, rows=rows, out=out)
    out, ldd = _output(out, m, n, out_dtype, a.device)
    _check(_lib.pts_gemm_fp8_experts(a.data_ptr(), have, _leading("a", a, 16), a_scale.data_ptr(),
                                     *_scale_strides(a_scale), b.data_ptr(), _leading("b", b, 16),
                                     b.stride(0) if experts > 1 else 0, b_scale.data_ptr(),
                                     b_scale.stride(0) if experts > 1 else 0, *_scale_strides(b_scale), experts,
                                     offsets.data_ptr(), index, out.data_ptr(), ldd, _DTYPES[out.dtype], m, n, k,
                                     _raw_stream(dev)))
    return out


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
    _expect("logits", logits, (torch.bfloat16, torch.float32), (None, None))
    m, experts = logits.shape
    if score not in _SCORES or group_score not in _GROUP_SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, group_score one of {sorted(_GROUP_SCORES)}")
    if bias is not None:
        _expect("bias", bias, (torch.float32,), (experts,))
        _contiguous("bias", bias)
    dev = _device(logits=logits, bias=bias)
    ld = _leading("logits", logits)
    device, top = logits.device, int(k)
    if not 1 <= top <= experts:
        raise ValueError(f"k must be in [1, {experts}], not {k}")
    ids = torch.empty((m, top), dtype=torch.int32, device=device)
    weights = torch.empty((m, top), dtype=torch.float32, device=device)
    offsets = torch.empty((experts + 1,), dtype=torch.int32, device=device)
    rows = torch.empty((m * top,), dtype=torch.int32, device=device)
    positions = torch.empty((m, top), dtype=torch.int32, device=device)
    need = _lib.pts_moe_route_workspace(m, experts, top)
    work = torch.empty((need,), dtype=torch.uint8, device=device) if need else None
    _check(_lib.pts_moe_route(logits.data_ptr(), _DTYPES[logits.dtype], ld, None if bias is None else bias.data_ptr(), m,
                              experts, top, _SCORES[score], groups, topk_groups, _GROUP_SCORES[group_score],
                              1 if renormalize else 0, scale, ids.data_ptr(), weights.data_ptr(), offsets.data_ptr(),
                              rows.data_ptr(), positions.data_ptr(), None if work is None else work.data_ptr(), need,
                              _raw_stream(dev)))
    return MoeRouting(ids, weights, offsets, rows, positions)


def moe_route_backward(dweights: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor, *, score: str = "softmax",
                       renormalize: bool = True, scale: float = 1.0) -> torch.Tensor:
    """The gradient of the logits (their dtype and shape) from that of
    :func:`moe_route`'s weights; ``ids``, ``score``, ``renormalize`` and ``scale``
    as in the forward call. The choice, and with it the bias, has no gradient."""
    _expect("logits", logits, (torch.bfloat16, torch.float32), (None, None))
    m, experts = logits.shape
    _expect("ids", ids, (torch.int32,), (m, None))
    top = ids.shape[1]
    _expect("dweights", dweights, (torch.float32,), (m, top))
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}")
    _contiguous("ids", ids)
    _contiguous("dweights", dweights)
    dev = _device(dweights=dweights, logits=logits, ids=ids)
    out = torch.empty((m, experts), dtype=logits.dtype, device=logits.device)
    _check(_lib.pts_moe_route_backward(dweights.data_ptr(), logits.data_ptr(), _DTYPES[logits.dtype],
                                       _leading("logits", logits), ids.data_ptr(), m, experts, top, _SCORES[score],
                                       1 if renormalize else 0, scale, out.data_ptr(), experts, _raw_stream(dev)))
    return out


def moe_combine(y: torch.Tensor, weights: torch.Tensor, positions: torch.Tensor) -> torch.Tensor:
    """out[t] = sum over j of ``weights[t, j] * y[positions[t, j]]``, in fp32, in
    ``y``'s dtype (bf16 or fp32). A position outside ``y`` adds nothing."""
    _expect("y", y, (torch.bfloat16, torch.float32), (None, None))
    _expect("positions", positions, (torch.int32,), (None, None))
    m, top = positions.shape
    _expect("weights", weights, (torch.float32,), (m, top))
    _contiguous("positions", positions)
    _contiguous("weights", weights)
    dev = _device(y=y, weights=weights, positions=positions)
    rows, n = y.shape
    out = torch.empty((m, n), dtype=y.dtype, device=y.device)
    _check(_lib.pts_moe_combine(y.data_ptr(), _DTYPES[y.dtype], _leading("y", y), rows, weights.data_ptr(),
                                positions.data_ptr(), m, n, top, out.data_ptr(), n, _raw_stream(dev)))
    return out


def moe_combine_backward(dout: torch.Tensor, y: torch.Tensor, weights: torch.Tensor,
                         positions: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """``(dy, dweights)`` of :func:`moe_combine`. Every row of ``y`` should be some
    slot's (as :func:`moe_route` numbers them: the rows of slots without an
    expert get a gradient of 0); a row that no position names is not set. No two
    slots may name the same row."""
    _expect("y", y, (torch.bfloat16, torch.float32), (None, None))
    _expect("positions", positions, (torch.int32,), (None, None))
    m, top = positions.shape
    rows, n = y.shape
    _expect("weights", weights, (torch.float32,), (m, top))
    _expect("dout", dout, (y.dtype,), (m, n))
    _contiguous("positions", positions)
    _contiguous("weights", weights)
    dev = _device(dout=dout, y=y, weights=weights, positions=positions)
    dy = torch.empty((rows, n), dtype=y.dtype, device=y.device)
    dweights = torch.empty((m, top), dtype=torch.float32, device=y.device)
    _check(_lib.pts_moe_combine_backward(dout.data_ptr(), _leading("dout", dout), y.data_ptr(), _DTYPES[y.dtype],
                                         _leading("y", y), rows, weights.data_ptr(), positions.data_ptr(), m, n, top,
                                         dy.data_ptr(), n, dweights.data_ptr(), _raw_stream(dev)))
    return dy, dweights


def moe_fp8(x: torch.Tensor, logits: torch.Tensor, k: int, gate_up: torch.Tensor, gate_up_scale: torch.Tensor,
            down: torch.Tensor, down_scale: torch.Tensor, **routing) -> torch.Tensor:
    """A layer of routed experts: each token's ``k`` experts' outputs
    ``down_e . (silu(gate_e x) * (up_e x))``, weighted and added.

    ``x``: (tokens, hidden) bf16; ``gate_up``: (experts, 2 inner, hidden) and
    ``down``: (experts, hidden, inner), e4m3 with 128 x 128 scales; ``routing``:
    keywords of :func:`moe_route`. Eight launches at most and no host
    synchronisation.
    """
    r = moe_route(logits, k, **routing)
    h = gemm_fp8_experts(*quantize_fp8(x), gate_up, gate_up_scale, r.offsets, r.rows)
    y = gemm_fp8_experts(*quantize_fp8(h, swiglu=True), down, down_scale, r.offsets)
    return moe_combine(y, r.weights, r.positions)
