"""Thin PyTorch binding of the expert-side calls (include/epdc_expert.h): the
experts' products for a few rows, a whole expert layer for a few tokens, the
gated activation with its 8-bit checkpoint, and the gradient of the combine.

As in ``ops``, the functions mirror the C entry points: they check dtypes,
shapes and devices, allocate outputs the caller did not pass, and enqueue on
the current (or given) HIP stream.  They run on the device of their tensors,
whichever is current.  They record nothing for autograd; the backward passes
are calls of their own."""

from __future__ import annotations

import functools
from typing import NamedTuple, Optional, Tuple, Union

import torch

from ._lib import EP_W_BF16, EP_W_FP4, EP_W_INT4, check, lib
from .ops import _gpu, _shape, _stream, _vp

__all__ = [
    "W4Weights",
    "ep_quantize_w4",
    "ep_expert_matvec",
    "ep_moe_tokens",
    "ep_moe_tokens_workspace_bytes",
    "ep_swiglu_fp8",
    "ep_swiglu_fp8_backward",
    "ep_combine_backward",
]

_BF16, _F32, _U8, _I32, _I64 = (torch.bfloat16, torch.float32, torch.uint8, torch.int32,
                                torch.int64)
_FP8 = torch.float8_e4m3fn
_W4_FMT = {"int4": EP_W_INT4, "fp4": EP_W_FP4}
_W4_SCALE = {"int4": _BF16, "fp4": _U8}


class W4Weights(NamedTuple):
    """4-bit matrices [.., N, K] with one scale for every ``group`` channels:
    ``fmt`` "int4" ((code - 8) times a bf16 scale; group 32, 64 or 128) or
    "fp4" (e2m1 times 2^(byte - 127); group 32).  Channel 2j sits in the low
    half of byte j of a row."""
    q: torch.Tensor                    # uint8 [.., N, K/2]
    scale: torch.Tensor                # [.., N, K/group]: bf16 (int4) or uint8 (fp4)
    fmt: str
    group: int


Weights = Union[torch.Tensor, W4Weights]


def _on_device(fn):
    """Run with the first tensor's device current, and the stream that was
    given, so that outputs allocated inside belong to both."""
    @functools.wraps(fn)
    def call(first, *args, stream=None, **kw):
        if not isinstance(first, torch.Tensor) or first.device.type != "cuda":
            return fn(first, *args, **kw)              # refused there, by its name
        if stream is not None:
            if stream.device != first.device:
                raise ValueError(f"stream is on {stream.device}, the tensors on {first.device}")
            with torch.cuda.stream(stream):
                return fn(first, *args, **kw)
        if first.device.index != torch.cuda.current_device():
            with torch.cuda.device(first.device):
                return fn(first, *args, **kw)
        return fn(first, *args, **kw)
    return call


def _on(t: torch.Tensor, name: str, dtype, shape, dev) -> torch.Tensor:
    _shape(_gpu(t, name, dtype), name, shape)
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, not on {dev}")
    return t


def _weights(w: Weights, name: str, dev):
    """(E, N, K, format, group, q, scale) of bf16 [E, N, K] or W4Weights."""
    if isinstance(w, W4Weights):
        if w.fmt not in _W4_FMT:
            raise ValueError(f"{name}.fmt must be one of {sorted(_W4_FMT)}")
        q, group = _gpu(w.q, f"{name}.q", _U8, 3), int(w.group)
        E, N, half = q.shape
        if group < 1:
            raise ValueError(f"{name}.group must be positive")
        _on(w.scale, f"{name}.scale", _W4_SCALE[w.fmt], (E, N, 2 * half // group), dev)
        out = E, N, 2 * half, _W4_FMT[w.fmt], group, q, w.scale
    else:
        q = _gpu(w, name, _BF16, 3)
        out = (*q.shape, EP_W_BF16, 0, q, None)
    if q.device != dev:
        raise ValueError(f"{name} is on {q.device}, not on {dev}")
    return out


@_on_device
def ep_quantize_w4(w: torch.Tensor, fmt: str = "int4", group: Optional[int] = None, *,
                   out: Optional[W4Weights] = None) -> W4Weights:
    """bf16 matrices [.., N, K] to 4 bits (int4: group 128 unless given; fp4:
    group 32).  K is a multiple of 128."""
    if fmt not in _W4_FMT:
        raise ValueError(f"fmt must be one of {sorted(_W4_FMT)}")
    _gpu(w, "w", _BF16)
    if w.dim() < 1:
        raise ValueError("w must be [.., N, K]")
    group = int(group) if group is not None else (32 if fmt == "fp4" else 128)
    K = w.shape[-1]
    if group < 1 or K < 1 or K % 128:
        raise ValueError("K must be a multiple of 128 and group positive")
    qs, ss = (*w.shape[:-1], K // 2), (*w.shape[:-1], K // group)
    if out is None:
        out = W4Weights(torch.empty(qs, dtype=_U8, device=w.device),
                        torch.empty(ss, dtype=_W4_SCALE[fmt], device=w.device), fmt, group)
    if out.fmt != fmt or int(out.group) != group:
        raise ValueError("out has another format")
    _on(out.q, "out.q", _U8, qs, w.device)
    _on(out.scale, "out.scale", _W4_SCALE[fmt], ss, w.device)
    st = lib().ep_quantize_w4(_vp(w), w.numel() // K, K, _W4_FMT[fmt], group, _vp(out.q),
                              _vp(out.scale), _stream(None))
    check(st, "ep_quantize_w4")
    return out


@_on_device
def ep_expert_matvec(x: torch.Tensor, weights: Weights, row_expert: Optional[torch.Tensor] = None,
                     *, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [R, N] bf16 with y[r] = W[row_expert[r]] x[r], for up to 1024 rows x
    [R, K] bf16 and matrices [E, N, K] (bf16 or W4Weights).  ``row_expert``
    [R] int32 may be left out for one matrix.  Rows whose id lies outside
    [0, E) are left as they are in ``out``; a result allocated here has zeros
    there."""
    _gpu(x, "x", _BF16, 2)
    R, K = x.shape
    dev = x.device
    E, N, wk, fmt, group, q, scale = _weights(weights, "weights", dev)
    if wk != K:
        raise ValueError(f"weights have {wk} channels, x has {K}")
    if row_expert is not None:
        _on(row_expert, "row_expert", _I32, (R,), dev)
    elif E != 1:
        raise ValueError("row_expert is needed for more than one expert")
    if out is None:
        out = (torch.empty if row_expert is None else torch.zeros)((R, N), dtype=_BF16, device=dev)
    else:
        _on(out, "out", _BF16, (R, N), dev)
    st = lib().ep_expert_matvec(_vp(x), _vp(row_expert), R, E, N, K, fmt, group, _vp(q),
                                _vp(scale), _vp(out), _stream(None))
    check(st, "ep_expert_matvec")
    return out


def ep_moe_tokens_workspace_bytes(num_tokens: int, num_topk: int, inner: int) -> int:
    return int(lib().ep_moe_tokens_workspace_bytes(int(num_tokens), int(num_topk), int(inner)))


@_on_device
def ep_moe_tokens(x: torch.Tensor, topk_idx: torch.Tensor, topk_weights: torch.Tensor,
                  w13: Weights, w2: Weights, first_expert: int = 0, *, bias=None,
                  out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out [T, H] bf16 of a whole expert layer for up to 128 tokens (T*K up to
    1024), in two launches: out[t] = sum over the slots whose expert e =
    topk_idx[t, k] - first_expert is one of the E here of topk_weights[t, k] *
    W2[e] (silu(gate) * up), the gate and up rows being W13[e] x[t].  ``w13``
    [E, 2I, H] (the gate rows, then the up rows) and ``w2`` [E, H, I] are bf16
    or W4Weights; ``bias`` is a [T, H] bf16 tensor or a pair, added in fp32
    before the one rounding, as in ep_combine.

    Without ``workspace`` (uint8, ep_moe_tokens_workspace_bytes of it) each
    call takes its own from PyTorch's allocator, so calls on several streams
    and captured graphs never share one."""
    _gpu(x, "x", _BF16, 2)
    T, H = x.shape
    dev = x.device
    _gpu(topk_idx, "topk_idx", _I64, 2)
    K = topk_idx.shape[1]
    _on(topk_idx, "topk_idx", _I64, (T, K), dev)
    _on(topk_weights, "topk_weights", _F32, (T, K), dev)
    E, N13, K13, fmt13, group13, q13, scale13 = _weights(w13, "w13", dev)
    E2, N2, I, fmt2, group2, q2, scale2 = _weights(w2, "w2", dev)
    if E2 != E or N2 != H or K13 != H or N13 != 2 * I:
        raise ValueError(f"w13 must be [E, 2I, {H}] and w2 [E, {H}, I], got "
                         f"[{E}, {N13}, {K13}] and [{E2}, {N2}, {I}]")
    biases = () if bias is None else (tuple(bias) if isinstance(bias, (tuple, list)) else (bias,))
    if len(biases) > 2:
        raise ValueError("bias is one [T, H] tensor or a pair")
    for i, b in enumerate(biases):
        _on(b, f"bias[{i}]", _BF16, (T, H), dev)
    if out is None:
        out = torch.empty((T, H), dtype=_BF16, device=dev)
    else:
        _on(out, "out", _BF16, (T, H), dev)
    if workspace is None:
        workspace = torch.empty(ep_moe_tokens_workspace_bytes(T, K, I), dtype=_U8, device=dev)
    else:
        _gpu(workspace, "workspace", _U8)
        if workspace.device != dev:
            raise ValueError(f"workspace is on {workspace.device}, not on {dev}")
    st = lib().ep_moe_tokens(
        _vp(x), _vp(topk_idx), _vp(topk_weights), T, K, H, I, int(first_expert), E, fmt13, group13,
        _vp(q13), _vp(scale13), fmt2, group2, _vp(q2), _vp(scale2),
        _vp(biases[0] if biases else None), _vp(biases[1] if len(biases) > 1 else None), _vp(out),
        _vp(workspace), workspace.numel(), _stream(None))
    check(st, "ep_moe_tokens")
    return out


def _row_count(t: Optional[torch.Tensor], dev):
    return None if t is None else _on(t, "row_count", _I32, (1,), dev)


@_on_device
def ep_swiglu_fp8(gate_up: torch.Tensor, *, row_count: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                  scale: Optional[torch.Tensor] = None
                  ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(h [R, I] bf16 = silu(gate) * up, q [R, 2I] float8_e4m3fn, scale
    [R, 2I/128] float32) of gate_up [R, 2I] bf16 (I gate channels, then I up
    channels; I a multiple of 128).  q and scale are the checkpoint that
    ep_swiglu_fp8_backward takes in place of gate_up and h.  Rows from
    ``row_count`` ([1] int32 on the device, e.g. ``expert_offsets[-1:]``) on
    are left as they are."""
    _gpu(gate_up, "gate_up", _BF16, 2)
    R, two = gate_up.shape
    if two % 256 or two == 0:
        raise ValueError("gate_up must be [R, 2I] with I a multiple of 128")
    I, dev = two // 2, gate_up.device
    count = _row_count(row_count, dev)
    h = torch.empty((R, I), dtype=_BF16, device=dev) if out is None else \
        _on(out, "out", _BF16, (R, I), dev)
    q = torch.empty((R, two), dtype=_FP8, device=dev) if q is None else \
        _on(q, "q", _FP8, (R, two), dev)
    scale = torch.empty((R, two // 128), dtype=_F32, device=dev) if scale is None else \
        _on(scale, "scale", _F32, (R, two // 128), dev)
    st = lib().ep_swiglu_fp8(_vp(gate_up), R, I, _vp(count), _vp(h), _vp(q), _vp(scale),
                             _stream(None))
    check(st, "ep_swiglu_fp8")
    return h, q, scale


@_on_device
def ep_swiglu_fp8_backward(dh: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, *,
                           row_count: Optional[torch.Tensor] = None, recompute: bool = True,
                           out: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None
                           ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(d_gate_up [R, 2I] bf16, h [R, I] bf16) from dh [R, I] bf16 and the
    checkpoint of ep_swiglu_fp8: the gradient of silu(gate) * up at the values
    the checkpoint stands for, and that product itself (what the second
    product's weight gradient takes), None without ``recompute``."""
    _gpu(dh, "dh", _BF16, 2)
    R, I = dh.shape
    if I % 128 or I == 0:
        raise ValueError("dh must be [R, I] with I a multiple of 128")
    dev = dh.device
    _on(q, "q", _FP8, (R, 2 * I), dev)
    _on(scale, "scale", _F32, (R, I // 64), dev)
    count = _row_count(row_count, dev)
    d = torch.empty((R, 2 * I), dtype=_BF16, device=dev) if out is None else \
        _on(out, "out", _BF16, (R, 2 * I), dev)
    if not recompute:
        if h is not None:
            raise ValueError("h is an output of recompute=True")
    elif h is None:
        h = torch.empty((R, I), dtype=_BF16, device=dev)
    else:
        _on(h, "h", _BF16, (R, I), dev)
    st = lib().ep_swiglu_fp8_backward(_vp(dh), _vp(q), _vp(scale), R, I, _vp(count), _vp(d),
                                      _vp(h), _stream(None))
    check(st, "ep_swiglu_fp8_backward")
    return d, h


@_on_device
def ep_combine_backward(dout: torch.Tensor, y: Optional[torch.Tensor], token_row: torch.Tensor,
                        topk_weights: Optional[torch.Tensor], *, weight_grad: Optional[bool] = None,
                        num_rows: Optional[int] = None, dy: Optional[torch.Tensor] = None,
                        dw: Optional[torch.Tensor] = None
                        ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gradient of ep_combine: (dy, shaped as y, bf16; dw [T, K] float32).
    dy[r] = (the sum of the weights of the slots that name row r) * dout[t],
    dw[t, k] = <dout[t], y[token_row[t, k]]>.  With ``topk_weights=None`` (the
    unweighted combine) or ``weight_grad=False`` dw is None and y is not read:
    it may then be None, with ``num_rows`` or ``dy`` giving the rows.  Rows no
    slot names are left as they are in ``dy``; a result allocated here has
    zeros there.  The gradient of a combine's bias is dout itself."""
    _gpu(dout, "dout", _BF16, 2)
    T, H = dout.shape
    dev = dout.device
    _gpu(token_row, "token_row", _I32, 2)
    K = token_row.shape[1]
    _on(token_row, "token_row", _I32, (T, K), dev)
    if topk_weights is not None:
        _on(topk_weights, "topk_weights", _F32, (T, K), dev)
    if weight_grad is None:
        weight_grad = topk_weights is not None
    elif weight_grad and topk_weights is None:
        raise ValueError("weight_grad needs topk_weights")
    if weight_grad and y is None:
        raise ValueError("the weights' gradient needs y")
    if y is not None:
        _gpu(y, "y", _BF16)
        if y.dim() < 2 or y.shape[-1] != H or y.device != dev:
            raise ValueError(f"y must be [.., {H}] on {dev}")
        shape = tuple(y.shape)
    elif dy is not None:
        shape = tuple(dy.shape)
    elif num_rows is not None:
        shape = (int(num_rows), H)
    else:
        raise ValueError("without y, num_rows or dy gives the rows")
    if dy is None:
        dy = torch.zeros(shape, dtype=_BF16, device=dev)
    elif len(shape) < 2 or shape[-1] != H:
        raise ValueError(f"dy must be [.., {H}]")
    else:
        _on(dy, "dy", _BF16, shape, dev)
    rows = dy.numel() // H if H else 0
    if num_rows is not None and int(num_rows) != rows:
        raise ValueError(f"num_rows is {num_rows}, the buffers have {rows}")
    if not weight_grad:
        if dw is not None:
            raise ValueError("dw is an output of weight_grad=True")
    elif dw is None:
        dw = torch.empty((T, K), dtype=_F32, device=dev)
    else:
        _on(dw, "dw", _F32, (T, K), dev)
    st = lib().ep_combine_backward(_vp(dout), _vp(y) if weight_grad else None, rows,
                                   _vp(token_row), _vp(topk_weights), T, K, H, _vp(dy), _vp(dw),
                                   _stream(None))
    check(st, "ep_combine_backward")
    return dy, dw
