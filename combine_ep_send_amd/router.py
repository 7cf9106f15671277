"""Thin PyTorch binding of the calls before the dispatch (include/epdc_router.h):
the RMS norm with the residual's addition and an 8-bit output, the router's
logits, the choice of the experts, their gradients, and the dispatch of rows
that are in 8 bits already.

As in ``ops`` and ``expert``, the functions mirror the C entry points: they check
dtypes, shapes and devices, allocate outputs the caller did not pass, and enqueue
on the current (or given) HIP stream, on the device of their tensors, whichever
is current.  They record nothing for autograd; the backward passes are calls of
their own."""

from __future__ import annotations

import functools
from typing import NamedTuple, Optional, Tuple

import torch

from ._lib import (EP_NORM_W_BF16, EP_NORM_W_F32, EP_OK, EP_SCALE_F32, EP_SCALE_POW2,
                   EP_SCORE_SIGMOID, EP_SCORE_SOFTMAX, check, lib)
from .expert import (_BF16, _F32, _FP8, _I32, _I64, _U8, _elsewhere, _first, _int, _on, _ptr,
                     _raw_stream, _there)

__all__ = [
    "RmsNorm",
    "ep_rms_norm",
    "ep_rms_norm_backward",
    "ep_rms_norm_backward_workspace_bytes",
    "ep_router_logits",
    "ep_router_logits_workspace_bytes",
    "ep_router_logits_backward",
    "ep_router_logits_backward_workspace_bytes",
    "ep_route",
    "ep_route_backward",
    "ep_dispatch_permute_quantized",
]

_NORM_SCALE = {"f32": EP_SCALE_F32, "pow2": EP_SCALE_POW2}
_SCORE = {"softmax": EP_SCORE_SOFTMAX, "sigmoid": EP_SCORE_SIGMOID}
_INT64_MAX = 0x7fffffffffffffff


class RmsNorm(NamedTuple):
    y: Optional[torch.Tensor]          # bf16 [T, H]
    q: Optional[torch.Tensor]          # float8_e4m3fn [T, H]
    scale: Optional[torch.Tensor]      # float32 [T, H/128]
    residual: Optional[torch.Tensor]   # bf16 [T, H]: x + residual, what was normalised
    rstd: Optional[torch.Tensor]       # float32 [T]


def _norm_weight(weight, H: int, index: int) -> int:
    f32 = isinstance(weight, torch.Tensor) and weight.dtype is _F32
    _on(weight, "weight", _F32 if f32 else _BF16, (H,), index)
    return EP_NORM_W_F32 if f32 else EP_NORM_W_BF16


def ep_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, *,
                residual: Optional[torch.Tensor] = None, bf16: bool = True, fp8: bool = False,
                rstd: bool = False, scale_fmt: str = "f32",
                residual_out: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                rstd_out: Optional[torch.Tensor] = None, stream=None) -> RmsNorm:
    """RMS norm of x [T, H] bf16 (H a multiple of 8) times ``weight`` [H] (bf16
    or float32), after the addition of ``residual`` [T, H] bf16 where it is
    given: the sum is rounded to bf16, returned as ``residual`` (it may be
    written over the residual: ``residual_out=residual``) and normalised.

    ``bf16``: the row in bf16 (``y``).  ``fp8``: e4m3 codes ``q`` and one fp32
    ``scale`` per 128 channels, quantized from fp32 (H a multiple of 128), which
    ``dispatch`` takes as (q, scale); ``scale_fmt="pow2"`` rounds the scales up
    to powers of two.  ``rstd``: 1 / the root mean square [T], for the backward
    pass.  What was not asked for is None."""
    index = _first(x, "x", _BF16, 2)
    if _elsewhere(index, stream):
        return _there(ep_rms_norm, index, stream, x, weight, eps, residual=residual, bf16=bf16,
                      fp8=fp8, rstd=rstd, scale_fmt=scale_fmt, residual_out=residual_out, out=out,
                      q=q, scale=scale, rstd_out=rstd_out)
    T, H = x.shape
    _int(H, "H")
    kind = _norm_weight(weight, H, index)
    fmt = _NORM_SCALE.get(scale_fmt)
    if fmt is None:
        raise ValueError(f"scale_fmt must be one of {sorted(_NORM_SCALE)}")
    if not bf16 and not fp8:
        raise ValueError("one of bf16 and fp8 must be asked for")
    if fp8 and H % 128:
        raise ValueError("fp8 needs H to be a multiple of 128")
    if residual is not None:
        _on(residual, "residual", _BF16, (T, H), index)
        residual_out = torch.empty_like(x) if residual_out is None else \
            _on(residual_out, "residual_out", _BF16, (T, H), index)
    elif residual_out is not None:
        raise ValueError("residual_out is an output of a call with a residual")
    if bf16:
        out = torch.empty_like(x) if out is None else _on(out, "out", _BF16, (T, H), index)
    elif out is not None:
        raise ValueError("out is an output of bf16=True")
    if fp8:
        q = x.new_empty((T, H), dtype=_FP8) if q is None else _on(q, "q", _FP8, (T, H), index)
        scale = x.new_empty((T, H // 128), dtype=_F32) if scale is None else \
            _on(scale, "scale", _F32, (T, H // 128), index)
    elif q is not None or scale is not None:
        raise ValueError("q and scale are outputs of fp8=True")
    if rstd:
        rstd_out = x.new_empty(T, dtype=_F32) if rstd_out is None else \
            _on(rstd_out, "rstd_out", _F32, (T,), index)
    elif rstd_out is not None:
        raise ValueError("rstd_out is an output of rstd=True")
    st = lib().ep_rms_norm(x.data_ptr(), _ptr(residual), weight.data_ptr(), kind, T, H, eps,
                           _ptr(residual_out), _ptr(out), _ptr(q), _ptr(scale), fmt,
                           _ptr(rstd_out), _raw_stream(index))
    if st != EP_OK:
        check(st, "ep_rms_norm")
    return RmsNorm(out, q, scale, residual_out, rstd_out)


def _bytes(name: str, *sizes) -> int:
    sizes = [int(v) for v in sizes]
    if abs(sizes[0]) > _INT64_MAX or any(abs(v) > 0x7fffffff for v in sizes[1:]):
        return 0                       # ctypes would drop the upper bits
    return int(getattr(lib(), name)(*sizes))


@functools.lru_cache(maxsize=1024)
def ep_rms_norm_backward_workspace_bytes(num_tokens: int, hidden: int) -> int:
    return _bytes("ep_rms_norm_backward_workspace_bytes", num_tokens, hidden)


@functools.lru_cache(maxsize=1024)
def ep_router_logits_workspace_bytes(num_tokens: int, num_experts: int, hidden: int) -> int:
    return _bytes("ep_router_logits_workspace_bytes", num_tokens, num_experts, hidden)


@functools.lru_cache(maxsize=1024)
def ep_router_logits_backward_workspace_bytes(num_tokens: int, num_experts: int,
                                              hidden: int) -> int:
    return _bytes("ep_router_logits_backward_workspace_bytes", num_tokens, num_experts, hidden)


def _workspace(workspace, nbytes: int, like: torch.Tensor, index: int) -> torch.Tensor:
    """The caller's, or one of this call's own from PyTorch's allocator, so that
    calls on several streams and captured graphs never share one."""
    if workspace is None:
        return like.new_empty(nbytes, dtype=_U8)
    if _first(workspace, "workspace", _U8, 1) != index:
        raise ValueError(f"workspace is on {workspace.device}, not on cuda:{index}")
    return workspace


def ep_rms_norm_backward(dy: torch.Tensor, s: torch.Tensor, weight: torch.Tensor,
                         rstd: torch.Tensor, *, d_residual: Optional[torch.Tensor] = None,
                         weight_grad: bool = True, out: Optional[torch.Tensor] = None,
                         dw: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None
                         ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gradient of ep_rms_norm: (dx [T, H] bf16, of x and of the residual alike;
    dw [H] float32, None without ``weight_grad``) from dy, the gradient of y, and
    what the forward normalised (``s``: its ``residual``, or x without one) with
    its ``rstd``.  ``d_residual``: the gradient that reaches the residual stream
    from elsewhere, added to dx (``out`` may be it, or dy)."""
    index = _first(dy, "dy", _BF16, 2)
    if _elsewhere(index, stream):
        return _there(ep_rms_norm_backward, index, stream, dy, s, weight, rstd,
                      d_residual=d_residual, weight_grad=weight_grad, out=out, dw=dw,
                      workspace=workspace)
    T, H = dy.shape
    _int(H, "H")
    _on(s, "s", _BF16, (T, H), index)
    kind = _norm_weight(weight, H, index)
    _on(rstd, "rstd", _F32, (T,), index)
    if d_residual is not None:
        _on(d_residual, "d_residual", _BF16, (T, H), index)
    out = torch.empty_like(dy) if out is None else _on(out, "out", _BF16, (T, H), index)
    if weight_grad:
        dw = dy.new_empty(H, dtype=_F32) if dw is None else _on(dw, "dw", _F32, (H,), index)
        workspace = _workspace(workspace, ep_rms_norm_backward_workspace_bytes(T, H), dy, index)
    elif dw is not None:
        raise ValueError("dw is an output of weight_grad=True")
    st = lib().ep_rms_norm_backward(dy.data_ptr(), s.data_ptr(), weight.data_ptr(), kind,
                                    rstd.data_ptr(), _ptr(d_residual), T, H, out.data_ptr(),
                                    _ptr(dw), _ptr(workspace),
                                    0 if workspace is None else workspace.numel(),
                                    _raw_stream(index))
    if st != EP_OK:
        check(st, "ep_rms_norm_backward")
    return out, dw


def ep_router_logits(x: torch.Tensor, w: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The router's logits [T, E] float32: x [T, H] bf16 times w [E, H] bf16
    (H a multiple of 8, E up to 1024), products exact, sums in fp32.  Without
    ``workspace`` (uint8, ep_router_logits_workspace_bytes of it) each call
    takes its own."""
    index = _first(x, "x", _BF16, 2)
    if _elsewhere(index, stream):
        return _there(ep_router_logits, index, stream, x, w, out=out, workspace=workspace)
    T, H = x.shape
    if _first(w, "w", _BF16, 2) != index:
        raise ValueError(f"w is on {w.device}, not on cuda:{index}")
    E = _int(w.shape[0], "E")
    if w.shape[1] != H:
        raise ValueError(f"w has {w.shape[1]} channels, x has {H}")
    out = x.new_empty((T, E), dtype=_F32) if out is None else _on(out, "out", _F32, (T, E), index)
    workspace = _workspace(workspace, ep_router_logits_workspace_bytes(T, E, H), x, index)
    st = lib().ep_router_logits(x.data_ptr(), w.data_ptr(), T, E, _int(H, "H"), out.data_ptr(),
                                workspace.data_ptr(), workspace.numel(), _raw_stream(index))
    if st != EP_OK:
        check(st, "ep_router_logits")
    return out


def ep_router_logits_backward(d_logits: torch.Tensor, x: Optional[torch.Tensor],
                              w: Optional[torch.Tensor], *, input_grad: bool = True,
                              weight_grad: bool = True, dx: Optional[torch.Tensor] = None,
                              dw: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None, stream=None
                              ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gradient of ep_router_logits from d_logits [T, E] float32: (dx [T, H]
    bf16, dw [E, H] float32), None where it is not asked for.  x is read for dw
    alone and w for dx alone; the other may then be None."""
    index = _first(d_logits, "d_logits", _F32, 2)
    if _elsewhere(index, stream):
        return _there(ep_router_logits_backward, index, stream, d_logits, x, w,
                      input_grad=input_grad, weight_grad=weight_grad, dx=dx, dw=dw,
                      workspace=workspace)
    T, E = d_logits.shape
    _int(E, "E")
    if not input_grad and not weight_grad:
        raise ValueError("one of input_grad and weight_grad must be asked for")
    if (input_grad and w is None) or (weight_grad and x is None):
        raise ValueError("input_grad needs w and weight_grad needs x")
    H = _int((w if w is not None else x).shape[-1], "H")
    if x is not None:
        _on(x, "x", _BF16, (T, H), index)
    if w is not None:
        _on(w, "w", _BF16, (E, H), index)
    if input_grad:
        dx = d_logits.new_empty((T, H), dtype=_BF16) if dx is None else \
            _on(dx, "dx", _BF16, (T, H), index)
    elif dx is not None:
        raise ValueError("dx is an output of input_grad=True")
    if weight_grad:
        dw = d_logits.new_empty((E, H)) if dw is None else _on(dw, "dw", _F32, (E, H), index)
    elif dw is not None:
        raise ValueError("dw is an output of weight_grad=True")
    workspace = _workspace(workspace, ep_router_logits_backward_workspace_bytes(T, E, H),
                           d_logits, index)
    st = lib().ep_router_logits_backward(d_logits.data_ptr(), _ptr(x), _ptr(w), T, E, H, _ptr(dx),
                                         _ptr(dw), workspace.data_ptr(), workspace.numel(),
                                         _raw_stream(index))
    if st != EP_OK:
        check(st, "ep_router_logits_backward")
    return dx, dw


def ep_route(logits: torch.Tensor, num_topk: int, *, score: str = "softmax",
             bias: Optional[torch.Tensor] = None, num_groups: int = 1, topk_groups: int = 1,
             group_top: int = 2, renormalize: bool = True, scale: float = 1.0,
             token_count: Optional[torch.Tensor] = None,
             topk_idx: Optional[torch.Tensor] = None,
             topk_weights: Optional[torch.Tensor] = None, stream=None
             ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(topk_idx [T, K] int64, topk_weights [T, K] float32) of the router's
    logits [T, E] float32, as ``dispatch`` takes them: the K experts of the
    largest ``score`` ("softmax" or "sigmoid") plus ``bias`` [E] float32, the
    largest first and ties to the lower number, weighted by their scores without
    the bias, over their sum with ``renormalize``, times ``scale``.

    With ``num_groups`` > 1 only the experts of the ``topk_groups`` worthiest
    groups take part, a group (E / num_groups neighbours) being worth the sum of
    its ``group_top`` (1 or 2) best.  Experts with a logit of -infinity or NaN
    are not chosen; a slot without an expert gets id -1 and weight 0.
    ``token_count`` ([1] int32 on the device): tokens from it on are padding and
    get -1 and 0 throughout."""
    index = _first(logits, "logits", _F32, 2)
    if _elsewhere(index, stream):
        return _there(ep_route, index, stream, logits, num_topk, score=score, bias=bias,
                      num_groups=num_groups, topk_groups=topk_groups, group_top=group_top,
                      renormalize=renormalize, scale=scale, token_count=token_count,
                      topk_idx=topk_idx, topk_weights=topk_weights)
    T, E = logits.shape
    K = _int(int(num_topk), "num_topk")
    if K < 1:
        raise ValueError("num_topk must be at least 1")
    kind = _SCORE.get(score)
    if kind is None:
        raise ValueError(f"score must be one of {sorted(_SCORE)}")
    if bias is not None:
        _on(bias, "bias", _F32, (E,), index)
    if token_count is not None:
        _on(token_count, "token_count", _I32, (1,), index)
    topk_idx = logits.new_empty((T, K), dtype=_I64) if topk_idx is None else \
        _on(topk_idx, "topk_idx", _I64, (T, K), index)
    topk_weights = logits.new_empty((T, K)) if topk_weights is None else \
        _on(topk_weights, "topk_weights", _F32, (T, K), index)
    st = lib().ep_route(logits.data_ptr(), T, _int(E, "E"), K, kind, _ptr(bias),
                        _int(int(num_groups), "num_groups"),
                        _int(int(topk_groups), "topk_groups"), _int(int(group_top), "group_top"),
                        bool(renormalize), scale, _ptr(token_count), topk_idx.data_ptr(),
                        topk_weights.data_ptr(), _raw_stream(index))
    if st != EP_OK:
        check(st, "ep_route")
    return topk_idx, topk_weights


def ep_route_backward(d_weights: torch.Tensor, logits: torch.Tensor, topk_idx: torch.Tensor, *,
                      score: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """d_logits [T, E] float32 of ep_route's weights from their gradient
    d_weights [T, K] float32 (combine_backward gives it), the choice topk_idx
    being constant.  ``score``, ``renormalize`` and ``scale`` as in the forward.
    Slots of id -1 are skipped."""
    index = _first(d_weights, "d_weights", _F32, 2)
    if _elsewhere(index, stream):
        return _there(ep_route_backward, index, stream, d_weights, logits, topk_idx, score=score,
                      renormalize=renormalize, scale=scale, out=out)
    T, K = d_weights.shape
    if _first(logits, "logits", _F32, 2) != index:
        raise ValueError(f"logits is on {logits.device}, not on cuda:{index}")
    E = _int(logits.shape[1], "E")
    _on(logits, "logits", _F32, (T, E), index)
    _on(topk_idx, "topk_idx", _I64, (T, K), index)
    kind = _SCORE.get(score)
    if kind is None:
        raise ValueError(f"score must be one of {sorted(_SCORE)}")
    out = torch.empty_like(logits) if out is None else _on(out, "out", _F32, (T, E), index)
    st = lib().ep_route_backward(d_weights.data_ptr(), logits.data_ptr(), topk_idx.data_ptr(), T,
                                 E, _int(K, "K"), kind, bool(renormalize), scale, out.data_ptr(),
                                 _raw_stream(index))
    if st != EP_OK:
        check(st, "ep_route_backward")
    return out


def ep_dispatch_permute_quantized(q: torch.Tensor, scale: torch.Tensor, token_row: torch.Tensor,
                                  num_send_capacity: int, *, out: Optional[torch.Tensor] = None,
                                  out_scale: Optional[torch.Tensor] = None, stream=None
                                  ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(send_q [cap, H] float8_e4m3fn, send_scale [cap, H/128] float32) of rows
    that are in 8 bits already: q [T, H] (H a multiple of 128) and scale
    [T, H/128], as ep_rms_norm makes them, moved unchanged to the rows that
    token_row [T, K] names, as in ep_dispatch_permute.  Other rows are left as
    they are."""
    index = _first(q, "q", _FP8, 2)
    if _elsewhere(index, stream):
        return _there(ep_dispatch_permute_quantized, index, stream, q, scale, token_row,
                      num_send_capacity, out=out, out_scale=out_scale)
    T, H = q.shape
    if _int(H, "H") % 128 or H == 0:
        raise ValueError("q must be [T, H] with H a multiple of 128")
    _on(scale, "scale", _F32, (T, H // 128), index)
    _first(token_row, "token_row", _I32, 2)
    K = _int(token_row.shape[1], "K")
    _on(token_row, "token_row", _I32, (T, K), index)
    cap = int(num_send_capacity)
    if not 0 <= cap <= 0x7fffffff:
        raise ValueError(f"num_send_capacity = {cap} is out of range")
    if out is None:
        out = q.new_empty((cap, H))
    elif out.dim() != 2 or out.shape[0] < cap:
        raise ValueError("out is too small")
    else:
        _on(out, "out", _FP8, (out.shape[0], H), index)
    if out_scale is None:
        out_scale = scale.new_empty((cap, H // 128))
    elif out_scale.dim() != 2 or out_scale.shape[0] < cap:
        raise ValueError("out_scale is too small")
    else:
        _on(out_scale, "out_scale", _F32, (out_scale.shape[0], H // 128), index)
    st = lib().ep_dispatch_permute_quantized(q.data_ptr(), scale.data_ptr(), H // 128, T, H,
                                             token_row.data_ptr(), K, cap, out.data_ptr(),
                                             out_scale.data_ptr(), _raw_stream(index))
    if st != EP_OK:
        check(st, "ep_dispatch_permute_quantized")
    return out, out_scale
