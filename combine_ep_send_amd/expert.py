"""Thin PyTorch binding of the expert-side calls (include/epdc_expert.h): the
experts' products for a few rows, a whole expert layer for a few tokens, the
gated activation with its 8-bit checkpoint, and the gradient of the combine.

As in ``ops``, the functions mirror the C entry points: they check dtypes,
shapes and devices, allocate outputs the caller did not pass, and enqueue on
the current (or given) HIP stream.  They run on the device of their tensors,
whichever is current.  They record nothing for autograd: outputs
do not require gradients even where an input does, without an error or a
warning.  The backward passes are calls of their own, to be made by hand or
from a ``torch.autograd.Function``."""

from __future__ import annotations

import functools
from typing import NamedTuple, Optional, Tuple, Union

import torch

from ._lib import EP_OK, EP_W_BF16, EP_W_FP4, EP_W_INT4, check, lib
from .ops import _gpu, _shape

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


# The calls take microseconds on the GPU, so the host's share counts: a check
# that passes costs a few attribute reads, and only one that fails goes through
# the named checks for its message.  The raw handle of the current stream costs
# a thirtieth of torch.cuda.current_stream() (0.1 against 2.9 us).

_INT_MAX = 0x7fffffff


def _int(v: int, name: str) -> int:
    # ctypes would drop the upper bits
    if not -_INT_MAX <= v <= _INT_MAX:
        raise ValueError(f"{name} = {v} is out of range")
    return v


def _raw_stream(index: int) -> int:
    return torch._C._cuda_getCurrentRawStream(index)


def _first(t, name: str, dtype, ndim: int) -> int:
    """Checks a call's first tensor and returns its device's index."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.dim() == ndim
            and t.is_contiguous()):
        _gpu(t, name, dtype, ndim)
    return t.get_device()


def _on(t, name: str, dtype, shape, index: int) -> torch.Tensor:
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == index and t.is_contiguous()):
        _shape(_gpu(t, name, dtype), name, shape)
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    return t


def _elsewhere(index: int, stream) -> bool:
    return stream is not None or index != torch._C._cuda_getDevice()


def _there(fn, index: int, stream, *args, **kw):
    """fn with its tensors' device current, and the stream that was given, so
    that outputs allocated inside belong to both."""
    if stream is None:
        with torch.cuda.device(index):
            return fn(*args, **kw)
    if stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _weights(w: Weights, name: str, index: int):
    """(E, N, K, format, group, q, scale) of bf16 [E, N, K] or W4Weights."""
    if isinstance(w, W4Weights):
        q, scale, form, group = w
        fmt = _W4_FMT.get(form)
        if fmt is None:
            raise ValueError(f"{name}.fmt must be one of {sorted(_W4_FMT)}")
        if _first(q, f"{name}.q", _U8, 3) != index:
            raise ValueError(f"{name}.q is on {q.device}, not on cuda:{index}")
        E, N, half = q.shape
        if group not in (32, 64, 128):
            raise ValueError(f"{name}.group must be 32, 64 or 128")
        if max(E, N, half) > _INT_MAX // 2:
            raise ValueError(f"{name} is too large: {tuple(q.shape)}")
        _on(scale, f"{name}.scale", _W4_SCALE[form], (E, N, 2 * half // group), index)
        return E, N, 2 * half, fmt, group, q.data_ptr(), scale.data_ptr()
    if _first(w, name, _BF16, 3) != index:
        raise ValueError(f"{name} is on {w.device}, not on cuda:{index}")
    E, N, K = w.shape
    if max(E, N, K) > _INT_MAX:
        raise ValueError(f"{name} is too large: {tuple(w.shape)}")
    return E, N, K, EP_W_BF16, 0, w.data_ptr(), None


def ep_quantize_w4(w: torch.Tensor, fmt: str = "int4", group: Optional[int] = None, *,
                   out: Optional[W4Weights] = None, stream=None) -> W4Weights:
    """bf16 matrices [.., N, K] to 4 bits (int4: group 128 unless given; fp4:
    group 32).  K is a multiple of 128."""
    if fmt not in _W4_FMT:
        raise ValueError(f"fmt must be one of {sorted(_W4_FMT)}")
    _gpu(w, "w", _BF16)
    if w.dim() < 1:
        raise ValueError("w must be [.., N, K]")
    index = w.get_device()
    if _elsewhere(index, stream):
        return _there(ep_quantize_w4, index, stream, w, fmt, group, out=out)
    group = int(group) if group is not None else (32 if fmt == "fp4" else 128)
    K = _int(w.shape[-1], "K")
    if group not in (32, 64, 128) or K < 1 or K % 128:
        raise ValueError("K must be a multiple of 128 and group 32, 64 or 128")
    qs, ss = (*w.shape[:-1], K // 2), (*w.shape[:-1], K // group)
    if out is None:
        out = W4Weights(w.new_empty(qs, dtype=_U8), w.new_empty(ss, dtype=_W4_SCALE[fmt]), fmt,
                        group)
    if out.fmt != fmt or int(out.group) != group:
        raise ValueError("out has another format")
    _on(out.q, "out.q", _U8, qs, index)
    _on(out.scale, "out.scale", _W4_SCALE[fmt], ss, index)
    st = lib().ep_quantize_w4(w.data_ptr(), w.numel() // K, K, _W4_FMT[fmt], group,
                              out.q.data_ptr(), out.scale.data_ptr(), _raw_stream(index))
    check(st, "ep_quantize_w4")
    return out


def ep_expert_matvec(x: torch.Tensor, weights: Weights, row_expert: Optional[torch.Tensor] = None,
                     *, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y [R, N] bf16 with y[r] = W[row_expert[r]] x[r], for up to 1024 rows x
    [R, K] bf16 and matrices [E, N, K] (bf16 or W4Weights).  ``row_expert``
    [R] int32 may be left out for one matrix.  Rows whose id lies outside
    [0, E) get zeros."""
    index = _first(x, "x", _BF16, 2)
    if _elsewhere(index, stream):
        return _there(ep_expert_matvec, index, stream, x, weights, row_expert, out=out)
    R, K = x.shape
    E, N, wk, fmt, group, q, scale = _weights(weights, "weights", index)
    if wk != K:
        raise ValueError(f"weights have {wk} channels, x has {K}")
    if row_expert is not None:
        _on(row_expert, "row_expert", _I32, (R,), index)
    elif E != 1:
        raise ValueError("row_expert is needed for more than one expert")
    if out is None:
        out = x.new_empty((R, N))
    else:
        _on(out, "out", _BF16, (R, N), index)
    st = lib().ep_expert_matvec(x.data_ptr(), _ptr(row_expert), R, E, N, K, fmt, group, q, scale,
                                out.data_ptr(), _raw_stream(index))
    if st != EP_OK:
        check(st, "ep_expert_matvec")
    return out


@functools.lru_cache(maxsize=1024)
def ep_moe_tokens_workspace_bytes(num_tokens: int, num_topk: int, hidden: int,
                                  inner: int) -> int:
    sizes = [int(v) for v in (num_tokens, num_topk, hidden, inner)]
    if max(map(abs, sizes)) > _INT_MAX:
        return 0
    return int(lib().ep_moe_tokens_workspace_bytes(*sizes))


def ep_moe_tokens(x: torch.Tensor, topk_idx: torch.Tensor, topk_weights: torch.Tensor,
                  w13: Weights, w2: Weights, first_expert: int = 0, *, bias=None,
                  out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """out [T, H] bf16 of a whole expert layer for up to 128 tokens (T*K up to
    1024), in two or three launches: out[t] = sum over the slots whose expert e =
    topk_idx[t, k] - first_expert is one of the E here of topk_weights[t, k] *
    W2[e] (silu(gate) * up), the gate and up rows being W13[e] x[t].  ``w13``
    [E, 2I, H] (the gate rows, then the up rows) and ``w2`` [E, H, I] are bf16 or
    W4Weights; ``bias`` is a [T, H] bf16 tensor or
    a pair, added in fp32 before the one rounding, as in ep_combine.

    Without ``workspace`` (uint8, ep_moe_tokens_workspace_bytes of it) each
    call takes its own from PyTorch's allocator, so calls on several streams
    and captured graphs never share one."""
    index = _first(x, "x", _BF16, 2)
    if _elsewhere(index, stream):
        return _there(ep_moe_tokens, index, stream, x, topk_idx, topk_weights, w13, w2,
                      first_expert, bias=bias, out=out, workspace=workspace)
    T, H = x.shape
    _first(topk_idx, "topk_idx", _I64, 2)
    K = _int(topk_idx.shape[1], "K")
    _on(topk_idx, "topk_idx", _I64, (T, K), index)
    _on(topk_weights, "topk_weights", _F32, (T, K), index)
    E, N13, K13, fmt13, group13, q13, scale13 = _weights(w13, "w13", index)
    E2, N2, I, fmt2, group2, q2, scale2 = _weights(w2, "w2", index)
    if E2 != E or N2 != H or K13 != H or N13 != 2 * I:
        raise ValueError(f"w13 must be [E, 2I, {H}] and w2 [E, {H}, I], got "
                         f"[{E}, {N13}, {K13}] and [{E2}, {N2}, {I}]")
    b0 = b1 = None
    if bias is not None:
        pair = tuple(bias) if isinstance(bias, (tuple, list)) else (bias,)
        if len(pair) > 2:
            raise ValueError("bias is one [T, H] tensor or a pair")
        ptrs = [_on(b, f"bias[{i}]", _BF16, (T, H), index).data_ptr() for i, b in enumerate(pair)]
        b0, b1 = (ptrs + [None, None])[:2]
    if out is None:
        out = torch.empty_like(x)
    else:
        _on(out, "out", _BF16, (T, H), index)
    if workspace is None:
        workspace = x.new_empty(ep_moe_tokens_workspace_bytes(T, K, H, I), dtype=_U8)
    elif _first(workspace, "workspace", _U8, 1) != index:
        raise ValueError(f"workspace is on {workspace.device}, not on cuda:{index}")
    st = lib().ep_moe_tokens(
        x.data_ptr(), topk_idx.data_ptr(), topk_weights.data_ptr(), T, K, H, I,
        _int(int(first_expert), "first_expert"), E, fmt13, group13, q13, scale13, fmt2, group2, q2,
        scale2, b0, b1, out.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _raw_stream(index))
    if st != EP_OK:
        check(st, "ep_moe_tokens")
    return out


def ep_swiglu_fp8(gate_up: torch.Tensor, *, row_count: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                  scale: Optional[torch.Tensor] = None, stream=None
                  ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(h [R, I] bf16 = silu(gate) * up, q [R, 2I] float8_e4m3fn, scale
    [R, 2I/128] float32) of gate_up [R, 2I] bf16 (I gate channels, then I up
    channels; I a multiple of 128).  q and scale are the checkpoint that
    ep_swiglu_fp8_backward takes in place of gate_up and h.  Rows from
    ``row_count`` ([1] int32 on the device, e.g. ``expert_offsets[-1:]``) on
    are left as they are."""
    index = _first(gate_up, "gate_up", _BF16, 2)
    if _elsewhere(index, stream):
        return _there(ep_swiglu_fp8, index, stream, gate_up, row_count=row_count, out=out, q=q,
                      scale=scale)
    R, two = gate_up.shape
    if two % 256 or two == 0:
        raise ValueError("gate_up must be [R, 2I] with I a multiple of 128")
    I = _int(two // 2, "I")
    if row_count is not None:
        _on(row_count, "row_count", _I32, (1,), index)
    h = gate_up.new_empty((R, I)) if out is None else _on(out, "out", _BF16, (R, I), index)
    q = gate_up.new_empty((R, two), dtype=_FP8) if q is None else \
        _on(q, "q", _FP8, (R, two), index)
    scale = gate_up.new_empty((R, two // 128), dtype=_F32) if scale is None else \
        _on(scale, "scale", _F32, (R, two // 128), index)
    st = lib().ep_swiglu_fp8(gate_up.data_ptr(), R, I, _ptr(row_count), h.data_ptr(), q.data_ptr(),
                             scale.data_ptr(), _raw_stream(index))
    if st != EP_OK:
        check(st, "ep_swiglu_fp8")
    return h, q, scale


def ep_swiglu_fp8_backward(dh: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, *,
                           row_count: Optional[torch.Tensor] = None, recompute: bool = True,
                           out: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                           stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(d_gate_up [R, 2I] bf16, h [R, I] bf16) from dh [R, I] bf16 and the
    checkpoint of ep_swiglu_fp8: the gradient of silu(gate) * up at the values
    the checkpoint stands for, and that product itself (what the second
    product's weight gradient takes), None without ``recompute``."""
    index = _first(dh, "dh", _BF16, 2)
    if _elsewhere(index, stream):
        return _there(ep_swiglu_fp8_backward, index, stream, dh, q, scale, row_count=row_count,
                      recompute=recompute, out=out, h=h)
    R, I = dh.shape
    if _int(I, "I") % 128 or I == 0:
        raise ValueError("dh must be [R, I] with I a multiple of 128")
    _on(q, "q", _FP8, (R, 2 * I), index)
    _on(scale, "scale", _F32, (R, I // 64), index)
    if row_count is not None:
        _on(row_count, "row_count", _I32, (1,), index)
    d = dh.new_empty((R, 2 * I)) if out is None else _on(out, "out", _BF16, (R, 2 * I), index)
    if not recompute:
        if h is not None:
            raise ValueError("h is an output of recompute=True")
    elif h is None:
        h = dh.new_empty((R, I))
    else:
        _on(h, "h", _BF16, (R, I), index)
    st = lib().ep_swiglu_fp8_backward(dh.data_ptr(), q.data_ptr(), scale.data_ptr(), R, I,
                                      _ptr(row_count), d.data_ptr(), _ptr(h), _raw_stream(index))
    if st != EP_OK:
        check(st, "ep_swiglu_fp8_backward")
    return d, h


def ep_combine_backward(dout: torch.Tensor, y: Optional[torch.Tensor], token_row: torch.Tensor,
                        topk_weights: Optional[torch.Tensor], *, weight_grad: Optional[bool] = None,
                        num_rows: Optional[int] = None, dy: Optional[torch.Tensor] = None,
                        dw: Optional[torch.Tensor] = None, stream=None
                        ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gradient of ep_combine: (dy, shaped as y, bf16; dw [T, K] float32).
    dy[r] = (the sum of the weights of the slots that name row r) * dout[t],
    dw[t, k] = <dout[t], y[token_row[t, k]]>.  With ``topk_weights=None`` (the
    unweighted combine) or ``weight_grad=False`` dw is None and y is not read:
    it may then be None, with ``num_rows`` or ``dy`` giving the rows.  Rows no
    slot names are left as they are in ``dy``, with what an earlier layout left
    there; a result allocated here has zeros.  The gradient of a combine's bias is dout itself.

    With a regroup's ``row_map`` and the received rows' weights in place of
    ``token_row`` and ``topk_weights`` it is the gradient of restore_by_expert;
    that of permute_by_expert is ``ep_combine(d_perm_x, row_map, None)``."""
    index = _first(dout, "dout", _BF16, 2)
    if _elsewhere(index, stream):
        return _there(ep_combine_backward, index, stream, dout, y, token_row, topk_weights,
                      weight_grad=weight_grad, num_rows=num_rows, dy=dy, dw=dw)
    T, H = dout.shape
    _int(H, "H")
    _first(token_row, "token_row", _I32, 2)
    K = _int(token_row.shape[1], "K")
    _on(token_row, "token_row", _I32, (T, K), index)
    if topk_weights is not None:
        _on(topk_weights, "topk_weights", _F32, (T, K), index)
    if weight_grad is None:
        weight_grad = topk_weights is not None
    elif weight_grad and topk_weights is None:
        raise ValueError("weight_grad needs topk_weights")
    if y is not None:
        shape = tuple(y.shape)
        _on(y, "y", _BF16, shape, index)
    elif weight_grad:
        raise ValueError("the weights' gradient needs y")
    elif dy is not None:
        shape = tuple(dy.shape)
    elif num_rows is not None:
        shape = (int(num_rows), H)
    else:
        raise ValueError("without y, num_rows or dy gives the rows")
    if len(shape) < 2 or shape[-1] != H:
        raise ValueError(f"y and dy must be [.., {H}], got {shape}")
    if dy is None:
        dy = dout.new_zeros(shape)
    else:
        _on(dy, "dy", _BF16, shape, index)
    rows = dy.numel() // H if H else 0
    if num_rows is not None and int(num_rows) != rows:
        raise ValueError(f"num_rows is {num_rows}, the buffers have {rows}")
    if not weight_grad:
        if dw is not None:
            raise ValueError("dw is an output of weight_grad=True")
    elif dw is None:
        dw = dout.new_empty((T, K), dtype=_F32)
    else:
        _on(dw, "dw", _F32, (T, K), index)
    st = lib().ep_combine_backward(dout.data_ptr(), y.data_ptr() if weight_grad else None, rows,
                                   token_row.data_ptr(), _ptr(topk_weights), T, K, H,
                                   dy.data_ptr(), _ptr(dw), _raw_stream(index))
    if st != EP_OK:
        check(st, "ep_combine_backward")
    return dy, dw
