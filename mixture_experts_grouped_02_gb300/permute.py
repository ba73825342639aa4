"""Token rows to the expert-sorted list of :func:`align` and back, with their
gradients: shape checks and output buffers around moe_permute_tokens,
moe_unpermute_tokens and their ``_backward`` entry points.

``plan`` is the dict :func:`align` (or :func:`route_align`) returns; its
``inv_perm`` (T*K) and ``sorted_ids`` (cap) are read.  Rows are contiguous
(rows, H) tensors; outputs are allocated when not given.

Like every call of the package these compute on tensors and record nothing for
autograd, also where an input requires a gradient: a training step calls the
``_backward`` functions, or wraps both in a torch.autograd.Function as
examples/fp8_expert_layer.py does.
"""
from __future__ import annotations

import contextlib

import torch

from . import _abi

_ROWS = {torch.bfloat16: _abi.MOE_BF16, torch.float32: _abi.MOE_F32}
_COPIED = {**_ROWS, torch.uint8: _abi.MOE_E4M3, torch.float8_e4m3fn: _abi.MOE_E4M3}


def _dtype(t, allowed):
    code = allowed.get(t.dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return code


def _lists(plan):
    inv, ids = plan["inv_perm"], plan["sorted_ids"]
    if inv.dtype != torch.int32 or ids.dtype != torch.int32:
        raise ValueError("inv_perm and sorted_ids are int32 tensors")
    return inv, ids, ids.numel()


def _rows(t, rows, H, dtype, what):
    if t.shape != (rows, H) or t.dtype != dtype:
        raise ValueError(f"{what}: expected a ({rows}, {H}) {dtype} tensor, got "
                         f"{tuple(t.shape)} {t.dtype}")
    return t


def _on(stream):
    """Context in which buffers for kernels on `stream` (None: the current
    one) are allocated, so that the allocator orders their reuse on it."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        # ExternalStream(0) would be a new stream of torch's pool; 1 is the
        # runtime's other handle of the default stream
        stream = (torch.cuda.default_stream() if stream in (0, 1)
                  else torch.cuda.ExternalStream(stream))
    return torch.cuda.stream(stream)


def _empty(shape, dtype, device, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _out(t, rows, H, like, what, stream):
    if t is None:
        return _empty((rows, H), like.dtype, like.device, stream)
    return _rows(t, rows, H, like.dtype, what)


def _topk(n_assign, T, what):
    if T == 0 or n_assign % T != 0:
        if T == 0 and n_assign == 0:
            return 1
        raise ValueError(f"{what}: inv_perm has {n_assign} entries for {T} tokens")
    return n_assign // T


def _weights(w, n_assign):
    if w.dim() != 2 or w.dtype != torch.float32 or w.numel() != n_assign:
        raise ValueError("topk_weights: expected (T, K) float32 as the plan's T*K assignments")
    return w.shape


def permute_tokens(x, plan, out=None, dev_status=None, stream=None):
    """Rows of x (T, H) at every slot their token occupies, (cap, H); rows of
    padding slots are zero.  bf16, fp32, or e4m3 codes (uint8 or
    float8_e4m3fn)."""
    code = _dtype(x, _COPIED)
    inv, ids, cap = _lists(plan)
    T, H = x.shape
    K = _topk(inv.numel(), T, "permute_tokens")
    out = _out(out, cap, H, x, "out", stream)
    _abi.moe_permute_tokens(x, code, T, H, K, inv, ids, cap, out, dev_status, stream)
    return out


def permute_tokens_backward(grad_sorted, plan, K, out=None, dev_status=None, stream=None):
    """Gradient of permute_tokens: for each token the sum of the rows of its
    K slots, (T, H).  Padding rows are not read."""
    code = _dtype(grad_sorted, _ROWS)
    inv, _, cap = _lists(plan)
    if K <= 0 or inv.numel() % K != 0:
        raise ValueError(f"permute_tokens_backward: {inv.numel()} assignments, K = {K}")
    T, H = inv.numel() // K, grad_sorted.shape[-1]
    _rows(grad_sorted, cap, H, grad_sorted.dtype, "grad_sorted")
    out = _out(out, T, H, grad_sorted, "out", stream)
    _abi.moe_permute_tokens_backward(grad_sorted, code, T, H, K, inv, cap, out, dev_status, stream)
    return out


def unpermute_tokens(y, plan, topk_weights, out=None, dev_status=None, stream=None):
    """out[t] = sum_k topk_weights[t, k] * (row of y at the slot of choice k),
    (T, H), summed in fp32.  Padding rows of y (cap, H) are not read."""
    code = _dtype(y, _ROWS)
    inv, _, cap = _lists(plan)
    T, K = _weights(topk_weights, inv.numel())
    H = y.shape[-1]
    _rows(y, cap, H, y.dtype, "y")
    out = _out(out, T, H, y, "out", stream)
    _abi.moe_unpermute_tokens(y, code, T, H, K, topk_weights, inv, cap, out, dev_status, stream)
    return out


def unpermute_tokens_backward(grad_out, y, plan, topk_weights, out=None, dev_status=None,
                              stream=None):
    """Gradients of unpermute_tokens: (grad_y (cap, H), zero in padding rows;
    grad_weights (T, K) fp32)."""
    code = _dtype(y, _ROWS)
    inv, ids, cap = _lists(plan)
    T, K = _weights(topk_weights, inv.numel())
    H = y.shape[-1]
    _rows(y, cap, H, y.dtype, "y")
    _rows(grad_out, T, H, y.dtype, "grad_out")
    out = _out(out, cap, H, y, "out", stream)
    grad_w = _empty((T, K), torch.float32, y.device, stream)
    _abi.moe_unpermute_tokens_backward(grad_out, y, code, T, H, K, topk_weights, inv, ids, cap,
                                       out, grad_w, dev_status, stream)
    return out, grad_w
