"""e4m3 operands with fp32 scales per block of 128: the quantiser, the plain
and the grouped product, and the expert FFN made of them.

Formats (those of DeepSeek-V3's fp8 checkpoints): activations (T, H) codes
with scales (T, ceil(H/128)); weights (..., N, K) codes with scales (...,
ceil(N/128), ceil(K/128)).  Codes are float8_e4m3fn or uint8 tensors.
"""
from __future__ import annotations

import torch

from . import _abi
from .permute import (_dtype, _empty, _lists, _on, _ROWS, permute_tokens,
                      unpermute_tokens)


def _nblk(n):
    return (n + 127) // 128


_CODES = (torch.float8_e4m3fn, torch.uint8)


def _codes(t, shape, what):
    if t.dtype not in _CODES:
        raise ValueError(f"{what}: expected e4m3 codes, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {shape}, got {tuple(t.shape)}")


def _scales(t, shape, what):
    if t.dtype != torch.float32 or t.shape != shape:
        raise ValueError(f"{what}: expected float32 {shape}, got {t.dtype} {tuple(t.shape)}")


def _result(out, rows, N, dtype, device, stream):
    if out is None:
        out = _empty((rows, N), dtype, device, stream)
    elif out.shape != (rows, N):
        raise ValueError(f"out: expected shape ({rows}, {N}), got {tuple(out.shape)}")
    return out, _dtype(out, _ROWS)


def quantize_fp8_block(x, gated=False, out=None, stream=None):
    """(codes (T, H) float8_e4m3fn, scales (T, ceil(H/128)) fp32) of x (T, H),
    or with gated of SiLU(gate) * up for x (T, 2H) holding gate then up.
    out: a (codes, scales) pair to write instead.  Every row is encoded: of a
    sorted list the padding rows too, whatever they hold."""
    code = _dtype(x, _ROWS)
    T, H = x.shape
    if gated:
        if H % 2 != 0:
            raise ValueError("gated: an even number of columns (gate, up) is needed")
        H //= 2
    if out is None:
        out = (_empty((T, H), torch.float8_e4m3fn, x.device, stream),
               _empty((T, _nblk(H)), torch.float32, x.device, stream))
    else:
        _codes(out[0], (T, H), "out codes")
        _scales(out[1], (T, _nblk(H)), "out scales")
    _abi.moe_quantize_fp8_block(x, code, T, H, gated, out[0], out[1], stream)
    return out


def gemm_fp8_block(a, a_scale, w, w_scale, out=None, out_dtype=torch.bfloat16, dev_status=None,
                   stream=None):
    """a (M, K) times w (N, K) transposed, (M, N) in out_dtype (bf16 or fp32)."""
    M, K = a.shape
    N = w.shape[0]
    _codes(a, (M, K), "a")
    _codes(w, (N, K), "w")
    _scales(a_scale, (M, _nblk(K)), "a_scale")
    _scales(w_scale, (_nblk(N), _nblk(K)), "w_scale")
    out, code = _result(out, M, N, out_dtype, a.device, stream)
    _abi.moe_gemm_fp8_block(a, a_scale, w, w_scale, M, N, K, out, code, dev_status, stream)
    return out


def grouped_gemm_fp8_block(a, a_scale, w, w_scale, plan, block_m=128, out=None,
                           out_dtype=torch.bfloat16, dev_status=None, stream=None):
    """The sorted rows a (cap, K) times their experts' w (E, N, K) transposed,
    (cap, N); `plan` and `block_m` as given to :func:`align`, over at most
    the E experts that w holds.  Rows of padding slots of out are not written."""
    rows, K = a.shape
    E, N = w.shape[0], w.shape[1]
    cap = _lists(plan)[2]
    info, num = plan["block_info"], plan["num_blocks"]
    if block_m <= 0 or info.shape != (cap // block_m, 4):
        raise ValueError(f"block_info {tuple(info.shape)} does not fit {cap} slots in blocks of "
                         f"{block_m}")
    if info.dtype != torch.int32 or num.dtype != torch.int32:
        raise ValueError("block_info and num_blocks are int32 tensors")
    # block_info's expert ids index w and w_scale: a list over other experts
    # would be read past their end
    counts = plan.get("counts")
    if counts is not None and counts.numel() > E:
        raise ValueError(f"the plan is over {counts.numel()} experts, w holds {E}")
    _codes(a, (cap, K), "a")
    _codes(w, (E, N, K), "w")
    _scales(a_scale, (cap, _nblk(K)), "a_scale")
    _scales(w_scale, (E, _nblk(N), _nblk(K)), "w_scale")
    out, code = _result(out, rows, N, out_dtype, a.device, stream)
    _abi.moe_grouped_gemm_fp8_block(a, a_scale, w, w_scale, E, N, K, cap, block_m, info, num, out,
                                    code, dev_status, stream)
    return out


def forward_fp8_block(x, topk_ids, topk_weights, w13, w13_scale, w2, w2_scale, block_m=None,
                      num_experts=None, expert_base=0, out=None, dev_status=None, stream=None):
    """The MoE expert FFN with 128-block fp8 weights: x (T, H) bf16 or fp32
    routed by (topk_ids, topk_weights) over w13 (L, 2I, H) (gate rows, then up
    rows) and w2 (L, H, I).  Both activations are quantised per 128 columns.
    With num_experts given, the weights are those of the shard [expert_base,
    expert_base + L) and out is its share of the layer output.  block_m: rows
    per align block, by default 16 while the experts receive at most 16 rows
    on average and 128 above.  dev_status: an int32 status word of the
    caller's, zero at the start (one is made otherwise): an expert id out of
    range is reported there; permutation and products then do nothing and out is
    not written, while the quantisers, which index nothing by the lists, encode
    what their buffers hold."""
    from . import align
    T, H = x.shape
    if topk_ids.dtype != torch.int32 or topk_ids.dim() != 2 or topk_ids.shape[0] != T:
        raise ValueError(f"topk_ids: expected (T, K) int32, got {tuple(topk_ids.shape)} "
                         f"{topk_ids.dtype}")
    L = w13.shape[0]
    K = topk_ids.shape[1]
    E = L if num_experts is None else num_experts
    if block_m is None:
        block_m = 16 if T * K <= 16 * E else 128
    # every buffer below is made and used on the one stream
    with _on(stream):
        if out is None:
            out = torch.empty((T, H), dtype=x.dtype, device=x.device)
        if T == 0:
            return out
        d = _abi._gpu(x)
        for t in (topk_ids, topk_weights, w13, w13_scale, w2, w2_scale, out, dev_status):
            _abi._p(t, d)  # before the first step
        if dev_status is None:
            dev_status = torch.zeros(1, dtype=torch.int32, device=x.device)
        plan = align(topk_ids, E, block_m, dev_status, None, expert_base,
                     0 if num_experts is None else L)
        xq, xs = quantize_fp8_block(x)
        a = permute_tokens(xq, plan, dev_status=dev_status)
        a_scale = permute_tokens(xs, plan, dev_status=dev_status)
        gu = grouped_gemm_fp8_block(a, a_scale, w13, w13_scale, plan, block_m,
                                    dev_status=dev_status)
        hq, hs = quantize_fp8_block(gu, gated=True)
        y = grouped_gemm_fp8_block(hq, hs, w2, w2_scale, plan, block_m, out_dtype=x.dtype,
                                   dev_status=dev_status)
        return unpermute_tokens(y, plan, topk_weights, out, dev_status)
