"""Activations kept in 8 bits for the backward pass: rows of bf16 to codes and
back, and the operators that keep or read them (the entry points of the same
names in include/moe.h).

What is kept of rows [R,W] is two tensors: codes int8 [R,W] and scales uint8
[R,ceil(W/32)], a byte X for every 32 columns; a value is code * 2^(X-133).
"""
from __future__ import annotations

from typing import Optional

import torch

from ._operators import (_BF16, _arg, _call, _fit, _gated, _new, _out, _p, _product_dw, _sizes, _weights_grad)

_I8, _U8 = torch.int8, torch.uint8


def _blocks(width: int) -> int:
    return (width + 31) // 32


def moe_ckpt_rows(x: torch.Tensor):
    """(codes int8 [R,W], scales uint8 [R,ceil(W/32)]) of rows bf16 [R,W]."""
    R, W = _sizes(x, "x", 2)
    dev = x.device
    _arg(x, "x", _BF16, (R, W), dev)
    _fit("moe_ckpt_rows", R, W)
    codes, scales = _new(_I8, dev, R, W), _new(_U8, dev, R, _blocks(W))
    _call(dev, "moe_ckpt_rows", _p(x), R, W, _p(codes), _p(scales))
    return codes, scales


def moe_ckpt_restore(codes: torch.Tensor, scales: torch.Tensor, *,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The rows that moe_ckpt_rows kept, bf16 [R,W]."""
    R, W = _sizes(codes, "codes", 2)
    dev = codes.device
    _arg(codes, "codes", _I8, (R, W), dev)
    _arg(scales, "scales", _U8, (R, _blocks(W)), dev)
    _fit("moe_ckpt_restore", R, W)
    out = _out(out, "out", _BF16, (R, W), dev)
    _call(dev, "moe_ckpt_restore", _p(codes), _p(scales), R, W, _p(out))
    return out


def moe_silu_mul_ckpt(g: torch.Tensor, topk_weights: Optional[torch.Tensor] = None, *,
                      sorted_ids: Optional[torch.Tensor] = None,
                      num_rows: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """moe_silu_mul that also keeps g for moe_silu_mul_bwd_ckpt: (a bf16 [R,N],
    codes int8 [R,2N], scales uint8 [R,2*ceil(N/32)], the halves of a row as rows
    of their own)."""
    dev, R, N, slots = _gated(g, topk_weights, sorted_ids, num_rows)
    _fit("moe_silu_mul_ckpt", R, N, slots)
    out = _out(out, "out", _BF16, (R, N), dev)
    codes, scales = _new(_I8, dev, R, 2 * N), _new(_U8, dev, R, 2 * _blocks(N))
    _call(dev, "moe_silu_mul_ckpt", _p(g), _p(topk_weights), _p(sorted_ids), _p(num_rows), slots, R, N,
          _p(out), _p(codes), _p(scales))
    return out, codes, scales


def moe_silu_mul_bwd_ckpt(da: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                          topk_weights: Optional[torch.Tensor] = None, *,
                          sorted_ids: Optional[torch.Tensor] = None,
                          num_rows: Optional[torch.Tensor] = None, again: bool = True):
    """Gradients of moe_silu_mul_ckpt from what it kept: (dg bf16 [R,2N],
    dtopk_weights in topk_weights' shape or None, a bf16 [R,N] -- the forward's
    output from what was kept, which the gradient of the down weights reads -- or
    None without ``again``).  Weights of slots that no row names get a gradient of
    zero; rows at and past num_rows are not written."""
    dev, R, N, slots = _gated(codes, topk_weights, sorted_ids, num_rows, "codes", _I8)
    _fit("moe_silu_mul_bwd_ckpt", R, N, slots)
    _arg(da, "da", _BF16, (R, N), dev)
    _arg(scales, "scales", _U8, (R, 2 * _blocks(N)), dev)
    dg = _new(_BF16, dev, R, 2 * N)
    dw = _weights_grad(topk_weights, sorted_ids, num_rows)
    a = _new(_BF16, dev, R, N) if again else None
    _call(dev, "moe_silu_mul_bwd_ckpt", _p(da), _p(codes), _p(scales), _p(topk_weights), _p(sorted_ids),
          _p(num_rows), slots, R, N, _p(dg), _p(dw), _p(a))
    return dg, dw, a


def moe_grouped_gemm_dw_ckpt(dy: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                             expert_offsets: torch.Tensor, *,
                             sorted_ids: Optional[torch.Tensor] = None, topk: int = 1,
                             num_tokens: Optional[int] = None, gather_dy: bool = False,
                             gather_x: bool = False, out_dtype: torch.dtype = torch.bfloat16,
                             out: Optional[torch.Tensor] = None, accumulate: bool = False,
                             workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_grouped_gemm_dw with x kept by moe_ckpt_rows: codes int8 [R,K] or,
    with ``gather_x``, [num_tokens,K], and their scales."""
    nx, K = _sizes(codes, "codes", 2)
    dev = codes.device
    _arg(codes, "codes", _I8, (nx, K), dev)
    _arg(scales, "scales", _U8, (nx, _blocks(K)), dev)
    return _product_dw("moe_grouped_gemm_dw_ckpt", dev, dy, (codes.data_ptr(), scales.data_ptr()),
                       codes.shape, expert_offsets, sorted_ids, topk, num_tokens, gather_dy, gather_x,
                       out_dtype, out, accumulate, workspace)
