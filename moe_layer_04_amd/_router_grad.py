"""The router's balance loss and gradients (the entry points of the same names in
include/moe.h)."""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from ._binding import _check
from ._operators import _BF16, _F32, _I32, _arg, _call, _fit, _fn, _new, _p, _sizes, _workspace


@functools.lru_cache(maxsize=256)
def _balance_workspace(M: int, E: int, topk: int) -> int:
    _fit("moe_balance", M, E, topk)
    nbytes = ctypes.c_size_t(0)
    _check(_fn("moe_balance")(None, None, None, M, E, topk, *[None] * 5, ctypes.byref(nbytes), None),
           "moe_balance (size query)")
    return nbytes.value


@functools.lru_cache(maxsize=256)
def _topk_bwd_workspace(rows: int, M: int, K: int, E: int, topk: int) -> int:
    _fit("moe_topk_bwd", rows, M, K, E, topk)
    nbytes = ctypes.c_size_t(0)
    _check(_fn("moe_topk_bwd")(*[None] * 7, rows, M, K, E, topk, *[None] * 4, ctypes.byref(nbytes), None),
           "moe_topk_bwd (size query)")
    return nbytes.value


def _mask(token_mask, M: int, device):
    """bool or uint8 [M], zero for tokens that do not count."""
    if token_mask is not None:
        dtype = torch.uint8 if getattr(token_mask, "dtype", None) is torch.uint8 else torch.bool
        _arg(token_mask, "token_mask", dtype, (M,), device)
    return token_mask


def moe_balance(logits: torch.Tensor, topk_ids: torch.Tensor, *,
                token_mask: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """The balance loss E * sum_e f_e probs[e] of moe_topk's logits [M,E] and ids
    [M,topk]: (loss fp32 [1], counts int32 [E], tokens int32 [1], probs fp32 [E]).
    counts[e]: slots that picked expert e, f_e = counts[e] / (tokens * topk),
    probs: the mean over the tokens of the softmax over all experts.  Tokens whose
    token_mask (bool or uint8 [M]) is zero do not count."""
    M, E = _sizes(logits, "logits", 2)
    dev = logits.device
    _arg(logits, "logits", _F32, (M, E), dev)
    topk = _sizes(topk_ids, "topk_ids", 2)[1]
    _arg(topk_ids, "topk_ids", _I32, (M, topk), dev)
    _mask(token_mask, M, dev)
    need = _balance_workspace(M, E, topk)
    workspace = _workspace(dev, workspace, need, True)
    loss, probs = _new(_F32, dev, 1), _new(_F32, dev, E)
    tokens, counts = _new(_I32, dev, 1), _new(_I32, dev, E)
    _call(dev, "moe_balance", _p(logits), _p(topk_ids), _p(token_mask), M, E, topk, _p(loss), _p(counts),
          _p(tokens), _p(probs), _p(workspace), ctypes.byref(ctypes.c_size_t(workspace.numel())))
    return loss, counts, tokens, probs


def moe_balance_bwd(dloss: torch.Tensor, logits: torch.Tensor, counts: torch.Tensor,
                    tokens: torch.Tensor, topk: int, *,
                    token_mask: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of moe_balance's loss with respect to the logits, fp32 [M,E],
    from dloss (fp32 [1], on the GPU) and the forward's counts and tokens, which
    may be sums over several batches."""
    M, E = _sizes(logits, "logits", 2)
    dev = logits.device
    _arg(logits, "logits", _F32, (M, E), dev)
    _arg(dloss, "dloss", _F32, (1,), dev)
    _arg(counts, "counts", _I32, (E,), dev)
    _arg(tokens, "tokens", _I32, (1,), dev)
    _mask(token_mask, M, dev)
    _fit("moe_balance_bwd", M, E, topk)
    out = _new(_F32, dev, M, E)
    _call(dev, "moe_balance_bwd", _p(dloss), _p(logits), _p(counts), _p(tokens), _p(token_mask), M, E, topk,
          _p(out))
    return out


def moe_topk_bwd(x: torch.Tensor, w_router: torch.Tensor, topk_ids: Optional[torch.Tensor] = None,
                 topk_weights: Optional[torch.Tensor] = None,
                 dtopk_weights: Optional[torch.Tensor] = None, *,
                 dlogits: Optional[torch.Tensor] = None, dx_rows: Optional[torch.Tensor] = None,
                 bias: bool = False, workspace: Optional[torch.Tensor] = None):
    """Gradients of moe_topk from those of its weights (dtopk_weights fp32 [M,topk],
    with topk_ids and topk_weights) and of its logits (dlogits fp32 [M,E]): (dx bf16
    [M,K], dw fp32 [E,K], dbias fp32 [E] or None without ``bias``).  dx_rows bf16
    [M*r,K]: gradients that reach the tokens another way, a token's r rows are
    added to its dx (moe_grouped_gemm_dx with ``scatter`` leaves them so; where
    slots are dropped into an ``out`` of zeros, as it writes the others' rows only).
    A token's dtopk_weights all enter its gradient, also those of ids outside the
    experts: a dropped slot's is zero, as moe_silu_mul_bwd returns it.
    Without topk_ids, topk_weights and dtopk_weights only dlogits is carried on."""
    M, K = _sizes(x, "x", 2)
    dev = x.device
    _arg(x, "x", _BF16, (M, K), dev)
    E = _sizes(w_router, "w_router", 2)[0]
    _arg(w_router, "w_router", _BF16, (E, K), dev)
    topk = 1
    if topk_ids is not None:
        topk = _sizes(topk_ids, "topk_ids", 2)[1]
        _arg(topk_ids, "topk_ids", _I32, (M, topk), dev)
    if (topk_weights is None) != (topk_ids is None) or (dtopk_weights is None) != (topk_ids is None):
        raise ValueError("topk_ids, topk_weights and dtopk_weights go together")
    if topk_ids is not None:
        _arg(topk_weights, "topk_weights", _F32, (M, topk), dev)
        _arg(dtopk_weights, "dtopk_weights", _F32, (M, topk), dev)
    elif dlogits is None:
        raise ValueError("nothing to differentiate: give dtopk_weights or dlogits")
    if dlogits is not None:
        _arg(dlogits, "dlogits", _F32, (M, E), dev)
    rows = 0
    if dx_rows is not None:
        count = _sizes(dx_rows, "dx_rows", 2)[0]
        rows = count // M if M else 0
        if count != rows * M or (M and rows == 0):
            raise ValueError(f"dx_rows must have a multiple of {M} rows, got {count}")
        _arg(dx_rows, "dx_rows", _BF16, (count, K), dev)
    need = _topk_bwd_workspace(rows, M, K, E, topk)
    workspace = _workspace(dev, workspace, need, True)
    dx, dw = _new(_BF16, dev, M, K), _new(_F32, dev, E, K)
    dbias = _new(_F32, dev, E) if bias else None
    _call(dev, "moe_topk_bwd", _p(x), _p(w_router), _p(topk_ids), _p(topk_weights), _p(dtopk_weights),
          _p(dlogits), _p(dx_rows), rows, M, K, E, topk, _p(dx), _p(dw), _p(dbias), _p(workspace),
          ctypes.byref(ctypes.c_size_t(workspace.numel())))
    return dx, dw, dbias
