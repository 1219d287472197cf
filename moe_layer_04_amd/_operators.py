"""The layer in pieces, with gradients: matrix products grouped by expert, the
gated activation between them and the norms around the block (the entry
points of the same names in include/moe.h).

As in the rest of the binding, tensors are dense and checked here, outputs
and workspaces are torch allocations unless given, and the work runs on the
current stream of the tensors' device.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from ._binding import MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MoEError, _check, load_library

MOE_ROWS_GATHER = 1
MOE_ROWS_SCATTER = 2
MOE_ROWS_GATHER_DY = 4

MOE_OUT_BF16 = 0
MOE_OUT_FP32 = 1
MOE_OUT_FP32_ADD = 2

MOE_PRODUCT_FWD = 0
MOE_PRODUCT_DX = 1
MOE_PRODUCT_DW = 2

MOE_PRODUCT_STREAM = 0
MOE_PRODUCT_TILES_64 = 1
MOE_PRODUCT_TILES_128 = 2
MOE_PRODUCT_TILES_256 = 3

_UNUSED = 256  # workspace bytes of a product that needs none

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _arg(t, name: str, dtype, shape, device):
    """A dense tensor of this dtype and shape (None: any) on this GPU.  One
    expression for the case that everything fits: these checks run before every
    call, and the shortest kernels here take a few microseconds."""
    try:
        if (t.dtype is dtype and (shape is None or t.shape == shape) and t.device == device
                and t.is_contiguous()):
            return t
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other tensors on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _sizes(t, name: str, dims: int):
    """The shape of the tensor whose device is the call's."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != dims:
        raise ValueError(f"{name} must be a {dims}-dimensional GPU tensor")
    return t.shape


def _fit(name: str, *sizes: int):
    """ctypes cuts sizes to 32 bits without an error: what does not fit is not
    supported (the library's own limits are lower)."""
    if max(sizes) > 0x7FFFFFFF or min(sizes) < -0x80000000:
        raise MoEError(MOE_ERR_UNSUPPORTED, name)


def _new(dtype, device, rows: int, cols: Optional[int] = None) -> torch.Tensor:
    # the cheapest of torch's allocations, 0.4 us below torch.empty
    if cols is None:
        return torch.empty_strided((rows,), (1,), dtype=dtype, device=device)
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=None)
def _fn(name: str):
    return getattr(load_library(), name)


def _call(device: torch.device, name: str, *args):
    """One library call on the device's current stream, with that device
    current."""
    index = device.index
    if torch._C._cuda_getDevice() == index:
        rc = _fn(name)(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            rc = _fn(name)(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc:
        _check(rc, name)


def _out(out, name: str, dtype, shape, device):
    if out is None:
        return (_new(dtype, device, *shape) if len(shape) == 2
                else torch.empty(shape, dtype=dtype, device=device))
    return _arg(out, name, dtype, shape, device)


@functools.lru_cache(maxsize=None)
def _unused(device) -> torch.Tensor:
    return torch.empty(_UNUSED, dtype=torch.uint8, device=device)


def _workspace(device, workspace, nbytes: int, product: bool = False):
    """The caller's workspace, or one allocated here; the library checks the
    size.  A product that reports the least size does not touch it: one buffer
    serves all of them."""
    if workspace is None:
        if product and nbytes == _UNUSED:
            return _unused(device)
        return _new(torch.uint8, device, nbytes)
    _arg(workspace, "workspace", torch.uint8, None, device)
    if workspace.numel() < nbytes:  # an empty one's null pointer would ask for the size
        raise MoEError(MOE_ERR_WORKSPACE, f"workspace of {workspace.numel()} bytes, {nbytes} needed:")
    return workspace


@functools.lru_cache(maxsize=1024)
def _product_workspace(name: str, *sizes) -> int:
    _fit(name, *sizes)
    nbytes = ctypes.c_size_t(0)
    _check(_fn(name)(None, None, None, None, *sizes, None, None, ctypes.byref(nbytes), None),
           f"{name} (size query)")
    return nbytes.value


@functools.lru_cache(maxsize=256)
def _norm_workspace(kind: int, M: int, K: int, topk: int, du_topk: int) -> int:
    _fit("moe_block_norm_bwd", M, K, topk, du_topk)
    nbytes = ctypes.c_size_t(0)
    _check(_fn("moe_block_norm_bwd")(*[None] * 9, kind, M, K, topk, du_topk, 1.0, *[None] * 6,
                                     ctypes.byref(nbytes), None),
           "moe_block_norm_bwd (size query)")
    return nbytes.value


class ProductPlan(ctypes.Structure):
    """moe_product_plan of include/moe.h."""
    _fields_ = [("kernel", ctypes.c_int32), ("splits", ctypes.c_int32),
                ("workgroups", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("workspace_bytes", ctypes.c_uint64)]


def grouped_plan(op: int, R: int, E: int, K: int, N: int) -> ProductPlan:
    """The library's launch plan of a product grouped by expert (MOE_PRODUCT_FWD,
    _DX or _DW) of R sorted rows; no GPU call is made."""
    _fit("moe_grouped_plan", op, R, E, K, N)
    plan = ProductPlan()
    _check(_fn("moe_grouped_plan")(op, R, E, K, N, ctypes.byref(plan)), "moe_grouped_plan")
    return plan


def _rows(sorted_ids, expert_offsets, num_tokens, gather_from, any_rows: bool, E: int, device):
    """Checks the row arguments; returns T.  gather_from: the rows of a
    gathered operand (the tokens), or None."""
    _arg(expert_offsets, "expert_offsets", _I32, (E + 1,), device)
    if sorted_ids is None:
        if any_rows:
            raise ValueError("gather and scatter need sorted_ids")
        return 0
    _arg(sorted_ids, "sorted_ids", _I32, None, device)
    if sorted_ids.dim() != 1:
        raise ValueError(f"sorted_ids must have one dimension, got {list(sorted_ids.shape)}")
    if gather_from is not None:
        if num_tokens is not None and num_tokens != gather_from:
            raise ValueError(f"num_tokens is {num_tokens}, the gathered operand has "
                             f"{gather_from} rows")
        return gather_from
    if num_tokens is None:
        raise ValueError("num_tokens is needed with sorted_ids when nothing is gathered")
    return int(num_tokens)


def _product(name, rows_in, w, expert_offsets, sorted_ids, topk, num_tokens, gather, scatter, out,
             workspace, dx: bool):
    E, N, K = _sizes(w, "w", 3)
    dev = w.device
    _arg(w, "w", _BF16, (E, N, K), dev)
    count, _ = _sizes(rows_in, "dy" if dx else "x", 2)
    _arg(rows_in, "dy" if dx else "x", _BF16, (count, N if dx else K), dev)
    T = _rows(sorted_ids, expert_offsets, num_tokens, count if gather else None,
              gather or scatter, E, dev)
    R = count if sorted_ids is None else sorted_ids.shape[0]
    if not gather and count != R:
        raise ValueError(f"the operand has {count} rows, sorted_ids {R}")
    rows = (MOE_ROWS_GATHER if gather else 0) | (MOE_ROWS_SCATTER if scatter else 0)
    sizes = (rows, T, topk, R, E, K, N)
    need = _product_workspace(name, *sizes)  # refuses sizes before anything is allocated for them
    out = _out(out, "out", _BF16, (T * topk if scatter else R, K if dx else N), dev)
    workspace = _workspace(dev, workspace, need, True)
    nbytes = ctypes.c_size_t(workspace.numel())
    _call(dev, name, _p(rows_in), _p(w), _p(expert_offsets), _p(sorted_ids), *sizes, _p(out),
          _p(workspace), ctypes.byref(nbytes))
    return out


def moe_grouped_gemm(x: torch.Tensor, w: torch.Tensor, expert_offsets: torch.Tensor, *,
                     sorted_ids: Optional[torch.Tensor] = None, topk: int = 1,
                     num_tokens: Optional[int] = None, gather: bool = False,
                     scatter: bool = False, out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[i] = w[e] x[i] for the sorted rows i of every expert e's range
    (expert_offsets, sorted_ids: moe_align's).

    x bf16 [R,K], or [num_tokens,K] with ``gather`` (row i reads the token of
    its slot); w bf16 [E,N,K]; returns bf16 [R,N], or with ``scatter``
    [num_tokens*topk,N] in slot order.  Rows of a new output that no sorted
    row writes are uninitialised."""
    return _product("moe_grouped_gemm", x, w, expert_offsets, sorted_ids, topk, num_tokens, gather,
                    scatter, out, workspace, False)


def moe_grouped_gemm_dx(dy: torch.Tensor, w: torch.Tensor, expert_offsets: torch.Tensor, *,
                        sorted_ids: Optional[torch.Tensor] = None, topk: int = 1,
                        num_tokens: Optional[int] = None, gather: bool = False,
                        scatter: bool = False, out: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dx[i] = w[e]^T dy[i]: the gradient of moe_grouped_gemm's input rows.
    dy bf16 [R,N] (or [num_tokens,N] with ``gather``); returns bf16 [R,K], or
    [num_tokens*topk,K] with ``scatter``."""
    return _product("moe_grouped_gemm_dx", dy, w, expert_offsets, sorted_ids, topk, num_tokens,
                    gather, scatter, out, workspace, True)


def moe_grouped_gemm_dw(dy: torch.Tensor, x: torch.Tensor, expert_offsets: torch.Tensor, *,
                        sorted_ids: Optional[torch.Tensor] = None, topk: int = 1,
                        num_tokens: Optional[int] = None, gather_dy: bool = False,
                        gather_x: bool = False, out_dtype: torch.dtype = torch.bfloat16,
                        out: Optional[torch.Tensor] = None, accumulate: bool = False,
                        workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dw[e] = sum over e's rows of dy[i] x[i]^T, the gradient of
    moe_grouped_gemm's weights: [E,N,K] in ``out_dtype`` (bf16 or fp32), or
    into ``out``; ``accumulate`` adds to an fp32 ``out``.  gather_dy /
    gather_x: that operand has num_tokens rows, read by the rows' tokens."""
    ny, N = _sizes(dy, "dy", 2)
    nx, K = _sizes(x, "x", 2)
    dev = dy.device
    _arg(dy, "dy", _BF16, (ny, N), dev)
    _arg(x, "x", _BF16, (nx, K), dev)
    if gather_dy and gather_x and ny != nx:
        raise ValueError("two gathered operands must have the same number of rows")
    E = _sizes(expert_offsets, "expert_offsets", 1)[0] - 1
    T = _rows(sorted_ids, expert_offsets, num_tokens, nx if gather_x else ny if gather_dy else None,
              gather_dy or gather_x, E, dev)
    R = ny if sorted_ids is None else sorted_ids.shape[0]
    for count, name, gathered in ((ny, "dy", gather_dy), (nx, "x", gather_x)):
        if not gathered and count != R:
            raise ValueError(f"{name} must have {R} rows, got {count}")
    if out is not None:
        out_dtype = out.dtype
    if out_dtype is not _BF16 and out_dtype is not _F32:
        raise ValueError(f"the gradient must be bfloat16 or float32, got {out_dtype}")
    if accumulate and (out is None or out_dtype is not _F32):
        raise ValueError("accumulate needs a float32 out")
    mode = MOE_OUT_FP32_ADD if accumulate else MOE_OUT_FP32 if out_dtype is _F32 else MOE_OUT_BF16
    rows = (MOE_ROWS_GATHER if gather_x else 0) | (MOE_ROWS_GATHER_DY if gather_dy else 0)
    sizes = (rows, T, topk, R, E, K, N, mode)
    need = _product_workspace("moe_grouped_gemm_dw", *sizes)
    out = _out(out, "out", out_dtype, (E, N, K), dev)
    workspace = _workspace(dev, workspace, need, True)
    nbytes = ctypes.c_size_t(workspace.numel())
    _call(dev, "moe_grouped_gemm_dw", _p(dy), _p(x), _p(expert_offsets), _p(sorted_ids), *sizes,
          _p(out), _p(workspace), ctypes.byref(nbytes))
    return out


def _gated(g, topk_weights, sorted_ids, num_rows):
    R, two_n = _sizes(g, "g", 2)
    dev = g.device
    _arg(g, "g", _BF16, (R, two_n), dev)
    if two_n % 2:
        raise ValueError("g must have an even number of columns (gate, up)")
    slots = 0
    if topk_weights is not None:
        _arg(topk_weights, "topk_weights", _F32, None, dev)
        slots = topk_weights.numel()
        if sorted_ids is None and slots != R:
            raise ValueError(f"without sorted_ids topk_weights must have {R} values, got {slots}")
    if sorted_ids is not None:
        _arg(sorted_ids, "sorted_ids", _I32, (R,), dev)
        if topk_weights is None:
            raise ValueError("sorted_ids is for topk_weights")
    if num_rows is not None:
        _arg(num_rows, "num_rows", _I32, (1,), dev)
    return dev, R, two_n // 2, slots


def moe_silu_mul(g: torch.Tensor, topk_weights: Optional[torch.Tensor] = None, *,
                 sorted_ids: Optional[torch.Tensor] = None,
                 num_rows: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """a[i] = wt * silu(g[i,:N]) * g[i,N:], bf16 [R,N], with the routing
    weight wt = topk_weights[sorted_ids[i]] (fp32, flat index; row i without
    sorted_ids, 1 without weights).  Padding rows are zero; rows at and past
    num_rows (moe_align's num_padded) are not written."""
    dev, R, N, slots = _gated(g, topk_weights, sorted_ids, num_rows)
    _fit("moe_silu_mul", R, N, slots)
    out = _out(out, "out", _BF16, (R, N), dev)
    _call(dev, "moe_silu_mul", _p(g), _p(topk_weights), _p(sorted_ids), _p(num_rows), slots, R, N,
          _p(out))
    return out


def moe_silu_mul_bwd(da: torch.Tensor, g: torch.Tensor,
                     topk_weights: Optional[torch.Tensor] = None, *,
                     sorted_ids: Optional[torch.Tensor] = None,
                     num_rows: Optional[torch.Tensor] = None):
    """Gradients of moe_silu_mul: (dg bf16 [R,2N], dtopk_weights in
    topk_weights' shape, or None without weights).  Weights of slots that no
    row names get an uninitialised gradient."""
    dev, R, N, slots = _gated(g, topk_weights, sorted_ids, num_rows)
    _fit("moe_silu_mul_bwd", R, N, slots)
    _arg(da, "da", _BF16, (R, N), dev)
    dg = torch.empty_like(g)
    dw = None if topk_weights is None else torch.empty_like(topk_weights)
    _call(dev, "moe_silu_mul_bwd", _p(da), _p(g), _p(topk_weights), _p(sorted_ids), _p(num_rows),
          slots, R, N, _p(dg), _p(dw))
    return dg, dw


def _stream_type(h, name: str) -> int:
    if not isinstance(h, torch.Tensor) or h.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"{name} must be a bfloat16 or float32 GPU tensor")
    return MOE_OUT_FP32 if h.dtype == torch.float32 else MOE_OUT_BF16


def moe_block_norm(h: torch.Tensor, o: Optional[torch.Tensor] = None,
                   gate: Optional[torch.Tensor] = None, w_post: Optional[torch.Tensor] = None,
                   w_pre: Optional[torch.Tensor] = None, *, topk: int = 1, res_scale: float = 1.0,
                   eps: float = 1e-6, out: Optional[torch.Tensor] = None):
    """The norm after a block, its gate and residual scale, and the norm
    before the next one:

      h_out = h + res_scale * gate[t] * rmsnorm(sum_j o[t*topk + j]) * w_post
      u     = rmsnorm(h_out) * w_pre

    h bf16 or fp32 [M,K]; o bf16 [M*topk,K]; gate fp32 [M]; w_post, w_pre
    fp32 [K].  Without o: only u, the norm of h.  Without w_post: the sum is
    added without a norm.  Without w_pre: no u.  Returns (h_out, u, rstd_post,
    rstd_pre), None where there is none; h_out is h without o.  ``out`` takes
    h_out and may be h."""
    kind = _stream_type(h, "h")
    dev = h.device
    M, K = _sizes(h, "h", 2)
    _fit("moe_block_norm", M, K, topk)
    _arg(h, "h", h.dtype, (M, K), dev)
    if w_pre is not None:
        _arg(w_pre, "w_pre", _F32, (K,), dev)
    if o is None:
        if gate is not None or w_post is not None or out is not None:
            raise ValueError("gate, w_post and out are for a block's output o")
        if w_pre is None:
            raise ValueError("one of o and w_pre is needed")
    else:
        _arg(o, "o", _BF16, (M * topk, K), dev)
        if gate is not None:
            _arg(gate, "gate", _F32, (M,), dev)
        if w_post is not None:
            _arg(w_post, "w_post", _F32, (K,), dev)
        out = _out(out, "out", h.dtype, (M, K), dev)
    u = None if w_pre is None else _new(_BF16, dev, M, K)
    r1 = None if w_post is None else _new(_F32, dev, M)
    r2 = None if w_pre is None else _new(_F32, dev, M)
    _call(dev, "moe_block_norm", _p(h), _p(o), _p(gate), _p(w_post), _p(w_pre), kind, M, K, topk,
          res_scale, eps, _p(out), _p(u), _p(r1), _p(r2))
    return (h if o is None else out), u, r1, r2


def moe_block_norm_bwd(dh_out: Optional[torch.Tensor], du: Optional[torch.Tensor],
                       h_out: torch.Tensor, o: Optional[torch.Tensor] = None,
                       gate: Optional[torch.Tensor] = None,
                       w_post: Optional[torch.Tensor] = None,
                       w_pre: Optional[torch.Tensor] = None,
                       rstd_post: Optional[torch.Tensor] = None,
                       rstd_pre: Optional[torch.Tensor] = None, *, topk: int = 1,
                       du_topk: int = 1, res_scale: float = 1.0,
                       workspace: Optional[torch.Tensor] = None):
    """Gradients of moe_block_norm from those of h_out ([M,K] in its type, or
    None) and of u (bf16 [M*du_topk,K], a token's rows are summed; None
    without w_pre).  h_out, rstd_post and rstd_pre are the forward's.  Returns
    (dh in h_out's type, do bf16 [M,K] -- the gradient of each of a token's
    slots -- dgate fp32 [M], dw_post, dw_pre fp32 [K]), None where there is
    none."""
    kind = _stream_type(h_out, "h_out")
    dev = h_out.device
    M, K = _sizes(h_out, "h_out", 2)
    _arg(h_out, "h_out", h_out.dtype, (M, K), dev)
    if dh_out is not None:
        _arg(dh_out, "dh_out", h_out.dtype, (M, K), dev)
    if (w_pre is None) != (du is None) or (w_pre is None) != (rstd_pre is None):
        raise ValueError("du, w_pre and rstd_pre go together")
    if (w_post is None) != (rstd_post is None):
        raise ValueError("w_post and rstd_post go together")
    if w_pre is not None:
        _arg(w_pre, "w_pre", _F32, (K,), dev)
        _arg(du, "du", _BF16, (M * du_topk, K), dev)
        _arg(rstd_pre, "rstd_pre", _F32, (M,), dev)
    elif dh_out is None or o is None:
        raise ValueError("nothing to differentiate: give du, or dh_out and o")
    if o is None:
        if gate is not None or w_post is not None:
            raise ValueError("gate and w_post are for a block's output o")
    else:
        _arg(o, "o", _BF16, (M * topk, K), dev)
        if gate is not None:
            _arg(gate, "gate", _F32, (M,), dev)
        if w_post is not None:
            _arg(w_post, "w_post", _F32, (K,), dev)
            _arg(rstd_post, "rstd_post", _F32, (M,), dev)
    need = _norm_workspace(kind, M, K, topk, du_topk)
    dh = _new(h_out.dtype, dev, M, K)
    do = None if o is None else _new(_BF16, dev, M, K)
    dgate = None if gate is None else _new(_F32, dev, M)
    dw_post = None if w_post is None else _new(_F32, dev, K)
    dw_pre = None if w_pre is None else _new(_F32, dev, K)
    workspace = _workspace(dev, workspace, need)
    nbytes = ctypes.c_size_t(workspace.numel())
    _call(dev, "moe_block_norm_bwd", _p(dh_out), _p(du), _p(h_out), _p(o), _p(gate), _p(w_post),
          _p(w_pre), _p(rstd_post), _p(rstd_pre), kind, M, K, topk, du_topk, res_scale, _p(dh),
          _p(do), _p(dgate), _p(dw_post), _p(dw_pre), _p(workspace), ctypes.byref(nbytes))
    return dh, do, dgate, dw_post, dw_pre
