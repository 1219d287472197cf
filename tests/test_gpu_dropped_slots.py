"""Slots that no sorted row names -- dropped by the caller's own sort, by a limit
on an expert's rows, or behind num_rows: their routing weights changed nothing,
so the gradient of these weights is zero, whatever the memory held before, and
goes on to the router as zero.

Bounds of the router's gradients: test_gpu_router_grad.py.
"""
import pytest
import torch

from tests._train_ref import U32, bf16, check, f32, silu_mul
from tests.test_gpu_router_grad import reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import moe_layer_04_amd as m
    m.load_library()
    return m


def note(msg):
    print(f"[gpu-test] {msg}", flush=True)


def stale(shape):
    """Leaves NaN in the memory that the next tensors of this size get."""
    held = [torch.full(shape, float("nan"), device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    del held


def backward(moe, kept, da, g, wt, **kw):
    """dg and dtopk_weights of the activation, plain or with its input kept in 8 bits."""
    if kept:
        codes, X = moe.moe_silu_mul_ckpt(g, wt, **kw)[1:]
        stale(wt.shape)
        return moe.moe_silu_mul_bwd_ckpt(da, codes, X, wt, **kw)[:2]
    stale(wt.shape)
    return moe.moe_silu_mul_bwd(da, g, wt, **kw)


@pytest.mark.parametrize("kept", [False, True], ids=["bf16", "kept"])
@pytest.mark.parametrize("T,topk,N", [(1, 1, 8), (40, 2, 24), (333, 3, 101)])
@pytest.mark.parametrize("how", ["sentinel", "fewer rows", "num_rows", "num_rows, slots in order", "no rows"])
def test_weights_without_a_row(moe, kept, T, topk, N, how):
    note(f"weights without a row T={T} topk={topk} N={N} {how} kept={kept}")
    slots = T * topk
    order = torch.randperm(slots, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    live = slots - (slots + 2) // 3
    num = None
    if how == "sentinel":                         # padding rows in their place
        order[live:] = slots
    elif how == "fewer rows":
        order = order[:live].contiguous()
    elif how == "no rows":
        order, live = order[:0].contiguous(), 0
    else:
        num = torch.tensor([live], dtype=torch.int32, device="cuda")
        if how != "num_rows":
            order = None
    R = slots if order is None else order.numel()
    g, da, wt = bf16((R, 2 * N), 2, 2.0), bf16((R, N), 3), f32((T, topk), 4, 0.2, 0.5)
    if order is None:
        wt = wt.view(-1)
    dw = backward(moe, kept, da, g, wt, sorted_ids=order, num_rows=num)[1]
    assert dw.shape == wt.shape
    at = (torch.arange(slots, device="cuda") if order is None else order[:live].long())[:live]
    dropped = torch.ones(slots, dtype=torch.bool, device="cuda")
    dropped[at] = False
    assert (dw.view(-1)[dropped] == 0).all()
    if not kept:                                  # and the others are what they are
        act = silu_mul(g[:live].double(), torch.ones(live, dtype=torch.float64, device="cuda"))[1]
        terms = da[:live].double() * act
        check(dw.view(-1)[at], terms.sum(1), (N + 64) * U32 * terms.abs().sum(1), "dtopk_weights")


@pytest.mark.parametrize("kept", [False, True], ids=["bf16", "kept"])
@pytest.mark.parametrize("T,topk,E,K,N", [(33, 2, 5, 40, 24), (300, 4, 70, 72, 48)])
def test_dropped_slots_and_the_router(moe, kept, T, topk, E, K, N):
    """From the activation's gradients on to the router's, with slots that an
    expert had no room for: their ids are -1, their rows of the tokens'
    gradients zeros."""
    note(f"dropped slots T={T} topk={topk} E={E} kept={kept}")
    x, w = bf16((T, K), 1), bf16((E, K), 2, K ** -0.5)
    ids, wts, _ = moe.moe_topk(x, w, torch.zeros(E, device="cuda"), topk)
    flat = ids.view(-1).long()
    room = max(1, T * topk // (2 * E))
    order = torch.sort(flat, stable=True)[1]
    start = torch.bincount(flat, minlength=E).cumsum(0) - torch.bincount(flat, minlength=E)
    place = torch.arange(flat.numel(), device="cuda") - start[flat[order]]
    sorted_ids = order[place < room].to(torch.int32).contiguous()
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.bincount(flat, minlength=E).clamp(max=room).cumsum(0)
    gone = torch.ones_like(flat, dtype=torch.bool)
    gone[sorted_ids.long()] = False
    assert gone.any()
    ids = torch.where(gone.view(T, topk), torch.full_like(ids, -1), ids)
    R = sorted_ids.numel()
    g, da, w1 = bf16((R, 2 * N), 3, 2.0), bf16((R, N), 4), bf16((E, 2 * N, K), 5, K ** -0.5)
    dg, dwts = backward(moe, kept, da, g, wts, sorted_ids=sorted_ids)
    rows = moe.moe_grouped_gemm_dx(dg, w1, off, sorted_ids=sorted_ids, topk=topk, num_tokens=T, scatter=True,
                                   out=torch.zeros((T * topk, K), dtype=torch.bfloat16, device="cuda"))
    s = dict(x=x, w_router=w, topk_ids=ids, topk_weights=wts, dtopk_weights=dwts, dlogits=None, dx_rows=rows)
    got = moe.moe_topk_bwd(**s, bias=True)
    want, bound = reference(dict(s, dtopk_weights=torch.where(gone.view(T, topk), torch.zeros_like(dwts), dwts)))
    for a, b, c, name in zip(got, want, bound, ("dx", "dw", "dbias")):
        check(a, b, c, name)


def test_dropped_slots_in_a_graph(moe):
    """The zeros are written by every replay, not by the capture alone."""
    note("dropped slots, graph")
    slots, N, live = 50, 40, 31
    order = torch.randperm(slots, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    order[live:] = slots
    g, da, wt = bf16((slots, 2 * N), 2), bf16((slots, N), 3), f32((slots,), 4)
    dropped = torch.ones(slots, dtype=torch.bool, device="cuda")
    dropped[order[:live].long()] = False
    moe.moe_silu_mul_bwd(da, g, wt, sorted_ids=order)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dw = moe.moe_silu_mul_bwd(da, g, wt, sorted_ids=order)[1]
    for rep in range(4):
        dw.fill_(float("nan"))
        da.copy_(bf16((slots, N), 10 + rep))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert (dw[dropped] == 0).all()
        assert torch.equal(dw, moe.moe_silu_mul_bwd(da, g, wt, sorted_ids=order)[1])
