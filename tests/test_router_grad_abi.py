"""The entry points of the router's balance loss and gradients on a host without
a GPU: every bad argument is answered with its documented status before any HIP
call, and the workspace queries make none."""
import ctypes

import pytest
import torch

import moe_layer_04_amd as moe
from moe_layer_04_amd import _binding as B
from tests.test_ckpt_abi import BAD, ptrs

INV, UNS, WSP, OK = (B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE, B.MOE_OK)


@pytest.fixture(scope="module")
def lib():
    return moe.load_library(build_if_missing=True)


SIZES = (dict(M=-1), dict(E=0), dict(topk=0), dict(topk=9))
BIG = (dict(E=257), dict(E=64, topk=17), dict(M=1 << 27))


def overlapping(call, outs, ins, size):
    """An output that starts with, ends in or lies before another buffer's first
    bytes."""
    for a in outs:
        for b in outs + ins:
            if a != b:
                for d in (0, (size[b] + 15) // 16 * 16 - 16, 16 - (size[a] + 15) // 16 * 16):
                    assert call(**{b: 0x900000, a: 0x900000 + d}) == INV, (a, b, d)


def test_balance_refusals(lib):
    n = ctypes.c_size_t(0)
    names = ("logits", "ids", "mask", "loss", "counts", "tokens", "probs", "ws")

    def call(M=16, E=8, topk=2, nbytes=1 << 40, **kw):
        n.value = nbytes
        p = ptrs(names, kw)
        return lib.moe_balance(*p[:3], M, E, topk, *p[3:], ctypes.byref(n), None)

    for kw in (*SIZES, *({k: None} for k in names if k not in ("mask", "ws")),
               *({k: BAD} for k in names), dict(ws=0x10010)):
        assert call(**kw) == INV, kw
    assert lib.moe_balance(*ptrs(names[:3], {}), 16, 8, 2, *ptrs(names[3:], {}), None, None) == INV
    for kw in BIG:
        assert call(**kw) == UNS, kw
    query = {k: None for k in names}
    assert call(**query) == OK and n.value == 256             # one workgroup: not used
    assert call(nbytes=255) == WSP
    assert call(**query, M=1 << 20, E=1, topk=1) == OK and n.value >= 512 and n.value % 256 == 0
    assert call(M=1 << 20, E=1, topk=1, nbytes=n.value - 1) == WSP
    assert call(**query, M=40, E=256) == OK and n.value >= 2 * 2 * 256 * 4
    outs, ins = ("loss", "counts", "tokens", "probs"), ("logits", "ids", "mask")
    overlapping(call, outs, ins, dict(loss=4, counts=32, tokens=4, probs=32, logits=512, ids=128, mask=16))


def test_balance_bwd_refusals(lib):
    names = ("dloss", "logits", "counts", "tokens", "mask", "dlogits")

    def call(M=16, E=8, topk=2, **kw):
        p = ptrs(names, kw)
        return lib.moe_balance_bwd(*p[:5], M, E, topk, p[5], None)

    for kw in (*SIZES, *({k: None} for k in names if k != "mask"), *({k: BAD} for k in names)):
        assert call(**kw) == INV, kw
    for kw in BIG:
        assert call(**kw) == UNS, kw
    assert call(M=0, **{k: None for k in names}) == OK
    overlapping(call, ("dlogits",), names[:5],
                dict(dloss=4, logits=512, counts=32, tokens=4, mask=16, dlogits=512))


def test_topk_bwd_refusals(lib):
    n = ctypes.c_size_t(0)
    names = ("x", "w", "ids", "wts", "dwts", "dl", "more", "dx", "dw", "db", "ws")

    def call(rows=2, M=16, K=64, E=8, topk=2, nbytes=1 << 40, **kw):
        n.value = nbytes
        p = ptrs(names, kw)
        return lib.moe_topk_bwd(*p[:7], rows, M, K, E, topk, *p[7:], ctypes.byref(n), None)

    for kw in (*SIZES, dict(K=0), dict(rows=-1), dict(rows=0), dict(more=None), dict(x=None), dict(w=None),
               dict(dx=None), dict(dw=None), dict(ids=None), dict(wts=None), dict(dwts=None),
               dict(ids=None, wts=None, dwts=None, dl=None), *({k: BAD} for k in names), dict(ws=0x10010)):
        assert call(**kw) == INV, kw
    assert lib.moe_topk_bwd(*ptrs(names[:7], {}), 2, 16, 64, 8, 2, *ptrs(names[7:], {}), None, None) == INV
    for kw in (*BIG, dict(K=1 << 20), dict(rows=17), dict(M=1 << 25, rows=16, topk=1), dict(M=1 << 24, K=1 << 14)):
        assert call(**kw) == UNS, kw
    query = {k: None for k in names}
    assert call(**query) == OK and n.value == 256              # few tokens and experts: not used
    assert call(nbytes=255) == WSP
    for kw in (dict(M=129), dict(E=65)):
        assert call(**query, **kw) == OK
        need = n.value
        assert need >= 3 * 16 * 64 * 2 and need % 256 == 0
        assert call(nbytes=need - 1, **kw) == WSP
    # the tokens in ranges: their sums
    assert call(**query, M=4096) == OK and n.value > 3 * 4096 * 64 * 2
    size = dict(x=2048, w=1024, ids=128, wts=128, dwts=128, dl=512, more=4096, dx=2048, dw=2048, db=32)
    overlapping(call, ("dx", "dw", "db"), names[:7], size)


@pytest.mark.parametrize("E,tokens", ((1, 16), (64, 16), (65, 8), (128, 8), (129, 4), (256, 4)))
def test_topk_bwd_tokens_of_a_launch(lib, E, tokens):
    """The launch for dl takes `tokens` tokens a workgroup of 256 threads and must have
    fewer than 2^32 threads."""
    n = ctypes.c_size_t(0)

    def query(M):
        return lib.moe_topk_bwd(*[None] * 7, 1, M, 8, E, 1, *[None] * 4, ctypes.byref(n), None)

    assert query(tokens * ((1 << 24) - 1)) == OK
    assert query(tokens * ((1 << 24) - 1) + 1) == UNS


def test_python_refuses_host_tensors(lib):
    l, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    for call in (lambda: moe.moe_balance(l, ids),
                 lambda: moe.moe_balance_bwd(l[0, :1], l, ids[0], ids[0, :1], 2),
                 lambda: moe.moe_topk_bwd(x, x, ids, l, l)):
        with pytest.raises(ValueError):
            call()


def test_sizes_past_32_bits_are_refused(lib):
    from moe_layer_04_amd import _router_grad as G
    far = (1 << 32) + 8
    for call in (lambda: G._balance_workspace(far, 8, 2), lambda: G._topk_bwd_workspace(2, far, 64, 8, 2),
                 lambda: G._topk_bwd_workspace(2, 16, far, 8, 2)):
        with pytest.raises(moe.MoEError) as err:
            call()
        assert err.value.status == UNS
