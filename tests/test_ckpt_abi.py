"""The entry points of activations kept in 8 bits on a host without a GPU: every
bad argument is answered with its documented status before any HIP call, and
the workspace queries make none."""
import ctypes

import pytest
import torch

import moe_layer_04_amd as moe
from moe_layer_04_amd import _binding as B

INV, UNS, WSP, OK = (B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE, B.MOE_OK)
BAD = 0x10004                                    # misaligned


@pytest.fixture(scope="module")
def lib():
    return moe.load_library(build_if_missing=True)


def ptrs(at, kw):
    """The pointers by name, far from one another; never dereferenced on error
    paths."""
    return [ctypes.c_void_p(kw[k]) if k in kw and kw[k] else
            (None if k in kw else ctypes.c_void_p(0x100000000 * (i + 1))) for i, k in enumerate(at)]


@pytest.mark.parametrize("name", ["moe_ckpt_rows", "moe_ckpt_restore"])
def test_rows_refusals(lib, name):
    ins, outs = (("x",), ("codes", "scales")) if name == "moe_ckpt_rows" else (("codes", "scales"), ("x",))

    def call(R=16, W=100, **kw):
        p = ptrs(ins + outs, kw)
        return getattr(lib, name)(*p[:len(ins)], R, W, *p[len(ins):], None)

    for kw in (dict(R=-1), dict(W=0), dict(W=-1), *({k: v} for k in ins + outs for v in (None, BAD))):
        assert call(**kw) == INV, kw
    for kw in (dict(R=1 << 28), dict(W=1 << 20), dict(R=1 << 27, W=4096), dict(R=(1 << 28) - 1, W=129)):
        assert call(**kw) == UNS, kw
    assert call(R=0, **{k: None for k in ins + outs}) == OK
    # an output that shares bytes with an input or with the other output
    n, nb = 16 * 100, 16 * 4
    size = {"x": 2 * n, "codes": n, "scales": nb}
    for a in outs:
        for b in ins + outs:
            if a != b:
                for d in (0, size[b] // 16 * 16 - 16, 16 - size[a] // 16 * 16):
                    assert call(**{b: 0x900000, a: 0x900000 + d}) == INV, (a, b, d)


def test_activation_refusals(lib):
    def fwd(slots=16, R=16, N=64, **kw):
        p = ptrs(("g", "wt", "ids", "num", "a", "codes", "scales"), kw)
        return lib.moe_silu_mul_ckpt(*p[:4], slots, R, N, *p[4:], None)

    def bwd(slots=16, R=16, N=64, **kw):
        p = ptrs(("da", "codes", "scales", "wt", "ids", "num", "dg", "dw", "a"), kw)
        return lib.moe_silu_mul_bwd_ckpt(*p[:6], slots, R, N, *p[6:], None)

    for call in (fwd, bwd):
        for kw in (dict(slots=-1), dict(R=-1), dict(N=0), dict(codes=None), dict(scales=None),
                   dict(codes=BAD), dict(scales=BAD), dict(wt=BAD), dict(ids=BAD), dict(num=BAD),
                   dict(a=BAD), dict(ids=None, slots=15)):
            assert call(**kw) == INV, kw
        for kw in (dict(R=1 << 28), dict(slots=1 << 28), dict(N=1 << 20),
                   dict(R=1 << 24, slots=1 << 24), dict(R=1 << 20, slots=1 << 20, N=1 << 15)):
            assert call(**kw) == UNS, kw
        assert call(R=0, codes=None) == OK
    for kw in (dict(g=None), dict(g=BAD), dict(a=None), dict(a=0x900000, codes=0x9007f0),
               dict(a=0x900000, g=0x900400), dict(scales=0x900000, g=0x900000),
               dict(codes=0x900000, scales=0x9007f0), dict(scales=0x900000, num=0x900010)):
        assert fwd(**kw) == INV, kw
    for kw in (dict(da=None), dict(da=BAD), dict(dg=None), dict(dg=BAD), dict(dw=BAD), dict(wt=None),
               dict(dg=0x900000, codes=0x900800), dict(dg=0x900000, da=0x900000),
               dict(dg=0x900000, a=0x900ff0), dict(a=0x900000, da=0x9007f0),
               dict(dw=0x900000, wt=0x900000), dict(dg=0x900000, scales=0x900010)):
        assert bwd(**kw) == INV, kw


def test_dw_refusals(lib):
    n = ctypes.c_size_t(0)

    def call(rows=1, T=8, topk=2, R=16, E=4, K=64, N=96, out=0, nbytes=1 << 40, **kw):
        n.value = nbytes
        p = ptrs(("dy", "codes", "scales", "off", "ids", "dw", "ws"), kw)
        return lib.moe_grouped_gemm_dw_ckpt(*p[:5], rows, T, topk, R, E, K, N, out, *p[5:],
                                            ctypes.byref(n), None)

    for kw in (dict(T=-1), dict(topk=0), dict(R=-1), dict(E=0), dict(K=0), dict(N=0), dict(rows=2),
               dict(rows=8), dict(out=3), dict(out=-1), dict(ids=None), dict(ids=None, rows=4),
               dict(dy=None), dict(codes=None), dict(scales=None), dict(off=None), dict(dw=None),
               dict(dy=BAD), dict(codes=BAD), dict(scales=BAD), dict(off=BAD), dict(ids=BAD),
               dict(dw=BAD), dict(ws=0x10010)):
        assert call(**kw) == INV, kw
    for kw in (dict(E=257), dict(topk=17), dict(R=1 << 28), dict(K=1 << 20), dict(K=1 << 15, N=1 << 15),
               dict(T=1 << 24), dict(T=1 << 24, rows=4), dict(R=1 << 27, K=4096, rows=0)):
        assert call(**kw) == UNS, kw
    size = {"dy": 16 * 96 * 2, "codes": 8 * 64, "scales": 8 * 2}
    for k, v in size.items():
        for d in (0, v - 16, 16 - 4 * 96 * 64 * 2):
            assert call(**{k: 0x900000, "dw": 0x900000 + d}) == INV, (k, d)
    query = {k: None for k in ("dy", "codes", "scales", "off", "ids", "dw", "ws")}
    for rows in (0, 1, 4, 5):
        assert call(**query, rows=rows) == OK
        need = n.value
        assert need >= 256 and need % 256 == 0
        assert call(rows=rows, nbytes=need - 1) == WSP
    assert call(R=0, out=2, rows=0, dy=None, codes=None, scales=None, ids=None) == OK   # nothing to add


def test_python_refuses_host_tensors():
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    codes, X = torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4, 1, dtype=torch.uint8)
    off = torch.tensor([0, 2, 4], dtype=torch.int32)
    for call in (lambda: moe.moe_ckpt_rows(x), lambda: moe.moe_ckpt_restore(codes, X),
                 lambda: moe.moe_silu_mul_ckpt(x), lambda: moe.moe_silu_mul_bwd_ckpt(x, codes, X),
                 lambda: moe.moe_grouped_gemm_dw_ckpt(x, codes, X, off)):
        with pytest.raises(ValueError):
            call()
