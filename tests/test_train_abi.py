"""The entry points of the layer in pieces on a host without a GPU: every bad
argument is answered with its documented status before any HIP call, and the
workspace queries make none."""
import ctypes

import pytest
import torch

import moe_layer_04_amd as moe
from moe_layer_04_amd import _binding as B

INV, UNS, WSP, OK = (B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE, B.MOE_OK)
FAKE = ctypes.c_void_p(0x10000)         # aligned, never dereferenced on error paths
MISALIGNED = ctypes.c_void_p(0x10004)


@pytest.fixture(scope="module")
def lib():
    return moe.load_library(build_if_missing=True)


@pytest.mark.parametrize("name", ["moe_grouped_gemm", "moe_grouped_gemm_dx"])
def test_grouped_rows_refusals(lib, name):
    n = ctypes.c_size_t(0)

    def call(a=FAKE, w=FAKE, off=FAKE, ids=FAKE, rows=1, T=8, topk=2, R=16, E=4, K=64, N=96,
             out=FAKE, ws=FAKE, nbytes=1 << 40):
        n.value = nbytes
        return getattr(lib, name)(a, w, off, ids, rows, T, topk, R, E, K, N, out, ws,
                                  ctypes.byref(n), None)

    for kw in (dict(T=-1), dict(topk=0), dict(R=-1), dict(E=0), dict(K=0), dict(N=0),
               dict(rows=4), dict(rows=8), dict(ids=None), dict(ids=None, rows=2), dict(a=None),
               dict(w=None), dict(off=None), dict(out=None), dict(a=MISALIGNED),
               dict(w=MISALIGNED), dict(off=MISALIGNED), dict(ids=MISALIGNED),
               dict(out=MISALIGNED), dict(ws=ctypes.c_void_p(0x10010))):
        assert call(**kw) == INV, kw
    assert getattr(lib, name)(FAKE, FAKE, FAKE, FAKE, 1, 8, 2, 16, 4, 64, 96, FAKE, FAKE, None,
                              None) == INV
    for kw in (dict(E=257), dict(topk=17), dict(R=1 << 28), dict(T=1 << 27), dict(K=1 << 20),
               dict(N=1 << 20), dict(K=1 << 15, N=1 << 15),      # one expert's weights: 2 GiB
               dict(T=1 << 24, K=64, N=64),                       # the gathered rows: 2 GiB
               dict(R=(1 << 28) - 1, K=1 << 19, N=64, T=8, rows=0),    # the grid
               dict(R=1 << 22, K=1 << 14, N=1 << 14, T=8, rows=0)):    # its threads
        assert call(**kw) == UNS, kw
    assert call(R=0, a=None, w=None, off=None, ids=None, out=None, rows=0) == OK
    query = dict(a=None, w=None, off=None, ids=None, out=None, ws=None)
    for rows in (0, 1, 2, 3):
        assert call(**query, rows=rows) == OK
        assert n.value == 256                                     # unused, never NULL-sized
        assert call(rows=rows, nbytes=255) == WSP
    # few output tiles of a long reduction: fp32 products of its ranges
    red, cols = ("K", "N") if name == "moe_grouped_gemm" else ("N", "K")
    for length, width, parts in ((2048, 8, 4), (2048, 7, 4), (4096, 2000, 8)):
        assert call(**query, R=64, E=1, rows=0, **{red: length, cols: width}) == OK
        assert n.value == parts * 64 * ((width + 3) // 4 * 4) * 4
    assert call(**query, R=1, E=1, rows=0, **{red: 2048, cols: 1}) == OK
    assert n.value == 512                                         # used, so not the least size


def test_grouped_dw_refusals(lib):
    f = lib.moe_grouped_gemm_dw
    n = ctypes.c_size_t(0)

    def call(dy=FAKE, x=FAKE, off=FAKE, ids=FAKE, rows=1, T=8, topk=2, R=16, E=4, K=64, N=96,
             out=0, dw=FAKE, ws=FAKE, nbytes=1 << 40):
        n.value = nbytes
        return f(dy, x, off, ids, rows, T, topk, R, E, K, N, out, dw, ws, ctypes.byref(n), None)

    for kw in (dict(T=-1), dict(topk=0), dict(R=-1), dict(E=0), dict(K=0), dict(N=0),
               dict(rows=2), dict(rows=8), dict(out=3), dict(out=-1), dict(ids=None),
               dict(ids=None, rows=4), dict(dy=None), dict(x=None), dict(off=None),
               dict(dw=None), dict(dy=MISALIGNED), dict(x=MISALIGNED), dict(dw=MISALIGNED),
               dict(ws=ctypes.c_void_p(0x10010))):
        assert call(**kw) == INV, kw
    for kw in (dict(E=257), dict(topk=17), dict(R=1 << 28), dict(K=1 << 20),
               dict(K=1 << 15, N=1 << 15), dict(T=1 << 24), dict(T=1 << 24, rows=4)):
        assert call(**kw) == UNS, kw
    assert f(FAKE, FAKE, FAKE, FAKE, 1, 8, 2, 16, 4, 64, 96, 0, FAKE, FAKE, None, None) == INV
    for rows in (0, 1, 4, 5):
        assert call(None, None, None, None, rows, dw=None, ws=None) == OK
        need = n.value
        assert need >= 256                                        # never NULL-sized
        assert call(rows=rows, nbytes=need - 1) == WSP
    # few output tiles over many rows: fp32 products of the rows' ranges
    assert call(None, None, None, None, 0, R=4096, E=1, dw=None, ws=None) == OK
    assert n.value == 8 * 96 * 64 * 4
    assert call(None, None, None, None, 0, R=4096, E=1, N=28672, K=4096, dw=None, ws=None) == OK
    assert n.value == 256
    assert call(None, None, None, None, 0, R=4096, E=1, N=97, dw=None, ws=None) == OK
    assert n.value == 256
    assert call(R=0, out=2, dy=None, x=None, ids=None, rows=0) == OK     # nothing to add


def test_silu_mul_refusals(lib):
    def fwd(g=FAKE, wt=FAKE, ids=FAKE, nr=None, slots=16, R=16, N=64, a=FAKE):
        return lib.moe_silu_mul(g, wt, ids, nr, slots, R, N, a, None)

    def bwd(da=FAKE, g=FAKE, wt=FAKE, ids=FAKE, nr=None, slots=16, R=16, N=64, dg=FAKE, dw=FAKE):
        return lib.moe_silu_mul_bwd(da, g, wt, ids, nr, slots, R, N, dg, dw, None)

    for call in (fwd, bwd):
        for kw in (dict(slots=-1), dict(R=-1), dict(N=0), dict(g=None), dict(g=MISALIGNED),
                   dict(wt=MISALIGNED), dict(ids=MISALIGNED), dict(nr=MISALIGNED),
                   dict(ids=None, slots=15)):
            assert call(**kw) == INV, kw
        for kw in (dict(R=1 << 28), dict(slots=1 << 28), dict(N=1 << 20),
                   dict(R=1 << 24, slots=1 << 24), dict(R=1 << 20, slots=1 << 20, N=1 << 15)):
            assert call(**kw) == UNS, kw
        assert call(R=0, g=None) == OK
    assert fwd(a=None) == INV and fwd(a=MISALIGNED) == INV
    for kw in (dict(da=None), dict(dg=None), dict(wt=None), dict(da=MISALIGNED),
               dict(dg=MISALIGNED), dict(dw=MISALIGNED)):
        assert bwd(**kw) == INV, kw


def test_block_norm_refusals(lib):
    def call(h=FAKE, o=FAKE, gate=FAKE, wp=FAKE, wn=FAKE, dt=0, M=4, K=64, topk=2, eps=1e-6,
             ho=FAKE, u=FAKE, r1=FAKE, r2=FAKE):
        return lib.moe_block_norm(h, o, gate, wp, wn, dt, M, K, topk, 1.0, eps, ho, u, r1, r2,
                                  None)

    for kw in (dict(dt=2), dict(dt=-1), dict(M=-1), dict(K=0), dict(topk=0), dict(eps=0.0),
               dict(eps=-1.0), dict(eps=float("nan")), dict(h=None), dict(ho=None), dict(u=None),
               dict(wn=None), dict(wn=None, u=None, r2=FAKE),
               dict(wp=None),                                      # its rstd is asked for
               dict(o=None), dict(o=None, gate=None, wp=None, r1=None),          # h_out given
               dict(o=None, gate=None, wp=None, wn=None, ho=None, u=None, r1=None, r2=None),
               dict(h=MISALIGNED), dict(o=MISALIGNED), dict(gate=MISALIGNED),
               dict(wp=MISALIGNED), dict(ho=MISALIGNED), dict(u=MISALIGNED), dict(r1=MISALIGNED)):
        assert call(**kw) == INV, kw
    for kw in (dict(K=1 << 20), dict(topk=17), dict(M=1 << 27), dict(M=1 << 22)):
        assert call(**kw) == UNS, kw
    assert call(M=0, h=None) == OK


def test_block_norm_bwd_refusals(lib):
    n = ctypes.c_size_t(0)
    names = ("dho", "du", "ho", "o", "gate", "wp", "wn", "r1", "r2")
    outs = ("dh", "do", "dgate", "dwp", "dwn")
    at = {k: 0x10000 + 0x1000 * i for i, k in enumerate(names + outs)}

    def call(dt=0, M=4, K=64, topk=2, dtopk=2, ws=FAKE, nbytes=1 << 40, **ptr):
        n.value = nbytes
        p = [ctypes.c_void_p(v) if (v := ptr.get(k, at[k])) else None for k in names]
        q = [ctypes.c_void_p(v) if (v := ptr.get(k, at[k])) else None for k in outs]
        return lib.moe_block_norm_bwd(*p, dt, M, K, topk, dtopk, 1.0, *q, ws, ctypes.byref(n),
                                      None)

    for kw in (dict(dt=2), dict(M=-1), dict(K=0), dict(topk=0), dict(dtopk=0), dict(dh=None),
               dict(du=None), dict(ho=None), dict(o=None), dict(wp=None), dict(wn=None),
               dict(gate=None), dict(dgate=None), dict(dwp=None), dict(dwn=None), dict(r1=None),
               dict(r2=None), dict(do=None), dict(dho=None, du=None, wn=None, dwn=None, r2=None),
               dict(o=None, do=None, gate=None, dgate=None, wp=None, dwp=None, wn=None, dwn=None,
                    du=None, r1=None, r2=None),
               dict(dh=at["dho"]), dict(dh=at["ho"]), dict(do=at["o"]), dict(do=at["du"]),
               dict(ws=ctypes.c_void_p(0x10010)), dict(dho=0x10004), dict(dwn=0x10004)):
        assert call(**kw) == INV, kw
    for kw in (dict(K=1 << 20), dict(topk=17), dict(dtopk=17), dict(M=1 << 27), dict(M=1 << 22)):
        assert call(**kw) == UNS, kw
    assert lib.moe_block_norm_bwd(*[FAKE] * 9, 0, 4, 64, 2, 2, 1.0, *[FAKE] * 5, FAKE, None,
                                  None) == INV
    assert call(ws=None, **{k: None for k in names + outs}) == OK and n.value >= 256
    assert call(nbytes=n.value - 1) == WSP


def test_python_refuses_host_tensors():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    w = torch.zeros(2, 8, 8, dtype=torch.bfloat16)
    off = torch.tensor([0, 2, 4], dtype=torch.int32)
    for call in (lambda: moe.moe_grouped_gemm(x, w, off),
                 lambda: moe.moe_grouped_gemm_dx(x, w, off),
                 lambda: moe.moe_grouped_gemm_dw(x, x, off),
                 lambda: moe.moe_silu_mul(x), lambda: moe.moe_silu_mul_bwd(x, x),
                 lambda: moe.moe_block_norm(x, w_pre=torch.ones(8)),
                 lambda: moe.moe_block_norm_bwd(None, x, x, w_pre=torch.ones(8),
                                                rstd_pre=torch.ones(4))):
        with pytest.raises(ValueError):
            call()


def test_sizes_past_32_bits_are_refused(lib):
    """They are not cut to the 32 bits of the library's arguments: 2^32 + 8
    rows are not 8."""
    from moe_layer_04_amd import _operators as O
    far = (1 << 32) + 8
    for call in (lambda: O._product_workspace("moe_grouped_gemm", 0, 0, 1, far, 2, 64, 64),
                 lambda: O._product_workspace("moe_grouped_gemm_dx", 0, far, 1, 16, 2, 64, 64),
                 lambda: O._product_workspace("moe_grouped_gemm_dw", 0, 0, 1, 16, 2, far, 64, 0),
                 lambda: O._product_workspace("moe_grouped_gemm", 0, 8, 1 - far, 16, 2, 64, 64),
                 lambda: O._norm_workspace(0, far, 64, 1, 1),
                 lambda: O._norm_workspace(0, 4, 64, far, 1)):
        with pytest.raises(moe.MoEError) as err:
            call()
        assert err.value.status == UNS


def test_products_over_their_operands_are_refused(lib):
    """An output that shares bytes with an operand: the same buffer, its end or
    its middle."""
    n = ctypes.c_size_t(1 << 40)
    R, E, K, N = 16, 4, 64, 64
    at = {"a": 0x100000, "w": 0x200000, "out": 0x300000, "off": 0x400000}
    size = {"a": R * K * 2, "w": E * N * K * 2}

    def call(name, **kw):
        p = {k: ctypes.c_void_p(kw.get(k, v)) for k, v in at.items()}
        return getattr(lib, name)(p["a"], p["w"], p["off"], None, 0, 0, 1, R, E, K, N, p["out"], FAKE,
                                  ctypes.byref(n), None)

    for name in ("moe_grouped_gemm", "moe_grouped_gemm_dx"):
        for k in ("a", "w"):
            for d in (0, 16, size[k] - 16, 16 - R * N * 2):
                assert call(name, out=at[k] + d) == INV, (name, k, d)
    bytes_dw = E * N * K * 4
    for k in ("dy", "x"):
        for d in (0, 16, R * K * 2 - 16, 16 - bytes_dw):
            p = {"dy": 0x100000, "x": 0x200000, "dw": 0x300000}
            p["dw"] = p[k] + d
            q = {i: ctypes.c_void_p(v) for i, v in p.items()}
            assert lib.moe_grouped_gemm_dw(q["dy"], q["x"], ctypes.c_void_p(0x400000), None, 0, 0, 1, R, E,
                                           K, N, 1, q["dw"], FAKE, ctypes.byref(n), None) == INV
