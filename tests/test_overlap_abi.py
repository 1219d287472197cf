"""Products whose output shares bytes with the lists that say which rows they take:
refused before any HIP call.  Workgroups read the lists while others write."""
import ctypes

import pytest

import moe_layer_04_amd as moe
from moe_layer_04_amd import _binding as B
from tests.test_ckpt_abi import ptrs

INV = B.MOE_ERR_INVALID_ARG
T, TOPK, R, E, K, N = 8, 2, 16, 4, 64, 80
AT = 0x900000


@pytest.fixture(scope="module")
def lib():
    return moe.load_library(build_if_missing=True)


def call(lib, name, rows, out=0, **kw):
    n = ctypes.c_size_t(1 << 40)
    ins = {"moe_grouped_gemm": ("x", "w"), "moe_grouped_gemm_dx": ("dy", "w"), "moe_grouped_gemm_dw": ("dy", "x"),
           "moe_grouped_gemm_dw_ckpt": ("dy", "codes", "scales")}[name]
    p = ptrs(ins + ("off", "ids", "y", "ws"), kw)
    mode = (out,) if "_dw" in name else ()
    return getattr(lib, name)(*p[:-2], rows, T, TOPK, R, E, K, N, *mode, *p[-2:], ctypes.byref(n), None)


@pytest.mark.parametrize("name,rows,size", [
    ("moe_grouped_gemm", 1, R * N * 2), ("moe_grouped_gemm", 3, T * TOPK * N * 2), ("moe_grouped_gemm", 0, R * N * 2),
    ("moe_grouped_gemm_dx", 1, R * K * 2), ("moe_grouped_gemm_dx", 2, T * TOPK * K * 2),
    ("moe_grouped_gemm_dw", 1, E * N * K * 2), ("moe_grouped_gemm_dw", 5, E * N * K * 2),
    ("moe_grouped_gemm_dw_ckpt", 0, E * N * K * 2), ("moe_grouped_gemm_dw_ckpt", 1, E * N * K * 2)])
def test_lists_of_rows(lib, name, rows, size):
    for k, held in (("off", 4 * (E + 1)), ("ids", 4 * R)):
        for d in (0, (held - 1) // 16 * 16, 16 - size):      # its start, its end, before it
            assert call(lib, name, rows, **{k: AT, "y": AT + d}) == INV, (k, d)


@pytest.mark.parametrize("name", ["moe_grouped_gemm_dw", "moe_grouped_gemm_dw_ckpt"])
@pytest.mark.parametrize("out,width", [(0, 2), (1, 4), (2, 4)])
def test_the_outputs_type_counts(lib, name, out, width):
    last = E * N * K * width - 16
    for k in ("off", "ids"):
        assert call(lib, name, 1, out=out, **{k: AT + last, "y": AT}) == INV
