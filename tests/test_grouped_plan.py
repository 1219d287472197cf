"""The launch plans of the grouped products, on a host without a GPU: bad
arguments, and that the shapes which stand for the paths in the GPU tests take
them."""
import ctypes

import pytest

import moe_layer_04_amd as moe
from moe_layer_04_amd import _binding as B
from moe_layer_04_amd import _operators as O
from tests._paths import DW, OP_PATHS, ROWS, T128, T256, T64, dw_R, rows_R

INV, UNS, OK = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_OK
OPS = {"fwd": moe.MOE_PRODUCT_FWD, "dx": moe.MOE_PRODUCT_DX, "dw": moe.MOE_PRODUCT_DW}


@pytest.fixture(scope="module")
def lib():
    return moe.load_library(build_if_missing=True)


def test_refusals(lib):
    plan = moe.ProductPlan()

    def call(op=0, R=16, E=4, K=64, N=96, out=ctypes.byref(plan)):
        return lib.moe_grouped_plan(op, R, E, K, N, out)

    assert call() == OK
    for kw in (dict(op=-1), dict(op=3), dict(R=-1), dict(E=0), dict(K=0), dict(N=0),
               dict(out=None)):
        assert call(**kw) == INV, kw
    for kw in (dict(R=1 << 28), dict(E=257), dict(K=1 << 20), dict(N=1 << 20),
               dict(K=1 << 15, N=1 << 15), dict(R=1 << 22, K=1 << 14, N=1 << 14)):
        assert call(**kw) == UNS, kw
    with pytest.raises(moe.MoEError):
        moe.grouped_plan(0, 1 << 32, 4, 64, 64)


@pytest.mark.parametrize("op", list(OPS))
def test_agrees_with_the_products_own_sizes(lib, op):
    """The workspace of the plan is the one the product reports."""
    name = "moe_grouped_gemm" + ("" if op == "fwd" else "_" + op)
    for R, E, K, N in ((0, 3, 64, 64), (1, 1, 2048, 1), (16, 8, 8200, 40), (64, 1, 2048, 7),
                       (1030, 1, 7304, 1096), (12000, 3, 136, 72), (8192, 8, 4096, 28672)):
        plan = moe.grouped_plan(OPS[op], R, E, K, N)
        sizes = (0, 0, 1, R, E, K, N) + ((0,) if op == "dw" else ())
        assert plan.workspace_bytes == O._product_workspace(name, *sizes)
        assert (plan.splits > 1) == (plan.workspace_bytes > 256)
        assert (plan.workgroups == 0) == (R == 0 and op != "dw")


@pytest.mark.parametrize("op,name", OP_PATHS)
def test_rows_paths(lib, op, name):
    _, _, E, _, red, width, kernel, splits = ROWS[name]
    K, N = (red, width) if op == "fwd" else (width, red)
    plan = moe.grouped_plan(OPS[op], rows_R(name), E, K, N)
    assert (plan.kernel, plan.splits) == (kernel, splits)


@pytest.mark.parametrize("padded", [True, False], ids=["sorted_ids", "plain"])
@pytest.mark.parametrize("name", list(DW))
def test_dw_paths(lib, name, padded):
    counts, _, _, K, N, kernel, splits = DW[name]
    plan = moe.grouped_plan(OPS["dw"], dw_R(name, padded), len(counts), K, N)
    assert (plan.kernel, plan.splits) == (kernel, splits)


def test_every_path_has_a_shape():
    assert {v[6] for v in ROWS.values()} == {0, T64, T128, T256}
    assert {v[5] for v in DW.values()} == {T64, T128, T256}
    for kernel in (0, T64, T256):
        assert {v[7] > 1 for v in ROWS.values() if v[6] == kernel} == {True, False}
    assert {v[6] > 1 for v in DW.values() if v[5] == T256} == {True, False}


@pytest.mark.parametrize("name", [n for n in DW if n.startswith("full, many tiles")])
def test_a_workgroup_has_several_tiles_of_several_steps(lib, name):
    """The tiles of the weight gradient's workgroups, as they walk them: XCD x
    takes an eighth of every expert's tiles, its workgroups every 32nd of the
    list."""
    counts, _, _, K, N, _, _ = DW[name]
    tiles = -(-K // 256) * -(-N // 256)
    per_xcd = -(-tiles // 8)
    grid = moe.grouped_plan(OPS["dw"], dw_R(name), len(counts), K, N).workgroups
    runs = []
    for wg in range(grid):
        xcd, at, run = wg % 8, wg // 8, []
        while at < len(counts) * per_xcd:
            e = at // per_xcd
            i = (xcd + e + e // 8 + e // 32) % 8 * per_xcd + at % per_xcd
            if i < tiles:
                run.append(-(-counts[e] // 64))
            at += grid // 8
        runs.append(run)
    assert sum(map(len, runs)) == tiles * len(counts)
    # two tiles of several steps one after the other, of unlike numbers of steps
    assert any(a >= 2 and b >= 2 and a != b for r in runs for a, b in zip(r, r[1:]))
    if 0 in counts:       # and with a tile without rows between them
        assert any(a >= 2 and b == 0 and c >= 2 for r in runs for a, b, c in zip(r, r[1:], r[2:]))
