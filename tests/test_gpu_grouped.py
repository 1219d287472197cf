"""Matrix products grouped by expert against fp64 products of the same rows.

Bounds, elementwise: an output of n products of bf16 values (exact in fp32)
summed in fp32 in any order is off by at most n half steps of the summed
magnitudes -- taken twice, for sums inside a matrix instruction that cut
instead of rounding -- and its rounding to bf16 by half a step of itself.
Where a bound says that a value is exactly zero, it has to be.
"""
import pytest
import torch

from tests._train_ref import U16, U32, bf16, check, f32, grouped_dw, grouped_rows, routing

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import moe_layer_04_amd as m
    m.load_library()
    return m


def note(msg):
    print(f"[gpu-test] {msg}", flush=True)


def bound(want, mag, n, out=torch.bfloat16):
    b = 2 * n * U32 * mag
    return b + U16 * (want.abs() + b) if out == torch.bfloat16 else b + U32 * want.abs()


# T, topk, E, K, N, block_m of moe_align, experts nobody picks
SHAPES = [
    (1, 2, 16, 256, 512, 1, ()),             # one token
    (1, 1, 1, 64, 64, 1, ()),
    (3, 2, 4, 8, 8, 1, ()),                  # narrower than any tile
    (5, 3, 7, 1, 1, 1, ()),
    (8, 2, 8, 512, 384, 16, ()),             # padded ranges
    (33, 2, 5, 72, 136, 1, (0, 4)),          # first and last expert empty
    (64, 8, 256, 128, 64, 1, ()),            # 256 experts, two rows each
    (100, 1, 3, 257, 129, 1, (1,)),          # odd widths
    (130, 2, 2, 331, 1000, 64, ()),
    (150, 4, 4, 520, 264, 1, ()),            # 150 rows an expert
    (600, 2, 2, 328, 256, 1, ()),            # 600 rows an expert
    (777, 2, 6, 192, 320, 128, (2,)),        # long, padded
    (1500, 2, 5, 640, 512, 1, (3,)),         # full tiles
    (1100, 1, 1, 1032, 776, 1, ()),          # one expert, widths that fill no tile
    (2100, 1, 2, 72, 136, 1, ()),            # few outputs, many rows: dw in ranges
    (3000, 1, 3, 264, 520, 1, (1,)),
    (1500, 2, 2, 136, 72, 64, ()),
    (4200, 1, 1, 8, 16, 1, ()),
    (40, 2, 4, 2056, 4104, 1, ()),           # few rows, wide: small tiles
    (9, 2, 16, 2048, 8200, 1, (3,)),
    (20, 2, 16, 200, 40, 4, ()),             # the weight stream, padded, a reduction tail
    (23, 1, 23, 4096, 24, 1, (0, 22)),
    (64, 1, 1, 2100, 13, 1, ()),             # few outputs of a long reduction: in ranges
    (64, 1, 1, 13, 2100, 1, ()),
    (70, 2, 2, 4096, 136, 16, ()),
    (70, 2, 2, 136, 4104, 16, ()),
    (2, 2, 8, 8200, 40, 4, ()),              # the same of the weight stream
    (3, 1, 3, 8704, 1000, 1, (1,)),
    (2100, 1, 2, 2056, 1032, 1, ()),         # and of full tiles
    (1100, 2, 4, 1032, 2056, 64, (1,)),
    (1030, 1, 1, 7304, 1096, 1, ()),
    (1030, 1, 1, 1096, 7304, 1, ()),
    (700, 2, 2, 65, 4100, 1, ()),            # odd widths, many outputs
    (700, 2, 2, 4100, 65, 16, ()),
    (300, 2, 4, 1030, 2051, 64, (2,)),
    (12000, 1, 3, 136, 72, 64, (1,)),        # dw in ranges, padded, an expert without rows
    (90, 2, 40, 520, 264, 1, (7,)),          # dw: few full tiles of many experts
    (500, 2, 60, 520, 776, 16, (7,)),
]


def setup(moe, T, topk, E, block_m, skip, seed):
    ids = routing(T, topk, E, seed, skip)
    sorted_ids, _, offsets, npad = moe.moe_align(ids, E, block_m)
    return sorted_ids, offsets, npad


@pytest.mark.parametrize("shape", SHAPES, ids=[str(s[:6]) for s in SHAPES])
@pytest.mark.parametrize("rows", ["sorted", "gather", "scatter", "both"])
@pytest.mark.parametrize("op", ["fwd", "dx"])
def test_rows(moe, op, rows, shape):
    T, topk, E, K, N, bm, skip = shape
    note(f"{op} {rows} {shape}")
    dx = op == "dx"
    ids, off, _ = setup(moe, T, topk, E, bm, skip, 11)
    gather, scatter = rows in ("gather", "both"), rows in ("scatter", "both")
    R = ids.shape[0]
    red, width = (N, K) if dx else (K, N)
    src = bf16((T if gather else R, red), 1)
    if not gather:
        src[off[-1]:] = float("nan")          # rows in no range
    w = bf16((E, N, K), 2, red ** -0.5)
    for e in skip:
        w[e] = float("nan")                   # an expert nobody picks
    out = torch.full((T * topk if scatter else R, width), 7.0, dtype=torch.bfloat16, device="cuda")
    call = moe.moe_grouped_gemm_dx if dx else moe.moe_grouped_gemm
    got = call(src, w, off, sorted_ids=ids, topk=topk, num_tokens=T, gather=gather,
               scatter=scatter, out=out.clone())
    want, mag = grouped_rows(src, w, off, ids, topk, T, gather, scatter, out, dx)
    torch.cuda.synchronize()
    check(got, want, torch.where(mag > 0, bound(want, mag, red), 0 * mag), op)


@pytest.mark.parametrize("shape", SHAPES, ids=[str(s[:6]) for s in SHAPES])
@pytest.mark.parametrize("rows", ["sorted", "gather_x", "gather_dy", "both"])
@pytest.mark.parametrize("out", ["bf16", "fp32", "add"])
def test_dw(moe, out, rows, shape):
    T, topk, E, K, N, bm, skip = shape
    note(f"dw {out} {rows} {shape}")
    ids, off, _ = setup(moe, T, topk, E, bm, skip, 12)
    gx, gy = rows in ("gather_x", "both"), rows in ("gather_dy", "both")
    R = ids.shape[0]
    x, dy = bf16((T if gx else R, K), 3), bf16((T if gy else R, N), 4)
    # padding rows and rows in no range are not read
    pad = (ids < 0) | (ids >= T * topk)
    for t, gathered in ((x, gx), (dy, gy)):
        if not gathered:
            t[pad] = float("nan")
    want, mag = grouped_dw(dy, x, off, ids, topk, T, gy, gx)
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    buf = f32((E, N, K), 5).to(dt)
    if out == "add":
        want = want + buf.double()
        mag = mag + buf.double().abs()
    got = moe.moe_grouped_gemm_dw(dy, x, off, sorted_ids=ids, topk=topk, num_tokens=T,
                                  gather_dy=gy, gather_x=gx, out=buf.clone(),
                                  accumulate=out == "add")
    torch.cuda.synchronize()
    most = int((off[1:] - off[:-1]).max())
    check(got, want, torch.where(mag > 0, bound(want, mag, most + 1, dt), 0 * mag), "dw")


def test_without_sorted_ids_and_a_gap(moe):
    """Ranges that do not start at row 0 and leave rows behind the last one."""
    note("offsets with gaps")
    off = torch.tensor([3, 3, 40, 90], dtype=torch.int32, device="cuda")
    for K, N in ((64, 72), (33, 19), (256, 512)):
        x, dy = bf16((100, K), 1), bf16((100, N), 2)
        for t in (x, dy):
            t[:3] = t[90:] = float("inf")
        w = bf16((3, N, K), 3)
        for dx in (False, True):
            out = torch.full((100, K if dx else N), -3.0, dtype=torch.bfloat16, device="cuda")
            call = moe.moe_grouped_gemm_dx if dx else moe.moe_grouped_gemm
            got = call(dy if dx else x, w, off, out=out.clone())
            want, mag = grouped_rows(dy if dx else x, w, off, None, 1, 0, False, False, out, dx)
            check(got, want, torch.where(mag > 0, bound(want, mag, N if dx else K), 0 * mag))
        got = moe.moe_grouped_gemm_dw(dy, x, off, out_dtype=torch.float32)
        want, mag = grouped_dw(dy, x, off, None, 1, 0, False, False)
        check(got, want, bound(want, mag, 50, torch.float32))
        assert not got[0].any()               # an expert without rows


def test_no_rows(moe):
    note("no rows")
    w = bf16((3, 24, 16), 1)
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    none = torch.empty((0,), dtype=torch.int32, device="cuda")
    x, dy = w.new_empty((0, 16)), w.new_empty((0, 24))
    assert moe.moe_grouped_gemm(x, w, off).shape == (0, 24)
    assert moe.moe_grouped_gemm_dx(dy, w, off, sorted_ids=none, gather=True).shape == (0, 16)
    got = moe.moe_grouped_gemm_dw(dy, x, off, out=torch.ones((3, 24, 16), device="cuda"))
    assert not got.any()
    got = moe.moe_grouped_gemm_dw(dy, x, off, out=torch.ones((3, 24, 16), device="cuda"),
                                  accumulate=True)
    assert (got == 1).all()
    # no tokens, but sorted rows: all of them padding
    ids = torch.zeros(5, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 2, 5, 5], dtype=torch.int32, device="cuda")
    y = moe.moe_grouped_gemm(x, w, off, sorted_ids=ids, gather=True)
    assert y.shape == (5, 24) and not y.any()
    got = moe.moe_grouped_gemm_dw(dy, x, off, sorted_ids=ids, gather_x=True, gather_dy=True)
    assert not got.any()
    assert moe.moe_grouped_gemm(bf16((5, 16), 3), w, off, sorted_ids=ids, num_tokens=0,
                                scatter=True).shape == (0, 24)


def test_offsets_out_of_range_stay_in_bounds(moe):
    """Offsets past the rows are cut to them: nothing is read or written
    outside, and the ranges inside keep their results."""
    note("offsets past the rows")
    K = N = 64
    x, w = bf16((40, K), 1), bf16((3, N, K), 2)
    off = torch.tensor([-5, 10, 40, 4000], dtype=torch.int32, device="cuda")
    buf = torch.full((80, N), 5.0, dtype=torch.bfloat16, device="cuda")
    got = moe.moe_grouped_gemm(x, w, off, out=buf[:40])
    cut = torch.tensor([0, 10, 40, 40], dtype=torch.int32, device="cuda")
    assert torch.equal(got, moe.moe_grouped_gemm(x, w, cut))
    assert (buf[40:] == 5).all()
    dw = moe.moe_grouped_gemm_dw(x, x, off)
    assert torch.equal(dw, moe.moe_grouped_gemm_dw(x, x, cut))


def test_special_values(moe):
    """Infinities and NaN stay in their rows, a value of the type's range
    comes out as infinity."""
    note("special values")
    for T, K, N in ((4, 64, 64), (300, 320, 512)):
        off = torch.tensor([0, T // 2, T], dtype=torch.int32, device="cuda")
        x, w = bf16((T, K), 1), bf16((2, N, K), 2)
        clean = moe.moe_grouped_gemm(x, w, off)
        x[1, 3] = float("inf")
        x[T - 1, 0] = float("nan")
        x[0] = 3e38
        got = moe.moe_grouped_gemm(x, w, off)
        keep = torch.ones(T, dtype=torch.bool)
        keep[[0, 1, T - 1]] = False
        assert torch.equal(got[keep.cuda()], clean[keep.cuda()])
        assert not torch.isfinite(got[1]).any() and torch.isnan(got[T - 1]).all()


def test_same_bits_every_time(moe):
    note("determinism")
    T, topk, E, K, N = 700, 2, 4, 512, 768
    ids, off, _ = setup(moe, T, topk, E, 1, (), 5)
    x, dy, w = bf16((T, K), 1), bf16((2 * T, N), 2), bf16((E, N, K), 3)

    def once():
        return (moe.moe_grouped_gemm(x, w, off, sorted_ids=ids, topk=topk, gather=True),
                moe.moe_grouped_gemm_dx(dy, w, off, sorted_ids=ids, topk=topk, num_tokens=T,
                                        scatter=True),
                moe.moe_grouped_gemm_dw(dy, x, off, sorted_ids=ids, topk=topk, gather_x=True,
                                        out_dtype=torch.float32))
    first = once()
    for _ in range(4):
        for a, b in zip(first, once()):
            assert torch.equal(a, b)


def test_ranges_in_a_graph(moe):
    """Products in ranges, captured: two graphs that replay in turn, with eager
    calls between them."""
    note("ranges in a graph")
    T, K, N = 150, 4096, 200
    off = torch.tensor([0, 70, 150], dtype=torch.int32, device="cuda")
    w = bf16((2, N, K), 2, K ** -0.5)
    xs = [bf16((T, K), 7), bf16((T, K), 8)]

    def run(x):
        return moe.moe_grouped_gemm(x, w, off)
    want = [run(x).clone() for x in xs]
    assert moe.moe_grouped_gemm(xs[0], w, off, workspace=torch.empty(
        1 << 24, dtype=torch.uint8, device="cuda")).equal(want[0])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run(xs[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(run(x))
        graphs.append(graph)
    for _ in range(3):
        for graph, out, y in zip(graphs, outs, want):
            out.zero_()
            graph.replay()
            assert torch.equal(run(xs[1]), want[1])
            torch.cuda.synchronize()
            assert torch.equal(out, y)


def test_two_streams(moe):
    """Calls that run at the same time on two streams."""
    note("two streams")
    sets = []
    for seed in (1, 2):
        T, topk, E, K, N = 900, 2, 3, 512, 512
        ids, off, _ = setup(moe, T, topk, E, 1, (), seed)
        sets.append((bf16((T, K), seed), bf16((2 * T, N), seed + 5), bf16((E, N, K), seed + 9), ids,
                     off))

    def run(s):
        x, dy, w, ids, off = s
        return (moe.moe_grouped_gemm(x, w, off, sorted_ids=ids, topk=2, gather=True),
                moe.moe_grouped_gemm_dw(dy, x, off, sorted_ids=ids, topk=2, gather_x=True))
    want = [run(s) for s in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(run(sets[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_refusals(moe):
    note("refusals")
    x, w = bf16((8, 32), 1), bf16((2, 16, 32), 2)
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    ids = torch.arange(8, dtype=torch.int32, device="cuda")
    f = moe.moe_grouped_gemm
    bad = [
        lambda: f(x.float(), w, off), lambda: f(x, w.float(), off), lambda: f(x, w, off.long()),
        lambda: f(x, w, off[:2].contiguous()), lambda: f(x[:, :16], w, off),
        lambda: f(bf16((32, 8), 1).t(), w, off), lambda: f(x, w[:, :, :16], off),
        lambda: f(x, w, off, gather=True), lambda: f(x, w, off, scatter=True),
        lambda: f(x, w, off, sorted_ids=ids),                       # no num_tokens
        lambda: f(x, w, off, sorted_ids=ids[:6], num_tokens=8),      # rows do not match
        lambda: f(x, w, off, sorted_ids=ids, gather=True, num_tokens=7),
        lambda: f(x, w, off, sorted_ids=ids.long(), gather=True),
        lambda: f(x, w, off, out=torch.empty((8, 16), device="cuda")),
        lambda: f(x, w, off, out=bf16((8, 17), 1)),
        lambda: f(x.cpu(), w, off), lambda: f(x, w, off.cpu()),
        lambda: moe.moe_grouped_gemm_dx(x, w, off),                 # rows of K, not of N
        lambda: moe.moe_grouped_gemm_dw(x, x[:4], off),
        lambda: moe.moe_grouped_gemm_dw(x, x, off, gather_x=True),
        lambda: moe.moe_grouped_gemm_dw(x, x, off, accumulate=True),
        lambda: moe.moe_grouped_gemm_dw(x, x, off, out=bf16((2, 32, 32), 1), accumulate=True),
        lambda: moe.moe_grouped_gemm_dw(x, x, off, out_dtype=torch.float16),
        lambda: moe.moe_grouped_gemm_dw(x, x[:5], off, sorted_ids=ids, gather_x=True,
                                        gather_dy=True),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"case {i} was taken")
    with pytest.raises(moe.MoEError):
        moe.moe_grouped_gemm(x, w, off, sorted_ids=ids, gather=True, topk=17)
    with pytest.raises(moe.MoEError):
        moe.moe_grouped_gemm(bf16((260,), 1)[4:].view(8, 32), w, off)   # 8-byte aligned
    with pytest.raises(moe.MoEError):
        moe.moe_grouped_gemm_dw(x, x, off, workspace=torch.empty(0, dtype=torch.uint8,
                                                                  device="cuda"))
