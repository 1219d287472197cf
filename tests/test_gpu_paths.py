"""The grouped products on every path that computes them (tests/_paths.py):
properties that must hold whichever kernel runs.

Where results are compared with fp64, operands are small integers: every
product, every partial sum in any order and every sum is then an integer below
2^24, exact in fp32, and the result has to be equal, rounded once to its type.
"""
import pytest
import torch

from tests._paths import DW, OP_PATHS, ROWS
from tests._train_ref import bf16, grouped_dw, grouped_rows, routing

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import moe_layer_04_amd as m
    m.load_library()
    return m


def note(msg):
    print(f"[gpu-test] {msg}", flush=True)


def rows_case(moe, name, seed):
    """(src [T,red], w [E,width,red], offsets, sorted ids)"""
    T, topk, E, bm, red, width = ROWS[name][:6]
    ids, _, off, _ = moe.moe_align(routing(T, topk, E, seed), E, bm)
    return bf16((T, red), seed + 1), bf16((E, width, red), seed + 2, red ** -0.5), off, ids


@pytest.mark.parametrize("op,name", OP_PATHS)
@pytest.mark.parametrize("gather", [True, False], ids=["gather", "sorted"])
def test_padding_rows_are_zeros_whatever_the_weights_hold(moe, op, name, gather):
    """Padding rows inside a range are written as zeros, also where the weights
    hold infinities and NaN (zero times either would be NaN)."""
    note(f"padding rows, {op} {name} gather={gather}")
    T, topk, E, bm, red, width = ROWS[name][:6]
    src, w, off, ids = rows_case(moe, name, 3)
    w[:, ::3, 0] = float("inf")
    w[:, 1::3, red // 2] = float("nan")
    w[:, 2::3, red - 1] = float("-inf")
    pad = (ids < 0) | (ids >= T * topk)
    last = int(off[-1])
    pad[last:] = False                        # in no range: left as they were
    assert int(pad.sum()) > 0
    if not gather:
        src = bf16((ids.shape[0], red), 4)
        src[(ids < 0) | (ids >= T * topk)] = float("nan")     # not read
    call = moe.moe_grouped_gemm
    if op == "dx":
        w = w.transpose(1, 2).contiguous()
        call = moe.moe_grouped_gemm_dx
    out = torch.full((ids.shape[0], width), 7.0, dtype=torch.bfloat16, device="cuda")
    got = call(src, w, off, sorted_ids=ids, topk=topk, num_tokens=T, gather=gather, out=out)
    assert (got[pad] == 0).all()
    assert (got[last:] == 7).all()
    real = ~pad
    real[last:] = False
    assert not torch.isfinite(got[real]).any()


def test_refusals_of_sizes_and_of_what_is_no_tensor(moe):
    """Errors are the binding's own, and come before anything is allocated."""
    note("refusals of sizes")
    x, w = bf16((8, 32), 1), bf16((2, 16, 32), 2)
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    ids = torch.arange(8, dtype=torch.int32, device="cuda")
    for call in (lambda: moe.moe_grouped_gemm(x, w, off, sorted_ids=[0] * 8, gather=True),
                 lambda: moe.moe_grouped_gemm(x, w, off, sorted_ids=ids.view(2, 4), gather=True),
                 lambda: moe.moe_grouped_gemm(x, w, off, workspace=bytearray(4096)),
                 lambda: moe.moe_silu_mul(x, [1.0] * 8)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: moe.moe_grouped_gemm(x, w, off, sorted_ids=ids, num_tokens=-3,
                                              scatter=True),
                 lambda: moe.moe_grouped_gemm_dx(bf16((8, 16), 3), w, off, sorted_ids=ids, topk=-2,
                                                 num_tokens=4, scatter=True),
                 # an output of 2^60 bytes and more
                 lambda: moe.moe_grouped_gemm(x, w, off, sorted_ids=ids, num_tokens=1 << 30,
                                              topk=1 << 26, scatter=True),
                 lambda: moe.moe_grouped_gemm_dw(x, x, off[:0])):
        with pytest.raises(moe.MoEError):
            call()


def ints(shape, seed, most=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(torch.bfloat16)


class Rows:
    """A rows product of one path on integers."""

    def __init__(self, moe, op, name, seed):
        self.T, self.topk, E, bm, self.red, self.width = ROWS[name][:6]
        self.dx = op == "dx"
        self.call = moe.moe_grouped_gemm_dx if self.dx else moe.moe_grouped_gemm
        self.ids, _, self.off, _ = moe.moe_align(routing(self.T, self.topk, E, seed), E, bm)
        self.R = self.ids.shape[0]
        shape = (E, self.red, self.width) if self.dx else (E, self.width, self.red)
        self.w = ints(shape, seed + 1)
        self.seed = seed

    def run(self, gather=False, scatter=False, src=None, out=None, **kw):
        return self.call(src, self.w, self.off, sorted_ids=self.ids, topk=self.topk,
                         num_tokens=self.T, gather=gather, scatter=scatter, out=out, **kw)

    def want(self, src, out, gather=False, scatter=False):
        y, _ = grouped_rows(src, self.w, self.off, self.ids, self.topk, self.T, gather, scatter, out,
                            self.dx)
        return y.to(torch.bfloat16)

    def src(self, gather, k=0):
        return ints((self.T if gather else self.R, self.red), self.seed + 10 + k)

    def out(self, scatter):
        rows = self.T * self.topk if scatter else self.R
        return torch.full((rows, self.width), 7.0, dtype=torch.bfloat16, device="cuda")


class Dw:
    """A weight gradient of one path on integers; rows: the operands' form."""

    def __init__(self, moe, name, seed, rows="sorted", bm=None):
        counts, self.topk, block, self.K, self.N = DW[name][:5]
        E, R = len(counts), sum(counts)
        self.call, self.E, self.T = moe.moe_grouped_gemm_dw, E, R // self.topk
        g = torch.Generator().manual_seed(seed)
        e = torch.repeat_interleave(torch.arange(E), torch.tensor(counts))[torch.randperm(R, generator=g)]
        self.ids, _, self.off, _ = moe.moe_align(
            e.to(torch.int32).view(self.T, self.topk).cuda(), E, 1 if rows == "plain" else block)
        self.gx, self.gy = rows in ("gather_x", "both"), rows in ("gather_dy", "both")
        if rows == "plain":
            self.ids = None
        self.R = R if self.ids is None else self.ids.shape[0]
        self.x = ints((self.T if self.gx else self.R, self.K), seed + 1)
        self.dy = ints((self.T if self.gy else self.R, self.N), seed + 2)
        if self.ids is not None:             # padding rows are not read
            pad = (self.ids < 0) | (self.ids >= R)
            for t, gathered in ((self.x, self.gx), (self.dy, self.gy)):
                if not gathered:
                    t[pad] = float("nan")

    def run(self, **kw):
        if self.ids is None:
            return self.call(self.dy, self.x, self.off, **kw)
        return self.call(self.dy, self.x, self.off, sorted_ids=self.ids, topk=self.topk,
                         num_tokens=self.T, gather_dy=self.gy, gather_x=self.gx, **kw)

    def want(self):
        return grouped_dw(self.dy, self.x, self.off, self.ids, self.topk, self.T, self.gy, self.gx)[0]


@pytest.mark.parametrize("op,name", OP_PATHS)
@pytest.mark.parametrize("scatter", [False, True], ids=["gather", "scatter"])
def test_rows_exactly(moe, op, name, scatter):
    note(f"exact rows, {op} {name} scatter={scatter}")
    c = Rows(moe, op, name, 21)
    src, out = c.src(not scatter), c.out(scatter)
    got = c.run(not scatter, scatter, src, out.clone())
    assert torch.equal(got, c.want(src, out, not scatter, scatter))


@pytest.mark.parametrize("name", list(DW))
@pytest.mark.parametrize("rows", ["plain", "sorted", "gather_x", "gather_dy", "both"])
def test_dw_exactly(moe, name, rows):
    """Every output type of one input: bf16, fp32, and fp32 added to what is
    there."""
    note(f"exact dw, {name} {rows}")
    c = Dw(moe, name, 31, rows)
    want = c.want()
    assert torch.equal(c.run(), want.to(torch.bfloat16))
    got = c.run(out_dtype=torch.float32)
    assert torch.equal(got, want.float())
    was = ints(got.shape, 39, 1000).float()
    assert torch.equal(c.run(out=was.clone(), accumulate=True), was + want.float())


def paths():
    return [(op, name) for op, name in OP_PATHS] + [("dw", name) for name in DW]


def job(moe, op, name, seed):
    """A call on arbitrary values (where the order of a sum changes its bits),
    as a function of its workspace."""
    if op == "dw":
        c = Dw(moe, name, seed, "gather_x")
        c.x = bf16(c.x.shape, seed + 3)
        c.dy = torch.where(c.dy.isnan(), c.dy, bf16(c.dy.shape, seed + 4))
        return lambda **kw: c.run(out_dtype=torch.float32, **kw)
    c = Rows(moe, op, name, seed)
    src = bf16((c.T, c.red), seed + 5)
    c.w = bf16(c.w.shape, seed + 6)
    return lambda **kw: c.run(True, True, src, **kw)


@pytest.mark.parametrize("op,name", paths())
def test_same_bits_every_time(moe, op, name):
    note(f"determinism, {op} {name}")
    run = job(moe, op, name, 41)
    first = run()
    for _ in range(4):
        assert torch.equal(run(), first)


@pytest.mark.parametrize("op,name", paths())
def test_two_streams_with_a_workspace_each(moe, op, name):
    note(f"two streams, {op} {name}")
    jobs = [job(moe, op, name, 51), job(moe, op, name, 52)]
    want = [run() for run in jobs]
    # more than any of these calls asks for
    spaces = [torch.empty(32 << 20, dtype=torch.uint8, device="cuda") for _ in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i].append(jobs[i](workspace=spaces[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(g, want[i]) for g in got[i])


@pytest.mark.parametrize("op,name", paths())
def test_two_graphs_replayed_in_turn(moe, op, name):
    note(f"graphs, {op} {name}")
    jobs = [job(moe, op, name, 61), job(moe, op, name, 62)]
    want = [run() for run in jobs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for run in jobs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(run())
        graphs.append(graph)
    for _ in range(3):
        for i in (0, 1):
            outs[i].zero_()
            graphs[i].replay()
            assert torch.equal(jobs[1 - i](), want[1 - i])     # eager work in between
            torch.cuda.synchronize()
            assert torch.equal(outs[i], want[i])


@pytest.mark.parametrize("op,name", OP_PATHS)
def test_rows_of_clamped_offsets_and_gaps(moe, op, name):
    """Offsets past the rows are cut to them, rows in no range stay as they
    were, and rows of no range may hold anything."""
    note(f"clamped offsets, {op} {name}")
    c = Rows(moe, op, name, 71)
    off = c.off.tolist()
    E, R = len(off) - 1, c.R
    for first, last in ((-5, R + 4000), (1, R - 1)):
        bad = [first] + off[1:-1] + [last]
        cut = torch.tensor([min(max(v, 0), R) for v in bad], dtype=torch.int32, device="cuda")
        src = c.src(False)
        src[:cut[0]] = src[cut[-1]:] = float("nan")
        buf = torch.full((R + 300, c.width), 7.0, dtype=torch.bfloat16, device="cuda")
        got = c.call(src, c.w, torch.tensor(bad, dtype=torch.int32, device="cuda"), out=buf[:R])
        want = grouped_rows(src, c.w, cut, None, 1, 0, False, False, torch.full_like(got, 7.0), c.dx)[0]
        assert torch.equal(got, want.to(torch.bfloat16))
        assert (buf[R:] == 7).all()


@pytest.mark.parametrize("name", list(DW))
def test_dw_of_clamped_offsets_and_gaps(moe, name):
    note(f"clamped offsets, dw {name}")
    c = Dw(moe, name, 81, "plain")
    off, R = c.off.tolist(), c.R
    for first, last in ((-5, R + 4000), (1, R - 1)):
        bad = [first] + off[1:-1] + [last]
        cut = torch.tensor([min(max(v, 0), R) for v in bad], dtype=torch.int32, device="cuda")
        x, dy = c.x.clone(), c.dy.clone()
        for t in (x, dy):
            t[:cut[0]] = t[cut[-1]:] = float("nan")
        want = grouped_dw(dy, x, cut, None, 1, 0, False, False)[0].float()
        buf = torch.full((want.numel() + 4096,), 7.0, device="cuda")
        got = moe.moe_grouped_gemm_dw(dy, x, torch.tensor(bad, dtype=torch.int32, device="cuda"),
                                      out=buf[:want.numel()].view(want.shape))
        assert torch.equal(got, want)
        assert (buf[want.numel():] == 7).all()


def test_neighbouring_buffers_are_taken(moe):
    """Operands and output side by side in one allocation, sharing no byte."""
    note("neighbouring buffers")
    R, K = 16, 64
    x, w = ints((R, K), 1), ints((1, K, K), 2)
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    buf = torch.empty((2 * R + K, K), dtype=torch.bfloat16, device="cuda")
    buf[R:2 * R], buf[2 * R:] = x, w[0]
    got = moe.moe_grouped_gemm(buf[R:2 * R], buf[2 * R:].view(1, K, K), off, out=buf[:R])
    assert torch.equal(got, moe.moe_grouped_gemm(x, w, off))
    with pytest.raises(moe.MoEError):
        moe.moe_grouped_gemm(buf[R:2 * R], w, off, out=buf[R - 8:2 * R - 8])
