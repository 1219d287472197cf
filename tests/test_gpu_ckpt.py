"""Activations kept in 8 bits: codes and values exactly, and the activation and
the weight gradient that read them against fp64 forms of the kept values.

Bounds of the activation and its gradients are those of the operators without
checkpoints (test_gpu_block_ops.py): kept values are inputs like others, and
bringing them back rounds nothing.
"""
import pytest
import torch

from tests._ckpt_ref import keep, keep_halves, spread
from tests._paths import DW
from tests._train_ref import U16, U32, bf16, check, f32, routing, silu_mul

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import moe_layer_04_amd as m
    m.load_library()
    return m


def note(msg):
    print(f"[gpu-test] {msg}", flush=True)


def equal(got, want):
    """equal values, NaN in the same places"""
    return torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))


# --------------------------------------------------------------------------
# rows
# --------------------------------------------------------------------------

ROWS = [(1, 1), (1, 8), (3, 31), (2, 32), (5, 33), (7, 100), (16, 1000), (203, 1001), (64, 4096),
        (3, 7), (9, 24), (1, 16391), (2, 40960), (1000, 40), (4099, 5)]


@pytest.mark.parametrize("R,W", ROWS)
def test_rows_exactly(moe, R, W):
    note(f"ckpt_rows {R} x {W}")
    x = spread(R, W, 10 + R)
    x[0, W // 2] = 255 * 2.0 ** 120
    if R > 6:
        x[1, 0], x[3, W - 1], x[5, W // 2] = float("inf"), float("nan"), float("-inf")
    x = x.cuda()
    codes, X, values = keep(x)
    got_codes, got_X = moe.moe_ckpt_rows(x)
    assert torch.equal(got_X, X)
    assert torch.equal(got_codes, codes)
    back = moe.moe_ckpt_restore(got_codes, got_X)
    assert equal(back.double(), values)
    again = moe.moe_ckpt_rows(back)
    assert torch.equal(again[0], codes) and torch.equal(again[1], X)   # nothing changes any more


def test_every_code_and_scale(moe):
    note("ckpt_restore, every code and scale")
    codes = torch.arange(-127, 128, dtype=torch.int8, device="cuda").repeat(256, 1)
    codes = torch.nn.functional.pad(codes, (0, 1))
    X = torch.arange(256, device="cuda").to(torch.uint8).view(256, 1).repeat(1, 8)
    # (Python's powers: those of the GPU's pow are not exact)
    step = torch.tensor([2.0 ** (e - 133) for e in range(256)], dtype=torch.float64, device="cuda")[:, None]
    want = codes.double() * step
    want[255] = float("nan")
    assert equal(moe.moe_ckpt_restore(codes, X).double(), want)


def test_rows_out_and_nothing_past_them(moe):
    note("ckpt, nothing past the rows")
    for R, W in ((5, 33), (3, 64), (1, 1)):
        x = spread(R, W, 5).cuda()
        codes, X = moe.moe_ckpt_rows(x)
        buf = torch.full((R * W + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
        got = moe.moe_ckpt_restore(codes, X, out=buf[:R * W].view(R, W))
        assert got.data_ptr() == buf.data_ptr()
        assert torch.equal(got.double(), keep(x)[2])
        assert (buf[R * W:] == 7).all()
    assert moe.moe_ckpt_rows(x[:0])[0].shape == (0, 1)
    assert moe.moe_ckpt_restore(codes[:0], X[:0]).shape == (0, 1)


# --------------------------------------------------------------------------
# the activation
# --------------------------------------------------------------------------

def rounded(want, err):
    return err + U16 * (want.abs() + err)


ACT = [(1, 1), (1, 8), (2, 14336), (3, 333), (5, 2048), (7, 2056), (16, 512), (40, 24), (300, 1000),
       (513, 64), (6, 31), (2, 4099)]


@pytest.mark.parametrize("R,N", ACT)
@pytest.mark.parametrize("mode", ["plain", "weights", "sorted", "padded"])
def test_silu_mul(moe, R, N, mode):
    note(f"silu_mul_ckpt R={R} N={N} {mode}")
    g = bf16((R, 2 * N), 1, 3.0)
    da = bf16((R, N), 2)
    wt = ids = num = None
    p = torch.arange(R, device="cuda")
    last = R
    if mode != "plain":
        wt = f32((R,), 3)
    if mode in ("sorted", "padded"):
        p = torch.randperm(R, generator=torch.Generator().manual_seed(4)).cuda()
        ids = p.to(torch.int32)
    if mode == "padded":
        ids[::3] = R                                   # moe_align's sentinel
        ids[R // 2] = -1
        last = R - R // 4
        num = torch.tensor([last], dtype=torch.int32, device="cuda")
    ok = torch.ones(R, dtype=torch.bool, device="cuda") if ids is None else (ids >= 0) & (ids < R)
    w = torch.ones(R, dtype=torch.float64, device="cuda") if wt is None else wt.double()[p]
    w = torch.where(ok, w, torch.zeros_like(w))
    g[~ok] = float("nan")                               # padding rows are not read
    gz = torch.where(ok[:, None], g, torch.zeros_like(g))
    out = torch.full((R, N), 9.0, dtype=torch.bfloat16, device="cuda")
    got, codes, X = moe.moe_silu_mul_ckpt(g, wt, sorted_ids=ids, num_rows=num, out=out.clone())
    want, _ = silu_mul(gz, w)
    check(got[:last], want[:last], rounded(want, 64 * U32 * want.abs())[:last], "a")
    assert (got[last:] == 9).all()
    k_codes, k_X, kept = keep_halves(gz)
    assert torch.equal(codes[:last], k_codes[:last]) and torch.equal(X[:last], k_X[:last])

    # rows that are not read may have kept anything
    codes[~ok], X[~ok] = 77, 255
    dg, dw, a = moe.moe_silu_mul_bwd_ckpt(da, codes, X, wt, sorted_ids=ids, num_rows=num)
    x = kept.requires_grad_()
    wl = w.clone().requires_grad_()
    again, act_u = silu_mul(x, wl)
    wx, ww = torch.autograd.grad(again, (x, wl), da.double())
    again, act_u = again.detach(), act_u.detach()
    check(a[:last], again[:last], rounded(again, 64 * U32 * again.abs())[:last], "a again")
    z, u, d = kept[:, :N].detach(), kept[:, N:].detach(), da.double()
    # s + z s (1 - s): its two terms may cancel
    s = torch.sigmoid(z)
    mag = torch.cat(((d * w[:, None] * u).abs() * (s + (z * s * (1 - s)).abs()), wx[:, N:].abs()), 1)
    check(dg[:last], wx[:last], rounded(wx, 64 * U32 * mag)[:last], "dg")
    if wt is not None:
        named = p[:last][ok[:last]]
        b = (N + 64) * U32 * (d * act_u).abs().sum(1)
        check(dw[named], ww[:last][ok[:last]], b[:last][ok[:last]], "dw")
    else:
        assert dw is None
    short = moe.moe_silu_mul_bwd_ckpt(da, codes, X, wt, sorted_ids=ids, num_rows=num, again=False)
    assert short[2] is None and torch.equal(short[0][:last], dg[:last])


def test_gradients_against_differences(moe):
    """The backward's gradients against central differences of the forward's
    formula in fp64 at the kept values."""
    note("silu_mul_bwd_ckpt, differences")
    R, N, h = 3, 40, 1e-5
    wt = f32((R,), 3, 0.3, 1.0)
    a, codes, X = moe.moe_silu_mul_ckpt(bf16((R, 2 * N), 1, 2.0), wt)
    da = bf16((R, N), 2)
    dg, dw, _ = moe.moe_silu_mul_bwd_ckpt(da, codes, X, wt)
    v = moe.moe_ckpt_restore(codes.view(2 * R, N), X.view(2 * R, -1)).view(R, 2 * N).double()

    def loss(v, w):
        return (silu_mul(v, w)[0] * da.double()).sum(1)

    for c in range(2 * N):
        e = torch.zeros_like(v)
        e[:, c] = h
        want = (loss(v + e, wt.double()) - loss(v - e, wt.double())) / (2 * h)
        # the difference is off by h^2/6 of the third derivative (below 2 |da u w|
        # here) and by 2^-52 of the sum over h; the gradient is rounded to bf16
        tol = U16 * want.abs() + 64 * U32 * 8 * da.double().abs().amax(1) * v.abs().amax(1) + 1e-8
        assert ((dg[:, c].double() - want).abs() <= tol).all(), c
    want = (loss(v, wt.double() + h) - loss(v, wt.double() - h)) / (2 * h)
    mag = (silu_mul(v, torch.ones_like(wt).double())[0] * da.double()).abs().sum(1)
    assert ((dw.double() - want).abs() <= (N + 64) * U32 * mag + 1e-8).all()


def test_a_block_that_is_not_finite(moe):
    """Comes back as NaN, its neighbours as they are."""
    note("silu_mul_ckpt, infinity")
    g = bf16((2, 2 * 96), 1)
    g[0, 40] = float("inf")
    g[1, 96 + 95] = float("nan")
    _, codes, X = moe.moe_silu_mul_ckpt(g)
    dg, _, a = moe.moe_silu_mul_bwd_ckpt(bf16((2, 96), 2), codes, X)
    nan = torch.zeros((2, 96), dtype=torch.bool, device="cuda")
    nan[0, 32:64] = nan[1, 64:] = True
    assert torch.equal(a.isnan(), nan)
    assert torch.equal(dg[:, :96].isnan(), nan)


# --------------------------------------------------------------------------
# the weight gradient
# --------------------------------------------------------------------------

def dw_case(moe, name, seed, rows, bm=None):
    counts, topk, block, K, N = DW[name][:5]
    E, R = len(counts), sum(counts)
    T = R // topk
    g = torch.Generator().manual_seed(seed)
    e = torch.repeat_interleave(torch.arange(E), torch.tensor(counts))[torch.randperm(R, generator=g)]
    ids, _, off, _ = moe.moe_align(e.to(torch.int32).view(T, topk).cuda(), E, block)
    gx, gy = rows in ("gather_x", "both"), rows in ("gather_dy", "both")
    x = bf16((T if gx else ids.shape[0], K), seed + 1)
    dy = bf16((T if gy else ids.shape[0], N), seed + 2)
    pad = (ids < 0) | (ids >= R)                # padding rows are not read
    for t, gathered in ((x, gx), (dy, gy)):
        if not gathered:
            t[pad] = float("nan")
    return x, dy, off, dict(sorted_ids=ids, topk=topk, num_tokens=T, gather_x=gx, gather_dy=gy)


@pytest.mark.parametrize("name", list(DW))
@pytest.mark.parametrize("rows", ["sorted", "gather_x", "gather_dy", "both"])
def test_dw_of_the_kept_rows(moe, name, rows):
    """Bit for bit the gradient of the rows that come back."""
    note(f"dw_ckpt {name} {rows}")
    x, dy, off, kw = dw_case(moe, name, 7, rows)
    codes, X = moe.moe_ckpt_rows(x)
    back = moe.moe_ckpt_restore(codes, X)
    for out in (torch.bfloat16, torch.float32):
        want = moe.moe_grouped_gemm_dw(dy, back, off, out_dtype=out, **kw)
        got = moe.moe_grouped_gemm_dw_ckpt(dy, codes, X, off, out_dtype=out, **kw)
        assert torch.isfinite(got).all()
        assert torch.equal(got, want)
    was = f32(want.shape, 9)
    got = moe.moe_grouped_gemm_dw_ckpt(dy, codes, X, off, out=was.clone(), accumulate=True, **kw)
    assert torch.equal(got, moe.moe_grouped_gemm_dw(dy, back, off, out=was.clone(), accumulate=True, **kw))


SMALL = [(1, 1, 1, 1, 1), (1, 2, 4, 8, 8), (3, 2, 4, 33, 65), (40, 2, 3, 100, 31), (65, 1, 2, 31, 200),
         (130, 3, 5, 7, 72), (333, 2, 8, 256, 1032)]


@pytest.mark.parametrize("T,topk,E,K,N", SMALL)
@pytest.mark.parametrize("gather", [True, False])
def test_dw_of_small_sizes(moe, T, topk, E, K, N, gather):
    note(f"dw_ckpt T={T} topk={topk} E={E} K={K} N={N} gather={gather}")
    ids, _, off, _ = moe.moe_align(routing(T, topk, E, 3), E, 1)
    x, dy = bf16((T if gather else T * topk, K), 1), bf16((T * topk, N), 2)
    codes, X = moe.moe_ckpt_rows(x)
    v = keep(x)[2]
    kw = dict(sorted_ids=ids, topk=topk, num_tokens=T)
    got = moe.moe_grouped_gemm_dw_ckpt(dy, codes, X, off, gather_x=gather, out_dtype=torch.float32, **kw)
    rows = v[ids.long() // topk] if gather else v
    o = off.tolist()
    for e in range(E):
        a, b = dy[o[e]:o[e + 1]].double().t(), rows[o[e]:o[e + 1]]
        check(got[e], a @ b, 2 * (o[e + 1] - o[e] + 1) * U32 * (a.abs() @ b.abs()), f"expert {e}")
    plain = moe.moe_grouped_gemm_dw_ckpt(dy, *moe.moe_ckpt_rows(rows.to(torch.bfloat16)), off,
                                         out_dtype=torch.float32)
    assert torch.equal(plain, got)


def test_dw_without_rows(moe):
    note("dw_ckpt without rows")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    codes = torch.empty((0, 40), dtype=torch.int8, device="cuda")
    X = torch.empty((0, 2), dtype=torch.uint8, device="cuda")
    got = moe.moe_grouped_gemm_dw_ckpt(bf16((0, 24), 1), codes, X, off)
    assert got.shape == (3, 24, 40) and (got == 0).all()
    # tokens that no row names
    ids = torch.full((5,), -1, dtype=torch.int32, device="cuda")
    off[1:] = 5
    codes, X = moe.moe_ckpt_rows(bf16((4, 40), 2))
    got = moe.moe_grouped_gemm_dw_ckpt(bf16((5, 24), 1), codes, X, off, sorted_ids=ids, topk=2, gather_x=True)
    assert (got == 0).all()


@pytest.mark.parametrize("E,N,K", [(3, 24, 40), (2, 2051, 1030), (16, 1024, 1024)])
def test_dw_without_rows_reads_nothing(moe, E, N, K):
    """R == 0 with tokens and no tensors of rows: null operands, zeros written."""
    note(f"dw_ckpt R=0, null operands, {E} x {N} x {K}")
    import ctypes
    lib = moe.load_library()
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    dw = torch.full((E, N, K), 7.0, dtype=torch.bfloat16, device="cuda")
    n = ctypes.c_size_t(0)
    sizes = (1, 8, 2, 0, E, K, N, 0)
    assert lib.moe_grouped_gemm_dw_ckpt(*[None] * 5, *sizes, None, None, ctypes.byref(n), None) == 0
    ws = torch.empty(n.value, dtype=torch.uint8, device="cuda")
    assert lib.moe_grouped_gemm_dw_ckpt(None, None, None, off.data_ptr(), None, *sizes, dw.data_ptr(),
                                        ws.data_ptr(), ctypes.byref(n),
                                        torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert (dw == 0).all()


# --------------------------------------------------------------------------
# refusals, streams, graphs
# --------------------------------------------------------------------------

def test_refusals(moe):
    x = bf16((4, 40), 1)
    codes, X = moe.moe_ckpt_rows(x)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    wt = f32((4,), 2)
    for call in (lambda: moe.moe_ckpt_rows(x.float()), lambda: moe.moe_ckpt_rows(x[:, :39]),
                 lambda: moe.moe_ckpt_rows(x[0]), lambda: moe.moe_ckpt_rows(x.cpu()),
                 lambda: moe.moe_ckpt_restore(codes, X[:, :1]), lambda: moe.moe_ckpt_restore(x, X),
                 lambda: moe.moe_ckpt_restore(codes, X.to(torch.int32)),
                 lambda: moe.moe_ckpt_restore(codes, X[:3]), lambda: moe.moe_ckpt_restore(codes, X, out=x.float()),
                 lambda: moe.moe_silu_mul_ckpt(x, wt[:3]), lambda: moe.moe_silu_mul_ckpt(codes),
                 lambda: moe.moe_silu_mul_ckpt(bf16((4, 15), 1)),
                 lambda: moe.moe_silu_mul_bwd_ckpt(x, codes, X),
                 lambda: moe.moe_silu_mul_bwd_ckpt(x[:, :20].contiguous(), codes, X[:, :1].contiguous()),
                 lambda: moe.moe_silu_mul_bwd_ckpt(x[:, :20].contiguous(), x, X),
                 lambda: moe.moe_grouped_gemm_dw_ckpt(x, x, X, off),
                 lambda: moe.moe_grouped_gemm_dw_ckpt(x, codes, X[:2], off),
                 lambda: moe.moe_grouped_gemm_dw_ckpt(x[:3], codes, X, off),
                 lambda: moe.moe_grouped_gemm_dw_ckpt(x, codes, X, off, gather_x=True),
                 lambda: moe.moe_grouped_gemm_dw_ckpt(x, codes, X, off, accumulate=True)):
        with pytest.raises(ValueError):
            call()
    # large tiles need the rows brought back in the workspace
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    big, off = bf16((4096, 512), 3), torch.tensor([0, 4096], dtype=torch.int32, device="cuda")
    with pytest.raises(moe.MoEError):
        moe.moe_grouped_gemm_dw_ckpt(big, *moe.moe_ckpt_rows(big), off, workspace=small)
    with pytest.raises(moe.MoEError):            # the output over the codes
        moe.moe_ckpt_restore(codes.view(-1)[:64].view(2, 32), X.view(-1)[:2].view(2, 1),
                             out=codes.view(-1)[32:160].view(torch.bfloat16).view(2, 32))


@pytest.mark.parametrize("R,N", [(6, 333), (200, 512)])
def test_streams_and_graphs(moe, R, N):
    """Forward and backward captured once and replayed on new inputs, with
    eager work in between, and the same calls on two other streams at once."""
    note(f"ckpt graph {R} x {N}")
    off = torch.tensor([0, R // 2, R], dtype=torch.int32, device="cuda")
    g, da, wt = bf16((R, 2 * N), 1), bf16((R, N), 2), f32((R,), 3)

    def step(g, da, wt):
        a, codes, X = moe.moe_silu_mul_ckpt(g, wt)
        dg, dw, again = moe.moe_silu_mul_bwd_ckpt(da, codes, X, wt)
        rows = moe.moe_ckpt_rows(a)
        return (a, dg, dw, again, moe.moe_ckpt_restore(*rows),
                moe.moe_grouped_gemm_dw_ckpt(dg, *rows, off, out_dtype=torch.float32))

    step(g, da, wt)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(g, da, wt)
    for rep in range(4):
        g.copy_(bf16((R, 2 * N), 10 + rep))
        da.copy_(bf16((R, N), 20 + rep))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in outs]
        eager = step(g, da, wt)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, eager))
    jobs = [(g, da, wt), (bf16((R, 2 * N), 31), bf16((R, N), 32), f32((R,), 33))]
    want = [step(*j) for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i].append(step(*jobs[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
