"""The pieces on tensors of more than 2^31 values: rows and columns behind every
32-bit border, compared with the same rows computed by themselves or in fp64.
Bounds as in the operators' own tests."""
import pytest
import torch

from tests._train_ref import U16, U32, bf16, check, f32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import moe_layer_04_amd as m
    m.load_library()
    yield m
    torch.cuda.empty_cache()


def note(msg):
    print(f"[gpu-test] {msg}", flush=True)


def big(rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    for i in range(0, rows, 1 << 16):
        n = min(1 << 16, rows - i)
        t[i:i + n] = torch.randn((n, cols), generator=g, device="cuda")
    return t


# rows whose values lie around 2^31 and 2^32 bytes and elements, and the ends
def picks(R, width):
    at = sorted({0, R - 1, *(min(R - 1, b // width + d) for b in (1 << 30, 1 << 31) for d in (-1, 0, 1))})
    return torch.tensor(at, device="cuda")


@pytest.mark.parametrize("K,N", [(64, 8192), (63, 8191)])
def test_grouped(moe, K, N):
    note(f"grouped, long, K={K} N={N}")
    R, E = 300_000, 3
    off = torch.tensor([0, 120_000, 120_000, R], dtype=torch.int32, device="cuda")
    x, w = big(R, K, 1), bf16((E, N, K), 2, 0.1)
    at = picks(R, N)
    e = torch.where(at < 120_000, 0, 2)
    y = moe.moe_grouped_gemm(x, w, off)                     # [R,N]: 4.9 GB
    want = torch.stack([w[int(i)].double() @ x[int(r)].double() for i, r in zip(e, at)])
    mag = torch.stack([w[int(i)].double().abs() @ x[int(r)].double().abs() for i, r in zip(e, at)])
    check(y[at], want, 2 * K * U32 * mag + U16 * want.abs() * 1.01, "y")
    dx = moe.moe_grouped_gemm_dx(y, w, off)                 # reads 4.9 GB
    yd = y[at].double()
    want = torch.stack([d @ w[int(i)].double() for d, i in zip(yd, e)])
    mag = torch.stack([d.abs() @ w[int(i)].double().abs() for d, i in zip(yd, e)])
    check(dx[at], want, 2 * N * U32 * mag + U16 * (want.abs() + 2 * N * U32 * mag), "dx")
    dw = moe.moe_grouped_gemm_dw(y, x, off, out_dtype=torch.float32)
    assert not dw[1].any()
    cols = torch.tensor([0, 1, N // 2, N - 1], device="cuda")
    for e_, a, b in ((0, 0, 120_000), (2, 120_000, R)):
        yc, xc = y[a:b][:, cols].t().double().contiguous(), x[a:b].double()
        want, mag = yc @ xc, yc.abs() @ xc.abs()
        # sums of as many terms as rows, in ranges and steps: twice the depth of
        # a running sum of 64-row steps covers them, and the products are exact
        check(dw[e_][cols], want, 2 * ((b - a) / 16 + 64) * U32 * mag, "dw")


def test_silu_mul(moe):
    note("silu_mul, long")
    R, N = 150_000, 8192
    g = big(R, 2 * N, 3)                                    # 4.9 GB
    at = picks(R, 2 * N)
    a = moe.moe_silu_mul(g)
    few = g[at].contiguous()
    assert torch.equal(a[at], moe.moe_silu_mul(few))
    dg, _ = moe.moe_silu_mul_bwd(a, g)
    assert torch.equal(dg[at], moe.moe_silu_mul_bwd(a[at].contiguous(), few)[0])


@pytest.mark.parametrize("K", [8192, 8191])
def test_block_norm(moe, K):
    note(f"block_norm, long, K={K}")
    M = 300_000
    h, o = big(M, K, 4), big(M, K, 5)
    wp, wn, gate = f32((K,), 6, 0.1, 1.0), f32((K,), 7, 0.1, 1.0), f32((M,), 8)
    ho, u, r1, r2 = moe.moe_block_norm(h, o, gate, wp, wn)
    at = picks(M, K)

    def few(t):
        return t[at].contiguous()
    sho, su, sr1, sr2 = moe.moe_block_norm(few(h), few(o), few(gate), wp, wn)
    for a, b in ((ho, sho), (u, su), (r1, sr1), (r2, sr2)):
        assert torch.equal(a[at], b)
    dh, do, dg, _, _ = moe.moe_block_norm_bwd(h, u, ho, o, gate, wp, wn, r1, r2)
    s = moe.moe_block_norm_bwd(few(h), su, sho, few(o), few(gate), wp, wn, sr1, sr2)
    for a, b in ((dh, s[0]), (do, s[1]), (dg, s[2])):
        assert torch.equal(a[at], b)


def test_rows_past_32_bits_are_refused(moe):
    """2^32 + 8 rows are not taken for 8."""
    note("rows past 32 bits")
    g = torch.empty(((1 << 32) + 8, 2), dtype=torch.bfloat16, device="cuda")
    a = g.view(-1)[:g.shape[0]].view(-1, 1)
    w = torch.ones((1,), device="cuda")
    x, off = torch.ones((1, 1, 2), dtype=torch.bfloat16, device="cuda"), torch.zeros(
        2, dtype=torch.int32, device="cuda")
    for call in (lambda: moe.moe_silu_mul(g), lambda: moe.moe_silu_mul_bwd(a, g),
                 lambda: moe.moe_block_norm(a, w_pre=w), lambda: moe.moe_grouped_gemm(g, x, off),
                 lambda: moe.moe_grouped_gemm_dw(a, g, off),
                 lambda: moe.moe_block_norm_bwd(None, a, a, w_pre=w, rstd_pre=torch.empty(
                     g.shape[0], device="cuda"))):
        with pytest.raises(moe.MoEError):
            call()


@pytest.mark.parametrize("slots", [False, True], ids=["plain", "sorted_ids"])
@pytest.mark.parametrize("K,N", [(64, 8192), (63, 8191)])
def test_grouped_dw_exactly(moe, K, N, slots):
    """Every value of the weight gradients of 300000 rows, on small integers:
    partial sums are at most 4 * 180000 < 2^24, exact in fp32, so that a step
    of rows lost or read from elsewhere cannot hide behind rounding.  With
    sorted_ids every 1000th row is padding."""
    note(f"grouped dw, long, exact, K={K} N={N} sorted_ids={slots}")
    R, cut = 300_000, 120_000
    off = torch.tensor([0, cut, cut, R], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(11)

    def few(rows, cols):
        t = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
        for i in range(0, rows, 1 << 14):
            n = min(1 << 14, rows - i)
            t[i:i + n] = torch.randint(-2, 3, (n, cols), generator=g, device="cuda")
        return t
    x, dy = few(R, K), few(R, N)                            # dy: 4.9 GB
    ids = None
    if slots:
        ids = torch.arange(R, dtype=torch.int32, device="cuda")
        ids[::1000] = R
        x[::1000] = float("nan")
    got = moe.moe_grouped_gemm_dw(dy, x, off, sorted_ids=ids, num_tokens=R, out_dtype=torch.float32)
    want = torch.zeros((3, N, K), dtype=torch.float64, device="cuda")
    for e, a, b in ((0, 0, cut), (2, cut, R)):
        for i in range(a, b, 1 << 13):
            j = min(b, i + (1 << 13))
            xs = x[i:j].double()
            if slots:
                xs[ids[i:j] == R] = 0
            want[e] += dy[i:j].double().t().contiguous() @ xs
    assert torch.equal(got, want.float())
