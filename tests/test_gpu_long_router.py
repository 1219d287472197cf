"""The router's gradients and kept activations on tensors of more than 2^31
values: rows behind every 32-bit border, compared with the same rows computed
by themselves, and weight gradients exactly on small integers."""
import pytest
import torch

from tests._train_ref import U32, check, f32
from tests.test_gpu_long import big, picks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import moe_layer_04_amd as m
    m.load_library()
    yield m
    torch.cuda.empty_cache()


def note(msg):
    print(f"[gpu-test] {msg}", flush=True)


def ints(rows, cols, seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty((rows, cols), dtype=dtype, device="cuda")
    for i in range(0, rows, 1 << 14):
        n = min(1 << 14, rows - i)
        t[i:i + n] = torch.randint(-2, 3, (n, cols), generator=g, device="cuda")
    return t


@pytest.mark.parametrize("W", [16384, 16381])
def test_rows(moe, W):
    note(f"ckpt_rows, long, W={W}")
    R = 150_000
    x = big(R, W, 3)                                        # 4.9 GB, 2.5 of codes
    at = picks(R, W)
    codes, X = moe.moe_ckpt_rows(x)
    few = moe.moe_ckpt_rows(x[at].contiguous())
    assert torch.equal(codes[at], few[0]) and torch.equal(X[at], few[1])
    back = moe.moe_ckpt_restore(codes, X)
    assert torch.equal(back[at], moe.moe_ckpt_restore(*few))


@pytest.mark.parametrize("N", [8192, 8190])
def test_silu_mul(moe, N):
    note(f"silu_mul_ckpt, long, N={N}")
    R = 150_000
    g = big(R, 2 * N, 3)
    at = picks(R, 2 * N)
    a, codes, X = moe.moe_silu_mul_ckpt(g)
    s = moe.moe_silu_mul_ckpt(g[at].contiguous())
    for t, few in zip((a, codes, X), s):
        assert torch.equal(t[at], few)
    dg, _, again = moe.moe_silu_mul_bwd_ckpt(a, codes, X)
    sdg, _, sagain = moe.moe_silu_mul_bwd_ckpt(*s)
    assert torch.equal(dg[at], sdg) and torch.equal(again[at], sagain)


def test_dw(moe):
    """Small integers are kept exactly, and so are their sums."""
    note("dw_ckpt, long")
    R, K, N = 300_000, 8192, 64
    off = torch.tensor([0, 120_000, 120_000, R], dtype=torch.int32, device="cuda")
    x, dy = ints(R, K, 1, torch.bfloat16), ints(R, N, 2, torch.bfloat16)
    got = moe.moe_grouped_gemm_dw_ckpt(dy, *moe.moe_ckpt_rows(x), off, out_dtype=torch.float32)
    assert torch.equal(got, moe.moe_grouped_gemm_dw(dy, x, off, out_dtype=torch.float32))


@pytest.mark.parametrize("K", [8192, 8190])
def test_topk_bwd(moe, K):
    note(f"topk_bwd, long, K={K}")
    M, E, topk = 300_000, 9, 2
    x, rows = ints(M, K, 1, torch.bfloat16), ints(M, K, 2, torch.bfloat16)      # 4.9 GB each
    w, dl = ints(E, K, 3, torch.bfloat16), ints(M, E, 4, torch.float32)
    dx, dw, db = moe.moe_topk_bwd(x, w, dlogits=dl, dx_rows=rows, bias=True)
    at = picks(M, K)
    assert torch.equal(dx[at].double(), dl[at].double() @ w.double() + rows[at].double())
    want = torch.zeros((E, K), dtype=torch.float64, device="cuda")
    for i in range(0, M, 1 << 13):
        want += dl[i:i + (1 << 13)].double().t() @ x[i:i + (1 << 13)].double()
    assert torch.equal(dw.double(), want)
    assert torch.equal(db.double(), dl.double().sum(0))


def test_balance(moe):
    note("balance, long")
    M, E, topk = 8_400_000, 256, 1                          # 2.15e9 logits, 8.6 GB
    logits = torch.empty((M, E), device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    P = torch.zeros(E, dtype=torch.float64, device="cuda")
    ids = torch.empty((M, 1), dtype=torch.int32, device="cuda")
    for i in range(0, M, 1 << 18):
        part = torch.randn((min(1 << 18, M - i), E), generator=g, device="cuda")
        logits[i:i + part.shape[0]] = part
        ids[i:i + part.shape[0], 0] = part.argmax(1)
        P += torch.softmax(part.double(), 1).sum(0)
    loss, counts, tokens, probs = moe.moe_balance(logits, ids)
    assert torch.equal(counts.long(), torch.bincount(ids.flatten().long(), minlength=E))
    assert tokens.tolist() == [M]
    # a lane adds 2051 tokens, then 24 additions; probabilities of logits within 13 of
    # their largest are off by 76 half steps (test_gpu_router_grad.py)
    check(probs, P / M, (2051 + 24 + 256 + 76) * U32 * P / M, "probs")
    at = picks(M, E)
    got = moe.moe_balance_bwd(loss, logits, counts, tokens, topk)
    assert torch.equal(got[at], moe.moe_balance_bwd(loss, logits[at].contiguous(), counts, tokens, topk))


def test_rows_past_32_bits_are_refused(moe):
    """2^32 + 8 rows are not taken for 8."""
    note("kept rows past 32 bits")
    far = (1 << 32) + 8
    x = torch.empty((far, 2), dtype=torch.bfloat16, device="cuda")
    codes, X = x.view(torch.int8).view(-1)[:far].view(-1, 1), x.view(torch.uint8).view(-1)[:far].view(-1, 1)
    ids, two = x.view(torch.int32), x.view(torch.uint8).view(-1)[:2 * far].view(far, 2)
    one, w = f32((1,), 1), torch.ones((1, 1), dtype=torch.bfloat16, device="cuda")
    logits = ids.view(torch.float32)
    for call in (lambda: moe.moe_ckpt_rows(x), lambda: moe.moe_ckpt_restore(codes, X),
                 lambda: moe.moe_silu_mul_ckpt(x),
                 lambda: moe.moe_silu_mul_bwd_ckpt(x.view(-1)[:far].view(-1, 1), two.view(torch.int8), two),
                 lambda: moe.moe_balance(logits, ids),
                 lambda: moe.moe_balance_bwd(one, logits, ids.view(-1)[:1], ids.view(-1)[:1], 1),
                 lambda: moe.moe_topk_bwd(x.view(-1)[:far].view(-1, 1), w, dlogits=logits)):
        with pytest.raises(moe.MoEError):
            call()
