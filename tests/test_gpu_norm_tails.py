"""The norms' statistics where one group of columns carries them: rows whose
only large values lie in the last columns, so that a group lost from a sum
changes its result by as much as itself, not by a rounding.

Bounds count the additions that a term of a row's sum passes: a thread adds
its columns one after the other, the 64 lanes of a wave in 6 steps and at most
16 waves in a row; 16 more half steps cover the products around the sum, the
reciprocal root and the weights.
"""
import pytest
import torch

from tests._train_ref import U16, U32, check, f32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import moe_layer_04_amd as m
    m.load_library()
    return m


def note(msg):
    print(f"[gpu-test] {msg}", flush=True)


def depth(K):
    """Additions behind a row's sum: the fewest threads of a row are K / 16 up to
    16384 columns and 512 for longer ones."""
    return (16 if K <= 16384 else -(-K // 4096) * 8) + 6 + 16 + 16


def tail(M, K, seed, dtype=torch.float32):
    """Rows of 2^-10, and values around 100 in the last one to eight columns."""
    t = f32((M, K), seed, 2.0 ** -10)
    n = (K - 1) % 8 + 1
    t[:, K - n:] = f32((M, n), seed + 1, 20.0, 100.0)
    return t.to(dtype)


KS = [1, 7, 9, 64, 513, 520, 1032, 2056, 4096, 4104, 8192, 8193, 8200, 16384, 16392, 20001, 40960]


@pytest.mark.parametrize("K", KS)
@pytest.mark.parametrize("h_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_statistics_of_the_last_columns(moe, K, h_dtype):
    note(f"norm tails, forward, K={K} {h_dtype}")
    M, eps = 5, 1e-6
    wp, wn = f32((K,), 3, 0.1, 1.0), f32((K,), 4, 0.1, 1.0)
    d = depth(K)

    def rstd(v):
        return (v.double().square().mean(1) + eps).rsqrt()
    h = tail(M, K, 1, h_dtype)
    _, u, _, r2 = moe.moe_block_norm(h, w_pre=wn, eps=eps)
    want = rstd(h)
    check(r2, want, d * U32 * want, "rstd_pre alone")
    wu = h.double() * want[:, None] * wn.double()
    check(u, wu, (1.01 * U16 + d * U32) * wu.abs(), "u")
    # the statistic of the block's output, then that of the stream as kept
    o = tail(M, K, 5, torch.bfloat16)
    ho, u, r1, r2 = moe.moe_block_norm(h, o, None, wp, wn, eps=eps)
    want = rstd(o)
    check(r1, want, d * U32 * want, "rstd_post")
    want = rstd(ho)
    check(r2, want, d * U32 * want, "rstd_pre")
    wu = ho.double() * want[:, None] * wn.double()
    check(u, wu, (1.01 * U16 + d * U32) * wu.abs(), "u of both")


@pytest.mark.parametrize("K", KS)
@pytest.mark.parametrize("h_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("which", ["du", "dh_out"])
def test_gradients_of_the_last_columns(moe, K, h_dtype, which):
    """The rows' sums of the backward, carried by the last columns of one
    incoming gradient."""
    note(f"norm tails, backward, K={K} {h_dtype} {which}")
    M, eps, scale = 5, 1e-6, 0.5
    # sums that follow one another: each result passes two of them
    err = 2 * depth(K) * U32
    h, o = f32((M, K), 10).to(h_dtype), f32((M, K), 11).to(torch.bfloat16)
    wp, wn, gate = f32((K,), 12, 0.1, 1.0), f32((K,), 13, 0.1, 1.0), f32((M,), 14, 0.3, 1.0)
    du, dho = (tail(M, K, 15, torch.bfloat16), torch.zeros_like(h)) if which == "du" else \
        (torch.zeros_like(o), tail(M, K, 17, h_dtype))
    r1, r2 = [(t.double().square().mean(1) + eps).rsqrt().float() for t in (o, h)]
    dh, do, dgate, dwp, dwn = moe.moe_block_norm_bwd(dho, du, h, o, gate, wp, wn, r1, r2,
                                                     res_scale=scale)
    n, z = h.double() * r2.double()[:, None], o.double() * r1.double()[:, None]
    c, g = du.double() * wn.double(), (scale * gate.double())[:, None]
    k1 = g.abs() * r1.double()[:, None]
    want = dho.double() + r2.double()[:, None] * (c - n * (c * n).mean(1, keepdim=True))
    mag = dho.double().abs() + r2.double()[:, None] * (
        c.abs() + n.abs() * (c * n).abs().mean(1, keepdim=True))
    half = U16 if h_dtype == torch.bfloat16 else U32
    check(dh, want, err * mag + half * (want.abs() + err * mag), "dh")
    b, bm = want * wp.double(), mag * wp.double().abs()
    wdo = g * r1.double()[:, None] * (b - z * (b * z).mean(1, keepdim=True))
    e = 2 * err * k1 * (bm + z.abs() * (bm * z.abs()).mean(1, keepdim=True))
    check(do, wdo, e + U16 * (wdo.abs() + e), "do")
    check(dgate, scale * (b * z).sum(1), 2 * err * scale * (bm * z.abs()).sum(1), "dgate")
    check(dwp, (g * want * z).sum(0), 2 * err * (g.abs() * mag * z.abs()).sum(0), "dw_post")
    check(dwn, (du.double() * n).sum(0), err * (du.double() * n).abs().sum(0), "dw_pre")
