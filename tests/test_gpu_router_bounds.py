"""The balance loss and its gradient against fp64 with the bounds of the sums as the
kernels form them, and values that are not finite in the router's calls.

In half steps of fp32 (U32), relative:

* a probability: d = l - max is off by |d| of them in e^d, the exponential by 4 (two
  of the hardware's, one to make the argument's rounding good, what is left of it
  below one); the sum of a token's by as much and 10 additions, its reciprocal by
  2, the quotient by 1: 2 D + 21 with D the largest |d|, 22 taken.
* a sum over tokens: a lane's tokens one after the other (additions() counts them),
  log2 of the lanes with the same experts, 8 waves, and of many workgroups at
  most 8 a slice and 32 slices; a division.
* the loss: f = count / (n k), two roundings, f P one, the experts' sum 8 levels or 6
  and 8 groups, times E: 20.
* the gradient: p; f, three; the sum of p f as p and f, a product and 10 additions;
  the difference, three products and what they are multiplied with, three.
"""
import math

import pytest
import torch

from tests._train_ref import U32, bf16, check, f32
from tests.test_gpu_router_grad import CASES, balance, grad

pytestmark = pytest.mark.gpu

TINY = 1e-37            # probabilities below fp32's normal range may be zeros


@pytest.fixture(scope="module")
def moe():
    import moe_layer_04_amd as m
    m.load_library()
    return m


def note(msg):
    print(f"[gpu-test] {msg}", flush=True)


def additions(M, E):
    """of a token's probability on its way to probs"""
    lanes = 1 if E <= 4 else 2 if E <= 8 else 4 if E <= 16 else 8 if E <= 32 else 16
    per = M if M * E <= 8192 else max(-(-2048 // E), -(-M // 256))
    groups = -(-M // per)
    lane = -(-per // (8 * (64 // lanes)))
    return lane + int(math.log2(64 // lanes)) + 8 + (-(-groups // 32) + 31 if groups > 1 else 0) + 1


@pytest.mark.parametrize("M,E,topk", CASES + [(131072, 64, 2), (300000, 8, 2), (65537, 100, 4)])
@pytest.mark.parametrize("mask", [None, 0.6])
def test_sums(moe, M, E, topk, mask):
    note(f"balance bounds M={M} E={E} topk={topk} mask={mask}")
    logits = f32((M, E), 21, 2.0) + f32((1, E), 22, 1.0)
    ids = logits.topk(topk, dim=1).indices.to(torch.int32)
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    if mask is not None:
        keep = (torch.rand(M, generator=torch.Generator().manual_seed(3)) < mask).cuda()
        keep[0] = True
    token_mask = None if mask is None else keep
    p, f, counts, n, P, loss, D = balance(logits, ids, keep, E, topk)
    got = moe.moe_balance(logits, ids, token_mask=token_mask)
    assert torch.equal(got[1].long(), counts) and got[2].tolist() == [n]
    off = (2 * D + 22 + additions(M, E)) * U32
    check(got[3], P, off * P + TINY, "probs")
    check(got[0], loss.view(1), (off + 20 * U32) * loss.view(1) + TINY * E, "loss")
    up = torch.tensor([0.37], device="cuda")
    d = moe.moe_balance_bwd(up, logits, got[1], got[2], topk, token_mask=token_mask)
    want, mag = torch.zeros((2, M, E), dtype=torch.float64, device="cuda")
    u = up.double().item()
    want[keep] = grad(p, f, n, u, E)
    mag[keep] = u * E / n * p * (f + (p * f).sum(1, keepdim=True))
    check(d, want, (4 * D + 64) * U32 * mag + TINY * E, "dlogits")


@pytest.mark.parametrize("M,E,topk", [(5, 3, 1), (64, 8, 2), (300, 64, 8), (3000, 130, 4)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_logit_that_is_not_finite(moe, M, E, topk, value):
    """The token's probabilities are NaN and so is what they are summed to; counts
    and the other tokens' gradients are as without it, and so is everything where
    the token does not count."""
    note(f"balance, {value} M={M} E={E}")
    good = f32((M, E), 1, 2.0)
    ids = good.topk(topk, dim=1).indices.to(torch.int32)
    bad, t = good.clone(), M // 2
    bad[t, E - 1] = value
    up = torch.ones(1, device="cuda")
    loss, counts, tokens, probs = moe.moe_balance(bad, ids)
    want = moe.moe_balance(good, ids)
    assert loss.isnan().all() and probs.isnan().all()
    assert torch.equal(counts, want[1]) and torch.equal(tokens, want[2])
    d, dw = (moe.moe_balance_bwd(up, l, counts, tokens, topk) for l in (bad, good))
    assert d[t].isnan().all()
    d[t] = dw[t]
    assert torch.equal(d, dw)
    mask = torch.ones(M, dtype=torch.bool, device="cuda")
    mask[t] = False
    for a, b in zip(moe.moe_balance(bad, ids, token_mask=mask), moe.moe_balance(good, ids, token_mask=mask)):
        assert torch.equal(a, b)
    d = moe.moe_balance_bwd(up, bad, counts, tokens, topk, token_mask=mask)
    assert (d[t] == 0).all() and torch.isfinite(d).all()


@pytest.mark.parametrize("M,K,E", [(70, 40, 9), (70, 41, 9), (200, 136, 70), (200, 333, 70), (130, 5, 65), (60, 3, 2),
                                   (900, 264, 8), (900, 267, 8)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_operands_that_are_not_finite(moe, M, K, E, value):
    """An infinity or a NaN in a row that is added stays in its value of dx, one in
    the tokens in its column of dw, one in the weights in its column of dx;
    everything else has the bits that it has without."""
    note(f"topk_bwd, {value} M={M} K={K} E={E}")
    rows = 2
    s = dict(x=bf16((M, K), 1), w_router=bf16((E, K), 2), dlogits=f32((M, E), 3), dx_rows=bf16((M * rows, K), 4))
    dx, dw, db = moe.moe_topk_bwd(**s, bias=True)
    for name in ("dx_rows", "x", "w_router"):
        n = s[name].shape[0]
        for i, c in ((0, 0), (n // 2, K // 2), (n - 1, K - 1)):
            t = s[name].clone()
            t[i, c] = value
            gx, gw, gb = moe.moe_topk_bwd(**{**s, name: t}, bias=True)
            odd = torch.zeros((M, K), dtype=torch.bool, device="cuda")
            odd_w = torch.zeros((E, K), dtype=torch.bool, device="cuda")
            if name == "dx_rows":
                odd[i // rows, c] = True
                assert gx[i // rows, c].item() == value or value != value and gx[i // rows, c].isnan()
            elif name == "w_router":
                odd[:, c] = True
            else:
                odd_w[:, c] = True
            assert torch.equal(~torch.isfinite(gx), odd) and torch.equal(~torch.isfinite(gw), odd_w)
            assert torch.equal(gx[~odd], dx[~odd]) and torch.equal(gw[~odd_w], dw[~odd_w])
            assert torch.equal(gb, db)
