"""The gated activation and the norms around a block against their fp64 forms.

Bounds: a rounding to bf16 is half a step of the value.  fp32 arithmetic is
counted in half steps of the magnitudes that enter a sum (K or N terms and a
few operations); the exponential of the activation is off by a few half
steps and one more for every unit of its argument, taken here as 64 for
arguments up to 30.
"""
import pytest
import torch

from tests._train_ref import U16, U32, bf16, block_norm, check, f32, silu_mul

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import moe_layer_04_amd as m
    m.load_library()
    return m


def note(msg):
    print(f"[gpu-test] {msg}", flush=True)


def rounded(want, err, dtype=torch.bfloat16):
    return err + (U16 if dtype == torch.bfloat16 else U32) * (want.abs() + err)


# --------------------------------------------------------------------------
# activation
# --------------------------------------------------------------------------

ACT = [(1, 1), (1, 8), (2, 14336), (3, 333), (5, 2048), (7, 2056), (16, 512), (40, 24), (300, 1000),
       (513, 64)]


@pytest.mark.parametrize("R,N", ACT)
@pytest.mark.parametrize("mode", ["plain", "weights", "sorted", "padded"])
def test_silu_mul(moe, R, N, mode):
    note(f"silu_mul R={R} N={N} {mode}")
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
    got = moe.moe_silu_mul(g, wt, sorted_ids=ids, num_rows=num, out=out.clone())
    want, act_u = silu_mul(gz, w)
    check(got[:last], want[:last], rounded(want, 64 * U32 * want.abs())[:last], "a")
    assert (got[last:] == 9).all()

    dg, dw = moe.moe_silu_mul_bwd(da, g, wt, sorted_ids=ids, num_rows=num)
    x = gz.double().requires_grad_()
    wl = w.clone().requires_grad_()
    a, _ = silu_mul(x, wl)
    wx, ww = torch.autograd.grad(a, (x, wl), da.double())
    z, u, d = gz[:, :N].double(), gz[:, N:].double(), da.double()
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


def test_silu_mul_range(moe):
    """Large gates: exactly the up value or zero, no NaN from the exponential."""
    note("silu_mul range")
    z = torch.tensor([-3e38, -1e4, -200.0, -100.0, -0.0, 0.0, 100.0, 1e4, 1e30], device="cuda")
    g = torch.stack((z, torch.ones_like(z)), 0).reshape(1, -1).to(torch.bfloat16)
    got = moe.moe_silu_mul(g)[0].float()
    want = torch.where(z > 0, z.to(torch.bfloat16).float(), torch.zeros_like(z))
    assert torch.equal(got.abs(), want)
    dg, _ = moe.moe_silu_mul_bwd(torch.ones((1, 9), dtype=torch.bfloat16, device="cuda"), g)
    assert torch.isfinite(dg).all()
    assert (dg[0, :4] == 0).all() and (dg[0, 6:9] == 1).all() and (dg[0, 4:6] == 0.5).all()


def test_silu_refusals(moe):
    g = bf16((4, 16), 1)
    wt = f32((4,), 2)
    ids = torch.arange(4, dtype=torch.int32, device="cuda")
    for call in (lambda: moe.moe_silu_mul(g.float()), lambda: moe.moe_silu_mul(g[:, :15]),
                 lambda: moe.moe_silu_mul(bf16((4, 15), 1)), lambda: moe.moe_silu_mul(g, wt[:3]),
                 lambda: moe.moe_silu_mul(g, wt.double()), lambda: moe.moe_silu_mul(g, sorted_ids=ids),
                 lambda: moe.moe_silu_mul(g, wt, sorted_ids=ids[:3]),
                 lambda: moe.moe_silu_mul(g, wt.cpu()),
                 lambda: moe.moe_silu_mul(g, num_rows=torch.tensor([4], device="cuda")),
                 lambda: moe.moe_silu_mul_bwd(g, g)):
        with pytest.raises(ValueError):
            call()
    assert moe.moe_silu_mul(g[:0]).shape == (0, 8)


# --------------------------------------------------------------------------
# norms
# --------------------------------------------------------------------------

# M, K, topk, du_topk
NORM = [(1, 1, 1, 1), (1, 64, 2, 2), (2, 100, 3, 1), (3, 512, 1, 4), (5, 520, 2, 2),
        (8, 4096, 2, 2), (4, 2048, 8, 8), (7, 7168, 8, 1), (3, 8200, 2, 2), (2, 16384, 2, 2),
        (2, 16392, 1, 2), (3, 333, 2, 2), (1030, 72, 2, 2), (600, 1032, 1, 1), (2, 20001, 2, 1),
        (4, 1000, 1, 1), (3, 3000, 2, 2), (520, 4096, 1, 2), (2, 6008, 3, 1), (1, 40960, 2, 2)]
PARTS = ["all", "no_gate", "no_post", "pre_only", "no_pre", "add"]


def norm_inputs(M, K, topk, parts, h_dtype, seed):
    h = f32((M, K), seed, 2.0).to(h_dtype)
    o = None if parts == "pre_only" else bf16((M * topk, K), seed + 1)
    gate = None if parts in ("no_gate", "pre_only", "add") else f32((M,), seed + 2)
    wp = None if parts in ("no_post", "pre_only", "add") else f32((K,), seed + 3, 0.2, 1.0)
    wn = None if parts in ("no_pre", "add") else f32((K,), seed + 4, 0.2, 1.0)
    return h, o, gate, wp, wn


def d(t):
    return None if t is None else t.double()


@pytest.mark.parametrize("M,K,topk,dtopk", NORM)
@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("h_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_block_norm(moe, M, K, topk, dtopk, parts, h_dtype):
    note(f"block_norm M={M} K={K} topk={topk} {parts} {h_dtype}")
    h, o, gate, wp, wn = norm_inputs(M, K, topk, parts, h_dtype, 20)
    scale, eps = 0.625, 1e-5
    ho, u, r1, r2 = moe.moe_block_norm(h, o, gate, wp, wn, topk=topk, res_scale=scale, eps=eps)
    # the second norm is of the stream as it was kept
    wh, wu, w1, w2 = block_norm(d(h), d(o), d(gate), d(wp), d(wn), topk, scale, eps, kept=ho.double())
    n = K + 32
    if o is None:
        assert ho is h
    else:
        # the slots' sum, the norm's statistic (K terms), the products
        mag = (wh - d(h)).abs()
        s = d(o).reshape(M, topk, K)
        lost = scale * s.abs().sum(1) * (1 if gate is None else d(gate).abs()[:, None])
        if wp is not None:
            lost = lost * w1[:, None] * d(wp).abs()
        err = n * U32 * mag + topk * U32 * lost * 2 + 2 * U32 * d(h).abs()
        check(ho, wh, rounded(wh, err, h_dtype), "h_out")
        # a sum of slots is off by topk half steps of its magnitudes
    if wp is not None:
        amp = (s.abs().sum(1) * s.sum(1).abs()).sum(1) / s.sum(1).square().sum(1).clamp_min(1e-30)
        check(r1, w1, w1 * U32 * (n + 4 * topk * amp), "rstd_post")
    if wn is not None:
        check(r2, w2, w2 * U32 * n, "rstd_pre")
        check(u, wu, rounded(wu, n * U32 * wu.abs()), "u")
    else:
        assert u is None and r2 is None

    # ---- backward: gradients of the fp64 form at the kept stream
    dho = None if parts == "no_gate" else f32((M, K), 31).to(h_dtype)
    du = None if wn is None else bf16((M * dtopk, K), 32)
    if parts == "pre_only":
        dho = None
    got = moe.moe_block_norm_bwd(dho, du, ho, o, gate, wp, wn, r1, r2, topk=topk, du_topk=dtopk,
                                 res_scale=scale)
    dus = None if du is None else du.double().reshape(M, dtopk, K)
    gh = torch.zeros((M, K), dtype=torch.float64, device="cuda") if dho is None else dho.double()
    err = U32 * gh.abs()
    if wn is not None:
        dsum = dus.sum(1)
        nn = ho.double().requires_grad_()
        wnl = d(wn).requires_grad_()
        _, uu, _, _ = block_norm(nn, None, None, None, wnl, 1, scale, eps)
        gn, gw = torch.autograd.grad(uu, (nn, wnl), dsum)
        gh = gh + gn
        nh = ho.double() * w2[:, None]
        c = dus.abs().sum(1) * d(wn).abs()
        err = err + (n + dtopk) * U32 * w2[:, None] * (c + nh.abs() * (c * nh.abs()).mean(1, keepdim=True))
        check(got[4], gw, (n + M + dtopk) * U32 * (dus.abs().sum(1) * nh.abs()).sum(0), "dw_pre")
    else:
        assert got[4] is None
    check(got[0], gh, rounded(gh, err, h_dtype), "dh")
    if o is None:
        assert got[1] is None and got[2] is None and got[3] is None
        return
    # the branch: its gradient starts from dh in fp32, which err bounds
    ol = d(o).reshape(M, topk, K).sum(1).requires_grad_()
    gl = None if gate is None else d(gate).requires_grad_()
    wl = None if wp is None else d(wp).requires_grad_()
    b, _, _, _ = block_norm(torch.zeros_like(ol), ol, gl, wl, None, 1, scale, eps)
    leaves = [t for t in (ol, gl, wl) if t is not None]
    grads = list(torch.autograd.grad(b, leaves, gh))
    g_abs = scale * (torch.ones(M, device="cuda", dtype=torch.float64) if gate is None else d(gate).abs())[:, None]
    oabs = d(o).abs().reshape(M, topk, K).sum(1)
    lost = 4 * (n + topk) * U32 * gh.abs() + err
    if wp is not None:
        z, za = ol.detach() * w1[:, None], oabs * w1[:, None]
        bw = lost * d(wp).abs()
        k1 = g_abs * w1[:, None]
        # z's own error comes with the slots' magnitudes; the statistic's with amp
        e_do = k1 * (bw + za * (bw * za).mean(1, keepdim=True)) * (1 + amp[:, None])
        e_gate = scale * (bw * za).sum(1) * (1 + amp)
        e_wp = (g_abs * lost * za * (1 + amp[:, None])).sum(0) + \
            (M + n) * U32 * (g_abs * gh.abs() * za).sum(0)
    else:
        e_do = g_abs * lost
        e_gate = scale * (lost * oabs).sum(1)
    check(got[1], grads[0], rounded(grads[0], e_do), "do")
    if gate is not None:
        check(got[2], grads[1], e_gate, "dgate")
    else:
        assert got[2] is None
    if wp is not None:
        check(got[3], grads[-1], e_wp, "dw_post")
    else:
        assert got[3] is None


def test_norm_gradients_against_differences(moe):
    """The gradients against central differences of the fp64 form, along a
    direction in all inputs at once."""
    note("norm differences")
    M, K, topk, scale, eps = 6, 256, 2, 0.5, 1e-4
    h, o, gate, wp, wn = norm_inputs(M, K, topk, "all", torch.float32, 50)
    gh, gu = f32((M, K), 60), bf16((M, K), 61)
    ho, u, r1, r2 = moe.moe_block_norm(h, o, gate, wp, wn, topk=topk, res_scale=scale, eps=eps)
    dh, do, dg, dwp, dwn = moe.moe_block_norm_bwd(gh, gu, ho, o, gate, wp, wn, r1, r2, topk=topk,
                                                  res_scale=scale)
    ins = [t.double() for t in (h, o, gate, wp, wn)]
    dirs = [torch.randn(t.shape, generator=torch.Generator().manual_seed(70 + i),
                        dtype=torch.float64).cuda() for i, t in enumerate(ins)]

    def loss(t):
        a, b, _, _ = block_norm(*[x + t * v for x, v in zip(ins, dirs)], topk, scale, eps)
        return ((a * gh.double()).sum() + (b * gu.double()).sum()).item()
    step = 1e-5
    num = (loss(step) - loss(-step)) / (2 * step)
    do_all = do.double().repeat_interleave(topk, 0)
    parts = [(x.double() * v) for x, v in zip((dh, do_all, dg, dwp, dwn), dirs)]
    ana = sum(p.sum().item() for p in parts)
    # half a bf16 step of do's terms, fp32 sums elsewhere, the differences' own
    # step^2 error and rounding (1e-6 of the terms covers both)
    tol = U16 * parts[1].abs().sum().item() + 1e-6 * sum(p.abs().sum().item() for p in parts)
    assert abs(ana - num) <= tol, (ana, num, tol)


def test_norm_in_place_and_empty(moe):
    note("norm in place")
    for K in (256, 333, 16392):
        h, o, gate, wp, wn = norm_inputs(5, K, 2, "all", torch.bfloat16, 80)
        a = moe.moe_block_norm(h, o, gate, wp, wn, topk=2)
        hh = h.clone()
        b = moe.moe_block_norm(hh, o, gate, wp, wn, topk=2, out=hh)
        assert b[0] is hh
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    h, o, gate, wp, wn = norm_inputs(3, 64, 2, "all", torch.float32, 81)
    ho, u, r1, r2 = moe.moe_block_norm(h[:0], o[:0], gate[:0], wp, wn, topk=2)
    assert ho.shape == (0, 64) and u.shape == (0, 64)
    got = moe.moe_block_norm_bwd(h[:0], o[:0], ho, o[:0], gate[:0], wp, wn, r1, r2, topk=2, du_topk=2)
    assert not got[3].any() and not got[4].any()
    # a row of zeros: finite, no gradient out of nothing
    z = torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda")
    ho, u, r1, r2 = moe.moe_block_norm(z, torch.cat((z, z)), None, wp, wn, topk=2)
    assert not ho.any() and not u.any() and torch.isfinite(r1).all()


def test_norm_same_bits_every_time(moe):
    note("norm determinism")
    h, o, gate, wp, wn = norm_inputs(1500, 512, 2, "all", torch.bfloat16, 90)
    ho, u, r1, r2 = moe.moe_block_norm(h, o, gate, wp, wn, topk=2)
    args = (h, u, ho, o, gate, wp, wn, r1, r2)
    first = moe.moe_block_norm_bwd(*args, topk=2)
    for _ in range(4):
        for a, b in zip(first, moe.moe_block_norm_bwd(*args, topk=2)):
            assert torch.equal(a, b)


def test_norm_refusals(moe):
    h, o, gate, wp, wn = norm_inputs(4, 64, 2, "all", torch.bfloat16, 95)
    f, b = moe.moe_block_norm, moe.moe_block_norm_bwd
    r = torch.ones(4, device="cuda")
    for call in (lambda: f(h), lambda: f(h.half(), w_pre=wn), lambda: f(h, o, gate, wp, wn),
                 lambda: f(h, o, gate.to(torch.bfloat16), wp, wn, topk=2),
                 lambda: f(h, o, gate[:3], wp, wn, topk=2), lambda: f(h, o, gate, wp[:32], wn, topk=2),
                 lambda: f(h, None, gate, None, wn), lambda: f(h, None, None, wp, wn),
                 lambda: f(h, o, gate, wp, wn, topk=2, out=h.float()),
                 lambda: f(h.t().contiguous().t(), o, gate, wp, wn, topk=2),
                 lambda: b(h, None, h, o, gate, wp, wn, r, r, topk=2),
                 lambda: b(h, h, h, o, gate, wp, wn, None, r, topk=2),
                 lambda: b(h, h, h, o, gate, wp, wn, r, None, topk=2),
                 lambda: b(h.float(), h, h, o, gate, wp, wn, r, r, topk=2),
                 lambda: b(None, None, h, o, gate, wp, None, r, None, topk=2),
                 lambda: b(h, h, h, o, gate, wp, wn, r, r, topk=2, du_topk=2)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(moe.MoEError):
        f(h, o, gate, wp, wn, topk=2, eps=0.0)
