"""A training step of a block with its router: the balance loss, the router's
gradients and activations kept in 8 bits, put together as they are used, against
the same step in fp64; captured into a graph; and what is kept against what it
replaces.

The fp64 step takes the routing of the step it is compared with, and in its
backward pass the values that the step kept (the gate and up rows and the block's
input), so what is left is roundings: as in test_gpu_train_step.py a tensor
passes at most 8 of them, 2^-8 of itself each, with maps that stretch by at most
1.2^2.  The router's gradients pass two more, of the rows that reach the tokens and
of their sum.
"""
import pytest
import torch

from tests._ckpt_ref import keep, keep_halves
from tests._train_ref import bf16, block_norm, f32

pytestmark = pytest.mark.gpu

TOL = 10 * 1.2 ** 2 * 2.0 ** -8
SCALE, EPS = 0.5, 1e-5


@pytest.fixture(scope="module")
def moe():
    import moe_layer_04_amd as m
    m.load_library()
    return m


def inputs(T, K, N, E, seed):
    g = torch.Generator().manual_seed(seed)
    return {
        "h": f32((T, K), seed, 1.0), "wr": bf16((E, K), seed + 1, K ** -0.5), "bias": f32((E,), seed + 2, 0.3),
        "w1": bf16((E, 2 * N, K), seed + 3, K ** -0.5), "w2": bf16((E, K, N), seed + 4, N ** -0.5),
        "w_in": f32((K,), seed + 5, 0.1, 1.0), "dh": f32((T, K), seed + 6, 0.1),
        "coef": f32((1,), seed + 7, 0.1, 5.0), "mask": (torch.rand(T, generator=g) < 0.8).cuda(),
    }


def forward(moe, s, topk, block_m):
    E, T = s["w1"].shape[0], s["h"].shape[0]
    f = dict(s)
    _, f["x"], _, f["r0"] = moe.moe_block_norm(s["h"], w_pre=s["w_in"], eps=EPS)
    f["ids"], f["wts"], f["logits"] = moe.moe_topk(f["x"], s["wr"], s["bias"], topk)
    f["loss"], f["counts"], f["tokens"], _ = moe.moe_balance(f["logits"], f["ids"], token_mask=s["mask"])
    f["sorted"], _, f["off"], f["num"] = moe.moe_align(f["ids"], E, block_m)
    f["g"] = moe.moe_grouped_gemm(f["x"], s["w1"], f["off"], sorted_ids=f["sorted"], topk=topk, gather=True)
    f["a"], *f["kept_g"] = moe.moe_silu_mul_ckpt(f["g"], f["wts"], sorted_ids=f["sorted"], num_rows=f["num"])
    f["kept_x"] = moe.moe_ckpt_rows(f["x"])
    f["o"] = moe.moe_grouped_gemm(f["a"], s["w2"], f["off"], sorted_ids=f["sorted"], topk=topk,
                                  num_tokens=T, scatter=True)
    f["ho"], _, _, _ = moe.moe_block_norm(s["h"], f["o"], topk=topk, res_scale=SCALE, eps=EPS)
    return f


def backward(moe, f, topk):
    T = f["h"].shape[0]
    rows = dict(sorted_ids=f["sorted"], topk=topk, num_tokens=T)
    g = {}
    dh, do, _, _, _ = moe.moe_block_norm_bwd(f["dh"], None, f["ho"], f["o"], topk=topk, res_scale=SCALE)
    da = moe.moe_grouped_gemm_dx(do, f["w2"], f["off"], gather=True, **rows)
    dg, dwts, a = moe.moe_silu_mul_bwd_ckpt(da, *f["kept_g"], f["wts"], sorted_ids=f["sorted"], num_rows=f["num"])
    g["w2"] = moe.moe_grouped_gemm_dw(do, a, f["off"], gather_dy=True, **rows)
    g["w1"] = moe.moe_grouped_gemm_dw_ckpt(dg, *f["kept_x"], f["off"], gather_x=True, out_dtype=torch.float32, **rows)
    dxs = moe.moe_grouped_gemm_dx(dg, f["w1"], f["off"], scatter=True, **rows)
    dl = moe.moe_balance_bwd(f["coef"], f["logits"], f["counts"], f["tokens"], topk, token_mask=f["mask"])
    g["x"], g["wr"], g["bias"] = moe.moe_topk_bwd(f["x"], f["wr"], f["ids"], f["wts"], dwts, dlogits=dl,
                                                  dx_rows=dxs, bias=True)
    g["h"], _, _, _, g["w_in"] = moe.moe_block_norm_bwd(dh, g["x"], f["h"], w_pre=f["w_in"], rstd_pre=f["r0"])
    return g


class Product(torch.autograd.Function):
    """x w^T, whose weights' gradient takes the kept x"""
    @staticmethod
    def forward(ctx, x, w, kept):
        ctx.save_for_backward(w, kept)
        return x @ w.t()

    @staticmethod
    def backward(ctx, dy):
        w, kept = ctx.saved_tensors
        return dy @ w, dy.t() @ kept, None


class Gated(torch.autograd.Function):
    """wt silu(g) u, whose gradients are those at the kept g"""
    @staticmethod
    def forward(ctx, g, wt, kept):
        ctx.save_for_backward(wt, kept)
        N = g.shape[1] // 2
        return wt[:, None] * torch.nn.functional.silu(g[:, :N]) * g[:, N:]

    @staticmethod
    def backward(ctx, da):
        wt, kept = ctx.saved_tensors
        with torch.enable_grad():
            g, w = kept.clone().requires_grad_(), wt.clone().requires_grad_()
            N = g.shape[1] // 2
            y = w[:, None] * torch.nn.functional.silu(g[:, :N]) * g[:, N:]
            return (*torch.autograd.grad(y, (g, w), da), None)


def reference(f, topk):
    """The step in fp64 with the step's own routing and kept values."""
    names = ("h", "wr", "bias", "w1", "w2", "w_in")
    p = {k: f[k].double().requires_grad_() for k in names}
    T, K = p["h"].shape
    E = p["w1"].shape[0]
    ids = f["ids"].long()
    _, x, _, _ = block_norm(p["h"], None, None, None, p["w_in"], 1, 1.0, EPS)
    logits = x @ p["wr"].t() + p["bias"]
    wts = torch.softmax(logits.gather(1, ids), 1)
    n = int(f["mask"].sum())
    counts = torch.bincount(ids[f["mask"]].flatten(), minlength=E)
    share = counts.double() / (n * topk)
    balance = E * (share * torch.softmax(logits, 1)[f["mask"]].sum(0) / n).sum()
    kept_x = keep(f["x"])[2]
    slots = f["sorted"].long()
    place = torch.full((T * topk,), -1, dtype=torch.long, device="cuda")       # a slot's sorted row
    real = (slots >= 0) & (slots < T * topk)
    place[slots[real]] = torch.arange(slots.numel(), device="cuda")[real]
    kept_g = keep_halves(torch.where(real[:, None], f["g"], torch.zeros_like(f["g"])))[2]
    o = torch.zeros((T, K), dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        g = Product.apply(x[t], p["w1"][e], kept_x[t])
        kg = kept_g[place[t * topk + j]]
        N = g.shape[1] // 2
        a = Gated.apply(g, wts[t, j], kg)
        again = wts[t, j, None].detach() * torch.nn.functional.silu(kg[:, :N]) * kg[:, N:]
        o = o.index_add(0, t, Product.apply(a, p["w2"][e], again))
    ho = p["h"] + SCALE * o
    total = (ho * f["dh"].double()).sum() + f["coef"].double().sum() * balance
    return balance, ho, dict(zip(names, torch.autograd.grad(total, [p[k] for k in names])))


CASES = [  # T, K, N, E, topk, block_m
    (1, 64, 40, 4, 2, 1), (24, 256, 384, 8, 2, 16), (77, 136, 72, 5, 3, 1), (40, 133, 65, 3, 2, 1),
    (700, 512, 256, 4, 2, 1), (520, 384, 320, 70, 4, 1),
]


@pytest.mark.parametrize("case", CASES, ids=[str(c) for c in CASES])
def test_step(moe, case):
    T, K, N, E, topk, bm = case
    print(f"[gpu-test] router step {case}", flush=True)
    s = inputs(T, K, N, E, 500)
    s["mask"][0] = True
    f = forward(moe, s, topk, bm)
    g = backward(moe, f, topk)
    torch.cuda.synchronize()
    balance, ho, want = reference(f, topk)
    assert abs(f["loss"].double().item() - balance.item()) <= TOL * balance.item()
    assert ((f["ho"].double() - ho).norm() / ho.norm()).item() <= TOL
    for k, v in want.items():
        assert torch.isfinite(g[k]).all(), k
        assert ((g[k].double() - v).norm() / v.norm()).item() <= TOL, k


def test_what_is_kept_replaces_bf16(moe):
    """Gradients of kept activations against those of bf16 ones: kept values are
    off by 1/127 of their block's largest at most, so by 2^-7 sqrt(32) of a block's
    2-norm, which the derivatives (below 1.2 each, of two factors) carry on."""
    print("[gpu-test] kept against bf16", flush=True)
    R, N = 96, 320
    g, da, wt = bf16((R, 2 * N), 1), bf16((R, N), 2), f32((R,), 3, 0.2, 1.0)
    a, codes, scales = moe.moe_silu_mul_ckpt(g, wt)
    assert torch.equal(a, moe.moe_silu_mul(g, wt))
    dg, dw, again = moe.moe_silu_mul_bwd_ckpt(da, codes, scales, wt)
    wg, ww = moe.moe_silu_mul_bwd(da, g, wt)
    bound = 2 * 1.2 * 32 ** 0.5 / 127 + 2.0 ** -7
    for got, want in ((dg, wg), (dw, ww), (again, a)):
        off = (got.double() - want.double()).norm() / want.double().norm()
        assert 0 < off.item() <= bound


@pytest.mark.parametrize("T,bm", [(6, 1), (300, 1), (200, 64)])
def test_step_in_a_graph(moe, T, bm):
    """The whole step captured once and replayed on new inputs, with eager work
    between the replays: the eager step's bits every time."""
    print(f"[gpu-test] router step graph T={T}", flush=True)
    K, N, E, topk = 256, 192, 4, 2
    s = inputs(T, K, N, E, 600)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                    # loads every kernel
        backward(moe, forward(moe, s, topk, bm), topk)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = forward(moe, s, topk, bm)
        g = backward(moe, f, topk)
    for rep in range(4):
        new = inputs(T, K, N, E, 700 + 20 * rep)
        for k in s:
            s[k].copy_(new[k])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept = {k: v.clone() for k, v in g.items()}
        kept.update({k: f[k].clone() for k in ("ho", "loss", "counts")})
        ef = forward(moe, s, topk, bm)
        eg = backward(moe, ef, topk)
        eg.update({k: ef[k] for k in ("ho", "loss", "counts")})
        torch.cuda.synchronize()
        for k, v in eg.items():
            assert torch.equal(kept[k], v), (rep, k)
