"""A block of the network put together from the pieces, forward and backward,
as a training step runs it; and the same step captured into a graph.

The step keeps its intermediate rows in bf16, so its results differ from the
fp64 step on the same inputs and the same routing by a few roundings of half
a bf16 step each.  In the 2-norm a rounding changes a tensor by at most 2^-8 of
itself; a tensor passes at most 8 of them, each carried on by linear maps of
random weights (which neither stretch nor shrink on average) and by norms and
activations whose derivatives are below 1.2: 8 * 1.2^2 * 2^-8 = 0.045.
"""
import pytest
import torch

from tests._train_ref import bf16, block_norm, f32

pytestmark = pytest.mark.gpu

TOL = 8 * 1.2 ** 2 * 2.0 ** -8
SCALE, EPS = 0.5, 1e-5


@pytest.fixture(scope="module")
def moe():
    import moe_layer_04_amd as m
    m.load_library()
    return m


def inputs(T, K, N, E, h_dtype, seed):
    return {
        "h": f32((T, K), seed, 1.0).to(h_dtype), "wr": bf16((E, K), seed + 1, K ** -0.5),
        "w1": bf16((E, 2 * N, K), seed + 2, K ** -0.5), "w2": bf16((E, K, N), seed + 3, N ** -0.5),
        "gate": f32((T,), seed + 4, 0.3, 1.0), "w_in": f32((K,), seed + 5, 0.1, 1.0),
        "w_post": f32((K,), seed + 6, 0.1, 1.0), "w_pre": f32((K,), seed + 7, 0.1, 1.0),
        "dh": f32((T, K), seed + 8, 0.1).to(h_dtype), "du": bf16((T, K), seed + 9, 0.1),
    }


def forward(moe, s, topk, block_m):
    E = s["w1"].shape[0]
    T = s["h"].shape[0]
    f = dict(s)
    _, f["x"], _, f["r0"] = moe.moe_block_norm(s["h"], w_pre=s["w_in"], eps=EPS)
    f["ids"], f["wts"], _ = moe.moe_topk(f["x"], s["wr"], None, topk)
    f["sorted"], _, f["off"], f["num"] = moe.moe_align(f["ids"], E, block_m)
    f["g"] = moe.moe_grouped_gemm(f["x"], s["w1"], f["off"], sorted_ids=f["sorted"], topk=topk,
                                  gather=True)
    f["a"] = moe.moe_silu_mul(f["g"], f["wts"], sorted_ids=f["sorted"], num_rows=f["num"])
    f["o"] = moe.moe_grouped_gemm(f["a"], s["w2"], f["off"], sorted_ids=f["sorted"], topk=topk,
                                  num_tokens=T, scatter=True)
    f["ho"], f["u"], f["r1"], f["r2"] = moe.moe_block_norm(
        s["h"], f["o"], s["gate"], s["w_post"], s["w_pre"], topk=topk, res_scale=SCALE, eps=EPS)
    return f


def backward(moe, f, topk):
    T = f["h"].shape[0]
    rows = dict(sorted_ids=f["sorted"], topk=topk, num_tokens=T)
    g = {}
    dh, do, g["gate"], g["w_post"], g["w_pre"] = moe.moe_block_norm_bwd(
        f["dh"], f["du"], f["ho"], f["o"], f["gate"], f["w_post"], f["w_pre"], f["r1"], f["r2"],
        topk=topk, res_scale=SCALE)
    da = f["da"] = moe.moe_grouped_gemm_dx(do, f["w2"], f["off"], gather=True, **rows)
    g["w2"] = moe.moe_grouped_gemm_dw(do, f["a"], f["off"], gather_dy=True, **rows)
    dg, g["wts"] = moe.moe_silu_mul_bwd(da, f["g"], f["wts"], sorted_ids=f["sorted"],
                                        num_rows=f["num"])
    dx = moe.moe_grouped_gemm_dx(dg, f["w1"], f["off"], scatter=True, **rows)
    g["w1"] = moe.moe_grouped_gemm_dw(dg, f["x"], f["off"], gather_x=True,
                                      out_dtype=torch.float32, **rows)
    g["h"], _, _, _, g["w_in"] = moe.moe_block_norm_bwd(dh, dx, f["h"], w_pre=f["w_in"],
                                                        rstd_pre=f["r0"], du_topk=topk)
    return g


def reference(f, topk):
    """The step in fp64 with the step's own routing: (outputs, gradients)."""
    names = ("h", "w1", "w2", "gate", "w_in", "w_post", "w_pre", "wts")
    p = {k: f[k].double().requires_grad_() for k in names}
    T, K = p["h"].shape
    ids = f["ids"].long()
    _, x, _, _ = block_norm(p["h"], None, None, None, p["w_in"], 1, 1.0, EPS)
    o = torch.zeros((T, K), dtype=torch.float64, device="cuda")
    for e in range(p["w1"].shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        g = x[t] @ p["w1"][e].t()
        N = g.shape[1] // 2
        a = p["wts"][t, j, None] * torch.nn.functional.silu(g[:, :N]) * g[:, N:]
        o = o.index_add(0, t, a @ p["w2"][e].t())
    ho, u, _, _ = block_norm(p["h"], o, p["gate"], p["w_post"], p["w_pre"], 1, SCALE, EPS)
    grads = torch.autograd.grad((ho, u), [p[k] for k in names], (f["dh"].double(), f["du"].double()))
    return {"ho": ho, "u": u}, dict(zip(names, grads))


def off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


CASES = [
    # T, K, N, E, topk, block_m, stream
    (1, 256, 128, 4, 2, 1, torch.bfloat16),
    (24, 256, 384, 8, 2, 16, torch.bfloat16),
    (77, 136, 72, 5, 3, 1, torch.float32),
    (40, 133, 65, 3, 1, 1, torch.float32),
    (700, 512, 256, 4, 2, 1, torch.bfloat16),
    (520, 384, 320, 6, 4, 128, torch.float32),
]


@pytest.mark.parametrize("case", CASES, ids=[str(c[:6]) for c in CASES])
def test_step(moe, case):
    T, K, N, E, topk, bm, dt = case
    print(f"[gpu-test] step {case}", flush=True)
    s = inputs(T, K, N, E, dt, 100)
    f = forward(moe, s, topk, bm)
    g = backward(moe, f, topk)
    torch.cuda.synchronize()
    out, want = reference(f, topk)
    for k in ("ho", "u"):
        assert off(f[k], out[k]) <= TOL, k
    for k, v in want.items():
        assert torch.isfinite(g[k]).all(), k
        size = v.norm()
        if k == "wts" and topk == 1:
            # One slot a token: rms(w y) = w rms(y), so the norm after the
            # block takes the weight w out again and its gradient sum_n da_n
            # (a_n / w) is zero but for eps, a sum whose terms cancel.  The
            # roundings act on the terms: |da| |a / w| a token.
            size = (f["da"].double().norm(dim=1) * f["a"].double().norm(dim=1) /
                    f["wts"].double().view(-1)[f["sorted"].long()]).norm()
        assert ((g[k].double() - v).norm() / size).item() <= TOL, k


def test_pieces_agree_with_the_fused_layer(moe):
    """The pieces' forward against moe_fused_forward on the same tokens,
    within that call's tolerance."""
    print("[gpu-test] pieces against the fused layer", flush=True)
    for T in (4, 300):
        s = inputs(T, 512, 256, 8, torch.bfloat16, 7)
        f = forward(moe, s, 2, 1)
        fused = moe.moe_fused_forward(f["x"], s["wr"], None, s["w1"], s["w2"], 2).double()
        mine = f["o"].double().view(T, 2, -1).sum(1)
        err = (mine - fused).abs().amax(1) / fused.abs().amax(1)
        assert err.max().item() <= 2e-2


@pytest.mark.parametrize("T,bm", [(6, 1), (300, 1), (200, 64)])
def test_step_in_a_graph(moe, T, bm):
    """The whole step captured once and replayed on new inputs, with eager
    work between the replays: the eager step's bits every time."""
    print(f"[gpu-test] step graph T={T}", flush=True)
    K, N, E, topk = 256, 192, 4, 2
    s = inputs(T, K, N, E, torch.bfloat16, 300)
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
        new = inputs(T, K, N, E, torch.bfloat16, 400 + 20 * rep)
        for k in s:
            s[k].copy_(new[k])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        keep = {k: v.clone() for k, v in g.items()}
        keep.update({k: f[k].clone() for k in ("ho", "u")})
        ef = forward(moe, s, topk, bm)
        eg = backward(moe, ef, topk)
        eg.update({k: ef[k] for k in ("ho", "u")})
        torch.cuda.synchronize()
        for k, v in eg.items():
            assert torch.equal(keep[k], v), (rep, k)
