"""Plain 64-bit forms of the operators around the experts, and helpers of
their tests.  Every form also returns, where asked, the sum of the magnitudes
of its terms: the scale of its fp32 rounding errors."""
import torch

U32 = 2.0 ** -24   # half a step of fp32, relative
U16 = 2.0 ** -8    # half a step of bf16, relative


def routing(T, topk, E, seed, skip=()):
    """Top-k ids [T,topk] without the experts in ``skip``, on the GPU."""
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn((T, E), generator=g)
    for e in skip:
        logits[:, e] = -1e9
    return logits.topk(topk, dim=1).indices.to(torch.int32).cuda()


def bf16(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).cuda()


def f32(shape, seed, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).cuda()


def read_rows(src, rows, sorted_ids, topk, slots, gather):
    """Rows of a (gathered) operand for the sorted rows ``rows``, in fp64;
    zeros where the slot says padding."""
    rows = torch.as_tensor(rows, device=src.device)
    if sorted_ids is None:
        return src[rows].double()
    p = sorted_ids[rows].long()
    ok = (p >= 0) & (p < slots)
    at = torch.where(ok, p // topk if gather else rows, torch.zeros_like(p))
    v = src[at].double() if src.shape[0] else torch.zeros((len(rows), src.shape[1]), device=src.device,
                                                          dtype=torch.float64)
    return torch.where(ok[:, None], v, torch.zeros_like(v))


def grouped_rows(src, w, offsets, sorted_ids, topk, T, gather, scatter, out, dx):
    """The rows product into a copy of ``out``: (result, magnitudes), fp64."""
    y = out.double().clone()
    mag = torch.zeros_like(y)
    off = offsets.tolist()
    for e in range(w.shape[0]):
        rows = range(off[e], off[e + 1])
        if len(rows) == 0:
            continue
        a = read_rows(src, list(rows), sorted_ids, topk, T * topk, gather)
        we = w[e].double() if dx else w[e].double().t().contiguous()
        v, m = a @ we, a.abs() @ we.abs()
        idx = torch.arange(off[e], off[e + 1], device=src.device)
        if scatter:
            p = sorted_ids[idx].long()
            ok = (p >= 0) & (p < T * topk)
            y[p[ok]], mag[p[ok]] = v[ok], m[ok]
        else:
            y[idx], mag[idx] = v, m
    return y, mag


def grouped_dw(dy, x, offsets, sorted_ids, topk, T, gather_dy, gather_x):
    off = offsets.tolist()
    E = len(off) - 1
    out = torch.zeros((E, dy.shape[1], x.shape[1]), dtype=torch.float64, device=dy.device)
    mag = torch.zeros_like(out)
    for e in range(E):
        rows = list(range(off[e], off[e + 1]))
        if rows:
            d = read_rows(dy, rows, sorted_ids, topk, T * topk, gather_dy).t().contiguous()
            v = read_rows(x, rows, sorted_ids, topk, T * topk, gather_x)
            out[e], mag[e] = d @ v, d.abs() @ v.abs()
    return out, mag


def check(got, want, bound, what=""):
    """|got - want| <= bound elementwise; both finite."""
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() - bound
    worst = over.max().item() if over.numel() else -1.0
    assert worst <= 0, f"{what}: over its bound by {worst:.3e} ({int((over > 0).sum())} values)"


def silu_mul(g, w):
    """(a, silu(gate) * up) in fp64; w per row."""
    N = g.shape[1] // 2
    z, u = g[:, :N].double(), g[:, N:].double()
    act = z * torch.sigmoid(z)
    return w[:, None] * act * u, act * u


def block_norm(h, o, gate, w_post, w_pre, topk, scale, eps, kept=None):
    """(h_out, u, rstd_post, rstd_pre) in the inputs' type (fp64 in the
    tests).  ``kept``: the stream as it was kept, which the second norm
    takes."""
    M, K = h.shape
    r1 = r2 = u = None
    if o is not None:
        s = o.reshape(M, topk, K).sum(1)
        if w_post is not None:
            r1 = (s.square().mean(1) + eps).rsqrt()
            s = s * r1[:, None] * w_post
        if gate is not None:
            s = s * gate[:, None]
        h = h + scale * s
    n = h if kept is None else kept
    if w_pre is not None:
        r2 = (n.square().mean(1) + eps).rsqrt()
        u = n * r2[:, None] * w_pre
    return h, u, r1, r2
