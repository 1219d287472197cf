"""What is measured of the operators around the experts of an MoE layer.

A case is one call (or, for the activation and the norms, one forward or one
backward call) of an operator:

  gemm      y[i] = W[e(i)] x[i], matrix products grouped by expert: row i of
            the expert-sorted rows belongs to the expert whose range
            [offsets[e], offsets[e+1]) holds it
  gemm_dx   dx[i] = W[e(i)]^T dy[i]
  gemm_dw   dW[e] = sum of dy[i] x[i]^T over the rows of expert e
  silu      a[i] = w[i] silu(g[i]) u[i] between the two products (forward), or
            its gradients with respect to g, u and the routing weight w
  norm      the norm after a block, its gate and residual scale and the norm
            before the next block: h' = h + s gate[t] rms(sum_j o[t,j]) w_post,
            u = rms(h') w_pre (forward), or all its gradients

`rows` says how a product takes its rows: "plain" (sorted rows in, sorted rows
out), "gather" (input row i is the token of slot sorted_ids[i]) or "scatter"
(output row goes to slot sorted_ids[i]).  The plain forms work on rows padded
to the longest expert, in fp32.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _gemm(name, op, T, k, E, K, N, rows, out="bf16", skew=0.5):
    """T tokens, k experts a token, E experts, W [E,N,K]; skew: variance of
    the per-expert bias of the routing logits."""
    return {"name": name, "op": op, "T": T, "topk": k, "E": E, "K": K, "N": N, "rows": rows,
            "out": out, "skew": skew}


def listed():
    return [
        # one token of a two-of-sixteen layer, its gate+up product: streaming
        # two experts' weights, the smallest serving call
        _gemm("up, one token", "gemm", 1, 2, 16, 4096, 16384, "gather"),
        # a decode batch of eight sequences, gate+up of eight experts
        _gemm("up, decode batch", "gemm", 8, 2, 8, 4096, 28672, "gather"),
        # 128 sequences over 256 small experts, the down product, about four
        # rows an expert
        _gemm("down, many experts", "gemm", 128, 8, 256, 2048, 7168, "scatter"),
        # a prompt batch of 4096 tokens, skewed routing: the largest forward
        _gemm("up, prompt batch", "gemm", 4096, 2, 8, 4096, 28672, "gather"),
        # the gradient of the activation rows from the layer's output
        # gradient, a training step of the same batch
        _gemm("down dx, training batch", "gemm_dx", 4096, 2, 8, 14336, 4096, "gather"),
        # a small layer of widths that fill no tile, a ragged micro-batch
        _gemm("up dx, odd widths", "gemm_dx", 203, 2, 7, 330, 1001, "scatter"),
        # the gradient of the gate+up weights in a training step
        _gemm("up dw, training batch", "gemm_dw", 4096, 2, 8, 4096, 28672, "gather"),
        # a small layer's gradient, kept in fp32 for accumulation over
        # micro-batches
        _gemm("up dw, small fp32", "gemm_dw", 333, 2, 8, 256, 1032, "gather", out="fp32"),
        # the activation between the products, decode
        {"name": "act, decode batch", "op": "silu", "T": 8, "topk": 2, "N": 14336, "back": False},
        # and its backward in a training step
        {"name": "act backward, training batch", "op": "silu", "T": 4096, "topk": 2, "N": 14336,
         "back": True},
        # around the layer: decode, bf16 residual stream
        {"name": "norms, decode batch", "op": "norm", "T": 8, "topk": 2, "K": 4096, "h": "bf16",
         "back": False},
        # and in a training step with an fp32 residual stream
        {"name": "norms backward, training batch", "op": "norm", "T": 4096, "topk": 2, "K": 4096,
         "h": "fp32", "back": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: mostly a multiple of 64 or 8, sometimes any."""
    v = _log(rng, lo, hi)
    r = rng.random()
    unit = 64 if r < 0.55 else 8 if r < 0.85 else 1
    return max(unit, v // unit * unit)


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gemm_dx", "gemm_dw", "silu", "norm"])
    T = _log(rng, 1, 4096)
    if op == "silu":
        return {"op": op, "T": T, "topk": rng.randint(1, 8) if T <= 1024 else rng.randint(1, 2),
                "N": _width(rng, 64, 14336), "back": rng.random() < 0.5}
    if op == "norm":
        return {"op": op, "T": T, "topk": rng.randint(1, 8) if T <= 1024 else rng.randint(1, 2),
                "K": _width(rng, 64, 4096 if T > 1024 else 8192), "h": rng.choice(["bf16", "fp32"]),
                "back": rng.random() < 0.5}
    E = _log(rng, 1, 256)
    k = rng.randint(1, min(E, 8))
    while True:
        K, N = _width(rng, 64, 14336), _width(rng, 64, 28672)
        t = T
        # at most the largest listed case's products and weights
        if E * N * K <= 1 << 30 and t * k * N * K <= 1 << 39 and t * k * max(N, K) <= 1 << 27:
            break
        T = max(1, T * 3 // 4)
    return {"op": op, "T": T, "topk": k, "E": E, "K": K, "N": N,
            "rows": rng.choice(["plain", "gather", "scatter"]) if op != "gemm_dw"
            else rng.choice(["plain", "gather"]),
            "out": rng.choice(["bf16", "fp32"]) if op == "gemm_dw" else "bf16",
            "skew": rng.choice([0.0, 0.5, 2.0])}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _route(case, gen, dev):
    """Top-k experts of random logits, and the expert-sorted slots."""
    T, k, E = case["T"], case["topk"], case["E"]
    logits = torch.randn((T, E), generator=gen, device=dev)
    logits += math.sqrt(case["skew"]) * torch.randn((1, E), generator=gen, device=dev)
    ids = logits.topk(k, dim=1).indices.reshape(-1)
    order = torch.sort(ids, stable=True)[1]
    counts = torch.bincount(ids, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    offsets[1:] = counts.cumsum(0)
    return order.to(torch.int32), offsets, int(counts.max())


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def rand(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device=dev).mul_(std).to(dtype)

    s = dict(case)
    T, k = case["T"], case["topk"]
    R = T * k
    if case["op"].startswith("gemm"):
        E, K, N = case["E"], case["K"], case["N"]
        s["sorted_ids"], s["offsets"], s["most"] = _route(case, gen, dev)
        gather = case["rows"] == "gather"
        if case["op"] != "gemm_dw":
            w = torch.empty((E, N, K), dtype=torch.bfloat16, device=dev)
            for e in range(E):
                w[e] = torch.randn((N, K), generator=gen, device=dev).mul_(1 / math.sqrt(K))
            s["w"] = w
        if case["op"] == "gemm":
            s["x"] = rand(T if gather else R, K)
        elif case["op"] == "gemm_dx":
            s["dy"] = rand(T if gather else R, N, std=0.01)
        else:
            s["x"], s["dy"] = rand(T if gather else R, K), rand(R, N, std=0.01)
    elif case["op"] == "silu":
        N = case["N"]
        s["g"] = rand(R, 2 * N)
        w = torch.rand((T, k), generator=gen, device=dev) + 0.1
        s["weights"] = w / w.sum(1, keepdim=True)
        s["sorted_ids"] = torch.randperm(R, generator=gen, device=dev).to(torch.int32)
        if case["back"]:
            s["da"] = rand(R, N, std=0.01)
    else:
        K = case["K"]
        s["o"] = rand(R, K)
        s["gate"] = torch.rand(T, generator=gen, device=dev)
        s["w_post"] = 1 + rand(K, std=0.1, dtype=torch.float32)
        s["w_pre"] = 1 + rand(K, std=0.1, dtype=torch.float32)
        s["scale"] = 0.5
        if not case["back"]:
            s["h"] = rand(T, K, std=2.0, dtype=DT[case["h"]])
        else:
            s["h_out"] = rand(T, K, std=2.0, dtype=DT[case["h"]])
            s["dh_out"] = rand(T, K, std=0.01, dtype=DT[case["h"]])
            s["du"] = rand(R, K, std=0.01)

            def rstd(v):
                return (v.square().mean(1) + EPS).rsqrt().float()

            # what the forward call of the same step left
            s["rstd_post"] = rstd(s["o"].double().view(T, k, K).sum(1))
            s["rstd_pre"] = rstd(s["h_out"].double())
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def _pad(rows, where, shape):
    """Sorted rows laid out [expert, place, width] in fp32, zeros elsewhere."""
    p = torch.zeros(shape + rows.shape[1:], dtype=torch.float32, device=rows.device)
    p[where] = rows.float()
    return p


def _plain_gemm(s):
    off, slots, E = s["offsets"], s["sorted_ids"].long(), s["E"]
    i = torch.arange(slots.numel(), device=off.device)
    e = torch.bucketize(i, off[1:].long(), right=True)
    where = (e, i - off.long()[e])
    shape = (E, s["most"])
    gather = s["rows"] == "gather"
    tokens = slots // s["topk"]
    if s["op"] == "gemm_dw":
        x = s["x"][tokens] if gather else s["x"]
        d = torch.bmm(_pad(s["dy"], where, shape).transpose(1, 2), _pad(x, where, shape))
        return d.to(DT[s["out"]])
    rows = s["x"] if s["op"] == "gemm" else s["dy"]
    w = s["w"].float()
    if s["op"] == "gemm":
        w = w.transpose(1, 2)
    y = torch.bmm(_pad(rows[tokens] if gather else rows, where, shape), w)[where]
    y = y.to(torch.bfloat16)
    if s["rows"] == "scatter":
        out = torch.empty_like(y)
        out[slots] = y
        return out
    return y


def _plain_silu(s):
    N = s["N"]
    g, u = s["g"][:, :N].float(), s["g"][:, N:].float()
    w = s["weights"].reshape(-1)[s["sorted_ids"].long()].unsqueeze(1)
    sig = 1 / (1 + torch.exp(-g))
    if not s["back"]:
        return (w * g * sig * u).to(torch.bfloat16)
    da = s["da"].float()
    dg = da * w * u * sig * (1 + g * (1 - sig))
    du = da * w * g * sig
    dw = torch.empty_like(s["weights"]).reshape(-1)
    dw[s["sorted_ids"].long()] = (da * g * sig * u).sum(1)
    return {"dg": torch.cat((dg, du), 1).to(torch.bfloat16), "dw": dw.view(s["T"], s["topk"])}


def _plain_norm(s):
    T, k, K = s["T"], s["topk"], s["K"]
    o = s["o"].float().view(T, k, K).sum(1)
    gate = s["gate"].unsqueeze(1) * s["scale"]
    if not s["back"]:
        r1 = torch.rsqrt(o.square().mean(1) + EPS)
        h = s["h"].float() + gate * (o * r1.unsqueeze(1)) * s["w_post"]
        # what the next block normalises is the stream as it is kept
        h = h.to(s["h"].dtype)
        f = h.float()
        r2 = torch.rsqrt(f.square().mean(1) + EPS)
        return {"h": h, "u": (f * r2.unsqueeze(1) * s["w_pre"]).to(torch.bfloat16),
                "rstd_post": r1, "rstd_pre": r2}
    r1, r2 = s["rstd_post"].unsqueeze(1), s["rstd_pre"].unsqueeze(1)
    du = s["du"].float().view(T, k, K).sum(1)
    n = s["h_out"].float() * r2
    c = du * s["w_pre"]
    dh = s["dh_out"].float() + r2 * (c - n * (c * n).mean(1, keepdim=True))
    z = o * r1
    b = dh * s["w_post"]
    do = gate * r1 * (b - z * (b * z).mean(1, keepdim=True))
    return {"dh": dh.to(s["h_out"].dtype), "do": do.to(torch.bfloat16),
            "dgate": s["scale"] * (b * z).sum(1), "dw_post": (gate * dh * z).sum(0),
            "dw_pre": (du * n).sum(0)}


def run(s):
    op = s["op"]
    if own:
        import moe_layer_04_amd as moe
        if op == "silu":
            if not s["back"]:
                return moe.moe_silu_mul(s["g"], s["weights"], sorted_ids=s["sorted_ids"])
            dg, dw = moe.moe_silu_mul_bwd(s["da"], s["g"], s["weights"],
                                          sorted_ids=s["sorted_ids"])
            return {"dg": dg, "dw": dw}
        if op == "norm":
            if not s["back"]:
                h, u, r1, r2 = moe.moe_block_norm(
                    s["h"], s["o"], s["gate"], s["w_post"], s["w_pre"], topk=s["topk"],
                    res_scale=s["scale"], eps=EPS)
                return {"h": h, "u": u, "rstd_post": r1, "rstd_pre": r2}
            dh, do, dgate, dw1, dw2 = moe.moe_block_norm_bwd(
                s["dh_out"], s["du"], s["h_out"], s["o"], s["gate"], s["w_post"], s["w_pre"],
                s["rstd_post"], s["rstd_pre"], topk=s["topk"], du_topk=s["topk"],
                res_scale=s["scale"])
            return {"dh": dh, "do": do, "dgate": dgate, "dw_post": dw1, "dw_pre": dw2}
        gather, scatter = s["rows"] == "gather", s["rows"] == "scatter"
        if op == "gemm_dw":
            return moe.moe_grouped_gemm_dw(s["dy"], s["x"], s["offsets"],
                                           sorted_ids=s["sorted_ids"] if gather else None,
                                           topk=s["topk"], gather_x=gather,
                                           out_dtype=DT[s["out"]])
        call = moe.moe_grouped_gemm if op == "gemm" else moe.moe_grouped_gemm_dx
        return call(s["x"] if op == "gemm" else s["dy"], s["w"], s["offsets"],
                    sorted_ids=s["sorted_ids"] if gather or scatter else None, topk=s["topk"],
                    num_tokens=s["T"], gather=gather, scatter=scatter)
    if op == "silu":
        return _plain_silu(s)
    if op == "norm":
        return _plain_norm(s)
    return _plain_gemm(s)


# --------------------------------------------------------------------------
# the work of a pass, and its result in 64 bits
# --------------------------------------------------------------------------

def work(case):
    T, k, op = case["T"], case["topk"], case["op"]
    R = T * k
    if op == "silu":
        N = case["N"]
        if not case["back"]:
            return {"bytes": R * N * 6 + R * 8, "flops": R * N * 6}
        return {"bytes": R * N * 10 + R * 12, "flops": R * N * 14}
    if op == "norm":
        K, hb = case["K"], 2 if case["h"] == "bf16" else 4
        if not case["back"]:
            return {"bytes": T * K * (2 * hb + 2 * k + 2) + 8 * K + 12 * T,
                    "flops": T * K * (k + 10)}
        return {"bytes": T * K * (3 * hb + 4 * k + 2) + 16 * K + 16 * T,
                "flops": T * K * (2 * k + 24)}
    E, K, N = case["E"], case["K"], case["N"]
    # weights of as many experts as R independent picks reach on average
    # (all, for the weight gradient)
    seen = E * (1 - (1 - k / E) ** T)
    src = T if case["rows"] == "gather" else R
    ids = 4 * (E + 1) + (0 if case["rows"] == "plain" else 4 * R)
    if op == "gemm_dw":
        return {"bytes": 2 * R * N + 2 * src * K + E * N * K * (2 if case["out"] == "bf16" else 4)
                + ids, "flops": 2 * R * N * K}
    read, write = (K, N) if op == "gemm" else (N, K)
    return {"bytes": int(2 * seen * N * K) + 2 * src * read + 2 * R * write + ids,
            "flops": 2 * R * N * K}


def exact(case, seed):
    s = prepare(case, seed)
    T, k, op = case["T"], case["topk"], case["op"]
    R = T * k
    if op == "silu":
        N = case["N"]
        gu = s["g"].double()
        g, u = gu[:, :N], gu[:, N:]
        slots = s["sorted_ids"].long()
        w = s["weights"].double().reshape(R)[slots][:, None]
        sg = torch.sigmoid(g)
        act = g * sg
        if not case["back"]:
            return w * act * u
        da = s["da"].double()
        dw = torch.zeros(R, dtype=torch.float64, device=g.device)
        dw[slots] = (da * act * u).sum(1)
        slope = sg + act * (1 - sg)
        return {"dg": torch.cat([da * w * u * slope, da * w * act], 1), "dw": dw.reshape(T, k)}
    if op == "norm":
        K = case["K"]
        o = s["o"].double().reshape(T, k, K).sum(1)
        wp, wn = s["w_post"].double(), s["w_pre"].double()
        gt = s["gate"].double()[:, None]
        sc = s["scale"]
        if not case["back"]:
            r1 = 1 / torch.sqrt((o * o).sum(1) / K + EPS)
            h = s["h"].double() + sc * gt * o * r1[:, None] * wp
            # the next block normalises the stream as it is kept
            kept = h.to(DT[case["h"]]).double()
            r2 = 1 / torch.sqrt((kept * kept).sum(1) / K + EPS)
            return {"h": h, "u": kept * r2[:, None] * wn, "rstd_post": r1, "rstd_pre": r2}
        r1, r2 = s["rstd_post"].double()[:, None], s["rstd_pre"].double()[:, None]
        du = s["du"].double().reshape(T, k, K).sum(1)
        n, z = s["h_out"].double() * r2, o * r1
        dn = du * wn
        dh = s["dh_out"].double() + r2 * dn - r2 * n * (dn * n).sum(1, keepdim=True) / K
        dz = dh * sc * gt * wp
        return {"dh": dh, "do": r1 * dz - r1 * z * (dz * z).sum(1, keepdim=True) / K,
                "dgate": (dh * sc * z * wp).sum(1), "dw_post": (dh * sc * gt * z).sum(0),
                "dw_pre": (du * n).sum(0)}
    E, K, N = case["E"], case["K"], case["N"]
    bounds = s["offsets"].tolist()
    slots = s["sorted_ids"].long()
    pick = (lambda t, a, b: t[slots[a:b] // k]) if case["rows"] == "gather" else \
        (lambda t, a, b: t[a:b])
    if op == "gemm_dw":
        out = torch.zeros((E, N, K), dtype=torch.float64, device=slots.device)
        for e in range(E):
            a, b = bounds[e], bounds[e + 1]
            if b > a:
                out[e] = s["dy"][a:b].double().t() @ pick(s["x"], a, b).double()
        return out
    out = torch.zeros((R, N if op == "gemm" else K), dtype=torch.float64, device=slots.device)
    for e in range(E):
        a, b = bounds[e], bounds[e + 1]
        if b == a:
            continue
        w = s["w"][e].double()
        y = pick(s["x"], a, b).double() @ w.t() if op == "gemm" else pick(s["dy"], a, b).double() @ w
        if case["rows"] == "scatter":
            out[slots[a:b]] = y
        else:
            out[a:b] = y
    return out
