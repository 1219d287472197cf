"""The router's balance loss, its gradient and the gradients of moe_topk against
fp64.

Bounds, elementwise, in half steps of fp32 (U32) of the magnitudes that enter:

* a probability: e^d with d = l - max is off by 2 |d| + 4 (the difference and its
  product with log2 e, each half a step of |d|; the exponential itself), their
  sum by as much and 10 additions, the quotient by 2 more: 4 D + 24 with D the
  largest |d|.
* a sum over tokens adds at most 9 + M/1024 values in a lane, then 6 lanes, 4
  waves and 64 + 2 workgroups one after the other: 96 + M/1024.
* dl takes topk + 6 operations on |dlogits| + |w| (|dw| + sum |w dw|).
* products as in test_gpu_grouped.py; dx takes dl in two bf16 parts, off by at most
  2^-8 * 2^-8 of it.
"""
import pytest
import torch

from tests._train_ref import U16, U32, bf16, check, f32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import moe_layer_04_amd as m
    m.load_library()
    return m


def note(msg):
    print(f"[gpu-test] {msg}", flush=True)


def ints(shape, seed, most=3):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g).cuda()


# --------------------------------------------------------------------------
# the balance loss
# --------------------------------------------------------------------------

def softmax(l):
    """fp64, zeros for a row of -inf; and the largest finite |l - max| (the others
    are zeros)"""
    l = l.double()
    m = l.amax(1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    e = torch.exp(l - m)
    s = e.sum(1, keepdim=True)
    d = (l - m).abs()
    D = d[(e > 1e-40) & torch.isfinite(d)]
    return torch.where(s > 0, e / s, torch.zeros_like(e)), (D.max().item() if D.numel() else 0.0)


def balance(logits, ids, keep, E, topk):
    p, D = softmax(logits[keep])
    n = int(keep.sum())
    k = ids[keep].long().flatten()
    counts = torch.bincount(k[(k >= 0) & (k < E)], minlength=E)
    f = counts.double() / max(n * topk, 1)
    P = p.sum(0) / max(n, 1)
    return p, f, counts, n, P, E * (f * P).sum(), D


def grad(p, f, n, up, E):
    return up * E / max(n, 1) * p * (f - (p * f).sum(1, keepdim=True))


CASES = [  # M, E, topk
    (1, 1, 1), (1, 8, 2), (3, 2, 2), (7, 5, 3), (64, 8, 2), (33, 4, 1), (100, 60, 4), (257, 63, 6),
    (300, 64, 8), (1000, 65, 2), (2100, 8, 2), (1025, 128, 8), (777, 130, 16), (515, 255, 1),
    (700, 256, 8), (9000, 17, 3), (5000, 256, 8), (20000, 1, 1), (70000, 3, 2),
]


@pytest.mark.parametrize("M,E,topk", CASES)
@pytest.mark.parametrize("mask", [None, "most", "few", "none", "bytes"])
def test_balance(moe, M, E, topk, mask):
    note(f"balance M={M} E={E} topk={topk} mask={mask}")
    logits = f32((M, E), 1, 2.0) + f32((1, E), 2, 1.0)
    ids = logits.topk(topk, dim=1).indices.to(torch.int32)
    if M > 5:
        logits[M // 2] = float("-inf")            # a token without an expert
        logits[M // 3] = torch.finfo(torch.float32).min
        logits[M // 4, 0] = float("-inf")
        ids[M // 5, 0] = -1                       # a dropped slot
        ids[M // 6, topk - 1] = E
    token_mask, keep = None, torch.ones(M, dtype=torch.bool, device="cuda")
    if mask is not None:
        share = {"most": 0.9, "few": 0.05, "none": 0.0, "bytes": 0.5}[mask]
        keep = (torch.rand(M, generator=torch.Generator().manual_seed(3)) < share).cuda()
        logits[~keep] = float("nan")              # not read
        ids[~keep] = 1 << 30
        token_mask = keep.to(torch.uint8) * 255 if mask == "bytes" else keep
    p, f, counts, n, P, loss, D = balance(logits, ids, keep, E, topk)
    got = moe.moe_balance(logits, ids, token_mask=token_mask)
    assert torch.equal(got[1].long(), counts)
    assert got[2].tolist() == [n]
    off = (4 * D + 24 + 96 + M / 1024) * U32
    check(got[3], P, off * P, "probs")
    check(got[0], loss.view(1), (off + 16 * U32) * loss.view(1), "loss")

    up = torch.tensor([0.37], device="cuda")
    d = moe.moe_balance_bwd(up, logits, got[1], got[2], topk, token_mask=token_mask)
    want = torch.zeros((M, E), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(want)
    want[keep] = grad(p, f, n, 0.37, E)
    mag[keep] = 0.37 * E / max(n, 1) * p * (f + (p * f).sum(1, keepdim=True))
    check(d, want, (8 * D + 64) * U32 * mag + U32 * want.abs(), "dlogits")


def test_balance_without_tokens(moe):
    note("balance M=0")
    for E in (1, 8, 256):
        loss, counts, tokens, probs = moe.moe_balance(f32((0, E), 1), torch.empty((0, 1), dtype=torch.int32,
                                                                                  device="cuda"))
        assert loss.tolist() == [0] and tokens.tolist() == [0]
        assert (counts == 0).all() and (probs == 0).all()
        assert moe.moe_balance_bwd(loss, f32((0, E), 1), counts, tokens, 1).shape == (0, E)


def test_counts_of_several_batches(moe):
    """Counts and tokens summed over two batches give the gradient of the loss
    over both."""
    note("balance, two batches")
    E, topk = 24, 3
    logits = f32((500, E), 1, 2.0)
    ids = logits.topk(topk, dim=1).indices.to(torch.int32)
    up = torch.ones(1, device="cuda")
    _, counts, tokens, _ = moe.moe_balance(logits, ids)
    whole = moe.moe_balance_bwd(up, logits, counts, tokens, topk)
    parts = [(logits[:200].contiguous(), ids[:200].contiguous()), (logits[200:].contiguous(), ids[200:].contiguous())]
    seen = [moe.moe_balance(*p) for p in parts]
    c, n = seen[0][1] + seen[1][1], seen[0][2] + seen[1][2]
    assert torch.equal(c, counts) and torch.equal(n, tokens)
    got = torch.cat([moe.moe_balance_bwd(up, l, c, n, topk) for l, _ in parts])
    assert torch.equal(got, whole)


def test_balance_gradient_against_differences(moe):
    note("balance, differences")
    M, E, topk, h = 5, 12, 2, 1e-6
    logits = f32((M, E), 1, 1.0)
    ids = logits.topk(topk, dim=1).indices.to(torch.int32)
    _, counts, tokens, _ = moe.moe_balance(logits, ids)
    got = moe.moe_balance_bwd(torch.ones(1, device="cuda"), logits, counts, tokens, topk).double()
    f = counts.double() / (M * topk)
    for e in range(E):
        for t in range(M):
            step = torch.zeros((M, E), dtype=torch.float64, device="cuda")
            step[t, e] = h
            hi, lo = (E * (f * softmax(logits.double() + s)[0].mean(0)).sum() for s in (step, -step))
            # h^2/6 of a third derivative below E/M, and 2^-52 of the loss (about 1) over h
            assert abs(got[t, e] - (hi - lo) / (2 * h)) <= 1e-9 + 64 * U32 * E / M, (t, e)


# --------------------------------------------------------------------------
# moe_topk's gradients
# --------------------------------------------------------------------------

def inputs(M, K, E, topk, rows, weights, dl, seed):
    logits = f32((M, E), seed, 2.0)
    ids = logits.topk(topk, dim=1).indices.to(torch.int32)
    s = {"x": bf16((M, K), seed + 1), "w_router": bf16((E, K), seed + 2, K ** -0.5)}
    if weights:
        w = torch.softmax(logits.gather(1, ids.long()), 1)
        s.update(topk_ids=ids, topk_weights=w, dtopk_weights=f32((M, topk), seed + 3))
    s["dlogits"] = f32((M, E), seed + 4, 0.1) if dl else None
    s["dx_rows"] = bf16((M * rows, K), seed + 5) if rows else None
    return s


def reference(s):
    """dx, dw, dbias and the bounds of what is off"""
    x, w = s["x"].double(), s["w_router"].double()
    M, K = x.shape
    E = w.shape[0]
    dl = torch.zeros((M, E), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(dl)
    topk = 0
    if s["dlogits"] is not None:
        dl += s["dlogits"].double()
        mag += dl.abs()
    if s.get("topk_ids") is not None:
        ids, wt, dwt = s["topk_ids"].long(), s["topk_weights"].double(), s["dtopk_weights"].double()
        topk = ids.shape[1]
        mean, size = (wt * dwt).sum(1), (wt * dwt).abs().sum(1)
        for j in range(topk):
            ok = (ids[:, j] >= 0) & (ids[:, j] < E)
            t = torch.arange(M, device="cuda")[ok]
            dl[t, ids[ok, j]] += (wt[:, j] * (dwt[:, j] - mean))[ok]
            mag[t, ids[ok, j]] += (wt[:, j].abs() * (dwt[:, j].abs() + size))[ok]
    err = (topk + 6) * U32 * mag
    r = torch.zeros((M, 1, K), dtype=torch.float64, device="cuda")
    if s["dx_rows"] is not None and M:
        r = s["dx_rows"].double().view(M, -1, K)
    dx = dl @ w + r.sum(1)
    n = 2 * E + r.shape[1] + 4
    b = (err + U16 * U16 * dl.abs()) @ w.abs() + 2 * n * U32 * (dl.abs() @ w.abs() + r.abs().sum(1))
    dx_b = b + U16 * (dx.abs() + b)
    dw = dl.t() @ x
    dw_b = err.t() @ x.abs() + 2 * (3 * M + 4) * U32 * (dl.abs().t() @ x.abs()) + U32 * dw.abs()
    db = dl.sum(0)
    db_b = err.sum(0) + 2 * (M + 4) * U32 * dl.abs().sum(0) + U32 * db.abs()
    return (dx, dw, db), (dx_b, dw_b, db_b)


SHAPES = [  # M, K, E, topk
    (1, 1, 1, 1), (1, 64, 8, 2), (2, 7, 3, 2), (64, 256, 8, 2), (65, 100, 5, 3), (63, 129, 64, 8),
    (130, 128, 65, 4), (77, 333, 127, 6), (200, 520, 256, 8), (300, 1001, 130, 16), (1100, 264, 8, 2),
    (1500, 1032, 60, 4), (3, 7168, 256, 8), (2050, 5, 2, 1), (600, 4096, 16, 2), (4100, 136, 200, 8),
    (40, 20001, 9, 1),
]


@pytest.mark.parametrize("M,K,E,topk", SHAPES)
@pytest.mark.parametrize("what", ["weights", "dlogits", "both", "rows"])
def test_topk_bwd(moe, M, K, E, topk, what):
    note(f"topk_bwd M={M} K={K} E={E} topk={topk} {what}")
    rows = {"rows": topk, "both": 1}.get(what, 0)
    s = inputs(M, K, E, topk, rows, what != "dlogits", what in ("dlogits", "both"), 5)
    if what == "both" and M > 3:
        s["topk_ids"][M // 2, 0] = -1            # a dropped slot passes nothing on
        s["topk_ids"][M // 3, topk - 1] = E
        if topk > 1:
            s["topk_ids"][1, 1] = s["topk_ids"][1, 0]
    want, bound = reference(s)
    got = moe.moe_topk_bwd(**s, bias=True)
    for g, w, b, name in zip(got, want, bound, ("dx", "dw", "dbias")):
        check(g, w, b, name)
    again = moe.moe_topk_bwd(**s)
    assert again[2] is None and torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


@pytest.mark.parametrize("M,K,E,topk", SHAPES)
def test_topk_bwd_exactly(moe, M, K, E, topk):
    """dlogits of 17 bits, tokens and weights of -1, 0 and 1: all three parts of dl
    are needed, every sum is an integer below 2^24, and dw and dbias are equal; and
    with dlogits of 7 bits dx is."""
    note(f"topk_bwd exactly M={M} K={K} E={E}")
    most = min(1 << 17, (1 << 23) // M)
    x, w = ints((M, K), 1, 1).to(torch.bfloat16), ints((E, K), 2, 1).to(torch.bfloat16)
    dl = ints((M, E), 3, most).float()
    _, dw, db = moe.moe_topk_bwd(x, w, dlogits=dl, bias=True)
    assert torch.equal(dw.double(), dl.double().t() @ x.double())
    assert torch.equal(db.double(), dl.double().sum(0))
    dl, rows = ints((M, E), 4, 100).float(), ints((2 * M, K), 5, 100).to(torch.bfloat16)
    dx, _, _ = moe.moe_topk_bwd(x, w, dlogits=dl, dx_rows=rows)
    want = dl.double() @ w.double() + rows.double().view(M, 2, K).sum(1)
    assert torch.equal(dx, want.to(torch.bfloat16))


def test_topk_bwd_without_tokens(moe):
    note("topk_bwd M=0")
    for K in (1, 136):
        dx, dw, db = moe.moe_topk_bwd(bf16((0, K), 1), bf16((9, K), 2), dlogits=f32((0, 9), 3),
                                      dx_rows=bf16((0, K), 4), bias=True)
        assert dx.shape == (0, K) and (dw == 0).all() and (db == 0).all()


def test_topk_bwd_not_finite(moe):
    """An infinity or a NaN of a gradient stays in its token's dx and its expert's
    dw, as in the product."""
    note("topk_bwd, infinity")
    M, K, E = 70, 40, 9
    x, w = bf16((M, K), 1).abs() + 1, bf16((E, K), 2).abs() + 1
    dl = f32((M, E), 3)
    dl[7, 2], dl[66, 8] = float("inf"), float("nan")
    dx, dw, db = moe.moe_topk_bwd(x, w, dlogits=dl, bias=True)
    row = torch.arange(M, device="cuda")
    assert (dx[7] == float("inf")).all() and dx[66].isnan().all()
    assert torch.isfinite(dx[(row != 7) & (row != 66)]).all()
    assert (dw[2] == float("inf")).all() and dw[8].isnan().all()
    assert db[2] == float("inf") and db[8].isnan()
    assert torch.isfinite(dw[[0, 1, 3, 4, 5, 6, 7]]).all()


def test_topk_bwd_against_differences(moe):
    """Gradients of sum(dwts * weights) with the weights that moe_topk's formula
    gives, against central differences in fp64."""
    note("topk_bwd, differences")
    M, K, E, topk, h = 4, 24, 6, 3, 1e-6
    x, w, dwt = bf16((M, K), 1), bf16((E, K), 2, K ** -0.5), f32((M, topk), 3)
    ids, wts, _ = moe.moe_topk(x, w, torch.zeros(E, device="cuda"), topk)
    dx, dw, db = moe.moe_topk_bwd(x, w, ids, wts, dwt, bias=True)

    def loss(x, w, b):
        l = (x @ w.t() + b).gather(1, ids.long())
        return (dwt.double() * torch.softmax(l, 1)).sum()

    at = [x.double(), w.double(), torch.zeros(E, dtype=torch.float64, device="cuda")]
    for i, got in enumerate((dx, dw, db)):
        flat = got.double().flatten()
        for c in range(flat.numel()):
            step = torch.zeros(flat.numel(), dtype=torch.float64, device="cuda")
            step[c] = h
            hi, lo = (loss(*[v + (s * step).view(v.shape) if j == i else v for j, v in enumerate(at)]) for s in (1, -1))
            want = (hi - lo) / (2 * h)
            # rounding of dx, fp32 of the terms (|dw| up to 3, |x|, |w| up to 4, a few of
            # them), and 1e-8 of the difference
            tol = (U16 * want.abs() + 2.0 ** -14 * 3 if i == 0 else 200 * U32 * 12) + 1e-8
            assert abs(flat[c] - want) <= tol, (i, c)


def test_refusals(moe):
    note("router refusals")
    s = inputs(4, 16, 8, 2, 2, True, True, 1)
    logits, ids = f32((4, 8), 1), s["topk_ids"]
    loss, counts, tokens, _ = moe.moe_balance(logits, ids)
    for call in (lambda: moe.moe_balance(logits.double(), ids), lambda: moe.moe_balance(logits, ids[:3]),
                 lambda: moe.moe_balance(logits, ids.long()), lambda: moe.moe_balance(logits[:, :7], ids),
                 lambda: moe.moe_balance(logits, ids, token_mask=torch.ones(3, dtype=torch.bool, device="cuda")),
                 lambda: moe.moe_balance(logits, ids, token_mask=torch.ones(4, device="cuda")),
                 lambda: moe.moe_balance_bwd(loss, logits, counts[:7], tokens, 2),
                 lambda: moe.moe_balance_bwd(loss.double(), logits, counts, tokens, 2),
                 lambda: moe.moe_balance_bwd(loss, logits, counts, counts, 2),
                 lambda: moe.moe_topk_bwd(s["x"], s["w_router"]),
                 lambda: moe.moe_topk_bwd(s["x"], s["w_router"], ids, dlogits=s["dlogits"]),
                 lambda: moe.moe_topk_bwd(**{**s, "x": s["x"].float()}),
                 lambda: moe.moe_topk_bwd(**{**s, "w_router": s["w_router"][:, :8]}),
                 lambda: moe.moe_topk_bwd(**{**s, "dx_rows": s["dx_rows"][:7]}),
                 lambda: moe.moe_topk_bwd(**{**s, "dx_rows": s["dx_rows"][:0]}),
                 lambda: moe.moe_topk_bwd(**{**s, "dlogits": s["dlogits"][:, :7].contiguous()}),
                 lambda: moe.moe_topk_bwd(**{**s, "topk_weights": None})):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: moe.moe_balance(logits, ids.repeat(1, 5)),          # topk above E
                 lambda: moe.moe_balance(f32((4, 257), 1), ids),
                 lambda: moe.moe_balance_bwd(loss, logits, counts, tokens, 9),
                 lambda: moe.moe_topk_bwd(**{**s, "dx_rows": bf16((4 * 17, 16), 1)}),
                 lambda: moe.moe_topk_bwd(**inputs(140, 16, 8, 2, 2, True, True, 1),
                                          workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(moe.MoEError):
            call()


@pytest.mark.parametrize("M,K,E,topk", [(6, 40, 8, 2), (1500, 136, 70, 4), (9000, 72, 16, 2)])
def test_streams_graphs_and_equal_bits(moe, M, K, E, topk):
    """The three calls of a step captured and replayed on new inputs, with eager
    work in between, and on two other streams at once: the same bits every
    time."""
    note(f"router graph M={M} K={K} E={E}")

    def new(seed):
        s = inputs(M, K, E, topk, topk, True, False, seed)
        return dict(s, logits=f32((M, E), seed, 2.0), up=f32((1,), seed + 9),
                    mask=(torch.rand(M, generator=torch.Generator().manual_seed(seed)) < 0.9).cuda())

    def step(s):
        b = moe.moe_balance(s["logits"], s["topk_ids"], token_mask=s["mask"])
        dl = moe.moe_balance_bwd(s["up"], s["logits"], b[1], b[2], topk, token_mask=s["mask"])
        names = ("x", "w_router", "topk_ids", "topk_weights", "dtopk_weights")
        return (*b, dl, *moe.moe_topk_bwd(*[s[k] for k in names], dlogits=dl, dx_rows=s["dx_rows"], bias=True))

    s = new(1)
    step(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(s)
    for rep in range(4):
        for k, v in new(20 * rep + 40).items():
            if v is not None:
                s[k].copy_(v)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in outs]
        eager = step(s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, eager))
    jobs = [s, new(200)]
    want = [step(j) for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i].append(step(jobs[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
