"""Workspaces of exactly the reported size, with anything in them; inputs that
end where values begin that must not count; outputs with guards behind them.
The bits are those of ordinary calls, and no guard changes.

The calls go to the C entry points, whose outputs are the caller's."""
import ctypes

import pytest
import torch

from tests._paths import DW
from tests._train_ref import bf16, f32
from tests.test_gpu_ckpt import dw_case
from tests.test_gpu_router_grad import inputs

pytestmark = pytest.mark.gpu

GUARD = 4096            # bytes before and behind


@pytest.fixture(scope="module")
def moe():
    import moe_layer_04_amd as m
    m.load_library()
    return m


def note(msg):
    print(f"[gpu-test] {msg}", flush=True)


class Held:
    """A tensor inside a buffer of one byte's copies: bytes of 0xff are NaN in every
    floating type and -1 in integers."""

    def __init__(self, shape, dtype, fill=0xff, value=None):
        n = torch.empty(shape, dtype=dtype, device="meta").nbytes
        self.fill, self.n = fill, n
        self.all = torch.full((2 * GUARD + (n + 15) // 16 * 16,), fill, dtype=torch.uint8, device="cuda")
        self.t = self.all[GUARD:GUARD + n].view(dtype).view(shape)
        if value is not None:
            self.t.copy_(value)

    @property
    def ptr(self):
        return self.all.data_ptr() + GUARD

    def unharmed(self):
        return bool((self.all[:GUARD] == self.fill).all() and (self.all[GUARD + self.n:] == self.fill).all())


def held(t, fill=0xff):
    return None if t is None else Held(t.shape, t.dtype, fill, t)


def ptr(h):
    return None if h is None else h.ptr


def outs(like, fill):
    return [None if t is None else Held(t.shape, t.dtype, fill) for t in like]


def run(lib, name, ins, sizes, out, fill=None):
    """One call with its workspace, if it takes one (fill: what that holds)."""
    f = getattr(lib, name)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    p, q = [ptr(h) for h in ins], [ptr(h) for h in out]
    ws = None
    if fill is None:
        assert f(*p, *sizes, *q, stream) == 0
    else:
        n = ctypes.c_size_t(0)
        assert f(*[None] * len(p), *sizes, *[None] * len(q), None, ctypes.byref(n), stream) == 0
        ws = Held((n.value,), torch.uint8, fill)
        assert ws.ptr % 256 == 0
        assert f(*p, *sizes, *q, ws.ptr, ctypes.byref(n), stream) == 0
    torch.cuda.synchronize()
    assert all(h is None or h.unharmed() for h in (*ins, *out, ws))


def same(out, want):
    for h, w in zip(out, want):
        if h is not None:
            bits = (lambda t: t.view(torch.uint8)) if w.dtype.itemsize == 1 else (lambda t: t)
            assert torch.equal(bits(h.t), bits(w))


FILLS = [0xff, 0x00, 0x55]


@pytest.mark.parametrize("M,E,topk", [(1, 1, 1), (64, 8, 2), (33, 5, 2), (2100, 8, 2), (9000, 17, 3), (5000, 256, 8),
                                      (777, 130, 16), (70000, 3, 2)])
@pytest.mark.parametrize("fill", FILLS)
def test_balance(moe, M, E, topk, fill):
    note(f"guards, balance M={M} E={E} fill={fill:#x}")
    lib = moe.load_library()
    logits = f32((M, E), 1, 2.0)
    ids = logits.topk(topk, dim=1).indices.to(torch.int32)
    mask = (f32((M,), 2) < 1).to(torch.uint8)
    want = moe.moe_balance(logits, ids, token_mask=mask)
    # (ids of zeros past the end would count)
    ins = [held(logits), held(ids, 0), held(mask)]
    out = outs(want, fill)
    run(lib, "moe_balance", ins, (M, E, topk), out, fill)
    same(out, want)
    up = f32((1,), 3)
    back = moe.moe_balance_bwd(up, logits, want[1], want[2], topk, token_mask=mask)
    d = outs([back], fill)
    run(lib, "moe_balance_bwd", [held(up), ins[0], held(want[1]), held(want[2]), ins[2]], (M, E, topk), d)
    same(d, [back])


@pytest.mark.parametrize("M,K,E,topk", [(1, 1, 1, 1), (64, 256, 8, 2), (65, 100, 5, 3), (130, 128, 65, 4), (77, 333, 127, 6),
                                        (300, 1001, 130, 16), (1100, 264, 8, 2), (1500, 1033, 60, 4), (2050, 5, 2, 1),
                                        (4100, 139, 200, 8), (129, 7, 3, 2)])
@pytest.mark.parametrize("fill", FILLS)
def test_topk_bwd(moe, M, K, E, topk, fill):
    note(f"guards, topk_bwd M={M} K={K} E={E} fill={fill:#x}")
    lib = moe.load_library()
    s = inputs(M, K, E, topk, topk, True, True, 7)
    want = moe.moe_topk_bwd(**s, bias=True)
    names = ("x", "w_router", "topk_ids", "topk_weights", "dtopk_weights", "dlogits", "dx_rows")
    ins = [held(s[k], 0 if k == "topk_ids" else 0xff) for k in names]
    out = outs(want, fill)
    run(lib, "moe_topk_bwd", ins, (topk, M, K, E, topk), out, fill)
    same(out, want)


@pytest.mark.parametrize("name", list(DW))
@pytest.mark.parametrize("rows", ["sorted", "gather_x"])
@pytest.mark.parametrize("fill", [0xff, 0x55])
def test_dw_ckpt(moe, name, rows, fill):
    note(f"guards, dw_ckpt {name} {rows} fill={fill:#x}")
    lib = moe.load_library()
    x, dy, off, kw = dw_case(moe, name, 7, rows)
    codes, X = moe.moe_ckpt_rows(x)
    ids, T, topk = kw["sorted_ids"], kw["num_tokens"], kw["topk"]
    sizes = (1 if kw["gather_x"] else 0, T, topk, ids.shape[0], off.shape[0] - 1, x.shape[1], dy.shape[1])
    for mode, dtype in ((0, torch.bfloat16), (1, torch.float32)):
        want = moe.moe_grouped_gemm_dw_ckpt(dy, codes, X, off, out_dtype=dtype, **kw)
        # (codes past the end are 0x77 with scales of 0x77: neither zeros nor NaN)
        for after in (0xff, 0x77):
            out = outs([want], fill)
            ins = [held(dy), held(codes, after), held(X, after), held(off), held(ids)]
            run(lib, "moe_grouped_gemm_dw_ckpt", ins, (*sizes, mode), out, fill)
            same(out, [want])


@pytest.mark.parametrize("R,W", [(1, 1), (3, 31), (5, 33), (7, 100), (64, 72), (203, 1001), (2, 4099)])
def test_rows(moe, R, W):
    note(f"guards, ckpt_rows {R} x {W}")
    lib = moe.load_library()
    x = bf16((R, W), 1)
    want = moe.moe_ckpt_rows(x)
    for fill in FILLS:
        out = outs(want, fill)
        run(lib, "moe_ckpt_rows", [held(x)], (R, W), out)
        same(out, want)
        back = outs([x], fill)
        run(lib, "moe_ckpt_restore", out, (R, W), back)
        same(back, [moe.moe_ckpt_restore(*want)])


@pytest.mark.parametrize("R,N", [(1, 1), (3, 31), (6, 33), (16, 512), (40, 24), (61, 333), (2, 4099), (5, 8200)])
@pytest.mark.parametrize("fill", FILLS)
def test_silu_mul_ckpt(moe, R, N, fill):
    note(f"guards, silu_mul_ckpt {R} x {N} fill={fill:#x}")
    lib = moe.load_library()
    g, da, wt = bf16((R, 2 * N), 1, 2.0), bf16((R, N), 2), f32((R,), 3)
    ids = torch.randperm(R, generator=torch.Generator().manual_seed(4)).to(torch.int32).cuda()
    num = torch.tensor([R], dtype=torch.int32, device="cuda")
    want = moe.moe_silu_mul_ckpt(g, wt, sorted_ids=ids, num_rows=num)
    rows = [held(wt), held(ids), held(num)]
    out = outs(want, fill)
    run(lib, "moe_silu_mul_ckpt", [held(g), *rows], (R, R, N), out)
    same(out, want)
    want = moe.moe_silu_mul_bwd_ckpt(da, want[1], want[2], wt, sorted_ids=ids, num_rows=num)
    back = outs(want, fill)
    run(lib, "moe_silu_mul_bwd_ckpt", [held(da), *out[1:], *rows], (R, R, N), back)
    same(back, want)
