"""Rows kept in 8 bits, from the format's definition: a block of 32 columns has
the least X of 0..254 with max |x| <= 127 * 2^(X-133), its codes are x * 2^(133-X)
rounded to the nearest integer, ties to even, within +-127; X = 255 and codes of
zero where the block holds an infinity or a NaN.  Everything is exact in 64
bits."""
import torch

BLOCK = 32


def keep(x):
    """(codes int8 [R,W], X uint8 [R,blocks], values fp64 [R,W])"""
    R, W = x.shape
    nb = -(-W // BLOCK)
    v = torch.zeros((R, nb * BLOCK), dtype=torch.float64, device=x.device)
    v[:, :W] = x.double()
    v = v.view(R, nb, BLOCK)
    bad = ~torch.isfinite(v).all(2)
    v = torch.where(bad[..., None], torch.zeros_like(v), v)
    amax = v.abs().amax(2)
    # 127 * 2^(X-133) for every X, ascending: exact
    reach = 127.0 * torch.pow(2.0, torch.arange(255, dtype=torch.float64) - 133).to(x.device)
    X = torch.searchsorted(reach, amax.contiguous()).clamp(max=254)     # least X with amax <= reach[X]
    step = reach[X] / 127
    codes = (v / step[..., None]).round().clamp(-127, 127)
    values = torch.where(bad[..., None], torch.full_like(v, float("nan")), codes * step[..., None])
    X = torch.where(bad, torch.full_like(X, 255), X)

    def flat(t):
        return t.reshape(R, nb * BLOCK)[:, :W].contiguous()

    return flat(codes).to(torch.int8), X.to(torch.uint8), flat(values)


def keep_halves(g):
    """The same of the activation's input: the two halves of a row as rows."""
    R, W = g.shape
    codes, X, values = keep(g.reshape(2 * R, W // 2))
    return codes.view(R, W), X.view(R, -1), values.view(R, W)


def spread(R, W, seed):
    """bf16 rows of every size: normal values, blocks of subnormal and of huge
    ones, zeros, ties between two codes."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((R, W), generator=g) * torch.exp(2 * torch.randn((R, 1), generator=g))
    nb = -(-W // BLOCK)
    kind = torch.randint(0, 8, (R, nb), generator=g).repeat_interleave(BLOCK, 1)[:, :W]
    far = torch.pow(2.0, torch.randint(-126, 127, (R, nb), generator=g).double())
    far = far.repeat_interleave(BLOCK, 1)[:, :W].float()
    halves = torch.randint(-255, 256, (R, W), generator=g) / 2
    x = torch.where(kind == 0, torch.zeros_like(x), x)
    x = torch.where(kind == 1, torch.randint(-255, 256, (R, W), generator=g) * 2.0 ** -133, x)
    x = torch.where(kind == 2, x.sign() * (x.abs() % 2) * far, x)
    x = torch.where(kind == 3, halves, x)
    x = x.clamp(-3.3895e38, 3.3895e38).to(torch.bfloat16)
    return x
