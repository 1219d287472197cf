"""The reference of the 8-bit format against its definition, value by value in
Python's own numbers."""
from fractions import Fraction

import pytest
import torch

from tests._ckpt_ref import BLOCK, keep, spread


def kept_block(values):
    """(X, codes) of one block of finite values, from the definition."""
    top = max(abs(v) for v in values)
    X = next((X for X in range(255) if top <= 127 * Fraction(2) ** (X - 133)), 254)
    step = Fraction(2) ** (X - 133)
    return X, [max(-127, min(127, round(v / step))) for v in values]   # round: ties to even


@pytest.mark.parametrize("R,W", [(1, 1), (3, 33), (20, 100)])
def test_reference(R, W):
    x = spread(R, W, R)
    if R == 20:
        x[0, :32] = 0
        x[0, 5] = 255 * 2.0 ** 120           # the largest value: no code reaches it
        x[1, 0], x[2, 40], x[3, 99] = float("inf"), float("nan"), float("-inf")
    codes, X, values = keep(x)
    for r in range(R):
        for b in range(-(-W // BLOCK)):
            part = slice(b * BLOCK, min(W, (b + 1) * BLOCK))
            row = x[r, part].double().tolist()
            if not all(abs(v) < float("inf") for v in row):
                assert X[r, b] == 255 and values[r, part].isnan().all() and (codes[r, part] == 0).all()
                continue
            want_X, want = kept_block([Fraction(v) for v in row])
            assert int(X[r, b]) == want_X and codes[r, part].tolist() == want
            assert values[r, part].tolist() == [float(c * Fraction(2) ** (want_X - 133)) for c in want]
    # every value is a bf16 number, and at most 1/127 of its block's largest off
    ok = torch.isfinite(values)
    assert torch.equal(values[ok].to(torch.bfloat16).double(), values[ok])
