"""Rotary positions far out against angles of sixty digits."""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TWO_PI = Decimal("6.283185307179586476925286766559005768394338798750211641949889")
POSITIONS = [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30 + 7, 1_234_567_891, 100_000_007, 23_000_003, 16_777_215, 131_071, 1]


def turns(dim, base=10000.0, scaling="none", factor=1.0, original=0, fast=32.0, slow=1.0):
    """Turns a position of each pair."""
    base, s = Decimal(base), Decimal(factor)
    if scaling == "ntk":
        base *= s ** (Decimal(dim) / (dim - 2))
    out = []
    for i in range(dim // 2):
        f = base ** (Decimal(-2 * i) / dim)
        if scaling == "linear":
            f /= s
        if scaling == "parts":
            keep = (Decimal(original) * f / TWO_PI - Decimal(slow)) / (Decimal(fast) - Decimal(slow))
            keep = min(max(keep, Decimal(0)), Decimal(1))
            f = f * keep + f / s * (1 - keep)
        out.append(f / TWO_PI)
    return out


@pytest.mark.parametrize("rope", [
    dict(), dict(base=500000.0), dict(base=1e6, dim=50), dict(scaling="linear", factor=3.0),
    dict(scaling="ntk", factor=7.0, base=500000.0), dict(scaling="parts", factor=16.0, original=8192, attention_factor=1.0),
])
def test_the_angle_of_any_position(rope):
    """Angles to 2^-32 of a turn, cosines and sines as if exact: a half step of fp32, 2^-24 of themselves, and 2 pi
    2^-32 (and 2^-28 of themselves for those that lie next to the middle of two numbers)."""
    import tensor_transformer_mlp_shard_gb300 as tp
    getcontext().prec = 60
    D, n = 128, len(POSITIONS)
    dim = rope.get("dim", D)
    half = dim // 2
    h = tp.TPRotary(n, 1, 1, 1, D, dtype="f32", rope=tp.Rope(**rope))
    x = torch.zeros(n, 3, D, device="cuda")
    x[:, 0, :half] = 1.0        # the query: cosine and sine
    x[:, 1, half:dim] = 1.0     # the key: minus the sine, and the cosine
    y = torch.empty_like(x)
    h.fwd(x, y, positions=torch.tensor(POSITIONS, dtype=torch.int32, device="cuda"))
    y = y.double().cpu().numpy()
    per = turns(dim, **{k: v for k, v in rope.items() if k not in ("dim", "attention_factor")})
    for j, p in enumerate(POSITIONS):
        angle = np.array([float((p * t) % 1) for t in per]) * 2.0 * math.pi
        c, s = np.cos(angle), np.sin(angle)
        for got, want in ((y[j, 0, :half], c), (y[j, 0, half:dim], s), (y[j, 1, :half], -s), (y[j, 1, half:dim], c)):
            bound = np.abs(want) * (2.0 ** -24 + 2.0 ** -28) + 2.0 * math.pi * 2.0 ** -32
            off = np.abs(got - want)
            assert (off <= bound).all(), (p, int(np.argmax(off - bound)), off.max())
