"""Pins of the attention oracle (no GPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as ref


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_rotation(interleaved):
    """Lengths and angles of pairs: scores depend on the distance of positions alone, position 0 turns nothing."""
    rng = np.random.default_rng(0)
    f, a = ref.rope_frequencies(16)
    x, y = rng.standard_normal((2, 1, 1, 20))
    turn = lambda v, p: ref.rotate(v, [p], f, a, interleaved)  # noqa: E731
    assert np.array_equal(turn(x, 0), x)
    assert abs(np.linalg.norm(turn(x, 77)) - np.linalg.norm(x)) < 1e-13
    dots = [float((turn(x, p) * turn(y, p + 5)).sum()) for p in (0, 1, 1000)]
    assert max(dots) - min(dots) < 1e-11
    assert np.allclose(ref.rotate(turn(x, 9), [9], f, a, interleaved, back=True), x, atol=1e-14)
    assert np.array_equal(turn(x, 3)[..., 16:], x[..., 16:])


def test_rotation_by_complex_numbers():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((4, 3, 12))
    f, a = ref.rope_frequencies(12, base=100.0)
    at = np.array([0, 3, 50, 7])
    z = torch.polar(torch.tensor(a, dtype=torch.float64).expand(4, 6).contiguous(), torch.tensor(np.outer(at, f)))[:, None]
    w = torch.view_as_real(torch.view_as_complex(torch.tensor(x).view(4, 3, 6, 2)) * z).view(4, 3, 12).numpy()
    assert np.allclose(ref.rotate(x, at, f, a, True), w, atol=1e-14)
    halves = np.concatenate([x[..., 0::2], x[..., 1::2]], -1)
    assert np.allclose(ref.rotate(halves, at, f, a), np.concatenate([w[..., 0::2], w[..., 1::2]], -1), atol=1e-14)


def test_frequencies():
    f, a = ref.rope_frequencies(64)
    assert f[0] == 1.0 and a == 1.0 and abs(f[16] - 0.01) < 1e-15
    assert np.allclose(ref.rope_frequencies(64, scaling="linear", factor=4.0)[0], f / 4)
    g = ref.rope_frequencies(64, scaling="ntk", factor=4.0)[0]
    assert g[0] == 1.0 and abs(g[-1] / (f[-1] / 4) - 1) < 1e-12
    p, a = ref.rope_frequencies(64, scaling="parts", factor=4.0, original=2048)
    turns = 2048 * f / (2 * math.pi)
    assert np.array_equal(p[turns >= 32], f[turns >= 32]) and np.allclose(p[turns <= 1], f[turns <= 1] / 4)
    assert abs(a - (0.1 * math.log(4.0) + 1)) < 1e-15
    assert np.all(np.diff(p) < 0)


def test_columns():
    assert ref.qkv_columns(4, 2, False) == ([0, 1, 2, 3], [4, 5], [6, 7])
    assert ref.qkv_columns(4, 2, True) == ([0, 1, 4, 5], [2, 6], [3, 7])


@pytest.mark.parametrize("window", [0, 5])
def test_decode_against_torch(window):
    rng = np.random.default_rng(2)
    n, hq, hk, D, page = 19, 6, 2, 8, 4
    k, v = rng.standard_normal((2, hk, n, D))
    table = np.array([[3, 0, 4, 1, 2, -1]])
    K, V = np.full((2, 6, hk, page, D), np.nan)
    for p in range(n):
        K[table[0, p // page], :, p % page] = k[:, p]
        V[table[0, p // page], :, p % page] = v[:, p]
    q = rng.standard_normal((2, hq, D))
    o, mag, _, seen = ref.decode(q, [n - 1, -1], [0, 9], table, K, V, D ** -0.5, window)
    lo = n - window if window else 0
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.tensor(q[0])[:, None], torch.tensor(k[:, lo:]).repeat_interleave(3, 0), torch.tensor(v[:, lo:]).repeat_interleave(3, 0))
    assert np.allclose(o[0], want[:, 0].numpy(), atol=1e-13)
    assert not o[1].any() and list(seen) == [n - lo, 0] and (mag[0] >= np.abs(o[0]) - 1e-15).all()


def test_slots():
    table = np.array([[5, 2], [7, -1]])
    got = ref.slots([0, 17, 32, -1, 3, 16, 1], [0, 0, 0, 0, 1, 1, 2], table, 16, 7)
    assert got == [(5, 0), (2, 1), None, None, None, None, None]
