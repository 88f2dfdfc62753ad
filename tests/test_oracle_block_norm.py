"""Pins of the fp64 block norm oracle: its gradients against central
differences of its forward, its norms against hand values, and the AdamW
oracle's number format and rounding bits."""
import numpy as np
import pytest

from oracle import adamw as oa
from oracle import block_norm as ob

EPS = 1e-5


def loss(x, f, gate, token, post, pw, pb, pre, nw, nb, a, c, zc, wy, wn):
    y = a * x + (0 if f is None else ob.added(f, post, pw, pb, gate, token, c, EPS, zc))
    return (wy * y).sum() + (0 if pre == "none" else (wn * ob.norm(y, pre, nw, nb, EPS, zc)).sum())


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
def test_gradients_against_differences(post, pre, gate):
    """Central differences at h = 1e-5: truncation h^2 |f'''| and rounding
    2^-52 |f| / h are both below 1e-7 of values near 1."""
    rng = np.random.default_rng(7)
    M, H, a, c, zc = 3, 6, 0.7, 1.3, gate == "token"
    t = {"x": rng.normal(size=(M, H)), "f": rng.normal(size=(M, H)) + 0.3, "pw": rng.normal(size=H) + 1,
         "pb": rng.normal(size=H), "nw": rng.normal(size=H) + 1, "nb": rng.normal(size=H),
         "g": {"none": None, "channel": rng.normal(size=H), "token": rng.normal(size=M),
               "element": rng.normal(size=(M, H))}[gate]}
    wy, wn = rng.normal(size=(M, H)), rng.normal(size=(M, H))

    def value(t):
        return loss(t["x"], t["f"], t["g"], gate == "token", post, t["pw"], t["pb"], pre, t["nw"], t["nb"], a, c, zc,
                    wy, wn)

    y = a * t["x"] + ob.added(t["f"], post, t["pw"], t["pb"], t["g"], gate == "token", c, EPS, zc)
    got = ob.grads(wy, wn, y, t["f"], t["g"], gate, post, t["pw"], t["pb"], pre, t["nw"], a, c, EPS, zc)
    for key, name in (("x", "dx"), ("f", "df"), ("g", "dgate"), ("pw", "dpost_w"), ("pb", "dpost_b"), ("nw", "dpre_w"),
                      ("nb", "dpre_b")):
        if got[name] is None:
            continue
        diff = np.zeros_like(t[key])
        for i in np.ndindex(diff.shape):
            ends = []
            for s in (1e-5, -1e-5):
                moved = {k: None if v is None else v.copy() for k, v in t.items()}
                moved[key][i] += s
                ends.append(value(moved))
            diff[i] = (ends[0] - ends[1]) / 2e-5
        np.testing.assert_allclose(got[name], diff, rtol=1e-6, atol=1e-6, err_msg=name)


def test_norms_by_hand():
    x = np.array([[3.0, 4.0], [0.0, 0.0]])
    np.testing.assert_allclose(ob.norm(x, "rms", [1, 2], None, 0.0 + 1e-300)[0], [3 / 12.5 ** 0.5, 8 / 12.5 ** 0.5])
    assert (ob.norm(x, "rms", [1, 1], None, EPS)[1] == 0).all()
    np.testing.assert_allclose(ob.norm(x, "layer", [0, 0], [5, 6], 1e-300, True)[0], [4, 7])


def test_e4m3_values():
    v = oa.e4m3_values()
    assert v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[0x7E] == 448 and np.isnan(v[0x7F]) and v[0x38] == 1
    assert (v[128:] == -v[:128])[:127].all()
    torch = pytest.importorskip("torch")
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(v, t)


def test_hash_bits_are_uniform():
    """2^20 hashes: every bit's share of ones, and the correlation of the two
    halves, within 6 standard deviations (6 / (2 sqrt n) and 6 / sqrt n)."""
    n = 1 << 20
    b = oa.random_bits(5, 3, 2, n)
    for k in range(32):
        ones = ((b >> np.uint64(k)) & np.uint64(1)).mean()
        assert abs(ones - 0.5) < 3 / n ** 0.5, k
    lo, hi = (b & np.uint64(0xFFFF)).astype(float), (b >> np.uint64(16)).astype(float)
    assert abs(np.corrcoef(lo, hi)[0, 1]) < 6 / n ** 0.5
    assert abs(np.corrcoef(lo[:-1], lo[1:])[0, 1]) < 6 / n ** 0.5
    # another step, tensor or seed: other bits
    for other in (oa.random_bits(5, 4, 2, n), oa.random_bits(5, 3, 1, n), oa.random_bits(6, 3, 2, n)):
        assert abs(np.corrcoef(lo, (other & np.uint64(0xFFFF)).astype(float))[0, 1]) < 6 / n ** 0.5


def test_rounding_keeps_the_expectation():
    """Mean of the rounded values of a constant: its error is at most 2^-16 of a
    step (16 random bits truncate) plus 6 standard deviations of the mean."""
    n = 1 << 18
    for value in (300.3, 1.01, 0.02, 0.0007):
        x = np.full(n, value)
        x[::256] = 448.0  # the block's scale is 1
        scales = oa.block_scales(x)
        _, step, at = oa.positions(x, scales, oa.random_bits(1, 1, 0, n) & np.uint64(0xFFFF))
        got = np.floor(at) * step
        rest = np.arange(n) % 256 != 0
        assert abs(got[rest].mean() - value) < step[1] * (2.0 ** -16 + 6 * 0.5 / n ** 0.5)


def test_update_by_hand():
    """First step of a zero state: m_hat = g and v_hat = g^2."""
    w, m, v = oa.update([1.0], [0.5], [0.0], [0.0], 1, 0.1, 0.9, 0.99, 1e-8, 0.2)
    np.testing.assert_allclose(w, 1 - 0.1 * 0.2 - 0.1 * 0.5 / (0.5 + 1e-8))
    np.testing.assert_allclose([m[0], v[0]], [0.05, 0.0025])
