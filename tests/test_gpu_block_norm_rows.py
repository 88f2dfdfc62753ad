"""The block norm's backward on rows whose mean lies far from zero, and on rows
with nothing in them, against the fp64 oracle.

A LayerNorm's statistics hold the mean rounded to fp32.  A row of mean 990 and
spread 1 is then off by up to 2^-15, the same for all its columns; a sum over
tokens adds that up.  The rows here have one mean between two fp32 values, so
nothing cancels.

Tolerances (u = 2^-24): x - mean is exact (both lie within a factor of two); the
normalised row carries the product with 1 / spread, the subtraction of its own
mean and the statistics' roundings, under 64 u of max(|xh|, 1).  A column's sum
adds at most 16 rows: 100 u of the sum of |d| (|xh| + 1).  Nothing in them grows
with the mean.
"""
import numpy as np
import pytest
import torch

from oracle import block_norm as ob
from test_gpu_block_norm import EPS, U, Case, _odd_rows, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tp():
    import tensor_transformer_mlp_shard_gb300 as tp
    from tensor_transformer_mlp_shard_gb300 import build
    build.build()
    return tp


def far_rows(M, H):
    """M rows of the same values in other orders, fp32, mean 990 and 0.4 of a step, spread 1."""
    step = 2.0 ** -14  # of fp32 between 512 and 1024
    row = np.rint((np.random.default_rng(H).normal(size=H) + 990.0) / step).astype(np.int64)
    over = int((row.sum() - (4 * H) // 10) % H)
    row[:(H - over) % H] += 1  # the sum is now 0.4 H above a multiple of H
    row = (row * step).astype(np.float32)
    at = (row.astype(np.float64).mean() / step) % 1.0
    assert abs(at - 0.4) < 1e-2 + 1.0 / H
    return torch.from_numpy(np.stack([np.roll(row, 7 * m) for m in range(M)])).cuda()


def close(got, ref, terms, name):
    err = np.abs(f64(got) - ref) / (100 * U * terms)
    assert (err <= 1).all(), (name, float(err.max()))


@pytest.mark.parametrize("H", [256, 512, 2056, 8192, 16384])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pre_norm_of_rows_far_from_zero(tp, H, dtype):
    """The stream in fp32, with activations of either type."""
    M = 16
    c = Case(M, H, dtype, "none", "layer", res32=True, block=False)
    c.x = far_rows(M, H)
    c.dn = (c.dn.float() * 0.25 + 1.0).to(c.act)
    h = c.handle(tp)
    c.run_fwd(h)
    c.run_bwd(h, tp)
    c.check_bwd()
    mean, rstd = ob.norm_stats(f64(c.x), "layer", EPS)
    hat, dn = (f64(c.x) - mean) * rstd, f64(c.dn)
    close(c.out["dpre_w"], (dn * hat).sum(0), (np.abs(dn) * (np.abs(hat) + 1)).sum(0), "dpre_w")


@pytest.mark.parametrize("gate", ["channel", "token"])
@pytest.mark.parametrize("H", [256, 512, 2056, 8192, 16384])
def test_post_norm_of_rows_far_from_zero(tp, H, gate):
    M = 16
    c = Case(M, H, "f32", "layer", "none", gate)
    c.f = far_rows(M, H)
    c.dy = c.dy * 0.25 + 1.0
    if gate == "token":
        c.g = c.g.abs() + 0.5
    h = c.handle(tp)
    c.run_fwd(h)
    c.run_bwd(h, tp)
    c.check_bwd()
    mean, rstd = ob.norm_stats(f64(c.f), "layer", EPS)
    hat, dy, g = (f64(c.f) - mean) * rstd, f64(c.dy), f64(c.g)
    e = dy * (g[:, None] if gate == "token" else g)
    close(c.out["dpost_w"], (e * hat).sum(0), (np.abs(e) * (np.abs(hat) + 1)).sum(0), "dpost_w")
    p = hat * f64(c.pw) + f64(c.pb)
    size = (np.abs(hat) + 1) * np.abs(f64(c.pw)) + np.abs(f64(c.pb))
    axis = 1 if gate == "token" else 0
    close(c.out["dgate"], (dy * p).sum(axis), (np.abs(dy) * size).sum(axis), "dgate")


@pytest.mark.parametrize("H", [512, 2056])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_odd_rows_backward(tp, kind, H):
    """Rows of zeros, without spread, with one channel far above the others, or tiny."""
    c = Case(9, H, "f32", kind, kind, "token", edit=_odd_rows)
    h = c.handle(tp)
    c.run_fwd(h)
    c.run_bwd(h, tp)
    c.check_bwd()
    assert all(torch.isfinite(t).all() for k, t in c.out.items() if kind == "layer" or not k.endswith("_b"))


@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
@pytest.mark.parametrize("H", [256, 2056, 16384])
def test_without_a_post_norm_df_does_not_depend_on_f(tp, H, gate):
    """y = a x + c g f: the gradient of f is c g dy, also where f is NaN or
    infinite (an expert's output that a token's gate of zero leaves out)."""
    def edit(c):
        c.f[3, 5], c.f[4, H - 1], c.f[5] = float("nan"), float("inf"), -float("inf")

    bad, clean = (Case(9, H, "bf16", "none", "none", gate, c=0.5, edit=e) for e in (edit, None))
    for c in (bad, clean):
        if gate != "none":
            c.g[..., 0] = 0.0
        h = c.handle(tp)
        c.run_fwd(h)
        c.run_bwd(h, tp)
    for k in ("dx", "df"):
        assert torch.equal(bad.out[k], clean.out[k]), k
    assert torch.isfinite(bad.out["df"]).all()
