"""The gradient norm over fp32's whole range, and what a clipped step does there.

Tolerances (u = 2^-24): every square is rounded once (u of it), the sums keep
their rounding errors and end in fp64, the norm is rounded once: 2 u of it.
16 u are allowed, as for gradients of ordinary size.  A subnormal gradient's
square is taken of an exactly scaled value.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
MAX = 3.4028234663852886e38


@pytest.fixture(scope="module")
def tp():
    import tensor_transformer_mlp_shard_gb300 as tp
    from tensor_transformer_mlp_shard_gb300 import build
    build.build()
    return tp


def optimizer(tp, grads, **kw):
    w = [torch.zeros(g.numel(), device="cuda") for g in grads]
    return w, tp.TPAdamW(w, grads, beta1=0.9, beta2=0.95, eps=1e-8, **kw)


def fp64_norm(grads):
    return float(np.sqrt(sum(float((g.double() ** 2).sum()) for g in grads)))


@pytest.mark.parametrize("n", [5, 8192, 1 << 22])
@pytest.mark.parametrize("size", [1e-44, 1e-40, 1e-30, 1e-24, 1e-21, 1e-19, 1e-14, 1e-12, 1.0, 1e13, 1e14, 1e18, 3e18,
                                  1e20, 1e30, 1e34])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm_of_any_size(tp, n, size, dtype):
    gen = torch.Generator(device="cuda").manual_seed(n)
    g = (torch.rand(n, generator=gen, device="cuda") + 0.5).double().mul_(size).float().to(dtype)
    _, opt = optimizer(tp, [g])
    total = fp64_norm([g])
    norm = opt.grad_norm(max_norm=1.0)
    # a norm that is subnormal itself is rounded to a multiple of 2^-149
    assert abs(float(norm.double()) - total) <= 16 * U * total + 2.0 ** -149
    assert int(opt.finite) == 1 and int(opt.steps) == 1
    # the clip factor is subnormal for the largest norms: 2^-149 of rounding
    scale = min(1.0, 1.0 / total) if total else 1.0
    assert abs(float(opt.scale.double()) - scale) <= 24 * U * scale + 2.0 ** -149


def test_large_and_small_side_by_side(tp):
    """Chunks and tensors of very different sizes: the norm is of all of them."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    grads = [torch.randn(n, generator=gen, device="cuda") * s
             for n, s in ((100003, 1e15), (40000, 1.0), (700, 3e14), (9000, 1e-30), (1 << 20, 1e12))]
    grads[0][5], grads[1][8191], grads[3][0] = 0.0, 3e15, 1e16
    for order in (grads, grads[::-1]):
        _, opt = optimizer(tp, order)
        total = fp64_norm(order)
        assert abs(float(opt.grad_norm()) - total) <= 16 * U * total


@pytest.mark.parametrize("bits", [32, 8])
def test_clipped_step_on_large_gradients(tp, bits):
    """Gradients of 1e18 whose squares add up beyond fp32: the clipped step is that of their direction."""
    n = 1 << 20
    g = torch.full((n,), 1e18, device="cuda")
    g[1::2] = -1e18
    w, opt = optimizer(tp, [g], state_bits=bits)
    norm = opt.grad_norm(max_norm=1.0)
    opt.step(1e-2)
    assert int(opt.finite) == 1 and int(opt.steps) == 1
    assert abs(float(norm) - 1e18 * 1024) <= 16 * U * 1e18 * 1024
    # the first step is lr g / (|g| + eps): g' is 2^-10, its roundings and eps are under 1e-4 of it
    assert torch.allclose(w[0], torch.sign(g) * -1e-2, rtol=1e-4, atol=0)


@pytest.mark.parametrize("scale,max_norm,steps", [(1.0, float("inf"), 0), (1.0, 1e25, 0), (1.0, 1e19, 1),
                                                   (1e-30, float("inf"), 1), (1e10, float("inf"), 0)])
def test_no_step_whose_squares_overflow(tp, scale, max_norm, steps):
    """The states hold g'^2: a clipped norm beyond fp32's largest root leaves everything as it was."""
    g = torch.full((1000,), 1e22, device="cuda")
    w, opt = optimizer(tp, [g])
    norm = opt.grad_norm(grad_scale=scale, max_norm=max_norm)
    opt.step(1e-2)
    total = 1e22 * 1000 ** 0.5 * scale
    assert abs(float(norm) - total) <= 32 * U * total
    assert int(opt.finite) == steps and int(opt.steps) == steps
    assert torch.isfinite(opt.v[0]).all() and bool((w[0] != 0).all()) == bool(steps)


def test_no_step_whose_squares_overflow_once_scaled(tp):
    """Gradients with a norm of 3e16 and a scale of 1e10 above it."""
    w, opt = optimizer(tp, [torch.full((1000,), 1e15, device="cuda")])
    norm = opt.grad_norm(grad_scale=1e10)
    opt.step(1e-2)
    total = 1e15 * 1000 ** 0.5 * 1e10
    assert abs(float(norm) - total) <= 32 * U * total
    assert int(opt.finite) == 0 and (opt.v[0] == 0).all() and (w[0] == 0).all()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("beside", [0.0, 1e-30, 1.0, 1e30])
def test_not_finite_whatever_lies_beside(tp, value, beside):
    g = torch.full((20000,), beside, device="cuda")
    g[9000] = value
    w, opt = optimizer(tp, [g])
    norm = opt.grad_norm(max_norm=1.0)
    opt.step(1e-2)
    assert not torch.isfinite(norm).any() and int(opt.finite) == 0 and int(opt.steps) == 0
    assert (w[0] == 0).all()


def test_norm_of_zeros(tp):
    _, opt = optimizer(tp, [torch.zeros(10000, device="cuda"), torch.full((3,), -0.0, device="cuda")])
    assert float(opt.grad_norm(max_norm=1.0)) == 0.0
    assert int(opt.finite) == 1 and float(opt.scale) == 1.0
