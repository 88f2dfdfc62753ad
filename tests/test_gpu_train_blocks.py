"""The training example runs the block norm, the MLP and AdamW together: its
gradients agree with autograd in fp64, captured steps are eager steps, and
training reduces the loss with states of either width."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from tensor_transformer_mlp_shard_gb300 import build
    build.build()
    import train_blocks
    return train_blocks


def reference(s):
    """Loss and parameter gradients of a stack by fp64 autograd."""
    names, leaves = [], []

    def leaf(t, name):
        v = t.detach().double().requires_grad_()
        names.append(name)
        leaves.append(v)
        return v

    def rms(x, w):
        return x * (x.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w

    nw = [leaf(w, f"norm{i}") for i, w in enumerate(s.norm_w)]
    x = s.x.double()
    for i, l in enumerate(s.layers):
        n = rms(x, nw[i])
        f = leaf(l["b2"], f"b2.{i}")
        for k, (w1, b1, w2) in enumerate(zip(l["W1"], l["b1"], l["W2"])):
            h = n @ leaf(w1, f"W1.{i}.{k}").T + leaf(b1, f"b1.{i}.{k}")
            f = f + torch.nn.functional.gelu(h, approximate="tanh") @ leaf(w2, f"W2.{i}.{k}").T
        x = x + leaf(l["gain"], f"gain.{i}") * rms(f, leaf(l["post_w"], f"post.{i}"))
    loss = (rms(x, nw[-1]) - s.target.double()).square().mean()
    return loss, dict(zip(names, torch.autograd.grad(loss, leaves)))


def test_gradients(ex):
    """bf16 rounds every activation by 2^-8: over the chain of 2 blocks and
    their backward some ten roundings stand between a gradient and its value,
    which average over its sums: 3 % of its norm."""
    s = ex.BlockStack(blocks=2, seed=3)
    s.forward()
    s.backward()
    loss, ref = reference(s)
    assert abs(float(s.loss) - float(loss.detach())) < 1e-2 * float(loss.detach())
    got = {f"norm{i}": g for i, g in enumerate(s.d_norm_w)}
    for i, l in enumerate(s.layers):
        got.update({f"b2.{i}": l["db2"], f"gain.{i}": l["dgain"], f"post.{i}": l["dpost_w"]})
        for k in range(len(l["W1"])):
            got.update({f"W1.{i}.{k}": l["dW1"][k], f"b1.{i}.{k}": l["db1"][k], f"W2.{i}.{k}": l["dW2"][k]})
    assert got.keys() == ref.keys()
    for k in ref:
        err = float((got[k].double() - ref[k]).norm() / ref[k].norm())
        assert err < 0.03, (k, err)


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_steps_are_eager_steps(ex, bits):
    a, b = (ex.BlockStack(blocks=2, state_bits=bits, seed=1) for _ in range(2))
    a.step()
    b.step()
    graph = b.capture()
    for _ in range(4):
        a.step()
        graph.replay()
    torch.cuda.synchronize()
    assert int(a.opt.steps) == int(b.opt.steps) == 5
    for p, q in zip(a.opt.params, b.opt.params):
        assert torch.equal(p, q)


@pytest.mark.parametrize("bits", [8, 32])
def test_training_reduces_the_loss(ex, bits):
    s = ex.BlockStack(blocks=3, state_bits=bits)
    s.step()
    start = float(s.loss)
    graph = s.capture()
    for _ in range(100):
        graph.replay()
    torch.cuda.synchronize()
    assert int(s.opt.finite) == 1 and float(s.loss) < 0.8 * start, (start, float(s.loss))


def test_launch_overlap_changes_nothing(ex):
    """Kernels that start while the one before them ends give the results of
    plain stream order."""
    import tensor_transformer_mlp_shard_gb300 as tp
    a, b = (ex.BlockStack(blocks=3, seed=2) for _ in range(2))
    try:
        for on, s in ((False, a), (True, b)):
            tp.set_launch_overlap(on)
            for _ in range(6):
                s.step()
            torch.cuda.synchronize()
    finally:
        tp.set_launch_overlap(True)
    for p, q in zip(a.opt.params, b.opt.params):
        assert torch.equal(p, q)
    assert torch.equal(a.out, b.out)
