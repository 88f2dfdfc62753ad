"""The 8-bit step's square roots are fp32's, rounded correctly.

A block of equal gradients, from states of zero, leaves the scale (root / 448)
of its one root: v = fl(fl(c2 g) g), scale = fl(fl(sqrt(v)) fl(1 / 448)).
IEEE fp32 on the host gives each of them exactly, so nothing may differ.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BETA2 = 0.95


def test_roots_are_rounded_correctly():
    import tensor_transformer_mlp_shard_gb300 as tp
    from tensor_transformer_mlp_shard_gb300 import build
    build.build()
    # 2^17 mantissas, the exponents of v from 2^-120 to 2^60: on both sides of
    # 2^-100, where the kernel's own root begins
    rng = np.random.default_rng(11)
    g = (rng.uniform(1.0, 2.0, 1 << 17) * 2.0 ** rng.integers(-58, 32, 1 << 17)).astype(np.float32)
    grad = torch.from_numpy(g).cuda().repeat_interleave(256)
    w = torch.zeros_like(grad)
    opt = tp.TPAdamW([w], [grad], state_bits=8, beta1=0.9, beta2=BETA2)
    opt.step(1e-3, step=1)
    c2 = np.float32(1.0 - BETA2)
    root = np.sqrt((c2 * g) * g)
    assert root.dtype == np.float32
    want = root * (np.float32(1.0) / np.float32(448.0))
    got = opt.v_scale[0].cpu().numpy()
    assert np.array_equal(got, want), int((got != want).sum())
