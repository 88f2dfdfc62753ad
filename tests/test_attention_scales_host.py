"""Scales and factors that stand for something else, or that fp32 does not hold (no GPU)."""
import pytest


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_shard_gb300 import build
    build.build()
    import tensor_transformer_mlp_shard_gb300 as tp
    return tp


@pytest.mark.parametrize("factor", [0, 0.0, -0.0])
def test_an_attention_factor_of_zero_is_no_default(tp, factor):
    """In the descriptor 0 stands for the default, which is None here."""
    with pytest.raises(ValueError, match="attention_factor"):
        tp.Rope(attention_factor=factor)
    assert tp.Rope().desc(64).attention_factor == 0.0
    assert tp.Rope(attention_factor=0.5).desc(64).attention_factor == 0.5


PAGED = dict(heads=8, kv_heads=4, head_dim=64, page_size=16, pages=10, T=2)


@pytest.mark.parametrize("scale", [1e-46, -1e-50, 5e-324])
def test_a_scale_below_fp32_is_no_default(tp, scale):
    """Zero in the descriptor, which stands for 1 / sqrt(head_dim)."""
    with pytest.raises(ValueError, match="scale"):
        tp.TPPagedAttention(**PAGED, scale=scale)
    tp.TPPagedAttention(**PAGED, scale=1e-44)


@pytest.mark.parametrize("scale", [2.4e38, -3e38, 3.4028e38])
def test_a_scale_beyond_base_two(tp, scale):
    """Scores of zero would become infinity times zero."""
    with pytest.raises(tp.TpError) as e:
        tp.TPPagedAttention(**PAGED, scale=scale)
    assert e.value.status == 1
    tp.TPPagedAttention(**PAGED, scale=2.3e38 if scale > 0 else -2.3e38)


def test_scales_of_any_number_type(tp):
    import numpy as np
    for scale in (1, np.float32(0.5), np.float16(0.5), np.int64(2)):
        tp.TPPagedAttention(**PAGED, scale=scale)
