"""A state given in part is refused: codes without their scales would decode to
zero, and m without v would be divided by eps (no GPU)."""
import pytest


@pytest.fixture(scope="module")
def whole():
    from tensor_transformer_mlp_shard_gb300 import build
    build.build()
    import tensor_transformer_mlp_shard_gb300 as tp
    return tp.TPAdamW._whole


def test_states_in_part(whole):
    torch = pytest.importorskip("torch")
    codes, scales = [torch.zeros(300, dtype=torch.uint8)], [torch.zeros(2)]
    empty = [torch.zeros(0, dtype=torch.uint8)]
    for a, b in ((None, None), (codes, scales), (codes, None), (None, scales), (empty, None), (empty + codes, None)):
        whole("m", a, "m_scale", b)  # whole, or zero
    codes[0][299], scales[0][1] = 3, 0.5
    whole("m", codes, "m_scale", scales)
    with pytest.raises(ValueError, match="m_scale: required with m"):
        whole("m", empty + codes, "m_scale", None)
    with pytest.raises(ValueError, match="m: required with m_scale"):
        whole("m", None, "m_scale", scales)
    with pytest.raises(ValueError, match="v: required with m"):
        whole("m", [torch.ones(3)], "v", None)
    with pytest.raises(ValueError, match="m: required with v"):
        whole("m", None, "v", [torch.ones(3)])
