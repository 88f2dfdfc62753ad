"""Calls of the C entry points that the binding does not make."""
import numpy as np
import pytest
import torch

from attention_cases import TORCH, cuda_i32, same_bits, table_for

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", [[100, 3], [9000, 5], [60] * 300])   # clusters; the list and its join; single warps
def test_calibration_is_of_codes_alone(dtype, lengths):
    """k_amax and v_amax change nothing where the cache holds numbers."""
    import tensor_transformer_mlp_shard_gb300 as tp
    from tensor_transformer_mlp_shard_gb300.binding import _pack1, _stream
    table, pages = table_for(np.random.default_rng(0), lengths, 16)
    cols = max(table.shape[1], 100)
    table = np.pad(table, ((0, 0), (0, cols - table.shape[1])), constant_values=-1)
    h = tp.TPPagedAttention(8, 2, 64, 16, pages, dtype=dtype)
    n, act = len(lengths), TORCH[dtype]
    K, V = (torch.randn(h.cache_shape, device="cuda").to(act) for _ in range(2))
    K2, V2 = K.clone(), V.clone()
    x = torch.randn(n, 12 * 64, device="cuda").to(act)
    q, q2 = (torch.zeros(n, 8 * 64, device="cuda", dtype=act) for _ in range(2))
    at, table, ws = cuda_i32(np.array(lengths) - 1), cuda_i32(table), tp.alloc_workspace(h.workspace_bytes())
    h.append(x, at, table, K, V, q)
    o, o2 = torch.empty_like(q), torch.empty_like(q)
    h.decode(q, at, table, K, V, o, ws)
    amax = torch.full((2,), 3.0, device="cuda")
    one = lambda t: _pack1(t.data_ptr())  # noqa: E731
    rows = (at.data_ptr(), None, n, table.data_ptr(), n, cols, amax.data_ptr(), amax.data_ptr())
    assert tp.lib().tp_paged_append(h._h, one(x), *rows, one(q2), one(K2), one(V2), _stream(None)) == 0
    assert tp.lib().tp_paged_decode(h._h, one(q2), *rows, one(K2), one(V2), one(o2), ws.data_ptr(), ws.numel(), _stream(None)) == 0
    assert h.sync_status() == 0
    assert same_bits(q, q2) and same_bits(K, K2) and same_bits(V, V2) and same_bits(o, o2)
