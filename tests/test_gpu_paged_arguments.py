"""Calls that the other tests do not make: arrays that a type has no use for, numbers that are none, launches in plain
stream order."""
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


@pytest.mark.parametrize("capacity", [1, 400])   # clusters; single warps of the list, its shares and its join
@pytest.mark.parametrize("gap", [0, 30])
def test_codes_that_are_not_numbers(capacity, gap):
    """NaN codes in keys and values that a row sees, and infinite and NaN queries, beside a dominant position or not."""
    import tensor_transformer_mlp_shard_gb300 as tp
    D, per, kv, rows = 64, 4, 2, 120
    rng = np.random.default_rng(1)
    lengths = [70] * (rows - 1) + [3000 if capacity > 1 else 70]
    table, pages = table_for(rng, lengths, 16)
    if capacity > table.shape[1]:
        table = np.pad(table, ((0, 0), (0, capacity - table.shape[1])), constant_values=-1)
    h = tp.TPPagedAttention(per * kv, kv, D, 16, pages, dtype="fp8", scale=1.0)
    K = (torch.randn(h.cache_shape) * 8).to(torch.float8_e4m3fn)
    V = (torch.randn(h.cache_shape) * 8).to(torch.float8_e4m3fn)
    K, V = K.view(torch.uint8), V.view(torch.uint8)
    K[..., 0] = 0
    K[table[:, 1], :, 3, 0] = int(torch.tensor(16.0 * gap / 4).to(torch.float8_e4m3fn).view(torch.uint8))
    q = (torch.randn(rows, per * kv, D) * 0.1).bfloat16()
    q[..., 0] = 4.0
    clean = (K.clone(), V.clone(), q.clone())
    last = lengths[-1] // 16 - 1
    V[table[1, 2], 0, 5, 7] = 0x7F
    V[table[rows - 1, last], 1, 5, 9] = 0xFF
    K[table[2, 0], 1, 15, 3] = 0x7F
    q[3, 1, 5] = float("nan")
    q[4, 6, 5] = float("inf")
    amax = torch.full((kv,), 28.0, device="cuda")
    out = []
    for k, v, x in (clean, (K, V, q)):
        o = torch.full((rows, per * kv * D), 9.0, dtype=torch.bfloat16, device="cuda")
        h.decode(x.view(rows, -1).cuda(), cuda_i32(np.array(lengths) - 1), cuda_i32(table), k.cuda(), v.cuda(), o,
                 tp.alloc_workspace(h.workspace_bytes()), k_amax=amax, v_amax=amax)
        assert h.sync_status() == 0
        out.append(o.view(rows, per * kv, D).cpu())
    good, o = out
    assert torch.isfinite(good).all()
    bad = torch.zeros(rows, per * kv, D, dtype=torch.bool)
    bad[1, :per, 7] = bad[rows - 1, per:, 9] = bad[2, per:] = bad[3, 1] = bad[4, 6] = True
    assert torch.isnan(o[bad]).all()
    assert same_bits(o[~bad], good[~bad])


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
def test_launch_overlap_changes_no_kernel_s_results(dtype):
    """Rotation, append and decode by clusters, one behind the other, in plain stream order and overlapped."""
    import tensor_transformer_mlp_shard_gb300 as tp
    act, n = TORCH[dtype], 300
    h = tp.TPPagedAttention(8, 2, 64, 16, 19, dtype=dtype)
    r = tp.TPRotary(n, 1, 8, 2, 64, dtype="f32" if dtype == "f32" else "bf16")
    x0 = torch.randn(n, 12 * 64, device="cuda").to(act)
    at, table = cuda_i32(np.arange(n)), cuda_i32(np.arange(19)[None])
    seq, last = torch.zeros(n, dtype=torch.int32, device="cuda"), cuda_i32([n - 1])
    amax = dict(k_amax=torch.full((2,), 6.0, device="cuda"), v_amax=torch.full((2,), 6.0, device="cuda")) if dtype == "fp8" else {}
    ws, got = tp.alloc_workspace(h.workspace_bytes()), []
    for on in (True, False):
        tp.set_launch_overlap(on)
        try:
            for _ in range(3):
                x = x0.clone()
                K, V = (torch.zeros(h.cache_shape, dtype=h.cache_dtype, device="cuda") for _ in range(2))
                q, o = torch.zeros(n, 8 * 64, dtype=act, device="cuda"), torch.zeros(1, 8 * 64, dtype=act, device="cuda")
                r.fwd(x)
                h.append(x, at, table, K, V, q, sequences=seq, **amax)
                h.decode(q[n - 1:], last, table, K, V, o, ws, **amax)
                r.bwd(x)
                got.append((x, K, V, q, o))
        finally:
            tp.set_launch_overlap(True)
    torch.cuda.synchronize()
    assert h.sync_status() == 0 and bool(got[0][4].any())
    for other in got[1:]:
        assert all(same_bits(a, b) for a, b in zip(got[0], other))


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("cols", [3, 4000])
@pytest.mark.parametrize("window", [1, 2, 17, 2 ** 31 - 1])
def test_padding_at_any_negative_position_with_a_window(dtype, cols, window):
    """The first position that a row sees, p - window + 1, does not exist for the smallest int32."""
    import tensor_transformer_mlp_shard_gb300 as tp
    h = tp.TPPagedAttention(4, 2, 32, 16, 3, dtype=dtype, window=window)
    act = TORCH[dtype]
    K, V = (torch.ones(h.cache_shape, device="cuda").to(h.cache_dtype) for _ in range(2))
    at = cuda_i32([-1, -2 ** 31, 40, -2 ** 31 + 1, -17])
    table = torch.full((5, cols), -1, dtype=torch.int32, device="cuda")
    table[2, :3] = cuda_i32([0, 1, 2])
    q = torch.randn(5, 4 * 32, device="cuda").to(act)
    o = torch.full_like(q, 5.0)
    amax = dict(k_amax=torch.ones(2, device="cuda"), v_amax=torch.ones(2, device="cuda")) if dtype == "fp8" else {}
    h.decode(q, at, table, K, V, o, tp.alloc_workspace(h.workspace_bytes()), **amax)
    assert h.sync_status() == 0
    assert not bool(o[[0, 1, 3, 4]].any()) and bool((o[2] != 0).all()) and bool(torch.isfinite(o[2]).all())
