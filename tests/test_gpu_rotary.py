"""Rotary positions of the QKV shards against the fp64 oracle."""
import numpy as np
import pytest
import torch

from attention_cases import HALF_STEP, check, cuda_i32, rotation_bound, same_bits, values
from oracle import attention as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tp():
    import tensor_transformer_mlp_shard_gb300 as tp
    return tp


def run(tp, S, B, heads, kv, D, T=1, dtype="bf16", grouped=False, positions=None, place=False, back=False, poke=None,
        **rope):
    rng = np.random.default_rng(S * 131 + heads * 17 + D)
    r = tp.Rope(**rope)
    h = tp.TPRotary(S, B, heads, kv, D, T=T, dtype=dtype, grouped=grouped, rope=r)
    M, hq, hk = S * B, heads // T, kv // T
    dim = D if rope.get("dim") is None else rope["dim"]
    f, a = ref.rope_frequencies(dim, **{k: v for k, v in rope.items() if k not in ("dim", "interleaved")}) if dim else \
        (np.zeros(0), 1.0)
    pairs = rope.get("interleaved", False)
    at = np.arange(M) // B if positions is None else np.asarray(positions)
    x, xf = zip(*[values(rng, (M, (hq + 2 * hk) * D), dtype) for _ in range(T)])
    if poke:
        for t in x:
            poke(t.view(M, hq + 2 * hk, D))
    kept = [t.clone() for t in x]
    y = None if place else [torch.full_like(t, float("nan")) for t in x]
    kw = {} if positions is None else {"positions": cuda_i32(positions)}
    (h.bwd if back else h.fwd)(list(x), y, **kw)
    torch.cuda.synchronize()
    out = x if place else y
    qc, kc, vc = ref.qkv_columns(hq, hk, grouped)
    for t in range(T):
        got = out[t].view(M, hq + 2 * hk, D)
        was = kept[t].view(M, hq + 2 * hk, D)
        assert same_bits(got[:, vc], was[:, vc])
        assert same_bits(got[:, qc + kc][:, :, dim:], was[:, qc + kc][:, :, dim:])
        if (at < 0).any():
            assert same_bits(got[torch.from_numpy(at < 0).cuda()], was[torch.from_numpy(at < 0).cuda()])
        if not poke:
            src = xf[t].reshape(M, hq + 2 * hk, D)[:, qc + kc]
            want = ref.rotate(src, at, f, a, pairs, back)
            bound = rotation_bound(src, want, f, a, HALF_STEP[dtype], pairs)
            check(got[:, qc + kc], want, bound, f"shard {t}")
        if not place:
            assert same_bits(x[t], kept[t])
    return out


SHAPES = [  # S, B, heads, kv, D, T
    (1, 1, 1, 1, 8, 1), (1, 1, 32, 8, 128, 1), (5, 3, 12, 4, 80, 2), (33, 1, 8, 8, 64, 4), (3, 2, 6, 2, 256, 1),
    (7, 1, 16, 16, 72, 16), (700, 2, 8, 2, 40, 2), (2501, 1, 4, 1, 128, 1),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_forward_and_back(tp, shape, dtype, interleaved):
    S, B, heads, kv, D, T = shape
    for grouped in (False, True):
        for place in (False, True):
            run(tp, S, B, heads, kv, D, T, dtype, grouped, place=place, back=place != grouped, interleaved=interleaved)


# part of the head: halves of 8, 12, 4, 9, 1 and 0 pairs (chunks of 8, 4 and 1 elements)
@pytest.mark.parametrize("dim", [16, 24, 8, 18, 2, 0, 42])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_part_of_the_head(tp, dim, dtype, interleaved):
    for place in (False, True):
        run(tp, 9, 2, 6, 2, 48, 2, dtype, dim == 24, place=place, dim=dim, interleaved=interleaved)


@pytest.mark.parametrize("rope", [
    dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0, base=500000.0),
    dict(scaling="parts", factor=16.0, original=4096), dict(scaling="parts", factor=8.0, original=8192, fast=4.0,
                                                            attention_factor=1.0, base=500000.0),
    dict(scaling="ntk", factor=2.0, dim=2), dict(attention_factor=0.7, interleaved=True),
])
def test_scaling(tp, rope):
    for back in (False, True):
        run(tp, 130, 2, 4, 2, 64, 1, "f32", positions=(np.arange(260) * 37) % 5000, back=back, **rope)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_negative_positions(tp, interleaved):
    """Angles stay exact wherever the token is; padding stays as it was."""
    at = [0, 1, 2 ** 31 - 1, 2 ** 30 + 7, 1_000_003, -1, 16_777_217, 2 ** 24 + 3, -2 ** 31, 131_071, 99_999_999]
    for place in (False, True):
        run(tp, len(at), 1, 4, 2, 128, 1, "f32", positions=at, place=place, interleaved=interleaved)
        run(tp, len(at), 1, 4, 2, 128, 2, "bf16", positions=at, place=place, grouped=True, interleaved=interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_what_is_not_rotated_may_be_anything(tp, interleaved, dtype):
    """Infinities and NaN behind the rotated part and in the values pass unchanged."""
    def poke(x):
        x[:, :, 20:] = float("inf")
        x[:, -1] = float("nan")
    for place in (False, True):
        run(tp, 6, 1, 2, 1, 32, 1, dtype, place=place, dim=20, interleaved=interleaved, poke=poke)


def test_gradient_is_the_transpose(tp):
    """<dY, R X> = <R' dY, X>, and the gradient against central differences."""
    rng = np.random.default_rng(5)
    S, B, heads, kv, D = 6, 2, 4, 2, 24
    h = tp.TPRotary(S, B, heads, kv, D, dtype="f32", rope=tp.Rope(dim=16, scaling="parts", factor=4.0, original=64))
    n = (heads + 2 * kv) * D
    x, xf = values(rng, (S * B, n), "f32")
    dy, dyf = values(rng, (S * B, n), "f32")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    h.fwd(x, y)
    h.bwd(dy, dx)
    size = 1.2 * np.abs(xf).sum() * np.abs(dyf).max() * 2.0 ** -20
    assert abs((y.double().cpu().numpy() * dyf).sum() - (dx.double().cpu().numpy() * xf).sum()) <= size
    step = 2.0 ** -4
    for i, j in ((0, 0), (3, 9), (11, 100), (7, 5 * D + 3), (5, 7 * D + 23)):
        up, down = x.clone(), x.clone()
        up[i, j] += step
        down[i, j] -= step
        h.fwd(up)
        h.fwd(down)
        slope = float(((up.double() - down.double()) / (up.new_tensor(2 * step).double()) * dy.double()).sum())
        # fp32 values up to ~6 with errors of 2^-21 of them, over a step of 2^-4, weighed by |dy| of two elements
        assert abs(slope - float(dx[i, j])) <= 6 * 2.0 ** -21 * 2.0 ** 4 * 4 * 4


def test_one_tensor_or_a_list(tp):
    h = tp.TPRotary(10, 1, 8, 4, 32, T=4)
    x = torch.randn(4, 10, 16 // 4 * 32, device="cuda").bfloat16()
    a, b = torch.empty_like(x), torch.empty_like(x)
    h.fwd(x, a)
    h.fwd(list(x.unbind(0)), list(b.unbind(0)))
    assert same_bits(a, b)


def test_stream_and_graph(tp):
    h = tp.TPRotary(300, 1, 8, 4, 64)
    x = torch.randn(300, 16 * 64, device="cuda").bfloat16()
    want, got = torch.empty_like(x), torch.empty_like(x)
    h.fwd(x, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        h.fwd(x, got)
    side.synchronize()
    assert same_bits(want, got)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h.fwd(x, got)
        h.bwd(got)
    x2 = torch.randn(300, 16 * 64, device="cuda").bfloat16()
    x.copy_(x2)
    g.replay()
    h.fwd(x2, want)
    h.bwd(want)
    torch.cuda.synchronize()
    assert same_bits(want, got)


def test_no_tokens(tp):
    h = tp.TPRotary(0, 4, 8, 4, 64)
    h.fwd(torch.empty(0, 16 * 64, device="cuda", dtype=torch.bfloat16))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,dim", [(200, 138), (128, 98), (256, 250), (72, 70), (40, 6)])
def test_halves_of_any_width(tp, dtype, D, dim):
    """Halves that are not whole chunks, heads over several rounds of a block's threads, several tokens a block."""
    for S, grouped, place, T in ((3, False, True, 2), (700, True, False, 1), (1301, False, True, 4)):
        run(tp, S, 1, 48 if S == 3 else 12, 16 if S == 3 else 4, D, T, dtype, grouped, place=place, back=grouped, dim=dim)
