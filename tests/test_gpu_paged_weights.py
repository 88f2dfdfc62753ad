"""Decode attention where one position dominates a softmax and its value says nothing: the output is made of
the small weights, which have to be as precise as the others."""
import numpy as np
import pytest
import torch

from attention_cases import HALF_STEP, TORCH, check, cuda_i32, e4m3, table_for
from oracle import attention as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tp():
    import tensor_transformer_mlp_shard_gb300 as tp
    return tp


AMAX = 28.0  # of every key head: codes are numbers times 16


def stored(x, dtype):
    """x as a cache of the type holds it: (CUDA tensor, its numbers in fp64)."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32))
    if dtype == "fp8":
        c = (t * 16).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return c.cuda(), e4m3(c) / 16
    t = t.to(TORCH[dtype])
    return t.cuda(), t.double().numpy()


def bound(o, mag, spread, seen, D, dtype):
    """As decode_bound, but `spread` is of the positions that the output is made of, and what the dominant score
    adds is a constant: its product is one number, exact, so that only its roundings to log2 units and the
    difference's count, six of 2^-24 of 92 at most (64 nats), 2^-14.7 of a weight; with 2^-17 for the weight's two
    parts and 2^-22 for the exponential, 2^-14.  Sums: two or three products follow one another for every 16
    positions of a warp (a few for every 8), four warps to a row of more than 128."""
    rel = 2 * (D + 4) * 2.0 ** -23 * spread + 2.0 ** -14 + ((seen / 8 + 64) * 2.0 ** -23)[:, None]
    err = rel[..., None] * mag
    return err + (np.abs(o) + err) * HALF_STEP[dtype]


def run(tp, rng, lengths, keys, vals, per, dtype, D, page_size=16, capacity=0, window=0, spread_keys=None):
    """keys, vals: [sequence] -> [kv, n, D].  One row a sequence, at its last position; queries begin with 4, a
    quarter of normal numbers follow; the scores' scale is 1."""
    kv = keys[0].shape[0]
    table, pages = table_for(rng, lengths, page_size)
    if capacity > table.shape[1] * page_size:
        wide = np.full((len(lengths), capacity // page_size), -1, dtype=np.int32)
        wide[:, :table.shape[1]] = table
        table = wide
    caches = []
    for parts in (keys, vals, spread_keys or keys):
        x = np.zeros((pages, kv, page_size, D), dtype=np.float32)
        for s, n in enumerate(lengths):
            for p0 in range(0, n, page_size):
                part = parts[s][:, p0:p0 + page_size]
                x[table[s, p0 // page_size], :, :part.shape[1]] = part
        caches.append(stored(x, dtype))
    h = tp.TPPagedAttention(per * kv, kv, D, page_size, pages, dtype=dtype, window=window, scale=1.0, rope=tp.Rope(dim=0))
    rows = len(lengths)
    q = rng.standard_normal((rows, per * kv, D)).astype(np.float32) * 0.25
    q[..., 0] = 4.0
    q = torch.from_numpy(q).to(TORCH[dtype])
    amax = torch.full((kv,), AMAX, device="cuda")
    kw = dict(k_amax=amax, v_amax=amax) if dtype == "fp8" else {}
    o = torch.full((rows, per * kv * D), float("nan"), device="cuda").to(TORCH[dtype])
    at = np.array(lengths) - 1
    h.decode(q.view(rows, -1).cuda(), cuda_i32(at), cuda_i32(table), caches[0][0], caches[1][0], o,
             tp.alloc_workspace(h.workspace_bytes()), **kw)
    assert h.sync_status() == 0
    args = (q.double().numpy(), at, np.arange(rows), table)
    want, mag, _, seen = ref.decode(*args, caches[0][1], caches[1][1], 1.0, window)
    spread = ref.decode(*args, caches[2][1], caches[1][1], 1.0, window)[2]
    check(o, want, bound(want, mag, spread, seen, D, dtype))


def sinks(rng, lengths, kv, D, gap, at):
    """Sequences whose positions at(n) score `gap`, a nat less each, and have values of zero; the others' scores
    are about normal, the first half of their values positive."""
    keys, vals, plain = [], [], []
    for n in lengths:
        k = (0.5 * rng.standard_normal((kv, n, D))).astype(np.float32)
        v = rng.standard_normal((kv, n, D)).astype(np.float32)
        v[..., :D // 2] = np.abs(v[..., :D // 2])
        k[..., 0] = 0.0
        for i in at(n):
            k[:, i], v[:, i] = 0.0, 0.0
        plain.append(k.copy())
        for j, i in enumerate(at(n)):
            k[:, i, 0] = (gap - j) / 4
        keys.append(k)
        vals.append(v)
    return keys, vals, plain


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("gap", [8, 12, 16, 20, 24, 48])
@pytest.mark.parametrize("lengths,capacity,window", [
    ([4000], 0, 0), ([4000], 40000, 0),              # one row, by a cluster and by the list
    ([2, 9, 40, 333], 0, 0), ([2, 9, 40, 333], 40000, 0),
    ([100, 17] * 90, 40000, 0),                      # single warps' rows
    ([700, 130, 64] * 8, 0, 0), ([900] * 3, 0, 300),  # (a window that the dominant position has left, or not)
])
def test_a_dominant_position_without_a_value(tp, dtype, gap, lengths, capacity, window):
    for per, D in ((4, 64), (6, 128)):
        for at in (lambda n: [0], lambda n: [n - 1]) if len(lengths) < 20 else (lambda n: [n // 2],):
            rng = np.random.default_rng(gap + D)
            keys, vals, plain = sinks(rng, lengths, 2, D, gap, at)
            run(tp, rng, lengths, keys, vals, per, dtype, D, capacity=capacity, window=window, spread_keys=plain)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("gap", [18, 24, 32])
def test_several_dominant_positions(tp, dtype, gap):
    """The first four, four in as many steps, and pairs that are far above the others."""
    for at in (lambda n: [0, 1, 2, 3], lambda n: [5, 90, 170, 299], lambda n: [40, 41, 100, 101]):
        for capacity in (0, 40000):
            rng = np.random.default_rng(gap)
            keys, vals, plain = sinks(rng, [300, 2000], 2, 64, gap, at)
            run(tp, rng, [300, 2000], keys, vals, 5, dtype, 64, capacity=capacity, spread_keys=plain)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("per", [1, 3, 12])
@pytest.mark.parametrize("D", [32, 96, 192, 256])
def test_a_dominant_position_by_width_and_queries(tp, dtype, per, D):
    for lengths in ([1500, 40], [130] * 100):
        rng = np.random.default_rng(per + D)
        keys, vals, plain = sinks(rng, lengths, 2, D, 20, lambda n: [n // 3])
        run(tp, rng, lengths, keys, vals, per, dtype, D, capacity=6000, spread_keys=plain)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("per", [2, 6, 12])
@pytest.mark.parametrize("scores", [
    [-1.5 * i for i in range(11)],                   # a staircase of 15 nats
    [0] + [-18] * 9, [0, -18] + [-36] * 9, [0, -1, -2, -20, -44] * 3, [-48] * 30 + [-24] * 20 + [0] * 3 + [-48] * 30,
])
def test_every_weight(tp, dtype, per, scores):
    """Each row's value is at one of the scores' positions alone, in a step and across steps."""
    D, n = 64, len(scores)
    rng = np.random.default_rng(per)
    k = np.zeros((2, n, D), dtype=np.float32)
    k[..., 0] = np.array(scores) / 4
    vals = []
    for i in range(n):
        v = np.zeros((2, n, D), dtype=np.float32)
        v[:, i] = rng.standard_normal((2, D)) + 3.0
        vals.append(v)
    for capacity in (0, 40000):
        run(tp, rng, [n] * n, [k] * n, vals, per, dtype, D, spread_keys=[0 * k] * n, capacity=capacity)


@pytest.mark.parametrize("per", [1, 5, 8, 12])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_fp32_products_to_their_last_digits(tp, per, D):
    """Scores of one product each, their mantissas just below a step of eleven bits: two positions a row, the
    first's weight is the output.  It is off by 2^-21 of the scores (64) for the products and, for both scores'
    sums and roundings to log2 units (92), four of 2^-24, times at most 1/4; its own products and sums add 2^-20."""
    rng = np.random.default_rng(per)
    rows = 64
    h = tp.TPPagedAttention(per, 1, D, 16, rows, dtype="f32", scale=64.0, rope=tp.Rope(dim=0))
    below = 2.0 ** -10 - rng.integers(1, 8, rows) * 2.0 ** -23
    x = np.float32(1 + rng.integers(0, 4, rows) * 2.0 ** -10 + below)
    q = np.zeros((rows, per, D), dtype=np.float32)
    q[..., 0] = x[:, None]
    K = np.zeros((rows, 1, 16, D), dtype=np.float32)
    V = K.copy()
    K[:, 0, 0, 0] = x
    K[:, 0, 1, 0] = np.float32(np.round(x.astype(np.float64) * 2 ** 10) / 2 ** 10 - rng.integers(0, 3, rows) * 2.0 ** -8)
    V[:, 0, 0] = 1.0
    o = torch.empty(rows, per * D, device="cuda")
    h.decode(torch.from_numpy(q).view(rows, -1).cuda(), cuda_i32([1] * rows), cuda_i32(np.arange(rows)[:, None]),
             torch.from_numpy(K).cuda(), torch.from_numpy(V).cuda(), o, tp.alloc_workspace(h.workspace_bytes()))
    score = 64.0 * x.astype(np.float64)[:, None] * K[:, 0, :2, 0].astype(np.float64)
    want = 1.0 / (1.0 + np.exp(score[:, 1] - score[:, 0]))
    off = np.abs(o.double().cpu().numpy() - want[:, None])
    assert off.max() <= 0.25 * (64 * 2.0 ** -21 + 4 * 92 * 2.0 ** -24 * np.log(2)) + 2.0 ** -20


@pytest.mark.parametrize("per", [1, 4, 5, 12])
@pytest.mark.parametrize("capacity", [1, 200])
def test_fp32_numbers_at_the_ends_of_their_range(tp, per, capacity):
    """NaN with its mark in the last place, and the largest numbers, in keys, queries and values."""
    D, top = 64, float(np.finfo(np.float32).max)
    h = tp.TPPagedAttention(per, 1, D, 16, 6, dtype="f32", scale=1.0, rope=tp.Rope(dim=0))
    K, V = np.zeros((6, 1, 16, D), dtype=np.float32), np.ones((6, 1, 16, D), dtype=np.float32)
    q = np.zeros((6, per, D), dtype=np.float32)
    q[0, :, 7] = -1.0                                    # NaN times a negative number
    K[0, 0, 3, 7] = np.array(0x7f800001, dtype=np.uint32).view(np.float32)
    K[1, 0, 3, 9], q[1, :, 9] = top, 2.0 ** -125         # scores of 8 and 0
    K[2, 0, 3, 9], q[2, :, 9] = 2.0 ** -125, -top        # of -8 and 0
    K[3, 0, 3, 9], q[3, :, 9] = -top, 1.0                # one weighs nothing
    K[4, 0, 3, 9], q[4, :, 9] = float("-inf"), 1.0
    V[5, 0, 3] = top                                     # a quarter of the largest number
    V[:5, 0, 3] = 3.0
    V[5, 0, :3] = 0.0
    table = np.full((6, capacity), -1, dtype=np.int32)
    table[:, 0] = np.arange(6)
    o = torch.empty(6, per * D, device="cuda")
    h.decode(torch.from_numpy(q).view(6, -1).cuda(), cuda_i32([3] * 6), cuda_i32(table), torch.from_numpy(K).cuda(),
             torch.from_numpy(V).cuda(), o, tp.alloc_workspace(h.workspace_bytes()))
    o = o.double().cpu().numpy()
    assert np.isnan(o[0]).all()
    for row, score in ((1, 8.0), (2, -8.0)):
        w = 1.0 / (1.0 + 3.0 * np.exp(-score))
        # scores of 8 to 2^-19 of themselves, products and sums to 2^-19
        assert np.abs(o[row] / (1.0 + 2.0 * w) - 1.0).max() <= 8 * 2.0 ** -19 + 2.0 ** -19
    assert (o[3] == 1.0).all() and (o[4] == 1.0).all()
    assert np.abs(o[5] / (top / 4) - 1.0).max() <= 2.0 ** -19


@pytest.mark.parametrize("v_amax", [2.0 ** -99, 2.0 ** -90, 2.9e38])
@pytest.mark.parametrize("lengths,capacity", [([3000, 60], 0), ([3000, 60], 40000), ([90] * 400, 40000), ([30000], 0)])
def test_value_scales_at_the_ends_of_their_range(tp, v_amax, lengths, capacity):
    """Many equal weights, and a dominant position without a value before them, over values as small or large as
    their calibration may be."""
    rng = np.random.default_rng(3)
    D, kv, per, rows = 64, 2, 4, len(lengths)
    table, pages = table_for(rng, lengths, 16)
    if capacity > table.shape[1] * 16:
        table = np.pad(table, ((0, 0), (0, capacity // 16 - table.shape[1])), constant_values=-1)
    h = tp.TPPagedAttention(per * kv, kv, D, 16, pages, dtype="fp8", scale=1.0, rope=tp.Rope(dim=0))
    amax = torch.full((kv,), v_amax, device="cuda")
    codes = torch.from_numpy(rng.integers(0x30, 0x78, (pages, kv, 16, D)).astype(np.uint8))   # 0.5 to 256
    scale = float(np.float32(448) / np.float32(v_amax))
    q = torch.zeros(rows, per * kv * D, dtype=torch.bfloat16)
    q.view(rows, -1, D)[..., 0] = 4.0
    for gap in (0, 20, 40):
        K = torch.zeros(pages, kv, 16, D)
        V = codes.clone()
        if gap:
            K[table[:, 0], :, 0, 0] = gap / 4
            V[table[:, 0], :, 0] = 0
        K = (K * 16).to(torch.float8_e4m3fn).view(torch.uint8)
        o = torch.empty(rows, per * kv * D, dtype=torch.bfloat16, device="cuda")
        at = np.array(lengths) - 1
        h.decode(q.cuda(), cuda_i32(at), cuda_i32(table), K.cuda(), V.cuda(), o, tp.alloc_workspace(h.workspace_bytes()),
                 k_amax=torch.full((kv,), AMAX, device="cuda"), v_amax=amax)
        assert h.sync_status() == 0
        want, mag, _, seen = ref.decode(q.view(rows, -1, D).double().numpy(), at, np.arange(rows), table, e4m3(K) / 16,
                                        e4m3(V) / scale, 1.0)
        # (the outputs at 2^-99 and 40 nats are 2^-148: bf16's own steps end at 2^-133, half of one is 2^-134)
        check(o, want, bound(want, mag, np.zeros(want.shape[:2]), seen, D, "fp8") + 2.0 ** -134)
