"""The paged cache and decode attention against the fp64 oracle."""
import numpy as np
import pytest
import torch

from attention_cases import (Cache, HALF_STEP, TORCH, check, cuda_i32, decode_bound, decode_case, e4m3, rotation_bound,
                             same_bits, table_for, values)
from oracle import attention as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tp():
    import tensor_transformer_mlp_shard_gb300 as tp
    return tp


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def append_case(tp, positions, sequences, table, pages, page_size, heads, kv, D, T=1, dtype="bf16", grouped=False,
                good=True, **rope):
    rng = np.random.default_rng(heads * 7 + D + len(positions))
    h = tp.TPPagedAttention(heads, kv, D, page_size, pages, T=T, dtype=dtype, grouped=grouped, rope=tp.Rope(**rope))
    n, hq, hk = len(positions), heads // T, kv // T
    dim = D if rope.get("dim") is None else rope["dim"]
    f, a = ref.rope_frequencies(dim, **{k: v for k, v in rope.items() if k not in ("dim", "interleaved")}) if dim else \
        (np.zeros(0), 1.0)
    pairs = rope.get("interleaved", False)
    x, xf = zip(*[values(rng, (n, (hq + 2 * hk) * D), dtype) for _ in range(T)])
    full = 0xA5 if dtype == "fp8" else float("nan")
    K = [torch.full(h.cache_shape, full, dtype=h.cache_dtype, device="cuda") for _ in range(T)]
    V = [k.clone() for k in K]
    Q = [torch.full((n, hq * D), float("nan"), dtype=TORCH[dtype], device="cuda") for _ in range(T)]
    before = [t.clone() for t in (K[0], Q[0])]
    kw, scale = {}, [None, None]
    if dtype == "fp8":
        # one head's amax is below what it meets (saturation), one is zero (scale 1)
        amax = [(2.0 + rng.random(kv)).astype(np.float32) for _ in range(2)]
        amax[0][-1], amax[1][0] = 0.5, 0.0
        kw = {"k_amax": torch.from_numpy(amax[0]).cuda(), "v_amax": torch.from_numpy(amax[1]).cuda()}
        scale = [np.where(m > 0, np.float32(448) / np.where(m > 0, m, 1), np.float32(1)).astype(np.float64) for m in amax]
    if sequences is not None:
        kw["sequences"] = cuda_i32(sequences)
    h.append(list(x), cuda_i32(positions), cuda_i32(table), K, V, Q, **kw)
    assert h.sync_status() == (0 if good else 6)
    assert h.sync_status() == 0
    at = ref.slots(positions, np.arange(n) if sequences is None else sequences, np.asarray(table), page_size, pages)
    rows = [j for j in range(n) if at[j] is not None]
    page, off = [at[j][0] for j in rows], [at[j][1] for j in rows]
    qc, kc, vc = ref.qkv_columns(hq, hk, grouped)
    untouched = torch.ones(pages, page_size, dtype=torch.bool)
    untouched[page, off] = False
    left = [j for j in range(n) if at[j] is None]
    for t in range(T):
        src = xf[t].reshape(n, hq + 2 * hk, D)[rows]
        p = np.asarray(positions)[rows]
        want = ref.rotate(src[:, qc], p, f, a, pairs)
        check(Q[t].view(n, hq, D)[rows], want, rotation_bound(src[:, qc], want, f, a, HALF_STEP[dtype], pairs), "Q")
        assert same_bits(Q[t][left], before[1][left])
        wk = ref.rotate(src[:, kc], p, f, a, pairs)
        kb = rotation_bound(src[:, kc], wk, f, a, 0.0 if dtype == "fp8" else HALF_STEP[dtype], pairs)
        for cache, new, bound, s in ((K[t], wk, kb, scale[0]), (V[t], src[:, vc], np.zeros_like(kb), scale[1])):
            assert same_bits(cache.permute(0, 2, 1, 3)[untouched.cuda()],
                             torch.full_like(cache.permute(0, 2, 1, 3)[untouched.cuda()], full))
            got = cache[page, :, off]
            if dtype != "fp8":
                check(got, new, bound, "cache")
                continue
            s = s[t * hk:(t + 1) * hk][None, :, None]
            u = np.clip(new * s, -448.0, 448.0)
            # half a step of the code, after the product's rounding
            err = bound * s + np.abs(u) * 2.0 ** -23
            check(torch.from_numpy(e4m3(got.contiguous())), u, np.maximum((np.abs(u) + err) * 2.0 ** -4, 2.0 ** -10) + err, "codes")
    return h


def ragged(rng, new, past, page_size):
    """Rows of sequences in turn: positions, sequences, table, pages."""
    lengths = [a + b for a, b in zip(new, past)]
    table, pages = table_for(rng, lengths, page_size)
    positions = np.concatenate([np.arange(p, p + k) for k, p in zip(new, past)])
    return positions, np.repeat(np.arange(len(new)), new), table, pages


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", [(1, 1, 16, 1), (12, 4, 80, 2), (8, 8, 64, 8), (10, 2, 256, 1), (32, 8, 128, 4)])
def test_append(tp, dtype, interleaved, shape):
    heads, kv, D, T = shape
    rng = np.random.default_rng(D)
    positions, sequences, table, pages = ragged(rng, [1, 40, 17, 3], [0, 5, 31, 100], 16)
    for grouped in (False, True):
        append_case(tp, positions, sequences, table, pages, 16, heads, kv, D, T, dtype, grouped, interleaved=interleaved)


@pytest.mark.parametrize("dim", [0, 24, 18, 48])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
def test_append_part_of_the_head(tp, dim, dtype):
    rng = np.random.default_rng(dim)
    positions, sequences, table, pages = ragged(rng, [30, 2], [7, 90], 48)
    for interleaved in (False, True):
        append_case(tp, positions, sequences, table, pages, 48, 6, 2, 48, 2, dtype, dim=dim, interleaved=interleaved)


def test_append_many_tokens(tp):
    """Several tokens a block, rows that do not divide by them."""
    rng = np.random.default_rng(2)
    positions, sequences, table, pages = ragged(rng, [5003], [77], 64)
    append_case(tp, positions, sequences, table, pages, 64, 4, 2, 64, 1, scaling="linear", factor=2.0)
    append_case(tp, positions, sequences, table, pages, 64, 4, 2, 64, 2, "fp8", interleaved=True)


def test_append_one_row_a_sequence(tp):
    rng = np.random.default_rng(3)
    table, pages = table_for(rng, [1, 16, 17, 300], 16)
    append_case(tp, [0, 15, 16, 299], None, table, pages, 16, 8, 4, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
def test_append_padding_and_bad_indices(tp, dtype):
    rng = np.random.default_rng(4)
    table, pages = table_for(rng, [40, 40], 16)
    positions = np.array([0, -1, 39, 3, -7, 8])
    append_case(tp, positions, [0, 99, 0, 1, -5, 1], table, pages, 16, 4, 2, 32, 1, dtype)  # padding: no error
    append_case(tp, np.full(4, -1), None, np.zeros((4, 1), np.int32), 1, 16, 4, 2, 32, 1, dtype)
    for sequences, positions in (([0, 2], [1, 1]), ([-1, 1], [1, 1]), ([0, 1], [48, 1]), ([0, 1], [2 ** 31 - 1, 1])):
        append_case(tp, np.array(positions), sequences, table, pages, 16, 4, 2, 32, 1, dtype, good=False)
    for page in (-1, pages, 2 ** 31 - 1, -2 ** 31):
        bad = table.copy()
        bad[0, 1] = page
        append_case(tp, np.array([0, 16, 5]), [0, 0, 1], bad, pages, 16, 4, 2, 32, 1, dtype, good=False)


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
LENGTHS = [1, 2, 15, 16, 17, 63, 64, 65, 0, 130, 1000, 255]


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("shape", [(8, 8, 64, 1), (8, 2, 128, 2), (12, 4, 80, 4), (16, 1, 112, 1), (6, 2, 256, 2), (3, 1, 16, 1),
                                   (5, 1, 192, 1)])
def test_decode(tp, dtype, shape):
    heads, kv, D, T = shape
    decode_case(tp, np.random.default_rng(heads + D), LENGTHS, heads, kv, D, 16, T, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [8, 24, 40, 72, 136, 248])
def test_decode_odd_widths(tp, dtype, D):
    decode_case(tp, np.random.default_rng(D), LENGTHS, 4, 2, D, 32, 1, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("per", [1, 2, 3, 4, 5, 7, 8, 9, 12, 16, 17, 33])
def test_decode_queries_of_a_key_head(tp, dtype, per):
    for D in (64, 128, 256):
        decode_case(tp, np.random.default_rng(per), [70, 1, 200], 2 * per, 2, D, 16, 1, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("page_size", [16, 48, 64, 272])
@pytest.mark.parametrize("window", [0, 1, 16, 50, 10000])
def test_decode_pages_and_windows(tp, dtype, page_size, window):
    decode_case(tp, np.random.default_rng(page_size + window), [1, 47, 48, 49, 500, 333, 0], 8, 2, 64, page_size, 2, dtype, window)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("lengths", [[40000], [9000, 3, 20000], [1] * 400, [100 + 7 * i for i in range(90)]])
def test_decode_split(tp, dtype, lengths):
    """One long row over all blocks, and more (row, head) pairs than blocks."""
    decode_case(tp, np.random.default_rng(len(lengths)), lengths, 8, 4 if len(lengths) > 50 else 2, 64, 64, 2, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
def test_decode_rows_share_a_sequence(tp, dtype):
    """The tokens of a short prompt, each over what is before it, rows in any order."""
    positions = [0, 5, 6, 7, 99, 98, -1, 20, 64, 63]
    sequences = [0, 1, 1, 1, 0, 0, 77, 1, 0, 0]
    decode_case(tp, np.random.default_rng(6), [100, 30], 4, 2, 64, 16, 1, dtype, sequences=sequences, positions=positions)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("scale,q_std", [(2.0, 8.0), (-0.3, 1.0), (1e-30, 1.0), (0.1, 1e15), (1.0, 1e-30)])
def test_decode_scales(tp, dtype, scale, q_std):
    """Peaked, flat and inverted softmaxes; queries outside fp16's range."""
    decode_case(tp, np.random.default_rng(7), [1, 100, 700], 4, 2, 64, 16, 1, dtype, scale=scale * (1e-15 if q_std == 1e15 else 1),
                q_std=q_std)


def plain(tp, dtype="bf16", n=4, D=64, length=100, **kw):
    """A handle and buffers without a reference."""
    rng = np.random.default_rng(8)
    table, pages = table_for(rng, [length] * n, 16)
    h = tp.TPPagedAttention(8, 2, D, 16, pages, dtype=dtype, **kw)
    act = TORCH[dtype]
    K, V = (torch.randn(h.cache_shape, device="cuda").to(act) for _ in range(2))
    q = torch.randn(n, 8 * D, device="cuda").to(act)
    return h, q, cuda_i32([length - 1] * n), cuda_i32(table), K, V, tp.alloc_workspace(h.workspace_bytes())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_infinities_and_nan(tp, dtype):
    h, q, at, table, K, V, ws = plain(tp, dtype)
    q.fill_(1.0)
    t = table.cpu().numpy()
    K[int(t[0, 2])] = float("-inf")              # positions 32..47 weigh nothing
    for p in t[1]:
        K[int(p)] = float("-inf")                # every score -infinity: zero
    V[int(t[2, 3]), 0, 5, 7] = float("nan")      # a value that is NaN shows in its element of head 0's queries
    K[int(t[3, 1]), 1, 2] = float("nan")         # a score that is NaN: the row of head 1's queries
    K[int(t[3, 0]), 0, 3, 0] = float("inf")      # a score of +infinity: inf - inf
    o = torch.full_like(q, 7.0)
    h.decode(q, at, table, K, V, o, ws)
    assert h.sync_status() == 0
    o = o.view(4, 8, 64).float().cpu()
    assert torch.isfinite(o[0]).all()
    k = K[table[0].long()].double()[:, :, :].permute(1, 0, 2, 3).reshape(2, -1, 64)[:, :100]
    v = V[table[0].long()].double().permute(1, 0, 2, 3).reshape(2, -1, 64)[:, :100]
    w = torch.softmax(k.sum(-1) / 8.0, -1)
    want = torch.einsum("hn,hnd->hd", w, v).repeat_interleave(4, 0).cpu()
    assert (o[0] - want).abs().max() <= 2.0 ** -7
    assert (o[1] == 0).all()
    assert torch.isnan(o[2, :4, 7]).all() and torch.isfinite(o[2, :4, :7]).all() and torch.isfinite(o[2, 4:]).all()
    assert torch.isnan(o[3]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_bad_indices(tp, dtype):
    """Bad rows give zero, bad pages are left out, and both are reported once."""
    h, q, at, table, K, V, ws = plain(tp, dtype, n=5)
    good, o = torch.empty_like(q), torch.full_like(q, 3.0)
    h.decode(q, at, table, K, V, good, ws)
    assert h.sync_status() == 0
    seq = cuda_i32([0, 5, -1, 3, 4])
    far = at.clone()
    far[3] = 16 * table.shape[1]
    h.decode(q, far, table, K, V, o, ws, sequences=seq)
    assert h.sync_status() == 6 and h.sync_status() == 0
    assert same_bits(o[0], good[0]) and same_bits(o[4], good[4]) and (o[1:4] == 0).all()
    for page in (-1, K.shape[0], 2 ** 31 - 1, -2 ** 31):
        bad = table.clone()
        bad[2, 6] = page                          # positions 96..99 of row 2
        h.decode(q, at, bad, K, V, o, ws)
        assert h.sync_status() == 6
        assert same_bits(o[[0, 1, 3, 4]], good[[0, 1, 3, 4]])
        short = at.clone()
        short[2] = 95
        h.decode(q, short, table, K, V, good, ws)
        assert h.sync_status() == 0
        rel = (o[2].float() - good[2].float()).abs().max() / good[2].float().abs().max()
        assert rel <= 2.0 ** -7                   # the same positions, dealt to the warps alike
        h.decode(q, at, table, K, V, good, ws)
    other = tp.TPPagedAttention(8, 2, 64, 16, 10)
    assert other.sync_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
def test_decode_repeats_bit_for_bit_and_in_place(tp, dtype):
    h, args, o, ws, kw = decode_case(tp, np.random.default_rng(9), [3000, 1, 77, 0, 900], 8, 2, 128, 32, 2, dtype)
    for _ in range(3):
        again = [torch.empty_like(x) for x in o]
        ws.fill_(0x7F)
        h.decode(*args, again, ws, **kw)
        assert all(same_bits(a, b) for a, b in zip(o, again))
    h.decode(*args, args[0], ws, **kw)            # over the queries
    assert all(same_bits(a, b) for a, b in zip(o, args[0]))


def test_decode_one_tensor_or_a_list(tp):
    h = tp.TPPagedAttention(8, 4, 64, 16, 12, T=4)
    K, V = (torch.randn(4, *h.cache_shape, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(4, 2, 2 * 64, device="cuda").bfloat16()
    a, b = torch.empty_like(q), torch.empty_like(q)
    at, table, ws = cuda_i32([60, 80]), cuda_i32(np.arange(12).reshape(2, 6)), tp.alloc_workspace(h.workspace_bytes())
    h.decode(q, at, table, K, V, a, ws)
    h.decode(list(q), at, table, list(K), list(V), list(b), ws)
    assert same_bits(a, b)


def test_decode_streams_and_graphs(tp):
    """Two streams with a workspace each, and a captured step replayed on other positions and pages."""
    h, q, at, table, K, V, ws = plain(tp, n=6, D=128, length=3000)
    want, one, two = (torch.empty_like(q) for _ in range(3))
    h.decode(q, at, table, K, V, want, ws)
    ws2 = tp.alloc_workspace(h.workspace_bytes())
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            h.decode(q, at, table, K, V, one, ws)
        with torch.cuda.stream(s2):
            h.decode(q, at, table, K, V, two, ws2)
    torch.cuda.synchronize()
    assert same_bits(want, one) and same_bits(want, two)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h.decode(q, at, table, K, V, one, ws)
    for length in (1, 50, 2999, 0):
        at.fill_(length - 1)
        table.copy_(table.roll(1, 0))
        one.fill_(9.0)
        g.replay()
        h.decode(q, at, table, K, V, two, ws2)
        torch.cuda.synchronize()
        assert same_bits(one, two)
    assert (one == 0).all() and h.sync_status() == 0


def test_launch_overlap_changes_nothing(tp):
    h, q, at, table, K, V, ws = plain(tp, n=3, length=5000)
    a, b = torch.empty_like(q), torch.empty_like(q)
    h.decode(q, at, table, K, V, a, ws)
    tp.set_launch_overlap(False)
    try:
        h.decode(q, at, table, K, V, b, ws)
    finally:
        tp.set_launch_overlap(True)
    assert same_bits(a, b)


def test_far_offsets(tp):
    """Slots whose byte and element offsets pass 32 bits, written and read."""
    pages, D = 70_000, 256                        # 70000 * 4 * 64 * 256 = 4.6e9 elements
    h = tp.TPPagedAttention(4, 4, D, 64, pages, dtype="fp8", rope=tp.Rope(dim=0))
    assert pages * 4 * 64 * D > 2 ** 32
    K, V = (torch.zeros(h.cache_shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    x = torch.randn(1, 12 * D, device="cuda").bfloat16()
    q, o = torch.empty(1, 4 * D, device="cuda", dtype=torch.bfloat16), torch.empty(1, 4 * D, device="cuda", dtype=torch.bfloat16)
    amax = torch.full((4,), 8.0, device="cuda")
    table = cuda_i32([[pages - 1]])
    h.append(x, cuda_i32([0]), table, K, V, q, k_amax=amax, v_amax=amax)
    ws = tp.alloc_workspace(h.workspace_bytes())
    h.decode(q, cuda_i32([0]), table, K, V, o, ws, k_amax=amax, v_amax=amax)
    assert h.sync_status() == 0
    assert bool(V[pages - 1, :, 0].any()) and not bool(V[:pages - 1].any()) and not bool(K[:pages - 1].any())
    v = x[0, 8 * D:].double()
    assert ((o[0].double() - v).abs() <= v.abs() * (2.0 ** -4 + 2.0 ** -7) + 2.0 ** -10 * 8 / 448).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("shape", [(4, 4, 64, 2), (8, 8, 128, 1), (12, 2, 80, 1), (2, 1, 256, 1)])
def test_decode_short_and_long_rows(tp, dtype, shape):
    """More (row, head) pairs than blocks, short rows between long and empty ones."""
    heads, kv, D, T = shape
    rng = np.random.default_rng(D)
    lengths = [int(x) for x in rng.integers(0, 140, size=1200 // kv)]
    for i in (0, 3, 4, 50, 51, 52, 149):
        lengths[i] = 700 + 130 * i
    lengths[5:9] = [128, 129, 127, 1]
    decode_case(tp, rng, lengths, heads, kv, D, 32, T, dtype)
    decode_case(tp, rng, lengths, heads, kv, D, 16, T, dtype, window=40)


@pytest.mark.parametrize("heads", [2, 16])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_infinite_values(tp, dtype, heads):
    """An infinite value leaves its element not finite, of the queries of its head alone, and nothing else; one or
    eight queries a key head."""
    rng = np.random.default_rng(13)
    table, pages = table_for(rng, [50, 50], 16)
    h = tp.TPPagedAttention(heads, 2, 64, 16, pages, dtype=dtype)
    K, V = (torch.randn(h.cache_shape, device="cuda").to(TORCH[dtype]) for _ in range(2))
    q = torch.randn(2, heads * 64, device="cuda").to(TORCH[dtype])
    V[int(table[1, 1]), 1, 4, 9] = float("-inf")
    K[int(table[0, 2]), 0, 3] = float("-inf")     # mixed signs of q: inf - inf
    o = torch.empty_like(q)
    h.decode(q, cuda_i32([49, 49]), cuda_i32(table), K, V, o, tp.alloc_workspace(h.workspace_bytes()))
    o = o.view(2, heads, 64).float().cpu()
    per = heads // 2
    assert torch.isnan(o[0, :per]).all() and torch.isfinite(o[0, per:]).all()
    assert not torch.isfinite(o[1, per:, 9]).any()   # infinite, or NaN: a weight's second part may be zero
    o[1, per:, 9] = 0
    assert torch.isfinite(o[1]).all()


FIRST_CALL = """
import torch, sys
sys.path.insert(0, {root!r})
import tensor_transformer_mlp_shard_gb300 as tp
dt = {dtype!r}
h = tp.TPPagedAttention(8, 2, 64, 16, 12, dtype=dt)
r = tp.TPRotary(3, 1, 8, 2, 64, dtype="f32" if dt == "f32" else "bf16")
act = torch.float32 if dt == "f32" else torch.bfloat16
x = torch.randn(3, 12 * 64, device="cuda").to(act)
K, V = (torch.zeros(h.cache_shape, dtype=h.cache_dtype, device="cuda") for _ in range(2))
q, o = (torch.zeros(3, 8 * 64, dtype=act, device="cuda") for _ in range(2))
at = torch.tensor([0, 40, -1], dtype=torch.int32, device="cuda")
table = torch.arange(9, dtype=torch.int32, device="cuda").view(3, 3)
ws = tp.alloc_workspace(h.workspace_bytes())
a = dict(k_amax=torch.ones(2, device="cuda"), v_amax=torch.ones(2, device="cuda")) if dt == "fp8" else dict()
def step(out):
    h.append(x, at, table, K, V, q, **a)
    h.decode(q, at, table, K, V, out, ws, **a)
    r.fwd(x)
    r.bwd(x)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):          # the process's first calls of these kernels
    step(o)
x0 = x.clone()
g.replay()
torch.cuda.synchronize()
x.copy_(x0)
want = torch.empty_like(o)
step(want)
torch.cuda.synchronize()
assert torch.equal(o, want) and bool(o[1].any()) and not bool(o[2].any()) and h.sync_status() == 0
print("same")
"""


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
def test_first_call_may_be_captured(dtype):
    """No call before the capture: what a kernel needs to be set up is not a stream's work."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(root=root, dtype=dtype)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
def test_the_last_positions(tp, dtype):
    """Positions up to the largest int32, through a window, in a table whose other pages are gone."""
    page_size, window, kv, D = 4096, 70, 2, 32
    cols = 2 ** 31 // page_size
    h = tp.TPPagedAttention(6, kv, D, page_size, 3, dtype=dtype, window=window, rope=tp.Rope(dim=0))
    table = torch.full((2, cols), -1, dtype=torch.int32, device="cuda")
    table[0, cols - 1], table[1, cols - 2], table[1, cols - 1] = 2, 0, 1
    at = [2 ** 31 - 1, (cols - 1) * page_size + 20]      # the second sees the end of a page and the beginning of the next
    rng = np.random.default_rng(14)
    n = window + 1
    amax = dict(k_amax=torch.full((kv,), 5.0, device="cuda"), v_amax=torch.full((kv,), 5.0, device="cuda")) if dtype == "fp8" else {}
    K, V = (torch.full(h.cache_shape, 0x7F if dtype == "fp8" else float("nan"), dtype=h.cache_dtype, device="cuda") for _ in range(2))
    q = torch.empty(n, 6 * D, dtype=TORCH[dtype], device="cuda")
    keys, values_ = [], []
    for s, p in enumerate(at):
        x, xf = values(rng, (n, (6 + 2 * kv) * D), dtype)
        positions = [p - window + 1 + i for i in range(window)] + [-1]
        h.append(x, cuda_i32(positions), table, K, V, q, sequences=cuda_i32([s] * n), **amax)
        keys.append(xf[:window, 6 * D:(6 + kv) * D].reshape(window, kv, D))
        values_.append(xf[:window, (6 + kv) * D:].reshape(window, kv, D))
    q, qf = values(rng, (2, 6 * D), dtype)
    o = torch.empty_like(q)
    h.decode(q, cuda_i32(at), table, K, V, o, tp.alloc_workspace(h.workspace_bytes()), **amax)
    assert h.sync_status() == 0
    for s in range(2):
        Kf, Vf = (x[s].transpose(1, 0, 2)[None] for x in (keys, values_))
        pad = np.zeros((1, kv, 80, D))
        pad_v = pad.copy()
        pad[:, :, :window], pad_v[:, :, :window] = Kf, Vf
        want = ref.decode(qf[s:s + 1].reshape(1, 6, D), [window - 1], [0], np.zeros((1, 1), int), pad, pad_v, D ** -0.5)
        bound = decode_bound(*want, D, dtype)
        if dtype == "fp8":   # the cache's own rounding, 2^-4 of keys and values: a score by 2^-4 spread
            bound = bound + want[1] * (2 * 2.0 ** -4 * want[2][..., None] + 2.0 ** -4)
        check(o[s:s + 1], want[0], bound, f"row {s}")


def test_no_rows(tp):
    h, q, at, table, K, V, ws = plain(tp)
    h.decode(q[:0], at[:0], table, K, V, q[:0], ws)
    h.append(torch.empty(0, 12 * 64, device="cuda", dtype=torch.bfloat16), at[:0], table, K, V, q[:0])
    assert h.sync_status() == 0


def test_more_queries_than_a_group(tp):
    for dtype in ("bf16", "f32", "fp8"):
        decode_case(tp, np.random.default_rng(15), [90, 3], 130, 1, 64, 16, 1, dtype)


def test_binding_refuses_on_the_gpu(tp):
    h, q, at, table, K, V, ws = plain(tp)
    o = torch.empty_like(q)
    for bad in (dict(Q=q.float()), dict(Q=q[:, ::2]), dict(Q=q.cpu()), dict(K=K[:-1]), dict(K=K.transpose(0, 1)), dict(positions=at.long()),
                dict(positions=at[:, None]), dict(table=table.t()), dict(table=table.float()), dict(O=o[:-1]), dict(workspace=ws.cpu())):
        kw = {**dict(Q=q, positions=at, table=table, K=K, V=V, O=o, workspace=ws), **bad}
        with pytest.raises(ValueError):
            h.decode(**kw)
    with pytest.raises(tp.TpError):
        h.decode(q, at, table, K, V, o, None)
    with pytest.raises(tp.TpError):
        h.decode(q, at, table, K, V, o, ws[:-256])
    with pytest.raises(tp.TpError):
        h.decode(q, at, table[:2].contiguous(), K, V, o, ws)    # more rows than sequences
    with pytest.raises(ValueError):
        tp.TPPagedAttention(8, 2, 64, 16, 8, dtype="fp8").decode(q, at, table, K[:8], V[:8], o, ws)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 256])
@pytest.mark.parametrize("per", [1, 3, 6, 13])
def test_decode_few_rows(tp, dtype, D, per):
    """Few short rows, which clusters of blocks take, and the same where the table could hold long ones, which are
    dealt out by the list."""
    for lengths in ([2000], [1, 0, 700, 65, 511]):
        for capacity in (0, 20000):
            decode_case(tp, np.random.default_rng(D + per), lengths, 2 * per, 2, D, 16, 1, dtype, capacity=capacity)
    decode_case(tp, np.random.default_rng(D + per), [5000, 333], 2 * per, 2, D, 32, 2, dtype, window=600)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("rows,length", [(1, 100), (2, 200), (3, 1000), (5, 450), (40, 480), (150, 500), (150, 120)])
def test_decode_clusters_of_all_sizes(tp, dtype, rows, length):
    """From eight blocks a segment to one, and more of them than are resident."""
    rng = np.random.default_rng(rows)
    lengths = [length] + [int(x) for x in rng.integers(0, length + 1, size=rows - 1)]
    for D in (64, 128) if rows < 100 else (128,):
        decode_case(tp, rng, lengths, 8, 4, D, 16, 2, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("D,dim", [(208, 138), (128, 98), (32, 6)])
def test_append_halves_of_any_width(tp, dtype, D, dim):
    rng = np.random.default_rng(dim)
    positions, sequences, table, pages = ragged(rng, [40, 3, 700], [0, 50, 9], 32)
    append_case(tp, positions, sequences, table, pages, 32, 32, 8, D, 2, dtype, dim=dim)
    append_case(tp, np.where(np.arange(len(positions)) % 7 == 0, -1, positions), sequences, table, pages, 32, 32, 8, D, 4, dtype, True, dim=dim)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("D,per", [(144, 9), (192, 16), (208, 12), (256, 16), (256, 17)])
def test_decode_wide_heads_and_groups(tp, dtype, D, per):
    """Long rows among short ones by the list, few rows by clusters, rows that a window bounds."""
    decode_case(tp, np.random.default_rng(D + per), [2100, 0, 1, 900, 17, 33] + [60] * 30, 4 * per, 4, D, 32, 2, dtype)
    decode_case(tp, np.random.default_rng(D - per), [1300, 129], 2 * per, 2, D, 16, 1, dtype)
    decode_case(tp, np.random.default_rng(per), [700, 3, 500, 200] * 20, 2 * per, 2, D, 64, 2, dtype, window=140)
