"""Inputs, references and error bounds shared by the attention tests."""
import numpy as np
import torch

from oracle import attention as ref

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.bfloat16}
# half a step of a stored number, relative to it
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp8": 2.0 ** -8}


def values(rng, shape, dtype):
    """Seeded normal numbers as the type holds them: (CUDA tensor, its numbers in fp64)."""
    t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(TORCH[dtype])
    return t.cuda(), t.double().numpy()


def rotation_bound(x, y, f, a, half_step, interleaved=False):
    """Bound on a rotated element's error, [n, heads, D].  In units of
    2^-24 a (|x1| + |x2|): a sine or cosine is off by 2 (the function) + 0.5 (its
    argument's rounding, an eighth of a turn at most) and 1 (times a), the
    products and their sum by 1 each, 5.5 in all; then half a step of the result."""
    half = len(f)
    size = np.zeros_like(y)
    i1 = np.arange(half) * 2 if interleaved else np.arange(half)
    i2 = i1 + 1 if interleaved else i1 + half
    both = a * (np.abs(x[..., i1]) + np.abs(x[..., i2])) * 2.0 ** -24 * 6
    size[..., i1], size[..., i2] = both, both
    return size + (np.abs(y) + size) * half_step


def decode_bound(o, mag, spread, seen, D, dtype):
    """Bound on decode's error.  A score is a sum of D products, each addition
    off by at most 2^-23 of the sum of magnitudes: (D + 4) 2^-23 spread, the 4
    for the scale and the exponent's argument; a weight's relative error is twice
    that (its own score and the normalisation's), 2^-15 for the sum of two
    16-bit numbers and the exponential (2^-20 in fp32), and the sum over
    positions adds (seen + 64) 2^-23 (the joins among it).  Then half a step of
    the result."""
    rel = 2 * (D + 4) * 2.0 ** -23 * spread + (2.0 ** -20 if dtype == "f32" else 2.0 ** -15)
    rel = rel + ((seen + 64) * 2.0 ** -23)[:, None]
    err = rel[..., None] * mag
    return err + (np.abs(o) + err) * HALF_STEP[dtype]


def check(got, want, bound, what=""):
    got = got.double().cpu().numpy().reshape(want.shape)
    off = np.abs(got - want)
    bad = ~(off <= bound + 1e-300) & ~((got == want) | (np.isnan(got) & np.isnan(want)))
    if bad.any():
        at = tuple(int(i[0]) for i in np.nonzero(bad))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first {at}: {got[at]} for {want[at]}, "
                             f"bound {bound[at]}")


def same_bits(a, b):
    v = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return bool((a.contiguous().view(v) == b.contiguous().view(v)).all())


def table_for(rng, lengths, page_size, spare=3):
    """A table of pages in no order, -1 behind each sequence's last; pages in all."""
    need = [-(-n // page_size) for n in lengths]
    order = rng.permutation(sum(need) + spare)
    table = np.full((len(lengths), max(1, max(need))), -1, dtype=np.int32)
    at = 0
    for s, k in enumerate(need):
        table[s, :k] = order[at:at + k]
        at += k
    return table, sum(need) + spare


def e4m3(codes):
    """fp64 values of uint8 E4M3 codes."""
    return codes.cpu().view(torch.float8_e4m3fn).double().numpy()


def cuda_i32(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()


class Cache:
    """The T shards of a cache whose slots all hold something: numbers in the
    slots of `lengths`, NaN everywhere else."""

    def __init__(self, rng, h, lengths, table, pages, page_size, dtype, amax=None):
        self.table, self.dtype = table, dtype
        T, hk, D = h.T, h.kv_heads // h.T, h.head_dim
        used = np.zeros((pages, page_size), dtype=bool)
        for s, n in enumerate(lengths):
            for p in range(n):
                used[table[s, p // page_size], p % page_size] = True
        self.K, self.V, self.Kf, self.Vf = [], [], [], []
        for t in range(T):
            for dev, host, key in ((self.K, self.Kf, 0), (self.V, self.Vf, 1)):
                x = torch.from_numpy(rng.standard_normal((pages, hk, page_size, D)).astype(np.float32))
                hole = torch.from_numpy(~used)[:, None, :, None].expand_as(x)
                if dtype == "fp8":
                    c = (x * 90).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                    c[hole] = 0x7F  # NaN
                    scale = (448.0 / amax[key][t * hk:(t + 1) * hk].float()).view(1, hk, 1, 1).double()
                    f = c.view(torch.float8_e4m3fn).double() / scale
                else:
                    c = x.to(TORCH[dtype])
                    c[hole] = float("nan")
                    f = c.double()
                dev.append(c.cuda())
                host.append(f.numpy())


def decode_case(tp, rng, lengths, heads, kv, D, page_size, T=1, dtype="bf16", window=0, sequences=None, positions=None,
                scale=None, q_std=1.0, capacity=0):
    """Runs decode on a seeded case and checks every shard; returns what it made."""
    table, pages = table_for(rng, lengths, page_size)
    if capacity > table.shape[1] * page_size:   # a table with room to grow
        wide = np.full((len(lengths), -(-capacity // page_size)), -1, dtype=np.int32)
        wide[:, :table.shape[1]] = table
        table = wide
    amax = None
    if dtype == "fp8":
        amax = [torch.from_numpy((3.0 + rng.random(kv)).astype(np.float32)) for _ in range(2)]
    h = tp.TPPagedAttention(heads, kv, D, page_size, pages, T=T, dtype=dtype, window=window, scale=scale)
    cache = Cache(rng, h, lengths, table, pages, page_size, dtype, amax)
    positions = np.asarray([n - 1 for n in lengths] if positions is None else positions)
    rows = len(positions)
    q, qf = zip(*[values(rng, (rows, heads // T * D), dtype) for _ in range(T)])
    if q_std != 1.0:
        q = [(x.float() * q_std).to(x.dtype) for x in q]
        qf = [x.double().cpu().numpy() for x in q]
    o = [torch.full_like(x, float("nan")) for x in q]
    ws = tp.alloc_workspace(h.workspace_bytes())
    ws.fill_(0xFF)
    kw = {}
    if amax:
        kw = dict(k_amax=amax[0].cuda(), v_amax=amax[1].cuda())
    if sequences is not None:
        kw["sequences"] = cuda_i32(sequences)
    args = (list(q), cuda_i32(positions), cuda_i32(table), cache.K, cache.V)
    h.decode(*args, o, ws, **kw)
    assert h.sync_status() == 0
    seqs = np.arange(rows) if sequences is None else np.asarray(sequences)
    for t in range(T):
        want = ref.decode(qf[t].reshape(rows, heads // T, D), positions, seqs, table, cache.Kf[t], cache.Vf[t],
                          D ** -0.5 if scale is None else scale, window)
        check(o[t], want[0], decode_bound(*want, D, dtype), f"shard {t}")
    return h, args, o, ws, kw
