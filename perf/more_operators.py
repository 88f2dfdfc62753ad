"""What stands between the QKV column layer and the output row layer, as cases to be measured.

Three operator families on the T shards of a tensor-parallel attention's QKV
tensor, x[t] = [tokens, (heads + 2 kv_heads) / T * D]:

* rotary: the position rotation of its queries and keys, and its gradient.  The
  pair (x1, x2) at position p turns by the angle p f_i:
      y1 = a (x1 cos - x2 sin)      y2 = a (x2 cos + x1 sin)
  with f_i = base^(-2i/dim), scaled for contexts longer than those trained on;
* append: new tokens enter a paged key-value cache.  Queries and keys are
  rotated, queries go to a tensor of their own, keys and values into the
  slots that a table of pages gives for (sequence, position), as they are or in
  8 bits;
* decode: attention of one new token a row over the pages of its sequence,
  positions max(0, p - window + 1) .. p; a row at position -1 is padding, whose
  output is zero.

`run` computes them with plain torch operations (own = False) or through this
package (own = True).
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _case(name, op, heads, kv_heads, D, T=1, dtype="bf16", grouped=False, dim=None, interleaved=False, base=10000.0,
          scaling="none", factor=1.0, original=0, **kw):
    return {"name": name, "op": op, "heads": heads, "kv_heads": kv_heads, "D": D, "T": T, "dtype": dtype,
            "grouped": grouped, "dim": D if dim is None else dim, "interleaved": interleaved, "base": base,
            "scaling": scaling, "factor": factor, "original": original, **kw}


def listed():
    return [
        # one token of one sequence while answering, in its place
        _case("rotary fwd one token", "rotary_fwd", 32, 8, 128, S=1, B=1, place=True, positions=True),
        # the attention projections' QKV tensor in 8 shards, 4096 positions and 2 sequences, in its place
        _case("rotary fwd projections", "rotary_fwd", 32, 32, 128, T=8, S=4096, B=2, place=True, positions=False),
        # training on packed long documents: positions start anew, frequencies for 16 times the length
        _case("rotary bwd long packed", "rotary_bwd", 32, 8, 128, T=4, S=32768, B=1, grouped=True, interleaved=True,
              base=500000.0, scaling="parts", factor=16.0, original=8192, place=False, positions=True),
        # a ragged fp32 batch whose heads are rotated in part
        _case("rotary bwd ragged f32", "rotary_bwd", 12, 4, 80, T=2, dtype="f32", dim=32, S=1021, B=3, place=False,
              positions=False),
        # one step of 64 sequences that answer
        _case("append one step", "append", 32, 8, 128, T=8, page=16, seqs=64, tokens=64, past=6000, pad=0),
        # the prompts of 7 sequences, some with a past, and rows behind the last
        _case("append prompts", "append", 32, 8, 128, T=4, grouped=True, page=64, seqs=7, tokens=8001, past=500, pad=91,
              scaling="linear", factor=4.0),
        # long prompts into a cache of 8 bits
        _case("append prompts 8-bit", "append", 64, 8, 128, T=8, dtype="fp8", interleaved=True, page=32, seqs=3,
              tokens=16384, past=0, pad=0, scaling="ntk", factor=8.0),
        # one sequence that answers alone
        _case("decode one sequence", "decode", 32, 8, 128, page=16, rows=1, length=2000, window=0),
        # a served batch of uneven lengths, every shard's heads, some rows empty
        _case("decode batch", "decode", 32, 8, 128, T=8, page=16, rows=64, length=8192, window=0, pad=3),
        # the same with more queries to a key head and the cache in 8 bits
        _case("decode batch 8-bit", "decode", 64, 8, 128, T=8, dtype="fp8", page=64, rows=96, length=8192, window=0),
        # one document of half a million tokens
        _case("decode long", "decode", 32, 8, 128, T=4, page=64, rows=1, length=500000, window=0),
        # fp32, a head for each query, an odd width, and a sliding window
        _case("decode window f32", "decode", 12, 12, 72, dtype="f32", page=48, rows=17, length=5000, window=1000),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary_fwd", "rotary_bwd", "append", "append", "decode", "decode", "decode"])
    dtype = rng.choice(["bf16", "bf16", "f32"] if op.startswith("rotary") else ["bf16", "bf16", "fp8", "f32"])
    D = rng.choice([128, 128, 64, 16 * rng.randint(2, 16), 8 * rng.randint(4, 32)])
    if dtype == "fp8":
        D = -(-D // 16) * 16
    kv = rng.choice([1, 2, 4, 8, 8, 16, rng.randint(1, 16)])
    heads = kv * rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 8, 12, 16])
    if heads > 128:
        heads = kv * 4
    case = _case("", op, heads, kv, D, T=rng.choice([t for t in (1, 2, 4, 8) if kv % t == 0]), dtype=dtype,
                 grouped=rng.random() < 0.4, interleaved=rng.random() < 0.4,
                 dim=rng.choice([D, D, 2 * rng.randint(2, D // 2), D // 2 // 2 * 2]),
                 base=rng.choice([10000.0, 500000.0, 1e6]), scaling=rng.choice(["none", "linear", "ntk", "parts"]))
    del case["name"]
    if case["scaling"] != "none":
        case["factor"], case["original"] = rng.choice([2.0, 4.0, 8.0, 32.0]), rng.choice([2048, 4096, 8192])
    size = {"bf16": 2, "fp8": 2, "f32": 4}[dtype]
    width = (heads + 2 * kv) * D * size
    most = max(1, min(32768, 400_000_000 // width))
    if op.startswith("rotary"):
        M = _log_int(rng, 1, most)
        B = min(M, rng.randint(1, 5))
        case.update(S=M // B, B=B, place=rng.random() < 0.5, positions=rng.random() < 0.5)
        if case["place"] and case["scaling"] == "parts":  # its factor would grow from pass to pass
            case.update(scaling="none", factor=1.0)
        return case
    case["page"] = rng.choice([16, 16, 32, 64, 128, 16 * rng.randint(1, 20)])
    row = 2 * kv * D * (1 if dtype == "fp8" else size)  # a position's bytes
    if op == "append":
        tokens = _log_int(rng, 1, most)
        seqs = _log_int(rng, 1, min(tokens, 128))
        case.update(seqs=seqs, tokens=tokens, past=_log_int(rng, 1, max(2, min(20000, 300_000_000 // (row * seqs)))),
                    pad=rng.choice([0, 0, rng.randint(1, 64)]))
        return case
    rows = _log_int(rng, 1, 256)
    length = _log_int(rng, 1, max(2, min(200_000, 800_000_000 // (row * rows))))
    case.update(rows=rows, length=length, window=rng.choice([0, 0, 0, _log_int(rng, 1, length)]))
    if rng.random() < 0.3:
        case["pad"] = rng.randint(1, 8)
    return case


def _share(total, parts, seed):
    """`total` things dealt out unevenly to `parts`, one at least to each."""
    rng = random.Random(seed)
    share = [rng.random() + 0.05 for _ in range(parts)]
    out = [1 + int((total - parts) * x / sum(share)) for x in share]
    out[0] += total - sum(out)
    return out


def _append_plan(case):
    """New tokens and past length of each sequence."""
    seqs, past = case["seqs"], case["past"]
    rng = random.Random(seqs * 1_000_003 + past)
    return _share(case["tokens"], seqs, case["tokens"]), [rng.randint(0, past) for _ in range(seqs)]


def _decode_lengths(case):
    """Length of each row's sequence, the new token among them (0: padding)."""
    rng = random.Random(case["rows"] * 1_000_003 + case["length"])
    out = [case["length"]] + [rng.randint(1, case["length"]) for _ in range(case["rows"] - 1)]
    for _ in range(case.get("pad", 0)):
        out.insert(rng.randint(0, len(out)), 0)
    return out


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    D, heads, kv = case["D"], case["heads"], case["kv_heads"]
    if case["op"] == "decode":
        c = 1 if case["dtype"] == "fp8" else e
        lengths = _decode_lengths(case)
        seen = sum(min(n, case["window"] or n) for n in lengths)
        return {"bytes": seen * 2 * kv * D * c + len(lengths) * 2 * heads * D * e + 4 * seen // case["page"],
                "flops": seen * heads * 4 * D}
    if case["op"] == "append":
        c = 1 if case["dtype"] == "fp8" else e
        return {"bytes": case["tokens"] * D * ((heads + 2 * kv) * e + heads * e + 2 * kv * c + 8),
                "flops": case["tokens"] * (heads + kv) * case["dim"] * 3}
    M = case["S"] * case["B"]
    moved = (heads + kv) * case["dim"] if case["place"] else (heads + 2 * kv) * D
    return {"bytes": M * moved * 2 * e + (4 * M if case["positions"] else 0),
            "flops": M * (heads + kv) * case["dim"] * 3}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _frequencies(case):
    """f_i of each pair, and a."""
    d, s = case["dim"], case["factor"]
    base = case["base"]
    if case["scaling"] == "ntk":  # a larger base: the slowest pair turns s times slower, the fastest as before
        base = base * s ** (d / (d - 2)) if d > 2 else base
    f = [base ** (-2.0 * i / d) for i in range(d // 2)]
    if case["scaling"] == "linear":
        f = [x / s for x in f]
    a = 1.0
    if case["scaling"] == "parts":
        # a pair that turns 32 times or more over the trained length keeps its frequency, one that turns once or
        # less is slowed s times, the others are between
        keep = [min(1.0, max(0.0, (case["original"] * x / (2 * math.pi) - 1.0) / 31.0)) for x in f]
        f = [x * k + x / s * (1.0 - k) for x, k in zip(f, keep)]
        a = 0.1 * math.log(s) + 1.0
    return f, a


def _normal(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device="cuda").mul_(std)


def _qkv(case, gen, n):
    """The T shards of a QKV tensor: some channels of the keys are far larger than the others."""
    T, D, hq, hk = case["T"], case["D"], case["heads"] // case["T"], case["kv_heads"] // case["T"]
    x = _normal(gen, T, n, (hq + 2 * hk) * D)
    q, k, _ = _split(case, x)
    k *= torch.exp(_normal(gen, hk, D, std=0.5))
    q *= 1.5
    return x.to(torch.float32 if case["dtype"] == "f32" else torch.bfloat16)


def _split(case, x):
    """Views of the queries [T, n, (kv heads,) heads, D], keys and values [T, n, kv heads, D] of the shards."""
    T, D, hq, hk = case["T"], case["D"], case["heads"] // case["T"], case["kv_heads"] // case["T"]
    if case["grouped"]:  # each key head's queries, its key, its value
        g = x.view(T, -1, hk, hq // hk + 2, D)
        return g[..., :-2, :], g[..., -2, :], g[..., -1, :]
    g = x.view(T, -1, hq + 2 * hk, D)
    return g[:, :, :hq], g[:, :, hq:hq + hk], g[:, :, hq + hk:]


def _table(case, gen, lengths):
    """Pages dealt out in no order: [sequences, most pages] with -1 behind a sequence's last, and how many there are."""
    page = case["page"]
    need = torch.tensor([-(-n // page) for n in lengths])
    used = int(need.sum())
    pages = used + 3
    order = torch.randperm(pages, generator=gen, device="cuda")[:used].int()
    table = torch.full((len(lengths), max(1, int(need.max()))), -1, dtype=torch.int32, device="cuda")
    table[(torch.arange(table.shape[1]) < need[:, None]).cuda()] = order
    return table, pages


def _cache(case, gen, pages):
    """Keys and values as earlier calls left them: [T, pages, kv heads, page, D]."""
    T, D, hk = case["T"], case["D"], case["kv_heads"] // case["T"]
    out = []
    for std in (1.2, 1.0):
        t = torch.empty(T, pages, hk, case["page"], D, device="cuda",
                        dtype={"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.uint8}[case["dtype"]])
        for shard in t:
            x = torch.randn(shard.shape, generator=gen, device="cuda", dtype=torch.bfloat16).mul_(std)
            if case["dtype"] == "fp8":
                shard.copy_((x * 90.0).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
            else:
                shard.copy_(x)
        out.append(t)
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    act = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    f, s["a"] = _frequencies(case)
    s["f"] = torch.tensor(f, dtype=torch.float64, device="cuda")
    T, D, heads, kv = case["T"], case["D"], case["heads"], case["kv_heads"]
    if case["op"].startswith("rotary"):
        M = case["S"] * case["B"]
        s["x"] = _qkv(case, gen, M)
        s["y"] = s["x"] if case["place"] else torch.empty_like(s["x"])
        s["positions"] = s["at"] = None
        s["at"] = torch.arange(M, device="cuda", dtype=torch.int32) // case["B"]
        if case["positions"]:  # documents one after the other, the first begun before
            lengths = torch.tensor(_share(M, min(M, 5), M), device="cuda")
            start = torch.cumsum(lengths, 0) - lengths
            which = torch.repeat_interleave(torch.arange(len(lengths), device="cuda"), lengths)
            at = torch.arange(M, device="cuda") - start[which] + torch.where(which == 0, 1717, 0)
            s["positions"] = s["at"] = at.int()
    elif case["op"] == "append":
        new, past = _append_plan(case)
        s["x"] = _qkv(case, gen, case["tokens"] + case["pad"])
        n = torch.tensor(new, device="cuda")
        which = torch.repeat_interleave(torch.arange(len(new), device="cuda"), n)
        at = torch.arange(len(which), device="cuda") - (torch.cumsum(n, 0) - n - torch.tensor(past, device="cuda"))[which]
        pad = torch.full((case["pad"],), -1, dtype=torch.int32, device="cuda")
        s["positions"] = torch.cat([at.int(), pad])
        s["sequences"] = torch.cat([which.int(), pad])
        s["table"], s["pages"] = _table(case, gen, [a + b for a, b in zip(new, past)])
        s["k"], s["v"] = _cache(case, gen, s["pages"])
        s["q"] = torch.zeros(T, case["tokens"] + case["pad"], heads // T * D, dtype=act, device="cuda")
    else:
        lengths = _decode_lengths(case)
        s["positions"] = torch.tensor(lengths, dtype=torch.int32, device="cuda") - 1
        s["table"], s["pages"] = _table(case, gen, lengths)
        s["k"], s["v"] = _cache(case, gen, s["pages"])
        sharp = 0.5 + 2.0 * torch.rand(T, 1, heads // T, 1, generator=gen, device="cuda")
        s["q"] = (_normal(gen, T, len(lengths), heads // T, D) * sharp).to(act).view(T, len(lengths), -1)
        s["o"] = torch.empty_like(s["q"])
    for key, top in (("k_amax", 6.0), ("v_amax", 5.0)):  # what calibration found for each key head
        s[key] = None
        if case["dtype"] == "fp8":
            s[key] = top * (0.8 + 0.4 * torch.rand(kv, generator=gen, device="cuda"))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"append": _own_append, "decode": _own_decode}.get(op, _own_rotary)(s)
    return {"append": _plain_append, "decode": _plain_decode}.get(op, _plain_rotary)(s)


def _own_rope(c):
    import tensor_transformer_mlp_shard_gb300 as tp
    return tp.Rope(dim=c["dim"], base=c["base"], interleaved=c["interleaved"], scaling=c["scaling"],
                   factor=c["factor"], original=c["original"])


def _own_rotary(s):
    import tensor_transformer_mlp_shard_gb300 as tp
    c = s["case"]
    if "rotary" not in s:  # one object for a shape, as a program keeps it
        s["rotary"] = tp.TPRotary(S=c["S"], B=c["B"], heads=c["heads"], kv_heads=c["kv_heads"], head_dim=c["D"],
                                  T=c["T"], dtype=c["dtype"], grouped=c["grouped"], rope=_own_rope(c))
    call = s["rotary"].fwd if c["op"] == "rotary_fwd" else s["rotary"].bwd
    call(s["x"], None if c["place"] else s["y"], positions=s["positions"])
    return s["y"]


def _own_attention(s):
    import tensor_transformer_mlp_shard_gb300 as tp
    c = s["case"]
    if "attention" not in s:
        s["attention"] = tp.TPPagedAttention(
            heads=c["heads"], kv_heads=c["kv_heads"], head_dim=c["D"], page_size=c["page"], pages=s["pages"], T=c["T"],
            dtype=c["dtype"], grouped=c["grouped"], rope=_own_rope(c), window=c.get("window", 0))
        s["ws"] = tp.alloc_workspace(s["attention"].workspace_bytes()) if c["op"] == "decode" else None
    return s["attention"]


def _own_append(s):
    _own_attention(s).append(s["x"], s["positions"], s["table"], s["k"], s["v"], s["q"], sequences=s["sequences"],
                             k_amax=s["k_amax"], v_amax=s["v_amax"])
    return _append_out(s)


def _own_decode(s):
    _own_attention(s).decode(s["q"], s["positions"], s["table"], s["k"], s["v"], s["o"], workspace=s["ws"],
                             k_amax=s["k_amax"], v_amax=s["v_amax"])
    return s["o"]


def _append_out(s):
    if s["case"]["dtype"] != "fp8":
        return {"q": s["q"], "k": s["k"], "v": s["v"]}
    return {"q": s["q"], "k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn)}


def _turns(s, positions):
    """a cos and a sin of every position and pair, the angles in 64 bits."""
    angle = positions.double()[:, None] * s["f"]
    return (s["a"] * angle.cos()).float(), (s["a"] * angle.sin()).float()


def _rotate(c, x, cos, sin):
    """x [T, n, ..., D] in 32 bits, turned."""
    d = c["dim"]
    shape = (1, x.shape[1]) + (1,) * (x.dim() - 3) + (d // 2,)
    cos, sin = cos.view(shape), sin.view(shape)
    x = x.float()
    if c["interleaved"]:
        x1, x2 = x[..., 0:d:2], x[..., 1:d:2]
        turned = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).flatten(-2)
    else:
        x1, x2 = x[..., :d // 2], x[..., d // 2:d]
        turned = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1)
    return turned if d == c["D"] else torch.cat([turned, x[..., d:]], -1)


def _plain_rotary(s):
    c = s["case"]
    cos, sin = _turns(s, s["at"])
    if c["op"] == "rotary_bwd":  # the transpose of a rotation is the one back
        sin = -sin
    to, (q, k, v) = _split(c, s["y"]), _split(c, s["x"])
    to[0].copy_(_rotate(c, q, cos, sin))
    to[1].copy_(_rotate(c, k, cos, sin))
    if not c["place"]:
        to[2].copy_(v)
    return s["y"]


def _scale(s, key):
    """fmax / amax of each key head, [T, 1, kv heads, 1]."""
    return (448.0 / s[key]).view(s["case"]["T"], 1, -1, 1)


def _plain_append(s):
    c = s["case"]
    rows = torch.nonzero(s["positions"] >= 0).flatten()
    at = s["positions"][rows].long()
    page = s["table"][s["sequences"][rows].long(), at // c["page"]].long()
    cos, sin = _turns(s, at)
    q, k, v = (t[:, rows] for t in _split(c, s["x"]))
    s["q"][:, rows] = _rotate(c, q, cos, sin).flatten(2).to(s["q"].dtype)
    k, v = _rotate(c, k, cos, sin), v.float()
    if c["dtype"] == "fp8":
        k, v = ((t * _scale(s, key)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                for t, key in ((k, "k_amax"), (v, "v_amax")))
    s["k"][:, page, :, at % c["page"]] = k.transpose(0, 1).to(s["k"].dtype)
    s["v"][:, page, :, at % c["page"]] = v.transpose(0, 1).to(s["v"].dtype)
    return _append_out(s)


def _plain_pages(s, key):
    """The cache's values of every row, [T, rows, kv heads, positions, D] in 32 bits."""
    c = s["case"]
    t = s[key][:, s["table"].clamp(min=0).long()].transpose(2, 3).flatten(3, 4)
    return t.view(torch.float8_e4m3fn).float() if c["dtype"] == "fp8" else t.float()


def _plain_decode(s):
    c = s["case"]
    T, D, hq, hk = c["T"], c["D"], c["heads"] // c["T"], c["kv_heads"] // c["T"]
    at = s["positions"]
    q = s["q"].view(T, -1, hk, hq // hk, D).float() * D ** -0.5
    if c["dtype"] == "fp8":
        q = q / _scale(s, "k_amax")[..., None]
    scores = q @ _plain_pages(s, "k").transpose(-1, -2)
    j = torch.arange(scores.shape[-1], device="cuda")
    seen = j <= at[:, None]
    if c["window"]:
        seen &= j > at[:, None] - c["window"]
    scores.masked_fill_(~seen[None, :, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out = p @ _plain_pages(s, "v") / torch.where(total > 0, total, 1.0)
    if c["dtype"] == "fp8":
        out = out / _scale(s, "v_amax")[..., None]
    s["o"].copy_(out.flatten(2))
    return s["o"]


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "decode": _exact_decode}.get(case["op"], _exact_rotary)(s)


def _exact_turn(s, x, at, back=False):
    """x [n, heads, D] in 64 bits: each pair as a complex number, times a e^(i p f)."""
    c, out = s["case"], x.clone()
    d = c["dim"]
    pairs = (slice(0, d, 2), slice(1, d, 2)) if c["interleaved"] else (slice(0, d // 2), slice(d // 2, d))
    angle = torch.outer(at.double(), s["f"])[:, None]
    z = torch.complex(x[..., pairs[0]], x[..., pairs[1]]) * torch.polar(torch.full_like(angle, s["a"]), -angle if back else angle)
    out[..., pairs[0]], out[..., pairs[1]] = z.real, z.imag
    return out


def _exact_columns(c):
    """The columns of a shard's queries, keys and values."""
    hq, hk = c["heads"] // c["T"], c["kv_heads"] // c["T"]
    per = hq // hk
    if c["grouped"]:
        first = [j * (per + 2) for j in range(hk)]
        return [i + r for i in first for r in range(per)], [i + per for i in first], [i + per + 1 for i in first]
    return list(range(hq)), list(range(hq, hq + hk)), list(range(hq + hk, hq + 2 * hk))


def _exact_rotary(s):
    c = s["case"]
    cols = _exact_columns(c)
    out = []
    for shard in s["x"]:
        y = shard.double().view(shard.shape[0], -1, c["D"])
        turned = cols[0] + cols[1]
        y[:, turned] = _exact_turn(s, y[:, turned], s["at"], c["op"] == "rotary_bwd")
        out.append(y.flatten(1))
    return torch.stack(out)


def _exact_codes(x, scale):
    """x in steps of e4m3: 8 between powers of two, none finer than 2^-9, halves to even."""
    u = (x * scale.double()[:, None]).clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(u / step) * step


def _exact_append(s):
    c, eight = s["case"], s["case"]["dtype"] == "fp8"
    hk = c["kv_heads"] // c["T"]
    cols = _exact_columns(c)
    real = s["positions"] >= 0
    at, seq = s["positions"][real].long(), s["sequences"][real].long()
    page = s["table"].long()[seq, torch.div(at, c["page"], rounding_mode="floor")]
    out = {"q": [], "k": [], "v": []}
    for t in range(c["T"]):
        x = s["x"][t].double().view(s["x"].shape[1], -1, c["D"])[real]
        q = s["q"][t].double()
        q[real] = _exact_turn(s, x[:, cols[0]], at).flatten(1)
        out["q"].append(q)
        for key, new in (("k", _exact_turn(s, x[:, cols[1]], at)), ("v", x[:, cols[2]])):
            cache = s[key][t].view(torch.float8_e4m3fn).double() if eight else s[key][t].double()
            if eight:
                new = _exact_codes(new, 448.0 / s[key + "_amax"][t * hk:(t + 1) * hk])
            flat = cache.transpose(1, 2).reshape(-1, hk, c["D"])
            flat[page * c["page"] + at % c["page"]] = new
            out[key].append(flat.view(-1, c["page"], hk, c["D"]).transpose(1, 2))
    return {key: torch.stack(v) for key, v in out.items()}


def _exact_decode(s):
    c, eight = s["case"], s["case"]["dtype"] == "fp8"
    T, D, hq, hk, page = c["T"], c["D"], c["heads"] // c["T"], c["kv_heads"] // c["T"], c["page"]
    out = torch.zeros(T, len(s["positions"]), hk, hq // hk, D, dtype=torch.float64, device="cuda")
    for row, at in enumerate(s["positions"].tolist()):
        if at < 0:
            continue
        lo = max(0, at - c["window"] + 1) if c["window"] else 0
        first = lo // page
        pages = s["table"][row, first:at // page + 1].long()
        got = []
        for key in ("k", "v"):
            x = s[key][:, pages].transpose(1, 2).flatten(2, 3)[:, :, lo - first * page:at + 1 - first * page]
            x = x.view(torch.float8_e4m3fn).double() if eight else x.double()
            if eight:
                x *= (s[key + "_amax"].double() / 448).view(T, hk, 1, 1)
            got.append(x)
        q = s["q"][:, row].double().view(T, hk, hq // hk, D)
        weights = torch.softmax(torch.einsum("thgd,thnd->thgn", q, got[0]) / math.sqrt(D), -1)
        out[:, row] = torch.einsum("thgn,thnd->thgd", weights, got[1])
    return out.view(T, len(s["positions"]), -1)
