"""The block norm and the AdamW step, as cases to be measured.

Two operator families that stand next to the tensor-parallel MLP in a training
step:

* the block norm: what happens to the residual stream x between one block and
  the next.  With the block's output f, its post-norm P, a gate g and the next
  block's pre-norm N:
      y = a x + c g * P(f)        n = N(y)
  (a the residual scale, c the block scale), and its backward pass;
* AdamW over a list of tensors (weights of every shard, biases, norm weights)
  with states in 32 bits or in 8, optionally after the global gradient norm
  that clips it.

`run` computes either with plain torch operations (own = False) or through
this package (own = True).
"""
import math
import random

import torch

own = False

BETA1, BETA2, EPS_ADAM, LR = 0.9, 0.95, 1e-8, 1e-3
QBLOCK = 256          # elements that share a scale of the 8-bit states
C1, C2, MASK = 0x9E3779B9, 0xB504F333, 0xFFFFFFFF


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _norm(name, op, S, B, H, T=1, dtype="bf16", post="none", pre="rms", gate="none", res32=False, train=True,
          zero=False, a=1.0, c=1.0):
    return {"name": name, "op": op, "S": S, "B": B, "H": H, "T": T, "dtype": dtype, "post": post, "pre": pre,
            "gate": gate, "res32": res32, "train": train, "zero": zero, "a": a, "c": c}


def _adamw(name, layout, param="bf16", grad="f32", bits=32, clip=False, **kw):
    return {"name": name, "op": "adamw", "layout": layout, "param": param, "grad": grad, "bits": bits, "clip": clip,
            **kw}


def listed():
    return [
        # one token of one sequence while answering: nothing is kept for a backward pass
        _norm("norm fwd one token", "norm_fwd", 1, 1, 4096, post="rms", train=False),
        # a ragged fp32 batch with LayerNorms and one gate value a token (a router's weight)
        _norm("norm fwd ragged f32", "norm_fwd", 77, 3, 1416, dtype="f32", post="layer", pre="layer", gate="token",
              a=0.5, c=1.25),
        # the GPT-size block: norms on both sides of the MLP and a learned gain per channel
        _norm("norm fwd gpt", "norm_fwd", 2048, 4, 4096, post="rms", gate="channel"),
        # the sequence-parallel block, its tokens in 8 shards: residual add and LayerNorm
        _norm("norm fwd sp", "norm_fwd", 4096, 4, 6144, T=8, pre="layer"),
        # gradients of a ragged batch with every kind of parameter, gated element by element
        _norm("norm bwd ragged", "norm_bwd", 129, 5, 2056, post="layer", pre="layer", gate="element", zero=True,
              a=0.7, c=0.9),
        _norm("norm bwd gpt", "norm_bwd", 2048, 4, 4096, post="rms", gate="channel"),
        # the SwiGLU-size block with its residual stream kept in fp32
        _norm("norm bwd swiglu f32 stream", "norm_bwd", 4096, 1, 8192, pre="layer", gate="channel", res32=True,
              c=0.25),
        # the parameters that are vectors, alone: every bias shard and norm weight of one block
        _adamw("adamw vectors", "vectors", param="f32", H=4096, F=16384, T=8, g=1),
        # all weights of the GPT-size block in 8 shards, clipped, states in 32 bits
        _adamw("adamw gpt clipped", "mlp", clip=True, H=4096, F=16384, T=8, g=1),
        # the same with states in 8 bits
        _adamw("adamw gpt 8-bit", "mlp", bits=8, H=4096, F=16384, T=8, g=1),
        # many tensors of uneven sizes, as a whole small model has them
        _adamw("adamw ragged 8-bit clipped", "ragged", bits=8, clip=True, count=301, total=24_000_007),
        _adamw("adamw ragged bf16 grads", "ragged", param="f32", grad="bf16", clip=True, count=97, total=40_000_003),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "adamw"])
    if op == "adamw":
        total = _log_int(rng, 1000, 50_000_000)
        return {"op": op, "layout": "ragged", "param": rng.choice(["bf16", "f32"]), "grad": rng.choice(["f32", "bf16"]),
                "bits": rng.choice([32, 8]), "clip": rng.random() < 0.5,
                "count": _log_int(rng, 1, min(400, total // 4)), "total": total}
    H = 8 * _log_int(rng, 8, 2048)
    B = rng.randint(1, 8)
    S = _log_int(rng, 1, max(1, min(8192, 32_000_000 // (H * B))))
    T = rng.choice([1, 1, 1, 2, 4, 8])
    if T > 1:
        S = T * max(1, S // T)
    block = rng.random() < 0.85
    case = _norm("", op, S, B, H, T=T, dtype=rng.choice(["bf16", "bf16", "f32"]),
                 post=rng.choice(["none", "rms", "layer"]),
                 pre=rng.choice(["rms", "layer"]) if not block else rng.choice(["none", "rms", "layer"]),
                 gate=rng.choice(["none", "channel", "token", "element"]), zero=rng.random() < 0.3,
                 train=op == "norm_bwd" or rng.random() < 0.7,
                 a=rng.choice([1.0, 0.5, 0.9]), c=rng.choice([1.0, 0.25, 1.5]))
    case["res32"] = case["dtype"] == "bf16" and rng.random() < 0.3
    if not block:  # the norm before the first block: there is no block output yet
        case["alone"] = True
        case["post"] = case["gate"] = "none"
        case["a"] = case["c"] = 1.0
    del case["name"]
    return case


def _sizes(case):
    """Element counts of the tensors of an AdamW case, and whether each is decayed."""
    if case["layout"] in ("mlp", "vectors"):
        H, F, T, g = case["H"], case["F"], case["T"], case["g"]
        vectors = [(g * F // T, False)] * T + [(H, False)] * 3
        if case["layout"] == "vectors":
            return vectors
        return [(g * F // T * H, True)] * T + [(H * (F // T), True)] * T + vectors
    rng = random.Random(case["count"] * 1_000_003 + case["total"])
    share = [math.exp(rng.gauss(0.0, 1.5)) for _ in range(case["count"])]
    left = max(0, case["total"] - case["count"])
    return [(1 + int(left * s / sum(share)), rng.random() < 0.6) for s in share]


def work(case):
    if case["op"] == "adamw":
        n = sum(k for k, _ in _sizes(case))
        b = (2 if case["grad"] == "bf16" else 4) + 8 + (2 if case["param"] == "bf16" else 0)
        b += 16 if case["bits"] == 32 else 4 + 16 / QBLOCK
        return {"bytes": n * b, "flops": n * (20 + (3 if case["clip"] else 0))}
    M, H = case["S"] * case["B"], case["H"]
    e = 4 if case["dtype"] == "f32" else 2
    r = 4 if case["res32"] else e
    block, pre = not case.get("alone"), case["pre"] != "none"
    gate = {"none": 0, "channel": 0, "token": 0, "element": e}[case["gate"]]
    if case["op"] == "norm_fwd":
        per = r + (e + gate + r if block else 0) + (e if pre else 0)
        return {"bytes": M * H * per, "flops": M * H * 12}
    # dy, y, dn (with a pre-norm), f; dx, df; a gate per element and its gradient
    per = r + (r + e if pre else 0) + (e if block and (case["post"] != "none" or case["gate"] != "none") else 0)
    per += r + (e + 2 * gate if block else 0)
    return {"bytes": M * H * per, "flops": M * H * 30}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return _prepare_adamw(case, gen) if case["op"] == "adamw" else _prepare_norm(case, gen)


def _stats(x, kind, eps):
    """(mean, 1 / spread) of each row, as the forward pass keeps them."""
    x = x.float()
    if kind == "none":
        return torch.zeros_like(x[:, 0]), torch.ones_like(x[:, 0])
    mean = x.mean(1) if kind == "layer" else torch.zeros_like(x[:, 0])
    return mean, ((x - mean[:, None]).square().mean(1) + eps).rsqrt()


def _prepare_norm(case, gen):
    M, H, T = case["S"] * case["B"], case["H"], case["T"]
    act = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    res = torch.float32 if case["res32"] else act

    def normal(*shape, std=1.0, mean=0.0, dtype=act):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(std).add_(mean).to(dtype)

    block, pre, post = not case.get("alone"), case["pre"], case["post"]
    s = {"case": case, "eps": 1e-5}
    # a residual stream has a few channels far larger than the others
    channel = torch.exp(torch.randn(H, generator=gen, device="cuda") * 0.4)
    channel[torch.randint(0, H, (max(1, H // 500),), generator=gen, device="cuda")] *= 12.0
    x = (torch.randn(M, H, generator=gen, device="cuda") * channel + 0.1).to(res)
    s["f"] = normal(M, H) if block else None
    s["gate"] = {"none": lambda: None, "channel": lambda: normal(H, std=0.3, mean=0.5),
                 "token": lambda: normal(M).sigmoid_(), "element": lambda: normal(M, H).sigmoid_()}[case["gate"]]()
    one = 0.0 if case["zero"] else 1.0
    for side, kind in (("post", post), ("pre", pre)):
        s[side + "_w"] = normal(H, std=0.2, mean=one) if kind != "none" else None
        s[side + "_b"] = normal(H, std=0.2) if kind == "layer" else None
    if case["op"] == "norm_fwd":
        s["x"] = x
        s["y"] = torch.empty_like(x) if block else None
        s["n"] = torch.empty(M, H, dtype=act, device="cuda") if pre != "none" else None
        s["stats"] = torch.empty(M, 4, device="cuda") if case["train"] else None
        shared = ("x", "f", "y", "n")
    else:
        s["y"] = x  # the stream after the block, as the forward pass stored it
        s["dy"] = normal(M, H, dtype=res)
        s["dn"] = normal(M, H) if pre != "none" else None
        st = _stats(s["f"], post, s["eps"]) if block else _stats(x, "none", s["eps"])
        s["stats"] = torch.stack(st + _stats(x, pre, s["eps"]), 1)
        s["dx"] = torch.empty_like(x)
        s["df"] = torch.empty_like(s["f"]) if block else None
        s["dgate"] = None if s["gate"] is None else torch.empty(
            s["gate"].shape, device="cuda", dtype=torch.float32 if case["gate"] == "channel" else act)
        for side in ("post_w", "post_b", "pre_w", "pre_b"):
            s["d" + side] = None if s[side] is None else torch.empty(H, device="cuda")
        shared = ("y", "f", "dy", "dn", "dx", "df")
    if case["gate"] in ("token", "element"):
        shared += ("gate", "dgate")
    # the token shards of each tensor, which are the tensor itself without sequence parallelism
    s["shards"] = {k: None if s.get(k) is None else list(s[k].chunk(T)) for k in shared}
    return s


def _prepare_adamw(case, gen):
    sizes = _sizes(case)
    blocks = torch.tensor([-(-n // QBLOCK) for n, _ in sizes])
    first = torch.cumsum(blocks, 0) - blocks
    total = int(blocks.sum()) * QBLOCK
    which = torch.repeat_interleave(torch.arange(len(sizes)), blocks)

    def views(t, per=QBLOCK):
        """The tensors inside a flat buffer that gives each a whole number of blocks."""
        if per == 1:
            return [t[a:a + b] for a, b in zip(first.tolist(), blocks.tolist())]
        return [t[a * per:a * per + n] for a, (n, _) in zip(first.tolist(), sizes)]

    s = {"case": case, "t": 10, "grad_scale": 0.125, "max_norm": 1.0, "seed": 12345}
    # what lies between the tensors is zero and stays so
    real = torch.zeros(total, dtype=torch.bool, device="cuda")
    for v in views(real):
        v.fill_(True)
    size = torch.exp(torch.randn(total // QBLOCK, 1, generator=gen, device="cuda") * 1.5) * 1e-3

    def normal(std=1.0):
        t = torch.randn(total // QBLOCK, QBLOCK, generator=gen, device="cuda").mul_(std)
        return t

    def flat(t):
        return t.reshape(-1).mul_(real)

    w = flat(normal(0.02))
    s["w"] = w
    s["p"] = w.to(torch.bfloat16) if case["param"] == "bf16" else None
    s["g"] = flat(normal() * size * 8).to(torch.float32 if case["grad"] == "f32" else torch.bfloat16)
    m, r = flat(normal() * size * 0.3), flat((normal() * 0.3 + 1.0).abs_() * size)
    if case["bits"] == 32:
        s["m"], s["v"], s["ms"], s["vs"] = m, r * r, None, None
    else:
        for key, t in (("m", m), ("v", r)):
            t = t.view(-1, QBLOCK)
            top = t.abs().amax(1, keepdim=True)
            scale = torch.where(top > 0, top / 448.0, 0.0)
            codes = torch.where(top > 0, t / scale, 0.0).to(torch.float8_e4m3fn)
            s[key], s[key + "s"] = codes.view(torch.uint8).reshape(-1), scale.reshape(-1).contiguous()
    s["which"] = which.cuda()
    s["block"] = torch.arange(total // QBLOCK, device="cuda") - first.cuda()[s["which"]]
    s["wd"] = [0.1 if d else 0.0 for _, d in sizes]
    s["lr_scale"] = [1.0 if i % 3 else 0.5 for i in range(len(sizes))]
    s["wd_block"] = torch.tensor(s["wd"], device="cuda")[s["which"]][:, None]
    s["lr_block"] = torch.tensor(s["lr_scale"], device="cuda")[s["which"]][:, None]
    s["tensors"] = {k: None if s[k] is None else views(s[k]) for k in ("w", "p", "g", "m", "v")}
    s["tensors"]["ms"] = None if s["ms"] is None else views(s["ms"], 1)
    s["tensors"]["vs"] = None if s["vs"] is None else views(s["vs"], 1)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"norm_fwd": _own_fwd, "norm_bwd": _own_bwd, "adamw": _own_adamw}[op](s)
    return {"norm_fwd": _plain_fwd, "norm_bwd": _plain_bwd, "adamw": _plain_adamw}[op](s)


def _own_handle(s):
    import tensor_transformer_mlp_shard_gb300 as tp
    c = s["case"]
    if "norm" not in s:  # one object for a shape, as a program keeps it
        s["norm"] = tp.TPBlockNorm(
            S=c["S"], B=c["B"], H=c["H"], T=c["T"], dtype=c["dtype"], post=c["post"], pre=c["pre"], gate=c["gate"],
            block=not c.get("alone"), residual_f32=c["res32"], seq_parallel=c["T"] > 1, zero_centered=c["zero"],
            eps=s["eps"], residual_scale=c["a"], block_scale=c["c"])
        s["ws"] = tp.alloc_workspace(s["norm"].workspace_bytes()) if c["op"] == "norm_bwd" else None
    return s["norm"]


def _own_fwd(s):
    h, t = _own_handle(s), s["shards"]
    h.fwd(t["x"], t["f"], t.get("gate", s["gate"]), s["post_w"], s["post_b"], s["pre_w"], s["pre_b"], t["y"], t["n"],
          stats=s["stats"])
    return {"y": s["y"], "n": s["n"], "stats": s["stats"]}


def _own_bwd(s):
    h, t = _own_handle(s), s["shards"]
    h.bwd(t["dy"], t["dn"], t["y"], t["f"], t.get("gate", s["gate"]), s["post_w"], s["post_b"], s["pre_w"],
          s["stats"], t["dx"], t["df"], t.get("dgate", s["dgate"]), s["dpost_w"], s["dpost_b"], s["dpre_w"],
          s["dpre_b"], workspace=s["ws"])
    return {k: s[k] for k in ("dx", "df", "dgate", "dpost_w", "dpost_b", "dpre_w", "dpre_b")}


def _own_adamw(s):
    import tensor_transformer_mlp_shard_gb300 as tp
    c, t = s["case"], s["tensors"]
    if "opt" not in s:
        bf16 = c["param"] == "bf16"
        s["opt"] = tp.TPAdamW(t["p"] if bf16 else t["w"], t["g"], master=t["w"] if bf16 else None, m=t["m"], v=t["v"],
                              m_scale=t["ms"], v_scale=t["vs"], state_bits=c["bits"], beta1=BETA1, beta2=BETA2,
                              eps=EPS_ADAM, weight_decay=s["wd"], lr_scale=s["lr_scale"], seed=s["seed"],
                              steps_done=s["t"])
    opt, norm = s["opt"], None
    if c["clip"]:
        norm = opt.grad_norm(grad_scale=s["grad_scale"], max_norm=s["max_norm"])
        opt.step(LR)
    else:
        s["t"] += 1
        opt.step(LR, step=s["t"], grad_scale=s["grad_scale"])
    return _adamw_out(s, norm)


def _adamw_out(s, norm):
    codes = s["case"]["bits"] == 8
    return {"w": s["w"], "p": s["p"], "m": s["m"].view(torch.float8_e4m3fn) if codes else s["m"],
            "v": s["v"].view(torch.float8_e4m3fn) if codes else s["v"], "ms": s["ms"], "vs": s["vs"], "norm": norm}


def _weight(w, zero):
    return None if w is None else w.float() + (1.0 if zero else 0.0)


def _plain_norm(x, kind, w, b, eps):
    if kind == "none":
        return x, torch.zeros_like(x[:, 0]), torch.ones_like(x[:, 0])
    mean = x.mean(1) if kind == "layer" else torch.zeros_like(x[:, 0])
    x = x - mean[:, None]
    rstd = torch.rsqrt((x * x).mean(1) + eps)
    out = x * rstd[:, None] * w
    return out if b is None else out + b.float(), mean, rstd


def _plain_gate(s):
    g = s["gate"]
    return None if g is None else g.float()[:, None] if s["case"]["gate"] == "token" else g.float()


def _plain_fwd(s):
    c, eps = s["case"], s["eps"]
    x = s["x"]
    st = [torch.zeros_like(x[:, 0], dtype=torch.float32), torch.ones_like(x[:, 0], dtype=torch.float32)]
    y = x
    if s["f"] is not None:
        p, *st = _plain_norm(s["f"].float(), c["post"], _weight(s["post_w"], c["zero"]), s["post_b"], eps)
        g = _plain_gate(s)
        y = (c["a"] * x.float() + c["c"] * (p if g is None else g * p)).to(x.dtype)
    # the next block's norm is of the stream as it is stored
    n, *st2 = _plain_norm(y.float(), c["pre"], _weight(s["pre_w"], c["zero"]), s["pre_b"], eps)
    return {"y": None if s["f"] is None else y, "n": None if c["pre"] == "none" else n.to(s["n"].dtype),
            "stats": torch.stack(st + st2, 1) if c["train"] else None}


def _plain_norm_bwd(d, hat, rstd, kind, w):
    """Gradient of a norm's input, from that of its output."""
    if kind == "none":
        return d
    h = d * w
    out = h - hat * (h * hat).mean(1, keepdim=True)
    if kind == "layer":
        out = out - h.mean(1, keepdim=True)
    return out * rstd


def _plain_bwd(s):
    c = s["case"]
    mp, rp, mn, rn = (s["stats"][:, k:k + 1] for k in range(4))
    out = {"dx": None, "df": None, "dgate": None, "dpost_w": None, "dpost_b": None, "dpre_w": None, "dpre_b": None}
    D = s["dy"].float()
    if c["pre"] != "none":
        dn, hat = s["dn"].float(), (s["y"].float() - mn) * rn
        D = D + _plain_norm_bwd(dn, hat, rn, c["pre"], _weight(s["pre_w"], c["zero"]))
        out["dpre_w"] = (dn * hat).sum(0)
        out["dpre_b"] = dn.sum(0) if c["pre"] == "layer" else None
    out["dx"] = (c["a"] * D).to(s["dy"].dtype)
    if s["f"] is not None:
        f, g, w = s["f"].float(), _plain_gate(s), _weight(s["post_w"], c["zero"])
        hat = (f - mp) * rp if c["post"] != "none" else f
        D = c["c"] * D
        if g is not None:
            p = hat if w is None else hat * w if s["post_b"] is None else hat * w + s["post_b"].float()
            kind = c["gate"]
            out["dgate"] = (D * p).sum(0) if kind == "channel" else (D * p).sum(1).to(s["gate"].dtype) \
                if kind == "token" else (D * p).to(s["gate"].dtype)
            D = D * g
        if c["post"] != "none":
            out["dpost_w"] = (D * hat).sum(0)
            out["dpost_b"] = D.sum(0) if c["post"] == "layer" else None
        out["df"] = _plain_norm_bwd(D, hat, rp, c["post"], w).to(s["f"].dtype)
    return out


def _mix(x):
    """32 bits to 32 well-spread bits: xor-shifts and odd multipliers."""
    x = x ^ (x >> 16)
    x = (x * C1) & MASK
    x = x ^ (x >> 15)
    x = (x * C2) & MASK
    return x ^ (x >> 16)


def _random_bits(s, t):
    """32 random bits for each element at step t, from its tensor and its place in it."""
    at_step = torch.tensor((s["seed"] + C1 * t) & MASK, device="cuda")
    of_tensor = _mix(_mix(at_step) ^ ((s["which"] * C2 + 1) & MASK))
    of_block = _mix((of_tensor + s["block"]) & MASK)
    return _mix(of_block[:, None] ^ ((torch.arange(QBLOCK, device="cuda") * C1) & MASK))


def _round_8(x, bits):
    """x >= 0 to a neighbouring e4m3 value, the upper one with a probability of its nearness (16 bits of it)."""
    small = x < 2.0 ** -6  # there the steps stop shrinking: 2^-9
    t = torch.where(small, x + 2.0 ** -6, x)
    t = ((t.view(torch.int32) + (bits << 4).int()) & ~0xFFFFF).view(torch.float32)
    return torch.where(small, t - 2.0 ** -6, t).clamp(max=448.0)


def _pack_8(x, bits, keep):
    """Codes and scales of x in blocks; with `keep` no value above zero becomes zero."""
    top = x.abs().amax(1, keepdim=True)
    some = top >= 2.0 ** -100
    code = _round_8(x.abs() * torch.where(some, 448.0 / top, 0.0), bits)
    if keep:
        code = torch.where((x > 0) & some, code.clamp(min=2.0 ** -9), code)
    return torch.copysign(code, x).to(torch.float8_e4m3fn).view(torch.uint8), torch.where(some, top / 448.0, 0.0)


def _plain_adamw(s):
    c = s["case"]
    s["t"] += 1
    t, scale, norm = s["t"], s["grad_scale"], None
    if c["clip"]:
        norm = (s["g"].float().square().sum(dtype=torch.float64).sqrt() * scale).float().reshape(1)
        scale = scale * torch.clamp(s["max_norm"] / norm, max=1.0)
    w, g = s["w"].view(-1, QBLOCK), s["g"].view(-1, QBLOCK).float() * scale
    if c["bits"] == 32:
        m, v = s["m"].view(-1, QBLOCK), s["v"].view(-1, QBLOCK)
    else:
        m = s["m"].view(torch.float8_e4m3fn).float().view(-1, QBLOCK) * s["ms"][:, None]
        v = (s["v"].view(torch.float8_e4m3fn).float().view(-1, QBLOCK) * s["vs"][:, None]).square()
    m, v = BETA1 * m + (1 - BETA1) * g, BETA2 * v + (1 - BETA2) * g * g
    lr = LR * s["lr_block"]
    root = v.sqrt()
    step = (lr / (1 - BETA1 ** t)) * m / (root / math.sqrt(1 - BETA2 ** t) + EPS_ADAM)
    s["w"].copy_((w - lr * s["wd_block"] * w - step).reshape(-1))
    if s["p"] is not None:
        s["p"].copy_(s["w"])
    if c["bits"] == 32:
        s["m"].copy_(m.reshape(-1))
        s["v"].copy_(v.reshape(-1))
    else:
        bits = _random_bits(s, t)
        for key, x, b in (("m", m, bits & 0xFFFF), ("v", root, bits >> 16)):
            codes, scales = _pack_8(x, b, key == "v")
            s[key].copy_(codes.reshape(-1))
            s[key + "s"].copy_(scales.reshape(-1))
    return _adamw_out(s, norm)


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_adamw(s) if case["op"] == "adamw" else _exact_norm(s)


def _exact_norm(s):
    c, eps = s["case"], s["eps"]
    get = {k: None if s.get(k) is None else s[k].double() for k in
           ("x", "f", "y", "gate", "post_w", "post_b", "pre_w", "pre_b", "dy", "dn")}
    bwd = c["op"] == "norm_bwd"
    if bwd:
        for k in ("f", "y", "gate", "post_w", "post_b", "pre_w", "pre_b"):
            if get[k] is not None:
                get[k].requires_grad_()

    def spread(v, kind):
        if kind == "layer":
            var, mean = torch.var_mean(v, 1, correction=0, keepdim=True)
            return mean, (var + eps) ** -0.5
        return torch.zeros_like(v[:, :1]), (torch.linalg.vector_norm(v, dim=1, keepdim=True) ** 2 / c["H"] + eps) ** -0.5

    def norm(v, kind, side):
        if kind == "none":
            return v, torch.zeros_like(v[:, :1]), torch.ones_like(v[:, :1])
        mean, r = spread(v, kind)
        weight = get[side + "_w"] + 1 if c["zero"] else get[side + "_w"]
        out = (v - mean) * r * weight
        return (out + get[side + "_b"] if kind == "layer" else out), mean, r

    one = torch.ones_like((get["y"] if bwd else get["x"])[:, :1])
    st, added = [0 * one, one], None
    if get["f"] is not None:
        p, *st = norm(get["f"], c["post"], "post")
        gate = get["gate"]
        added = c["c"] * (p if gate is None else p * (gate[:, None] if c["gate"] == "token" else gate))
    if not bwd:
        y = get["x"] if added is None else c["a"] * get["x"] + added
        # by definition the next norm is of the stream as it is stored
        n, *st2 = norm(y.to(s["x"].dtype).double(), c["pre"], "pre")
        return {"y": None if added is None else y, "n": None if c["pre"] == "none" else n,
                "stats": torch.cat(st + st2, 1) if c["train"] else None}
    # y is given as stored: first the gradient that reaches it, then that of what was added into it
    D, out = get["dy"], {}
    if c["pre"] != "none":
        wrt = ["y", "pre_w"] + (["pre_b"] if c["pre"] == "layer" else [])
        got = torch.autograd.grad(norm(get["y"], c["pre"], "pre")[0], [get[k] for k in wrt], get["dn"])
        D = D + got[0]
        out.update(zip(wrt[1:], got[1:]))
    if added is not None:
        wrt = [k for k in ("f", "gate", "post_w", "post_b") if get[k] is not None]
        out.update(zip(wrt, torch.autograd.grad(added, [get[k] for k in wrt], D)))
    return {"dx": c["a"] * D, "df": out.get("f"), "dgate": out.get("gate"), "dpost_w": out.get("post_w"),
            "dpost_b": out.get("post_b"), "dpre_w": out.get("pre_w"), "dpre_b": out.get("pre_b")}


def _exact_adamw(s):
    c, t, scale, norm = s["case"], s["t"] + 1, s["grad_scale"], None
    g = s["g"].double()
    if c["clip"]:
        norm = torch.linalg.vector_norm(g).reshape(1) * scale
        scale = scale * min(1.0, s["max_norm"] / float(norm))
    g *= scale
    scale_of = lambda k: s[k].double().repeat_interleave(QBLOCK)  # noqa: E731
    of_element = lambda v: torch.tensor(v, dtype=torch.float64, device="cuda")[s["which"]].repeat_interleave(QBLOCK)  # noqa: E731
    if c["bits"] == 32:
        m, v = s["m"].double(), s["v"].double()
    else:
        m = s["m"].view(torch.float8_e4m3fn).double() * scale_of("ms")
        v = (s["v"].view(torch.float8_e4m3fn).double() * scale_of("vs")) ** 2
    m = torch.lerp(g, m, BETA1)
    v = torch.lerp(g ** 2, v, BETA2)
    m_hat, v_hat = m / (1 - BETA1 ** t), v / (1 - BETA2 ** t)
    lr = of_element(s["lr_scale"]) * LR
    w = s["w"].double()
    w = w * (1 - lr * of_element(s["wd"])) - lr * m_hat / (v_hat.sqrt() + EPS_ADAM)
    out = {"w": w, "p": None if s["p"] is None else w, "m": m, "v": v, "ms": None, "vs": None, "norm": norm}
    if c["bits"] == 32:
        return out
    bits = _random_bits(s, t)
    for key, x, b in (("m", m, bits & 0xFFFF), ("v", v.sqrt(), bits >> 16)):
        x = x.view(-1, QBLOCK)
        top = x.abs().amax(1, keepdim=True)
        u = (x.abs() / top.clamp(min=2.0 ** -100)) * 448
        # e4m3 has 8 steps between powers of two, and none finer than 2^-9
        step = torch.exp2(torch.floor(torch.log2(u.clamp(min=2.0 ** -6))) - 3)
        code = torch.floor(u / step + b.double() / 65536) * step
        code = code.clamp(max=448.0)
        if key == "v":
            code = torch.where(x > 0, code.clamp(min=2.0 ** -9), code)
        out[key], out[key + "s"] = (torch.sign(x) * code).reshape(-1), (top / 448).reshape(-1)
    return out
