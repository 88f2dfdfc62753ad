"""GPU parity of the block norm against its fp64 oracle.

Tolerances, from the arithmetic (u = 2^-24, an fp32 rounding):
* an output stored in bf16 is rounded once: 2^-8 of its value;
* before that it is a few fp32 operations and sums of at most 32 elements a
  thread, 5 shuffles and 16 warps, less than 64 roundings: 64 u of the largest
  term of its row;
* a sum over tokens adds at most M / blocks + 304 / 8 + 8 terms in a row of
  its own and each term carries under 16 roundings; with the sizes here that
  is below 100 u of the sum of the terms' magnitudes.
n is compared with the norm of the stored y, which is what it is of.
"""
import numpy as np
import pytest
import torch

from oracle import block_norm as ob

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5
GUARD = 64  # elements around every output that must stay as they are


@pytest.fixture(scope="module")
def tp():
    import tensor_transformer_mlp_shard_gb300 as tp
    from tensor_transformer_mlp_shard_gb300 import build
    build.build()
    return tp


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


class Guarded:
    """An output inside a larger buffer filled with a pattern."""

    def __init__(self, shape, dtype):
        n = int(np.prod(shape))
        self.buf = torch.full((n + 2 * GUARD,), 7.5, dtype=dtype, device="cuda")
        self.t = self.buf[GUARD:GUARD + n].view(shape)
        self.t.fill_(float("nan"))

    def intact(self):
        return bool((self.buf[:GUARD] == 7.5).all() and (self.buf[self.buf.numel() - GUARD:] == 7.5).all())


class Case:
    def __init__(self, M, H, dtype="bf16", post="rms", pre="rms", gate="none", res32=False, block=True, zc=False, T=1,
                 a=1.0, c=1.0, seed=0, edit=None):
        self.__dict__.update({k: v for k, v in locals().items() if k != "self"})
        act = torch.float32 if dtype == "f32" else torch.bfloat16
        res = torch.float32 if res32 else act
        gen = torch.Generator(device="cuda").manual_seed(1000 + seed)

        def normal(*shape, dtype=act, mean=0.0):
            return (torch.randn(*shape, generator=gen, device="cuda") + mean).to(dtype)

        self.act, self.res = act, res
        self.x, self.dy, self.dn = normal(M, H, dtype=res, mean=0.2), normal(M, H, dtype=res), normal(M, H)
        self.f = normal(M, H, mean=-0.3) if block else None
        self.g = {"none": None, "channel": normal(H), "token": normal(M), "element": normal(M, H)}[gate]
        self.pw, self.pb, self.nw, self.nb = (normal(H) for _ in range(4))
        if edit:
            edit(self)

    def split(self, t):
        return None if t is None else list(t.view(self.T, -1).unbind(0)) if self.T > 1 else t

    def handle(self, tp):
        S, B = (self.M, 1)
        return tp.TPBlockNorm(S, B, self.H, T=self.T, dtype=self.dtype, post=self.post, pre=self.pre, gate=self.gate,
                              block=self.block, residual_f32=self.res32, seq_parallel=self.T > 1,
                              zero_centered=self.zc, eps=EPS, residual_scale=self.a, block_scale=self.c)

    def run_fwd(self, h, y=None, stream=None):
        M, H = self.M, self.H
        self.o = {"y": Guarded((M, H), self.res), "n": Guarded((M, H), self.act), "stats": Guarded((M, 4), torch.float32)}
        self.y = (self.o["y"].t if y is None else y) if self.block else self.x
        sp = self.split
        gate = self.g if self.gate == "channel" else sp(self.g)
        h.fwd(sp(self.x), sp(self.f), gate, self.pw, self.pb, self.nw, self.nb, sp(self.y) if self.block else None,
              sp(self.o["n"].t), stats=self.o["stats"].t, stream=stream)
        self.n, self.stats = self.o["n"].t, self.o["stats"].t

    def check_fwd(self):
        half = 2.0 ** -8 if self.act == torch.bfloat16 else U
        half_y = 2.0 ** -8 if self.res == torch.bfloat16 else U
        if self.block:
            add = ob.added(f64(self.f), self.post, f64(self.pw), f64(self.pb), f64(self.g), self.gate == "token", self.c,
                           EPS, self.zc)
            ref = self.a * f64(self.x) + add
            self.near(self.y, ref, half_y, np.abs(f64(self.x)) + np.abs(add), "y")
        if self.pre != "none":
            ref = ob.norm(f64(self.y), self.pre, f64(self.nw), f64(self.nb), EPS, self.zc)
            terms = np.abs(ref) + (np.abs(f64(self.nb)) if self.pre == "layer" else 0)
            self.near(self.n, ref, half, terms, "n")
        mp, rp = ob.norm_stats(f64(self.f), self.post, EPS) if self.block else (np.zeros((self.M, 1)), np.ones((self.M, 1)))
        mn, rn = ob.norm_stats(f64(self.y), self.pre, EPS)
        self.near(self.stats, np.concatenate([mp, rp, mn, rn], 1), 0.0, None, "stats")
        assert all(g.intact() for g in self.o.values())

    @staticmethod
    def near(got, ref, half, terms, name):
        """|got - ref| <= half |ref| + 64 u (largest term of the row)."""
        got, ref = f64(got), np.asarray(ref)
        scale = np.abs(ref) if terms is None else terms
        tol = half * np.abs(ref) + 64 * U * scale.max(-1, keepdims=True)
        bad = ~(np.abs(got - ref) <= tol)
        assert not bad.any(), (name, int(bad.sum()), float(np.nanmax(np.abs(got - ref) / (tol + 1e-300))))

    def run_bwd(self, h, tp, dy=True, stream=None, inplace=False):
        M, H, f32 = self.M, self.H, torch.float32
        o = self.o = {"dx": Guarded((M, H), self.res), "df": Guarded((M, H), self.act)}
        if self.gate != "none":
            o["dgate"] = Guarded(tuple(self.g.shape), f32 if self.gate == "channel" else self.act)
        for k in ("dpost_w", "dpost_b", "dpre_w", "dpre_b"):
            o[k] = Guarded((H,), f32)
        ws = tp.alloc_workspace(h.workspace_bytes())
        sp = self.split
        chan = self.gate == "channel"
        dg = o["dgate"].t if "dgate" in o else None
        self.dy_used = f64(self.dy) if dy else None
        dx = self.dy if inplace else o["dx"].t
        h.bwd(sp(self.dy) if dy else None, sp(self.dn), sp(self.y), sp(self.f), self.g if chan else sp(self.g), self.pw,
              self.pb, self.nw, self.stats, sp(dx), sp(o["df"].t), dg if chan else sp(dg), o["dpost_w"].t,
              o["dpost_b"].t, o["dpre_w"].t, o["dpre_b"].t, workspace=ws, stream=stream)
        self.out = {k: v.t for k, v in o.items()}
        self.out["dx"] = dx

    def check_bwd(self):
        half = 2.0 ** -8 if self.act == torch.bfloat16 else U
        half_x = 2.0 ** -8 if self.res == torch.bfloat16 else U
        g, f, y, dn = f64(self.g), f64(self.f), f64(self.y), f64(self.dn)
        pw, pb, nw = f64(self.pw), f64(self.pb), f64(self.nw)
        ref = ob.grads(self.dy_used, dn, y, f, g, self.gate, self.post, pw, pb, self.pre, nw, self.a, self.c, EPS, self.zc)
        zc = 1.0 if self.zc else 0.0
        # magnitudes of the terms, row by row
        size = np.zeros_like(y) if self.dy_used is None else np.abs(self.dy_used)
        if self.pre != "none":
            mean, rstd = ob.norm_stats(y, self.pre, EPS)
            yh = np.abs(y - mean) * rstd
            size = size + rstd * np.abs(dn * (nw + zc)).max(1, keepdims=True) * (2 + yh)
        self.near(self.out["dx"], ref["dx"], half_x, size, "dx")
        sums = {"dpre_w": dn * ((np.abs(y) + np.abs(mean)) * rstd if self.pre != "none" else 0), "dpre_b": dn}
        if self.block:
            mean, rstd = ob.norm_stats(f, self.post, EPS)
            fh = (np.abs(f) + np.abs(mean)) * rstd
            pv = (fh * np.abs(pw + zc) + (np.abs(pb) if self.post == "layer" else 0)) if self.post != "none" else np.abs(f)
            e = abs(self.c) * size * (1.0 if g is None else np.abs(g[:, None] if self.gate == "token" else g))
            hp = e * (np.abs(pw + zc) if self.post != "none" else 1)
            self.near(self.out["df"], ref["df"], half, hp if self.post == "none" else rstd * hp.max(1, keepdims=True) * (2 + fh),
                      "df")
            sums.update(dpost_w=e * fh, dpost_b=e)
            dg = abs(self.c) * size * pv
            if self.gate == "element":
                self.near(self.out["dgate"], ref["dgate"], half, dg, "dgate")
            elif self.gate == "token":
                tol = half * np.abs(ref["dgate"]) + 100 * U * dg.sum(1)
                assert (np.abs(f64(self.out["dgate"]) - ref["dgate"]) <= tol).all()
            sums["dgate"] = dg
        for k, terms in sums.items():
            if ref[k] is None or (k == "dgate" and self.gate != "channel"):
                continue
            err = np.abs(f64(self.out[k]) - ref[k])
            assert (err <= 100 * U * np.abs(terms).sum(0)).all(), (k, float((err / (U * np.abs(terms).sum(0))).max()))
        assert all(v.intact() for v in self.o.values())


KINDS = [(p, q, g) for p in ("none", "rms", "layer") for q in ("none", "rms", "layer")
         for g in ("none", "channel", "token", "element")]


@pytest.mark.parametrize("post,pre,gate", KINDS)
def test_every_combination(tp, post, pre, gate):
    """Each norm on each side with each gate, on a warp's and a block's row."""
    for i, (M, H, dtype, res32) in enumerate([(13, 72, "bf16", False), (37, 1032, "bf16", True), (5, 264, "f32", False)]):
        c = Case(M, H, dtype, post, pre, gate, res32=res32, zc=i == 1, a=0.75, c=1.5, seed=i)
        h = c.handle(tp)
        c.run_fwd(h)
        c.check_fwd()
        c.run_bwd(h, tp)
        c.check_bwd()


# widths at both ends of every kernel variant (a warp up to 1024 columns with 8, 16 or 32 elements a lane, then a block
# with 8, 16 or 32 a thread), and token counts from one to more than one pass of the grid
WIDTHS = [8, 248, 256, 264, 512, 520, 1024, 1032, 2056, 4096, 4104, 8192, 8200, 16376, 16384]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dtype,res32", [("bf16", False), ("bf16", True), ("f32", False)])
def test_widths(tp, H, dtype, res32):
    for M in (1, 3, 29):
        c = Case(M, H, dtype, "layer", "rms", "channel", res32=res32, seed=H + M)
        h = c.handle(tp)
        c.run_fwd(h)
        c.check_fwd()
        c.run_bwd(h, tp)
        c.check_bwd()


@pytest.mark.parametrize("M,H", [(1501, 520), (3001, 96), (701, 2056), (613, 4096)])
def test_many_tokens(tp, M, H):
    c = Case(M, H, "bf16", "rms", "layer", "token", a=0.5, c=2.0)
    h = c.handle(tp)
    c.run_fwd(h)
    c.check_fwd()
    c.run_bwd(h, tp)
    c.check_bwd()


@pytest.mark.parametrize("gate", ["channel", "token", "element"])
@pytest.mark.parametrize("H", [264, 2056])
def test_token_shards(tp, gate, H):
    """T token shards hold what one buffer holds; M/T is odd (M = 5 * 8 tokens a shard of 16-byte aligned gates)."""
    c = Case(40, H, "bf16", "rms", "layer", gate, T=5)
    h = c.handle(tp)
    c.run_fwd(h)
    c.check_fwd()
    c.run_bwd(h, tp)
    c.check_bwd()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_token_gate_shards_need_no_vector_alignment(tp, dtype):
    """7 tokens a shard: a shard's gates start at any multiple of their type's size."""
    c = Case(35, 264, dtype, "rms", "layer", "token", T=5)
    h = c.handle(tp)
    c.run_fwd(h)
    c.check_fwd()
    c.run_bwd(h, tp)
    c.check_bwd()


def test_handles_of_one_kernel_take_turns(tp):
    """Configurations that stage more and less of a row run the same kernels:
    neither may keep the other from its shared memory."""
    cases = [Case(9, 4096, "bf16", "rms", "rms", "channel"), Case(9, 4096, "bf16", "none", "rms", "none"),
             Case(9, 2056, "bf16", "rms", "rms", "element"), Case(9, 2056, "bf16", "none", "rms", "none", block=False)]
    handles = [c.handle(tp) for c in cases]
    for _ in range(2):
        for dy in (True, False):
            for c, h in zip(cases, handles):
                c.run_fwd(h)
                c.check_fwd()
                c.run_bwd(h, tp, dy=dy)
                c.check_bwd()


def test_norm_without_a_block(tp):
    for kind in ("rms", "layer"):
        c = Case(19, 776, "bf16", "none", kind, block=False)
        h = c.handle(tp)
        c.run_fwd(h)
        c.check_fwd()
        c.run_bwd(h, tp)
        c.check_bwd()


def test_no_gradient_from_past_the_norm(tp):
    c = Case(19, 1544, "bf16", "rms", "rms", "channel")
    h = c.handle(tp)
    c.run_fwd(h)
    c.run_bwd(h, tp, dy=False)
    c.check_bwd()


@pytest.mark.parametrize("H", [512, 4096])
def test_in_place(tp, H):
    """Y may be X and dX may be dY; the results are those of separate buffers."""
    a, b = (Case(33, H, "bf16", "layer", "rms", "token") for _ in range(2))
    h = a.handle(tp)
    a.run_fwd(h)
    b.run_fwd(h, y=b.x)
    assert torch.equal(a.y, b.x) and torch.equal(a.n, b.n) and torch.equal(a.stats, b.stats)
    a.run_bwd(h, tp)
    b.run_bwd(h, tp, inplace=True)
    assert torch.equal(a.out["dx"], b.dy) and torch.equal(a.out["df"], b.out["df"])


def _odd_rows(c):
    c.f[0], c.x[0] = 0, 0                                  # nothing there: 1 / spread = 1 / sqrt(eps)
    c.f[1], c.x[1] = 300.0, 0                              # a constant row has no spread about its mean
    c.x[2] = 1000.0 + c.x[2].float()                       # a mean far above the spread
    c.x[3, 0], c.f[3, 0] = 30000.0, -20000.0               # one channel far above the others
    c.f[4], c.x[4] = c.f[4].float() * 1e-20, c.x[4].float() * 1e-20


@pytest.mark.parametrize("H", [512, 2056])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_odd_rows(tp, kind, H):
    c = Case(9, H, "f32", kind, kind, "token", edit=_odd_rows)
    h = c.handle(tp)
    c.run_fwd(h)
    c.check_fwd()
    assert torch.isfinite(c.n).all()


@pytest.mark.parametrize("H", [512, 2056])
def test_nan_and_infinity_stay_in_their_row(tp, H):
    def edit(c):
        c.f[3, 5], c.x[7, 9] = float("nan"), float("inf")

    c, clean = Case(12, H, "bf16", "rms", "layer", "element", edit=edit), Case(12, H, "bf16", "rms", "layer", "element")
    h = c.handle(tp)
    c.run_fwd(h)
    clean.run_fwd(h)
    rows = [i for i in range(12) if i not in (3, 7)]
    assert torch.equal(c.n[rows], clean.n[rows]) and torch.equal(c.y[rows], clean.y[rows])
    assert c.y[3].isnan().all() and c.y[7, 9].isinf() and c.n[7, 9].isnan()


def test_no_tokens(tp):
    c = Case(0, 520, "bf16", "layer", "layer", "channel")
    h = c.handle(tp)
    c.run_fwd(h)
    c.run_bwd(h, tp)
    for k in ("dpost_w", "dpost_b", "dpre_w", "dpre_b", "dgate"):
        assert (c.out[k] == 0).all(), k
    assert all(v.intact() for v in c.o.values())


@pytest.mark.parametrize("H", [264, 4096])
def test_same_results_every_time(tp, H):
    a, b = (Case(2000, H, "bf16", "rms", "layer", "channel") for _ in range(2))
    h = a.handle(tp)
    for c in (a, b):
        c.run_fwd(h)
        c.run_bwd(h, tp)
    for k in a.out:
        if k != "dpost_b":
            assert torch.equal(a.out[k], b.out[k]), k


def test_other_stream_and_graph(tp):
    """On a stream of the caller's, and captured: replays redo the whole pass."""
    c, ref = (Case(300, 2056, "bf16", "layer", "rms", "channel") for _ in range(2))
    h = c.handle(tp)
    ref.run_fwd(h)
    ref.run_bwd(h, tp)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        c.run_fwd(h)
        c.run_bwd(h, tp)
    st.synchronize()
    for k in c.out:
        assert torch.equal(c.out[k], ref.out[k]) or k in ("dpre_b",), k
    g = torch.cuda.CUDAGraph()
    ws = tp.alloc_workspace(h.workspace_bytes())
    o = c.out
    with torch.cuda.graph(g):
        h.fwd(c.x, c.f, c.g, c.pw, c.pb, c.nw, c.nb, c.y, c.n, stats=c.stats)
        h.bwd(c.dy, c.dn, c.y, c.f, c.g, c.pw, c.pb, c.nw, c.stats, o["dx"], o["df"], o["dgate"], o["dpost_w"],
              o["dpost_b"], o["dpre_w"], o["dpre_b"], workspace=ws)
    for _ in range(2):
        for t in (c.y, c.n, c.stats, *o.values()):
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for k in o:
            if k != "dpre_b":
                assert torch.equal(o[k], ref.out[k]), k


def test_binding_refuses(tp):
    c = Case(8, 64, "bf16", "rms", "rms", "token")
    h = c.handle(tp)
    good = dict(X=c.x, F=c.f, gate=c.g, post_w=c.pw, pre_w=c.nw, Y=torch.empty_like(c.x), N=torch.empty_like(c.f))
    h.fwd(**good)
    for key, bad in (("X", c.x.float()), ("F", c.f[:, :32]), ("gate", c.g[:4]), ("post_w", c.pw[:8]), ("pre_w", None),
                     ("Y", torch.empty(64, 8, dtype=c.act, device="cuda").t()), ("N", c.f.cpu()), ("X", [c.x, c.x])):
        with pytest.raises(ValueError, match=key):
            h.fwd(**{**good, key: bad})
    with pytest.raises(ValueError, match="stats"):
        h.fwd(**good, stats=torch.empty(8, 2, device="cuda"))


def test_offsets_beyond_32_bits(tp):
    """More than 2^31 elements: the last rows are as a small problem's."""
    H, M = 16384, 131072 + 77
    act = torch.bfloat16
    f = torch.empty(M, H, dtype=act, device="cuda").fill_(1.0)
    x = torch.empty_like(f).fill_(0.5)
    small = Case(3, H, "bf16", "rms", "rms")
    f[-3:], x[-3:] = small.f, small.x
    y, n, stats = torch.empty_like(f), torch.empty_like(f), torch.empty(M, 4, device="cuda")
    h = tp.TPBlockNorm(M, 1, H, post="rms", pre="rms", eps=EPS)
    h.fwd(x, f, None, small.pw, None, small.nw, None, y, n, stats=stats)
    hs = small.handle(tp)
    small.run_fwd(hs)
    assert torch.equal(n[-3:], small.n) and torch.equal(y[-3:], small.y) and torch.equal(stats[-3:], small.stats)
    dx, df = y, n  # the forward's outputs have been compared: their memory serves again
    dy, dn = x, f
    dy[-3:], dn[-3:] = small.dy, small.dn
    yy = torch.empty_like(f).fill_(1.0)
    yy[-3:] = small.y
    ff = torch.empty_like(f).fill_(1.0)
    ff[-3:] = small.f
    dw = [torch.empty(H, device="cuda") for _ in range(2)]
    h.bwd(dy, dn, yy, ff, None, small.pw, None, small.nw, stats, dx, df, None, dw[0], None, dw[1], None,
          workspace=tp.alloc_workspace(h.workspace_bytes()))
    small.run_bwd(hs, tp)
    assert torch.equal(dx[-3:], small.out["dx"]) and torch.equal(df[-3:], small.out["df"])
