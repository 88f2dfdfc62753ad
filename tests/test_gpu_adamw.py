"""GPU parity of the AdamW step and the gradient norm against the fp64 oracle.

Tolerances (u = 2^-24): m is three fp32 roundings of terms of at most |m| +
|g'|, v four; the weight's change carries the roundings of m, v, a square
root, a division and six products, under 24 u of it, and the new weight three
of its own magnitude.  A bf16 parameter is exactly the rounded master copy.
An 8-bit code may differ from the oracle's only where the value lies within
the fp32 error of the random threshold it is compared with: 2^-24 * 32 of its
position, in steps.  Norms: fp32 squares, 8 of them added in fp32: 16 u.
"""
import numpy as np
import pytest
import torch

from oracle import adamw as oa

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SIZES = [1, 3, 4, 255, 256, 257, 0, 2047, 2048, 2049, 5000, 16, 40001]
B1, B2, EPS = 0.9, 0.95, 1e-8


@pytest.fixture(scope="module")
def tp():
    import tensor_transformer_mlp_shard_gb300 as tp
    from tensor_transformer_mlp_shard_gb300 import build
    build.build()
    return tp


def f64(t):
    return t.detach().double().cpu().numpy()


class Setup:
    """Tensors inside guarded buffers, their optimizer and copies of the start."""

    def __init__(self, tp, sizes=SIZES, param="bf16", grad="f32", bits=32, seed=0, state=True, g_scale=1e-2, **kw):
        gen = torch.Generator(device="cuda").manual_seed(77 + seed)
        self.bits, self.half, self.sizes = bits, param == "bf16", sizes
        self.buffers = []

        def place(values, dtype, pad=64):
            """values in the middle of a buffer of a known pattern"""
            n = values.numel()
            room = -(-n // 64) * 64
            buf = torch.full((pad + room + pad,), 3, dtype=dtype, device="cuda")
            t = buf[pad:pad + n]
            t.copy_(values)
            self.buffers.append((buf, pad, n))
            return t

        def normal(n, std=1.0):
            return torch.randn(n, generator=gen, device="cuda") * std

        f32 = torch.float32
        w = [normal(n, 0.02) for n in sizes]
        self.w = [place(t, f32) for t in w]
        self.p = [place(t.bfloat16(), torch.bfloat16) for t in w] if self.half else None
        gt = f32 if grad == "f32" else torch.bfloat16
        self.g = [normal(n, g_scale).to(gt) for n in sizes]
        m, r = [normal(n, g_scale / 3) for n in sizes], [normal(n, g_scale).abs() for n in sizes]
        if not state:
            m, r = [torch.zeros_like(t) for t in m], [torch.zeros_like(t) for t in r]
        self.ms = self.vs = None
        if bits == 32:
            self.m, self.v = [place(t, f32) for t in m], [place(t * t, f32) for t in r]
        else:
            self.m, self.v, self.ms, self.vs = [], [], [], []
            for src, codes, scales in ((m, self.m, self.ms), (r, self.v, self.vs)):
                for t in src:
                    s = torch.from_numpy(oa.block_scales(f64(t))).float().cuda()
                    full = s.repeat_interleave(256)[:t.numel()]
                    q = torch.where(full > 0, t / full, 0.0).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                    codes.append(place(q, torch.uint8))
                    scales.append(place(s, f32))
        self.lr_scale = [1.0 + 0.5 * (i % 2) for i in range(len(sizes))]
        self.wd = [0.1 * (i % 3) for i in range(len(sizes))]
        self.before = self.state()
        self.opt = tp.TPAdamW(self.p if self.half else self.w, self.g, master=self.w if self.half else None, m=self.m,
                              v=self.v, m_scale=self.ms, v_scale=self.vs, state_bits=bits, beta1=B1, beta2=B2, eps=EPS,
                              weight_decay=self.wd, lr_scale=self.lr_scale, seed=9, **kw)

    def state(self):
        out = {"w": [f64(t) for t in self.w], "g": [f64(t) for t in self.g]}
        if self.bits == 32:
            out["m"], out["v"] = [f64(t) for t in self.m], [f64(t) for t in self.v]
        else:
            out["mc"], out["vc"] = [t.cpu().numpy().copy() for t in self.m], [t.cpu().numpy().copy() for t in self.v]
            out["ms"], out["vs"] = [f64(t) for t in self.ms], [f64(t) for t in self.vs]
            out["m"] = [oa.decode(a, b) for a, b in zip(out["mc"], out["ms"])]
            out["v"] = [oa.decode(a, b) ** 2 for a, b in zip(out["vc"], out["vs"])]
        return out

    def intact(self):
        return all(bool((b[:p] == 3).all() and (b[p + n:] == 3).all()) for b, p, n in self.buffers)

    def tensors(self):
        return [t for k in (self.w, self.p, self.m, self.v, self.ms, self.vs) if k is not None for t in k]

    def check(self, t, lr, scale, before=None):
        """The state now is one step from `before`."""
        before, now = before or self.before, self.state()
        for i, n in enumerate(self.sizes):
            w0, g, m0, v0 = (before[k][i] for k in ("w", "g", "m", "v"))
            l = lr * self.lr_scale[i]
            w, m, v = oa.update(w0, g, m0, v0, t, l, B1, B2, EPS, self.wd[i], scale)
            change = np.abs(w - w0) + l * np.abs(g * scale) / (np.sqrt(v) + EPS)
            assert (np.abs(now["w"][i] - w) <= 3 * U * np.abs(w0) + 24 * U * change).all(), (i, n)
            if self.half:
                assert torch.equal(self.p[i], self.w[i].bfloat16())
            if self.bits == 32:
                assert (np.abs(now["m"][i] - m) <= 4 * U * (np.abs(m0) + np.abs(g * scale))).all(), (i, n)
                assert (np.abs(now["v"][i] - v) <= 8 * U * v + 2.0 ** -148).all(), (i, n)
            else:
                bits = oa.random_bits(9, t, i, n)
                # rounding of m cancels against terms of |m0| and |g'|; relative to the block's largest value it is small
                for x, size, codes, scales, b, root in (
                        (m, B1 * np.abs(m0) + (1 - B1) * np.abs(g * scale), now["mc"][i], now["ms"][i],
                         bits & np.uint64(0xFFFF), False),
                        (np.sqrt(v), np.sqrt(v), now["vc"][i], now["vs"][i], bits >> np.uint64(16), True)):
                    want = oa.block_scales(x)
                    assert (np.abs(scales - want) <= 16 * U * (want + oa.block_scales(size))).all(), (i, n)
                    _, step, at = oa.positions(x, want, b)
                    err = 32 * U * (1 + at + np.abs(size) / np.where(np.abs(x) > 0, np.abs(x), 1) * at)
                    got = np.abs(oa.e4m3_values()[codes])
                    low = np.minimum(np.floor(at - err) * step, 448)
                    high = np.minimum(np.floor(at + err) * step, 448)
                    if root:
                        some = (x > 0) & (np.repeat(want, 256)[:n] > 0)
                        low, high = (np.where(some, np.maximum(a, 2.0 ** -9), a) for a in (low, high))
                    # at - err may fall below a power of two, where the steps are half as large
                    ok = (got >= low - step / 2 * (low < got)) & (got <= high)
                    ok &= (got == low) | (got == high) | (np.floor(at - err) != np.floor(at + err))
                    assert ok.all(), (i, n, root, int((~ok).sum()))
                    signs = np.sign(oa.e4m3_values()[codes])
                    assert (signs * np.sign(x) >= 0).all()
        assert self.intact()


TYPES = [(p, g, b) for p in ("bf16", "f32") for g in ("f32", "bf16") for b in (32, 8)]


@pytest.mark.parametrize("param,grad,bits", TYPES)
def test_step(tp, param, grad, bits):
    s = Setup(tp, param=param, grad=grad, bits=bits)
    s.opt.step(1e-2, step=7, grad_scale=0.25)
    s.check(7, 1e-2, 0.25)
    before = s.state()
    s.opt.step(3e-3, step=8)
    s.check(8, 3e-3, 1.0, before)


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_from_zero_states(tp, bits):
    s = Setup(tp, bits=bits, state=False)
    s.opt.step(1e-3, step=1)
    s.check(1, 1e-3, 1.0)


@pytest.mark.parametrize("param,grad,bits", TYPES[::3])
def test_clipped_step(tp, param, grad, bits):
    s = Setup(tp, param=param, grad=grad, bits=bits, steps_done=4)
    total = float(np.sqrt(sum((g ** 2).sum() for g in s.before["g"]))) * 0.5
    norm = s.opt.grad_norm(grad_scale=0.5, max_norm=total / 3)
    s.opt.step(1e-2)
    assert abs(float(norm) - total) <= 16 * U * total
    assert int(s.opt.finite) == 1 and int(s.opt.steps) == 5
    assert abs(float(s.opt.scale) - 0.5 / 3) <= 24 * U
    s.check(5, 1e-2, float(s.opt.scale))
    before = s.state()
    s.opt.grad_norm(max_norm=1e9)  # above the norm: nothing is clipped
    s.opt.step(1e-2)
    assert float(s.opt.scale) == 1.0
    s.check(6, 1e-2, 1.0, before)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_step_that_is_not_finite_changes_nothing(tp, bits, value):
    s = Setup(tp, bits=bits, steps_done=3)
    s.g[12][777] = value
    was = [t.clone() for t in s.tensors()]
    s.opt.grad_norm(max_norm=1.0)
    s.opt.step(1e-2)
    assert int(s.opt.finite) == 0 and int(s.opt.steps) == 3
    assert all(torch.equal(a, b) for a, b in zip(was, s.tensors()))
    s.g[12][777] = 0.01
    before = s.state()
    s.opt.grad_norm()
    s.opt.step(1e-2)
    assert int(s.opt.finite) == 1 and int(s.opt.steps) == 4
    s.check(4, 1e-2, 1.0, before)


def test_a_step_before_any_norm_changes_nothing(tp):
    s = Setup(tp)
    was = [t.clone() for t in s.tensors()]
    s.opt.step(1e-2)
    assert all(torch.equal(a, b) for a, b in zip(was, s.tensors()))


@pytest.mark.parametrize("count", [40, 41, 360, 361, 420, 421, 860])
@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(tp, count, bits):
    """Lists around the sizes of one launch's tables; the norm is of all of them."""
    s = Setup(tp, sizes=[(i * 37) % 700 for i in range(count)], bits=bits)
    total = float(np.sqrt(sum((g ** 2).sum() for g in s.before["g"])))
    norm = s.opt.grad_norm(max_norm=total / 2)
    s.opt.step(1e-2)
    assert abs(float(norm) - total) <= 16 * U * total
    s.check(1, 1e-2, float(s.opt.scale))


def test_blocks_of_zeros_and_tiny_values(tp):
    """A block without a gradient or a state stays zero; a root above zero keeps a code above zero."""
    s = Setup(tp, sizes=[1024], bits=8, state=False)
    s.g[0][256:512] = 0
    s.g[0][512:768] = 1e-33                # its root's block scale is below 2^-100: kept as zero
    s.g[0][768:] = 1e-9
    s.g[0][768] = 1.0                      # 2^30 above the rest of its block
    s.before = s.state()
    s.opt.step(1e-2, step=1)
    s.check(1, 1e-2, 1.0)
    assert (s.m[0][256:768] == 0).all() and (s.v[0][256:768] == 0).all()
    assert (s.ms[0][1:3] == 0).all() and (s.vs[0][1:3] == 0).all()
    assert (s.v[0][768:] > 0).all() and s.v[0][769] == 1


@pytest.mark.parametrize("g_scale", [3e3, 1e6, 1e12, 1e-6, 1e-12])
def test_states_of_any_size(tp, g_scale):
    """Block scales far from 1 on either side, up to squares near fp32's largest."""
    s = Setup(tp, sizes=[5000, 257], bits=8, g_scale=g_scale)
    s.opt.step(1e-2, step=3)
    s.check(3, 1e-2, 1.0)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_bad_gradient_without_the_norm_stays_in_its_block(tp, value):
    """Its block's states become NaN, which no later step hides; the others are as without it."""
    s, clean = (Setup(tp, sizes=[1024], bits=8) for _ in range(2))
    s.g[0][300] = value
    s.opt.step(1e-2, step=1)
    clean.opt.step(1e-2, step=1)
    assert not torch.isfinite(s.w[0][300])
    rest = torch.arange(1024, device="cuda") != 300
    assert torch.equal(s.w[0][rest], clean.w[0][rest])
    far = torch.arange(1024, device="cuda") // 256 != 1
    for a, b in ((s.m, clean.m), (s.v, clean.v)):
        assert torch.equal(a[0][far], b[0][far]) and ((a[0][~far] & 0x7F) == 0x7F).all()


def test_set_grads(tp):
    s, ref = Setup(tp), Setup(tp)
    other = [g * -2 for g in s.g]
    s.opt.set_grads(other)
    for g in ref.g:
        g.mul_(-2)
    s.opt.step(1e-2, step=1)
    ref.opt.step(1e-2, step=1)
    assert all(torch.equal(a, b) for a, b in zip(s.tensors(), ref.tensors()))
    with pytest.raises(ValueError, match="grads"):
        s.opt.set_grads(other[:-1])
    with pytest.raises(ValueError, match="grads"):
        s.opt.set_grads([g.bfloat16() for g in other])


@pytest.mark.parametrize("bits", [32, 8])
def test_same_results_every_time_on_any_stream_and_in_a_graph(tp, bits):
    a, b, c = (Setup(tp, bits=bits) for _ in range(3))
    for _ in range(3):
        a.opt.grad_norm(max_norm=0.5)
        a.opt.step(1e-2)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        b.opt.grad_norm(max_norm=0.5, stream=st)
        b.opt.step(1e-2, stream=st)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.opt.grad_norm(max_norm=0.5)
        c.opt.step(1e-2)
    for _ in range(3):  # each replay is the next step
        g.replay()
    torch.cuda.synchronize()
    assert int(c.opt.steps) == 3
    for x, y, z in zip(a.tensors(), b.tensors(), c.tensors()):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_long_training_in_8_bits_keeps_up(tp):
    """400 steps on gradients of a fixed variance: v's mean must reach it,
    although a step moves v by 5 %, less than half a step of its codes.  The
    variance of the rounding adds to v: under 10 %."""
    n = 1 << 16
    w, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    opt = tp.TPAdamW([w], [g], state_bits=8, beta1=B1, beta2=0.99, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(5)
    for t in range(1, 1001):
        g.normal_(generator=gen)
        opt.step(1e-4, step=t)
    r = opt.v[0].view(torch.float8_e4m3fn).float() * opt.v_scale[0].repeat_interleave(256)
    assert abs(float((r * r).mean()) - 1.0) < 0.1


def test_offsets_beyond_32_bits(tp):
    n = (1 << 31) + 4099
    w = torch.zeros(n, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    opt = tp.TPAdamW([w], [g], m=[m], v=[v], state_bits=8, beta1=B1, beta2=B2)
    g[-5000:] = 0.5
    norm = opt.grad_norm()
    opt.step(1e-2)
    assert abs(float(norm) - (5000 * 0.25) ** 0.5) < 1e-4
    assert (w[:-5000] == 0).all()
    np.testing.assert_allclose(f64(w[-5000:]), -1e-2, rtol=1e-5)
    assert (m[-5000:] > 0).all() and (m[:-5000] == 0).all()
