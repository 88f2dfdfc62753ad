"""An optimizer rebuilt from saved states goes on where the first one stopped,
and refuses a state of which a part is missing."""
import pytest
import torch

pytestmark = pytest.mark.gpu

N = [300, 5000, 1]


@pytest.fixture(scope="module")
def tp():
    import tensor_transformer_mlp_shard_gb300 as tp
    from tensor_transformer_mlp_shard_gb300 import build
    build.build()
    return tp


def trained(tp, bits, steps=3):
    gen = torch.Generator(device="cuda").manual_seed(4)
    w = [torch.randn(n, generator=gen, device="cuda") for n in N]
    g = [torch.randn(n, generator=gen, device="cuda") for n in N]
    opt = tp.TPAdamW(w, g, state_bits=bits, seed=2)
    for t in range(1, steps + 1):
        opt.step(1e-2, step=t)
    return w, g, opt


@pytest.mark.parametrize("bits", [32, 8])
def test_resumed(tp, bits):
    w, g, opt = trained(tp, bits)
    copy = lambda ts: None if ts is None else [t.clone() for t in ts]  # noqa: E731
    w2 = copy(w)
    again = tp.TPAdamW(w2, g, state_bits=bits, seed=2, m=copy(opt.m), v=copy(opt.v), m_scale=copy(opt.m_scale),
                       v_scale=copy(opt.v_scale))
    for o in (opt, again):
        o.step(1e-2, step=4)
    for a, b in ((w, w2), (opt.m, again.m), (opt.v, again.v)):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("bits,left_out,message", [
    (8, "m_scale", "m_scale: required with m"), (8, "v_scale", "v_scale: required with v"),
    (8, "m", "m: required with m_scale"), (32, "v", "v: required with m"), (32, "m", "m: required with v")])
def test_a_state_in_part_is_refused(tp, bits, left_out, message):
    w, g, opt = trained(tp, bits)
    parts = dict(m=opt.m, v=opt.v, m_scale=opt.m_scale, v_scale=opt.v_scale)
    parts[left_out] = None
    with pytest.raises(ValueError, match=message):
        tp.TPAdamW(w, g, state_bits=bits, **parts)


def test_zero_states_may_come_in_part(tp):
    """A caller's buffers for a run that starts: nothing is lost."""
    zeros = lambda dtype: [torch.zeros(n, dtype=dtype, device="cuda") for n in N]  # noqa: E731
    w, g = zeros(torch.float32), [torch.ones(n, device="cuda") for n in N]
    for kw in (dict(state_bits=8, m=zeros(torch.uint8), v=zeros(torch.uint8)), dict(m=zeros(torch.float32)),
               dict(state_bits=8, v=zeros(torch.uint8))):
        tp.TPAdamW(w, g, **kw).step(0.0, step=1)
