"""Refusals of the block norm and AdamW entry points (no GPU): every bad
descriptor, constant or pointer is an error before anything is enqueued."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_shard_gb300 import build
    build.build()
    import tensor_transformer_mlp_shard_gb300 as tp
    return tp


NORM_BASE = dict(S=16, B=2, H=64, T=1, dtype="bf16", post="rms", pre="layer", gate="channel")


def norm_create(tp, raw=None, **kw):
    base = {**NORM_BASE, **kw}
    try:
        h = tp.TPBlockNorm(**base)
    except tp.TpError as e:
        return e.status
    if raw:
        from tensor_transformer_mlp_shard_gb300.binding import VP
        for k, v in raw.items():
            setattr(h._d, k, v)
        out = VP()
        s = tp.lib().tp_block_norm_create(ctypes.byref(h._d), ctypes.byref(out))
        if s == 0:
            tp.lib().tp_block_norm_destroy(out)
        return s
    return 0


@pytest.mark.parametrize("kw,raw,expect", [
    ({}, None, 0),
    ({"H": 60}, None, 2),
    ({"H": 0}, None, 2),
    ({"H": 16384}, None, 0),
    ({"H": 16392}, None, 3),
    ({"T": 0}, None, 2),
    ({"T": 17}, None, 2),
    ({"S": 15, "T": 4, "seq_parallel": True}, None, 2),
    ({"S": 20, "T": 4, "seq_parallel": True}, None, 0),
    ({"S": -1}, None, 2),
    ({"S": 1 << 23, "B": 4}, None, 2),
    ({"S": 0}, None, 0),
    ({"eps": 0.0}, None, 1),
    ({"eps": float("nan")}, None, 1),
    ({"residual_scale": float("inf")}, None, 1),
    ({"block_scale": float("nan")}, None, 1),
    ({"dtype": "fp8"}, None, 1),
    ({"block": False}, None, 1),                                  # a post-norm and a gate without a block
    ({"block": False, "post": "none", "gate": "none"}, None, 0),
    ({"block": False, "post": "none", "gate": "none", "pre": "none"}, None, 1),
    ({"block": False, "post": "none", "gate": "none", "block_scale": 0.5}, None, 1),
    ({}, {"post": 3}, 1),
    ({}, {"pre": -1}, 1),
    ({}, {"gate": 4}, 1),
    ({}, {"zero_centered": 2}, 1),
    ({}, {"has_block": -1}, 1),
])
def test_block_norm_create(tp, kw, raw, expect):
    assert norm_create(tp, raw, **kw) == expect


def test_block_norm_create_null(tp):
    from tensor_transformer_mlp_shard_gb300.binding import VP, BlockNormDesc
    out = VP()
    assert tp.lib().tp_block_norm_create(None, ctypes.byref(out)) == 1
    assert tp.lib().tp_block_norm_create(ctypes.byref(BlockNormDesc()), None) == 1
    tp.lib().tp_block_norm_destroy(None)
    assert tp.lib().tp_block_norm_workspace_bytes(None) == 0


@pytest.mark.parametrize("drop", ["X", "F", "gate", "post_w", "pre_w", "pre_b", "Y", "N"])
@pytest.mark.parametrize("how", ["null", "misaligned"])
def test_block_norm_fwd_pointers(tp, drop, how):
    from tensor_transformer_mlp_shard_gb300.binding import _arr
    h = tp.TPBlockNorm(**NORM_BASE)
    at = {k: 0x10000 * (i + 1) for i, k in enumerate(("X", "F", "gate", "post_w", "post_b", "pre_w", "pre_b", "Y", "N"))}
    at[drop] = None if how == "null" else at[drop] + 8
    a = lambda k: _arr([at[k]])  # noqa: E731
    s = tp.lib().tp_block_norm_fwd(h._h, a("X"), a("F"), a("gate"), at["post_w"], at["post_b"], at["pre_w"],
                                   at["pre_b"], a("Y"), a("N"), None, None)
    assert s == 1 and drop.encode() in tp.lib().tp_last_error()
    if drop in ("X", "F", "gate", "Y", "N") and how == "null":
        arrays = {k: None if k == drop else a(k) for k in ("X", "F", "gate", "Y", "N")}
        s = tp.lib().tp_block_norm_fwd(h._h, arrays["X"], arrays["F"], arrays["gate"], at["post_w"], at["post_b"],
                                       at["pre_w"], at["pre_b"], arrays["Y"], arrays["N"], None, None)
        assert s == 1 and drop.encode() in tp.lib().tp_last_error()


@pytest.mark.parametrize("drop", ["dY", "dN", "Y", "F", "gate", "post_w", "pre_w", "stats", "dX", "dF", "dgate",
                                  "dpost_w", "dpre_w", "dpre_b", "ws"])
def test_block_norm_bwd_pointers(tp, drop):
    from tensor_transformer_mlp_shard_gb300.binding import _arr
    h = tp.TPBlockNorm(**NORM_BASE)
    keys = ("dY", "dN", "Y", "F", "gate", "post_w", "post_b", "pre_w", "stats", "dX", "dF", "dgate", "dpost_w",
            "dpost_b", "dpre_w", "dpre_b", "ws")
    at = {k: 0x10000 * (i + 1) for i, k in enumerate(keys)}
    at[drop] += 8
    a = lambda k: _arr([at[k]])  # noqa: E731

    def call(nbytes):
        return tp.lib().tp_block_norm_bwd(
            h._h, a("dY"), a("dN"), a("Y"), a("F"), a("gate"), at["post_w"], at["post_b"], at["pre_w"], at["stats"],
            a("dX"), a("dF"), a("dgate"), at["dpost_w"], at["dpost_b"], at["dpre_w"], at["dpre_b"], at["ws"], nbytes,
            None)

    assert call(1 << 30) == 1
    if drop == "ws":
        at["ws"] -= 8
        assert call(h.workspace_bytes() - 1) == 1 and b"workspace" in tp.lib().tp_last_error()
    else:
        assert drop.encode() in tp.lib().tp_last_error()


def test_block_norm_workspace(tp):
    """One row of partial sums a block (at most 304 from 4096 columns on, 1216 up
    to 1024, and at most one a token) for each of the sums the parameters need."""
    assert tp.TPBlockNorm(**{**NORM_BASE, "S": 1000}).workspace_bytes() == 4 * 3 * 1216 * 64
    assert tp.TPBlockNorm(**{**NORM_BASE, "S": 1000, "H": 4096}).workspace_bytes() == 4 * 3 * 304 * 4096
    assert tp.TPBlockNorm(**{**NORM_BASE, "S": 1000, "H": 2048}).workspace_bytes() == 4 * 3 * 608 * 2048
    assert tp.TPBlockNorm(**{**NORM_BASE, "S": 3}).workspace_bytes() == 4 * 3 * 6 * 64
    assert tp.TPBlockNorm(16, 2, 64, post="none", pre="none", gate="element").workspace_bytes() == 0


def adamw_create(tp, n=3, sizes=(100, 0, 300), edit=None, **kw):
    from tensor_transformer_mlp_shard_gb300.binding import VP, AdamWDesc, AdamWTensor
    d = AdamWDesc(n, 1, 0, 8, 0.9, 0.95, 1e-8, 0)
    t = (AdamWTensor * max(1, len(sizes)))()
    for i, k in enumerate(sizes):
        if k:
            base = 0x100000 * (i + 1)
            t[i].param, t[i].master, t[i].grad, t[i].m, t[i].v = (base + 0x1000 * j for j in range(5))
            t[i].m_scale, t[i].v_scale = base + 0x8004, base + 0x9004
        t[i].n, t[i].lr_scale, t[i].weight_decay = k, 1.0, 0.1
    for k, v in kw.items():
        setattr(d, k, v)
    if edit:
        setattr(t[edit[0]], edit[1], edit[2])
    out = VP()
    s = tp.lib().tp_adamw_create(ctypes.byref(d), t, ctypes.byref(out))
    return s, out


@pytest.mark.parametrize("kw,edit,expect", [
    ({}, None, 0),
    ({"n_tensors": 0}, None, 2),
    ({"n_tensors": 65537}, None, 2),
    ({"param_dtype": 2}, None, 1),
    ({"grad_dtype": 2}, None, 1),
    ({"state_bits": 16}, None, 1),
    ({"beta1": 1.0}, None, 1),
    ({"beta2": -0.1}, None, 1),
    ({"beta2": float("nan")}, None, 1),
    ({"eps": 0.0}, None, 1),
    ({}, (0, "n", -1), 2),
    ({}, (2, "n", 1 << 39), 2),
    ({}, (0, "param", None), 1),
    ({}, (0, "param", 0x100008), 1),
    ({}, (2, "master", None), 1),
    ({"param_dtype": 0}, (2, "master", None), 0),
    ({}, (2, "grad", 0x300004), 1),
    ({}, (0, "m", None), 1),
    ({}, (0, "v", 0x100001), 1),
    ({}, (0, "m_scale", None), 1),
    ({}, (0, "v_scale", 0x100002), 1),
    ({"state_bits": 32}, (0, "v_scale", None), 0),
    ({}, (1, "lr_scale", float("inf")), 1),
    ({}, (1, "weight_decay", float("nan")), 1),
])
def test_adamw_create(tp, kw, edit, expect):
    s, h = adamw_create(tp, edit=edit, **kw)
    assert s == expect
    if s == 0:
        tp.lib().tp_adamw_destroy(h)


def test_adamw_calls(tp):
    from tensor_transformer_mlp_shard_gb300.binding import VP, _arr
    L = tp.lib()
    s, h = adamw_create(tp)
    assert s == 0
    ctl = VP(0x10000)
    assert L.tp_adamw_create(None, None, ctypes.byref(VP())) == 1
    assert L.tp_adamw_step(None, 0.1, 1.0, 1, None, None) == 1
    assert L.tp_adamw_step(h, float("nan"), 1.0, 1, None, None) == 1
    assert L.tp_adamw_step(h, 0.1, 1.0, 0, None, None) == 1            # steps count from 1
    assert L.tp_adamw_step(h, 0.1, float("inf"), 1, None, None) == 1
    assert L.tp_adamw_step(h, 0.1, 1.0, 1, VP(0x10010), None) == 1     # misaligned control block
    assert L.tp_adamw_grad_norm(h, 1.0, 1.0, None, None) == 1
    assert L.tp_adamw_grad_norm(h, 0.0, 1.0, ctl, None) == 1
    assert L.tp_adamw_grad_norm(h, 1.0, 0.0, ctl, None) == 1
    assert L.tp_adamw_grad_norm(h, 1.0, float("nan"), ctl, None) == 1
    assert L.tp_adamw_grad_norm(None, 1.0, 1.0, ctl, None) == 1
    assert L.tp_adamw_ctl_init(None, 0, None) == 1
    assert L.tp_adamw_ctl_init(ctl, -1, None) == 1
    assert L.tp_adamw_set_grads(h, None) == 1
    assert L.tp_adamw_set_grads(h, _arr([0x1000, None, None])) == 1    # the third has elements
    assert L.tp_adamw_set_grads(h, _arr([0x1000, None, 0x2004])) == 1
    assert L.tp_adamw_set_grads(h, _arr([0x1000, None, 0x2000])) == 0
    L.tp_adamw_destroy(h)
    L.tp_adamw_destroy(None)


def test_binding_refuses_cpu_tensors(tp):
    torch = pytest.importorskip("torch")
    h = tp.TPBlockNorm(4, 1, 64, pre="rms")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="X"):
        h.fwd(x, x, None, None, None, x[0], None, x, x)
    with pytest.raises(ValueError, match="params"):
        tp.TPAdamW([torch.zeros(8)], [torch.zeros(8)])
    with pytest.raises(ValueError, match="state_bits"):
        tp.TPAdamW([torch.zeros(8)], [torch.zeros(8)], state_bits=4)
