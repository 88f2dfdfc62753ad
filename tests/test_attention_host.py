"""Refusals of the rotary and paged-attention entry points (no GPU): every bad
descriptor, size or pointer is an error before anything is enqueued."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_shard_gb300 import build
    build.build()
    import tensor_transformer_mlp_shard_gb300 as tp
    return tp


ROTARY = dict(S=16, B=2, heads=8, kv_heads=4, head_dim=64, T=2)
PAGED = dict(heads=8, kv_heads=4, head_dim=64, page_size=16, pages=10, T=2)
NAN, INF = float("nan"), float("inf")

# (keyword arguments, rope's, fields of the descriptor, status)
HEADS = [
    ({}, {}, {}, 0),
    ({"T": 0}, {}, {}, 2),
    ({"T": 17}, {}, {}, 2),
    ({"T": 3}, {}, {}, 2),                      # kv_heads % T
    ({"kv_heads": 0}, {}, {}, 2),
    ({"heads": 10}, {}, {}, 2),                 # heads % kv_heads
    ({"heads": 0}, {}, {}, 2),
    ({"heads": 4100}, {}, {}, 2),
    ({"head_dim": 0}, {}, {}, 2),
    ({"head_dim": 60}, {}, {}, 2),
    ({"head_dim": 264}, {}, {}, 3),
    ({"head_dim": 256}, {}, {}, 0),
    ({}, {}, {"grouped": 2}, 1),
    ({}, {"dim": 66}, {}, 1),
    ({}, {"dim": 31}, {}, 1),
    ({}, {"dim": -2}, {}, 1),
    ({}, {"dim": 0}, {}, 0),
    ({}, {"base": 0.5}, {}, 1),
    ({}, {"base": NAN}, {}, 1),
    ({}, {"base": INF}, {}, 1),
    ({}, {"scaling": "linear", "factor": 0.5}, {}, 1),
    ({}, {"scaling": "linear", "factor": NAN}, {}, 1),
    ({}, {"factor": 2.0}, {}, 1),               # a factor without a scaling
    ({}, {"scaling": "parts", "factor": 2.0}, {}, 1),  # no length trained on
    ({}, {"scaling": "parts", "factor": 2.0, "original": 100}, {}, 0),
    ({}, {"scaling": "parts", "factor": 2.0, "original": 100, "fast": 1.0}, {}, 1),
    ({}, {"scaling": "parts", "factor": 2.0, "original": 100, "slow": -1.0}, {}, 1),
    ({}, {"scaling": "parts", "factor": 2.0, "original": NAN}, {}, 1),
    ({}, {"attention_factor": -1.0}, {}, 1),
    ({}, {"attention_factor": NAN}, {}, 1),
    ({}, {}, {"dtype": 5}, 1),
]


def create(tp, cls, name, base, kw, rope, raw):
    try:
        h = cls(**{**base, **kw}, rope=tp.Rope(**rope))
    except tp.TpError as e:
        return e.status
    if raw:
        from tensor_transformer_mlp_shard_gb300.binding import VP
        for k, v in raw.items():
            setattr(h._d.rope if k in ("pairs", "scaling") else h._d, k, v)
        out = VP()
        s = getattr(tp.lib(), f"tp_{name}_create")(ctypes.byref(h._d), ctypes.byref(out))
        if s == 0:
            getattr(tp.lib(), f"tp_{name}_destroy")(out)
        return s
    return 0


@pytest.mark.parametrize("kw,rope,raw,expect", HEADS + [
    ({"S": -1}, {}, {}, 2),
    ({"S": 0}, {}, {}, 0),
    ({"S": 1 << 23, "B": 4}, {}, {}, 2),
    ({"dtype": "fp8"}, {}, {}, 1),
    ({}, {}, {"pairs": 2}, 1),
    ({}, {}, {"scaling": 4}, 1),
])
def test_rotary_create(tp, kw, rope, raw, expect):
    assert create(tp, tp.TPRotary, "rotary", ROTARY, kw, rope, raw) == expect


@pytest.mark.parametrize("kw,rope,raw,expect", HEADS + [
    ({"page_size": 0}, {}, {}, 2),
    ({"page_size": 8}, {}, {}, 2),
    ({"page_size": 24}, {}, {}, 2),
    ({"page_size": 48}, {}, {}, 0),
    ({"pages": 0}, {}, {}, 2),
    ({"window": -1}, {}, {}, 1),
    ({"scale": NAN}, {}, {}, 1),
    ({"scale": INF}, {}, {}, 1),
    ({"dtype": "fp8"}, {}, {}, 0),
    ({"dtype": "fp8", "head_dim": 72}, {}, {}, 2),
    ({"head_dim": 72}, {}, {}, 0),
])
def test_paged_create(tp, kw, rope, raw, expect):
    assert create(tp, tp.TPPagedAttention, "paged", PAGED, kw, rope, raw) == expect


def test_null_handles(tp):
    from tensor_transformer_mlp_shard_gb300.binding import VP, PagedDesc, RotaryDesc
    L, out = tp.lib(), VP()
    for name, desc in (("rotary", RotaryDesc()), ("paged", PagedDesc())):
        make = getattr(L, f"tp_{name}_create")
        assert make(None, ctypes.byref(out)) == 1 and make(ctypes.byref(desc), None) == 1
        getattr(L, f"tp_{name}_destroy")(None)
    assert L.tp_paged_workspace_bytes(None) == 0
    assert L.tp_paged_sync_status(None, None) == 1
    assert L.tp_rotary_fwd(None, None, None, None, None) == 1
    assert L.tp_paged_append(None, None, None, None, 1, None, 1, 1, None, None, None, None, None, None) == 1
    assert L.tp_paged_decode(None, None, None, None, 1, None, 1, 1, None, None, None, None, None, None, 0, None) == 1
    assert L.tp_status_str(6) == b"TP_ERR_INDEX"


def shards(n, at):
    from tensor_transformer_mlp_shard_gb300.binding import _pack
    return _pack[n](*[at + 0x1000 * i if at else 0 for i in range(n)])


@pytest.mark.parametrize("back", [False, True])
def test_rotary_pointers(tp, back):
    from tensor_transformer_mlp_shard_gb300.binding import _pack
    h = tp.TPRotary(**ROTARY)
    call = tp.lib().tp_rotary_bwd if back else tp.lib().tp_rotary_fwd
    x, y = (b"dY", b"dX") if back else (b"X", b"Y")
    err = tp.lib().tp_last_error
    assert call(h._h, None, None, shards(2, 0x20000), None) == 1 and x in err()
    assert call(h._h, shards(2, 0x10000), None, None, None) == 1 and y in err()
    assert call(h._h, shards(2, 0x10008), None, shards(2, 0x20000), None) == 1 and x in err()
    assert call(h._h, shards(2, 0x10000), None, shards(2, 0x20004), None) == 1 and y in err()
    assert call(h._h, shards(2, 0x10000), 0x30002, shards(2, 0x20000), None) == 1 and b"positions" in err()
    assert call(h._h, _pack[2](0x10000, 0x20000), None, _pack[2](0x10000, 0x30000), None) == 1 and b"in place" in err()


PAGED_KEYS = ("X", "positions", "sequences", "table", "k_amax", "v_amax", "Q", "K", "V", "O", "ws")


def paged_call(tp, h, which, at, n=4, rows=4, cols=5, nbytes=1 << 40):
    a = lambda k: shards(2, at[k])  # noqa: E731
    if which == "append":
        return tp.lib().tp_paged_append(h._h, a("X"), at["positions"], at["sequences"], n, at["table"], rows, cols,
                                        at["k_amax"], at["v_amax"], a("Q"), a("K"), a("V"), None)
    return tp.lib().tp_paged_decode(h._h, a("Q"), at["positions"], at["sequences"], n, at["table"], rows, cols,
                                    at["k_amax"], at["v_amax"], a("K"), a("V"), a("O"), at["ws"], nbytes, None)


@pytest.mark.parametrize("which", ["append", "decode"])
@pytest.mark.parametrize("how", ["null", "misaligned"])
def test_paged_pointers(tp, which, how):
    h = tp.TPPagedAttention(**PAGED, dtype="fp8")
    for key in PAGED_KEYS:
        if key in (("O", "ws") if which == "append" else ("X",)) or (key == "sequences" and how == "null"):
            continue
        at = {k: 0x100000 * (i + 1) for i, k in enumerate(PAGED_KEYS)}
        at[key] = 0 if how == "null" else at[key] + (2 if key in PAGED_KEYS[1:6] else 8)
        assert paged_call(tp, h, which, at) == 1
        assert ("workspace" if key == "ws" else key).encode() in tp.lib().tp_last_error(), key


@pytest.mark.parametrize("which", ["append", "decode"])
def test_paged_sizes(tp, which):
    h = tp.TPPagedAttention(**PAGED)
    at = {k: 0x100000 * (i + 1) for i, k in enumerate(PAGED_KEYS)}
    assert paged_call(tp, h, which, at, n=-1) == 2
    assert paged_call(tp, h, which, at, n=(1 << 20) + 1) == 2
    assert paged_call(tp, h, which, at, rows=0) == 2
    assert paged_call(tp, h, which, at, cols=0) == 2
    assert paged_call(tp, h, which, at, cols=(1 << 20) + 1) == 2
    assert paged_call(tp, h, which, dict(at, sequences=None), n=5) == 2  # more rows than the table has
    assert paged_call(tp, h, which, at, n=0) == 0                         # nothing to do
    if which == "decode":
        assert paged_call(tp, h, which, at, nbytes=h.workspace_bytes() - 1) == 1
        assert b"workspace" in tp.lib().tp_last_error()


def test_index_words(tp):
    """As many handles as there are index words, and their words come back."""
    live = [tp.TPPagedAttention(**PAGED) for _ in range(1024)]
    with pytest.raises(tp.TpError) as e:
        tp.TPPagedAttention(**PAGED)
    assert e.value.status == 3
    live.pop()
    live.append(tp.TPPagedAttention(**PAGED))
    live.clear()


def test_binding_refuses(tp):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="scale"):
        tp.TPPagedAttention(**PAGED, scale=0.0)
    with pytest.raises(KeyError):
        tp.TPRotary(**ROTARY, rope=tp.Rope(scaling="other"))
    h = tp.TPPagedAttention(**PAGED)
    x = torch.zeros(2, 4, 64)
    for positions, table in ((x, x), (torch.zeros(4, dtype=torch.int32), x), ([1], torch.zeros(1, 1, dtype=torch.int32))):
        with pytest.raises(ValueError):
            h._rows(positions, None, table, None, None, 0)
    from tensor_transformer_mlp_shard_gb300.binding import _shards
    with pytest.raises(ValueError, match="X"):
        _shards("X", x, 2, 256, torch.float32, 0)
    with pytest.raises(ValueError, match="X"):
        _shards("X", [x[0], x[1]], 2, 256, torch.float32, 0)
    with pytest.raises(ValueError, match="X"):
        _shards("X", None, 2, 256, torch.float32, 0)
