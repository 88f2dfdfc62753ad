"""The block norm's kernels for wide rows, with everything a row can have.

Rows of 4104 to 8192 columns are a block's, 16 elements a thread in the backward
(whose weights are read at every row under two LayerNorms in bf16); wider ones
are a block's with 32 elements a thread in the forward and a cluster's of two or
four blocks in the backward, as are narrower rows whose staged arrays exceed an
SM's shared memory (fp32 from 6616 columns, 5192 with an element gate, an fp32
stream with an element gate from 7632), and in the forward fp32 rows from 13224
columns (8472 with an element gate) and those of an fp32 stream with an element
gate from 13224.  200 tokens give
every block or cluster several rows: both stages, both buffers of the
reductions, and column sums of more than one row.

Tolerances as in test_gpu_block_norm: a worker adds at most 8 rows, the
parameter gradients at most 200 partial rows in a tree of 4 + 16 + 4 additions.
"""
import numpy as np
import pytest
import torch

from oracle import block_norm as ob
from test_gpu_block_norm import EPS, U, Case, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tp():
    import tensor_transformer_mlp_shard_gb300 as tp
    from tensor_transformer_mlp_shard_gb300 import build
    build.build()
    return tp


BLOCK = [  # H, types, post, pre, gate, token shards, dY
    (4104, "bf16", "rms", "rms", "token", 1, True),
    (8192, "bf16", "rms", "rms", "element", 1, True),
    (8192, "bf16", "layer", "layer", "channel", 1, True),
    (5000, "bf16", "layer", "layer", "token", 1, True),
    (7992, "bf16", "layer", "layer", "element", 5, True),
    (8192, "bf16", "layer", "rms", "channel", 4, True),
    (6144, "bf16", "rms", "layer", "none", 8, False),
    (8192, "bf16", "layer", "layer", "channel", 1, False),
    (4104, "mixed", "layer", "layer", "token", 1, True),
    (8192, "mixed", "layer", "layer", "channel", 1, True),
    (8192, "mixed", "rms", "layer", "token", 4, True),
    (7624, "mixed", "layer", "rms", "element", 1, False),
    (8192, "mixed", "none", "layer", "channel", 1, False),
    (6608, "f32", "layer", "layer", "channel", 1, True),
    (5184, "f32", "layer", "layer", "element", 1, True),
    (4104, "f32", "rms", "layer", "token", 5, True),
    (6608, "f32", "layer", "rms", "token", 1, False),
]
CLUSTER = [
    (6616, "f32", "layer", "layer", "channel", 1, True),
    (5192, "f32", "layer", "layer", "element", 1, True),
    (8192, "f32", "rms", "rms", "token", 5, True),
    (7632, "mixed", "layer", "layer", "element", 1, True),
    (8200, "bf16", "rms", "rms", "channel", 1, True),
    (8200, "bf16", "layer", "layer", "token", 5, True),
    (12000, "bf16", "layer", "layer", "channel", 1, True),
    (16384, "bf16", "layer", "layer", "token", 1, True),
    (16384, "bf16", "rms", "layer", "element", 1, True),
    (16384, "bf16", "layer", "rms", "channel", 8, True),
    (16384, "bf16", "rms", "rms", "token", 1, False),
    (16384, "bf16", "layer", "none", "element", 1, True),
    (8200, "mixed", "rms", "layer", "token", 1, True),
    (16384, "mixed", "layer", "layer", "element", 4, True),
    (16384, "mixed", "layer", "layer", "channel", 1, False),
    (13224, "mixed", "layer", "rms", "element", 1, True),
    (8200, "f32", "layer", "layer", "element", 1, True),
    (8472, "f32", "rms", "rms", "element", 1, True),
    (13224, "f32", "rms", "layer", "channel", 1, True),
    (16384, "f32", "layer", "layer", "token", 4, True),
    (16384, "f32", "layer", "layer", "channel", 1, True),
    (16384, "f32", "none", "layer", "channel", 1, False),
    (16376, "f32", "layer", "rms", "none", 1, True),
]


@pytest.mark.parametrize("H,types,post,pre,gate,T,dy", BLOCK + CLUSTER)
def test_wide_rows(tp, H, types, post, pre, gate, T, dy):
    c = Case(200, H, "f32" if types == "f32" else "bf16", post, pre, gate, res32=types == "mixed", zc=T > 1, T=T,
             a=0.75, c=1.5, seed=H)
    h = c.handle(tp)
    c.run_fwd(h)
    c.check_fwd()
    c.run_bwd(h, tp, dy=dy)
    c.check_bwd()


@pytest.mark.parametrize("H,dtype,gate", [(8192, "f32", "token"), (16384, "bf16", "element"), (16384, "f32", "channel")])
def test_wide_rows_in_place(tp, H, dtype, gate):
    """Y may be X and dX may be dY; the results are those of separate buffers."""
    a, b = (Case(170, H, dtype, "layer", "layer", gate) for _ in range(2))
    h = a.handle(tp)
    a.run_fwd(h)
    b.run_fwd(h, y=b.x)
    assert torch.equal(a.y, b.x) and torch.equal(a.n, b.n) and torch.equal(a.stats, b.stats)
    a.run_bwd(h, tp)
    b.run_bwd(h, tp, inplace=True)
    assert torch.equal(a.out["dx"], b.dy)
    assert all(torch.equal(a.out[k], b.out[k]) for k in a.out if k != "dx")


def test_parameter_gradients_beyond_32_bits(tp):
    """More than 2^31 elements: the parameter gradients are the sums over all
    tokens.  All but three are alike, so the sums are known.  A cluster of two
    blocks adds 131149 / 76 rows in turn and the partial rows add 76 / 64 + 24
    more: 1752 u of the sum of magnitudes, and 16 u for each term."""
    H, M = 16384, 131072 + 77
    act = torch.bfloat16
    small = Case(4, H, "bf16", "rms", "rms")
    for t, v in ((small.x, 0.5), (small.f, 1.0), (small.dy, 0.5), (small.dn, 1.0)):
        t[0] = v  # the row that all others are
    hs = small.handle(tp)
    small.run_fwd(hs)
    small.run_bwd(hs, tp)
    small.check_bwd()

    def whole(t):
        out = torch.empty(M, *t.shape[1:], dtype=t.dtype, device="cuda")
        out[:] = t[0]
        out[-3:] = t[1:]
        return out

    dy, dn, y, f, stats = (whole(t) for t in (small.dy, small.dn, small.y, small.f, small.stats))
    h = tp.TPBlockNorm(M, 1, H, post="rms", pre="rms", eps=EPS)
    dw = [torch.empty(H, device="cuda") for _ in range(2)]
    df = torch.empty(M, H, dtype=act, device="cuda")
    h.bwd(dy, dn, y, f, None, small.pw, None, small.nw, stats, dy, df, None, dw[0], None, dw[1], None,
          workspace=tp.alloc_workspace(h.workspace_bytes()))
    assert torch.equal(dy[-3:], small.out["dx"][1:]) and torch.equal(df[-3:], small.out["df"][1:])
    for key, got in (("dpost_w", dw[0]), ("dpre_w", dw[1])):
        ref, size = np.zeros(H), np.zeros(H)
        for i in range(4):  # a row's own gradients, and how often the row is there
            row = lambda t: f64(t[i:i + 1])  # noqa: E731
            g = ob.grads(row(small.dy), row(small.dn), row(small.y), row(small.f), None, "none", "rms", f64(small.pw),
                         None, "rms", f64(small.nw), 1.0, 1.0, EPS)[key]
            ref += g * (M - 3 if i == 0 else 1)
            # D is a difference of terms as large as those of the oracle's bound on dx
            size += (np.abs(g) + np.abs(row(small.dy)[0]) + 3 * np.abs(f64(small.nw)) * np.abs(row(small.dn)[0])) \
                * (M - 3 if i == 0 else 1)
        assert (np.abs(f64(got) - ref) <= (1752 + 16) * U * size).all(), key
