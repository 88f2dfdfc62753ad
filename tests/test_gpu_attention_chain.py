"""The operators as they are used together: the QKV column layer, the rotation on
the way into the paged cache, decode attention, the output row layer; and, in
training, the rotation between the QKV layer and what reads it, with its gradient."""
import numpy as np
import pytest
import torch

import oracle
from attention_cases import TORCH, cuda_i32, table_for
from harness import TOL, dev, rel_err
from oracle import attention as ref
from oracle.fp8 import round_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tp():
    import tensor_transformer_mlp_shard_gb300 as tp
    return tp


H, HEADS, KV, D, T = 256, 8, 4, 64, 2
WIDTH = (HEADS + 2 * KV) * D


def weights(rng, dtype):
    rnd = (lambda a: a) if dtype == "f32" else round_bf16
    wq = [rnd(rng.standard_normal((WIDTH // T, H)) * 0.08) for _ in range(T)]
    wo = [rnd(rng.standard_normal((H, HEADS // T * D)) * 0.05) for _ in range(T)]
    return wq, wo, rnd


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
def test_prompt_and_answers(tp, dtype):
    """A prompt of three sequences, then steps of one token each, every step one replay of a captured graph; a
    sequence ends on the way and its row becomes padding."""
    rng = np.random.default_rng(11)
    act = "f32" if dtype == "f32" else "bf16"
    wq, wo, rnd = weights(rng, act)
    prompt, steps, n = [37, 5, 64], 4, 3
    table, pages = table_for(rng, [k + steps for k in prompt], 16)
    h = tp.TPPagedAttention(HEADS, KV, D, 16, pages, T=T, dtype=dtype, grouped=True, rope=tp.Rope(dim=32))
    K = torch.zeros(T, *h.cache_shape, dtype=h.cache_dtype, device="cuda")
    V = torch.zeros_like(K)
    ws = tp.alloc_workspace(h.workspace_bytes())
    amax = {}
    if dtype == "fp8":
        amax = dict(k_amax=torch.full((KV,), 8.0, device="cuda"), v_amax=torch.full((KV,), 8.0, device="cuda"))
    wqd, wod = [dev(w, act) for w in wq], [dev(w, act) for w in wo]
    f, a = ref.rope_frequencies(32)
    total = [k + steps for k in prompt]
    x_all = [rnd(rng.standard_normal((k, H))) for k in total]

    def buffers(m):
        e = dict(dtype=TORCH[dtype], device="cuda")
        col = tp.Layout(m, 1, H, WIDTH, T, act="none", dtype=act)
        row = tp.Layout(m, 1, H, HEADS * D, T, act="none", dtype=act)
        return (col, row, torch.zeros(m, H, **e), torch.empty(T, m, WIDTH // T, **e), torch.empty(T, m, HEADS // T * D, **e),
                torch.empty(m, H, **e))

    def step(b, at, seq):
        col, row, x, qkv, q, y = b
        tp.linear_col(col, [x], wqd, None, list(qkv))
        h.append(qkv, at, tab, K, V, q, sequences=seq, **amax)
        h.decode(q, at, tab, K, V, q, ws, sequences=seq, **amax)   # over the queries
        tp.linear_row(row, list(q), wod, None, None, [y])

    tab = cuda_i32(table)
    got = [np.zeros((k, H)) for k in total]
    # the prompts, every token a row of its own
    first = buffers(sum(prompt))
    first[2].copy_(dev(np.concatenate([x[:k] for x, k in zip(x_all, prompt)]), act))
    step(first, cuda_i32(np.concatenate([np.arange(k) for k in prompt])), cuda_i32(np.repeat(np.arange(n), prompt)))
    y = first[5].double().cpu().numpy()
    for s, k in enumerate(prompt):
        got[s][:k] = y[sum(prompt[:s]):sum(prompt[:s]) + k]
    # the answers
    b = buffers(n)
    at, seq = cuda_i32([-1] * n), cuda_i32(np.arange(n))
    step(b, at, seq)                                                # warm up: padding alone
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(b, at, seq)
    for i in range(steps):
        live = [s for s in range(n) if not (s == 1 and i >= 2)]     # sequence 1 ends after two
        at.copy_(cuda_i32([prompt[s] + i if s in live else -1 for s in range(n)]))
        b[2].copy_(dev(np.stack([x_all[s][prompt[s] + i] for s in range(n)]), act))
        g.replay()
        y = b[5].double().cpu().numpy()
        for s in live:
            got[s][prompt[s] + i] = y[s]
    assert h.sync_status() == 0
    total[1] = prompt[1] + 2
    # the same in fp64, a sequence at a time
    want = []
    for s in range(n):
        x, m, out = x_all[s][:total[s]], total[s], np.zeros((total[s], H))
        own = np.arange(-(-m // 16))[None]
        for t in range(T):
            qkv = (x @ wq[t].T).reshape(m, -1, D)
            qc, kc, vc = ref.qkv_columns(HEADS // T, KV // T, True)
            q = ref.rotate(qkv[:, qc], np.arange(m), f, a)
            Kc, Vc = np.zeros((2, own.shape[1], KV // T, 16, D))
            for p in range(m):
                Kc[p // 16, :, p % 16] = ref.rotate(qkv[p:p + 1, kc], [p], f, a)[0]
                Vc[p // 16, :, p % 16] = qkv[p, vc]
            o = ref.decode(q, np.arange(m), np.zeros(m, int), own, Kc, Vc, D ** -0.5)[0]
            out += o.reshape(m, -1) @ wo[t].T
        want.append(out)
    got, want = np.concatenate([x[:k] for x, k in zip(got, total)]), np.concatenate(want)
    # the layers' own tolerances; E4M3 keys and values are off by 2^-4, which the sums over positions and heads
    # average: a half of it of the largest output
    assert rel_err(got, want) <= {"f32": TOL["f32"], "bf16": TOL["bf16"], "fp8": 2.0 ** -5}[dtype]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_training_layer(tp, dtype):
    """QKV layer and rotation, forward and backward, captured as one step."""
    rng = np.random.default_rng(12)
    S, B = 48, 2
    M = S * B
    wq, _, rnd = weights(rng, dtype)
    x, dy = rnd(rng.standard_normal((M, H))), rnd(rng.standard_normal((T, M, WIDTH // T)))
    col = tp.Layout(S, B, H, WIDTH, T, act="none", dtype=dtype)
    rot = tp.TPRotary(S, B, HEADS, KV, D, T=T, dtype=dtype, rope=tp.Rope(scaling="linear", factor=2.0))
    e = dict(dtype=TORCH[dtype], device="cuda")
    xd, wqd = dev(x, dtype), [dev(w, dtype) for w in wq]
    qkv, grad = torch.empty(T, M, WIDTH // T, **e), torch.empty(T, M, WIDTH // T, **e)
    upstream = torch.stack([dev(t, dtype) for t in dy])
    dx, dw = torch.empty(M, H, **e), [torch.empty(WIDTH // T, H, device="cuda") for _ in range(T)]
    ws = tp.alloc_workspace(tp.linear_workspace_bytes(col))

    def step():
        tp.linear_col(col, [xd], wqd, None, list(qkv))
        rot.fwd(qkv)
        rot.bwd(upstream, grad)
        tp.linear_col_bwd(col, list(grad), [xd], wqd, [dx], dw, None, ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for t in (qkv, grad, dx):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    f, a = ref.rope_frequencies(D, scaling="linear", factor=2.0)
    at = np.arange(M) // B
    want_dx = 0
    for t in range(T):
        y = ref.rotary(x @ wq[t].T, at, HEADS // T, KV // T, D, False, f, a)
        back = ref.rotary(dy[t], at, HEADS // T, KV // T, D, False, f, a, back=True)
        assert rel_err(qkv[t].double().cpu().numpy(), y) <= TOL[dtype]
        assert rel_err(grad[t].double().cpu().numpy(), back) <= TOL[dtype]
        assert rel_err(dw[t].double().cpu().numpy(), back.T @ x) <= TOL[dtype]
        want_dx = want_dx + back @ wq[t]
    assert rel_err(dx.double().cpu().numpy(), want_dx) <= TOL[dtype]
