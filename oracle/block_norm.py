"""fp64 block norm (numpy): the residual stream between one block and the next,
and its gradients, from the definitions.

    p = P(f),  y = a x + c g p,  n = N(y)

norms: "none", "rms" (x / sqrt(mean x^2 + eps) * w) or "layer" ((x - mean) /
sqrt(var + eps) * w + b).  gate: None, [H], [M] or [M, H]."""
from __future__ import annotations

import numpy as np


def norm_stats(x, kind, eps):
    """(mean, 1 / spread) of every row, as [M, 1]."""
    x = np.asarray(x, np.float64)
    if kind == "none":
        return np.zeros((len(x), 1)), np.ones((len(x), 1))
    mean = x.mean(1, keepdims=True) if kind == "layer" else np.zeros((len(x), 1))
    return mean, 1.0 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)


def norm(x, kind, w, b, eps, zero_centered=False):
    x = np.asarray(x, np.float64)
    if kind == "none":
        return x
    mean, rstd = norm_stats(x, kind, eps)
    out = (x - mean) * rstd * (np.asarray(w, np.float64) + (1.0 if zero_centered else 0.0))
    return out + np.asarray(b, np.float64) if kind == "layer" else out


def _gate(g):
    return 1.0 if g is None else np.asarray(g, np.float64)


def added(f, post, post_w, post_b, gate, token, c, eps, zero_centered=False):
    """c g P(f): what the block adds to the stream."""
    g = _gate(gate)
    return c * (g[:, None] if token else g) * norm(f, post, post_w, post_b, eps, zero_centered)


def norm_grad(d, x, kind, w, eps, zero_centered=False):
    """Gradients of norm(x) given that of its output: (dx, dw, db)."""
    d, x = np.asarray(d, np.float64), np.asarray(x, np.float64)
    if kind == "none":
        return d, None, None
    mean, rstd = norm_stats(x, kind, eps)
    hat = (x - mean) * rstd
    h = d * (np.asarray(w, np.float64) + (1.0 if zero_centered else 0.0))
    dx = h - hat * (h * hat).mean(1, keepdims=True)
    if kind == "layer":
        dx = dx - h.mean(1, keepdims=True)
    return rstd * dx, (d * hat).sum(0), d.sum(0)


def grads(dy, dn, y, f, gate, kind_of_gate, post, post_w, post_b, pre, pre_w, a, c, eps, zero_centered=False):
    """All gradients, as a dict (None where there is nothing)."""
    D = np.zeros_like(np.asarray(y, np.float64)) if dy is None else np.asarray(dy, np.float64)
    out = dict.fromkeys(("dx", "df", "dgate", "dpost_w", "dpost_b", "dpre_w", "dpre_b"))
    if pre != "none":
        up, out["dpre_w"], db = norm_grad(dn, y, pre, pre_w, eps, zero_centered)
        out["dpre_b"] = db if pre == "layer" else None
        D = D + up
    out["dx"] = a * D
    if f is None:
        return out
    g = _gate(gate)
    if kind_of_gate != "none":
        dg = c * D * norm(f, post, post_w, post_b, eps, zero_centered)
        out["dgate"] = dg.sum(0) if kind_of_gate == "channel" else dg.sum(1) if kind_of_gate == "token" else dg
    dp = c * D * (g[:, None] if kind_of_gate == "token" else g)
    out["df"], dw, db = norm_grad(dp, f, post, post_w, eps, zero_centered)
    if post != "none":
        out["dpost_w"], out["dpost_b"] = dw, db if post == "layer" else None
    return out
