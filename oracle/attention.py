"""fp64 numpy oracle of the operators around the attention projections: rotary
positions, the paged key-value cache, decode attention.  Test infrastructure
only, written from the definitions in include/tp_mlp.h."""
from __future__ import annotations

import math

import numpy as np


def rope_frequencies(dim, base=10000.0, scaling="none", factor=1.0, original=0, fast=32.0, slow=1.0,
                     attention_factor=None):
    """(radians a position of each pair, attention factor)."""
    if scaling == "ntk" and dim > 2:
        base = base * factor ** (dim / (dim - 2))
    f = np.array([base ** (-2.0 * i / dim) for i in range(dim // 2)], dtype=np.float64)
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        keep = np.clip((original * f / (2 * math.pi) - slow) / (fast - slow), 0.0, 1.0)
        f = keep * f + (1.0 - keep) * f / factor
    if attention_factor is None:
        attention_factor = 0.1 * math.log(factor) + 1.0 if scaling == "parts" else 1.0
    return f, attention_factor


def rotate(x, positions, f, a, interleaved=False, back=False):
    """x [n, heads, D], token j at positions[j] (negative: as it is)."""
    x = np.asarray(x, np.float64)
    out = x.copy()
    half = len(f)
    for j, p in enumerate(positions):
        if p < 0:
            continue
        c, s = a * np.cos(int(p) * f), a * np.sin(int(p) * f)
        if back:
            s = -s
        i1 = np.arange(half) * 2 if interleaved else np.arange(half)
        i2 = i1 + 1 if interleaved else i1 + half
        x1, x2 = x[j][:, i1], x[j][:, i2]
        out[j][:, i1] = x1 * c - x2 * s
        out[j][:, i2] = x2 * c + x1 * s
    return out


def qkv_columns(hq, hk, grouped):
    """The heads (of head_dim columns) of a shard's queries, keys and values."""
    per = hq // hk
    if not grouped:
        return list(range(hq)), list(range(hq, hq + hk)), list(range(hq + hk, hq + 2 * hk))
    start = [j * (per + 2) for j in range(hk)]
    return [s + i for s in start for i in range(per)], [s + per for s in start], [s + per + 1 for s in start]


def rotary(x, positions, hq, hk, D, grouped, f, a, interleaved=False, back=False):
    """One shard's QKV rows [n, (hq + 2 hk) D] with queries and keys rotated."""
    y = np.asarray(x, np.float64).reshape(len(positions), hq + 2 * hk, D).copy()
    q, k, _ = qkv_columns(hq, hk, grouped)
    y[:, q + k] = rotate(y[:, q + k], positions, f, a, interleaved, back)
    return y.reshape(len(positions), -1)


def slots(positions, sequences, table, page_size, pages):
    """(page, place in it) of every row, None for padding and indices out of range."""
    out = []
    for p, s in zip(positions, sequences):
        ok = p >= 0 and 0 <= s < table.shape[0] and p // page_size < table.shape[1]
        page = int(table[s, p // page_size]) if ok else -1
        out.append((page, int(p) % page_size) if 0 <= page < pages else None)
    return out


def decode(q, positions, sequences, table, K, V, scale, window=0):
    """q [n, hq, D] over one shard's caches [pages, hk, page_size, D] -> (o, sum_j w_j |v_j|,
    largest scale * sum |q k| of a row, positions that a row sees)."""
    n, hq, D = q.shape
    pages, hk, page_size, _ = K.shape
    o, mag = np.zeros((n, hq, D)), np.zeros((n, hq, D))
    spread, seen = np.zeros((n, hq)), np.zeros(n, dtype=np.int64)
    for r, (p, s) in enumerate(zip(positions, sequences)):
        if p < 0 or not 0 <= s < table.shape[0] or p // page_size >= table.shape[1]:
            continue
        at = np.arange(max(0, p - window + 1) if window else 0, p + 1)
        page = table[s, at // page_size].astype(np.int64)
        good = (page >= 0) & (page < pages)
        at, page = at[good], page[good]
        seen[r] = len(at)
        if not len(at):
            continue
        for h in range(hq):
            k = K[page, h // (hq // hk), at % page_size].astype(np.float64)
            v = V[page, h // (hq // hk), at % page_size].astype(np.float64)
            with np.errstate(invalid="ignore", over="ignore"):
                x = scale * (k @ q[r, h].astype(np.float64))
                spread[r, h] = abs(scale) * np.max(np.abs(k) @ np.abs(q[r, h].astype(np.float64)))
                top = x.max()
                if top == -np.inf:
                    continue
                w = np.exp(x - top)
                w /= w.sum()
                o[r, h], mag[r, h] = w @ v, w @ np.abs(v)
    return o, mag, spread, seen
