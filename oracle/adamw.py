"""fp64 AdamW (numpy) and the 8-bit form of its states.

States in 8 bits: E4M3 codes of m and of r = sqrt(v), one scale (largest
magnitude / 448) for 256 consecutive elements, rounded to a neighbouring code
by 16 bits of a hash of (seed, step, tensor, block, element)."""
from __future__ import annotations

import numpy as np

QBLOCK = 256
_M1, _M2 = np.uint64(0x9E3779B9), np.uint64(0xB504F333)
_MASK = np.uint64(0xFFFFFFFF)


def mix(x):
    """32 bits to 32 well-spread bits (xor-shifts and odd multipliers)."""
    x = np.asarray(x, np.uint64) & _MASK
    x = ((x ^ (x >> np.uint64(16))) * _M1) & _MASK
    x = ((x ^ (x >> np.uint64(15))) * _M2) & _MASK
    return x ^ (x >> np.uint64(16))


def random_bits(seed, step, tensor, n, first_block=0):
    """The 32 bits of elements [256 first_block, 256 first_block + n) of a tensor."""
    with np.errstate(over="ignore"):
        at_step = mix(np.uint64(seed) + _M1 * np.uint64(step))
        of_tensor = mix(at_step ^ ((np.uint64(tensor) * _M2 + np.uint64(1)) & _MASK))
        e = np.arange(n, dtype=np.uint64)
        block = mix(of_tensor + np.uint64(first_block) + e // np.uint64(QBLOCK))
        return mix(block ^ ((e % np.uint64(QBLOCK)) * _M1 & _MASK))


def e4m3_values():
    """The values of the 256 E4M3 codes (no infinities; NaN at 0x7F and 0xFF)."""
    code = np.arange(256)
    exp, man = (code >> 3) & 15, code & 7
    v = np.where(exp == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (exp - 10.0))
    v[(code & 127) == 127] = np.nan
    return np.where(code & 128, -v, v)


def decode(codes, scales):
    """Values of a tensor's codes (bytes) and scales."""
    return e4m3_values()[np.asarray(codes)] * np.repeat(np.asarray(scales, np.float64), QBLOCK)[:len(codes)]


def block_scales(x):
    """Scale of every block of x (0 for a block below 2^-100)."""
    pad = np.zeros(-(-len(x) // QBLOCK) * QBLOCK)
    pad[:len(x)] = np.abs(x)
    top = pad.reshape(-1, QBLOCK).max(1)
    return np.where(top < 2.0 ** -100, 0.0, top / 448.0)


def positions(x, scales, bits):
    """(magnitude in units of the local E4M3 step, that step, its position plus
    the random fraction): the rounded magnitude is floor(position) * step."""
    s = np.repeat(scales, QBLOCK)[:len(x)]
    u = np.abs(x) / np.where(s > 0, s, 1.0) * (s > 0)
    step = 2.0 ** (np.floor(np.log2(np.maximum(u, 2.0 ** -6))) - 3)
    return u / step, step, u / step + np.asarray(bits, np.float64) / 65536.0


def update(w, g, m, v, t, lr, beta1, beta2, eps, weight_decay, scale=1.0):
    """One step: (w, m, v) after it, in fp64."""
    w, g, m, v = (np.asarray(a, np.float64) for a in (w, g, m, v))
    g = g * scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    w = w - lr * weight_decay * w - lr * (m / (1 - beta1 ** t)) / (np.sqrt(v / (1 - beta2 ** t)) + eps)
    return w, m, v
