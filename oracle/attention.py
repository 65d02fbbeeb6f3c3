"""Plain fp64 statement of the rotary positions, the paged key/value cache and
the attention over it (the calls around the weight products of a decode step).

The cache is held here as a user thinks of it: one array of tokens per page,
[pages][page_size][heads][dim]; `cache_memory` lays it out as the GPU library
keeps it.
"""
from __future__ import annotations

import functools
import math

import numpy as np

from .rfp2 import dequantize_acts, quantize_acts


def rope_freqs(rot, base, factor=1.0, orig_len=0.0, low_turns=0.0, high_turns=1.0):
    """Angle per position of pair i, one pair at a time."""
    out = []
    for i in range(rot // 2):
        f = math.pow(base, -2.0 * i / rot)
        keep = 0.0
        if orig_len > 0:
            turns = orig_len * f / (2.0 * math.pi)
            keep = min(max((turns - low_turns) / (high_turns - low_turns), 0.0), 1.0)
        out.append((1.0 - keep) * f / factor + keep * f)
    return np.array(out)


def rope(x, pos, freqs, rot, interleaved, mscale=1.0):
    """x [T][H][D] -> fp64 rotated values (not rounded)."""
    y = np.asarray(x, dtype=np.float64).copy()
    a = np.asarray(pos, dtype=np.float64)[:, None] * np.asarray(freqs)[None, :]
    c, s = np.cos(a)[:, None, :], np.sin(a)[:, None, :]
    h = rot // 2
    i1, i2 = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, h), slice(h, rot))
    x1, x2 = y[..., i1].copy(), y[..., i2].copy()
    y[..., i1] = mscale * (x1 * c - x2 * s)
    y[..., i2] = mscale * (x2 * c + x1 * s)
    return y


def quantize_heads(x):
    """x [T][H][D] fp32 -> (codes int8 of the same shape, scales [T][H][D/32])."""
    T, H, D = x.shape
    q, d = quantize_acts(np.ascontiguousarray(x, dtype=np.float32).reshape(T * H, D))
    return q.reshape(T, H, D), d.reshape(T, H, D // 32)


def held(x, i8):
    """The values the cache stands for once fp32 x [T][H][D] has been written."""
    if not i8:
        return np.asarray(x, dtype=np.float32).astype(np.float16).astype(np.float64)
    q, d = quantize_heads(x)
    T, H, D = q.shape
    return np.asarray(dequantize_acts(q.reshape(T * H, D), d.reshape(T * H, D // 32)),
                      dtype=np.float64).reshape(T, H, D)


def keys_in_memory(x):
    """[pages][page_size][heads][n] -> [pages][heads][page_size][n]."""
    return np.ascontiguousarray(np.swapaxes(x, 1, 2))


def eights_in_memory(x):
    """[pages][page_size][heads][n] -> [pages][heads][page_size/8][n][8] (values, scales)."""
    G, P, H, n = x.shape
    out = np.empty((G, H, P // 8, n, 8), dtype=x.dtype)
    for r in range(P):
        out[:, :, r // 8, :, r % 8] = x[:, r]
    return out


def attention(q, k, v, pos, scale, window=0):
    """One query q [H][D] at position pos over tokens k, v [n][Hkv][D] at positions
    0 .. n-1: (y [H][D], sum_j w_j |v_j| / sum_j w_j, largest scale * sum |q k|)."""
    H, D = q.shape
    hkv = k.shape[1]
    y, mag, big = np.zeros((H, D)), np.zeros((H, D)), np.zeros(H)
    lo = max(0, pos - window + 1) if window else 0
    hi = min(pos + 1, k.shape[0])
    if hi <= lo:
        return y, mag, big
    q = np.asarray(q, dtype=np.float64)
    for h in range(H):
        kk, vv = k[lo:hi, h // (H // hkv)], v[lo:hi, h // (H // hkv)]
        s = scale * (kk @ q[h])
        w = np.exp(s - s.max())
        y[h] = w @ vv / w.sum()
        mag[h] = w @ np.abs(vv) / w.sum()
        big[h] = abs(scale) * (np.abs(kk) @ np.abs(q[h])).max()
    return y, mag, big


@functools.lru_cache
def _pi_in_bits(bits):
    """pi * 2^bits, by Machin's formula in whole numbers."""
    one = 1 << (bits + 32)

    def arctan_of_one_over(x):
        term, total, n = one // x, 0, 1
        while term:
            total += term // n if n % 4 == 1 else -(term // n)
            term //= x * x
            n += 2
        return total
    return 4 * (4 * arctan_of_one_over(5) - arctan_of_one_over(239)) >> 32


def turn_fraction(pos, f):
    """pos * f radians as a fraction of a turn in [-1/2, 1/2], rounded once: the product
    and its division by 2 pi are whole-number arithmetic, however far the position."""
    num, den = float(f).as_integer_ratio()
    bits = 256
    turns = (int(pos) * num << (2 * bits)) // (den * 2 * _pi_in_bits(bits))   # * 2^bits
    rest = turns & ((1 << bits) - 1)
    if rest >> (bits - 1):
        rest -= 1 << bits
    return rest / (1 << bits)


def rope_far(x, pos, freqs, rot, interleaved, mscale=1.0):
    """`rope` with the angles of `turn_fraction`: for positions where the product
    pos * f no longer fits 53 bits well enough."""
    a = np.array([[2.0 * math.pi * turn_fraction(p, f) for f in freqs] for p in pos])
    return np.concatenate([rope(x[t:t + 1], [1], a[t], rot, interleaved, mscale)
                           for t in range(len(a))])
