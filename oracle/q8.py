"""Prompt attention and the 8-bit slot cache, in float64 numpy, one unit at a time.

The scales and codes follow float32 operations (each rounded to nearest), so they are
computed in float32 here too and must match bit for bit; everything else is float64.
"""
from __future__ import annotations

import numpy as np

TOP = {"s8": 127.0, "e4m3": 448.0}


def attn_prompt(q, k, v, scale):
    """One sequence and head: q [nq][d], k, v [nk][d] -> (o [nq][d], lse [nq], mass [nq][d]):
    mass = sum_j p_j |v_j|, what rounding errors of p are weighed with."""
    nq, nk = len(q), len(k)
    o = np.zeros((nq, v.shape[1]))
    mass = np.zeros_like(o)
    lse = np.full(nq, -np.inf)
    for i in range(nq):
        n = min(nk, i + nk - nq + 1)
        if n <= 0:
            continue
        x = scale * (k[:n] @ q[i])
        m = x.max()
        w = np.exp(x - m)
        lse[i] = m + np.log(w.sum())
        w /= w.sum()
        o[i] = w @ v[:n]
        mass[i] = w @ np.abs(v[:n])
    return o, lse, mass


def to_e4m3(y):
    """float32 values -> the nearest e4m3 values (ties to even, at most 448), as float64."""
    y = np.asarray(y, dtype=np.float64)
    a = np.abs(y)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -40)))
    step = 2.0 ** (np.maximum(e, -6) - 3)
    return np.copysign(np.minimum(np.round(a / step) * step, 448.0), y)


def quantise(x, fmt):
    """x [rows][d] float32 -> (code values [rows][d] float64, scale float32)."""
    x = np.asarray(x, dtype=np.float32)
    big = np.abs(x).max() if x.size else np.float32(0)
    scale = max(np.float32(big) / np.float32(TOP[fmt]), np.float32(2.0 ** -126))
    y = x * (np.float32(1) / np.float32(scale))
    return (np.clip(np.rint(y.astype(np.float64)), -127, 127) if fmt == "s8" else to_e4m3(y)), np.float32(scale)


def rows(codes, scales, tail, n, block):
    """The float64 rows that a unit's n slots stand for (codes as values)."""
    f = n // block * block
    out = np.asarray(codes[:f], dtype=np.float64) * np.repeat(np.asarray(scales[:f // block], np.float64), block)[:, None]
    return np.concatenate([out, np.asarray(tail[:n - f], dtype=np.float64)])


def decode(q, k, v, scale):
    """q [G][d] over rows k, v [n][d] -> (o [G][d], p [G][n], mass [G][d])."""
    x = scale * (q @ k.T)
    w = np.exp(x - x.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    return w @ v, w, w @ np.abs(v)


def evict(acc, pos, n, keep, recent, sink):
    """The slots that stay, ascending: the (acc, slot)-smallest unprotected ones go, one by one."""
    left = list(range(n))
    while len(left) > keep:
        free = [i for i in left if i < n - recent and pos[i] >= sink]
        left.remove(min(free, key=lambda i: (acc[i], i)))
    return np.array(left, dtype=np.int64)
