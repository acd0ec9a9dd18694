"""Plain 64-bit forms of the paged 4-bit KV cache operators (numpy, float64, host loops),
and the error bounds their tests use.

The bounds count roundings.  Half a step of bf16 is 2^-8 of the value, of fp32 2^-24.
"""
from __future__ import annotations

import numpy as np
import torch

BF16 = 2.0 ** -8
FP32 = 2.0 ** -24


def f64(t) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def bf16(x) -> torch.Tensor:
    return torch.as_tensor(np.asarray(x), dtype=torch.float64).to(torch.bfloat16)


# ------------------------------------------------------------------ page tables
def page_table(old, new, free, cursor, table, page, sink=0, window=0, n_slots=None):
    """Request by request: (table, slots, positions, cu, cursor)."""
    table = np.array(table, np.int64)
    slots, pos, cu = [], [], [0]
    for b, (o, n) in enumerate(zip(old, new)):
        last = -(-n // page)
        for j in range(-(-o // page), last):
            if window and j >= sink + window:
                table[b, j] = table[b, j - window]
            else:
                table[b, j] = free[cursor]
                cursor += 1
        for p in range(o, n):
            j = p // page
            live = not window or j < sink or j >= last - window
            slots.append(table[b, j] * page + p % page if live else -1)
            pos.append(p)
        cu.append(len(pos))
    rest = (n_slots if n_slots is not None else len(pos)) - len(pos)
    return table, np.array(slots + [-1] * rest), np.array(pos + [0] * rest), np.array(cu), cursor


# ------------------------------------------------------------------ quantisation
def quantise(x):
    """(codes, scales) of x [..., d], the scales with a last axis per group of 32."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    a = np.max(np.abs(g), -1)
    odd = ~(a <= 2.0 ** 120)
    small = a < 2.0 ** -100
    with np.errstate(all="ignore"):
        m, e = np.frexp(np.where(odd | small, 1.0, a) / 7)
        s = np.ldexp(np.floor(m * 32) / 32, e)
        n = np.round(np.where(odd[..., None], 0, g) / s[..., None])
    n = np.where((odd | small)[..., None], 0, n)
    return n, np.where(odd, np.nan, np.where(small, 0, s))


def values(x):
    n, s = quantise(x)
    with np.errstate(all="ignore"):
        return (n * s[..., None]).reshape(np.shape(x))


# ------------------------------------------------------------------ norm + rotation
def norm_rope(x, w, eps, pos, inv_freq, interleaved):
    """x [N, H, d] -> (y, bound): bound counts one bf16 rounding of y, and in fp32 the d-term
    sum of squares (half of d roundings after the root), about 8 roundings of the two products
    and 4 of the angle and its sine, each on |a| + |b|."""
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    h = len(inv_freq)
    ang = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    y, size = x.copy(), np.abs(x)
    i0 = np.arange(0, 2 * h, 2) if interleaved else np.arange(h)
    i1 = i0 + 1 if interleaved else i0 + h
    a, b = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = a * c - b * s, b * c + a * s
    size[..., i0] = size[..., i1] = np.abs(a) + np.abs(b)
    return y, BF16 * np.abs(y) + (d / 2 + 12) * FP32 * size


# ------------------------------------------------------------------ decode
def live_tokens(s, fa, sink=1, window=16, block=128):
    u = np.arange(s)
    if fa:
        return u
    nb = -(-s // block)
    return u[(u // block < sink) | (u // block >= nb - window)]


def decode_row(q, k, v, scale):
    """One query row over live keys: (o, lse, bound on o, bound on lse).

    q [d], k / v [n, d] stored values.  Scores: the kernel may sum a group's products with
    codes shifted by up to 24 (its operand stands for 16 + code), so a term is at most
    31 s |q| and a score has d / 4 + 8 fp32 roundings (the tensor core's may be cuts: whole
    steps, 2^-23) of their sum.  exp, the sums and the merge: 16 more roundings.  p enters the
    value product in bf16, o leaves in bf16."""
    d = q.shape[-1]
    if len(k) == 0:
        return np.zeros(d), -np.inf, np.zeros(d), 0.0
    x = scale * (k @ q)
    top = x.max()
    p = np.exp(x - top)
    lse = top + np.log(p.sum())
    p /= p.sum()
    s = np.abs(k).reshape(len(k), d // 32, 32).max(-1) / 7        # the scales
    size = (scale * 31 * s * np.abs(q).reshape(d // 32, 32).sum(-1)).sum(-1)
    err = ((d / 4 + 8) * 2 * FP32 * size).max() + 16 * FP32 * (1 + np.abs(x - top).max())
    o, weight = p @ v, p @ np.abs(v)
    bound = BF16 * np.abs(o) + (BF16 + 2 * err) * weight * (1 + 2 * BF16)
    return o, lse, bound, err + 4 * FP32 * abs(lse) + 4 * FP32
