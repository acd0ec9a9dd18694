"""Decode over the 4-bit cache in float64 with the error bound of the kernel's present arithmetic,
roundings counted.  Half a step of fp32 is 2^-24 of the value, of bf16 2^-8."""
from __future__ import annotations

import numpy as np

BF16 = 2.0 ** -8
FP32 = 2.0 ** -24


def decode_rows(q, k, v, scale):
    """The G query rows of one kv head over its live keys: o, lse and the bounds on both.

    q [G, d], k / v [n, d] stored values.

    Scores.  An operand is code + 8, at most 15, and 8 sum(q) comes off, so the terms of a group
    add up to at most 23 s sum|q| (s its scale).  Two MMAs of 17 addends a group and one for the
    8 sum(q), each addend cut at 2^-24 of the sum (51), the groups' sums (4), sum(q) itself in
    fp32 (10) and in three bf16 pieces (1), scale, log2(e), their product and the score's (4):
    70, taken as 72, half steps of the sum of the terms.
    exp2 to 2^-22, its argument to half a step of it, sums and merges: 16 half steps of
    1 + |score - maximum|.

    Weights.  Two bf16 pieces: the low one is at most 2^-8 of p and is rounded to 2^-8 of itself.
    An accumulator is cut by at most one step for each 16 tokens, and 32 more in merges and
    rescalings.  o leaves in bf16.
    """
    d = q.shape[1]
    n = len(k)
    if n == 0:
        z = np.zeros(q.shape)
        return z, np.full(len(q), -np.inf), z, np.zeros(len(q))
    x = scale * (q @ k.T)                                             # [G, n]
    top = x.max(1, keepdims=True)
    p = np.exp(x - top)
    total = p.sum(1, keepdims=True)
    lse = (top + np.log(total))[:, 0]
    p /= total
    s = np.abs(k).reshape(n, d // 32, 32).max(-1) / 7
    size = scale * 23 * np.abs(q).reshape(len(q), d // 32, 32).sum(-1) @ s.T
    err = 72 * FP32 * size.max(1) + 16 * FP32 * (1 + np.abs(x - top).max(1))
    o, weight = p @ v, p @ np.abs(v)
    bound = BF16 * np.abs(o) + (2.0 ** -16 + 2 * err[:, None] + (n / 16 + 32) * 2 * FP32) * weight * (1 + 2 * BF16)
    return o, lse, bound, err + 4 * FP32 * np.abs(lse) + 4 * FP32
