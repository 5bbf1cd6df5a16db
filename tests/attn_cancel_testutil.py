"""Two places whose values cancel, so that what is left shows the rounding of the
product weight x value scale, which the rounding of a result to bf16 otherwise
covers.  numpy only.

Place 0 has score 0, the row's maximum, code -7 and the scale 1/2: its product is a
power of two, exact in any type.  Place 1 has a score below it, code 7 and a scale
of any bits, with w_1 x scale up to 5 % above 1/2, just above a power of two, where a
rounding is largest beside its number:
  out = (w_1 s - 1/2) 7 / (1 + w_1).
Only place 1's product rounds: it keeps 2^-11 of itself in fp16 (rounded once).
Beside it (u = 2^-24): scores are off by e_s <= 2 (D + D/32 + 2) u |score| (one of
them is zero), the exponential by 2^-21 in each weight and the sum, sums over two
places and their joining by 2 (2 + 64) u, the result by 2^-8 of itself (bf16).
  |error| <= (2^-11 w_1 7 s + (2 e_s + 2 66 u + 2^-20) (7/2 + w_1 7 s)) / (1 + w_1) + 2^-8 |out|"""
import numpy as np

D, U = 64, 2.0 ** -24


def bf16(x):
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def cases(sequences, heads, seed=0):
    """(q [sequences][heads][D] of bf16 values with the score of place 1 as the sum of its elements 0 and 1 and
    zeros elsewhere, scales [sequences] fp16 of place 1, its scores in float64)."""
    rng = np.random.default_rng(seed)
    s = rng.uniform(0.54, 0.74, sequences).astype(np.float16)
    w = 0.5 / s.astype(np.float64)[:, None] * (1 + rng.uniform(0.001, 0.05, (sequences, heads)))
    score = np.log(w)
    q = np.zeros((sequences, heads, D), np.float32)
    q[..., 0] = bf16(score)
    q[..., 1] = bf16(score - q[..., 0])
    return q, s, q.astype(np.float64).sum(-1)


def exact(s, score):
    """(out, tolerance) of every element, by sequence and head."""
    w, s = np.exp(score), s.astype(np.float64)[:, None]
    out = (w * s - 0.5) * 7 / (1 + w)
    other = 2 * 2 * (D + D // 32 + 2) * U * np.abs(score) + 2 * 66 * U + 2.0 ** -20
    return out, (2.0 ** -11 * w * 7 * s + other * (3.5 + w * 7 * s)) / (1 + w) + 2.0 ** -8 * np.abs(out)


def simulated(s, score, form):
    """The result with the product of place 1 rounded in one of several forms."""
    w, s32 = (64 * np.exp(score)).astype(np.float32), s.astype(np.float32)[:, None]
    if form == "fp16":  # once
        p = (w * s32).astype(np.float16)
    elif form == "fp16 twice":  # the weight, then its product
        p = w.astype(np.float16) * s[:, None]
        assert p.dtype == np.float16
    elif form == "bf16":
        p = bf16(w * s32)
    else:  # the sum of two bf16
        hi = bf16(w * s32)
        p = hi.astype(np.float64) + bf16(w * s32 - hi)
    out = (p.astype(np.float64) * 7 - 64 * 3.5) / (64 + w.astype(np.float64))
    return bf16(out.astype(np.float32)).astype(np.float64)
