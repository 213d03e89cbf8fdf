"""Inputs and derived tolerances of the prompt-side GPU tests.

A rounding to a type is off by at most half a step, relative to the value:
bf16 2^-8, fp32 2^-24, E4M3 2^-4 (2^-10 absolute below 2^-6).  fp32 sums of n
terms are off by at most n 2^-23 of the sum of magnitudes (2^-23 a step also
where the tensor cores cut instead of rounding).
"""
from __future__ import annotations

import numpy as np

BF16, FP32, E4M3 = 2.0 ** -8, 2.0 ** -24, 2.0 ** -4


def f64(t):
    return t.detach().double().cpu().numpy()


def assert_within(got, ref, tol, what=""):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= tol)
    if bad.any():
        i = tuple(int(x) for x in np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} values out of tolerance, first at {i}: "
                             f"got {got[i]!r}, want {ref[i]!r} +- {np.broadcast_to(tol, ref.shape)[i]!r}")


def rope_tol(kv, rows, cos_sin, positions, norm):
    """Of the stored row before its last rounding.  Latent: 16 squares a lane
    and five shuffles, a mean, a square root, a reciprocal and two products
    (fp32, each 2^-24, a root halving what went before) stay below 32 2^-24 of
    the value.  Rotation: two products and a sum, 3 2^-24 of |a cos| + |b sin|."""
    tol = np.zeros_like(rows)
    if norm:
        tol[:, :512] = 32 * FP32 * np.abs(rows[:, :512])
    tol[:, 512:] = 3 * FP32 * pair_size(kv[:, 512:])
    return tol


def pair_size(x):
    """An upper bound of |a| + |b| for the pair of every element."""
    top = np.abs(x).max(-1, keepdims=True)
    return np.broadcast_to(2 * top, x.shape)


def expand_tol(rows, w_uk, w_uv, k, v):
    """512 products summed in fp32, one rounding to bf16."""
    ck = np.stack([np.abs(rows[:, :512]) @ np.abs(w).T for w in w_uk], 1)
    cv = np.stack([np.abs(rows[:, :512]) @ np.abs(w) for w in w_uv], 1)
    return BF16 * np.abs(k) + 512 * 2 ** -23 * ck, BF16 * np.abs(v) + 512 * 2 ** -23 * cv


def attend_tol(out, lse, mag, size, nk):
    """out: its own rounding; the weights' rounding to bf16 (2^-8 of sum p|v|);
    the scores' fp32 error d = 192 2^-23 sum|q k| (192 products) plus the
    exponential's and its argument's (2^-21 and 2^-22 of the score), once in
    each weight and once in their sum; nk products summed in fp32.
    lse: d, the sum of nk weights, and its own rounding."""
    d = 192 * 2 ** -23 * size + 2.0 ** -21 + 2.0 ** -22 * size
    tol = BF16 * np.abs(out) + mag * (BF16 + (2 * d + 2 * nk * 2.0 ** -23)[..., None])
    with np.errstate(invalid="ignore"):
        lse_tol = np.where(np.isinf(lse), 0.0, d + nk * 2.0 ** -23 + 4 * FP32 * np.abs(lse) + 2.0 ** -20)
    return tol, lse_tol
