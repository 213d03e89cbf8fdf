"""The prompt side in numpy fp64: the oracle of mla_rope_append, mla_expand_kv
and mla_prefill.

TEST INFRASTRUCTURE ONLY (same rule as the rest of ``oracle/``).  Everything
takes fp64 arrays of the values that the device's operands hold and follows the
definitions in include/mla.h one to one; nothing is rounded.
"""
from __future__ import annotations

import numpy as np

LORA, ROPE = 512, 64


def rotate(x, cos, sin, interleaved):
    """x [..., 64] with each of its 32 pairs (a, b) replaced by
    (a cos - b sin, b cos + a sin); cos, sin [..., 32] broadcast against it."""
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    out = np.empty(np.broadcast_shapes(x.shape, a.shape[:-1] + (ROPE,)), np.float64)
    ra, rb = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        out[..., 0::2], out[..., 1::2] = ra, rb
    else:
        out[..., :32], out[..., 32:] = ra, rb
    return out


def rope_rows(kv, cos_sin, positions, norm_weight, eps, interleaved):
    """The rows that mla_rope_append stores, before their one rounding."""
    row = cos_sin[positions]
    latent = kv[:, :LORA]
    if norm_weight is not None:
        latent = norm_weight * latent / np.sqrt((latent ** 2).mean(1, keepdims=True) + eps)
    return np.concatenate([latent, rotate(kv[:, LORA:], row[:, :32], row[:, 32:], interleaved)], 1)


def expand(rows, w_uk, w_uv):
    """k_nope [T, H, 128] and v [T, H, 128] of latent rows [T, 576]."""
    c = rows[:, :LORA]
    k = np.stack([c @ w.T for w in w_uk], 1)
    v = np.stack([c @ w for w in w_uv], 1)
    return k, v


def attend(q_nope, q_pe, k_nope, k_pe, v, softmax_scale, causal):
    """One request: queries [nq, H, .] over keys [nk, H, .].  Returns out
    [nq, H, 128], lse [nq, H], and two per-row magnitudes for error bounds:
    sum_j p_j |v_j| and max_j scale * sum_d |q_d k_jd| over the visible keys."""
    nq, H = q_nope.shape[:2]
    nk = k_nope.shape[0]
    out, mag = np.zeros((nq, H, 128)), np.zeros((nq, H, 128))
    lse, size = np.full((nq, H), -np.inf), np.zeros((nq, H))
    seen = np.ones((nq, nk), bool)
    if causal:
        seen = np.arange(nk)[None] <= np.arange(nq)[:, None] + (nk - nq)
    rows = seen.any(1)
    for h in range(H):
        if not rows.any():
            break
        q = np.concatenate([q_nope[rows, h], q_pe[rows, h]], 1)
        k = np.concatenate([k_nope[:, h], k_pe], 1)
        s = np.where(seen[rows], softmax_scale * (q @ k.T), -np.inf)
        top = s.max(1, keepdims=True)
        p = np.exp(s - top)
        total = p.sum(1, keepdims=True)
        out[rows, h] = p / total @ v[:, h]
        mag[rows, h] = p / total @ np.abs(v[:, h])
        lse[rows, h] = (top + np.log(total))[:, 0]
        size[rows, h] = (np.where(seen[rows], softmax_scale * (np.abs(q) @ np.abs(k).T), 0)).max(1)
    return out, lse, mag, size
