"""Decode over a shared prefix, attention weights, the choice of tokens that stay
and their move, in numpy fp64: the oracle of mla_decode_shared,
mla_attention_mass, mla_evict_select and mla_cache_compact.

TEST INFRASTRUCTURE ONLY (same rule as the rest of ``oracle/``).  Everything
takes the values that the device's operands hold and follows the definitions in
include/mla.h one to one; nothing is rounded.
"""
from __future__ import annotations

import numpy as np

LORA = 512


def rows_of(cache, table, b, n, shared=()):
    """Rows 0 .. n-1 of request b of cache [NB, BS, 576]; its first blocks are `shared`."""
    page = cache.shape[1]
    t = np.arange(n)
    blocks = np.array([shared[i] if i < len(shared) else table[b][i] for i in range(-(-n // page))], np.int64)
    return cache[blocks[t // page], t % page]


def scores(q, rows, scale):
    """q [H, 576] on rows [n, 576]: [H, n]."""
    return (q @ rows.T) * scale


def decode(q, rows, scale):
    """One request: out [H, 512], lse [H]."""
    if len(rows) == 0:
        return np.zeros((len(q), LORA)), np.full(len(q), -np.inf)
    x = scores(q, rows, scale)
    top = x.max(1, keepdims=True)
    w = np.exp(x - top)
    total = w.sum(1, keepdims=True)
    return (w / total) @ rows[:, :LORA], (top + np.log(total))[:, 0]


def mass(q, rows, scale, lse):
    """One request: the weight that its heads give each row, summed over heads."""
    live = lse != -np.inf
    return np.exp(scores(q, rows, scale)[live] - lse[live][:, None]).sum(0)


def select(weights, n, budget, sink, recent):
    """The positions that stay of tokens 0 .. n-1, by going through them one at a time."""
    if n <= budget:
        return list(range(n))
    middle = list(range(sink, n - recent))
    value = lambda t: -np.inf if np.isnan(weights[t]) else float(weights[t])  # noqa: E731
    # NaN lowest, below -inf too; the earlier one first
    middle.sort(key=lambda t: (np.isnan(weights[t]), -value(t), t))
    return sorted(list(range(sink)) + middle[:budget - sink - recent] + list(range(n - recent, n)))


def compact(cache, table, keep, lens, weights=None):
    """cache [layers, NB, BS, ...] and weights [B, S] after the move, as copies; keep: a list of
    positions for each request."""
    page = cache.shape[2]
    out = cache.copy()
    new = None if weights is None else weights.copy()
    for b, kept in enumerate(keep):
        for j, t in enumerate(kept):
            out[:, table[b][j // page], j % page] = cache[:, table[b][t // page], t % page]
        if new is not None:
            new[b, :lens[b]] = 0
            new[b, :len(kept)] = weights[b][list(kept)]
    return out, new
