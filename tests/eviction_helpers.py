"""Inputs and derived tolerances of the tests of decode over a shared prefix and of
cache eviction (see prompt_helpers for the roundings that they count)."""
from __future__ import annotations

import numpy as np

import oracle.eviction as oe
from prompt_helpers import BF16, FP32, f64

SCALE = 192.0 ** -0.5


def i32(a):
    import torch
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def word():
    return i32([0])


def bf16(rng, *shape, by=1.0):
    import torch
    return torch.from_numpy((rng.standard_normal(shape) * by).astype(np.float32)).cuda().to(torch.bfloat16)


def paged(rng, lens, page, first=0, spare=3):
    """A table over a shuffled pool (entries that nobody reads: -7), the shared blocks, the pool's size."""
    need = [max(0, -(-n // page) - first) for n in lens]
    blocks = first + sum(need) + spare
    order = rng.permutation(blocks).astype(np.int32)
    table = np.full((len(lens), max(1, first + max(need))), -7, np.int32)
    at = first
    for b, n in enumerate(need):
        table[b, first:first + n] = order[at:at + n]
        at += n
    return table, order[:first], blocks


def poisoned(cache, table, shared, lens, page):
    """NaN in every row that no request sees; shared blocks are seen up to the longest length."""
    import torch
    seen = torch.zeros(cache.shape[:2], dtype=torch.bool)
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            block = shared[i] if i < len(shared) else table[b][i]
            seen[int(block), :max(0, min(page, n - i * page))] = True
    cache[~seen.cuda()] = float("nan")
    return cache


def score_error(q, rows, scale):
    """Of a score before the softmax, per head: 576 products summed in fp32 (2^-23 of the sum of
    magnitudes a step), the scale's product and the exponential's argument (2^-22 of the score) and
    the exponential itself (2^-21)."""
    size = (np.abs(q) @ np.abs(rows).T).max(1) * scale
    return 576 * 2.0 ** -23 * size + 2.0 ** -21 + 2.0 ** -22 * size


def decode_tol(q, rows, scale, out, lse):
    """out: its own rounding, the weights' to bf16 and a partial result's to bf16 (both of the
    weighted sum of magnitudes), the scores' error once in each weight and once in their sum, and the
    sums over the tokens.  lse: the scores' error, the sum's and its own rounding."""
    if len(rows) == 0:
        return np.zeros_like(out), np.zeros_like(lse)
    d = score_error(q, rows, scale)
    mag = oe.decode(q, np.concatenate([np.abs(rows[:, :512]), rows[:, 512:]], 1), scale)[0]
    x = oe.scores(q, rows, scale)
    w = np.exp(x - lse[:, None])
    mag = w @ np.abs(rows[:, :512])
    n = len(rows)
    tol = BF16 * np.abs(out) + mag * (2 * BF16 + 2 * d + 2 * n * 2.0 ** -23)[:, None]
    return tol, d + n * 2.0 ** -23 + 4 * FP32 * np.abs(lse) + 2.0 ** -20


def mass_tol(q, rows, scale, lse, given, before, fp8):
    """The scores' error (with an E4M3 cache also what two E4M3 numbers leave of a dim of q, 2^-17 of
    its head's largest), the argument's subtraction (2^-22 of the score and of the lse), the sum over
    heads, and the sum with what was there.  A weight below 2^-126, the smallest normal fp32 number,
    becomes 0: 2^-126 a head."""
    size = (np.abs(q) @ np.abs(rows).T) * scale
    d = 576 * 2.0 ** -23 * size + 2.0 ** -20 + 2.0 ** -22 * (size + np.abs(lse)[:, None])
    if fp8:
        d = d + 2.0 ** -17 * np.abs(q).max(1)[:, None] * np.abs(rows).sum(1)[None] * scale
    w = np.exp(oe.scores(q, rows, scale) - lse[:, None])
    return (w * np.expm1(d)).sum(0) + len(q) * (2.0 ** -23 * given + 2.0 ** -126) + 2.0 ** -22 * np.abs(before)


def check_shared(c):
    """Every request of a case against its definition."""
    from prompt_helpers import assert_within
    cache, q, out, lse = f64(c["cache"]), f64(c["q"]), f64(c["out"]), f64(c["lse"])
    n_shared = int(c["shared_blocks"])
    for b, n in enumerate(c["lens"]):
        rows = oe.rows_of(cache, c["table"], b, n, c["shared"][:n_shared])
        ref, ref_lse = oe.decode(q[b], rows, SCALE)
        tol, ltol = decode_tol(q[b], rows, SCALE, ref, ref_lse)
        assert_within(out[b], ref, tol, f"out of request {b}")
        if n == 0:
            assert np.isneginf(lse[b]).all()
        else:
            assert_within(lse[b], ref_lse, ltol, f"lse of request {b}")


def shared_case(rng, heads, page, shared_blocks, lens, by=1.0, table_blocks=None):
    import torch
    table, shared, blocks = paged(rng, lens, page, shared_blocks)
    B = len(lens)
    c = dict(lens=lens, table=table, shared=shared, q=bf16(rng, B, heads, 576, by=by), cache=bf16(rng, blocks, page, 576),
             shared_table=i32(shared), shared_blocks=i32([shared_blocks]), block_table=i32(table), seq_lens=i32(lens),
             out=torch.full((B, heads, 512), 7.0, dtype=torch.bfloat16, device="cuda"),
             lse=torch.full((B, heads), 7.0, dtype=torch.float32, device="cuda"), status=word())
    poisoned(c["cache"], table, shared, lens, page)
    return c


def run_shared(mla, c, **kw):
    mla.mla_decode_shared(c["q"], c["cache"], c["shared_table"], c["shared_blocks"], c["block_table"], c["seq_lens"], SCALE, c["out"],
                          c["lse"], dev_status=c["status"], **kw)


def mass_case(rng, heads, page, lens, fp8=False, width=None, by=1.0):
    import torch
    table, _, blocks = paged(rng, lens, page)
    B, S = len(lens), width or max(max(lens), 1)
    c = dict(lens=lens, table=table, q=bf16(rng, B, heads, 576, by=by), cache=bf16(rng, blocks, page, 576), block_table=i32(table), fp8=fp8,
             seq_lens=i32(lens), kv_scale=0.037 if fp8 else 1.0, status=word(), mass=torch.full((B, S), 3.0, device="cuda"),
             previous=torch.from_numpy(rng.random((B, S)).astype(np.float32)).cuda())
    poisoned(c["cache"], table, [], lens, page)
    if fp8:
        c["cache"] = (c["cache"].float() / 0.037).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    lse = np.full((B, heads), -np.inf)
    for b, n in enumerate(lens):
        if n:
            lse[b] = oe.decode(f64(c["q"])[b], mass_rows(c, b), SCALE)[1]
    c["lse"] = torch.from_numpy(lse).float().cuda()
    return c


def mass_rows(c, b):
    import torch
    cache = c["cache"] if not c["fp8"] else c["cache"].view(torch.float8_e4m3fn).double()
    return oe.rows_of(f64(cache), c["table"], b, c["lens"][b]) * c["kv_scale"]


def run_mass(mla, c, **kw):
    if c["fp8"]:
        kw["kv_scale"] = c["kv_scale"]
    (mla.mla_attention_mass_fp8 if c["fp8"] else mla.mla_attention_mass)(
        c["q"], c["cache"], c["block_table"], c["seq_lens"], SCALE, c["lse"], c["mass"], dev_status=c["status"], **kw)


def check_mass(c, decay, before, behind=3.0):
    """before: what `previous` held, or None; behind: what stood behind each request's end."""
    from prompt_helpers import assert_within
    got = f64(c["mass"])
    for b, n in enumerate(c["lens"]):
        rows, q, lse = mass_rows(c, b), f64(c["q"])[b], f64(c["lse"])[b]
        old = np.zeros(n) if before is None else decay * before[b, :n]
        given = oe.mass(q, rows, SCALE, lse)
        assert_within(got[b, :n], old + given, mass_tol(q, rows, SCALE, lse, given, old, c["fp8"]), f"mass of request {b}")
        assert (got[b, n:] == (behind if np.isscalar(behind) else behind[b, n:])).all()
