"""Decode over a shared prefix and cache eviction on the GPU: operands that are not
finite, pieces of many tiles, and what rounding may cost.  (Tolerances:
eviction_helpers; a head with a log-sum-exp of -inf has no part in them.)"""
import numpy as np
import pytest

import oracle.eviction as oe
from eviction_helpers import (SCALE, bf16, check_mass, check_shared, i32, mass_case, mass_rows, mass_tol, paged, run_mass, run_shared,
                              shared_case, word)
from prompt_helpers import assert_within, f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def mla():
    import mla_latent_cache_decode_gb300 as mla
    torch.cuda.set_device(0)
    return mla


def weigh(mla, c, scale=SCALE, **kw):
    """The weights at this scale (a cache of E4M3 has its own)."""
    if c["fp8"]:
        mla.mla_attention_mass_fp8(c["q"], c["cache"], c["block_table"], c["seq_lens"], scale, c["lse"], c["mass"], kv_scale=c["kv_scale"], **kw)
    else:
        mla.mla_attention_mass(c["q"], c["cache"], c["block_table"], c["seq_lens"], scale, c["lse"], c["mass"], **kw)
    return f64(c["mass"])


def weights_of(c, b, heads):
    """Request b's weights from these heads alone, and their tolerance."""
    q, rows, lse = f64(c["q"])[b][heads], mass_rows(c, b), f64(c["lse"])[b][heads]
    given = oe.mass(q, rows, SCALE, lse)
    return given, mass_tol(q, rows, SCALE, lse, given, 0.0 * given, c["fp8"]) if len(q) else 0.0 * given


@pytest.mark.parametrize("heads", [16, 128])
def test_shared_and_mass_with_nothing_to_do_for_most(mla, heads):
    """One token, or none: all pairs of SMs but one set up their barriers, have no tiles and leave; three
    hundred calls in a row."""
    rng = np.random.default_rng(60)
    for lens in ([1], [0, 0]):
        c, d = shared_case(rng, heads, 16, 0, lens), mass_case(rng, heads, 16, lens, heads == 16)
        ws = mla.make_shared_workspace(len(lens), heads)
        run_shared(mla, c, workspace=ws)
        run_mass(mla, d)
        first = c["out"].clone(), c["lse"].clone(), d["mass"].clone()
        for _ in range(300):
            run_shared(mla, c, workspace=ws)
            run_mass(mla, d)
        assert int(c["status"]) == 0 and int(d["status"]) == 0
        assert all(torch.equal(a, b) for a, b in zip(first, (c["out"], c["lse"], d["mass"])))
        check_shared(c)
        check_mass(d, 0.0, None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("what", ["nan", "inf", "one nan", "one inf", "one -inf"])
def test_mass_heads_of_no_weight_hold_anything(mla, what, fp8):
    """A head whose lse is -inf gives nothing, whatever its query: a padding head's may never have been
    set.  Of a request that has only such heads not even a row of NaN counts."""
    c = mass_case(np.random.default_rng(61), 20, 32, [100, 64, 70], fp8)
    live = np.ones((3, 20), bool)
    live[0, 3] = live[1, ::2] = live[2] = False
    dead = torch.from_numpy(~live).cuda()
    c["lse"][dead] = -float("inf")
    queries = c["q"][dead]
    queries[:, 100 if what.startswith("one") else slice(None)] = float(what.split()[-1])
    c["q"][dead] = queries
    if fp8:
        c["cache"][int(c["table"][2][1]), 5] = 0x7F  # token 37 of request 2
    else:
        c["cache"][int(c["table"][2][1]), 5] = float("nan")
    got = weigh(mla, c, dev_status=c["status"])
    assert int(c["status"]) == 0
    for b in range(2):
        want, tol = weights_of(c, b, np.flatnonzero(live[b]))
        assert_within(got[b, :c["lens"][b]], want, tol, f"request {b}")
    assert (got[2, :70] == 0).all()
    before = f64(c["previous"])
    assert np.array_equal(weigh(mla, c, previous=c["previous"], decay=0.5)[2, :70], 0.5 * before[2, :70])


@pytest.mark.parametrize("scale", [SCALE, 0.1, 0.1352, 0.125, 1.0])  # scale * log2(e) rounds up in some, down in others
@pytest.mark.parametrize("row", [float("inf"), -float("inf")])
def test_mass_rows_that_score_plus_infinity(mla, row, scale):
    """One head of forty scores a token +inf, the others -inf: its weight is +inf by the definition, at
    any scale; the other tokens' are what they were."""
    c = mass_case(np.random.default_rng(62), 40, 32, [200, 100], False)
    sign = torch.full((40,), -1.0, device="cuda")
    sign[27] = 1.0
    c["q"][:, :, 3] = (c["q"][:, :, 3].abs() + 1) * (sign * np.sign(row)).to(torch.bfloat16)
    for b in range(2):
        c["lse"][b] = torch.from_numpy(oe.decode(f64(c["q"])[b], mass_rows(c, b), scale)[1]).float().cuda()
    clean = weigh(mla, c, scale)
    c["cache"][int(c["table"][0][2]), 7, 3] = row  # token 71
    got = weigh(mla, c, scale)
    assert got[0, 71] == np.inf
    assert np.array_equal(np.delete(got[0], 71), np.delete(clean[0], 71)) and np.array_equal(got[1], clean[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [3, 100, 200, 575])  # of each of the parts that a score is summed in
def test_mass_queries_that_are_not_finite(mla, dim, fp8):
    """An infinite dim of a query gives each token +inf, nothing or NaN, by the sign of its row there
    (E4M3 has no infinities: NaN); a NaN gives every token of its request NaN.  Other requests are
    not touched."""
    c = mass_case(np.random.default_rng(63), 16, 32, [200, 100, 90], fp8)
    clean = weigh(mla, c)
    zero = int(c["table"][2][1]), 9  # token 41 of request 2
    c["cache"][zero[0], zero[1], dim] = 0
    c["q"][2, 5, dim] = float("inf")
    got = weigh(mla, c)
    assert np.array_equal(got[:2], clean[:2])
    at = mass_rows(c, 2)[:, dim]
    assert at[41] == 0
    if fp8:
        assert np.isnan(got[2, :90]).all()
    else:
        assert (got[2, :90][at > 0] == np.inf).all() and np.isnan(got[2, :90][at == 0]).all()
        want, tol = weights_of(c, 2, [h for h in range(16) if h != 5])
        assert_within(got[2, :90][at < 0], want[at < 0], tol[at < 0])
    c["q"][2, 5, dim] = float("nan")
    got = weigh(mla, c)
    assert np.array_equal(got[:2], clean[:2]) and np.isnan(got[2, :90]).all()


@pytest.mark.parametrize("share", [0.0, 0.95])
def test_mass_waits_for_as_long_as_a_piece_takes(mla, share):
    """Every pair of SMs weighs 27 million tokens (more than 0.1 s), one of them 95% of its own before it
    comes to the next request's: no wait runs out while tiles go by.  All pages are one."""
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    # of two requests' tokens every pair gets 1 / pairs: the pair whose share ends the first has this part of its own there
    n = [1 << 30, int((1 << 30) * (pairs / (pairs // 2 + share) - 1)) // 256 * 256]
    rng = np.random.default_rng(64)
    cache, q = bf16(rng, 1, 256, 576), bf16(rng, 2, 1, 576)
    lse = torch.logsumexp((q.double() @ cache[0].double().T) * SCALE, -1).float()
    mass, status = torch.zeros(2, 1 << 30, device="cuda"), word()
    mla.mla_attention_mass(q, cache, torch.zeros(2, 1 << 22, dtype=torch.int32, device="cuda"), i32(n), SCALE, lse, mass, dev_status=status)
    assert int(status) == 0
    for b in range(2):
        rows, qb, lb = f64(cache)[0], f64(q)[b], f64(lse)[b]
        want = oe.mass(qb, rows, SCALE, lb)
        assert_within(f64(mass[b, :256]), want, mass_tol(qb, rows, SCALE, lb, want, 0.0, False))
        pages = mass[b, :n[b]].view(-1, 256)
        assert bool((pages == pages[0]).all())
        assert not mass[b, n[b]:].any()


def peaks_case(rng, heads, page, shared_blocks, lens, every=700, rise=11.0):
    """Scores that are nearly flat but for a token in every 700, four kinds of them in turn: a head of
    the same kind scores it 2^11 times as high.  A run of tiles that meets its first such token behind
    its first tile takes what it has so far to the new scale, and by then that is a good part of the
    result (some 2,800 tokens of 2^-11 a peak)."""
    table, shared, blocks = paged(rng, lens, page, shared_blocks)
    B = len(lens)
    q, cache = bf16(rng, B, heads, 576, by=0.2), bf16(rng, blocks, page, 576)
    kind = torch.arange(heads, device="cuda") % 4
    q[..., 512:] = 0
    q[:, torch.arange(heads, device="cuda"), 512 + kind] = 8.0
    cache[..., 512:] = 0
    for b, n in enumerate(lens):
        for i, t in enumerate(range(every // 2, n, every)):
            block = shared[t // page] if t < shared_blocks * page else table[b][t // page]
            cache[int(block), t % page, 512 + i % 4] = rise * np.log(2) / SCALE / 8
    return dict(lens=lens, table=table, shared=shared, q=q, cache=cache, shared_table=i32(shared), shared_blocks=i32([shared_blocks]),
                block_table=i32(table), seq_lens=i32(lens), out=torch.full((B, heads, 512), 7.0, dtype=torch.bfloat16, device="cuda"),
                lse=torch.full((B, heads), 7.0, dtype=torch.float32, device="cuda"), status=word())


@pytest.mark.parametrize("heads,page,shared,lens", [
    (16, 64, 0, [100001]),                                        # a request's own tokens, few heads
    (128, 128, 0, [90007, 3000]),                                 # ... a full set
    (16, 64, 700, [44800 + n for n in (1, 77, 600) * 5]),         # packed rows on the shared part, 15 requests
    (5, 16, 3000, [48000 + n for n in (1, 300) * 13]),            # ... on short pages, a block's second half of the rows empty
])
def test_shared_maxima_that_rise_within_a_piece(mla, heads, page, shared, lens):
    """Pieces of four tiles and more, most of which rescale what they have summed up."""
    c = peaks_case(np.random.default_rng(65), heads, page, shared, lens)
    run_shared(mla, c)
    assert int(c["status"]) == 0
    some = sorted({0, 1, len(lens) // 2, len(lens) - 1} & set(range(len(lens))))
    check_shared(dict(c, lens=[lens[b] for b in some], table=c["table"][some], **{k: c[k][some] for k in ("q", "out", "lse")}))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads", [3, 40, 100])
def test_mass_pieces_of_many_tiles(mla, heads, fp8):
    """Ten tiles and more on every pair of SMs: several rounds of the rings and of S's buffers in a piece."""
    c = mass_case(np.random.default_rng(66), heads, 64, [100001, 700, 5000], fp8)
    run_mass(mla, c, previous=c["previous"], decay=0.5)
    assert int(c["status"]) == 0
    check_mass(c, 0.5, f64(c["previous"]))


@pytest.mark.parametrize("heads,shared,lens", [(128, 0, [3000] * 6), (16, 32, [2048 + n for n in (100, 700, 300, 500, 600)])])
def test_shared_partial_results_cost_next_to_nothing(mla, heads, shared, lens):
    """out's error in units of what two roundings alone leave, the weights' to bf16 and out's own
    (0.0018 of its size here).  Partial results add at most 2^-12 of the largest of 64 dims, some 2^-10.5
    of a dim's size; by half steps evenly spread (1 / sqrt 3) and independent of the others' that is
    0.0004, 2% together.  In bf16 they would add as much as out's own rounding: 20% and more."""
    c = shared_case(np.random.default_rng(67), heads, 64, shared, lens)
    run_shared(mla, c)
    error = least = 0.0
    for b, n in enumerate(lens):
        rows = torch.from_numpy(oe.rows_of(f64(c["cache"]), c["table"], b, n, c["shared"])).cuda()
        x = (c["q"][b].double() @ rows.T) * SCALE
        w = (x - x.amax(1, keepdim=True)).exp()
        out, total = w @ rows[:, :512], w.sum(1, keepdim=True)
        rounded = ((w.to(torch.bfloat16).double() @ rows[:, :512]) / total).to(torch.bfloat16).double()
        out = out / total
        least += float(((rounded - out) ** 2).sum())
        error += float(((c["out"][b].double() - out) ** 2).sum())
    assert (error / least) ** 0.5 < 1.1
