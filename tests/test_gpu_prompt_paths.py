"""The prompt side's kernels on the paths that only long contexts and many
items take: mla_prefill's straight-line softmax with claimed items, pairs of
heads and tiles that are not full, and mla_expand_kv over many changes of rows.
Against the fp64 oracle, with the derived tolerances of prompt_helpers."""
import numpy as np
import pytest

import oracle.prompt as op
from prompt_helpers import assert_within, attend_tol, f64
from test_gpu_prompt import bits, check_expand, expand_case, mla, prefill_case, run_expand, run_prefill, word  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def check_heads(c, heads, causal, scale=0.07):
    """check_prefill on some heads: every row of out and lse of each request."""
    qn, qp, kn, v = (f64(c[n][:, heads]) for n in ("qn", "qp", "kn", "v"))
    kp = f64(c["kp"])
    got, got_lse = f64(c["out"][:, heads]), f64(c["lse"][:, heads])
    q0 = k0 = 0
    for nq, nk in zip(c["q_lens"], c["kv_lens"]):
        q, k = slice(q0, q0 + nq), slice(k0, k0 + nk)
        out, lse, mag, size = op.attend(qn[q], qp[q], kn[k], kp[k], v[k], float(np.float32(scale)), causal)
        tol, lse_tol = attend_tol(out, lse, mag, size, nk)
        empty = np.isneginf(lse)
        assert_within(got[q], out, tol, f"out of {nq} queries on {nk} keys")
        assert np.array_equal(np.isneginf(got_lse[q]), empty) and (got[q][empty] == 0).all()
        assert_within(np.where(empty, 0, got_lse[q]), np.where(empty, 0, lse), lse_tol, f"lse of {nq} queries on {nk} keys")
        q0, k0 = q0 + nq, k0 + nk


# Tiles of up to 256 queries a request; the last with 1 to 128 rows runs odd and
# even key tiles, or pairs of heads from 304 tiles and heads on.  Means above
# 2,048 keys (causal) and 512 (not) run the straight-line softmax, those below the loops.
SHAPES = [
    ([300], [2600], 3),                                    # two tiles, then 44 rows
    ([257, 129], [2500, 2100], 5),                         # a last tile of one row, 129 rows
    ([90], [2700], 2), ([1], [2305], 1), ([33], [4100], 3),  # odd and even key tiles
    ([300, 129], [2600, 2300], 64),                        # claimed items, two tiles
    ([700, 40], [3000, 1700], 61),
    ([40, 100, 127], [2500, 2100, 3001], 125),             # claimed pairs of heads, one left over
    ([300, 1], [2200, 2100], 128),                         # two tiles and pairs of heads in one call
    ([40, 100, 127], [300, 210, 1300], 125),               # the same with loops when causal
    ([300, 129], [400, 135], 64),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,kv_lens,H", SHAPES)
def test_prefill_long_without_workspace(mla, q_lens, kv_lens, H, causal):
    c = prefill_case(np.random.default_rng(sum(q_lens) + H), q_lens, kv_lens, H)
    run_prefill(mla, c, causal=causal)
    check_heads(c, sorted({0, H // 2, H - 1, max(H - 2, 0)}), causal)
    assert torch.isfinite(c["out"]).all() and torch.isfinite(c["lse"]).all()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,kv_lens,H", [([300, 129], [2600, 2300], 64), ([40, 100, 127], [2500, 2100, 3001], 125),
                                              ([40, 100, 127], [300, 210, 1300], 125)])
def test_prefill_claimed_items_repeat_bit_for_bit(mla, q_lens, kv_lens, H, causal):
    """Which block claims an item changes from run to run; what comes out does not."""
    c = prefill_case(np.random.default_rng(7), q_lens, kv_lens, H)
    first = None
    for _ in range(10):
        c["out"].fill_(float("nan"))
        run_prefill(mla, c, causal=causal)
        got = (bits(c["out"]), bits(c["lse"]))
        if first is None:
            first = got
        assert np.array_equal(got[0], first[0]) and np.array_equal(got[1], first[1])


@pytest.mark.parametrize("causal", [True, False])
def test_prefill_long_rows_behind_a_request_never_matter(mla, causal):
    """Straight-line softmax, claimed items: NaN behind every request's rows, key counts that
    leave 1 to 15 rows of a step of 16."""
    lens_q, lens_k, H = [130, 300, 65], [2113, 2575, 2305], 51
    c = prefill_case(np.random.default_rng(8), lens_q, lens_k, H, q_behind=200, kv_behind=300)
    run_prefill(mla, c, causal=causal)
    rows = sum(lens_q)
    assert torch.isnan(c["out"][rows:]).all() and torch.isnan(c["lse"][rows:]).all()
    check_heads(c, [0, 25, 50], causal)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,H", [([60001], 1), ([20000, 1, 0, 25003], 2)])
def test_expand_many_changes_of_rows(mla, lens, H, fp8):
    """Few heads on many rows: a block walks through several tiles of rows."""
    c = expand_case(np.random.default_rng(9), lens, H, 64, fp8, behind=70)
    st = word()
    run_expand(mla, c, 0.37 if fp8 else None, dev_status=st)
    assert int(st) == 0
    check_expand(c, 0.37 if fp8 else 1.0)


# ------------------------------------------------------------------- scores of -inf

INF = float("inf")

# every form of an item: two tiles, odd and even key tiles, pairs of heads (and one left over), keys
# in parts; with loops and straight-line
FORMS = [([300], [300], 2, False), ([300], [2600], 2, False), ([60], [60], 3, False), ([60], [2600], 3, False), ([1], [1], 1, False),
         ([40, 100, 127], [60, 130, 130], 125, False), ([40, 100, 127], [2500, 2100, 3001], 125, False), ([5, 3], [2000, 900], 2, True),
         ([140], [2500], 1, True), ([3], [9], 1, True)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,kv_lens,H,split", FORMS)
def test_prefill_query_whose_scores_are_all_minus_infinity(mla, q_lens, kv_lens, H, split, causal):
    """An infinite query dim against keys of the other sign: NaN, not the row of a query that sees nothing."""
    c = prefill_case(np.random.default_rng(51), q_lens, kv_lens, H)
    c["kn"][:, :, 9] = -c["kn"][:, :, 9].abs() - 1
    starts = np.concatenate([[0], np.cumsum(q_lens)])
    rows = sorted({int(r) for b, n in enumerate(q_lens) for r in (starts[b], starts[b] + n // 2, starts[b] + n - 1)})
    keep = np.setdiff1d(np.arange(sum(q_lens)), rows)
    run_prefill(mla, c, causal=causal, ws=mla.make_prefill_workspace() if split else None)
    before = bits(c["out"][keep]), bits(c["lse"][keep])
    c["qn"][rows, :, 9] = INF
    run_prefill(mla, c, causal=causal, ws=mla.make_prefill_workspace() if split else None)
    assert torch.isnan(c["out"][rows]).all() and torch.isnan(c["lse"][rows]).all()
    assert np.array_equal(bits(c["out"][keep]), before[0]) and np.array_equal(bits(c["lse"][keep]), before[1])


@pytest.mark.parametrize("q_len,H,split", [(300, 2, False), (60, 3, False), (100, 128, False), (60, 1, True)])
def test_prefill_key_whose_scores_are_minus_infinity(mla, q_len, H, split):
    """The first key of a causal prompt: its own query sees only it (NaN), for the others it has no weight."""
    c = prefill_case(np.random.default_rng(52), [q_len] * 3, [q_len] * 3, H)
    c["qn"][:, :, 7] = c["qn"][:, :, 7].abs() + 1
    first = [0, q_len, 2 * q_len]
    c["kn"][first, :, 7] = -INF
    run_prefill(mla, c, ws=mla.make_prefill_workspace() if split else None)
    assert torch.isnan(c["out"][first]).all() and torch.isnan(c["lse"][first]).all()
    heads = sorted({0, H - 1})
    qn, qp, kn, kp, v = (f64(c[n] if n == "kp" else c[n][:, heads]) for n in ("qn", "qp", "kn", "kp", "v"))
    for a in first:
        rows = slice(a + 1, a + q_len)
        out, lse, mag, size = op.attend(qn[rows], qp[rows], kn[rows], kp[rows], v[rows], float(np.float32(0.07)), True)
        tol, lse_tol = attend_tol(out, lse, mag, size, q_len)
        assert_within(f64(c["out"][rows][:, heads]), out, tol)
        assert_within(f64(c["lse"][rows][:, heads]), lse, lse_tol)


@pytest.mark.parametrize("split", [False, True])
def test_prefill_infinite_query_that_sees_no_key(mla, split):
    """More queries than keys: rows in front of the first key stay 0 and -inf whatever the query holds."""
    c = prefill_case(np.random.default_rng(53), [200, 30], [40, 3], 2)
    c["qn"][:160], c["qp"][200:227] = INF, float("nan")
    run_prefill(mla, c, ws=mla.make_prefill_workspace() if split else None)
    for rows in (slice(0, 160), slice(200, 227)):
        assert (c["out"][rows] == 0).all() and torch.isneginf(c["lse"][rows]).all()
    assert torch.isfinite(c["out"][160:200]).all() and torch.isfinite(c["lse"][227:]).all()


# ------------------------------------------------------------------- append, smallest scale

def test_append_e4m3_zeros_stay_zero_at_the_smallest_scales(mla):
    """1 / kv_scale next to fp32's largest: everything but zero saturates, in rows that are computed
    in pairs of fp32 (some 3% of them here) as in those that are not."""
    rng = np.random.default_rng(54)
    T = 4096
    kv = torch.from_numpy((rng.standard_normal((T, 576)) * 0.1).astype(np.float32)).cuda().to(torch.bfloat16)
    weight = torch.from_numpy((1 + 0.1 * rng.standard_normal(512)).astype(np.float32)).cuda().to(torch.bfloat16)
    kv[:, 5], kv[::2, 300:340] = 0, 0
    table = torch.cat([torch.ones(1, 32), torch.zeros(1, 32)], 1).cuda()
    cache = torch.zeros(T // 64, 64, 576, dtype=torch.uint8, device="cuda")
    mla.mla_rope_append_fp8(kv, torch.zeros(T, dtype=torch.int64, device="cuda"), table, torch.arange(T, device="cuda"), cache, kv_scale=1e-38,
                            norm_weight=weight)
    got = cache.view(torch.float8_e4m3fn).float().view(T, 576)
    assert torch.equal(got, torch.sign(kv.float()) * 448)


# ------------------------------------------------------------------- several calls

def several(mla):
    """Split, straight-line and short calls, each with what it gives alone."""
    rng = np.random.default_rng(55)
    cases = [prefill_case(rng, *shape) for shape in (([5, 1, 3], [2000, 1097, 1600], 4), ([300, 40], [2600, 1900], 32), ([1, 17, 64, 200],) * 2 + (64,))]
    ws = mla.make_prefill_workspace()
    for c in cases:
        run_prefill(mla, c, ws=ws)
        c["alone"] = bits(c["out"]), bits(c["lse"])
        c["out"].zero_()
    return cases


def call(mla, c, ws, stream=None):
    mla.mla_prefill(c["qn"], c["qp"], c["kn"], c["kp"], c["v"], c["qo"], c["ko"], 0.07, c["out"], c["lse"], workspace=ws, stream=stream)


def test_prefill_calls_at_once(mla):
    """Three streams, a workspace each."""
    cases = several(mla)
    streams, ws = [torch.cuda.Stream() for _ in cases], [mla.make_prefill_workspace() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, w in zip(cases, streams, ws):
            call(mla, c, w, s)
    torch.cuda.synchronize()
    for c in cases:
        assert np.array_equal(bits(c["out"]), c["alone"][0]) and np.array_equal(bits(c["lse"]), c["alone"][1])


def test_prefill_graphs_that_share_a_workspace(mla):
    """Captured apart, replayed one after the other on one stream."""
    cases, ws, graphs = several(mla), mla.make_prefill_workspace(), []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for c in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call(mla, c, ws)
        graphs.append(graph)
    for _ in range(10):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for c in cases:
        assert np.array_equal(bits(c["out"]), c["alone"][0]) and np.array_equal(bits(c["lse"]), c["alone"][1])
