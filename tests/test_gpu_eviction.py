"""Decode over a shared prefix and cache eviction on the GPU, against their
definitions in fp64 (tolerances: eviction_helpers)."""
import numpy as np
import pytest

import oracle.eviction as oe
from eviction_helpers import (SCALE, bf16, check_mass, check_shared, i32, mass_case, mass_rows, paged, run_mass, run_shared, shared_case, word)
from prompt_helpers import f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def mla():
    import mla_latent_cache_decode_gb300 as mla
    torch.cuda.set_device(0)
    return mla


# ------------------------------------------------------------------------- shared prefix

SHARED = [
    # heads, page, shared blocks, lengths
    (1, 16, 1, [16]),
    (1, 16, 3, [49]),
    (16, 16, 4, [65, 64, 81, 128, 264]),
    (16, 64, 8, [512 + n for n in (1, 17, 64, 200)]),
    (5, 32, 9, [288 + n for n in (1, 2, 3, 63, 64, 65, 127, 128, 129, 255, 256, 257)]),
    (32, 128, 5, [641, 900, 640, 1100, 777]),
    (40, 64, 7, [449, 512, 600, 700]),
    (100, 16, 20, [321, 400, 336]),
    (128, 64, 5, [321, 320, 577, 1000]),
    (128, 256, 3, [769, 1300, 768]),
    (64, 256, 4, [1025, 1024, 1500]),
    (8, 16, 33, [529 + n for n in range(20)]),
]


@pytest.mark.parametrize("heads,page,shared,lens", SHARED)
def test_shared_against_definition(mla, heads, page, shared, lens):
    c = shared_case(np.random.default_rng(heads + page), heads, page, shared, lens)
    run_shared(mla, c)
    assert int(c["status"]) == 0
    check_shared(c)


@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("lens", [[0], [0, 300, 0], [1, 5, 31, 32, 33, 400], [160, 159, 161, 0, 1]])
def test_shared_short_and_empty_requests(mla, heads, lens):
    """Lengths below the shared part, 0 and 1 among them: they see their own first tokens only, also
    when the rows behind those hold NaN."""
    rng = np.random.default_rng(5)
    c = shared_case(rng, heads, 16, 10, lens)
    run_shared(mla, c)
    assert int(c["status"]) == 0
    check_shared(c)


@pytest.mark.parametrize("heads", [16, 128])
def test_shared_non_finite_rows_stay_with_those_that_see_them(mla, heads):
    c = shared_case(np.random.default_rng(6), heads, 32, 10, [330, 350, 100, 321, 0])
    rows = f64(c["cache"]).copy()
    c["cache"][int(c["table"][1][10]), 20] = float("inf")  # token 340 of request 1
    c["cache"][int(c["shared"][4]), 3] = float("nan")      # token 131: everybody's but request 2's
    run_shared(mla, c)
    out = f64(c["out"])
    assert np.isnan(out[[0, 1, 3]]).any(-1).all()
    ref, _ = oe.decode(f64(c["q"])[2], oe.rows_of(rows, c["table"], 2, 100, c["shared"]), SCALE)
    assert np.isfinite(out[2]).all() and np.abs(out[2] - ref).max() < 0.05
    assert (out[4] == 0).all()


@pytest.mark.parametrize("heads,batch", [(16, 40), (2, 200), (128, 30), (100, 12), (33, 21)])
def test_shared_many_requests(mla, heads, batch):
    rng = np.random.default_rng(batch)
    lens = [int(512 + n) for n in rng.integers(1, 300, batch)]
    c = shared_case(rng, heads, 64, 8, lens)
    run_shared(mla, c)
    assert int(c["status"]) == 0
    check_shared(c)


@pytest.mark.parametrize("heads,batch", [(1, 1500), (16, 385), (128, 386)])
def test_shared_more_requests_than_threads(mla, heads, batch):
    """Lengths are summed up a block's threads at a time; empty requests and short ones among them."""
    rng = np.random.default_rng(batch)
    lens = [int(n) for n in rng.choice([0, 1, 33, 64, 65, 90], batch)]
    c = shared_case(rng, heads, 32, 2, lens)
    run_shared(mla, c)
    assert int(c["status"]) == 0
    check_shared(c)


@pytest.mark.parametrize("heads", [16, 128])
def test_shared_nothing_in_common(mla, heads):
    c = shared_case(np.random.default_rng(8), heads, 64, 0, [300, 1, 64, 0, 999])
    run_shared(mla, c)
    check_shared(c)


@pytest.mark.parametrize("heads", [16, 128])
def test_shared_long(mla, heads):
    c = shared_case(np.random.default_rng(9), heads, 256, 30, [7680 + 3000, 7681])
    run_shared(mla, c)
    check_shared(c)


def test_shared_large_scores(mla):
    """Scores that rise and fall by hundreds over the tokens: every rescale is taken."""
    c = shared_case(np.random.default_rng(10), 16, 64, 12, [768 + 400, 769, 1000], by=20.0)
    run_shared(mla, c)
    check_shared(c)
    ramp = torch.linspace(0, 40, c["cache"].shape[0] * 64, device="cuda").view(-1, 64, 1)
    c["cache"][..., 512:] = (ramp * 0.2 + 0 * c["cache"][..., 512:].nan_to_num()).to(torch.bfloat16)
    c["q"][..., 512:] = 1.0
    c["cache"] = c["cache"].nan_to_num()
    run_shared(mla, c)
    check_shared(c)


def test_shared_equals_decode(mla):
    """The same numbers, within both calls' tolerance, as mla_decode over whole tables."""
    c = shared_case(np.random.default_rng(11), 128, 64, 6, [384 + n for n in (1, 100, 500)])
    whole = c["table"].copy()
    whole[:, :6] = c["shared"]
    other = torch.empty_like(c["out"])
    run_shared(mla, c)
    mla.mla_decode(c["q"], c["cache"], i32(whole), c["seq_lens"], SCALE, other)
    assert (c["out"].float() - other.float()).abs().max() < 0.02


def test_shared_without_lse_and_twice_the_same_bits(mla):
    c = shared_case(np.random.default_rng(12), 16, 64, 10, [640 + n for n in (3, 90, 700)])
    ws = mla.make_shared_workspace(3, 16)
    run_shared(mla, c, workspace=ws)
    first = c["out"].clone()
    ws.fill_(255)
    c["lse"] = None
    run_shared(mla, c, workspace=ws)
    assert torch.equal(first, c["out"])


def test_shared_replayed_with_other_lengths(mla):
    """A captured call follows the lengths, the shared count and the tables."""
    rng = np.random.default_rng(13)
    c = shared_case(rng, 16, 64, 8, [512 + 300, 512 + 700, 900])
    d = shared_case(rng, 16, 64, 3, [193, 800, 0])
    ws = mla.make_shared_workspace(3, 16)
    pool = max(c["cache"].shape[0], d["cache"].shape[0])
    width = max(c["table"].shape[1], d["table"].shape[1])
    live = dict(cache=torch.zeros(pool, 64, 576, dtype=torch.bfloat16, device="cuda"), q=c["q"].clone(),
                shared_table=torch.zeros(8, dtype=torch.int32, device="cuda"), shared_blocks=word(),
                block_table=torch.full((3, width), -7, dtype=torch.int32, device="cuda"), seq_lens=i32([0, 0, 0]), out=c["out"], lse=c["lse"],
                status=word())

    def load(x):
        live["cache"][:x["cache"].shape[0]] = x["cache"]
        live["q"].copy_(x["q"])
        live["shared_table"][:len(x["shared"])] = x["shared_table"]
        live["shared_blocks"].copy_(x["shared_blocks"])
        live["block_table"][:, :x["table"].shape[1]] = x["block_table"]
        live["seq_lens"].copy_(x["seq_lens"])

    load(c)
    run_shared(mla, live, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_shared(mla, live, workspace=ws)
    for x in (c, d, c):
        load(x)
        live["out"].fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        check_shared(dict(x, out=live["out"], lse=live["lse"], cache=x["cache"]))
    assert int(live["status"]) == 0


def test_shared_two_at_once(mla):
    """Two streams, a workspace each."""
    cases = [shared_case(np.random.default_rng(s), h, 64, 6, [384 + 100 * i + s for i in range(5)]) for s, h in ((14, 16), (15, 128))]
    ws = [mla.make_shared_workspace(5, c["q"].shape[1]) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, w, st in zip(cases, ws, streams):
            run_shared(mla, c, workspace=w, stream=st)
    torch.cuda.synchronize()
    for c in cases:
        check_shared(c)


def test_shared_on_another_stream_without_workspace(mla):
    """Its workspace is that stream's, whatever the current one allocates next."""
    c = shared_case(np.random.default_rng(17), 16, 64, 6, [384 + 100 * i + 5 for i in range(8)])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        c["out"].zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            run_shared(mla, c, stream=stream)
            torch.full((mla.mla_decode_shared_workspace_size(8, 16),), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        check_shared(c)


@pytest.mark.parametrize("heads", [16, 128])
def test_shared_reports_what_lies_outside(mla, heads):
    c = shared_case(np.random.default_rng(16), heads, 64, 5, [320 + 100, 320 + 90, 500])
    c["cache"] = c["cache"].nan_to_num()
    for key, bad in (("shared_blocks", i32([6])), ("shared_blocks", i32([-1])), ("seq_lens", i32([420, -3, 500])),
                     ("seq_lens", i32([420, 100000, 500])), ("shared_table", i32([0, 1, 2, 3, 1 << 30])),
                     ("block_table", torch.full_like(c["block_table"], -1)), ("block_table", torch.full_like(c["block_table"], 2 ** 31 - 1))):
        x = dict(c, status=word(), **{key: bad})
        run_shared(mla, x)
        assert int(x["status"]) == 5, key
    run_shared(mla, c)
    assert int(c["status"]) == 0
    check_shared(c)


# ------------------------------------------------------------------------- weights

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,page,lens", [
    (128, 64, [201]), (128, 16, [2, 18, 65, 201]), (16, 64, [1, 127, 128, 129, 700]), (1, 16, [5, 33]), (5, 32, [64, 63, 300, 1]),
    (40, 256, [1000, 256]), (128, 128, [129, 511, 1024]), (100, 64, [77]), (128, 64, [0, 0]), (32, 64, [0, 100, 0, 3]), (17, 16, [640] * 9)])
def test_mass_against_definition(mla, heads, page, lens, fp8):
    c = mass_case(np.random.default_rng(heads + page), heads, page, lens, fp8)
    run_mass(mla, c)
    assert int(c["status"]) == 0
    check_mass(c, 0.0, None)
    run_mass(mla, c, previous=c["previous"], decay=0.75)
    check_mass(c, 0.75, f64(c["previous"]))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,batch", [(2, 1200), (40, 390)])
def test_mass_more_requests_than_threads(mla, heads, batch, fp8):
    rng = np.random.default_rng(batch)
    c = mass_case(rng, heads, 16, [int(n) for n in rng.choice([0, 1, 33, 64, 65, 130], batch)], fp8)
    run_mass(mla, c)
    assert int(c["status"]) == 0
    check_mass(c, 0.0, None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads", [3, 40])
def test_mass_long(mla, heads, fp8):
    """More tiles than the rings' rounds and S's buffers, on every pair of SMs."""
    c = mass_case(np.random.default_rng(28), heads, 64, [12001, 700, 3000], fp8)
    run_mass(mla, c)
    assert int(c["status"]) == 0
    check_mass(c, 0.0, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_mass_rows_and_queries_that_are_not_finite(mla, fp8):
    """A token's weight is its own row's affair; a head's query is every token's of its request."""
    c = mass_case(np.random.default_rng(29), 16, 32, [200, 100, 90], fp8)
    run_mass(mla, c)
    clean = f64(c["mass"])
    if fp8:
        c["cache"][int(c["table"][0][2]), 7, 3] = 0x7F  # token 71: a NaN
    else:
        c["cache"][int(c["table"][0][2]), 7, 3] = float("nan")
    c["q"][2, 5, 100] = float("inf")
    run_mass(mla, c)
    got = f64(c["mass"])
    assert np.isnan(got[0, 71]) and np.array_equal(np.delete(got[0], 71), np.delete(clean[0], 71)) and np.array_equal(got[1], clean[1])
    assert not np.isfinite(got[2, :90]).any() or not fp8


@pytest.mark.parametrize("scale", [SCALE, 0.1, 0.125, 1.0])  # scale * log2(e) rounds up in some, down in others
@pytest.mark.parametrize("low", [-float("inf"), torch.finfo(torch.bfloat16).min])
def test_mass_rows_of_nothing(mla, low, scale):
    """A row that every head scores -inf, or lowest, has weight 0; what was there before stays."""
    c = mass_case(np.random.default_rng(30), 40, 32, [200, 100], False)
    c["q"][:, :, 3] = c["q"][:, :, 3].abs() + 1
    for b in range(2):
        c["lse"][b] = torch.from_numpy(oe.decode(f64(c["q"])[b], mass_rows(c, b), scale)[1]).float().cuda()

    def weigh(**kw):
        mla.mla_attention_mass(c["q"], c["cache"], c["block_table"], c["seq_lens"], scale, c["lse"], c["mass"], **kw)
        return f64(c["mass"])
    clean = weigh()
    c["cache"][int(c["table"][0][2]), 7, 3] = low  # token 71
    got = weigh()
    assert got[0, 71] == 0 and np.array_equal(np.delete(got[0], 71), np.delete(clean[0], 71)) and np.array_equal(got[1], clean[1])
    assert weigh(previous=c["previous"], decay=0.5)[0, 71] == 0.5 * f64(c["previous"])[0, 71]


@pytest.mark.parametrize("fp8", [False, True])
def test_mass_in_place_and_wide_rows(mla, fp8):
    """previous is mass itself, rows of a wider tensor; what is behind each end stays."""
    c = mass_case(np.random.default_rng(21), 16, 64, [300, 5, 129], fp8, width=400)
    wide = torch.rand(3, 1000, device="cuda")
    start = f64(wide)
    c["mass"] = wide[:, 100:500]
    run_mass(mla, c, previous=c["mass"], decay=0.5)
    check_mass(c, 0.5, start[:, 100:500], behind=start[:, 100:500])
    assert (f64(wide)[:, :100] == start[:, :100]).all() and (f64(wide)[:, 500:] == start[:, 500:]).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_mass_heads_without_weight(mla, fp8):
    c = mass_case(np.random.default_rng(22), 20, 32, [100, 64], fp8)
    c["lse"][0, 3] = -float("inf")
    c["lse"][1, ::2] = -float("inf")
    run_mass(mla, c)
    check_mass(c, 0.0, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_mass_sums_to_the_heads(mla, fp8):
    """With the decode's own lse the weights of a request add up to its number of heads."""
    c = mass_case(np.random.default_rng(23), 128, 64, [4096, 1000, 1], fp8)
    out, lse = torch.empty(3, 128, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 128, device="cuda")
    if fp8:
        mla.mla_decode_fp8(c["q"], c["cache"], c["block_table"], c["seq_lens"], SCALE, out, lse, kv_scale=c["kv_scale"])
    else:
        mla.mla_decode(c["q"], c["cache"], c["block_table"], c["seq_lens"], SCALE, out, lse)
    c["lse"] = lse
    c["mass"].zero_()
    run_mass(mla, c)
    total = f64(c["mass"]).sum(1)
    assert np.abs(total - 128).max() < 128 * 1e-3  # the two products' errors in the scores, about 576 2^-23 of some hundred


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("by", [1e-3, 30.0])
def test_mass_small_and_large_queries(mla, by, fp8):
    c = mass_case(np.random.default_rng(24), 16, 64, [333, 64], fp8, by=by)
    c["q"][:, :, 7] *= 50  # one dim far above the others
    lse = np.stack([oe.decode(f64(c["q"])[b], __import__("eviction_helpers").mass_rows(c, b), SCALE)[1] for b in range(2)])
    c["lse"] = torch.from_numpy(lse).float().cuda()
    run_mass(mla, c)
    check_mass(c, 0.0, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_mass_reports_what_lies_outside(mla, fp8):
    c = mass_case(np.random.default_rng(25), 16, 64, [300, 200], fp8)
    for key, bad in (("seq_lens", i32([300, -1])), ("seq_lens", i32([301, 200])), ("block_table", torch.full_like(c["block_table"], 1 << 30)),
                     ("block_table", torch.full_like(c["block_table"], -1))):
        x = dict(c, status=word(), mass=torch.full((4, 300), 3.0, device="cuda")[1:3], **{key: bad})
        run_mass(mla, x)
        assert int(x["status"]) == 5, key
        assert (x["mass"]._base[[0, 3]] == 3.0).all()


def test_mass_two_at_once_and_replayed(mla):
    cases = [mass_case(np.random.default_rng(s), h, 64, [700, 1, 300 + s], fp8) for s, h, fp8 in ((26, 128, False), (27, 16, True))]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for c, st in zip(cases, streams):
        run_mass(mla, c, stream=st)
    torch.cuda.synchronize()
    for c in cases:
        check_mass(c, 0.0, None)
    c = cases[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_mass(mla, c, previous=c["previous"], decay=0.5)
    c["lens"] = [20, 699, 0]
    c["table"] = np.concatenate([c["table"][:1], c["table"][:1], c["table"][2:]])
    c["block_table"].copy_(i32(c["table"]))
    c["seq_lens"].copy_(i32(c["lens"]))
    c["mass"].fill_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    check_mass(c, 0.5, f64(c["previous"]))


# ------------------------------------------------------------------------- choice

def check_select(mla, mass, lens, budget, sink, recent):
    B = len(lens)
    whole = torch.full((B + 2, budget), 99, dtype=torch.int32, device="cuda")
    new, st = torch.full((B,), 99, dtype=torch.int32, device="cuda"), word()
    mla.mla_evict_select(mass, i32(lens), whole[1:-1], new, sink=sink, recent=recent, dev_status=st)
    keep, w = whole.cpu().numpy(), f64(mass)
    assert int(st) == 0 and (keep[[0, -1]] == 99).all()
    for b, n in enumerate(lens):
        want = oe.select(w[b], n, budget, sink, recent)
        assert int(new[b]) == len(want)
        assert keep[b + 1].tolist() == want + [-1] * (budget - len(want)), (b, n)
    return whole[1:-1], new


@pytest.mark.parametrize("lens,budget,sink,recent", [
    ([2, 18, 65, 201], 32, 4, 8), ([1], 1, 0, 0), ([5, 0, 3], 2, 1, 1), ([5, 0, 3], 2, 0, 0), ([100, 31, 32, 33], 31, 0, 1),
    ([1000, 4096, 2049], 2048, 0, 2048), ([1000, 4096, 2049], 2048, 2048, 0), ([5000, 777, 4097], 1001, 5, 77), ([20000, 16384, 9000], 16383, 1, 1),
    ([3000] * 300, 17, 1, 2)])
def test_select_against_definition(mla, lens, budget, sink, recent):
    rng = np.random.default_rng(sum(lens) % 1000 + budget)
    mass = np.exp(2 * rng.standard_normal((len(lens), max(lens) + 3)) - 3).astype(np.float32)
    check_select(mla, torch.from_numpy(mass).cuda(), lens, budget, sink, recent)


@pytest.mark.parametrize("kind", ["equal", "two", "zeros", "signs", "nan", "inf", "ramp", "down", "tiny"])
@pytest.mark.parametrize("lens,budget", [([700, 40, 999], 300), ([40000, 33000], 9999)])
def test_select_ties_and_odd_values(mla, kind, lens, budget):
    rng = np.random.default_rng(31)
    S = max(lens)
    x = rng.standard_normal((len(lens), S)).astype(np.float32)
    mass = {"equal": np.ones_like(x), "two": (x > 1).astype(np.float32), "zeros": np.where(x > 0, 0.0, -0.0).astype(np.float32),
            "signs": np.sign(x) * np.float32(0.5), "nan": np.where(x > 0.3, np.nan, x), "inf": np.where(x > 1, np.inf, np.where(x < -1, -np.inf, x)),
            "ramp": np.broadcast_to(np.arange(S, dtype=np.float32), x.shape).copy(),
            "down": np.broadcast_to(-np.arange(S, dtype=np.float32), x.shape).copy(), "tiny": x * np.float32(1e-42)}[kind].astype(np.float32)
    check_select(mla, torch.from_numpy(mass).cuda(), lens, budget, 3, 10)


def test_select_very_long_and_strided(mla):
    rng = np.random.default_rng(32)
    mass = torch.from_numpy(np.exp(rng.standard_normal((2, 140000))).astype(np.float32)).cuda()
    check_select(mla, mass[:, 3:131075], [131072, 1024], 16001, 64, 1000)
    check_select(mla, mass[:, 1:], [139999, 70001], 100, 64, 10)


def test_select_reports_what_lies_outside(mla):
    mass = torch.rand(3, 100, device="cuda")
    for lens in ([100, 101, 5], [100, -1, 5], [2 ** 31 - 1, 1, 1]):
        keep, new, st = torch.zeros(3, 10, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"), word()
        mla.mla_evict_select(mass, i32(lens), keep, new, dev_status=st)
        assert int(st) == 5
        assert ((keep >= -1) & (keep < 100)).all() and ((new >= 0) & (new <= 10)).all()


# ------------------------------------------------------------------------- move

def compact_case(rng, lens, page, budget, layers, fp8, sink=2, recent=3):
    table, _, blocks = paged(rng, lens, page)
    shape = (layers, blocks, page, 576)
    cache = torch.from_numpy(rng.integers(0, 256, shape, dtype=np.uint8) if fp8 else rng.integers(0, 1 << 15, shape, dtype=np.int16)).cuda()
    cache = cache if fp8 else cache.view(torch.bfloat16)
    weights = rng.random((len(lens), max(lens) + 5)).astype(np.float32)
    keep = [oe.select(weights[b], n, budget, sink, recent) for b, n in enumerate(lens)]
    array = np.full((len(lens), budget), -1, np.int32)
    for b, k in enumerate(keep):
        array[b, :len(k)] = k
    return dict(lens=lens, table=table, keep=keep, cache=cache, block_table=i32(table), keep_t=i32(array), seq_lens=i32(lens),
                new_lens=i32([len(k) for k in keep]), mass=torch.from_numpy(weights).cuda(), fp8=fp8, status=word())


def bits(t):
    return (t if t.dtype == torch.uint8 else t.view(torch.int16)).cpu().numpy()


def run_compact(mla, c, mass=True, **kw):
    (mla.mla_cache_compact_fp8 if c["fp8"] else mla.mla_cache_compact)(c["cache"], c["block_table"], c["keep_t"], c["seq_lens"], c["new_lens"],
                                                                      mass=c["mass"] if mass else None, dev_status=c["status"], **kw)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,page,budget,layers", [
    ([40], 16, 20, 1), ([2, 18, 65, 201], 16, 32, 2), ([100, 0, 7], 7, 10, 1), ([700, 3000, 5], 64, 1000, 1), ([5000], 64, 4321, 1),
    ([300] * 40, 32, 100, 3), ([9000, 20], 128, 8999, 1), ([4097, 4096], 256, 2049, 2), ([33, 34], 1, 30, 1)])
def test_compact_against_definition(mla, lens, page, budget, layers, fp8):
    c = compact_case(np.random.default_rng(41), lens, page, budget, layers, fp8)
    want, weights = oe.compact(bits(c["cache"]), c["table"], c["keep"], c["lens"], f64(c["mass"]))
    run_compact(mla, c)
    assert int(c["status"]) == 0
    assert np.array_equal(bits(c["cache"]), want)
    assert np.array_equal(f64(c["mass"]), weights)


@pytest.mark.parametrize("fp8", [False, True])
def test_compact_one_layer_without_weights(mla, fp8):
    c = compact_case(np.random.default_rng(42), [500, 90], 32, 64, 1, fp8)
    want, _ = oe.compact(bits(c["cache"]), c["table"], c["keep"], c["lens"])
    before = c["mass"].clone()
    c["cache"] = c["cache"][0]
    run_compact(mla, c, mass=False)
    assert np.array_equal(bits(c["cache"]), want[0]) and torch.equal(before, c["mass"])


@pytest.mark.parametrize("kind", ["last", "first", "all", "even", "one", "none"])
def test_compact_shapes_of_what_stays(mla, kind):
    """The longest moves, none at all, every other token."""
    n = 6000
    c = compact_case(np.random.default_rng(43), [n, 50], 64, 6000, 1, False)
    kept = {"last": range(n - 3000, n), "first": range(3000), "all": range(n), "even": range(0, n, 2), "one": [n - 1], "none": []}[kind]
    c["keep"] = [list(kept), [49]]
    array = np.full((2, 6000), -1, np.int32)
    for b, k in enumerate(c["keep"]):
        array[b, :len(k)] = k
    c["keep_t"], c["new_lens"] = i32(array), i32([len(k) for k in c["keep"]])
    want, weights = oe.compact(bits(c["cache"]), c["table"], c["keep"], c["lens"], f64(c["mass"]))
    run_compact(mla, c)
    assert int(c["status"]) == 0
    assert np.array_equal(bits(c["cache"]), want) and np.array_equal(f64(c["mass"]), weights)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("requests,n,layers", [(1, 30000, 1), (3, 9000, 2), (20, 4096, 1), (40, 700, 4)])
def test_compact_again_and_again(mla, requests, n, layers, fp8):
    """Targets that are other blocks' sources: fresh rows, moved a little each time, always the same bits."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    page, blocks = 64, requests * -(-n // 64)
    table = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32).view(requests, -1)
    cache = torch.randint(0, 256, (layers, blocks, page, 576 if fp8 else 1152), generator=gen, device="cuda", dtype=torch.uint8)
    cache = cache if fp8 else cache.view(torch.bfloat16)
    slots = (table.long()[..., None] * page + torch.arange(page, device="cuda")).flatten(1)
    for gone in (1, 7, n // 2, n // 3, 1, 2, 3, 40, 50, 60):
        keep = torch.stack([torch.randperm(n, generator=gen, device="cuda")[gone:].sort()[0] for _ in range(requests)])
        want = cache.clone()
        rows = want.view(layers, blocks * page, -1).view(torch.uint8)
        rows[:, slots[:, :n - gone].flatten()] = rows[:, slots.gather(1, keep).flatten()]
        c = dict(cache=cache.clone(), block_table=table, keep_t=keep.to(torch.int32), seq_lens=i32([n] * requests),
                 new_lens=i32([n - gone] * requests), mass=torch.rand(requests, n, generator=gen, device="cuda"), fp8=fp8, status=word())
        weights = torch.cat([c["mass"].gather(1, keep), torch.zeros(requests, gone, device="cuda")], 1)
        run_compact(mla, c)
        assert torch.equal(c["mass"], weights)
        assert int(c["status"]) == 0 and torch.equal(c["cache"].view(torch.uint8), want.view(torch.uint8))


def test_compact_reports_what_lies_outside(mla):
    c = compact_case(np.random.default_rng(44), [300, 200], 16, 100, 1, False)
    start = c["cache"].clone()
    pool = torch.zeros(3, *start.shape[1:], dtype=torch.bfloat16, device="cuda")
    for key, bad in (("keep_t", c["keep_t"].flip(1)), ("keep_t", c["keep_t"] + 250), ("keep_t", c["keep_t"] * 0 - 5), ("new_lens", i32([101, 5])),
                     ("new_lens", i32([-1, 5])), ("seq_lens", i32([100000, 200])), ("seq_lens", i32([-7, 200])),
                     ("block_table", c["block_table"] + 1000), ("block_table", c["block_table"] * 0 - 1)):
        pool.zero_()
        pool[1] = start[0]
        wide = torch.full((4, 305), 3.0, device="cuda")
        x = dict(c, cache=pool[1:2], status=word(), mass=wide[1:3])
        x[key] = bad
        run_compact(mla, x)
        assert int(x["status"]) == 5, key
        assert (pool[0] == 0).all() and (pool[2] == 0).all() and (wide[[0, 3]] == 3.0).all()


def test_compact_keeps_shared_pages(mla):
    """Two requests with their first two pages in common, whose tokens stay: the pages are not written."""
    c = compact_case(np.random.default_rng(45), [200, 150], 16, 60, 1, False, sink=32)
    c["table"][1, :2] = c["table"][0, :2]
    c["block_table"] = i32(c["table"])
    want, _ = oe.compact(bits(c["cache"]), c["table"], c["keep"], c["lens"])
    run_compact(mla, c, mass=False)
    assert np.array_equal(bits(c["cache"]), want)


# ------------------------------------------------------------------------- together

@pytest.mark.parametrize("heads", [16, 128])
def test_decode_weigh_choose_move_decode(mla, heads):
    """A step with a shared prefix, its weights, a cut to a budget that keeps the prefix, and the next
    decode over what is left: the same as attention over the rows that stayed."""
    rng = np.random.default_rng(51)
    page, first, lens, budget = 16, 4, [64 + n for n in (10, 300, 171)], 120
    c = shared_case(rng, heads, page, first, lens)
    whole = c["table"].copy()
    whole[:, :first] = c["shared"]
    run_shared(mla, c)
    check_shared(c)
    mass = torch.zeros(3, 400, device="cuda")
    for _ in range(2):  # two layers' worth
        mla.mla_attention_mass(c["q"], c["cache"], i32(whole), c["seq_lens"], SCALE, c["lse"], mass, previous=mass)
    w = f64(mass)
    assert np.abs(w.sum(1) - 2 * heads).max() < 0.01 * heads
    keep, new = torch.empty(3, budget, dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    mla.mla_evict_select(mass, c["seq_lens"], keep, new, sink=64, recent=16)
    before = f64(c["cache"]).copy()
    mla.mla_cache_compact(c["cache"], i32(whole), keep, c["seq_lens"], new, mass=mass, dev_status=c["status"])
    mla.mla_decode_shared(c["q"], c["cache"], c["shared_table"], c["shared_blocks"], c["block_table"], new, SCALE, c["out"], c["lse"],
                          dev_status=c["status"])
    assert int(c["status"]) == 0
    for b, n in enumerate(lens):
        kept = oe.select(w[b], n, budget, 64, 16)
        rows = oe.rows_of(before, whole, b, n)[kept]
        ref, ref_lse = oe.decode(f64(c["q"])[b], rows, SCALE)
        from eviction_helpers import decode_tol
        from prompt_helpers import assert_within
        tol, ltol = decode_tol(f64(c["q"])[b], rows, SCALE, ref, ref_lse)
        assert_within(f64(c["out"])[b], ref, tol, f"request {b}")
        assert_within(f64(c["lse"])[b], ref_lse, ltol, f"lse of request {b}")
        assert np.array_equal(f64(mass)[b, :len(kept)], w[b, kept]) and (f64(mass)[b, len(kept):] == 0).all()
