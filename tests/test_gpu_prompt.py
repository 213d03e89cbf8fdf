"""GPU tests of the prompt side: mla_rope_append, mla_expand_kv, mla_prefill and
the run of them that hands a prompt over to the decode, against the fp64 oracle
with derived tolerances (prompt_helpers)."""
import numpy as np
import pytest

import mla_inputs as mi
import oracle
import oracle.prompt as op
from prompt_helpers import BF16, E4M3, assert_within, attend_tol, expand_tol, f64, pair_size, rope_tol

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

NAN = float("nan")


@pytest.fixture(scope="module")
def mla():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    import mla_latent_cache_decode_gb300 as m
    return m


def bf16(rng, *shape, by=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * by).astype(np.float32)).cuda().to(torch.bfloat16)


def i32(values):
    return torch.tensor(np.asarray(values), dtype=torch.int32, device="cuda")


def offsets(lens, start=0):
    return i32(start + np.concatenate([[0], np.cumsum(lens)]))


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def rope_table(n):
    angle = np.arange(n)[:, None] * 10000.0 ** (-np.arange(32) / 32)
    return torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).cuda()


# ------------------------------------------------------------------- append

def append_case(rng, T, H, norm=True, positions=5000):
    return dict(kv=bf16(rng, T, 576, by=2.0), q=bf16(rng, T, H, 64), weight=bf16(rng, 512) if norm else None, table=rope_table(positions),
                positions=torch.from_numpy(rng.integers(0, positions, T)).cuda())


def append_ref(c, interleaved, eps=1e-6):
    kv, table, pos = f64(c["kv"]), f64(c["table"]), c["positions"].cpu().numpy()
    rows = op.rope_rows(kv, table, pos, None if c["weight"] is None else f64(c["weight"]), eps, interleaved)
    tol = rope_tol(kv, rows, table, pos, c["weight"] is not None)
    a = table[pos]
    q = op.rotate(f64(c["q"]), a[:, None, :32], a[:, None, 32:], interleaved)
    return rows, tol, q, BF16 * np.abs(q) + 3 * 2.0 ** -24 * pair_size(f64(c["q"]))


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("T,H,page", [(1, 128, 64), (3, 1, 1), (20, 16, 16), (57, 5, 48), (130, 33, 256)])
def test_append_bf16(mla, T, H, page, norm, interleaved):
    rng = np.random.default_rng(T + H)
    c = append_case(rng, T, H, norm)
    blocks = -(-T // page) + 2
    cache = torch.full((blocks, page, 576), NAN, dtype=torch.bfloat16, device="cuda")
    slots = rng.permutation(blocks * page)[:T]
    slots[T // 2] = -1  # this one's row is not stored, its query is rotated all the same
    out, st = torch.full_like(c["q"], NAN), word()
    mla.mla_rope_append(c["kv"], c["positions"], c["table"], torch.from_numpy(slots).cuda(), cache, norm_weight=c["weight"],
                        interleaved=interleaved, q_pe=c["q"], q_pe_out=out, dev_status=st)
    rows, tol, q, q_tol = append_ref(c, interleaved)
    keep = slots >= 0
    got = f64(cache).reshape(-1, 576)
    assert int(st) == 0
    assert_within(got[slots[keep]], rows[keep], (BF16 * np.abs(rows) + tol)[keep], "rows")
    assert np.isnan(np.delete(got, slots[keep], 0)).all()
    assert_within(f64(out), q, q_tol, "q")
    if not norm:  # untouched dims are copied bit for bit
        assert np.array_equal(got[slots[keep], :512], f64(c["kv"])[keep, :512])


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("scale", [1.0, 0.037, 4.0])
@pytest.mark.parametrize("T,H", [(1, 128), (70, 3)])
def test_append_e4m3(mla, T, H, scale, interleaved):
    rng = np.random.default_rng(11)
    c = append_case(rng, T, H)
    c["kv"][0, :8] *= 300.0
    cache = torch.full((T + 3, 16, 576), 0x5A, dtype=torch.uint8, device="cuda")
    slots = rng.permutation((T + 3) * 16)[:T]
    out, st = torch.full_like(c["q"], NAN), word()
    mla.mla_rope_append_fp8(c["kv"], c["positions"], c["table"], torch.from_numpy(slots).cuda(), cache, kv_scale=scale, norm_weight=c["weight"],
                            interleaved=interleaved, q_pe=c["q"], q_pe_out=out, dev_status=st)
    rows, tol, q, q_tol = append_ref(c, interleaved)
    assert int(st) == 0
    x = np.clip(rows / scale, -448, 448)
    # half a step, and what fp32 is off by before it (the reciprocal's and the product's rounding too)
    bound = np.maximum(E4M3 * np.abs(x), 2.0 ** -10) + tol / scale + 4 * 2.0 ** -24 * np.abs(x)
    got = cache.cpu().numpy().reshape(-1, 576)
    assert_within(oracle.e4m3_value(got[slots].ravel()).reshape(T, 576), x, bound, "codes")
    assert (np.delete(got, slots, 0) == 0x5A).all()
    assert_within(f64(out), q, q_tol, "q")


def e4m3_nearest(x):
    """The E4M3 value nearest to x (fp64), ties to even."""
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)
    return np.clip(np.round(x / step) * step, -448, 448)


@pytest.mark.parametrize("interleaved", [True, False])
def test_append_e4m3_codes_are_those_of_the_exact_values(mla, interleaved):
    """Next to the middle of two codes fp32 would take the wrong one of one value in a million."""
    rng = np.random.default_rng(14)
    T = 16000
    c = append_case(rng, T, 1)
    c["table"][0] = torch.cat([torch.ones(32), torch.zeros(32)]).cuda()
    cache = torch.zeros(T // 64, 64, 576, dtype=torch.uint8, device="cuda")
    mla.mla_rope_append_fp8(c["kv"], c["positions"], c["table"], torch.arange(T, device="cuda"), cache, kv_scale=0.037, norm_weight=c["weight"],
                            interleaved=interleaved)
    rows = append_ref(c, interleaved)[0]
    rows *= float(np.float32(1) / np.float32(0.037))
    turned = c["positions"].cpu().numpy() != 0  # (x itself is scaled in fp32)
    got = cache.view(torch.float8_e4m3fn).double().cpu().numpy().reshape(T, 576)
    assert np.array_equal(got[turned], e4m3_nearest(rows[turned]))


def test_append_without_query_equals_finished_rows(mla):
    """No weight and position 0 (cos 1, sin 0): what mla_cache_append(_fp8) stores, bit for bit."""
    rng = np.random.default_rng(5)
    T = 37
    kv, slots = bf16(rng, T, 576), torch.from_numpy(rng.permutation(64)[:T]).cuda()
    zeros = torch.zeros(T, dtype=torch.int64, device="cuda")
    a, b = (torch.zeros(4, 16, 576, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mla.mla_rope_append(kv, zeros, rope_table(2), slots, a)
    mla.mla_cache_append(kv, slots, b)
    assert np.array_equal(bits(a), bits(b))
    a, b = (torch.zeros(4, 16, 576, dtype=torch.uint8, device="cuda") for _ in range(2))
    mla.mla_rope_append_fp8(kv, zeros, rope_table(2), slots, a, kv_scale=0.3)
    mla.mla_cache_append_fp8(kv, slots, b, kv_scale=0.3)
    assert np.array_equal(bits(a), bits(b))


def test_append_strides_in_place_and_into_the_absorbed_query(mla):
    rng = np.random.default_rng(6)
    T, H = 9, 7
    c = append_case(rng, T, H)
    wide = bf16(rng, T, 1536 + 576)  # a fused projection's output: the latent rows are its tail
    wide[:, 1536:] = c["kv"]
    full = bf16(rng, T, H, 192)      # heads of 128 + 64
    full[..., 128:] = c["q"]
    absorbed = torch.full((T, H, 576), NAN, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(T, device="cuda")
    cache = torch.zeros(1, 16, 576, dtype=torch.bfloat16, device="cuda")
    args = (wide[:, 1536:], c["positions"], c["table"], slots, cache)
    mla.mla_rope_append(*args, norm_weight=c["weight"], q_pe=full[..., 128:], q_pe_out=absorbed[..., 512:])
    rows, tol, q, q_tol = append_ref(c, True)
    assert_within(f64(cache)[0, :T], rows, BF16 * np.abs(rows) + tol)
    assert_within(f64(absorbed)[..., 512:], q, q_tol)
    assert torch.isnan(absorbed[..., :512]).all()
    before = full[..., :128].clone()
    mla.mla_rope_append(*args, norm_weight=c["weight"], q_pe=full[..., 128:], q_pe_out=full[..., 128:])
    assert np.array_equal(bits(full[..., 128:]), bits(absorbed[..., 512:]))
    assert np.array_equal(bits(full[..., :128]), bits(before))
    # heads outermost
    swapped = torch.full((H, T, 64), NAN, dtype=torch.bfloat16, device="cuda")
    mla.mla_rope_append(*args, q_pe=c["q"], q_pe_out=swapped.transpose(0, 1))
    assert np.array_equal(bits(swapped.transpose(0, 1)), bits(absorbed[..., 512:]))


def test_append_reports_what_lies_outside(mla):
    rng = np.random.default_rng(7)
    for fp8 in (False, True):
        c = append_case(rng, 4, 2, positions=50)
        c["positions"] = torch.tensor([3, 50, -1, 4], device="cuda")
        cache = torch.zeros(2, 16, 576, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
        out, st = torch.full_like(c["q"], NAN), word()
        fn = mla.mla_rope_append_fp8 if fp8 else mla.mla_rope_append
        fn(c["kv"], c["positions"], c["table"], torch.tensor([0, 1, 2, 3], device="cuda"), cache, q_pe=c["q"], q_pe_out=out, dev_status=st)
        assert int(st) == 5
        wrote = (f64(cache.float())[0] != 0).any(1)
        assert wrote[[0, 3]].all() and not wrote[[1, 2]].any() and not wrote[4:].any()
        assert torch.isfinite(out[[0, 3]]).all() and torch.isnan(out[[1, 2]]).all()
        st = word()
        fn(c["kv"][:2], torch.zeros(2, dtype=torch.int64, device="cuda"), c["table"], torch.tensor([32, -2], device="cuda"), cache, dev_status=st)
        assert int(st) == 5


def test_append_zero_rows_and_special_values(mla):
    """A zero row stays zero under the norm; infinities and NaN stay in their own token."""
    rng = np.random.default_rng(8)
    c = append_case(rng, 4, 1)
    c["kv"][1] = 0
    c["kv"][2, 5], c["kv"][2, 520] = float("inf"), NAN
    cache = torch.zeros(1, 16, 576, dtype=torch.bfloat16, device="cuda")
    mla.mla_rope_append(c["kv"], c["positions"], c["table"], torch.arange(4, device="cuda"), cache, norm_weight=c["weight"])
    got = f64(cache)[0]
    with np.errstate(invalid="ignore"):
        rows, tol, _, _ = append_ref(c, True)
    assert (got[1] == 0).all() and np.isnan(got[2]).any()
    # E4M3: an infinity saturates, where the rotation or a row without a weight keeps it one
    codes = torch.zeros(1, 16, 576, dtype=torch.uint8, device="cuda")
    c["kv"][3], c["kv"][3, 7], c["kv"][3, 530] = 1, -float("inf"), float("inf")
    mla.mla_rope_append_fp8(c["kv"], c["positions"], c["table"], torch.arange(len(c["kv"]), device="cuda"), codes, kv_scale=0.25)
    val = codes.view(torch.float8_e4m3fn).float().cpu().numpy()[0]
    assert val[3, 7] == -448 and (val[3, :7] == 4).all() and set(np.abs(val[3, 530:532])) == {448.0} and np.isnan(val[2, 520])
    assert_within(got[[0, 3]], rows[[0, 3]], (BF16 * np.abs(rows) + tol)[[0, 3]])


# ------------------------------------------------------------------- expand

def expand_case(rng, lens, H, page, fp8=False, start=0, behind=0):
    B, total = len(lens), sum(lens)
    need = [-(-n // page) for n in lens]
    blocks = max(1, sum(need)) + 3
    table = mi.make_block_table(rng, lens, page, blocks)
    cache = mi.poison_unused(mi.f32_to_bf16_bits(rng.standard_normal((blocks, page, 576), dtype=np.float32)), table, lens, page)
    rows = np.concatenate([mi.gather_rows(cache, table, b, n, page) for b, n in enumerate(lens)]) if total else np.zeros((0, 576), np.uint16)
    rows = mi.bf16_bits_to_f32(rows).astype(np.float64)
    t = torch.from_numpy(cache.view(np.int16)).cuda().view(torch.bfloat16)
    if fp8:
        t = t.float().to(torch.float8_e4m3fn).view(torch.uint8)
        rows = torch.from_numpy(rows).float().to(torch.float8_e4m3fn).double().numpy()
    T = start + total + behind
    full = lambda *s: torch.full(s, NAN, dtype=torch.bfloat16, device="cuda")
    return dict(cache=t, table=i32(table), offsets=offsets(lens, start), w_uk=bf16(rng, H, 128, 512, by=0.05), w_uv=bf16(rng, H, 512, 128, by=0.05),
                k=full(T, H, 128), v=full(T, H, 128), pe=full(T, 64), rows=rows, start=start, total=total)


def run_expand(mla, c, scale=None, **kw):
    args = [c[n] for n in ("cache", "table", "offsets", "w_uk", "w_uv", "k", "v", "pe")]
    if scale is None:
        mla.mla_expand_kv(*args, **kw)
    else:
        mla.mla_expand_kv_fp8(*args, kv_scale=scale, **kw)


def check_expand(c, scale=1.0):
    rows = c["rows"] * np.float64(np.float32(scale))
    k, v = op.expand(rows, f64(c["w_uk"]), f64(c["w_uv"]))
    k_tol, v_tol = expand_tol(rows, f64(c["w_uk"]), f64(c["w_uv"]), k, v)
    mine = slice(c["start"], c["start"] + c["total"])
    assert_within(f64(c["k"])[mine], k, k_tol, "k_nope")
    assert_within(f64(c["v"])[mine], v, v_tol, "v")
    assert_within(f64(c["pe"])[mine], rows[:, 512:], (BF16 if scale != 1.0 else 0) * np.abs(rows[:, 512:]), "k_pe")
    for name in ("k", "v", "pe"):  # rows of no request are left as they were
        assert torch.isnan(c[name][:c["start"]]).all() and torch.isnan(c[name][c["start"] + c["total"]:]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,H,page", [
    ([1], 1, 16), ([1], 128, 64), ([2, 18, 65, 201], 3, 16), ([127], 2, 64), ([128], 16, 64), ([129], 5, 32), ([0, 5, 0, 130, 0], 4, 16),
    ([257, 1, 255], 7, 256), ([33] * 9, 2, 48), ([1] * 300, 1, 1), ([640], 33, 128), ([300, 90], 128, 64)])
def test_expand(mla, lens, H, page, fp8):
    c = expand_case(np.random.default_rng(sum(lens) + H), lens, H, page, fp8)
    st = word()
    run_expand(mla, c, 0.37 if fp8 else None, dev_status=st)
    assert int(st) == 0
    check_expand(c, 0.37 if fp8 else 1.0)


@pytest.mark.parametrize("start,behind", [(3, 0), (0, 40), (130, 200)])
def test_expand_leaves_rows_of_no_request(mla, start, behind):
    c = expand_case(np.random.default_rng(21), [70, 150], 3, 32, start=start, behind=behind)
    run_expand(mla, c)
    check_expand(c)


def test_expand_e4m3_code_values(mla):
    """Every finite code comes out as its value: a unit weight copies latent dims to key dims."""
    c = expand_case(np.random.default_rng(22), [4], 2, 16, True)
    codes = np.arange(256, dtype=np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x38
    c["w_uk"].zero_()
    c["w_uv"].zero_()
    for h in range(2):
        c["w_uk"][h, torch.arange(128), 128 * h + torch.arange(128)] = 1
        c["w_uv"][h, 256 + 128 * h + torch.arange(128), torch.arange(128)] = 1
    row = np.concatenate([codes, codes[::-1], codes[:64]])
    c["cache"][int(c["table"][0, 0]), :4] = torch.from_numpy(np.ascontiguousarray(row)).cuda()
    run_expand(mla, c, 1.0)
    val = oracle.e4m3_value(row)
    assert np.array_equal(f64(c["k"])[2], val[:256].reshape(2, 128)) and np.array_equal(f64(c["v"])[1], val[256:512].reshape(2, 128))
    assert np.array_equal(f64(c["pe"])[3], val[512:])


@pytest.mark.parametrize("fp8", [False, True])
def test_expand_reports_pages_outside(mla, fp8):
    """Tables checked on the device: a block outside the pool, a request longer than its table."""
    rng = np.random.default_rng(23)
    for bad in (1 << 20, -5, 2 ** 31 - 1):
        c = expand_case(rng, [40, 20], 2, 16, fp8)
        c["table"][1, 0] = bad
        st = word()
        run_expand(mla, c, 1.0 if fp8 else None, dev_status=st)
        assert int(st) == 5
        k, _ = op.expand(c["rows"][:40], f64(c["w_uk"]), f64(c["w_uv"]))
        assert_within(f64(c["k"])[:40], k, 1e-2 * np.abs(k).max())
    c = expand_case(rng, [40, 20], 2, 16, fp8)
    c["offsets"] = i32([0, 60, 60])  # 60 tokens, three pages of 16
    st = word()
    run_expand(mla, c, 1.0 if fp8 else None, dev_status=st)
    assert int(st) == 5


@pytest.mark.parametrize("fp8", [False, True])
def test_expand_thousands_of_short_requests(mla, fp8):
    """More requests than are compared one by one, every fourth of them empty, the first and the last too."""
    lens = [0, 1, 2, 3] * 400 + [0]
    c = expand_case(np.random.default_rng(25), lens, 2, 2, fp8)
    st = word()
    run_expand(mla, c, 0.37 if fp8 else None, dev_status=st)
    assert int(st) == 0
    check_expand(c, 0.37 if fp8 else 1.0)


def test_expand_offsets_beyond_the_rows_are_cut(mla):
    c = expand_case(np.random.default_rng(24), [40, 20], 2, 16)
    c["offsets"] = i32([-3, 40, 1000])
    st = word()
    run_expand(mla, c, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 5


# ------------------------------------------------------------------- prefill

def prefill_case(rng, q_lens, kv_lens, H, by=1.5, q_start=0, kv_start=0, q_behind=0, kv_behind=0):
    Tq, Tk = q_start + sum(q_lens) + q_behind, kv_start + sum(kv_lens) + kv_behind
    c = dict(qn=bf16(rng, Tq, H, 128, by=by), qp=bf16(rng, Tq, H, 64, by=by), kn=bf16(rng, Tk, H, 128), kp=bf16(rng, Tk, 64), v=bf16(rng, Tk, H, 128),
             qo=offsets(q_lens, q_start), ko=offsets(kv_lens, kv_start), q_lens=q_lens, kv_lens=kv_lens, q_start=q_start, kv_start=kv_start,
             out=torch.full((Tq, H, 128), NAN, dtype=torch.bfloat16, device="cuda"), lse=torch.full((Tq, H), NAN, device="cuda"))
    for name in ("qn", "qp"):
        c[name][:q_start] = NAN
        c[name][Tq - q_behind:] = NAN
    for name in ("kn", "kp", "v"):
        c[name][:kv_start] = NAN
        c[name][Tk - kv_behind:] = NAN
    return c


def run_prefill(mla, c, scale=0.07, causal=True, ws=None, **kw):
    st = word()
    mla.mla_prefill(c["qn"], c["qp"], c["kn"], c["kp"], c["v"], c["qo"], c["ko"], scale, c["out"], c["lse"], causal=causal, workspace=ws,
                    dev_status=st, **kw)
    torch.cuda.synchronize()
    assert int(st) == 0


def check_prefill(c, scale=0.07, causal=True, only=None):
    qn, qp, kn, kp, v = (f64(c[n]) for n in ("qn", "qp", "kn", "kp", "v"))
    got, got_lse = f64(c["out"]), f64(c["lse"])
    q0, k0 = c["q_start"], c["kv_start"]
    scale = float(np.float32(scale))
    used = np.zeros(len(got), bool)
    for b, (nq, nk) in enumerate(zip(c["q_lens"], c["kv_lens"])):
        if only is None or b in only:
            q, k = slice(q0, q0 + nq), slice(k0, k0 + nk)
            out, lse, mag, size = op.attend(qn[q], qp[q], kn[k], kp[k], v[k], scale, causal)
            tol, lse_tol = attend_tol(out, lse, mag, size, nk)
            assert_within(got[q], out, tol, f"out of request {b} ({nq} on {nk})")
            empty = np.isneginf(lse)
            assert np.array_equal(np.isneginf(got_lse[q]), empty)
            assert_within(np.where(empty, 0, got_lse[q]), np.where(empty, 0, lse), lse_tol, f"lse of request {b}")
            assert (got[q][empty] == 0).all()
        used[q0:q0 + nq] = True
        q0, k0 = q0 + nq, k0 + nk
    assert np.isnan(got[~used]).all() and np.isnan(got_lse[~used]).all()


EDGES = [1, 2, 15, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 300]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", EDGES)
def test_prefill_prompt_of_every_edge(mla, n, causal):
    c = prefill_case(np.random.default_rng(n), [n], [n], 3)
    run_prefill(mla, c, causal=causal)
    check_prefill(c, causal=causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,kv_lens,H", [
    ([1], [1], 128), ([1, 17, 64, 200], [1, 17, 64, 200], 5), ([5, 1, 3], [800, 411, 600], 4), ([130, 300], [700, 513], 2),
    ([128, 256, 384], [385, 256, 512], 2), ([0, 7, 0, 9], [5, 7, 0, 300], 3), ([7, 4], [0, 129], 3), ([300, 20], [40, 3], 2),
    ([257, 1], [129, 640], 1), ([1] * 70, list(range(1, 71)), 2), ([3, 129] * 12, [10, 200] * 12, 2), ([33], [1500], 33)])
def test_prefill_ragged(mla, q_lens, kv_lens, H, causal):
    """Contexts before the prompt, prompts longer than their keys (rows that see nothing), empty requests."""
    c = prefill_case(np.random.default_rng(len(q_lens) + H), q_lens, kv_lens, H)
    run_prefill(mla, c, causal=causal)
    check_prefill(c, causal=causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,kv_lens,H", [([1], [3500], 1), ([5, 1, 3], [2000, 1097, 1600], 2), ([1, 1], [129, 1], 3), ([140], [2500], 1),
                                              ([3, 0, 2], [0, 900, 1], 2), ([40, 9], [25, 1100], 1)])
def test_prefill_with_workspace(mla, q_lens, kv_lens, H, causal):
    """Few queries on long contexts: the keys may be spread over the GPU and joined."""
    c = prefill_case(np.random.default_rng(31), q_lens, kv_lens, H, q_start=2, q_behind=3, kv_behind=5)
    ws = mla.make_prefill_workspace()
    ws.fill_(0xFF)
    run_prefill(mla, c, causal=causal, ws=ws)
    check_prefill(c, causal=causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,kv_lens,H", [([3, 100, 128, 129, 257, 40], [3, 350, 128, 129, 400, 20], 65), ([1] * 70, [5] * 70, 5),
                                              ([200, 1, 64], [200, 130, 64], 128), ([90] * 40, [90, 300] * 20, 8)])
def test_prefill_many_items(mla, q_lens, kv_lens, H, causal):
    """Several items a block: heads in pairs (an odd head left over), more requests than a warp holds."""
    c = prefill_case(np.random.default_rng(38), q_lens, kv_lens, H)
    run_prefill(mla, c, causal=causal, ws=mla.make_prefill_workspace())
    check_prefill(c, causal=causal)


def test_prefill_overlapping_offsets_in_the_split_form(mla):
    """Offsets that give every request all rows: more parts than blocks, reported, nothing out of place."""
    c = prefill_case(np.random.default_rng(39), [4] * 30, [1000] * 30, 2)
    ws, st = mla.make_prefill_workspace(), word()
    bad = i32([0, 120] * 15 + [120])
    mla.mla_prefill(c["qn"], c["qp"], c["kn"], c["kp"], c["v"], bad, i32([0, 30000] * 15 + [30000]), 0.07, c["out"], c["lse"], workspace=ws,
                    dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 5
    run_prefill(mla, c, ws=ws)
    check_prefill(c)


@pytest.mark.parametrize("causal", [True, False])
def test_prefill_rows_of_no_request_never_matter(mla, causal):
    """NaN in front of, behind and (as the neighbours' values) beside a request's rows."""
    c = prefill_case(np.random.default_rng(32), [100, 70, 140], [100, 131, 270], 2, q_start=5, kv_start=9, q_behind=77, kv_behind=300)
    for name in ("kn", "kp", "v"):
        c[name][9 + 100:9 + 231] = NAN  # the middle request's own keys: only its own outputs may show it
    c["qn"][105:175] = float("inf")
    run_prefill(mla, c, causal=causal)
    c["kv_lens"], c["q_lens"] = [100, 131, 270], [100, 70, 140]
    check_prefill(c, causal=causal, only=(0, 2))


@pytest.mark.parametrize("q_len", [0, 1])
def test_prefill_thousands_of_short_requests(mla, q_len):
    """A block's items lie many groups of 32 requests apart (q_len 0: but the last request has none)."""
    n = 3000
    q_lens, kv_lens = [q_len] * (n - 1) + [3], [2] * (n - 1) + [70]
    c = prefill_case(np.random.default_rng(42), q_lens, kv_lens, 3)
    run_prefill(mla, c)
    check_prefill(c)


@pytest.mark.parametrize("q_len,kv_len,H,split", [(200, 700, 2, False), (50, 700, 2, False), (50, 700, 2, True), (200, 2600, 2, True)])
def test_prefill_query_that_is_not_finite(mla, q_len, kv_len, H, split):
    """A query of NaN or infinity shows in its own rows of out and lse, and nowhere else."""
    c = prefill_case(np.random.default_rng(41), [q_len], [kv_len], H)
    c["qn"][17], c["qp"][33] = float("inf"), NAN
    run_prefill(mla, c, ws=mla.make_prefill_workspace() if split else None)
    for row in (17, 33):
        assert torch.isnan(c["out"][row]).all() and torch.isnan(c["lse"][row]).all()
    keep = [r for r in range(q_len) if r not in (17, 33)]
    args = [f64(c[n]) for n in ("qn", "qp", "kn", "kp", "v")]
    args[0][17], args[1][33] = 0, 0
    out, lse, mag, size = op.attend(*args, float(np.float32(0.07)), True)
    tol, lse_tol = attend_tol(out, lse, mag, size, kv_len)
    assert_within(f64(c["out"])[keep], out[keep], tol[keep])
    assert_within(f64(c["lse"])[keep], lse[keep], lse_tol[keep])


@pytest.mark.parametrize("q_len,split", [(300, False), (100, False), (100, True)])
def test_prefill_key_that_is_not_finite_is_masked(mla, q_len, split):
    """Causal: queries before such a key do not notice it, those that see it give NaN."""
    c = prefill_case(np.random.default_rng(43), [q_len], [700], 2)
    at = 700 - q_len + 40
    c["kn"][at], c["kp"][at + 2] = NAN, float("inf")
    run_prefill(mla, c, ws=mla.make_prefill_workspace() if split else None)
    args = [f64(c[n]) for n in ("qn", "qp", "kn", "kp", "v")]
    args[2][at], args[3][at + 2] = 0, 0
    out, lse, mag, size = op.attend(*args, float(np.float32(0.07)), True)
    tol, lse_tol = attend_tol(out, lse, mag, size, 700)
    assert_within(f64(c["out"])[:40], out[:40], tol[:40])
    assert_within(f64(c["lse"])[:40], lse[:40], lse_tol[:40])
    assert torch.isnan(c["out"][40:]).all() and torch.isnan(c["lse"][40:]).all()


def test_prefill_sharp_and_flat_scores(mla):
    """Scores of hundreds (one key takes all, maxima that keep rising) and of nearly nothing."""
    rng = np.random.default_rng(33)
    c = prefill_case(rng, [150, 260], [400, 260], 2, by=4.0)
    run_prefill(mla, c, scale=2.0)
    check_prefill(c, scale=2.0)
    c = prefill_case(rng, [150, 260], [400, 260], 2)
    run_prefill(mla, c, scale=1e-6)
    check_prefill(c, scale=1e-6)
    # scores rising along the keys by far more than a weight can hold
    c = prefill_case(rng, [130], [520], 1)
    c["qn"][:] = 1
    c["kn"][:] = (torch.arange(520, device="cuda").float() / 4)[:, None, None].to(torch.bfloat16)
    run_prefill(mla, c, scale=0.25)
    check_prefill(c, scale=0.25)
    c["kn"][:] = -c["kn"]
    run_prefill(mla, c, scale=0.25)
    check_prefill(c, scale=0.25)


def test_prefill_strided_operands_and_no_lse(mla):
    rng = np.random.default_rng(34)
    c = prefill_case(rng, [90, 150], [200, 150], 3)
    run_prefill(mla, c)
    want, H = bits(c["out"]), 3
    q = bf16(rng, 240, H, 192)
    q[..., :128], q[..., 128:] = c["qn"], c["qp"]
    kv = bf16(rng, 350, H, 256)
    kv[..., :128], kv[..., 128:] = c["kn"], c["v"]
    row = bf16(rng, 350, 576)
    row[:, 512:] = c["kp"]
    s = dict(c, qn=q[..., :128], qp=q[..., 128:], kn=kv[..., :128], v=kv[..., 128:], kp=row[:, 512:], out=torch.zeros_like(c["out"]), lse=None)
    run_prefill(mla, s)
    assert np.array_equal(bits(s["out"]), want)
    # heads outermost
    s = dict(s, kn=c["kn"].transpose(0, 1).contiguous().transpose(0, 1), qp=c["qp"].transpose(0, 1).contiguous().transpose(0, 1))
    s["out"].zero_()
    run_prefill(mla, s)
    assert np.array_equal(bits(s["out"]), want)


def test_prefill_repeats_bit_for_bit(mla):
    c = prefill_case(np.random.default_rng(35), [700, 33, 1000], [1500, 900, 1000], 4)
    ws = mla.make_prefill_workspace()
    first = None
    for _ in range(20):
        run_prefill(mla, c, ws=ws)
        got = (bits(c["out"]), bits(c["lse"]))
        if first is None:
            first = got
            check_prefill(c)
        else:
            assert np.array_equal(got[0], first[0]) and np.array_equal(got[1], first[1])


def test_prefill_rows_more_than_32_bits_apart(mla):
    """Keys at a token stride that takes element offsets past 2^31."""
    rng = np.random.default_rng(36)
    c = prefill_case(rng, [40], [1100], 1)
    run_prefill(mla, c)
    want = bits(c["out"])
    stride = (1 << 31) // 1024
    far = torch.zeros(stride * 1100, dtype=torch.bfloat16, device="cuda").view(1100, 1, stride)
    far[..., :128], far[..., 128:256] = c["kn"], c["v"]
    far[:, 0, 256:320] = c["kp"]
    s = dict(c, kn=far[..., :128], v=far[..., 128:256], kp=far[:, 0, 256:320])
    s["out"].zero_()
    run_prefill(mla, s)
    assert np.array_equal(bits(s["out"]), want)


@pytest.mark.parametrize("qo,ko", [([0, 30, 20], [0, 20, 40]), ([0, 20, 31], [0, 20, 40]), ([0, 10, 30], [0, 41, 40]), ([0, 10, 30], [0, 20, 41]),
                                   ([-1, 10, 30], [0, 20, 40]), ([0, 10, 30], [-7, 20, 40]), ([0, 10, 2 ** 31 - 1], [0, 2 ** 31 - 1, -2 ** 31])])
def test_prefill_reports_bad_offsets(mla, qo, ko):
    """Offsets that fall or leave the rows: reported, nothing out of place, the context stays usable."""
    c = prefill_case(np.random.default_rng(37), [10, 20], [20, 20], 2)
    st = word()
    mla.mla_prefill(c["qn"], c["qp"], c["kn"], c["kp"], c["v"], i32(qo), i32(ko), 0.07, c["out"], c["lse"], dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 5
    run_prefill(mla, c)
    check_prefill(c)


# ------------------------------------------------------------------- together

def test_streams_and_graphs(mla):
    """The three calls on a side stream, captured and replayed on other inputs."""
    rng = np.random.default_rng(41)
    e = expand_case(rng, [200, 77], 4, 16)
    p = prefill_case(rng, [60, 77], [200, 77], 4)
    p.update(kn=e["k"], v=e["v"], kp=e["pe"])
    a = append_case(rng, 277, 4)
    slots = torch.from_numpy(np.concatenate([[mi.slot_of(e["table"].cpu().numpy(), b, t, 16) for t in range(n)] for b, n in enumerate([200, 77])])).cuda()
    ws, st = mla.make_prefill_workspace(), word()
    new, absorbed = e["cache"], torch.zeros_like(a["q"])

    def step(stream):
        mla.mla_rope_append(a["kv"], a["positions"], a["table"], slots, new, norm_weight=a["weight"], q_pe=a["q"], q_pe_out=absorbed, dev_status=st,
                            stream=stream)
        mla.mla_expand_kv(new, e["table"], e["offsets"], e["w_uk"], e["w_uv"], e["k"], e["v"], e["pe"], dev_status=st, stream=stream)
        mla.mla_prefill(p["qn"], p["qp"], e["k"], e["pe"], e["v"], p["qo"], p["ko"], 0.07, p["out"], p["lse"], workspace=ws, dev_status=st,
                        stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    eager = bits(p["out"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(torch.cuda.current_stream())
    p["out"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(bits(p["out"]), eager) and int(st) == 0
    a["kv"].copy_(bf16(rng, 277, 576))
    p["qn"].copy_(bf16(rng, *p["qn"].shape))
    graph.replay()
    torch.cuda.synchronize()
    check_prefill(p)
    rows = append_ref(a, True)[0]
    assert_within(f64(new).reshape(-1, 576)[slots.cpu().numpy()], rows, BF16 * np.abs(rows) + 1e-4)


def test_prompt_then_decode(mla):
    """A prompt taken in by append, expand and prefill, then its last token decoded again in
    the absorbed form over the same cache and weights: one attention, two forms."""
    rng = np.random.default_rng(42)
    H, page, lens, new = 128, 16, [130, 37], [50, 37]
    blocks = 16
    table = mi.make_block_table(rng, lens, page, blocks)
    cache = torch.full((blocks, page, 576), NAN, dtype=torch.bfloat16, device="cuda")
    w_uk, w_uv, weight = bf16(rng, H, 128, 512, by=0.05), bf16(rng, H, 512, 128, by=0.05), bf16(rng, 512)
    cos_sin = rope_table(256)
    # each context arrives in two chunks (the first request's), the second one's queries are attended
    kv = bf16(rng, sum(lens), 576)
    q = bf16(rng, sum(new), H, 192)
    q_pe = torch.empty(sum(new), H, 64, dtype=torch.bfloat16, device="cuda")
    slot = [[mi.slot_of(table, b, t, page) for t in range(n)] for b, n in enumerate(lens)]
    pos = [np.arange(n) for n in lens]
    dev = lambda x: torch.from_numpy(np.asarray(x)).cuda()
    mla.mla_rope_append(kv[:80], dev(pos[0][:80]), cos_sin, dev(slot[0][:80]), cache, norm_weight=weight)
    mla.mla_rope_append(kv[80:], dev(np.concatenate([pos[0][80:], pos[1]])), cos_sin, dev(slot[0][80:] + slot[1]), cache, norm_weight=weight,
                        q_pe=q[..., 128:], q_pe_out=q_pe)
    Tk = sum(lens)
    k, v = (torch.empty(Tk, H, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k_pe, st = torch.empty(Tk, 64, dtype=torch.bfloat16, device="cuda"), word()
    mla.mla_expand_kv(cache, i32(table), offsets(lens), w_uk, w_uv, k, v, k_pe, dev_status=st)
    out, lse = torch.empty(sum(new), H, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(sum(new), H, device="cuda")
    mla.mla_prefill(q[..., :128], q_pe, k, k_pe, v, offsets(new), offsets(lens), mi.SOFTMAX_SCALE, out, lse, dev_status=st)
    assert int(st) == 0
    last = torch.tensor([new[0] - 1, sum(new) - 1], device="cuda")
    q_abs = torch.empty(2, H, 576, dtype=torch.bfloat16, device="cuda")
    mla.mla_absorb_q(q[last][..., :128].contiguous(), q_pe[last], w_uk, q_abs)
    latent, lse2 = torch.empty(2, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(2, H, device="cuda")
    mla.mla_decode(q_abs, cache, i32(table), i32(lens), mi.SOFTMAX_SCALE, latent, lse2)
    o = torch.empty(2, H, 128, dtype=torch.bfloat16, device="cuda")
    mla.mla_absorb_out(latent, w_uv, o)
    # both forms round q or k, the weights, and the result to bf16: 2e-2 of the largest value covers
    # those few half steps of 2^-8 each
    a, b = f64(out[last]), f64(o)
    assert np.abs(a - b).max() <= 2e-2 * np.abs(b).max()
    # scores of 192 (576) rounded products: their sum's error is that of the bf16 keys (queries),
    # 2^-8 of |q k| summed in quadrature over the dims, far below 0.05 here
    assert np.abs(f64(lse[last]) - f64(lse2)).max() <= 0.05
