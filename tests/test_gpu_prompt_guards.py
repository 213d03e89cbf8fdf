"""What the prompt side's kernels leave alone when offsets, pages, positions or
slots lie outside: every tensor that they write stands between rows of a known
pattern, which has to be the same bits after the call."""
import numpy as np
import pytest

import oracle.prompt as op
from prompt_helpers import assert_within, expand_tol, f64
from test_gpu_prompt import append_case, check_prefill, expand_case, i32, mla, prefill_case, run_prefill, word  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

MARGIN = 256  # rows in front and behind


class Guarded:
    """Tensors of the given first dims between MARGIN rows of 0xA5 bytes on either side."""

    def __init__(self):
        self.all = []

    def like(self, t):
        rows = t.shape[0]
        whole = torch.empty((rows + 2 * MARGIN, *t.shape[1:]), dtype=t.dtype, device="cuda")
        whole.view(torch.uint8).fill_(0xA5)
        whole[MARGIN:MARGIN + rows] = t
        self.all.append((whole, rows))
        return whole[MARGIN:MARGIN + rows]

    def check(self):
        torch.cuda.synchronize()
        for whole, rows in self.all:
            raw = whole.view(torch.uint8)
            assert (raw[:MARGIN] == 0xA5).all() and (raw[MARGIN + rows:] == 0xA5).all(), "written outside the tensor"


BAD = [([0, 30, 20], [0, 20, 40]), ([0, 20, 31], [0, 20, 40]), ([0, 10, 30], [0, 41, 40]), ([0, 10, 30], [0, 20, 41]),
       ([-1, 10, 30], [0, 20, 40]), ([0, 10, 30], [-7, 20, 40]), ([0, 10, 2 ** 31 - 1], [0, 2 ** 31 - 1, -2 ** 31]),
       ([-2 ** 31, 2 ** 31 - 1, 2 ** 31 - 1], [-2 ** 31, 2 ** 31 - 1, 2 ** 31 - 1]), ([0, 1000, 1000], [0, 1000, 1000])]


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("H", [2, 128])
@pytest.mark.parametrize("qo,ko", BAD)
def test_prefill_bad_offsets_write_nothing_outside(mla, qo, ko, H, split):
    c = prefill_case(np.random.default_rng(61), [10, 20], [20, 20], H)
    g = Guarded()
    c["out"], c["lse"] = g.like(c["out"]), g.like(c["lse"])
    ws = g.like(torch.zeros(mla.make_prefill_workspace().numel() // 1024, 1024, dtype=torch.uint8, device="cuda")).view(-1) if split else None
    for causal in (True, False):
        st = word()
        mla.mla_prefill(c["qn"], c["qp"], c["kn"], c["kp"], c["v"], i32(qo), i32(ko), 0.07, c["out"], c["lse"], causal=causal, workspace=ws,
                        dev_status=st)
        g.check()
        assert int(st) == 5
    run_prefill(mla, c, ws=ws)
    g.check()
    check_prefill(c)


@pytest.mark.parametrize("split", [False, True])
def test_prefill_bad_request_beside_good_ones(mla, split):
    """The first request's offsets are fine: its rows come out whole, whatever the others' say."""
    c = prefill_case(np.random.default_rng(62), [33, 20], [700, 20], 2)
    g = Guarded()
    c["out"], c["lse"] = g.like(c["out"]), g.like(c["lse"])
    ws, st = mla.make_prefill_workspace() if split else None, word()
    mla.mla_prefill(c["qn"], c["qp"], c["kn"], c["kp"], c["v"], i32([0, 33, 900]), i32([0, 700, 2 ** 31 - 1]), 0.07, c["out"], c["lse"],
                    workspace=ws, dev_status=st)
    g.check()
    assert int(st) == 5
    check_prefill(dict(c, lse=c["lse"]), only=(0,))


@pytest.mark.parametrize("split", [False, True])
def test_prefill_overlapping_offsets_write_nothing_outside(mla, split):
    """Offsets that give every other request all rows: more work than the call was sized for."""
    c = prefill_case(np.random.default_rng(63), [4] * 30, [1000] * 30, 2)
    g = Guarded()
    c["out"], c["lse"] = g.like(c["out"]), g.like(c["lse"])
    ws = g.like(torch.zeros(mla.make_prefill_workspace().numel() // 1024, 1024, dtype=torch.uint8, device="cuda")).view(-1) if split else None
    st = word()
    mla.mla_prefill(c["qn"], c["qp"], c["kn"], c["kp"], c["v"], i32([0, 120] * 15 + [120]), i32([0, 30000] * 15 + [30000]), 0.07, c["out"],
                    c["lse"], workspace=ws, dev_status=st)
    g.check()
    assert int(st) == 5


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("offs", [[0, 40, 1000], [0, 40, 2 ** 31 - 1], [0, 40, 20], [0, 40, -2 ** 31], [-3, 40, 60], [-2 ** 31, 40, 60],
                                  [0, 1000, 60], [500, 600, 700]])
def test_expand_bad_offsets_write_nothing_outside(mla, offs, fp8):
    c = expand_case(np.random.default_rng(64), [40, 20], 3, 16, fp8)
    g = Guarded()
    for name in ("k", "v", "pe"):
        c[name] = g.like(c[name])
    c["offsets"] = i32(offs)
    st, scale = word(), 0.37
    args = [c[n] for n in ("cache", "table", "offsets", "w_uk", "w_uv", "k", "v", "pe")]
    if fp8:
        mla.mla_expand_kv_fp8(*args, kv_scale=scale, dev_status=st)
    else:
        mla.mla_expand_kv(*args, dev_status=st)
    g.check()
    assert int(st) == 5
    if offs[:2] == [0, 40] and offs[2] >= 40:  # the first request's rows are right
        rows = c["rows"][:40] * (np.float64(np.float32(scale)) if fp8 else 1.0)
        k, v = op.expand(rows, f64(c["w_uk"]), f64(c["w_uv"]))
        k_tol, v_tol = expand_tol(rows, f64(c["w_uk"]), f64(c["w_uv"]), k, v)
        assert_within(f64(c["k"])[:40], k, k_tol)
        assert_within(f64(c["v"])[:40], v, v_tol)


@pytest.mark.parametrize("fp8", [False, True])
def test_append_writes_nothing_outside(mla, fp8):
    c = append_case(np.random.default_rng(65), 8, 5, positions=50)
    c["positions"] = torch.tensor([3, 50, -1, 4, 2 ** 62, -2 ** 63, 7, 8], device="cuda")
    slots = torch.tensor([0, 1, 2, 32, 4, 5, 2 ** 62, -2 ** 63], device="cuda")
    g = Guarded()
    cache = g.like(torch.zeros(2, 16, 576, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda"))
    out, st = g.like(torch.zeros_like(c["q"])), word()
    fn = mla.mla_rope_append_fp8 if fp8 else mla.mla_rope_append
    fn(c["kv"], c["positions"], c["table"], slots, cache, norm_weight=c["weight"], q_pe=c["q"], q_pe_out=out, dev_status=st)
    g.check()
    assert int(st) == 5
    wrote = (cache.view(-1, 576) != 0).any(1).cpu().numpy()
    assert wrote[0] and not wrote[1:].any()
    assert [bool((out[t] != 0).any()) for t in range(8)] == [True, False, False, True, False, False, True, True]
