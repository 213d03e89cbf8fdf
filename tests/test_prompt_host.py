"""The prompt-side entry points without a GPU: refusals before any launch, and
pins of their fp64 oracle."""
import ctypes

import numpy as np
import pytest

import oracle.nonabsorbed as na
import oracle.prompt as op


@pytest.fixture(scope="module")
def lib():
    from mla_latent_cache_decode_gb300 import build
    lib = ctypes.CDLL(build.build())
    import mla_latent_cache_decode_gb300 as mla
    for name in ("mla_rope_append", "mla_rope_append_fp8", "mla_expand_kv", "mla_expand_kv_fp8", "mla_prefill",
                 "mla_prefill_workspace_size", "mla_last_error_detail"):
        getattr(lib, name).argtypes = getattr(mla.get_lib(), name).argtypes
        getattr(lib, name).restype = getattr(mla.get_lib(), name).restype
    return lib


A = 1 << 20  # an aligned address that no test lets a kernel touch


def append(lib, fp8=False, **kw):
    a = dict(kv=A, kv_stride=576, positions=A, cos_sin=A, max_position=8, slots=A, tokens=2, weight=None, eps=1e-6, interleaved=1, cache=A,
             num_blocks=4, block_size=16, scale=1.0, q=A, qt=128 * 64, qh=64, qo=2 * A, qot=128 * 64, qoh=64, heads=128)
    a.update(kw)
    args = [a[k] for k in ("kv", "kv_stride", "positions", "cos_sin", "max_position", "slots", "tokens", "weight", "eps", "interleaved",
                           "cache", "num_blocks", "block_size")]
    args += [a["scale"]] if fp8 else []
    args += [a[k] for k in ("q", "qt", "qh", "qo", "qot", "qoh", "heads")] + [None, None]
    return (lib.mla_rope_append_fp8 if fp8 else lib.mla_rope_append)(*args)


@pytest.mark.parametrize("bad, status", [
    (dict(tokens=-1), 1), (dict(tokens=1 << 27), 1), (dict(block_size=0), 1), (dict(num_blocks=0), 1), (dict(max_position=0), 1),
    (dict(interleaved=2), 1), (dict(weight=A, eps=float("nan")), 1), (dict(weight=A, eps=-1.0), 1), (dict(q=None), 1), (dict(qo=None), 1),
    (dict(heads=0), 2), (dict(heads=129), 2), (dict(kv=None), 1), (dict(positions=None), 1), (dict(cos_sin=None), 1), (dict(slots=None), 1),
    (dict(cache=None), 1), (dict(kv=A + 8), 1), (dict(cos_sin=A + 4), 1), (dict(cache=A + 8), 1), (dict(weight=A + 2), 1), (dict(q=A + 2), 1),
    (dict(qo=A + 8), 1), (dict(positions=A + 4), 1), (dict(slots=A + 4), 1), (dict(kv_stride=568), 1), (dict(kv_stride=580), 1),
    (dict(qt=100), 1), (dict(qh=-64), 1), (dict(qoh=32), 1), (dict(qot=64), 1), (dict(qot=8128), 1)])
def test_append_refusals(lib, bad, status):
    assert append(lib, **bad) == status
    assert lib.mla_last_error_detail() != b""
    assert append(lib, True, **bad) == status


def test_append_no_ops_and_scales(lib):
    assert append(lib, tokens=0, kv=None, cache=None) == 0
    for scale in (0.0, -1.0, float("inf"), float("nan"), 1e-45):
        assert append(lib, True, scale=scale, tokens=0) == 1
        assert b"kv_scale" in lib.mla_last_error_detail()
    assert append(lib, True, scale=0.5, tokens=0) == 0


def expand(lib, fp8=False, **kw):
    a = dict(cache=A, num_blocks=4, block_size=16, table=A, width=2, offsets=A, batch=2, total=20, w_uk=A, w_uv=A, heads=16, scale=1.0,
             k=A, v=A, pe=A)
    a.update(kw)
    args = [a[k] for k in ("cache", "num_blocks", "block_size", "table", "width", "offsets", "batch", "total", "w_uk", "w_uv", "heads")]
    args += [a["scale"]] if fp8 else []
    return (lib.mla_expand_kv_fp8 if fp8 else lib.mla_expand_kv)(*args, a["k"], a["v"], a["pe"], None, None)


@pytest.mark.parametrize("bad, status", [
    (dict(batch=-1), 1), (dict(total=-1), 1), (dict(total=1 << 30), 1), (dict(block_size=0), 1), (dict(num_blocks=0), 1), (dict(width=0), 1),
    (dict(heads=0), 2), (dict(heads=129), 2), (dict(cache=None), 1), (dict(table=None), 1), (dict(offsets=None), 1), (dict(w_uk=None), 1),
    (dict(w_uv=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(pe=None), 1), (dict(cache=A + 8), 1), (dict(w_uk=A + 2), 1),
    (dict(k=A + 8), 1), (dict(table=A + 2), 1), (dict(offsets=A + 1), 1)])
def test_expand_refusals(lib, bad, status):
    assert expand(lib, **bad) == status
    assert lib.mla_last_error_detail() != b""
    assert expand(lib, True, **bad) == status


def test_expand_no_ops_and_scales(lib):
    assert expand(lib, batch=0, table=None) == 0
    assert expand(lib, total=0, k=None, v=None, pe=None) == 0
    assert expand(lib, True, total=0, scale=0.0) == 1
    assert expand(lib, True, total=0, scale=float("inf")) == 1


def prefill(lib, **kw):
    a = dict(qn=A, qnt=16 * 192, qnh=192, qp=A, qpt=16 * 64, qph=64, kn=A, knt=16 * 128, knh=128, kp=A, kpt=64, v=A, vt=16 * 128, vh=128,
             qo=A, ko=A, batch=2, tq=20, tk=30, heads=16, causal=1, scale=0.1, out=A, lse=A, ws=None, wsb=0)
    a.update(kw)
    return lib.mla_prefill(*[a[k] for k in ("qn", "qnt", "qnh", "qp", "qpt", "qph", "kn", "knt", "knh", "kp", "kpt", "v", "vt", "vh", "qo",
                                            "ko", "batch", "tq", "tk", "heads", "causal", "scale", "out", "lse", "ws", "wsb")], None, None)


@pytest.mark.parametrize("bad, status", [
    (dict(batch=-1), 1), (dict(tq=-1), 1), (dict(tk=-1), 1), (dict(tq=1 << 30), 1), (dict(tk=(1 << 26) + 1), 1), (dict(heads=0), 2),
    (dict(heads=129), 2), (dict(causal=2), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(scale=-1.0), 1), (dict(qn=None), 1), (dict(qp=None), 1), (dict(kn=None), 1), (dict(kp=None), 1), (dict(v=None), 1),
    (dict(qo=None), 1), (dict(ko=None), 1), (dict(out=None), 1), (dict(qn=A + 2), 1), (dict(kp=A + 8), 1), (dict(out=A + 8), 1),
    (dict(qo=A + 2), 1), (dict(lse=A + 1), 1), (dict(qnt=100), 1), (dict(qnh=120), 1), (dict(vh=0), 1), (dict(kpt=56), 1),
    (dict(knt=1 << 38), 1), (dict(ws=A + 16, wsb=1 << 30), 1), (dict(ws=A, wsb=1024), 3)])
def test_prefill_refusals(lib, bad, status):
    assert prefill(lib, **bad) == status
    assert lib.mla_last_error_detail() != b""


def test_prefill_no_ops_and_workspace(lib):
    assert prefill(lib, batch=0, qo=None, ko=None) == 0
    assert prefill(lib, tq=0, qn=None, qp=None, out=None) == 0
    assert 0 < lib.mla_prefill_workspace_size() <= 32 << 20


def test_bindings_refuse_what_the_abi_cannot_see():
    torch = pytest.importorskip("torch")
    import mla_latent_cache_decode_gb300 as mla
    x = torch.zeros(2, 576, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # not on a GPU
        mla.mla_rope_append(x, torch.zeros(2, dtype=torch.int64), torch.zeros(4, 64), torch.zeros(2, dtype=torch.int64),
                            torch.zeros(2, 16, 576, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        mla.mla_prefill(None, None, None, None, None, None, None, 1.0, None)
    t = torch.zeros(3, 1, 7, 128)
    assert mla._strides(t[:, 0], 128) == [7 * 128, 128]
    assert mla._strides(torch.zeros(1, 5, 192)[:, :1, :128], 128) == [128, 128]
    assert mla._strides(torch.zeros(4, 192)[:, 128:], 64) == [192]


# ------------------------------------------------------------------- the oracle

def test_oracle_rotation_is_a_rotation():
    rng = np.random.default_rng(1)
    x, angle = rng.standard_normal((5, 64)), rng.standard_normal((5, 32))
    for interleaved in (True, False):
        y = op.rotate(x, np.cos(angle), np.sin(angle), interleaved)
        assert np.allclose((y ** 2).sum(1), (x ** 2).sum(1))
        assert np.allclose(op.rotate(y, np.cos(angle), -np.sin(angle), interleaved), x)
    # pair 0 of a quarter turn: (a, b) -> (-b, a)
    z = op.rotate(x, np.zeros((5, 32)), np.ones((5, 32)), True)
    assert np.allclose(z[:, 0], -x[:, 1]) and np.allclose(z[:, 1], x[:, 0])
    z = op.rotate(x, np.zeros((5, 32)), np.ones((5, 32)), False)
    assert np.allclose(z[:, 0], -x[:, 32]) and np.allclose(z[:, 32], x[:, 0])


def test_oracle_rotated_scores_depend_on_distance_only():
    rng = np.random.default_rng(2)
    q, k, freq = rng.standard_normal(64), rng.standard_normal(64), 10000.0 ** (-np.arange(32) / 32)
    for interleaved in (True, False):
        s = [op.rotate(q, np.cos(n * freq), np.sin(n * freq), interleaved) @ op.rotate(k, np.cos((n - 7) * freq), np.sin((n - 7) * freq), interleaved)
             for n in (7, 100, 5000)]
        assert np.allclose(s, s[0])


def test_oracle_expanded_attention_is_the_non_absorbed_one():
    """expand + attend of a context's last token = explicit 192-dim attention."""
    rng = np.random.default_rng(3)
    H, L = 3, 40
    rows = rng.standard_normal((L, 576))
    w_uk, w_uv = rng.standard_normal((H, 128, 512)) / 20, rng.standard_normal((H, 512, 128)) / 20
    qn, qp = rng.standard_normal((5, H, 128)), rng.standard_normal((5, H, 64))
    k, v = op.expand(rows, w_uk, w_uv)
    out, lse, _, _ = op.attend(qn, qp, k, rows[:, 512:], v, 0.07, True)
    for i in range(5):
        want = na.mha_nonabsorbed(qn[i], qp[i], w_uk, w_uv.transpose(0, 2, 1), rows[:L - 4 + i], 0.07)
        assert np.allclose(out[i], want)


def test_oracle_rows_that_see_nothing():
    rng = np.random.default_rng(4)
    g = lambda *s: rng.standard_normal(s)
    out, lse, _, _ = op.attend(g(5, 2, 128), g(5, 2, 64), g(3, 2, 128), g(3, 64), g(3, 2, 128), 1.0, True)
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.isfinite(lse[2:]).all()
    assert np.isfinite(op.attend(g(5, 2, 128), g(5, 2, 64), g(3, 2, 128), g(3, 64), g(3, 2, 128), 1.0, False)[1]).all()
    out, lse, _, _ = op.attend(g(5, 2, 128), g(5, 2, 64), g(0, 2, 128), g(0, 64), g(0, 2, 128), 1.0, False)
    assert (out == 0).all() and np.isneginf(lse).all()
