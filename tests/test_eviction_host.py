"""Decode over a shared prefix and cache eviction without a GPU: refusals before any
launch, and pins of their fp64 oracle."""
import ctypes

import numpy as np
import pytest

import oracle.eviction as oe

A = 1 << 20  # an aligned address that no test lets a kernel touch


@pytest.fixture(scope="module")
def lib():
    from mla_latent_cache_decode_gb300 import build
    lib = ctypes.CDLL(build.build())
    import mla_latent_cache_decode_gb300 as mla
    for name in ("mla_decode_shared", "mla_attention_mass", "mla_attention_mass_fp8", "mla_evict_select", "mla_cache_compact",
                 "mla_cache_compact_fp8", "mla_decode_shared_workspace_size", "mla_last_error_detail"):
        getattr(lib, name).argtypes = getattr(mla.get_lib(), name).argtypes
        getattr(lib, name).restype = getattr(mla.get_lib(), name).restype
    return lib


def shared(lib, **kw):
    a = dict(q=A, cache=A, num_blocks=9, block_size=64, shared_table=A, shared_blocks=A, max_shared=4, table=A, width=4, lens=A, batch=2,
             heads=16, scale=0.1, out=A, lse=A, ws=A, ws_bytes=0)
    a.update(kw)
    return lib.mla_decode_shared(*a.values(), None, None)


@pytest.mark.parametrize("bad, status", [
    (dict(batch=-1), 1), (dict(batch=(1 << 20) + 1), 1), (dict(heads=0), 2), (dict(heads=129), 2), (dict(block_size=0), 1),
    (dict(block_size=48), 2), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(num_blocks=0), 1), (dict(num_blocks=1 << 31), 1),
    (dict(width=0), 1), (dict(width=1 << 25), 1), (dict(max_shared=-1), 1), (dict(max_shared=1 << 25), 1), (dict(q=None), 1),
    (dict(cache=None), 1), (dict(shared_table=None), 1), (dict(shared_blocks=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(out=None), 1), (dict(ws=None), 1), (dict(q=A + 8), 1), (dict(cache=A + 2), 1), (dict(out=A + 8), 1), (dict(lse=A + 2), 1),
    (dict(table=A + 2), 1), (dict(shared_table=A + 1), 1), (dict(shared_blocks=A + 2), 1), (dict(lens=A + 2), 1), (dict(ws=A + 16), 1)])
def test_shared_refusals(lib, bad, status):
    assert shared(lib, **bad) == status
    assert lib.mla_last_error_detail() != b""


def test_shared_no_op(lib):
    assert shared(lib, batch=0, q=None, table=None, ws=None) == 0
    for batch, heads in ((-1, 16), (4, 0), (4, 129)):
        assert lib.mla_decode_shared_workspace_size(batch, heads) == 0


def mass(lib, fp8=False, **kw):
    a = dict(q=A, cache=A, num_blocks=9, block_size=64, table=A, width=4, lens=A, batch=2, heads=16, scale=0.1, kv=1.0, lse=A, previous=A,
             previous_stride=256, decay=1.0, mass=A, stride=256, tokens=256)
    a.update(kw)
    if not fp8:
        a.pop("kv")
    return (lib.mla_attention_mass_fp8 if fp8 else lib.mla_attention_mass)(*a.values(), None, None)


@pytest.mark.parametrize("bad, status", [
    (dict(batch=-1), 1), (dict(batch=1 << 24), 1), (dict(heads=0), 2), (dict(heads=129), 2), (dict(block_size=0), 1), (dict(block_size=48), 2),
    (dict(scale=-1.0), 1), (dict(scale=float("inf")), 1), (dict(num_blocks=0), 1), (dict(width=0), 1), (dict(width=1 << 25), 1),
    (dict(decay=-0.5), 1), (dict(decay=float("nan")), 1), (dict(tokens=-1), 1), (dict(stride=255), 1), (dict(previous_stride=255), 1),
    (dict(q=None), 1), (dict(cache=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(lse=None), 1), (dict(mass=None), 1),
    (dict(q=A + 8), 1), (dict(cache=A + 8), 1), (dict(lse=A + 2), 1), (dict(mass=A + 2), 1), (dict(previous=A + 1), 1)])
def test_mass_refusals(lib, bad, status):
    assert mass(lib, **bad) == status
    assert lib.mla_last_error_detail() != b""
    assert mass(lib, True, **bad) == status


def test_mass_no_ops_and_scales(lib):
    assert mass(lib, batch=0, q=None) == 0
    assert mass(lib, tokens=0, mass=None) == 0
    for kv in (0.0, -1.0, float("nan"), float("inf"), 1e-45):
        assert mass(lib, True, kv=kv, batch=0, scale=1e-3) == 1


def select(lib, **kw):
    a = dict(mass=A, stride=100, tokens=100, lens=A, batch=2, sink=1, recent=2, keep=A, budget=10, new=A)
    a.update(kw)
    return lib.mla_evict_select(*a.values(), None, None)


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(sink=-1), dict(recent=-1), dict(budget=0), dict(budget=2),
    dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), dict(mass=None), dict(lens=None), dict(keep=None), dict(new=None), dict(mass=A + 2),
    dict(lens=A + 2), dict(keep=A + 2), dict(new=A + 1), dict(stride=99)])
def test_select_refusals(lib, bad):
    assert select(lib, **bad) == 1
    assert lib.mla_last_error_detail() != b""


def test_select_no_op(lib):
    assert select(lib, batch=0, mass=None, keep=None) == 0


def compact(lib, fp8=False, **kw):
    a = dict(cache=A, layers=2, num_blocks=9, block_size=16, table=A, width=4, batch=2, keep=A, budget=10, lens=A, new=A, mass=A, stride=64,
             tokens=64)
    a.update(kw)
    return (lib.mla_cache_compact_fp8 if fp8 else lib.mla_cache_compact)(*a.values(), None, None)


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(budget=-1), dict(layers=-1), dict(layers=1 << 31), dict(num_blocks=0), dict(num_blocks=1 << 31), dict(block_size=0),
    dict(width=0), dict(width=1 << 27), dict(cache=None), dict(table=None), dict(keep=None), dict(lens=None), dict(new=None),
    dict(cache=A + 8), dict(table=A + 2), dict(keep=A + 2), dict(lens=A + 2), dict(new=A + 2), dict(mass=A + 2), dict(stride=63),
    dict(tokens=-1)])
def test_compact_refusals(lib, bad):
    for fp8 in (False, True):
        assert compact(lib, fp8, **bad) == 1
        assert lib.mla_last_error_detail() != b""


def test_compact_no_ops(lib):
    assert compact(lib, batch=0, cache=None, table=None) == 0
    assert compact(lib, layers=0, mass=None) == 0


# ------------------------------------------------------------------------- the oracle

def test_select_by_hand():
    w = np.array([5.0, 1, 4, 4, np.nan, 4, 0, 9])
    assert oe.select(w, 8, 8, 0, 0) == list(range(8))
    assert oe.select(w, 8, 3, 0, 0) == [0, 2, 7]
    assert oe.select(w, 8, 4, 1, 1) == [0, 2, 3, 7]
    assert oe.select(w, 8, 4, 0, 2) == [0, 2, 6, 7]
    assert oe.select(w, 8, 7, 0, 0) == [0, 1, 2, 3, 5, 6, 7]
    assert oe.select(w, 3, 5, 1, 1) == [0, 1, 2]


def test_compact_by_hand():
    cache = np.arange(6.0).reshape(1, 3, 2)  # blocks 0..2 of two rows
    out, w = oe.compact(cache, [[2, 0]], [[1, 3]], [4], np.array([[10.0, 11, 12, 13, 14]]))
    assert out.tolist() == [[[0, 1], [2, 3], [5, 1]]]
    assert w.tolist() == [[11, 13, 0, 0, 14]]


def test_weights_add_up_and_decode_splits():
    """The weights are those that decode averages the rows with, and a prefix is no different."""
    rng = np.random.default_rng(1)
    q, cache = rng.standard_normal((3, 576)), rng.standard_normal((9, 16, 576))
    table = [[0, 0, 4, 7, 2]]
    rows = oe.rows_of(cache, table, 0, 70, [5, 1])
    assert np.array_equal(rows[16:48], np.concatenate([cache[1], cache[4]]))
    out, lse = oe.decode(q, rows, 0.07)
    one = oe.decode(q[:1], rows, 0.07)
    w = oe.mass(q[:1], rows, 0.07, one[1])
    assert abs(w.sum() - 1) < 1e-12 and np.allclose(w @ rows[:, :512], one[0][0], atol=1e-12)
    assert np.allclose(oe.mass(q, rows, 0.07, lse), sum(oe.mass(q[h:h + 1], rows, 0.07, lse[h:h + 1]) for h in range(3)))


# ------------------------------------------------------------------------- sizes whose products wrap

@pytest.mark.parametrize("call", [shared, mass, lambda lib, **kw: mass(lib, True, **kw), compact, lambda lib, **kw: compact(lib, True, **kw)])
def test_pools_beyond_64_bits_are_refused(lib, call):
    assert call(lib, block_size=64, num_blocks=(1 << 58) + 1) == 1  # 64 rows more than 2^64
    assert lib.mla_last_error_detail() != b""


def test_moves_beyond_64_bits_are_refused(lib):
    assert compact(lib, batch=1 << 30, layers=(1 << 31) - 1) == 1
    assert b"num_layers" in lib.mla_last_error_detail()
    assert compact(lib, width=(1 << 26) + 1) == 1
    assert compact(lib, width=1 << 26, layers=0, mass=None) == 0  # 2^30 tokens
