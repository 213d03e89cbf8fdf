"""Decode over a shared prefix and cache eviction on the GPU: operands that are not
finite, pieces of many tiles, and what rounding may cost.  (Tolerances:
eviction_helpers; a head with a log-sum-exp of -inf has no part in them.)"""
import numpy as np
import pytest

from eviction_helpers import check_mass, check_shared, mass_case, run_mass, run_shared, shared_case

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def mla():
    import mla_latent_cache_decode_gb300 as mla
    torch.cuda.set_device(0)
    return mla


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
