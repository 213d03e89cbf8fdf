"""What the calls for a full cache refuse or promise at their limits, without a GPU."""
import pytest

from test_eviction_host import A, lib, select  # noqa: F401


@pytest.mark.parametrize("batch,budget", [(2, 10), (1, 1)])
@pytest.mark.parametrize("what", ["keep", "new"])
def test_select_refuses_to_write_over_the_lengths(lib, what, batch, budget):  # noqa: F811
    """Blocks read a request's length each for itself, so neither output may lie over the lengths: not
    at the same address, nor by their last or first entry."""
    size = 4 * batch * (budget if what == "keep" else 1)
    other = {"keep": "new", "new": "keep"}[what]
    # (a stride below the tokens is refused too: what does not overlap gets as far as that, and no further)
    a = dict(batch=batch, budget=budget, sink=0, recent=0, lens=A, stride=99, **{other: A + (1 << 16)})
    if batch == 1:
        a["mass"] = None
    for at in (A, A + 4 * batch - 4, A - size + 4):
        assert select(lib, **dict(a, mass=A), **{what: at}) == 1
        assert b"overlap" in lib.mla_last_error_detail()
    for at in (A + 4 * batch, A - size):
        assert select(lib, **a, **{what: at}) == 1
        assert b"overlap" not in lib.mla_last_error_detail()
