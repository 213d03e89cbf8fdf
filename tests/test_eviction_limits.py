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


def test_a_query_in_two_e4m3_numbers():
    """What the header says of q over an E4M3 cache, for every bf16 number and every largest one of a head,
    scaled to (224, 448] by a power of two: hi = E4M3(x) and lo = E4M3(x - hi) hold it exactly from 2^-9
    of the largest on (some from 2^-10 on they do not), and to 2^-17 of the largest below."""
    torch = pytest.importorskip("torch")
    x = (torch.arange(0, 1 << 15, dtype=torch.int32) << 16).view(torch.float32)  # all that are not negative
    x = x[(x <= 448) & (x > 2.0 ** -60)]

    def e4m3(v):
        return v.to(torch.float8_e4m3fn).float()
    hi = e4m3(x)
    left = (x.double() - (hi + e4m3(x - hi)).double()).abs().numpy()
    x = x.double().numpy()
    largest = x[x > 224]
    assert len(largest) == 128  # every mantissa
    for top in largest:
        assert not left[(x >= top * 2.0 ** -9) & (x <= top)].any()
        assert left[x <= top].max() <= top * 2.0 ** -17
    assert left[(x >= 225 * 2.0 ** -10) & (x < 0.25)].any() and not left[x >= 0.25].any()
