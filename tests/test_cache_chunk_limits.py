"""What the host refuses of chunk attention because the kernel counts in 32 bits (no GPU: every
pointer is a made-up number, and what passes the checks ends for want of a device)."""
import pytest

from test_cache_chunk_refusals import P, call  # noqa: F401  (P: the fixture)
from test_cache_refusals import cache

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("diff", [False, True])
def test_rows_end_below_31_bits(P, diff):  # noqa: F811
    """The last item's rows are counted to its end, 256 above its first."""
    one = dict(c=cache(P, heads=1, max_blocks=4), batch=1, qs=64, qhs=64, max_len=64, hq=1)
    for tokens in (MOST, MOST - 1, MOST - 255, MOST - 511):
        assert call(P, diff, tokens=tokens, **one) == P.SKV_ERR_ARG, tokens
    assert call(P, diff, tokens=MOST - 512, **one) != P.SKV_ERR_ARG
    two = dict(one, hq=2, qs=128)
    assert call(P, diff, tokens=2 ** 30 - 1, **two) == P.SKV_ERR_ARG
    assert call(P, diff, tokens=2 ** 30 - 512, **two) != P.SKV_ERR_ARG


@pytest.mark.parametrize("diff", [False, True])
def test_units_of_all_rows_are_below_31_bits(P, diff):  # noqa: F811
    """Sequences of one row each count for their blocks and what an item costs beside them."""
    for max_len, cost in ((64, 13), (500, 19), (4096, 76), (2 ** 20, 16396)):
        batch = 2 ** 31 // cost // 2                      # two kv heads
        one = dict(hq=2, qs=128, max_len=max_len)
        assert call(P, diff, batch=batch + cost, tokens=batch + cost, **one) == P.SKV_ERR_ARG, max_len
        less = (2 ** 31 - 1) // (2 * cost) * 32 // 33     # (tokens / 64 more items)
        assert call(P, diff, batch=less - less // 64, tokens=less - less // 64, **one) != P.SKV_ERR_ARG
