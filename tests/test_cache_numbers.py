"""Numbers that do not fit the library's 32 bits are refused by the binding, not cut (no GPU)."""
import pytest
import torch

from test_cache_binding import D, HEADS, Library, P, host_cache, ints  # noqa: F401  (P: the fixture)


@pytest.mark.parametrize("bad", [2 ** 31, 2 ** 32, 2 ** 32 + 8, -1, -2 ** 32 + 8])
def test_numbers_beyond_32_bits(P, bad):  # noqa: F811
    library = Library()
    c = host_cache(P, library)
    c._chunk_bytes = {4: 4096}
    q, lam = torch.zeros(2, 4, D, dtype=torch.bfloat16), torch.zeros(4)
    two, starts = ints(0, 1), ints(0, 1, 2)
    kv = torch.zeros(2, HEADS, D, dtype=torch.bfloat16)
    for call in (lambda: c.attend_chunk(0, two, two, starts, q, bad),
                 lambda: c.attend_chunk(0, two, two, starts, q, 8, window=bad),
                 lambda: c.attend_chunk(bad, two, two, starts, q, 8),
                 lambda: c.attend_diff(0, two, two, q, lam, bad),
                 lambda: c.attend_diff(0, two, two, q, lam, 8, window=bad),
                 lambda: c.attend_diff(bad, two, two, q, lam, 8, starts=starts),
                 lambda: c.attend(0, two, two, q, bad), lambda: c.attend(bad, two, two, q, 8),
                 lambda: c.append(bad, two, two, q, kv, kv)):
        with pytest.raises(P.SkvError) as e:
            call()
        assert e.value.status == P.SKV_ERR_ARG
    assert not library.calls


def test_the_largest_numbers_are_passed_on(P):  # noqa: F811
    library = Library()
    c = host_cache(P, library)
    c._chunk_bytes = {4: 4096}
    q = torch.zeros(2, 4, D, dtype=torch.bfloat16)
    two, most = ints(0, 1), 2 ** 31 - 1
    c.attend(0, two, two, q, most)
    c.attend_chunk(0, two, two, ints(0, 1, 2), q, most, window=most)
    assert library.calls[0][1][11] == most
    k = library.calls[1][1][2]._obj
    assert (k.max_len, k.window) == (most, most)
