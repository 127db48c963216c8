"""Lengths that another stream overwrites while a request runs: what comes of it is not
defined, but it stays inside the table, the counts and the pool."""
import pytest
import torch

from cache_helpers import ints, skv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages", [400, 20000])          # one block, and several
def test_requests_keep_to_the_pages_they_were_counted_for(pages):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    P = skv()
    rows, tb = 40, 4
    c = P.PagedCache(P.SKV_BF16, 1, rows // 2, 8, tb, num_pages=pages, max_seqs=6, max_blocks=4)
    side = torch.cuda.Stream()
    slots, parents, children = ints([0, 1]), ints([0, 1, 0]), ints([2, 3, 4])
    zero, full = ints([0, 0]), ints([2 * tb, 2 * tb + 1])
    lens, new = ints([0, 0, 0]), ints([0, 0])
    torch.cuda.synchronize()
    for i in range(200):
        c.clear()
        c.reserve(slots, zero, full)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for j in range(12):
                lens.fill_((tb, tb + 1, 0, 2 * tb)[(i + j) % 4])
                new.fill_((2 * tb, 3 * tb, 4 * tb, 2 * tb + 1)[(i + j) % 4])
        c.fork(parents, children, lens)
        c.reserve(slots, full, new)
        torch.cuda.synchronize()
        assert int(c.table.min()) >= -1 and int(c.table.max()) < pages
        named = torch.bincount(c.table[c.table >= 0].long(), minlength=pages)
        assert torch.all(c.refs[named > 0] > 0) and int(c.refs.min()) >= 0
        try:
            c.status()
        except P.SkvError:
            pass
