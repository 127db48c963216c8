"""How blocks of keys and values reach shared memory: rows and whole boxes in turns through the
same places, values taken out on the way, pages that are missing or that change meanwhile."""
import math

import pytest
import torch

from cache_helpers import ints, skv
from chunk_helpers import check
from test_gpu_cache_attend import filled
from test_gpu_cache_chunk import queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tb", [24, 128])
def test_values_taken_out_of_blocks_that_are_followed_by_boxes(dtype, d, tb):
    """NaN in every 37th token, so that each item takes values out of its partly masked blocks
    and goes on with whole ones in the same places: rows keep the bits of what they see."""
    n, new, window, h = 3000, 1500, 700, 4
    c = filled(dtype, 1, h, d, tb, 1, n)
    q = queries(new, 2 * h, d)
    args = (0, ints([0]), ints([n]), ints([0, new]), q, n)
    out, lse = c.attend_chunk(*args, window=window, lse=True)
    t = torch.arange(5, n, 37, device="cuda")
    for head in range(h):
        c.pool[c.table[0, 0, 1, head, t // tb].long(), t % tb, 3 + 8 * head] = 0x7FC0 if dtype == 0 else 0x7F
    o2, l2 = c.attend_chunk(*args, window=window, lse=True)
    assert torch.equal(l2, lse)
    for head in range(h):
        rest = [i for i in range(d) if i != 3 + 8 * head]
        for j in (2 * head, 2 * head + 1):
            assert torch.equal(o2[:, j, rest], out[:, j, rest])
            assert torch.all(torch.isnan(o2[:, j, 3 + 8 * head]))
    for _ in range(20):
        o3, l3 = c.attend_chunk(*args, window=window, lse=True)
        assert torch.equal(o3.view(torch.int16), o2.view(torch.int16)) and torch.equal(l3, lse)
    c.status()
