"""How blocks of keys and values reach shared memory: rows and whole boxes in turns through the
same places, values taken out on the way, pages that are missing or that change meanwhile."""
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


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tb", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("missing", [-1, 1 << 30])
def test_pages_that_are_missing_in_blocks_that_all_rows_see(dtype, d, tb, missing):
    """Their tokens are left out, whatever the side, and reported; other heads keep their bits."""
    P = skv()
    n, new = 2500, 40
    c = filled(dtype, 1, 2, d, tb, 1, n)
    q = queries(new, 4, d)
    args = (0, ints([0]), ints([n]), ints([0, new]), q, n)
    out, lse = c.attend_chunk(*args, lse=True)
    c.status()
    gone = torch.zeros(n, dtype=torch.bool, device="cuda")
    for side, t in ((0, 300), (1, 700), (0, 1100), (1, 1105), (1, 2000)):
        c.table[0, 0, side, 1, t // tb] = missing
        gone[t // tb * tb:(t // tb + 1) * tb] = True
    o2, l2 = c.attend_chunk(*args, lse=True)
    with pytest.raises(P.SkvError) as e:
        c.status()
    assert e.value.status == P.SKV_ERR_ARG
    assert torch.equal(o2[:, :2], out[:, :2]) and torch.equal(l2[:, :2], lse[:, :2])
    # the tokens that are left, as a sequence of their own
    rest = torch.nonzero(~gone)[:, 0]
    old = torch.nonzero(~gone[:n - new]).numel()
    assert rest.numel() == old + new
    e = filled(dtype, 1, 1, d, tb, 1, n)
    if dtype:
        e.scale.copy_(c.scale[:, 1:])
    t = torch.arange(rest.numel(), device="cuda")
    keep = c.table.clone()
    keep[(keep < 0) | (keep >= c.pool.shape[0])] = 0
    for side in (0, 1):
        e.pool[e.table[0, 0, side, 0, t // tb].long(), t % tb] = \
            c.pool[keep[0, 0, side, 1, rest // tb].long(), rest % tb]
    check(e, dtype, 0, [0], [rest.numel()], [0, new], q[:, 2:].contiguous(), o2[:, 2:], l2[:, 2:])


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("tb", [16, 128])
def test_a_table_that_is_overwritten_meanwhile(dtype, d, tb):
    """Pages go and come back on another stream: what comes of it is not defined, but no part of the
    kernel waits for bytes that do not come, and calls after it are right."""
    P = skv()
    n, new = 20000, 33
    c = filled(dtype, 1, 2, d, tb, 1, n)
    q = queries(new, 4, d)
    args = (0, ints([0]), ints([n]), ints([0, new]), q, n)
    out, lse = c.attend_chunk(*args, lse=True)
    c.status()
    full = c.table.clone()
    some = torch.where(torch.rand(full.shape, device="cuda") < 0.5, full, -1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(50):
        with torch.cuda.stream(side):
            for j in range(20):
                c.table.copy_(some if j % 2 else full)
        for j in range(8):
            c.attend_chunk(*args)
        torch.cuda.synchronize()
        try:
            c.status()
        except P.SkvError as e:
            assert e.status == P.SKV_ERR_ARG
    c.table.copy_(full)
    o2, l2 = c.attend_chunk(*args, lse=True)
    c.status()
    assert torch.equal(o2, out) and torch.equal(l2, lse)
