"""Page operations on pools and requests that take more than one block (more than 16384
pages, 2048 entries of a sequence, 1024 sequences of a request), against the plain loops:
tables, counts and contents are equal, and what is refused changes nothing."""
import numpy as np
import pytest
import torch

from cache_helpers import Pages, ints, skv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def make(layers, heads, seqs, blocks, free, pages=20000, tb=2, seed=0):
    """A cache without sequences in a pool of which `free` pages, spread over all of it, are
    free; the others are counted once and no entry names them."""
    P = skv()
    c = P.PagedCache(P.SKV_BF16, layers, heads, 8, tb, num_pages=pages, max_seqs=seqs,
                     max_blocks=blocks)
    g = torch.Generator(device="cuda").manual_seed(seed)
    c.pool.copy_(torch.randint(-2 ** 15, 2 ** 15, c.pool.shape, generator=g, device="cuda"))
    c.refs.fill_(1)
    c.refs[torch.randperm(pages, generator=g, device="cuda")[:free]] = 0
    return P, c


def stepper(c):
    ref = Pages(c)

    def step(name, *args):
        getattr(c, name)(*(ints(a) for a in args))
        getattr(ref, name)(*args)
        c.status()
        ref.same(c.table, c.refs, c.pool)

    return ref, step


def refused(P, c, status, *calls):
    before = c.table.clone(), c.refs.clone(), c.pool.clone()
    for name, args in calls:
        getattr(c, name)(*(ints(a) for a in args))
        with pytest.raises(P.SkvError) as e:
            c.status()
        assert e.value.status == status, (name, args)
        for x, y in zip(before, (c.table, c.refs, c.pool)):
            assert torch.equal(x, y), (name, args)


@pytest.mark.parametrize("pages", [16384, 16385, 20000, 50000])
@pytest.mark.parametrize("layers,heads,blocks", [(1, 1, 5), (2, 3, 5), (1, 3, 7), (1, 1, 4)])
def test_a_life_of_sequences(pages, layers, heads, blocks):
    """Entries of a sequence that are and are not a multiple of 4 (10, 60, 42, 8)."""
    tb, rows = 2, layers * 2 * heads
    P, c = make(layers, heads, 6, blocks, rows * 23 + 3, pages, tb, seed=blocks)
    ref, step = stepper(c)
    step("reserve", [3, 0], [0, 0], [2 * tb + 1, 3 * tb])
    step("reserve", [3], [2 * tb + 1], [3 * tb])
    step("fork", [3, 0, 3], [1, 5, 2], [2 * tb + 1, 3 * tb, tb])
    step("fork", [0], [4], [0])
    step("reserve", [4, 1], [0, 2 * tb + 1], [tb, 4 * tb])
    step("free", [3])
    step("free", [4, 2])
    ref.compact()
    c.compact()
    c.status()
    ref.same(c.table, c.refs, c.pool)
    step("reserve", [2], [0], [2 * tb])
    step("free", [0, 1, 2, 3, 4, 5])


@pytest.mark.parametrize("pages", [16385, 20000])
def test_bad_requests_change_nothing(pages):
    P, c = make(2, 2, 6, 5, 200, pages)
    c.reserve(ints([0]), ints([0]), ints([5]))
    c.status()
    refused(P, c, P.SKV_ERR_ARG,
            ("reserve", ([6], [0], [3])), ("reserve", ([-1], [0], [3])),
            ("reserve", ([1], [-1], [3])), ("reserve", ([1], [4], [3])),
            ("reserve", ([1], [0], [11])), ("reserve", ([2, 2], [0, 0], [3, 3])),
            ("reserve", ([0], [0], [3])), ("reserve", ([1, 0], [0, 4], [3, 6])),
            ("fork", ([0], [0], [3])), ("fork", ([0], [6], [3])), ("fork", ([6], [1], [3])),
            ("fork", ([0], [1], [-1])), ("fork", ([0], [1], [11])),
            ("fork", ([0, 0], [1, 1], [3, 3])), ("fork", ([0, 1], [1, 2], [3, 0])),
            ("fork", ([0], [1], [7])), ("fork", ([1], [0], [0])))


@pytest.mark.parametrize("layers,heads", [(16, 16), (7, 37)], ids=["2560", "2590"])
def test_one_bad_entry_among_thousands(layers, heads):
    """2560 and 2590 entries of a sequence: two parts of 2048 (whole quads and single ones)."""
    rows, tb = layers * 2 * heads, 2
    P, c = make(layers, heads, 4, 5, rows * 10, 20000, tb)
    c.reserve(ints([0]), ints([0]), ints([3 * tb]))
    c.status()
    for r in (0, rows // 2, rows - 1):
        entry = c.table.view(4, rows, 5)
        for slot, b, value in ((0, 2, -1), (0, 1, 20000), (1, 4, 7), (1, 0, 7)):
            old = int(entry[slot, r, b])
            entry[slot, r, b] = value                # a parent's page missing, a child's entry taken
            refused(P, c, P.SKV_ERR_ARG, ("fork", ([0, 0], [2, 1], [2 * tb + 1] * 2)))
            if slot == 1 and b == 0:
                refused(P, c, P.SKV_ERR_ARG, ("reserve", ([2, 1], [0, 0], [1, 1])))
            entry[slot, r, b] = old
    ref, step = stepper(c)
    step("fork", [0, 0], [2, 1], [2 * tb + 1, 3 * tb])
    step("reserve", [1, 2], [3 * tb, 2 * tb + 1], [4 * tb, 4 * tb])
    step("free", [0, 1])


@pytest.mark.parametrize("n", [257, 600, 1500])
@pytest.mark.parametrize("pages", [9000, 20000])
def test_requests_of_many_sequences(n, pages):
    tb, rows = 2, 2
    P, c = make(1, 1, 2 * n + 3, 3, rows * 3 * n - 5, pages, tb, seed=n)
    g = np.random.default_rng(n)
    lens = g.integers(0, 3, n).tolist()
    slots = g.permutation(n).tolist()
    ref, step = stepper(c)
    step("reserve", slots, [0] * n, lens)
    at = dict(zip(slots, lens))
    parents = g.permutation(n).tolist()
    step("fork", parents, list(range(n, 2 * n)), [at[p] for p in parents])
    spare = 2 * n
    refused(P, c, P.SKV_ERR_ARG,
            ("reserve", (slots[:-1] + [slots[0]], [2] * n, [3] * n)),        # first and last
            ("fork", (parents[:2], [spare, spare], [0, 0])),
            ("fork", ([0] * n, [spare] + list(range(n + 1, 2 * n)), [0] * n)))
    step("free", list(range(n, 2 * n)))
    free = int((c.refs == 0).sum())
    # all that is left, and one more
    take = list(range(n))
    old = [at[s] for s in take]
    want = sum(rows * (3 - (a + 1) // 2) for a in old)
    assert want > free
    refused(P, c, P.SKV_ERR_CAPACITY, ("reserve", (take, old, [6] * n)))
    step("reserve", take[::2], old[::2], [2 * (-(-a // 2)) + 2 for a in old[::2]])
    step("free", take)


def test_the_last_free_page_and_one_too_many():
    P, c = make(1, 2, 4, 5, 4 * 3, 20000)
    refused(P, c, P.SKV_ERR_CAPACITY, ("reserve", ([0], [0], [7])),
            ("reserve", ([0, 1], [0, 0], [6, 1])))
    ref, step = stepper(c)
    step("reserve", [0, 1], [0, 0], [4, 1])
    assert int((c.refs == 0).sum()) == 0
    refused(P, c, P.SKV_ERR_CAPACITY, ("fork", ([0], [2], [3])))
    step("fork", [0], [2], [4])                       # full pages only
