"""Page operations of the paged cache against plain loops on the host: tables, counts
and page contents are equal, and what is refused changes nothing."""
import numpy as np
import pytest
import torch

from cache_helpers import Pages, ints, skv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def make(dtype=0, layers=2, heads=2, d=64, tb=16, pages=300, seqs=6, blocks=5, seed=0):
    P = skv()
    g = torch.Generator(device="cuda").manual_seed(seed)
    hi = 1 << 15 if dtype == 0 else 256
    pool = torch.randint(0, hi, (pages, tb, d), generator=g, device="cuda",
                         dtype=torch.int16 if dtype == 0 else torch.uint8) if dtype else \
        torch.randint(-hi, hi, (pages, tb, d), generator=g, device="cuda", dtype=torch.int16)
    c = P.PagedCache(dtype, layers, heads, d, tb, max_seqs=seqs, max_blocks=blocks, pool=pool)
    return P, c


def test_a_new_cache_is_empty():
    P, c = make()
    assert torch.all(c.table == -1) and torch.all(c.refs == 0)
    c.status()


@pytest.mark.parametrize("dtype,d,tb", [(0, 64, 16), (0, 8, 5), (1, 16, 1), (1, 48, 33),
                                        (0, 72, 128)])
@pytest.mark.parametrize("layers,heads", [(1, 1), (2, 3)])
def test_a_life_of_sequences(dtype, d, tb, layers, heads):
    """reserve, fork, reserve more, free, compact (aside and in place), reserve again."""
    rows = layers * 2 * heads
    P, c = make(dtype, layers, heads, d, tb, pages=rows * 23 + 3)
    ref = Pages(c)

    def step(name, *args):
        getattr(c, name)(*(ints(a) for a in args))
        getattr(ref, name)(*args)
        c.status()
        ref.same(c.table, c.refs, c.pool)

    step("reserve", [3, 0], [0, 0], [2 * tb + 1, 3 * tb])
    step("reserve", [3], [2 * tb + 1], [min(2 * tb + 2, 3 * tb)])       # inside the last block
    step("fork", [3, 0, 3], [1, 5, 2], [2 * tb + 1, 3 * tb, tb])         # a tail, none, a shorter one
    step("fork", [0], [4], [0])                                          # nothing to share
    step("reserve", [4, 1], [0, 2 * tb + 1], [tb, 4 * tb])
    step("free", [3])
    step("free", [4, 2])
    step("free", [4])                                                    # empty already
    t, r = torch.empty_like(c.table), torch.empty_like(c.refs)
    before = c.table.clone(), c.refs.clone()
    c.compact(t, r)
    c.status()
    assert torch.equal(c.table, before[0]) and torch.equal(c.refs, before[1])
    ref.compact()
    ref.same(t, r, c.pool)
    c.compact()                                                          # the same in place
    c.status()
    ref.same(c.table, c.refs, c.pool)
    c.compact()                                                          # nothing left to move
    ref.same(c.table, c.refs, c.pool)
    step("reserve", [2], [0], [2 * tb])
    step("free", [0, 1, 2, 3, 4, 5])
    assert torch.all(c.refs == 0)


def test_compact_random_pools():
    for seed, (pages, live) in enumerate([(1, 0), (1, 1), (40, 0), (40, 40), (4096, 4000),
                                          (4097, 1000), (9001, 4500), (20000, 37)]):
        P, c = make(0, 1, 1, 8, 1, pages=pages, seqs=4, blocks=max(1, -(-live // 8)), seed=seed)
        rng = np.random.default_rng(seed)
        t = np.full(c.table.numel(), -1, dtype=np.int64)
        t[:live] = rng.permutation(pages)[:live]
        rng.shuffle(t)
        c.table.copy_(torch.from_numpy(t.astype(np.int32)).view(c.table.shape))
        c.refs.copy_(torch.from_numpy(np.bincount(t[t >= 0], minlength=pages).astype(np.int32)))
        ref = Pages(c)
        c.compact()
        c.status()
        ref.compact()
        ref.same(c.table, c.refs, c.pool)


def test_reserve_takes_the_lowest_free_pages_of_a_large_pool():
    P, c = make(1, 1, 1, 16, 1, pages=50000, seqs=2, blocks=9000)
    used = torch.rand(50000, device="cuda", generator=torch.Generator("cuda").manual_seed(3)) < 0.6
    c.refs.copy_(used.int())
    want = torch.nonzero(~used).flatten()[:18000].int()
    c.reserve(ints([1]), ints([0]), ints([9000]))
    c.status()
    assert torch.equal(c.table[1].flatten(), want)
    assert int(c.refs.sum()) == int(used.sum()) + 18000


BAD = [("reserve", ([6], [0], [3])), ("reserve", ([-1], [0], [3])), ("reserve", ([1], [-1], [3])),
       ("reserve", ([1], [4], [3])), ("reserve", ([1], [0], [81])),
       ("reserve", ([2, 2], [0, 0], [3, 3])), ("reserve", ([0], [0], [3])),   # entries taken
       ("fork", ([0], [0], [3])), ("fork", ([0], [6], [3])), ("fork", ([6], [1], [3])),
       ("fork", ([0], [1], [-1])), ("fork", ([0], [1], [81])), ("fork", ([0, 0], [1, 1], [3, 3])),
       ("fork", ([0, 1], [1, 2], [3, 0])),                                    # a child as a parent
       ("fork", ([0], [1], [50])),                                            # no page there
       ("fork", ([1], [0], [0])),                                             # a child with pages
       ("free", ([6],)), ("free", ([-1],))]


@pytest.mark.parametrize("name,args", BAD)
def test_bad_requests_change_nothing(name, args):
    P, c = make()
    c.reserve(ints([0]), ints([0]), ints([40]))
    c.status()
    before = c.table.clone(), c.refs.clone(), c.pool.clone()
    getattr(c, name)(*(ints(a) for a in args))
    with pytest.raises(P.SkvError) as e:
        c.status()
    assert e.value.status == P.SKV_ERR_ARG
    c.status()                                                                # cleared
    for x, y in zip(before, (c.table, c.refs, c.pool)):
        assert torch.equal(x, y)


def test_no_pages_left_changes_nothing():
    P, c = make(pages=8 * 4 - 1)
    c.reserve(ints([0]), ints([0]), ints([40]))                               # 24 of 31
    c.status()
    before = c.table.clone(), c.refs.clone()
    for call in (lambda: c.reserve(ints([1]), ints([0]), ints([1])),
                 lambda: c.reserve(ints([1, 2]), ints([0, 0]), ints([0, 16])),
                 lambda: c.fork(ints([0]), ints([1]), ints([33]))):
        call()
        with pytest.raises(P.SkvError) as e:
            c.status()
        assert e.value.status == P.SKV_ERR_CAPACITY
        assert torch.equal(before[0], c.table) and torch.equal(before[1], c.refs)
    c.fork(ints([0]), ints([1]), ints([32]))                                  # full pages only
    c.status()


def test_free_reports_bad_entries_and_a_slot_twice_counts_once():
    P, c = make()
    c.reserve(ints([0, 1]), ints([0, 0]), ints([16, 16]))
    c.status()
    c.free(ints([0, 0]))
    c.status()
    assert int(c.refs.sum()) == 8
    c.table[1, 0, 0, 0, 1] = 300                                              # past the pool
    c.table[1, 0, 0, 0, 2] = 0                                                # a free page
    c.free(ints([1]))
    with pytest.raises(P.SkvError):
        c.status()
    assert torch.all(c.table[1] == -1) and torch.all(c.refs == 0)


def test_free_of_entries_that_name_one_free_page():
    P, c = make()
    c.table[1] = 7                                                            # count 0, 40 times
    c.free(ints([1]))
    with pytest.raises(P.SkvError):
        c.status()
    assert torch.all(c.table == -1) and torch.all(c.refs == 0)


def test_compact_reports_entries_that_name_free_pages():
    P, c = make()
    c.reserve(ints([0, 1]), ints([0, 0]), ints([16, 16]))
    c.free(ints([0]))
    c.status()
    c.table[2, 0, 0, 0, 0] = 3
    c.table[2, 0, 0, 0, 1] = 299
    c.table[2, 0, 0, 0, 2] = 300
    c.compact()
    with pytest.raises(P.SkvError):
        c.status()
    assert c.table[2, 0, 0, 0, :3].tolist() == [3, 299, 300]
    assert sorted(c.table[1][c.table[1] >= 0].tolist()) == list(range(8))


@pytest.mark.parametrize("dtype,d,tb,n", [(0, 64, 16, 100), (1, 16, 1, 7), (0, 8, 3, 1),
                                          (0, 128, 256, 40), (1, 48, 33, 140)])
def test_copy_pages(dtype, d, tb, n):
    P, c = make(dtype, d=d, tb=tb)
    order = np.random.default_rng(n).permutation(300)
    src, dst = order[:n], order[n:2 * n]
    want = c.pool.clone()
    want[torch.from_numpy(dst).cuda()] = want[torch.from_numpy(src).cuda()]
    c.copy_pages(ints(src), ints(dst))
    c.status()
    assert torch.equal(c.pool, want)
    # out to pinned host memory and back to other places
    host = torch.zeros(n + 2, tb, d, dtype=c.pool.dtype).pin_memory()
    c.copy_pages(ints(src), ints(np.arange(n) + 1), dst_pool=host)
    c.copy_pages(ints(np.arange(n) + 1), ints(dst[::-1].copy()), src_pool=host)
    c.status()
    assert torch.equal(host[1:n + 1], want[torch.from_numpy(src).cuda()].cpu())
    assert torch.equal(c.pool[torch.from_numpy(dst[::-1].copy()).cuda()].cpu(), host[1:n + 1])
    # out of range: reported, the others copied
    before = c.pool.clone()
    c.copy_pages(ints([300, int(src[0])]), ints([int(dst[0]), 300]))
    with pytest.raises(P.SkvError):
        c.status()
    assert torch.equal(before, c.pool)
    with pytest.raises(P.SkvError):
        c.copy_pages(ints([0]), ints([1]), src_pool=torch.zeros(4, tb, d, dtype=c.pool.dtype))


def test_page_offsets_past_32_bits():
    P = skv()
    tb, d, pages = 2048, 128, (5 << 30) // (2048 * 128 * 2)
    c = P.PagedCache(P.SKV_BF16, 1, 1, d, tb, num_pages=pages, max_seqs=3, max_blocks=3)
    c.refs[:pages - 6] = 1
    c.reserve(ints([0]), ints([0]), ints([2 * tb - 1]))                       # the last pages
    c.status()
    assert c.table[0].flatten()[:2].tolist() == [pages - 6, pages - 5]
    top = torch.randint(-2 ** 15, 2 ** 15, (4, tb, d), dtype=torch.int16, device="cuda")
    c.pool[pages - 6:pages - 2] = top
    c.fork(ints([0]), ints([1]), ints([2 * tb - 1]))
    c.status()
    assert torch.equal(c.pool[pages - 2, :tb - 1], top[1, :tb - 1])
    assert torch.equal(c.pool[pages - 1, :tb - 1], top[3, :tb - 1])
    c.refs[1:5] = 0
    c.copy_pages(ints([pages - 6]), ints([1]))
    assert torch.equal(c.pool[1], top[0])
    c.compact()
    c.status()
    assert torch.equal(c.pool[int(c.table[0, 0, 0, 0, 0])], top[0])
    assert int(c.table.max()) < int((c.refs > 0).sum())


def test_in_a_graph_with_new_lengths():
    P, c = make()
    old, new = ints([0, 0]), ints([20, 33])
    slots = ints([4, 1])
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ref = Pages(c)
    with torch.cuda.graph(graph, stream=s):
        c.reserve(slots, old, new)
    for a, b in (([0, 0], [20, 33]), ([20, 33], [40, 34])):
        old.copy_(ints(a))
        new.copy_(ints(b))
        graph.replay()
        ref.reserve([4, 1], a, b)
        c.status()
        ref.same(c.table, c.refs, c.pool)


def test_wrapper_refusals():
    P, c = make()
    i = ints([0, 1])
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    rope = P.Rope(torch.ones(32, dtype=torch.float64, device="cuda"))
    for call in (lambda: c.reserve(i, i, i.long()), lambda: c.reserve(i, i, i.cpu()),
                 lambda: c.fork(i, i[:1], i), lambda: c.free(i.long()),
                 lambda: c.compact(table_out=c.table.clone()),
                 lambda: c.compact(c.table.clone(), c.refs[:2]),
                 lambda: c.append(0, i, i, x, x.float(), x),
                 lambda: c.append(0, i, i, x, x[:, :1], x),
                 lambda: c.append(0, i, i, x, x, x, rope),                    # positions missing
                 lambda: c.append(0, i, i, x, x, x, rope, i),                 # not [axes, n]
                 lambda: c.append(9, i, i, x, x, x),
                 lambda: c.attend(0, i, i, x.float(), 4), lambda: c.attend(0, i, i[:1], x, 4),
                 lambda: c.attend(0, i, i, x[:, :1], 4),                      # 1 head of 2
                 lambda: c.attend(0, i, i, x, 4, out=x[:, :, :32])):
        with pytest.raises(P.SkvError):
            call()
    c.status()
