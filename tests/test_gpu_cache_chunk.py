"""Attention of chunks of new tokens over the paged cache against float64 (tolerances derived
in chunk_helpers)."""
import math

import pytest
import torch

from cache_helpers import ints, skv
from chunk_helpers import check
from test_gpu_cache_attend import filled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def queries(n, hq, d, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, hq, d, generator=g, device="cuda").bfloat16()


def starts_of(news, first=0):
    s = [first]
    for n in news:
        s.append(s[-1] + n)
    return s


def run(c, dtype, layer, slots, lens, news, hq, begins=None, window=0, causal=True, seed=1, q=None,
        scale=None, max_len=None, heads=None):
    starts = starts_of(news)
    if q is None:
        q = queries(starts[-1], hq, c.head_dim, seed)
    out, lse = c.attend_chunk(layer, ints(slots), ints(lens), ints(starts), q,
                              max(lens) if max_len is None else max_len, window=window, causal=causal,
                              begins=None if begins is None else ints(begins), scale=scale, lse=True)
    c.status()
    check(c, dtype, layer, slots, lens, starts, q, out, lse, begins, window, causal, scale, heads=heads)
    return q, out, lse


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [16, 64, 80, 96, 128, 192, 256])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 4), (3, 5), (1, 8), (2, 9), (1, 16), (1, 200)])
def test_head_layouts(dtype, d, heads, group):
    c = filled(dtype, 2, heads, d, 16, 3, 150, seed=d)
    run(c, dtype, 1, [2, 0, 1], [150, 37, 64], [9, 37, 1], heads * group)


def test_bf16_head_dims_of_8():
    for d in (8, 24, 72, 136, 248):
        c = filled(0, 1, 2, d, 16, 2, 70, seed=d)
        run(c, 0, 0, [1, 0], [70, 5], [33, 5], 4)


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("tb", [1, 5, 16, 24, 32, 33, 128, 256])
@pytest.mark.parametrize("d", [64, 256])
def test_page_sizes_and_lengths(dtype, tb, d):
    lens = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300]
    c = filled(dtype, 1, 2, d, tb, len(lens), 300, seed=tb)
    slots = list(range(len(lens)))[::-1]
    run(c, dtype, 0, slots, lens, [min(n, 7) for n in lens], 4)
    run(c, dtype, 0, slots, lens, lens, 4)                    # all tokens are new
    run(c, dtype, 0, [3], [1], [1], 4)


@pytest.mark.parametrize("dtype,d,group", [(0, 128, 8), (1, 128, 8), (0, 64, 2), (1, 64, 16),
                                           (0, 256, 4), (1, 256, 12), (0, 96, 3)])
@pytest.mark.parametrize("n,new", [(1000, 1), (5003, 40), (20011, 3), (2500, 700)])
def test_long_rows_are_split_and_joined(dtype, d, group, n, new):
    c = filled(dtype, 1, 2, d, 128, 1, n, seed=n)
    q, out, lse = run(c, dtype, 0, [0], [n], [new], 2 * group)
    for _ in range(3):                                    # the same bits every time
        o2, l2 = c.attend_chunk(0, ints([0]), ints([n]), ints([0, new]), q, n, lse=True)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    assert torch.equal(c.attend_chunk(0, ints([0]), ints([n]), ints([0, new]), q, n), out)


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("window", [0, 1, 3, 64, 129, 1000])
@pytest.mark.parametrize("causal", [True, False])
def test_ragged_batch_with_windows(dtype, d, window, causal):
    lens = [0, 700, 1, 333, 700, 64, 512, 5, 690, 100]
    news = [0, 300, 1, 333, 2, 64, 129, 0, 1, 50]
    begins = [0, 100, 0, 333, 699, 60, 257, 9, 16, -3]     # some leave rows empty, one is clamped
    c = filled(dtype, 2, 4, d, 64, len(lens), 700)
    run(c, dtype, 0, list(range(10)), lens, news, 8, begins=begins, window=window, causal=causal)


@pytest.mark.parametrize("group", [1, 3])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_long_prompts(d, group):
    """Several tiles of rows and of tokens, some of them without a mask."""
    c = filled(0, 1, 2, d, 64, 2, 1500)
    run(c, 0, 0, [0, 1], [1500, 1111], [1500, 600], 2 * group)
    run(c, 0, 0, [0, 1], [1500, 1111], [1500, 600], 2 * group, window=400)
    c = filled(1, 1, 2, d, 64, 2, 1500)
    run(c, 1, 0, [0, 1], [1500, 1111], [1500, 600], 2 * group)


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("tb", [16, 33, 128])
def test_nan_and_infinities_that_are_not_seen_have_no_effect(dtype, tb):
    """Outside the range, and at tokens that only later rows see (or, with a window, earlier
    ones): rows that do not see them keep their bits."""
    c = filled(dtype, 1, 2, 64, tb, 2, 400)
    lens, news, begins = [390, 77], [200, 30], [21, 0]
    bad = [0x7FC0, 0x7F80, -128] if dtype == 0 else [0x7F, 0xFF, 0x7F]   # NaN, inf, -inf; NaN
    clean = c.pool.clone()
    for window in (0, 50):
        c.pool.copy_(clean)
        q, out, lse = run(c, dtype, 0, [0, 1], lens, news, 4, begins, window)
        for s in (0, 1):
            for t in list(range(begins[s])) + list(range(lens[s], c.table.shape[-1] * tb)):
                pages = c.table[s, 0, :, :, t // tb].flatten().long()
                c.pool[pages, t % tb] = bad[t % 3]
        args = (0, ints([0, 1]), ints(lens), ints(starts_of(news)), q, 400)
        more = dict(begins=ints(begins), window=window, lse=True)
        o2, l2 = c.attend_chunk(*args, **more)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
        for side in (1, 0):                               # a value, then also a key, of one token
            t = 300
            c.pool[int(c.table[0, 0, side, 1, t // tb]), t % tb, 5] = bad[1]
            o2, l2 = c.attend_chunk(*args, **more)
            first = t - (lens[0] - news[0])
            last = min(news[0], first + window) if window else news[0]
            see = torch.zeros(sum(news), 4, dtype=torch.bool, device="cuda")
            see[first:last, 2:] = True
            assert torch.equal(o2[~see], out[~see]) and torch.equal(l2[~see], lse[~see])
            others = [i for i in range(64) if i != 5]
            if side == 1:
                assert torch.equal(l2, lse)
                assert torch.equal(o2[see][:, others], out[see][:, others])
                assert not torch.any(torch.isfinite(o2[see][:, 5]))
            elif dtype == 1:                              # a NaN among the scores
                assert torch.all(torch.isnan(o2[see])) and torch.all(torch.isnan(l2[see]))
        c.status()
    # pages beyond the length, or before the range, may be missing
    c.pool.copy_(clean)
    c.table[0, 0, :, :, -(-390 // tb):] = -1
    c.table[0, 0, :, :, :21 // tb] = -1
    o2, l2 = c.attend_chunk(*args, begins=ints(begins), lse=True)
    c.status()
    check(c, dtype, 0, [0, 1], lens, starts_of(news), q, o2, l2, begins)


@pytest.mark.parametrize("d", [128, 256])
def test_infinite_values_that_some_rows_see(d):
    """In a tile that is partly masked and in one that is not: +inf, -inf, both."""
    c = filled(0, 1, 1, d, 64, 1, 600)
    n, new = 600, 150
    q, out, lse = run(c, 0, 0, [0], [n], [new], 2)
    v = lambda t: c.pool.view(torch.bfloat16)[int(c.table[0, 0, 1, 0, t // 64]), t % 64]  # noqa: E731
    v(3)[7] = math.inf                                     # every row sees it
    v(500)[9], v(560)[9], v(590)[11] = math.inf, -math.inf, math.nan
    o2, l2 = c.attend_chunk(0, ints([0]), ints([n]), ints([0, new]), q, n, lse=True)
    c.status()
    assert torch.equal(l2, lse)
    want = out.clone()
    want[:, :, 7] = math.inf
    want[50:, :, 9] = math.inf
    want[110:, :, 9] = math.nan
    want[140:, :, 11] = math.nan
    assert torch.equal(torch.isnan(o2), torch.isnan(want))
    assert torch.equal(o2.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d,n", [(64, 40), (128, 3000), (256, 40), (256, 3000)])
def test_rows_without_a_place_see_nothing(dtype, d, n):
    """More new tokens than the sequence has, all of which see all of it, among whose values are
    infinities and NaN; in one block of threads and in several."""
    c = filled(dtype, 1, 1, d, 64, 1, n)
    new = n + 5
    q = queries(new, 2, d)
    args = (0, ints([0]), ints([n]), ints([0, new]), q, n)
    out, lse = c.attend_chunk(*args, causal=False, lse=True)
    check(c, dtype, 0, [0], [n], [0, new], q, out, lse, causal=False)
    for t in (3, n - 1):
        c.pool[int(c.table[0, 0, 1, 0, t // 64]), t % 64, 7] = 0x7F80 if dtype == 0 else 0x7F
    o2, l2 = c.attend_chunk(*args, causal=False, lse=True)
    c.status()
    assert torch.equal(lse, l2) and torch.all(o2[:5] == 0) and torch.all(l2[:5] == -math.inf)
    rest = [i for i in range(d) if i != 7]
    assert torch.equal(o2[:, :, rest], out[:, :, rest]) and not torch.any(torch.isfinite(o2[5:, :, 7]))


def test_special_scores():
    c = filled(0, 1, 1, 64, 16, 1, 40)
    q = torch.ones(8, 1, 64, device="cuda").bfloat16()
    pool = c.pool.view(torch.bfloat16)
    k = lambda t: pool[int(c.table[0, 0, 0, 0, t // 16]), t % 16]  # noqa: E731
    for t in range(36):
        k(t)[3] = -math.inf                               # scores of -inf: weight 0
    args = (0, ints([0]), ints([40]), ints([0, 8]), q, 40)
    out, lse = c.attend_chunk(*args, lse=True)
    assert torch.all(out[:4] == 0) and torch.all(lse[:4] == -math.inf)
    assert torch.all(torch.isfinite(out[4:])) and torch.all(torch.isfinite(lse[4:]))
    k(38)[3] = math.nan
    o2, l2 = c.attend_chunk(*args, lse=True)
    assert torch.equal(o2[:6], out[:6]) and torch.equal(l2[:6], lse[:6])
    assert torch.all(torch.isnan(o2[6:])) and torch.all(torch.isnan(l2[6:]))


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 256])
def test_large_and_growing_scores(dtype, d):
    """Scores that grow along the row by far more than the slack of the running maximum,
    large q, tiny q, zero q, a negative softmax scale."""
    c = filled(dtype, 1, 1, d, 16, 1, 2000)
    f = torch.linspace(0.01, 2.0, 2000)
    for t in range(2000):
        p = int(c.table[0, 0, 0, 0, t // 16])
        if dtype == 0:
            v = c.pool.view(torch.bfloat16)
            v[p, t % 16] = (v[p, t % 16].float() * float(f[t])).bfloat16()
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(20, 4, d, generator=g, device="cuda")
    for mul, scale in ((8.0, None), (1e-6, None), (0.0, None), (1.0, -0.3), (1e4, 1e-5)):
        run(c, dtype, 0, [0], [2000], [20], 4, q=(q * mul).bfloat16(), scale=scale)
    wide = q.clone()
    wide[..., ::2] *= 2.0 ** -20                          # a wide range of channels within a head
    run(c, dtype, 0, [0], [2000], [20], 4, q=wide.bfloat16())


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 256])
def test_rows_of_very_different_size_with_a_negative_scale(dtype, d):
    """Rows whose scores have no sign left next to large ones, in one warp."""
    c = filled(dtype, 1, 1, d, 16, 1, 700)
    q = queries(20, 4, d).float()
    q[::2] *= 2.0 ** -126
    run(c, dtype, 0, [0], [700], [20], 4, q=q.bfloat16(), scale=-0.3)
    run(c, dtype, 0, [0], [700], [20], 4, q=(q * 2.0 ** -10).bfloat16(), scale=-2.0 ** -20)


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
def test_strides_in_place_padding_and_rows_of_no_sequence(dtype):
    c = filled(dtype, 1, 2, 64, 16, 2, 90)
    g = torch.Generator(device="cuda").manual_seed(4)
    wide = torch.randn(60, 8, 80, generator=g, device="cuda").bfloat16()
    q = wide[:, 2:6, 8:72]
    q1 = q.contiguous()
    args = (0, ints([1, -1, 0]), ints([90, 50, 33]), ints([3, 33, 40, 50]))
    mark = torch.full((60, 4, 64), 7.0, device="cuda").bfloat16()
    want, lse = c.attend_chunk(*args, q1, 90, out=mark.clone(), lse=True)
    c.status()
    check(c, dtype, 0, [1], [90], [3, 33], q1, want, lse)
    check(c, dtype, 0, [0], [33], [40, 50], q1, want, lse)
    assert torch.all(want[33:40] == 0) and torch.all(lse[33:40] == -math.inf)
    assert torch.all(want[:3] == 7) and torch.all(want[50:] == 7)
    assert torch.equal(c.attend_chunk(*args, q, 90, out=mark.clone()), want)
    assert c.attend_chunk(*args, q1, 90, out=q1) is q1
    assert torch.equal(q1[3:50], want[3:50])
    assert torch.equal(q1[:3], q.contiguous()[:3]) and torch.equal(q1[50:], q.contiguous()[50:])


def test_the_same_sequence_twice():
    """Two chunks of one slot: each sees the tokens up to its own places."""
    c = filled(0, 1, 2, 64, 16, 2, 90)
    run(c, 0, 0, [1, 1, 0, 1], [60, 90, 10, 61], [30, 30, 10, 1], 4)


def test_bad_data_is_reported():
    P = skv()
    c = filled(0, 1, 2, 64, 16, 2, 90)
    q = queries(50, 4, 64, 4)
    mark = torch.full((50, 4, 64), 7.0, device="cuda").bfloat16()

    def call(slots, lens, starts, max_len):
        return c.attend_chunk(0, ints(slots), ints(lens), ints(starts), q, max_len, out=mark.clone(),
                              lse=True)

    good, gl = call([1, 0], [90, 33], [0, 30, 50], 90)
    c.status()
    for slots, lens, max_len in (([1, 2], [90, 33], 90), ([1, 0], [90, -1], 90),
                                 ([1, 0], [90, 97], 100), ([1, 0], [90, 91], 90)):
        out, lse = call(slots, lens, [0, 30, 50], max_len)
        with pytest.raises(P.SkvError):
            c.status()
        assert torch.equal(out[:30], good[:30]) and torch.all(out[30:] == 0)
        assert torch.all(lse[30:] == -math.inf)
    for starts in ([0, 30, 51], [0, 30, 29], [0, 30, 1 << 30], [0, 30, -5]):
        out, lse = call([1, 0], [90, 33], starts, 90)
        with pytest.raises(P.SkvError):
            c.status()
        assert torch.equal(out[:30], good[:30]) and torch.all(out[30:] == 7)
    out, lse = call([1, 0], [90, 33], [-1, 30, 50], 90)
    with pytest.raises(P.SkvError):
        c.status()
    assert torch.equal(out[30:], good[30:]) and torch.all(out[:30] == 7)
    # more new tokens than the sequence has: those before its first see nothing
    out, lse = call([1, 0], [90, 12], [0, 30, 50], 90)
    c.status()
    assert torch.all(out[30:38] == 0) and torch.all(lse[30:38] == -math.inf)
    check(c, 0, 0, [0], [12], [38, 50], q, out, lse)
    # a key or value page that is missing or past the pool: its tokens are left out
    for side, page in ((0, -1), (1, c.pool.shape[0])):
        old = c.table[0, 0, side, 1, 1].clone()
        c.table[0, 0, side, 1, 1] = page
        out, lse = call([1, 0], [90, 33], [0, 30, 50], 90)
        with pytest.raises(P.SkvError):
            c.status()
        c.table[0, 0, side, 1, 1] = old
        assert torch.equal(out[:30], good[:30]) and torch.equal(out[30:, :2], good[30:, :2])
        pool = c.pool.view(torch.bfloat16)
        for j in (0, 5, 19):                              # places 13, 18 and 32
            tok = [t for t in range(14 + j) if t // 16 != 1]
            for i in (2, 3):
                kk, vv = (torch.stack([pool[int(c.table[0, 0, s, 1, t // 16]), t % 16] for t in tok]
                                      ).double() for s in (0, 1))
                s = kk @ q[30 + j, i].double() / 8
                w = torch.softmax(s, 0)
                assert abs(float(lse[30 + j, i]) - float(torch.logsumexp(s, 0))) < 1e-4
                assert torch.all((out[30 + j, i].double() - w @ vv).abs() <= 2.0 ** -6 * (w @ vv.abs()))


def test_empty_calls():
    c = filled(0, 1, 2, 64, 16, 2, 90)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    e = torch.empty(0, 4, 64, device="cuda").bfloat16()
    assert c.attend_chunk(0, none, none, ints([0]), e, 90).shape == (0, 4, 64)
    assert c.attend_chunk(0, ints([0, 1]), ints([5, 6]), ints([0, 0, 0]), e, 90).shape == (0, 4, 64)
    q = torch.ones(5, 4, 64, device="cuda").bfloat16()
    for max_len in (0, 90):
        out, lse = c.attend_chunk(0, ints([0, 1]), ints([0, 0]), ints([0, 2, 5]), q, max_len, lse=True)
        c.status()
        assert torch.all(out == 0) and torch.all(lse == -math.inf)


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("batch", [33, 700])
def test_many_sequences(dtype, batch):
    """More sequences than a warp has lanes and a block threads, most of them short."""
    c = filled(dtype, 1, 1, 64, 32, 4, 4100)
    g = torch.Generator().manual_seed(batch)
    lens = torch.randint(0, 30, (batch,), generator=g)
    long = torch.randperm(batch, generator=g)[:6]
    lens[long] = torch.tensor([4100, 3000, 4099, 1, 2048, 777])
    news = [min(int(n), int(k)) for n, k in zip(lens, torch.randint(0, 70, (batch,), generator=g))]
    run(c, dtype, 0, [i % 4 for i in range(batch)], lens.tolist(), news, 2)


def test_pool_offsets_past_32_bits():
    P = skv()
    tb, d = 2048, 128
    pages = (5 << 30) // (tb * d * 2)
    pool = torch.empty(pages, tb, d, dtype=torch.int16, device="cuda")
    table = torch.tensor([pages - 1, pages - 3, pages - 2, pages - 4], dtype=torch.int32,
                         device="cuda").view(1, 1, 2, 1, 2)
    for p in table.flatten().tolist():
        pool[p] = torch.randn(tb, d, device="cuda").bfloat16().view(torch.int16)
    c = P.PagedCache(0, 1, 1, d, tb, pool=pool, table=table,
                     refs=torch.ones(pages, dtype=torch.int32, device="cuda"))
    run(c, 0, 0, [0], [3001], [77], 4)


def test_query_offsets_past_32_bits():
    c = filled(0, 1, 1, 64, 16, 1, 90)
    wide = torch.empty(3, (3 << 30) // 2, dtype=torch.bfloat16, device="cuda")
    q = torch.as_strided(wide, (3, 2, 64), (wide.shape[1], wide.shape[1] - 64, 1))
    q.copy_(queries(3, 2, 64))
    run(c, 0, 0, [0], [90], [3], 2, q=q)


def test_graph_replay_with_new_lengths():
    c = filled(1, 1, 2, 128, 64, 2, 900)
    q = queries(40, 8, 128, 4)
    lens, slots, starts = ints([0, 0]), ints([0, 1]), ints([0, 0, 0])
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        out, lse = c.attend_chunk(0, slots, lens, starts, q, 900, lse=True)
    for n, st in (([900, 1], [0, 39, 40]), ([64, 0], [0, 1, 1]), ([513, 900], [3, 9, 40])):
        lens.copy_(ints(n))
        starts.copy_(ints(st))
        graph.replay()
        torch.cuda.synchronize()
        check(c, 1, 0, [0, 1], n, st, q, out, lse)


def test_two_graphs_and_an_eager_call_at_once():
    """Each captured call has a workspace of its own."""
    c = filled(0, 1, 4, 128, 64, 4, 3000)
    q = [queries(60, 16, 128, i) for i in range(3)]
    lens = [ints([3000, 20, 0, 1234]), ints([77, 2999, 3000, 64]), ints([3000, 3000, 3000, 3000])]
    slots, starts = ints(range(4)), ints([0, 20, 40, 40, 60])
    want = [c.attend_chunk(0, slots, n, starts, x, 3000, lse=True) for n, x in zip(lens, q)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    graphs, got = [], []
    for i in (0, 1):
        g = torch.cuda.CUDAGraph()
        streams[i].wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=streams[i]):
            got.append(c.attend_chunk(0, slots, lens[i], starts, q[i], 3000, lse=True))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(10):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        o, l = c.attend_chunk(0, slots, lens[2], starts, q[2], 3000, lse=True, stream=streams[2])
        torch.cuda.synchronize()
        for (x, y), (wo, wl) in zip(got + [(o, l)], want):
            assert torch.equal(x, wo) and torch.equal(y, wl)
    c.status()


def test_written_just_before():
    """Lengths, starts and queries come from work that is enqueued right before the call, on the
    same stream, without a wait."""
    c = filled(1, 1, 2, 128, 128, 2, 9000)
    q0 = queries(30, 16, 128, 4).float()
    slots = ints([0, 1])
    cases = [([9000, 17], [0, 10, 27], 1.0), ([64, 9000], [0, 3, 30], 0.5),
             ([8999, 8999], [0, 1, 2], 2.0), ([0, 5000], [0, 0, 30], 1.0)]
    want = []
    for n, st, f in cases:
        out = torch.zeros(30, 16, 128, device="cuda").bfloat16()
        want.append(c.attend_chunk(0, slots, ints(n), ints(st), (q0 * f).bfloat16(), 9000, out=out))
        torch.cuda.synchronize()
    slow = torch.randn(4096, 4096, device="cuda")
    lens, starts, q = ints([0, 0]), ints([0, 0, 0]), torch.zeros(30, 16, 128, device="cuda").bfloat16()
    new = [(ints(n), ints(st)) for n, st, _ in cases]
    got = []
    outs = [torch.zeros(30, 16, 128, device="cuda").bfloat16() for _ in range(16)]
    torch.cuda.synchronize()
    for r in range(4):
        for i, (_, _, f) in enumerate(cases):
            slow = slow @ slow * 1e-3
            lens.copy_(new[i][0])
            starts.copy_(new[i][1])
            q.copy_(q0 * f)
            got.append((i, c.attend_chunk(0, slots, lens, starts, q, 9000, out=outs[r * 4 + i])))
    torch.cuda.synchronize()
    for i, o in got:
        assert torch.equal(o, want[i])


def test_threads_on_one_stream():
    import threading
    c = filled(0, 2, 2, 128, 64, 2, 3000)
    q = [queries(12, 8, 128, i) for i in range(3)]
    lens = [ints(v) for v in ([3000, 10], [77, 2999], [2500, 2500])]
    slots, starts = ints([0, 1]), ints([0, 7, 12])
    want = [c.attend_chunk(i % 2, slots, lens[i], starts, q[i], 3000, lse=True) for i in range(3)]
    got = [[] for _ in range(3)]
    torch.cuda.synchronize()

    def work(i):
        for _ in range(100):
            got[i].append(c.attend_chunk(i % 2, slots, lens[i], starts, q[i], 3000, lse=True))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    c.status()
    for i in range(3):
        assert len(got[i]) == 100
        for o, l in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


def test_chunks_agree_with_single_tokens():
    """A chunk's rows are what `attend` gives for each token as the last one."""
    for dtype in (0, 1):
        c = filled(dtype, 1, 2, 128, 64, 1, 700)
        q, out, lse = run(c, dtype, 0, [0], [650], [25], 8)
        n = torch.arange(626, 651, dtype=torch.int32, device="cuda")
        o1, l1 = c.attend(0, torch.zeros_like(n), n, q, 650, lse=True)
        scale = o1.float().abs().amax()
        assert float((o1.float() - out.float()).abs().max()) <= 2.0 ** -6 * float(scale)
        assert torch.allclose(lse, l1, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
def test_a_run_of_append_chunk_and_single_token(dtype):
    """A prompt in two chunks, then single tokens: reserve, append with rotary positions,
    attend to what is there."""
    P = skv()
    h, group, d, tb = 2, 4, 64, 32
    scale = torch.full((1, h), 0.02, device="cuda") if dtype else None
    c = P.PagedCache(dtype, 1, h, d, tb, num_pages=64, max_seqs=2, max_blocks=6, scale=scale)
    c.pool.zero_()
    rope = P.Rope(1e4 ** (-2.0 * torch.arange(d // 2, device="cuda").double() / d))
    g = torch.Generator(device="cuda").manual_seed(3)
    lens = [0, 0]
    for news in ([70, 33], [40, 50], [1, 1], [1, 1]):
        new = [a + b for a, b in zip(lens, news)]
        c.reserve(ints([0, 1]), ints(lens), ints(new))
        qkv = torch.randn(sum(news), h * (group + 2), d, generator=g, device="cuda").bfloat16()
        q, k, v = qkv.split([h * group, h, h], 1)
        slots = ints([0] * news[0] + [1] * news[1])
        at = ints(list(range(lens[0], new[0])) + list(range(lens[1], new[1])))
        q = c.append(0, slots, at, q, k, v, rope, at.view(1, -1))
        starts = starts_of(news)
        out, lse = c.attend_chunk(0, ints([0, 1]), ints(new), ints(starts), q, max(new), lse=True)
        c.status()
        check(c, dtype, 0, [0, 1], new, starts, q, out, lse)
        if news == [1, 1]:
            o1 = c.attend(0, ints([0, 1]), ints(new), q, max(new))
            assert float((o1.float() - out.float()).abs().max()) <= 2.0 ** -6 * float(o1.abs().max())
        lens = new
