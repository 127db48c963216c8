"""Attention of one new token over the paged cache against float64 (tolerances derived
in cache_helpers.check_attend)."""
import math

import pytest
import torch

from cache_helpers import check_attend, ints, skv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def filled(dtype, layers, heads, d, tb, seqs, max_len, seed=0, scaled=True, outside=None):
    """A cache whose every sequence has pages for max_len tokens, in a random order;
    `outside`: the pattern in all places that no test fills."""
    P = skv()
    g = torch.Generator(device="cuda").manual_seed(seed)
    blocks = max(1, -(-max_len // tb))
    pages = seqs * layers * 2 * heads * blocks + 2
    x = torch.randn(pages, tb, d, generator=g, device="cuda") * \
        torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))
    pool = x.bfloat16().view(torch.int16) if dtype == 0 else \
        (x * 16).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    table = torch.randperm(pages, generator=g, device="cuda")[:pages - 2].int().view(
        seqs, layers, 2, heads, blocks)
    scale = torch.rand(layers, heads, generator=g, device="cuda") * 0.1 + 0.02 \
        if dtype and scaled else None
    return P.PagedCache(dtype, layers, heads, d, tb, pool=pool.contiguous(),
                        table=table.contiguous(), scale=scale,
                        refs=torch.ones(pages, dtype=torch.int32, device="cuda"))


def run(c, dtype, layer, slots, lens, hq, begins=None, seed=1, q=None, scale=None, max_len=None):
    if q is None:
        g = torch.Generator(device="cuda").manual_seed(seed)
        q = torch.randn(len(slots), hq, c.head_dim, generator=g, device="cuda").bfloat16()
    out, lse = c.attend(layer, ints(slots), ints(lens), q, max(lens) if max_len is None else max_len,
                        begins=None if begins is None else ints(begins), scale=scale, lse=True)
    c.status()
    check_attend(c, dtype, layer, slots, begins or [0] * len(slots), lens, q,
                 c.head_dim ** -0.5 if scale is None else scale, out, lse)
    return q, out, lse


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [16, 64, 80, 96, 128, 192, 256])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 4), (3, 5), (1, 8), (2, 9), (1, 16), (1, 20)])
def test_head_layouts(dtype, d, heads, group):
    c = filled(dtype, 2, heads, d, 16, 3, 150, seed=d)
    run(c, dtype, 1, [2, 0, 1], [150, 37, 64], heads * group)


def test_bf16_head_dims_of_8():
    for d in (8, 24, 72, 136, 248):
        c = filled(0, 1, 2, d, 16, 2, 70, seed=d)
        run(c, 0, 0, [1, 0], [70, 5], 4)


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("tb", [1, 5, 16, 24, 32, 33, 128, 256])
def test_page_sizes_and_lengths(dtype, tb):
    lens = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300]
    c = filled(dtype, 1, 2, 64, tb, len(lens), 300, seed=tb)
    run(c, dtype, 0, list(range(len(lens)))[::-1], lens, 4)
    # all in one short row: one block, no join
    run(c, dtype, 0, [3], [1], 4)


@pytest.mark.parametrize("dtype,d,group", [(0, 128, 8), (1, 128, 8), (0, 64, 2), (1, 64, 16),
                                           (0, 256, 4), (1, 256, 12)])
@pytest.mark.parametrize("n", [1000, 5003, 20011])
def test_long_rows_are_split_and_joined(dtype, d, group, n):
    c = filled(dtype, 1, 2, d, 128, 1, n, seed=n)
    q, out, lse = run(c, dtype, 0, [0], [n], 2 * group)
    for _ in range(3):                                    # the same bits every time
        o2, l2 = c.attend(0, ints([0]), ints([n]), q, n, lse=True)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    # the result alone, and a larger bound on the lengths
    assert torch.equal(c.attend(0, ints([0]), ints([n]), q, n), out)


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
def test_ragged_batch_with_windows(dtype):
    lens = [0, 700, 1, 333, 700, 64, 512, 5, 690, 100]
    begins = [0, 100, 0, 333, 699, 0, 257, 9, 16, -3]     # some leave nothing, one is clamped
    c = filled(dtype, 2, 4, 128, 64, len(lens), 700)
    g = torch.Generator(device="cuda").manual_seed(9)
    q = torch.randn(len(lens), 8, 128, generator=g, device="cuda").bfloat16()
    out, lse = c.attend(0, ints(range(10)), ints(lens), q, 700, begins=ints(begins), lse=True)
    c.status()
    check_attend(c, dtype, 0, range(10), [max(0, b) for b in begins], lens, q, 128 ** -0.5, out, lse)


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("tb", [16, 33])
def test_nan_and_infinities_outside_the_range_have_no_effect(dtype, tb):
    c = filled(dtype, 1, 2, 64, tb, 2, 200)
    begins, lens = [21, 0], [150, 77]
    q, out, lse = run(c, dtype, 0, [0, 1], lens, 4, begins)
    bad = [0x7FC0, 0x7F80, -128] if dtype == 0 else [0x7F, 0xFF, 0x7F]   # NaN, inf, -inf; NaN
    for s in (0, 1):
        for t in list(range(begins[s])) + list(range(lens[s], c.table.shape[-1] * tb)):
            pages = c.table[s, 0, :, :, t // tb].flatten().long()
            c.pool[pages, t % tb] = bad[t % 3]
    o2, l2 = c.attend(0, ints([0, 1]), ints(lens), q, 200, begins=ints(begins), lse=True)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    # pages beyond the length may be missing
    c.table[0, 0, :, :, -(-150 // tb):] = -1
    o2, l2 = c.attend(0, ints([0, 1]), ints(lens), q, 200, begins=ints(begins), lse=True)
    c.status()
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_special_values_inside_the_range():
    c = filled(0, 1, 1, 64, 16, 1, 40)
    q = torch.ones(1, 1, 64, device="cuda").bfloat16()
    pool = c.pool.view(torch.bfloat16)
    k = lambda t: pool[int(c.table[0, 0, 0, 0, t // 16]), t % 16]  # noqa: E731
    k(7)[3] = -math.inf                                   # a score of -inf: weight 0
    out, lse = c.attend(0, ints([0]), ints([40]), q, 40, lse=True)
    check = [t for t in range(40) if t != 7]
    ks = torch.stack([k(t) for t in check]).double()
    vs = torch.stack([pool[int(c.table[0, 0, 1, 0, t // 16]), t % 16] for t in check]).double()
    s = ks.sum(1) / 8
    assert abs(float(lse) - float(torch.logsumexp(s, 0))) < 1e-4
    ref = torch.softmax(s, 0) @ vs
    assert torch.all((out[0, 0].double() - ref).abs() <= 2.0 ** -6 * (torch.softmax(s, 0) @ vs.abs()))
    for t in range(40):
        k(t)[3] = -math.inf                               # nothing has weight
    out, lse = c.attend(0, ints([0]), ints([40]), q, 40, lse=True)
    assert torch.all(out == 0) and float(lse) == -math.inf
    k(11)[3] = math.nan
    out, lse = c.attend(0, ints([0]), ints([40]), q, 40, lse=True)
    assert torch.all(torch.isnan(out)) and math.isnan(float(lse))


def test_nan_codes_inside_the_range():
    c = filled(1, 1, 2, 64, 16, 1, 40)
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(1, 4, 64, generator=g, device="cuda").bfloat16()
    want, wl = c.attend(0, ints([0]), ints([40]), q, 40, lse=True)
    c.pool[int(c.table[0, 0, 1, 0, 1]), 3, 7] = 0x7F          # a value of kv head 0
    out, lse = c.attend(0, ints([0]), ints([40]), q, 40, lse=True)
    assert torch.all(torch.isnan(out[0, :2, 7])) and torch.equal(lse, wl)
    rest = [d for d in range(64) if d != 7]
    assert torch.equal(out[0, :2, rest], want[0, :2, rest]) and torch.equal(out[0, 2:], want[0, 2:])
    c.pool[int(c.table[0, 0, 0, 1, 2]), 1, 0] = 0xFF          # a key of kv head 1
    out, lse = c.attend(0, ints([0]), ints([40]), q, 40, lse=True)
    assert torch.all(torch.isnan(out[0, 2:])) and torch.all(torch.isnan(lse[0, 2:]))
    assert torch.equal(lse[0, :2], wl[0, :2])


def test_infinite_values_inside_the_range():
    c = filled(0, 1, 1, 64, 16, 1, 40)
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(1, 4, 64, generator=g, device="cuda").bfloat16()
    want = c.attend(0, ints([0]), ints([40]), q, 40)
    v = lambda t: c.pool.view(torch.bfloat16)[int(c.table[0, 0, 1, 0, t // 16]), t % 16]  # noqa: E731
    for t in range(0, 40, 3):
        v(t)[5], v(t)[9] = math.inf, -math.inf
    v(0)[11], v(1)[11] = math.inf, -math.inf
    out = c.attend(0, ints([0]), ints([40]), q, 40)
    assert torch.all(out[0, :, 5] == math.inf) and torch.all(out[0, :, 9] == -math.inf)
    assert torch.all(torch.isnan(out[0, :, 11]))
    rest = [d for d in range(64) if d not in (5, 9, 11)]
    assert torch.equal(out[0, :, rest], want[0, :, rest])


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
def test_large_and_growing_scores(dtype):
    """Scores that grow along the row by far more than the slack of the running maximum,
    large q, tiny q, zero q, a negative softmax scale."""
    c = filled(dtype, 1, 1, 64, 16, 1, 2000)
    f = torch.linspace(0.01, 2.0, 2000)
    for t in range(2000):
        p = int(c.table[0, 0, 0, 0, t // 16])
        if dtype == 0:
            v = c.pool.view(torch.bfloat16)
            v[p, t % 16] = (v[p, t % 16].float() * float(f[t])).bfloat16()
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(1, 4, 64, generator=g, device="cuda")
    for mul, scale in ((8.0, None), (1e-6, None), (0.0, None), (1.0, -0.3), (1e4, 1e-5)):
        run(c, dtype, 0, [0], [2000], 4, q=(q * mul).bfloat16(), scale=scale)
    wide = q.clone()
    wide[..., ::2] *= 2.0 ** -20                          # a wide range of channels within a head
    run(c, dtype, 0, [0], [2000], 4, q=wide.bfloat16())


def test_strides_in_place_and_padding_slots():
    c = filled(0, 1, 2, 64, 16, 2, 90)
    g = torch.Generator(device="cuda").manual_seed(4)
    wide = torch.randn(3, 8, 80, generator=g, device="cuda").bfloat16()
    q = wide[:, 2:6, 8:72]
    q1 = q.contiguous()
    want, lse = c.attend(0, ints([1, -1, 0]), ints([90, 50, 33]), q1, 90, lse=True)
    c.status()
    assert torch.all(want[1] == 0) and torch.all(lse[1] == -math.inf)
    assert torch.equal(c.attend(0, ints([1, -1, 0]), ints([90, 50, 33]), q, 90), want)
    assert c.attend(0, ints([1, -1, 0]), ints([90, 50, 33]), q1, 90, out=q1) is q1
    assert torch.equal(q1, want)


def test_bad_data_is_reported():
    P = skv()
    c = filled(0, 1, 2, 64, 16, 2, 90)
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn(2, 4, 64, generator=g, device="cuda").bfloat16()
    good = c.attend(0, ints([1, 0]), ints([90, 33]), q, 90)
    c.status()
    for slots, lens, max_len in (([1, 2], [90, 33], 90), ([1, 0], [90, -1], 90),
                                 ([1, 0], [90, 97], 100), ([1, 0], [90, 91], 90)):
        out, lse = c.attend(0, ints(slots), ints(lens), q, max_len, lse=True)
        with pytest.raises(P.SkvError):
            c.status()
        assert torch.equal(out[0], good[0]) and torch.all(out[1] == 0)
        assert torch.all(lse[1] == -math.inf)
    # a key or value page that is missing or past the pool: its tokens are left out
    for side, page in ((0, -1), (1, c.pool.shape[0])):
        old = c.table[0, 0, side, 1, 1].clone()
        c.table[0, 0, side, 1, 1] = page
        out, lse = c.attend(0, ints([1, 0]), ints([90, 33]), q, 90, lse=True)
        with pytest.raises(P.SkvError):
            c.status()
        c.table[0, 0, side, 1, 1] = old
        assert torch.equal(out[0], good[0]) and torch.equal(out[1, :2], good[1, :2])
        tok = [t for t in range(33) if t // 16 != 1]
        for i in (2, 3):
            pool = c.pool.view(torch.bfloat16)
            kk, vv = (torch.stack([pool[int(c.table[0, 0, s, 1, t // 16]), t % 16] for t in tok]
                                  ).double() for s in (0, 1))
            s = kk @ q[1, i].double() / 8
            w = torch.softmax(s, 0)
            assert abs(float(lse[1, i]) - float(torch.logsumexp(s, 0))) < 1e-4
            assert torch.all((out[1, i].double() - w @ vv).abs() <= 2.0 ** -6 * (w @ vv.abs()))


def test_empty_batch_and_all_rows_empty():
    c = filled(0, 1, 2, 64, 16, 2, 90)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    e = torch.empty(0, 4, 64, device="cuda").bfloat16()
    assert c.attend(0, none, none, e, 90).shape == (0, 4, 64)
    q = torch.ones(2, 4, 64, device="cuda").bfloat16()
    for max_len in (0, 90):
        out, lse = c.attend(0, ints([0, 1]), ints([0, 0]), q, max_len, lse=True)
        c.status()
        assert torch.all(out == 0) and torch.all(lse == -math.inf)


def test_many_sequences():
    """More batch entries than a block's threads, most of them short."""
    n = 700
    c = filled(1, 1, 2, 64, 16, 50, 40)
    g = torch.Generator().manual_seed(0)
    lens = torch.randint(0, 41, (n,), generator=g).tolist()
    run(c, 1, 0, [i % 50 for i in range(n)], lens, 4, max_len=40)


@pytest.mark.parametrize("batch", [33, 70, 1100])
@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
def test_many_sequences_with_long_ones_among_them(dtype, batch):
    """Cut rows in a batch of more entries than a warp has lanes (and than their square)."""
    c = filled(dtype, 1, 1, 64, 32, 4, 4100)
    g = torch.Generator().manual_seed(batch)
    lens = torch.randint(0, 30, (batch,), generator=g)
    long = torch.randperm(batch, generator=g)[:6]
    lens[long] = torch.tensor([4100, 3000, 4099, 1, 2048, 777])
    lens = lens.tolist()
    slots = [i % 4 for i in range(batch)]
    gq = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(batch, 2, 64, generator=gq, device="cuda").bfloat16()
    out, lse = c.attend(0, ints(slots), ints(lens), q, 1 << 17 if batch == 1100 else 4100, lse=True)
    c.status()
    sel = sorted(set(long.tolist() + [i for i in range(0, batch, 1 + batch // 40)]))
    check_attend(c, dtype, 0, [slots[i] for i in sel], [0] * len(sel), [lens[i] for i in sel],
                 q[sel], 64 ** -0.5, out[sel], lse[sel])


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
    run(c, 0, 0, [0], [3001], 4)


def test_graph_replay_with_new_lengths():
    c = filled(1, 1, 2, 128, 64, 2, 900)
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn(2, 8, 128, generator=g, device="cuda").bfloat16()
    lens, slots = ints([0, 0]), ints([0, 1])
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        out, lse = c.attend(0, slots, lens, q, 900, lse=True)
    for n in ([900, 1], [64, 0], [513, 900]):
        lens.copy_(ints(n))
        graph.replay()
        torch.cuda.synchronize()
        check_attend(c, 1, 0, [0, 1], [0, 0], n, q, 128 ** -0.5, out, lse)


def test_two_streams_at_once():
    c = filled(0, 1, 4, 128, 64, 4, 3000)
    g = torch.Generator(device="cuda").manual_seed(4)
    q = [torch.randn(4, 16, 128, generator=g, device="cuda").bfloat16() for _ in range(2)]
    lens = [ints([3000, 10, 0, 1234]), ints([77, 2999, 3000, 64])]
    slots = ints(range(4))
    want = [c.attend(0, slots, n, x, 3000) for n, x in zip(lens, q)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in (0, 1):
            got[i].append(c.attend(0, slots, lens[i], q[i], 3000, stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(want[i], o) for o in got[i])
    c.status()


def test_lengths_and_queries_written_just_before():
    """The lengths, the queries and the pages come from work that is enqueued right before
    the call, on the same stream, without a wait: long rows that are split and joined."""
    c = filled(1, 1, 2, 128, 128, 2, 9000)
    g = torch.Generator(device="cuda").manual_seed(4)
    q0 = torch.randn(2, 16, 128, generator=g, device="cuda")
    slots = ints([0, 1])
    cases = [([9000, 17], 1.0), ([64, 9000], 0.5), ([8999, 8999], 2.0), ([0, 5000], 1.0)]
    want = []
    for n, f in cases:
        want.append(c.attend(0, slots, ints(n), (q0 * f).bfloat16(), 9000, lse=True))
        torch.cuda.synchronize()
    slow = torch.randn(4096, 4096, device="cuda")
    lens, q = ints([0, 0]), torch.zeros(2, 16, 128, device="cuda").bfloat16()
    new = [ints(n) for n, _ in cases]
    got = []
    torch.cuda.synchronize()
    for _ in range(4):
        for i, (n, f) in enumerate(cases):
            slow = slow @ slow * 1e-3
            lens.copy_(new[i])
            q.copy_(q0 * f)
            got.append((i, c.attend(0, slots, lens, q, 9000, lse=True)))
    torch.cuda.synchronize()
    for i, (o, l) in got:
        assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])
