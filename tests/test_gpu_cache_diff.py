"""Differential attention over the paged cache against float64 (tolerances derived in
chunk_helpers)."""
import math

import pytest
import torch

from cache_helpers import ints, skv
from chunk_helpers import check, check_norm
from test_gpu_cache_attend import filled
from test_gpu_cache_chunk import queries, starts_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def weights(hq, d, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.rand(hq, generator=g, device="cuda") * 0.8 - 0.1,
            torch.rand(d, generator=g, device="cuda") + 0.2)


def run(c, dtype, layer, slots, lens, news, hq, norm=False, q=None, max_len=None, begins=None, **more):
    """news None: one new token per sequence, the form without starts."""
    starts = None if news is None else starts_of(news)
    n = len(slots) if news is None else starts[-1]
    if q is None:
        q = queries(n, hq, c.head_dim)
    lam, w = weights(hq, c.head_dim)
    w = w if norm else None
    args = (layer, ints(slots), ints(lens), q, lam, max(lens) if max_len is None else max_len)
    kw = dict(starts=None if news is None else ints(starts),
              begins=None if begins is None else ints(begins), **more)
    out, lse = c.attend_diff(*args, norm=w, lse=True, **kw)
    c.status()
    if norm:
        check_norm(c.attend_diff(*args, **kw), out, w)
    check(c, dtype, layer, slots, lens, starts, q, out, lse, begins=begins, lam=lam, norm=w, **more)
    return q, lam, w, out, lse


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [16, 48, 64, 80, 96, 128, 192, 256])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 4), (3, 5), (2, 9), (1, 16), (1, 70)])
def test_head_layouts(dtype, d, heads, group):
    c = filled(dtype, 2, heads, d, 16, 3, 150, seed=d)
    run(c, dtype, 1, [2, 0, 1], [150, 37, 64], [9, 37, 1], heads * group)
    run(c, dtype, 1, [2, 0, 1], [150, 37, 64], None, heads * group)
    run(c, dtype, 1, [2, 0, 1], [150, 37, 64], [9, 37, 1], heads * group, norm=True)
    run(c, dtype, 1, [2, 0, 1], [150, 37, 64], None, heads * group, norm=True)


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("tb", [1, 16, 33, 128])
def test_page_sizes_and_lengths(dtype, tb):
    lens = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300]
    c = filled(dtype, 1, 2, 64, tb, len(lens), 300, seed=tb)
    slots = list(range(len(lens)))[::-1]
    run(c, dtype, 0, slots, lens, [min(n, 7) for n in lens], 4, norm=True)
    run(c, dtype, 0, slots, lens, lens, 4)
    run(c, dtype, 0, slots, lens, None, 4)
    run(c, dtype, 0, slots, lens, None, 4, norm=True)


@pytest.mark.parametrize("dtype,d,group", [(0, 128, 4), (1, 128, 4), (0, 64, 2), (1, 64, 16),
                                           (0, 256, 4), (1, 256, 12)])
@pytest.mark.parametrize("n,new", [(1000, 1), (5003, 40), (20011, None), (2500, 400)])
def test_long_rows_are_split_and_joined(dtype, d, group, n, new):
    c = filled(dtype, 1, 2, d, 128, 1, n, seed=n)
    for norm in (False, True):
        q, lam, w, out, lse = run(c, dtype, 0, [0], [n], None if new is None else [new], 2 * group, norm)
        for _ in range(3):                                # the same bits every time
            o2, l2 = c.attend_diff(0, ints([0]), ints([n]), q, lam, n, norm=w, lse=True,
                                   starts=None if new is None else ints([0, new]))
            assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("window", [0, 3, 129])
@pytest.mark.parametrize("causal", [True, False])
def test_ragged_batch_with_windows(dtype, window, causal):
    lens = [0, 700, 1, 333, 700, 64, 512, 5, 690, 100]
    news = [0, 300, 1, 333, 2, 64, 129, 0, 1, 50]
    begins = [0, 100, 0, 333, 699, 60, 257, 9, 16, -3]
    for d in (128, 256):
        c = filled(dtype, 2, 2, d, 64, len(lens), 700)
        run(c, dtype, 0, list(range(10)), lens, news, 4, begins=begins, window=window, causal=causal)
        run(c, dtype, 0, list(range(10)), lens, None, 4, begins=begins, window=window, causal=causal)


def test_one_token_with_and_without_starts():
    for dtype in (0, 1):
        c = filled(dtype, 1, 2, 128, 64, 4, 3000)
        lens = [3000, 0, 77, 1234]
        q, lam, w, out, lse = run(c, dtype, 0, [0, 1, 2, 3], lens, None, 8, norm=True)
        o2, l2 = c.attend_diff(0, ints([0, 1, 2, 3]), ints(lens), q, lam, 3000, norm=w, lse=True,
                               starts=ints(range(5)))
        assert float((o2.float() - out.float()).abs().max()) <= 2.0 ** -5 * float(out.float().abs().max())
        assert torch.allclose(lse, l2, rtol=1e-5, atol=1e-5)


def test_lambda_zero_is_the_first_map():
    c = filled(0, 1, 2, 64, 64, 1, 300)
    q = queries(20, 4, 64)
    out, lse = c.attend_diff(0, ints([0]), ints([300]), q, torch.zeros(4, device="cuda"), 300,
                             starts=ints([0, 20]), lse=True)
    q0 = q.clone()
    q0[..., 32:] = 0
    o1, l1 = c.attend_chunk(0, ints([0]), ints([300]), ints([0, 20]), q0, 300, scale=32 ** -0.5, lse=True)
    c.status()
    assert torch.allclose(out.float(), o1.float(), rtol=2.0 ** -6, atol=2.0 ** -6)
    assert torch.allclose(lse[..., 0], l1, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("new", [None, 60])
def test_values_that_are_not_seen_have_no_effect(new):
    c = filled(0, 1, 1, 128, 64, 1, 300)
    n = 290
    q, lam, w, out, lse = run(c, 0, 0, [0], [n], None if new is None else [new], 4)
    bad = c.pool.view(torch.bfloat16)
    for t in range(n, 300):
        bad[int(c.table[0, 0, 1, 0, t // 64]), t % 64] = math.nan
        bad[int(c.table[0, 0, 0, 0, t // 64]), t % 64] = math.inf
    call = lambda: c.attend_diff(0, ints([0]), ints([n]), q, lam, n, lse=True,  # noqa: E731
                                 starts=None if new is None else ints([0, new]))
    o2, l2 = call()
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    if new:
        bad[int(c.table[0, 0, 1, 0, 270 // 64]), 270 % 64, 3] = math.nan
        o2, l2 = call()
        assert torch.equal(l2, lse) and torch.equal(o2[:40], out[:40])
        assert torch.all(torch.isnan(o2[40:, :, 3]))
        assert torch.equal(o2[40:, :, 4:], out[40:, :, 4:])
    c.status()


def test_strides_in_place_and_padding():
    c = filled(0, 1, 2, 64, 16, 2, 90)
    g = torch.Generator(device="cuda").manual_seed(4)
    wide = torch.randn(3, 8, 80, generator=g, device="cuda").bfloat16()
    q = wide[:, 2:6, 8:72]
    q1 = q.contiguous()
    lam, w = weights(4, 64)
    args = (0, ints([1, -1, 0]), ints([90, 50, 33]))
    for starts in (None, ints([0, 1, 2, 3])):
        q1 = q.contiguous()
        want, lse = c.attend_diff(*args, q1, lam, 90, starts=starts, norm=w, lse=True)
        c.status()
        assert torch.all(want[1] == 0) and torch.all(lse[1] == -math.inf)
        assert torch.equal(c.attend_diff(*args, q, lam, 90, starts=starts, norm=w), want)
        assert c.attend_diff(*args, q1, lam, 90, starts=starts, norm=w, out=q1) is q1
        assert torch.equal(q1, want)


def test_bad_data_is_reported():
    P = skv()
    c = filled(0, 1, 2, 64, 16, 2, 90)
    q = queries(2, 4, 64)
    lam, _ = weights(4, 64)
    good = c.attend_diff(0, ints([1, 0]), ints([90, 33]), q, lam, 90)
    c.status()
    for slots, lens in (([1, 2], [90, 33]), ([1, 0], [90, -1]), ([1, 0], [90, 97])):
        out, lse = c.attend_diff(0, ints(slots), ints(lens), q, lam, 90, lse=True)
        with pytest.raises(P.SkvError):
            c.status()
        assert torch.equal(out[0], good[0]) and torch.all(out[1] == 0)
        assert torch.all(lse[1] == -math.inf)


@pytest.mark.parametrize("starts", [False, True])
def test_graph_streams_and_new_lengths(starts):
    c = filled(1, 1, 2, 128, 64, 2, 2000)
    q = queries(2, 8, 128, 4)
    lam, w = weights(8, 128)
    lens, slots = ints([0, 0]), ints([0, 1])
    st = ints([0, 1, 2]) if starts else None
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        out, lse = c.attend_diff(0, slots, lens, q, lam, 2000, starts=st, norm=w, lse=True)
    for n in ([2000, 1], [64, 0], [513, 1900]):
        lens.copy_(ints(n))
        graph.replay()
        other = c.attend_diff(0, slots, lens, q, lam, 2000, starts=st, norm=w, stream=torch.cuda.Stream())
        torch.cuda.synchronize()
        check(c, 1, 0, [0, 1], n, [0, 1, 2], q, out, lse, lam=lam, norm=w)
        assert torch.equal(other, out)


def test_many_sequences():
    n = 700
    c = filled(1, 1, 2, 64, 16, 50, 40)
    g = torch.Generator().manual_seed(0)
    lens = torch.randint(0, 41, (n,), generator=g).tolist()
    run(c, 1, 0, [i % 50 for i in range(n)], lens, None, 4, max_len=40)
    run(c, 1, 0, [i % 50 for i in range(n)], lens, [min(m, 3) for m in lens], 4, max_len=40)
