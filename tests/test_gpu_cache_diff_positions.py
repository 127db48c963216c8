"""Append with rotary positions, then differential attention of a chunk and of single tokens."""
import math

import pytest
import torch

from cache_helpers import ints, skv
from chunk_helpers import check, rows_of, seen
from test_gpu_cache_chunk import starts_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


H, GROUP = 2, 3


def cache_and_rope(dtype, d, interleaved=True):
    P = skv()
    scale = torch.full((1, H), 0.02, device="cuda") if dtype else None
    c = P.PagedCache(dtype, 1, H, d, 32, num_pages=64, max_seqs=2, max_blocks=6, scale=scale)
    c.pool.zero_()
    half = 1e4 ** (-2.0 * torch.arange(d // 4, device="cuda").double() / (d // 2))
    return c, P.Rope(half.repeat(2), interleaved=interleaved)


def grow(c, rope, lens, news, g, shift=0):
    """The new tokens of two sequences appended: their lengths and turned queries."""
    new = [a + b for a, b in zip(lens, news)]
    c.reserve(ints([0, 1]), ints(lens), ints(new))
    qkv = torch.randn(sum(news), H * (GROUP + 2), c.head_dim, generator=g, device="cuda").bfloat16()
    q, k, v = qkv.split([H * GROUP, H, H], 1)
    slots = ints([0] * news[0] + [1] * news[1])
    at = ints(list(range(lens[0], new[0])) + list(range(lens[1], new[1])))
    return new, c.append(0, slots, at, q, k, v, rope, (at + shift).view(1, -1))


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 96, 256])
def test_a_run_of_append_chunk_and_single_tokens(dtype, d):
    c, rope = cache_and_rope(dtype, d)
    g = torch.Generator(device="cuda").manual_seed(3)
    lam = torch.rand(H * GROUP, generator=g, device="cuda")
    lens = [0, 0]
    for news in ([70, 33], [40, 50], [1, 1], [1, 1]):
        lens, q = grow(c, rope, lens, news, g)
        starts = starts_of(news)
        out, lse = c.attend_diff(0, ints([0, 1]), ints(lens), q, lam, max(lens), starts=ints(starts), lse=True)
        c.status()
        check(c, dtype, 0, [0, 1], lens, starts, q, out, lse, lam=lam)
        if news == [1, 1]:
            out, lse = c.attend_diff(0, ints([0, 1]), ints(lens), q, lam, max(lens), lse=True)
            c.status()
            check(c, dtype, 0, [0, 1], lens, starts, q, out, lse, lam=lam)


@pytest.mark.parametrize("d", [64, 256])
def test_only_the_distance_of_two_tokens_counts(d):
    """All positions moved by the same number: both maps' results stay within the roundings of the turned
    queries and keys (2^-8 of each channel, so 2^-7 + 2^-16 of sum |q_d k_d| per score and run, where
    a pair's two products are at most the product of its lengths) and of weights and results."""
    res = []
    for shift, kind in ((0, True), (777, True), (0, False), (777, False)):
        c, rope = cache_and_rope(0, d, kind)
        g = torch.Generator(device="cuda").manual_seed(5)
        lens, q = grow(c, rope, [0, 0], [120, 77], g, shift)
        lam = torch.full((H * GROUP,), 0.7, device="cuda")
        out, lse = c.attend_diff(0, ints([0, 1]), ints(lens), q, lam, max(lens), starts=ints([0, 120, 197]),
                                 lse=True)
        c.status()
        res.append((c, q, out.double(), lse.double()))
    c, q, out, lse = res[0]
    scale = (d // 2) ** -0.5
    apart = 0.0                                     # of pairs in both halves, in bounds
    for i, (a, z) in enumerate(((0, 120), (120, 197))):
        n = z - a
        ok = seen(torch.arange(n, device="cuda"), n, 0, 0, True)
        for h in range(H * GROUP):
            k, v = rows_of(c, 0, 0, i, h // GROUP, n)
            tol = 0
            for m in (0, 1):
                part = slice(m * d // 2, (m + 1) * d // 2)
                qh, kh = q[a:z, h, part].double(), k[:, part]
                most = qh.view(n, -1, 2).norm(dim=2) @ kh.view(n, -1, 2).norm(dim=2).T
                e = 2 * (2.0 ** -7 + 2.0 ** -16) * scale * most.masked_fill(~ok, 0).amax(1)
                w = torch.softmax((qh @ kh.T * scale).masked_fill(~ok, -math.inf), 1)
                apart = max(apart, float(((res[3][3] - res[2][3])[a:z, h, m].abs() / (e + 2.0 ** -12)).max()))
                assert torch.all((res[1][3][a:z, h, m] - lse[a:z, h, m]).abs() <= e + 2.0 ** -12)
                near = torch.expm1(2 * e)[:, None] + 2 * 2.0 ** -8
                tol = tol + (1.0 if m == 0 else 0.7) * near * (w @ v.abs())
            off = (res[1][2][a:z, h] - out[a:z, h]).abs()
            assert torch.all(off <= tol + 2 * 2.0 ** -8 * (out[a:z, h].abs() + tol))
    assert apart > 2.0                              # the other kind of pairs is seen by this test
