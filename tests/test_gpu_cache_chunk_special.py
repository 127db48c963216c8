"""Infinities, NaN and scores beyond the ordinary that rows do see, in chunk and differential
attention.  What exact arithmetic gives is asked for, whatever route the row takes: in one block
of threads or several, in one tile or two, one token or a chunk."""
import math

import pytest
import torch

from cache_helpers import ints
from chunk_helpers import one_map, rows_of, seen
from test_gpu_cache_attend import filled
from test_gpu_cache_chunk import queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def place(c, side, t, head=0):
    """A token's row of the pool, layer 0 of sequence 0."""
    tb = c.page_tokens
    pool = c.pool.view(torch.bfloat16) if c.pool.dtype == torch.int16 else c.pool
    return pool[int(c.table[0, 0, side, head, t // tb]), t % tb]


FORMS = [(300, None), (9000, None), (150, 60), (300, 40), (300, 150), (9000, 40), (2500, 300)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,new", FORMS)
def test_an_infinite_value_with_a_norm(d, n, new):
    """Heads with lambda above, below and at 0.  The difference is NaN, infinite and NaN in the value's
    channel; with a norm the root of the mean square is infinite or NaN with it."""
    c = filled(0, 1, 1, d, 64, 1, n)
    rows = new or 1
    q = queries(rows, 3, d)
    lam = torch.tensor([0.5, -0.5, 0.0], device="cuda")
    norm = torch.rand(d, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") + 0.2
    args = (0, ints([0]), ints([n]), q, lam, n)
    starts = None if new is None else ints([0, new])
    plain, lse = c.attend_diff(*args, starts=starts, lse=True)
    normed = c.attend_diff(*args, starts=starts, norm=norm)
    t = n - rows // 2 - 1
    place(c, 1, t)[5] = math.inf
    first = t - (n - rows)                         # rows from here on see it
    rest = [i for i in range(d) if i != 5]
    o, l = c.attend_diff(*args, starts=starts, lse=True)
    assert torch.equal(l, lse) and torch.equal(o[:first], plain[:first])
    assert torch.equal(o[first:][:, :, rest], plain[first:][:, :, rest])
    assert torch.all(torch.isnan(o[first:, 0, 5])) and torch.all(torch.isnan(o[first:, 2, 5]))
    assert torch.all(o[first:, 1, 5] == math.inf)
    o = c.attend_diff(*args, starts=starts, norm=norm)
    assert torch.equal(o[:first], normed[:first])
    assert torch.all(torch.isnan(o[first:, 0])) and torch.all(torch.isnan(o[first:, 2]))
    assert torch.all(torch.isnan(o[first:, 1, 5])) and torch.all(o[first:, 1][:, rest] == 0)
    c.status()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,new", FORMS)
@pytest.mark.parametrize("power", [-120, -60, -20, 40, 64, 90])
def test_the_norm_of_small_and_large_results(d, n, new, power):
    """Without eps the normalised result does not change when all values take the same power of two,
    although the squares of the results leave the range of a float."""
    c = filled(0, 1, 1, d, 64, 1, n)
    rows = new or 1
    q = queries(rows, 2, d)
    lam = torch.tensor([0.5, -0.5], device="cuda")
    norm = torch.rand(d, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") + 0.2
    args = (0, ints([0]), ints([n]), q, lam, n)
    more = dict(starts=None if new is None else ints([0, new]), norm=norm)
    v = c.table[0, 0, 1, 0].long()
    pool = c.pool.view(torch.bfloat16)
    x = pool[v]
    pool[v] = torch.where(x.abs() < 2.0 ** -5, 0.0, x)     # (no power of two makes a subnormal)
    want = c.attend_diff(*args, eps=0.0, **more)
    one = c.attend_diff(*args, eps=1e-5, **more)
    pool[v] = (pool[v].float() * 2.0 ** power).bfloat16()
    got = c.attend_diff(*args, eps=0.0, **more)
    assert torch.all(torch.isfinite(want)) and torch.any(want != 0)
    # (2^-22 of the sum of squares and of each product; half a step of bf16 on either side)
    off = (got.double() - want.double()).abs()
    assert torch.all(off <= 2.0 ** -7 * want.double().abs() + 2.0 ** -18)
    # with eps: large results do not feel it, small ones have the root of eps for a divisor
    got = c.attend_diff(*args, eps=1e-5, **more).double()
    if power > 0:
        assert torch.all((got - want.double()).abs() <= 2.0 ** -7 * want.double().abs() + 2.0 ** -18)
    elif power < -20:
        plain = c.attend_diff(*args, eps=0.0, starts=more["starts"]).double()
        ref = plain * norm.double() / math.sqrt(1e-5)
        # (`plain` is bf16: below 2^-126 its half step is 2^-134 whatever its size, which enters times
        # norm / sqrt(eps); the same of the result itself)
        half = 2.0 ** -134
        assert torch.all((got - ref).abs() <= 2.0 ** -7 * ref.abs() + half * (norm.double() / math.sqrt(1e-5) + 2))
    assert torch.all(torch.isfinite(one))
    c.status()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,new", [(300, 5), (3000, 5), (20000, 60), (3000, 100)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_values_of_tokens_whose_weight_is_next_to_nothing(d, n, new, bad):
    """Scores of the odd blocks lie 150 below those of the even ones; an infinity or NaN among the
    values of the former is not lost, other channels keep their bits."""
    c = filled(0, 1, 1, d, 64, 1, n)
    for t in range(n):
        place(c, 0, t).zero_()
        place(c, 0, t)[0] = 0.0 if t // 128 % 2 else 150.0
    q = torch.zeros(new, 2, d, device="cuda").bfloat16()
    q[:, :, 0] = 1.0
    args = (0, ints([0]), ints([n]), ints([0, new]), q, n)
    out, lse = c.attend_chunk(*args, scale=1.0, lse=True)
    place(c, 1, 131)[7] = bad
    o, l = c.attend_chunk(*args, scale=1.0, lse=True)
    rest = [i for i in range(d) if i != 7]
    assert torch.equal(l, lse) and torch.equal(o[:, :, rest], out[:, :, rest])
    assert not torch.any(torch.isfinite(o[:, :, 7]))
    c.status()


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [4, 90])
@pytest.mark.parametrize("n", [600, 5000])
def test_scores_that_get_huge_next_to_rows_whose_are(dtype, d, new, n):
    """Of two heads, neighbours in a warp, one has huge scores from the first token on, the other from
    token 400 on, which takes all of the weight: its result is that token's value."""
    c = filled(dtype, 1, 1, d, 64, 1, n, scaled=False)
    for t in range(n):
        row = place(c, 0, t)
        row.zero_()
        row[0] = 1.0 if dtype == 0 else 0x38           # 1
    place(c, 0, 400)[1] = 2.0 ** 14 if dtype == 0 else 0x7E      # 448
    q = torch.zeros(new, 2, d, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(6)
    q[:, 0, 0] = 2.0 ** 25
    q[:, 1, 1] = 2.0 ** 26 * (1 + 63 / 64 * torch.rand(new, generator=g, device="cuda")) * (1 if dtype == 0 else 2.0 ** 4)
    q = q.bfloat16()
    args = (0, ints([0]), ints([n]), ints([0, new]))
    out, lse = c.attend_chunk(*args, q, n, lse=True)
    k, v = rows_of(c, dtype, 0, 0, 0, n)
    assert torch.equal(out[:, 1].double(), v[400].expand(new, d))
    want = q[:, 1, 1].double() * k[400, 1] * d ** -0.5
    assert torch.all((lse[:, 1].double() - want).abs() <= 2.0 ** -21 * want)
    calm = q.clone()
    calm[:, 0, 0] = 1.0
    o, l = c.attend_chunk(*args, calm, n, lse=True)        # the other head does not matter
    assert torch.equal(o[:, 1], out[:, 1]) and torch.equal(l[:, 1], lse[:, 1])
    c.status()


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [16, 48, 64, 80, 128, 192, 256])
@pytest.mark.parametrize("n,new", FORMS)
@pytest.mark.parametrize("half", [0, 1])
def test_keys_that_are_not_finite_in_one_half(dtype, d, n, new, half):
    """An infinity that gives a token no weight in one map, or a NaN, has no effect on the other map."""
    c = filled(dtype, 1, 1, d, 64, 1, n, seed=d)
    rows = new or 1
    q = queries(rows, 3, d, 5)
    lam = torch.tensor([0.5, -0.3, 1.1], device="cuda")
    ch = half * d // 2 + d // 2 - 1
    q[:, :, ch] = q[:, :, ch].abs() + 0.1
    args = (0, ints([0]), ints([n]), q, lam, n)
    starts = None if new is None else ints([0, new])
    k, v = rows_of(c, dtype, 0, 0, 0, n)
    ok = seen(n - rows + torch.arange(rows, device="cuda"), n, 0, 0, True)
    at = torch.cat([torch.arange(2, n, 61), torch.tensor([n - rows])]).tolist()
    for t in at:
        if dtype == 0:
            place(c, 0, t)[ch] = -math.inf
        else:
            place(c, 0, t)[ch] = 0x7F
    o, l = c.attend_diff(*args, starts=starts, lse=True)
    there = ok.clone()
    there[:, at] = False                               # what the map with the infinities sees
    for h in range(3):
        res = []
        for m in (0, 1):
            part = slice(m * d // 2, (m + 1) * d // 2)
            see = there if m == half and dtype == 0 else ok
            w = k.clone()
            w[at, ch] = 0.0 if m == half else w[at, ch]
            res.append(one_map(dtype, q[:, h, part].double(), w[:, part], v, see, (d // 2) ** -0.5))
            if m != half or dtype == 0:
                assert torch.all((l[:, h, m].double() - res[m][1]).abs() <= res[m][3]), (h, m)
        if dtype == 0:
            f = float(lam[h])
            ref = res[0][0] - f * res[1][0]
            tol = res[0][2] + abs(f) * res[1][2] + 2.0 ** -22 * ref.abs()
            assert torch.all((o[:, h].double() - ref).abs() <= tol + 2.0 ** -8 * (ref.abs() + tol)), h
        else:
            last = ok[:, at].any(1)
            assert torch.all(torch.isnan(l[last, h, half])) and torch.all(torch.isnan(o[last, h]))
    # a NaN: its map and the result are NaN where the token is seen
    t = n - rows // 2 - 1
    place(c, 0, t)[ch] = math.nan if dtype == 0 else 0xFF
    o2, l2 = c.attend_diff(*args, starts=starts, lse=True)
    first = t - (n - rows)
    assert torch.all(torch.isnan(o2[first:])) and torch.all(torch.isnan(l2[first:, :, half]))
    for h in range(3):
        m = 1 - half
        part = slice(m * d // 2, (m + 1) * d // 2)
        _, rl, _, tl = one_map(dtype, q[:, h, part].double(), k[:, part], v, ok, (d // 2) ** -0.5)
        assert torch.all((l2[:, h, m].double() - rl).abs() <= tl)
    c.status()


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 256])
def test_the_c_call_without_starts(dtype, d):
    """starts NULL: one new token per sequence, as starts = 0 .. batch."""
    import ctypes

    from cache_helpers import skv
    P = skv()
    lens = [3000, 0, 77, 1234, 1]
    c = filled(dtype, 1, 2, d, 64, 5, 3000)
    q = queries(5, 8, d)
    slots, n = ints([4, 2, 0, 1, 3]), ints(lens)
    want, wl = c.attend_chunk(0, slots, n, ints(range(6)), q, 3000, lse=True)
    out, lse = torch.empty_like(want), torch.empty_like(wl)
    nb = P.skv_cache_attend_chunk_workspace_bytes(c.struct, 8)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    k = P.SkvChunk(5, 5, 3000, 0, 0, 0, slots.data_ptr(), n.data_ptr(), None, None)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    rc = P.skv_cache_attend_chunk(c.struct, 0, k, q.data_ptr(), q.stride(0), q.stride(1), 8, d ** -0.5,
                                  out.data_ptr(), lse.data_ptr(), ws.data_ptr(), nb, stream)
    assert rc == P.SKV_OK
    c.status()
    assert torch.equal(out, want) and torch.equal(lse, wl)
