"""How exactly the softmax weights of attention meet the values.

Queries with one channel that is not zero make the scores exact (the matrix unit adds
zeros to one product, and what is multiplied here are few bits), so what is left of the
error are the roundings of the weights, of the sums and of the result:
  - the exponent's argument, one multiplication: 2^-23 * (|score| / ln 2), the exponential
    2^-22, the sums in fp32 with at most one cut of 2^-23 for each of n + 64 additions:
    e = (2 |score| + n + 80) * 2^-23, of the numerator and of the sum: 2 e;
  - the weight as an operand of the matrix unit: bf16 caches 2^-16 (two bf16 parts); e4m3
    caches 2^-11 (fp16), and where that is less, 2^-36 of the row's largest weight;
  - the result in bf16: 2^-8 of it (torch.finfo(bfloat16).eps / 2, and its own step)."""
import math

import pytest
import torch

from cache_helpers import ints, skv

FLOOR = 2.0 ** -36


def exact(q, k, v, scale):
    """q [d], k and v [n, d], float64: the result, sum w |v|, sum |v| / (sum of weights relative
    to the largest), lse, max |score|."""
    s = k @ q * scale
    w = torch.softmax(s, 0)
    total = torch.exp(s - s.max()).sum()
    return w @ v, w @ v.abs(), v.abs().sum(0) / total, torch.logsumexp(s, 0), float(s.abs().max())


def tolerance(dtype, n, ref, absw, absv, top):
    e = (2 * top + n + 80) * 2.0 ** -23
    tol = 2.0 ** -8 * ref.abs() + (2 * e + (2.0 ** -16 if dtype == 0 else 2.0 ** -11)) * absw
    return tol + (FLOOR * absv if dtype == 1 else 0) + 1e-30


def make_bf16(n, d, seed):
    """Keys and values [1, 2, 1, n, d], a query whose scores spread over a few units."""
    g = torch.Generator().manual_seed(seed)
    kv = torch.randn(2, n, d, generator=g).bfloat16()
    q = torch.zeros(d).bfloat16()
    q[3] = 8.0
    return kv[0], kv[1], q


def cut(p, bits):
    """float64 weights cut to `bits` significant bits."""
    m, e = torch.frexp(p)
    return torch.ldexp(torch.floor(m * 2.0 ** bits), e - bits)


def test_the_bound_for_bf16_caches_tells_one_part_from_two():
    """On the host: weights of 8 bits (one bf16 part) leave the bound, those of 16 keep it."""
    for seed in range(3):
        k, v, q = (x.double() for x in make_bf16(64, 128, seed))
        ref, absw, absv, _, top = exact(q, k, v, 128 ** -0.5)
        tol = tolerance(0, 64, ref, absw, absv, top)
        s = k @ q * 128 ** -0.5
        p = torch.exp(s - s.max())
        off = [(((cut(p, bits) @ v / p.sum()).bfloat16().double() - ref).abs() / tol).max()
               for bits in (8, 16)]
        assert off[0] > 1 and off[1] <= 1, off


def one_row(dtype, k, v, tb, batch=1):
    """A cache whose one sequence has these keys and values."""
    P = skv()
    n, d = k.shape
    blocks = -(-n // tb)
    pool = torch.zeros(2 * blocks, tb, d, dtype=k.dtype)
    pool.view(2, blocks * tb, d)[0, :n] = k
    pool.view(2, blocks * tb, d)[1, :n] = v
    pool = pool.view(torch.int16 if dtype == 0 else torch.uint8).cuda()
    table = torch.arange(2 * blocks, dtype=torch.int32, device="cuda").view(1, 1, 2, 1, blocks)
    return P.PagedCache(dtype, 1, 1, d, tb, pool=pool, table=table,
                        refs=torch.ones(2 * blocks, dtype=torch.int32, device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [16, 64, 400, 3000])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_weights_of_bf16_caches_keep_16_bits(n, d):
    for seed in range(3):
        k, v, q = make_bf16(n, d, seed)
        c = one_row(0, k, v, 32)
        out, lse = c.attend(0, ints([0]), ints([n]), q.view(1, 1, d).cuda(), n, lse=True)
        c.status()
        ref, absw, absv, rl, top = exact(q.double(), k.double(), v.double(), d ** -0.5)
        tol = tolerance(0, n, ref, absw, absv, top)
        off = (out[0, 0].double().cpu() - ref).abs()
        assert torch.all(off <= tol), float((off / tol).max())
        assert abs(float(lse) - float(rl)) <= (2 * top + n + 80) * 2.0 ** -23


def make_sink(n, d, code, at, seed):
    """Keys whose scores lie within half a unit of 0 but for one, `code` / 2 above, whose value
    is zero; the other values around 1."""
    g = torch.Generator().manual_seed(seed)
    k = torch.zeros(n, d)
    k[:, 5] = torch.rand(n, generator=g) * 2 - 1
    v = 0.5 + torch.rand(n, d, generator=g)
    k[at, 5], v[at] = code, 0.0
    q = torch.zeros(d).bfloat16()
    q[5] = 1.0
    return k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn), q


@pytest.mark.gpu
@pytest.mark.parametrize("code", [16, 24, 28, 32, 36, 40])       # 8 to 20 units
@pytest.mark.parametrize("n,d,batch", [(300, 128, 1), (600, 128, 1), (600, 64, 1), (300, 256, 2),
                                       (5003, 128, 1), (4100, 128, 1500)])
def test_weights_of_e4m3_caches_far_below_the_largest(n, d, batch, code):
    """A sink: one token takes nearly all of the weight and has no value, so the result is
    what the others add up to.  (With 1500 rows a block takes rows whole, so the sink's
    warp holds a quarter of them.)"""
    for at in (0, n // 2):
        k, v, q = make_sink(n, d, code, at, code + n)
        c = one_row(1, k, v, 64)
        out, lse = c.attend(0, ints([0] * batch), ints([n] * batch),
                            q.cuda().expand(batch, 1, d), n, scale=0.5, lse=True)
        c.status()
        ref, absw, absv, rl, top = exact(q.double(), k.double(), v.double(), 0.5)
        tol = tolerance(1, n, ref, absw, absv, top)
        off = (out[:, 0].double().cpu() - ref).abs()
        assert torch.all(off <= tol), float((off / tol).max())
        off = (lse.double().cpu() - rl).abs()
        assert float(off.max()) <= (2 * top + n + 80) * 2.0 ** -23
        assert math.isfinite(float(out.double().sum()))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("power", range(16, 31))
def test_scores_whose_steps_are_larger_than_one(dtype, power):
    """Scores of 2^16 to 2^31, growing along the row: the largest ones share the weight, all
    others are e^-1000 or less, and nothing overflows on the way."""
    n, d = 400, 128
    g = torch.Generator().manual_seed(power)
    v = torch.randn(n, d, generator=g)
    k = torch.zeros(n, d)
    k[:, 5] = 1 + (torch.arange(n) * 8 // n).float() / 8              # 1 to 1.875, in e4m3's steps
    order = torch.randperm(n, generator=g)
    for rows in (torch.arange(n), order):
        t = torch.bfloat16 if dtype == 0 else torch.float8_e4m3fn
        kk, vv = k[rows].to(t), v[rows].to(t)
        q = torch.zeros(d).bfloat16()
        q[5] = 2.0 ** power
        for sign in (1, -1):
            c = one_row(dtype, (sign * kk.float()).to(t), vv, 32)
            out, lse = c.attend(0, ints([0]), ints([n]), q.view(1, 1, d).cuda(), n, scale=1.0,
                                lse=True)
            c.status()
            best = kk[:, 5].float() == (1.875 if sign == 1 else 1.0)
            x = vv.double()[best]
            # equal weights: 2^-22 for the sums, 2^-8 for the result
            tol = 2.0 ** -8 * x.mean(0).abs() + 2.0 ** -20 * x.abs().mean(0)
            assert torch.all((out[0, 0].double().cpu() - x.mean(0)).abs() <= tol)
            want = sign * (1.875 if sign == 1 else 1.0) * 2.0 ** power + math.log(len(x))
            assert abs(float(lse) - want) <= 2.0 ** -21 * abs(want)
