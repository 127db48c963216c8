"""Plain 64-bit forms of attention of chunks of new tokens and of differential attention
over a paged cache, and the tolerances that the roundings allow.

Scores: exact products summed in fp32 by the matrix unit, whose additions may cut instead
of round (2^-23 each), one multiplication and the exponential (2^-22): the weights are off by
e = (2 (d + 8) * max_t sum_d |q_d k_d| * scale + tokens + 64) * 2^-23 relative (their sum is
taken in fp32).  e4m3: q is held in fp16 after a power of two per row, which leaves at most
2^-25 of its largest channel in each: e grows by that times sum_d |k_d|.  Weights round to
bf16 (2^-8) or, for e4m3, to fp16 (2^-11; where that is more, half of fp16's smallest step, 2^-25,
with the row's largest weight at 2^8 or above: 2^-33 of that one).  The result rounds to bf16 (2^-8)."""
import math

import torch

from cache_helpers import values


def rows_of(cache, dtype, layer, slot, head, n):
    """Keys and values [n, d] of one head of a sequence, float64."""
    t = torch.arange(n, device="cuda")
    res = []
    for side in (0, 1):
        page = cache.table[slot, layer, side, head].long()[t // cache.page_tokens]
        x = values(cache.pool[page, t % cache.page_tokens], dtype)
        if cache.scale is not None:
            x = x * cache.scale[layer, head].double()
        res.append(x)
    return res


def seen(at, n, begin, window, causal):
    """[rows, n]: which of a sequence's n tokens the rows at these places see."""
    t = torch.arange(n, device="cuda")
    at = at[:, None]
    ok = (t >= max(begin, 0)) & (at >= 0)
    if causal:
        ok = ok & (t <= at)
    if window:
        ok = ok & (t > at - window)
    return ok


def one_map(dtype, q, k, v, ok, scale):
    """q [rows, width], k [n, width], v [n, d], ok [rows, n]: the result and its log-sum in
    64 bits, and how far each may be off before the last rounding."""
    n, width = k.shape
    s = (q @ k.T * scale).masked_fill(~ok, -math.inf)
    lse = torch.logsumexp(s, 1)
    none = ~ok.any(1)
    w = torch.softmax(s, 1)
    w[none] = 0
    top = torch.where(none, 0.0, s.amax(1))
    least = torch.exp(torch.where(none, 0.0, top - lse))       # the largest weight
    out, absw = w @ v, w @ v.abs()
    absv = (ok.double() @ v.abs()) * least[:, None]
    mag = ((q.abs() @ k.abs().T) * abs(scale)).masked_fill(~ok, 0).amax(1)
    e = (2 * (width + 8) * mag + n + 64) * 2.0 ** -23
    if dtype == 1:
        e = e + 2.0 ** -25 * q.abs().amax(1) * k.abs().sum(1).amax() * abs(scale)
    p = 2.0 ** -8 if dtype == 0 else 2.0 ** -11
    tol = (p + 2 * e[:, None]) * absw + (2.0 ** -33 * absv if dtype == 1 else 0) + 1e-30
    return out, lse, tol, e + 2.0 ** -22 * torch.where(none, 0.0, lse.abs())


def check(cache, dtype, layer, slots, lens, starts, q, out, lse, begins=None, window=0, causal=True,
          scale=None, lam=None, norm=None, eps=1e-5, heads=None):
    """out and lse of attend_chunk (lam None) or attend_diff against 64 bits; heads: only these."""
    hq, d = q.shape[1:]
    g = hq // cache.heads
    maps = 1 if lam is None else 2
    width = d // maps
    scale = width ** -0.5 if scale is None else scale
    starts = list(range(len(slots) + 1)) if starts is None else starts
    for i, slot in enumerate(slots):
        a, z = starts[i], starts[i + 1]
        n = lens[i]
        if z == a:
            continue
        for h in range(hq) if heads is None else heads:
            got = out[a:z, h].double()
            gl = (lse[a:z, h] if maps == 2 else lse[a:z, h, None]).double()
            if slot < 0 or n == 0:
                assert torch.all(got == 0) and torch.all(gl == -math.inf)
                continue
            k, v = rows_of(cache, dtype, layer, slot, h // g, n)
            ok = seen(n - (z - torch.arange(a, z, device="cuda")), n,
                      begins[i] if begins is not None else 0, window, causal)
            k, v = k.masked_fill(~ok.any(0)[:, None], 0), v.masked_fill(~ok.any(0)[:, None], 0)
            ref = tol = None
            for m in range(maps):
                part = slice(m * width, (m + 1) * width)
                o, rl, t, tl = one_map(dtype, q[a:z, h, part].double(), k[:, part], v, ok, scale)
                off = (gl[:, m] - rl).abs()
                some = ok.any(1)
                assert torch.all(gl[~some, m] == -math.inf)
                assert torch.all(off[some] <= tl[some]), (i, h, m, float((off / tl)[some].max()))
                f = float(lam[h]) if m else 1.0
                ref, tol = (o, t) if not m else (ref - f * o, tol + abs(f) * t)
            tol = tol + 2.0 ** -22 * ref.abs()
            if norm is not None:
                # (a bound that is as large as the result says nothing: see check_norm)
                # R = sqrt(mean o^2 + eps) is a 2-norm of (o / sqrt(d), sqrt(eps)), so by the triangle
                # inequality it is off by at most T = sqrt(mean tol^2), and o / R by at most
                # (|o| + tol) / (R - T) - |o| / R; 2^-20 for the mean, the root and two products
                r = torch.rsqrt(ref.square().mean(1, keepdim=True) + eps)
                t = tol.square().mean(1, keepdim=True).sqrt()
                tol = norm.double().abs() * ((ref.abs() + tol) / (1 / r - t) - ref.abs() * r +
                                             2.0 ** -20 * r * ref.abs())
                tol = torch.where(r * t < 0.5, tol, math.inf)
                ref = ref * r * norm.double()
            tol = tol + 2.0 ** -8 * ref.abs()
            off = (got - ref).abs()
            assert torch.all(got[~ok.any(1)] == 0)
            assert torch.all(off <= tol), (i, h, float((off / tol).max()))


def check_norm(plain, normed, norm, eps=1e-5):
    """The result with a norm against the one without, whose rounding (2^-8 of each channel)
    enters as tol does above; the last rounding 2^-8."""
    o = plain.double()
    r = torch.rsqrt(o.square().mean(-1, keepdim=True) + eps)
    t = 2.0 ** -8 * o.square().mean(-1, keepdim=True).sqrt()
    ref = o * r * norm.double()
    tol = norm.double().abs() * o.abs() * ((1 + 2.0 ** -8) / (1 / r - t) - r + 2.0 ** -20 * r)
    assert torch.all((normed.double() - ref).abs() <= tol + 2.0 ** -8 * (ref.abs() + tol) + 1e-30)
