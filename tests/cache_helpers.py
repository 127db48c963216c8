"""Plain 64-bit forms of the paged cache's operators, and caches to run them on."""
import math

import numpy as np
import torch

NO = 0xFFFFFFFF


def skv():
    import lossless_kv_cache_fixed_gb300 as P
    P.build()
    return P


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Pages:
    """Table and counts of a cache on the host, with the page operations in plain loops.
    pool [pages, tokens, d] holds page contents."""

    def __init__(self, cache):
        self.table = cache.table.cpu().numpy().view(np.uint32).copy()
        self.refs = cache.refs.cpu().numpy().copy()
        self.pool = cache.pool.cpu().numpy().copy()
        self.tb = cache.page_tokens

    def rows(self, slot):
        return self.table[slot].reshape(-1, self.table.shape[-1])

    def lowest(self):
        return int(np.flatnonzero(self.refs == 0)[0])

    def reserve(self, slots, old, new):
        for s, a, b in zip(slots, old, new):
            for row in self.rows(s):
                for blk in range(-(-a // self.tb), -(-b // self.tb)):
                    assert row[blk] == NO
                    row[blk] = p = self.lowest()
                    self.refs[p] = 1

    def fork(self, parents, children, lens):
        for p, c, n in zip(parents, children, lens):
            full, tail = divmod(n, self.tb)
            for src, dst in zip(self.rows(p), self.rows(c)):
                for blk in range(full):
                    dst[blk] = src[blk]
                    self.refs[src[blk]] += 1
                if tail:
                    q = self.lowest()
                    dst[full] = q
                    self.refs[q] = 1
                    self.pool[q, :tail] = self.pool[src[full], :tail]

    def free(self, slots):
        for s in slots:
            for row in self.rows(s):
                for p in row[row != NO]:
                    self.refs[p] -= 1
                row[:] = NO

    def compact(self):
        live = int((self.refs > 0).sum())
        moved = {}
        while True:
            holes = np.flatnonzero(self.refs[:live] == 0)
            if not len(holes):
                break
            h, p = int(holes[0]), int(np.flatnonzero(self.refs > 0)[-1])
            self.refs[h], self.refs[p] = self.refs[p], 0
            self.pool[h] = self.pool[p]
            moved[p] = h
        for p, h in moved.items():
            self.table[self.table == p] = h

    def same(self, table, refs, pool):
        assert np.array_equal(table.cpu().numpy().view(np.uint32), self.table)
        assert np.array_equal(refs.cpu().numpy(), self.refs)
        if pool is not None:
            assert np.array_equal(pool.cpu().numpy(), self.pool)


def values(pool, dtype):
    """Page contents as float64."""
    if dtype == 0:
        return pool.view(torch.bfloat16).double()
    return pool.view(torch.float8_e4m3fn).double()


def attend64(cache, dtype, layer, slot, a, n, q, scale):
    """One sequence in float64: out [q_heads, d], lse [q_heads] and, for the tolerances,
    sum_t w_t |v_t|, max_t scale * sum_d |q_d k_d|, max over channels of |v|, sum over tokens."""
    hq, d = q.shape
    h = cache.heads
    g = hq // h
    out = torch.zeros(hq, d, dtype=torch.float64)
    absw, absv = torch.zeros(hq, d).double(), torch.zeros(hq, d).double()
    lse = torch.full((hq,), -math.inf, dtype=torch.float64)
    mag = torch.zeros(hq, dtype=torch.float64)
    if n > a:
        tab = cache.table[slot, layer].cpu().long()
        for i in range(hq):
            kv = []
            for side in (0, 1):
                t = torch.arange(a, n)
                page = tab[side, i // g, t // cache.page_tokens]
                x = values(cache.pool[page.cuda(), (t % cache.page_tokens).cuda()], dtype).cpu()
                if cache.scale is not None:
                    x = x * cache.scale[layer, i // g].double().cpu()
                kv.append(x)
            qd = q[i].double().cpu()
            s = kv[0] @ qd * scale
            mag[i] = (kv[0].abs() @ qd.abs() * abs(scale)).max()
            lse[i] = torch.logsumexp(s, 0)
            w = torch.softmax(s, 0)
            out[i] = w @ kv[1]
            absw[i] = w @ kv[1].abs()
            absv[i] = kv[1].abs().sum(0)
    return out, lse, absw, absv, mag


def check_attend(cache, dtype, layer, slots, begins, lens, q, scale, out, lse):
    """out and lse against float64, within what the roundings allow.

    Scores: exact products summed in fp32 by the matrix unit, whose additions may cut
    instead of round (2^-23 each), one multiplication and the exponential (2^-22): the
    weights are off by e = (d + 8) * 2^-23 * max_t sum_d |q_d k_d| * scale + (tokens + 64)
    * 2^-23 relative (their sum is taken in fp32).  Weights round to bf16 (2^-8) or, for
    e4m3, to fp16 (2^-11, and 2^-25 absolute below its normal range; q's channels below
    2^-24 of the largest likewise enter through e, doubled for it).  The result rounds
    to bf16 (2^-8)."""
    d = q.shape[2]
    for b, (s, a, n) in enumerate(zip(slots, begins, lens)):
        ref, rl, absw, absv, mag = attend64(cache, dtype, layer, s, a, n, q[b], scale)
        got, gl = out[b].double().cpu(), lse[b].double().cpu()
        if n <= a:
            assert torch.all(got == 0) and torch.all(gl == -math.inf)
            continue
        e = (2 * (d + 8) * mag + (n - a) + 64) * 2.0 ** -23
        p = 2.0 ** -8 if dtype == 0 else 2.0 ** -11
        tol = (p + 2 * e[:, None]) * absw + 2.0 ** -8 * ref.abs() + 1e-30
        if dtype == 1:
            tol = tol + 2.0 ** -25 * absv
        assert torch.all((got - ref).abs() <= tol), (b, ((got - ref).abs() / tol).max())
        assert torch.all((gl - rl).abs() <= e + 2.0 ** -22 * rl.abs()), (b, (gl - rl).abs().max())
