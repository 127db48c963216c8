#!/usr/bin/env python3
"""From a coded cache in host memory to decoding on its pages.

A prompt's cache is encoded, its container kept in pinned host memory, and later
decoded straight into the pages of a serving cache.  The sequence is forked into
continuations that share the prompt's full pages, every continuation appends new
tokens (rotary positions, keys and values written to their pages) and attends to
its cache; then all but one are dropped, the pool is compacted and the last one goes
on.  Every step is checked against plain torch.

    python examples/paged_decode.py [--e4m3] [--tokens 700] [--steps 3] [--branches 3]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import lossless_kv_cache_fixed_gb300 as P  # noqa: E402
import synth  # noqa: E402


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def coded_prompt(spec):
    """The prompt's cache, its predictions, the codec and the container (pinned host)."""
    w = synth.make(spec, device="cuda")
    ecdf = phat = None
    if spec.dtype == synth.BF16:
        import numpy as np
        E, ph = P.skv_build_ecdf(w.counts.cpu().numpy().astype(np.uint64))
        ecdf, phat = torch.from_numpy(E.view(np.int32)).cuda(), torch.from_numpy(ph).cuda()
    codec = P.Codec(spec.dtype, spec.L, spec.H, spec.T, spec.D, spec.Tb, spec.G, w.sigma, ecdf, phat)
    kv = w.kv.view(torch.int16) if spec.dtype == synth.BF16 else w.kv
    mu = w.mu.view(torch.int16)
    buf, nbytes = codec.encode(kv, mu)
    host = torch.empty(nbytes, dtype=torch.uint8).pin_memory()
    host.copy_(buf[:nbytes])
    print("prompt of %d tokens: %.1f MB coded as %.1f MB" % (
        spec.T, kv.numel() * kv.element_size() / 1e6, nbytes / 1e6))
    return w, kv, mu, codec, host


def paged(x, table, pages, page_tokens):
    """[L, 2, H, T, D] laid out in the pages that `table` [L, 2, H, blocks] names."""
    blocks = table.shape[-1]
    pad = blocks * page_tokens - x.shape[3]
    x = torch.nn.functional.pad(x, (0, 0, 0, pad)).view(-1, page_tokens, x.shape[4])
    pool = torch.zeros((pages, page_tokens, x.shape[2]), dtype=x.dtype, device=x.device)
    pool[table.reshape(-1).long()] = x
    return pool


def values(cache, slot, layer, side, head, n):
    """Plain form: the first n rows of one head of a sequence, float64."""
    t = torch.arange(n, device="cuda")
    page = cache.table[slot, layer, side, head][t // cache.page_tokens].long()
    x = cache.pool[page, t % cache.page_tokens]
    x = x.view(torch.bfloat16).double() if x.dtype == torch.int16 else \
        x.view(torch.float8_e4m3fn).double()
    return x if cache.scale is None else x * cache.scale[layer, head].double()


def check_attention(cache, layer, slots, lens, q, out):
    group = q.shape[1] // cache.heads
    for b, (slot, n) in enumerate(zip(slots, lens)):
        for h in range(q.shape[1]):
            k, v = (values(cache, slot, layer, s, h // group, n) for s in (0, 1))
            w = torch.softmax(k @ q[b, h].double() / math.sqrt(cache.head_dim), 0)
            off = (out[b, h].double() - w @ v).abs() / (w @ v.abs())
            assert float(off.max()) < 2.0 ** -7, float(off.max())


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--e4m3", action="store_true")
    ap.add_argument("--tokens", type=int, default=700)
    ap.add_argument("--steps", type=int, default=3)
    ap.add_argument("--branches", type=int, default=3)
    a = ap.parse_args(argv)
    base = synth.WORKLOADS["qwen3-0.6b-e4m3" if a.e4m3 else "qwen3-0.6b-bf16"]
    spec = base.scaled(name="paged-decode", L=2, H=2, T=a.tokens, calib_draws=min(2, base.calib_draws))
    group, n = 2, a.tokens
    w, kv, mu, codec, host = coded_prompt(spec)

    # a cache with room for the prompt and its branches; slot 0 takes the prompt
    rows = spec.L * 2 * spec.H
    blocks = -(-(n + a.steps + 1) // spec.Tb)
    cache = P.PagedCache(spec.dtype, spec.L, spec.H, spec.D, spec.Tb,
                         num_pages=rows * (blocks + 2 * a.branches) + 5, max_seqs=1 + a.branches,
                         max_blocks=blocks,
                         scale=None if w.fp8_scale is None else w.fp8_scale.float().contiguous())
    cache.pool.zero_()
    cache.reserve(i32([0]), i32([0]), i32([n]))
    cache.status()

    # decode from the host container into those pages (the predictions lie in pages, too)
    used = cache.table[0][..., :-(-n // spec.Tb)]
    mu_pool = paged(mu, used, cache.pool.shape[0], spec.Tb)
    pages = cache.page_of_chunk(0, n)
    codec.decode_range(host, host.numel(), 0, codec.num_chunks(), mu_pool, cache.pool, pages=pages,
                       num_pages=cache.pool.shape[0], first=True)
    codec.decode_status()
    assert torch.equal(paged(kv, used, cache.pool.shape[0], spec.Tb), cache.pool)
    print("decoded into %d pages, exact" % pages.numel())

    # fork: full pages are shared, the last one is copied
    branches = list(range(1, 1 + a.branches))
    cache.fork(i32([0] * a.branches), i32(branches), i32([n] * a.branches))
    cache.free(i32([0]))
    cache.status()
    print("%d branches on %d pages" % (a.branches, int((cache.refs > 0).sum())))

    # decode steps: room, append (positions on time, height, width; text: all the same), attend
    pairs = spec.D // 2
    freqs = 1e6 ** (-2.0 * torch.arange(pairs, device="cuda").double() / spec.D)
    axis = (torch.arange(pairs, device="cuda") % 3).to(torch.uint8)
    rope = P.Rope(freqs, axis, axes=3)
    g = torch.Generator(device="cuda").manual_seed(0)

    def step(slots, length):
        m = len(slots)
        s, at = i32(slots), i32([length] * m)
        cache.reserve(s, at, at + 1)
        for layer in range(spec.L):
            heads = spec.H * (group + 2)
            qkv = torch.randn(m, heads, spec.D, generator=g, device="cuda").bfloat16()
            q, k, v = qkv.split([spec.H * group, spec.H, spec.H], 1)
            q = cache.append(layer, s, at, q, k, v, rope, at.expand(3, m).contiguous())
            out = cache.attend(layer, s, at + 1, q, length + 1)
            check_attention(cache, layer, slots, [length + 1] * m, q, out)
        cache.status()

    for i in range(a.steps):
        step(branches, n + i)
    print("%d steps of %d branches" % (a.steps, a.branches))

    # drop all but the last, close the holes, go on
    cache.free(i32(branches[:-1]))
    before = int((cache.refs > 0).nonzero().max()) + 1
    cache.compact()
    cache.status()
    after = int((cache.refs > 0).sum())
    assert int((cache.refs > 0).nonzero().max()) + 1 == after
    step(branches[-1:], n + a.steps)
    print("compacted from %d to %d pages, and one more step" % (before, after))


if __name__ == "__main__":
    main()
