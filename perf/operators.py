"""What is measured of the operators on a paged KV cache: attention of one new
token per sequence over its pages, the append of new tokens (rotary positions on
one or more axes, keys and values written to their pages) and the page
operations (fork, reserve, free, compact, copy).

A cache is a pool of pages, each page_tokens x head_dim scalars of one (layer,
key/value, head, token block), and a table of page numbers [sequence][layer][2]
[head][block], -1 where there is no page.  The shapes are those of the synthetic
caches (28 x 8 x 4096 x 128, 64 x 8 x 8192 x 128, 36 x 8 x 16384 x 128 as e4m3,
64 x 8 x 32768 x 128), their pages the coder's chunks of 128 and 256 tokens.
"""
import math

import torch

own = False  # True: the framework's operators; False: their plain form

DEV = "cuda"
E4M3_MAX = 448.0
ROPE_BASE = 1e6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the tiny cache's shape (2 heads x 300 tokens x 64): the latency of one call
        dict(name="attend-tiny", op="attend", dtype="bf16", batch=1, layers=2, kv_heads=2,
             group=4, head_dim=64, page=128, max_len=300, window=0, empty=0),
        # a small model's decode step: ragged sequences, two of them without a token yet
        dict(name="attend-0.6b-ragged", op="attend", dtype="bf16", batch=24, layers=1,
             kv_heads=8, group=2, head_dim=128, page=256, max_len=4096, window=0, empty=2),
        # a large model's decode step over the 8192-token cache
        dict(name="attend-32b", op="attend", dtype="bf16", batch=16, layers=1, kv_heads=8,
             group=8, head_dim=128, page=256, max_len=8192, window=0, empty=0),
        # the FP8 cache, ragged up to 16384 tokens
        dict(name="attend-8b-e4m3", op="attend", dtype="e4m3", batch=32, layers=1, kv_heads=8,
             group=4, head_dim=128, page=256, max_len=16384, window=0, empty=0),
        # one long sequence in FP8: few rows, a long axis
        dict(name="attend-long-e4m3", op="attend", dtype="e4m3", batch=1, layers=1, kv_heads=8,
             group=8, head_dim=128, page=128, max_len=131071, window=0, empty=0),
        # one new token for each of 8 running sequences
        dict(name="append-step", op="append", dtype="bf16", seqs=8, tokens=8, start=4001,
             kv_heads=8, group=2, head_dim=128, rotary=128, page=256, axes=1, interleaved=False,
             far=0),
        # a prompt with images for a large model: positions in time, height and width
        dict(name="append-prompt-3axes", op="append", dtype="bf16", seqs=1, tokens=8190, start=0,
             kv_heads=8, group=8, head_dim=128, rotary=128, page=256, axes=3, interleaved=False,
             far=500000),
        # prompts into an FP8 cache, half of each head rotated, neighbouring pairs
        dict(name="append-prompts-e4m3", op="append", dtype="e4m3", seqs=5, tokens=16001,
             start=77, kv_heads=8, group=4, head_dim=128, rotary=64, page=256, axes=1,
             interleaved=True, far=0),
        # parallel sampling on a small model: 4 continuations of one prompt are dropped and
        # forked again, each with room for one more token
        dict(name="fork-0.6b", op="fork", dtype="bf16", parents=1, children=4, rows=448,
             head_dim=128, page=256, length=3990, extra=1),
        # beams of a large model's 2 prompts
        dict(name="fork-32b", op="fork", dtype="bf16", parents=2, children=8, rows=1024,
             head_dim=128, page=256, length=8100, extra=300),
        # the pool after sequences of the FP8 model have left: holes everywhere
        dict(name="compact-8b-e4m3", op="compact", dtype="e4m3", seqs=24, rows=576, blocks=6,
             head_dim=128, page=256, live=0.7),
        # some thousand pages moved to other places of the pool
        dict(name="copy-pages", op="copy", dtype="bf16", pages=5000, head_dim=128, page=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "fork", "compact", "copy"])
    dtype = rng.choice(["bf16", "e4m3"])
    size = 2 if dtype == "bf16" else 1
    if op == "attend":
        while True:
            c = dict(op=op, dtype=dtype, batch=_log(rng, 1, 64), layers=rng.choice([1, 2]),
                     kv_heads=rng.choice([1, 2, 4, 8]), group=rng.choice([1, 2, 3, 4, 5, 8, 12, 16]),
                     head_dim=rng.choice([64, 96, 128, 128, 128, 256]),
                     page=rng.choice([16, 33, 64, 128, 128, 256, 256]),
                     max_len=_log(rng, 1, 131072), window=0, empty=0)
            if rng.random() < 0.3:
                c["window"] = _log(rng, 1, 8192)
            if c["batch"] > 2 and rng.random() < 0.3:
                c["empty"] = 1
            if (c["batch"] * c["layers"] * c["kv_heads"] * c["head_dim"] * c["max_len"] * 2 * size
                    <= 5 << 28 and c["batch"] * c["kv_heads"] * c["group"] * c["max_len"] <= 1 << 24):
                return c
    if op == "append":
        seqs = _log(rng, 1, 64)
        d = rng.choice([64, 96, 128, 128])
        return dict(op=op, dtype=dtype, seqs=seqs, tokens=max(seqs, _log(rng, 1, 8192)),
                    start=rng.randrange(0, 3000), kv_heads=rng.choice([1, 2, 4, 8]),
                    group=rng.choice([1, 2, 3, 4, 8]), head_dim=d,
                    rotary=rng.choice([d, d, d // 2]), page=rng.choice([16, 33, 64, 128, 256]),
                    axes=rng.choice([1, 1, 2, 3]), interleaved=rng.random() < 0.4,
                    far=rng.choice([0, 0, _log(rng, 1000, 1000000)]))
    if op == "fork":
        while True:
            c = dict(op=op, dtype=dtype, parents=_log(rng, 1, 8), children=_log(rng, 1, 16),
                     rows=2 * _log(rng, 1, 512), head_dim=rng.choice([64, 96, 128]),
                     page=rng.choice([16, 33, 128, 256]), length=_log(rng, 1, 8192),
                     extra=_log(rng, 1, 600))
            blocks = c["length"] // c["page"] + c["extra"] // c["page"] + 3
            if ((c["parents"] + c["children"]) * c["rows"] * blocks * c["page"] * c["head_dim"] * size
                    <= 3 << 30 and (c["parents"] + c["children"]) * c["rows"] * blocks <= 1 << 19):
                return c
    if op == "compact":
        while True:
            c = dict(op=op, dtype=dtype, seqs=_log(rng, 1, 32), rows=2 * _log(rng, 1, 512),
                     blocks=rng.randrange(1, 12), head_dim=rng.choice([64, 96, 128]),
                     page=rng.choice([16, 33, 128, 256]), live=round(rng.uniform(0.3, 0.95), 3))
            if (c["seqs"] * c["rows"] * c["blocks"] * c["page"] * c["head_dim"] * size
                    <= 5 << 29 and c["seqs"] * c["rows"] * c["blocks"] <= 1 << 18):
                return c
    return dict(op=op, dtype=dtype, pages=_log(rng, 1, 10000),
                head_dim=rng.choice([64, 96, 128]), page=rng.choice([16, 33, 128, 256]))


def _bytes(case):
    return 2 if case["dtype"] == "bf16" else 1


def _lens(case):
    """Lengths of the sequences of an attend case: the longest first, the others spread over
    (1/4, 1], `empty` at the end without a token."""
    b, n = case["batch"], case["max_len"]
    lens = [n] + [max(1, int(n * (0.25 + 0.75 * math.modf(i * 0.6180339887)[0])))
                  for i in range(1, b)]
    for i in range(case["empty"]):
        lens[b - 1 - i] = 0
    return lens


def _begins(case):
    w = case["window"]
    return [max(0, n - w) if w else 0 for n in _lens(case)]


def _counts(case):
    """Tokens of each sequence of an append case."""
    s, n = case["seqs"], case["tokens"]
    return [n // s + (1 if i < n % s else 0) for i in range(s)]


def _fork_lens(case):
    """Length of each child's parent when it is forked."""
    n = case["length"]
    by_parent = [max(1, n - 37 * i) for i in range(case["parents"])]
    return [by_parent[i % case["parents"]] for i in range(case["children"])]


def _fork_blocks(case):
    return -(-(case["length"] + case["extra"]) // case["page"])


def _fork_pages(case):
    p, n = case["page"], case["length"]
    own_pages = sum(-(-max(1, n - 37 * i) // p) for i in range(case["parents"]))
    fresh = sum(-(-(m + case["extra"]) // p) - m // p for m in _fork_lens(case))
    return case["rows"] * (own_pages + fresh) + 7


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _rand(shape, g):
    return torch.randn(shape, generator=g, device=DEV)


def _pool(case, pages, g):
    """Page contents: normal values, every channel with a scale of its own and a few of them
    ten times that, as in key-value caches; e4m3 codes span the type's range."""
    d = case["head_dim"]
    chan = torch.exp(0.5 * _rand((d,), g))
    chan[torch.randperm(d, generator=g, device=DEV)[:4]] *= 5.0
    pool = torch.empty((pages, case["page"], d), device=DEV,
                       dtype=torch.bfloat16 if case["dtype"] == "bf16" else torch.float8_e4m3fn)
    step = max(1, (1 << 27) // (case["page"] * d))
    for a in range(0, pages, step):
        x = _rand((min(step, pages - a), case["page"], d), g) * chan
        if case["dtype"] == "e4m3":
            x = (x * 8.0).clamp_(-E4M3_MAX, E4M3_MAX)
        pool[a:a + step] = x.to(pool.dtype)
    return pool


def _codes(pool):
    """The pool as the codec's symbols: bf16 patterns or e4m3 codes."""
    return pool.view(torch.int16) if pool.dtype == torch.bfloat16 else pool.view(torch.uint8)


def _handle(case, s, layers, heads):
    """The framework's view of the cache that a serving program keeps: it holds s's own tensors."""
    import lossless_kv_cache_fixed_gb300 as P
    return P.PagedCache(P.SKV_BF16 if case["dtype"] == "bf16" else P.SKV_E4M3, layers, heads,
                        case["head_dim"], case["page"], pool=_codes(s["pool"]), table=s["table"],
                        refs=s["refs"], scale=s.get("scale"))


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    op, d, tb = case["op"], case["head_dim"], case["page"]
    if op == "attend":
        b, layers, h = case["batch"], case["layers"], case["kv_heads"]
        lens = _lens(case)
        blocks = max(1, -(-max(lens) // tb))
        need = [-(-n // tb) for n in lens]
        have = torch.arange(blocks, device=DEV) < _ints(need)[:, None]
        have = have[:, None, None, None, :].expand(b, layers, 2, h, blocks)
        pages = int(sum(need)) * layers * 2 * h
        s["pool"] = _pool(case, pages, g)
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        s["table"] = torch.full((b, layers, 2, h, blocks), -1, dtype=torch.int32, device=DEV)
        s["table"][have] = order
        s["refs"] = torch.ones(pages, dtype=torch.int32, device=DEV)
        if case["dtype"] == "e4m3":
            s["scale"] = torch.exp(0.3 * _rand((layers, h), g)) / 8.0
        s["q"] = (0.5 * _rand((b, h * case["group"], d), g)).to(torch.bfloat16)
        s["slots"] = torch.randperm(b, generator=g, device=DEV).to(torch.int32)
        # slot i of the table holds the sequence of length lens[i]
        s["lens"] = _ints(lens)[s["slots"].long()].contiguous()
        s["begins"] = _ints(_begins(case))[s["slots"].long()].contiguous() if case["window"] else None
        s["layer"] = layers - 1
        s["max_len"] = max(lens)
        if own:
            s["cache"] = _handle(case, s, layers, h)
    elif op == "append":
        h, n, seqs = case["kv_heads"], case["tokens"], case["seqs"]
        hq, r = h * case["group"], case["rotary"]
        counts = _counts(case)
        blocks = -(-(case["start"] + max(counts)) // tb)
        pages = seqs * 2 * h * blocks
        s["pool"] = _pool(case, pages, g)
        s["table"] = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).view(
            seqs, 1, 2, h, blocks)
        s["refs"] = torch.ones(pages, dtype=torch.int32, device=DEV)
        # one row of q, k and v heads per token, as a fused projection leaves them
        qkv = (_rand((n, hq + 2 * h, d), g) * torch.exp(0.5 * _rand((hq + 2 * h, d), g))).to(
            torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + h], qkv[:, hq + h:]
        if case["dtype"] == "e4m3":
            s["scale"] = (0.02 * torch.exp(0.3 * _rand((1, h), g)))
        c = _ints(counts)
        s["slots"] = torch.repeat_interleave(torch.arange(seqs, device=DEV), c.long(),
                                             output_size=n).to(torch.int32)
        first = (torch.cumsum(c, 0) - c)[s["slots"].long()]
        s["at"] = (case["start"] + torch.arange(n, device=DEV) - first).to(torch.int32)
        t = s["at"] + case["far"] + torch.randint(0, 1000, (1,), generator=g, device=DEV).to(torch.int32)
        s["positions"] = torch.stack([t, case["far"] + s["at"] % 37, case["far"] + s["at"] % 53])[
            :case["axes"]].to(torch.int32).contiguous()
        pair = torch.arange(r // 2, device=DEV)
        s["freqs"] = ROPE_BASE ** (-2.0 * pair.double() / r)
        s["axis"] = (pair * case["axes"] // (r // 2)).to(torch.uint8)
        if own:
            import lossless_kv_cache_fixed_gb300 as P
            s["cache"] = _handle(case, s, 1, h)
            s["rope"] = P.Rope(s["freqs"], s["axis"], axes=case["axes"],
                               interleaved=case["interleaved"])
    elif op == "fork":
        p, c, rows = case["parents"], case["children"], case["rows"]
        blocks, pages = _fork_blocks(case), _fork_pages(case)
        need = _ints([-(-max(1, case["length"] - 37 * i) // tb) for i in range(p)])
        have = (torch.arange(blocks, device=DEV) < need[:, None])[:, None, :].expand(p, rows, blocks)
        s["pool"] = _pool(case, pages, g)
        s["table"] = torch.full((p + c, rows // 2, 2, 1, blocks), -1, dtype=torch.int32, device=DEV)
        used = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)[:int(have.sum())]
        s["table"][:p].view(p, rows, blocks)[have] = used
        s["refs"] = torch.zeros(pages, dtype=torch.int32, device=DEV)
        s["refs"][used.long()] = 1
        s["parents"] = _ints([i % p for i in range(c)])
        s["children"] = _ints([p + i for i in range(c)])
        s["lens"] = _ints(_fork_lens(case))
        s["new_lens"] = s["lens"] + case["extra"]
        if own:
            s["cache"] = _handle(case, s, rows // 2, 1)
    elif op == "compact":
        rows, seqs, blocks = case["rows"], case["seqs"], case["blocks"]
        n = seqs * rows * blocks
        pages = int(n / case["live"]) + 1
        s["pool"] = _pool(case, pages, g)
        table = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)[:n].view(
            seqs, rows, blocks).clone()
        # every second sequence shares the first half of its blocks with the one before it
        half, pairs = blocks // 2, seqs // 2
        table[1:2 * pairs:2, :, :half] = table[0:2 * pairs:2, :, :half]
        s["table"] = table.view(seqs, rows // 2, 2, 1, blocks)
        s["refs"] = torch.bincount(table.reshape(-1).long(), minlength=pages).to(torch.int32)
        s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
        if own:
            s["cache"] = _handle(case, s, rows // 2, 1)
    else:
        n = case["pages"]
        s["pool"] = _pool(case, 2 * n + 1, g)
        order = torch.randperm(2 * n + 1, generator=g, device=DEV).to(torch.int32)
        s["src"], s["dst"] = order[:n].contiguous(), order[n:2 * n].contiguous()
        s["table"] = torch.full((1, 1, 2, 1, 1), -1, dtype=torch.int32, device=DEV)
        s["refs"] = torch.zeros(2 * n + 1, dtype=torch.int32, device=DEV)
        if own:
            s["cache"] = _handle(case, s, 1, 1)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if op == "attend":
        if own:
            return s["cache"].attend(s["layer"], s["slots"], s["lens"], s["q"], s["max_len"],
                                     begins=s["begins"], lse=True)
        return _attend_plain(s, case)
    if op == "append":
        if own:
            q = s["cache"].append(0, s["slots"], s["at"], s["q"], s["k"], s["v"], s["rope"],
                                  s["positions"])
        else:
            q = _append_plain(s, case)
        return q, s["pool"]
    if op == "fork":
        if own:
            s["cache"].free(s["children"])
            s["cache"].fork(s["parents"], s["children"], s["lens"])
            s["cache"].reserve(s["children"], s["lens"], s["new_lens"])
        else:
            _fork_plain(s, case)
        return s["table"], s["refs"], _codes(s["pool"])
    if op == "compact":
        if own:
            s["cache"].compact(table_out=s["table_out"], refs_out=s["refs_out"])
        else:
            _compact_plain(s, case)
        return s["table_out"], s["refs_out"], _codes(s["pool"])
    if own:
        s["cache"].copy_pages(s["src"], s["dst"])
    else:
        pool = _codes(s["pool"])
        pool[s["dst"].long()] = pool[s["src"].long()]
    return _codes(s["pool"])


def _attend_plain(s, case):
    b, h, d = case["batch"], case["kv_heads"], case["head_dim"]
    page = s["table"][s["slots"].long(), s["layer"]].clamp(min=0).long()   # [b, 2, h, blocks]
    kv = s["pool"][page].view(b, 2, h, -1, d)
    k, v = kv[:, 0].float(), kv[:, 1].float()
    del kv
    pos = torch.arange(k.shape[2], device=DEV)
    seen = pos < s["lens"][:, None]
    if s["begins"] is not None:
        seen = seen & (pos >= s["begins"][:, None])
    seen = seen[:, None, None, :]
    x = s["q"].float().view(b, h, case["group"], d) @ k.transpose(2, 3) / math.sqrt(d)
    if "scale" in s:
        x = x * s["scale"][s["layer"]][:, None, None]
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m0)
    total = p.sum(-1, keepdim=True)
    o = p @ v / torch.where(total == 0, 1.0, total)
    if "scale" in s:
        o = o * s["scale"][s["layer"]][:, None, None]
    lse = (m0 + torch.log(total)).view(b, -1)
    return o.to(torch.bfloat16).view(b, -1, d), lse


def _angles(s):
    """cos and sin [tokens, 1, pairs] of every token's angles, in 64 bits."""
    at = s["positions"].double()[s["axis"].long()]            # [pairs, tokens]
    a = (at * s["freqs"][:, None]).T[:, None, :]
    return torch.cos(a), torch.sin(a)


def _append_plain(s, case):
    cos, sin = (t.float() for t in _angles(s))
    r = case["rotary"]

    def rotate(x):
        y = x.float().clone()
        if case["interleaved"]:
            a, b = x[..., 0:r:2].float(), x[..., 1:r:2].float()
            y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, a * sin + b * cos
        else:
            a, b = x[..., :r // 2].float(), x[..., r // 2:r].float()
            y[..., :r // 2], y[..., r // 2:r] = a * cos - b * sin, a * sin + b * cos
        return y

    q, k, v = rotate(s["q"]), rotate(s["k"]), s["v"].float()
    kv = torch.stack([k, v], 1)                               # [tokens, 2, heads, d]
    if "scale" in s:
        kv = (kv / s["scale"][0][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    at = s["at"].long()
    page = s["table"][s["slots"].long(), 0][torch.arange(at.numel(), device=DEV), :, :,
                                            at // case["page"]].long()
    s["pool"].view(-1, case["head_dim"])[page * case["page"] + (at % case["page"])[:, None, None]] = \
        kv.to(s["pool"].dtype)
    return q.to(torch.bfloat16)


def _fork_plain(s, case):
    rows, tb = case["rows"], case["page"]
    blocks = s["table"].shape[-1]
    refs, pages = s["refs"], s["refs"].numel()
    table = s["table"].view(-1, rows, blocks)
    pool = _codes(s["pool"])
    child = s["children"].long()
    block = torch.arange(blocks, device=DEV)
    # free: drop the children's references
    old = table[child]
    refs.index_add_(0, old.clamp(min=0).reshape(-1).long(), -(old >= 0).reshape(-1).to(torch.int32))
    # the lowest free pages, in order
    fresh = torch.argsort(refs != 0, stable=True)
    # fork: full blocks are shared, the last one is copied if it is not full
    parent = table[s["parents"].long()]
    full = (s["lens"] // tb)[:, None]
    tail = (s["lens"] % tb)[:, None]
    shared = (block < full)[:, None, :].expand(-1, rows, -1)
    new = torch.where(shared, parent, -1)
    part = ((block == full) & (tail > 0))[:, None, :].expand(-1, rows, -1)
    rank = torch.cumsum(part.reshape(-1), 0) - 1
    page = fresh[rank.clamp(min=0)].view(part.shape).to(torch.int32)
    taken = rank[-1] + 1
    new = torch.where(part, page, new)
    refs.index_add_(0, new.clamp(min=0).reshape(-1).long(), (new >= 0).reshape(-1).to(torch.int32))
    last = full.long().clamp(max=blocks - 1)[:, :, None].expand(-1, rows, 1)
    # [children, rows, page, d]: the parent's values where it has some, the new page's elsewhere
    has = tail.expand(-1, rows) > 0
    src = parent.gather(2, last)[:, :, 0].clamp(min=0).long()
    dst = torch.where(has, new.gather(2, last)[:, :, 0].clamp(min=0).long(), src)
    filled = (torch.arange(tb, device=DEV) < torch.where(tail > 0, tail, tb))[:, None, :, None]
    pool[dst] = torch.where(filled, pool[src], pool[dst])
    # reserve: the next lowest free pages for the blocks still missing
    want = (block < (-(-s["new_lens"] // tb))[:, None]) & (block >= (-(-s["lens"] // tb))[:, None])
    want = want[:, None, :].expand(-1, rows, -1)
    rank = taken + torch.cumsum(want.reshape(-1), 0) - 1
    page = fresh[rank.clamp(min=0, max=pages - 1)].view(want.shape).to(torch.int32)
    new = torch.where(want, page, new)
    refs.index_add_(0, page.reshape(-1).long(), want.reshape(-1).to(torch.int32))
    table[child] = new


def _compact_plain(s, case):
    refs, pages = s["refs"], s["refs"].numel()
    pool = _codes(s["pool"])
    live = refs > 0
    at = torch.arange(pages, device=DEV)
    count = live.sum()
    # the lowest hole takes the highest live page, until no live page is above a hole
    holes = torch.argsort(live, stable=True)
    high = torch.argsort(~live, stable=True)
    k = at.clamp(max=pages - 1)
    high = high[(count - 1 - k).clamp(min=0)]
    move = (k < count) & (holes < count) & ~live[holes] & (high >= count) & live[high]
    moves = int(move.sum())                                   # the new size of a copy
    src, dst = high[:moves], holes[:moves]
    where_to = at.clone()
    where_to[src] = dst
    pool[dst] = pool[src]
    s["refs_out"].copy_(refs)
    s["refs_out"][dst] = refs[src]
    s["refs_out"][src] = 0
    t = s["table"]
    s["table_out"].copy_(torch.where(t >= 0, where_to[t.clamp(min=0).long()].to(torch.int32), t))


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    op, d = case["op"], case["head_dim"]
    if op not in ("attend", "append"):
        return None                                           # whole numbers, compared as they are
    s = prepare(case, seed)
    if op == "attend":
        h, group = case["kv_heads"], case["group"]
        scale = s["scale"][s["layer"]].double() if "scale" in s else torch.ones(h, device=DEV).double()
        out = torch.zeros(case["batch"], h, group, d, dtype=torch.float64, device=DEV)
        lse = torch.full((case["batch"], h, group), -math.inf, dtype=torch.float64, device=DEV)
        lens = s["lens"].tolist()
        begins = s["begins"].tolist() if s["begins"] is not None else [0] * len(lens)
        q = s["q"].double().view(case["batch"], h, group, d)
        for i, slot in enumerate(s["slots"].tolist()):
            a, n = begins[i], lens[i]
            if n <= a:
                continue
            for j in range(h):
                rows = []
                for side in (0, 1):
                    pages = s["table"][slot, s["layer"], side, j, :-(-n // case["page"])].long()
                    rows.append(s["pool"][pages].double().reshape(-1, d)[a:n] * scale[j])
                w = (rows[0] @ q[i, j].T) / math.sqrt(d)      # [tokens, group]
                lse[i, j] = torch.logsumexp(w, 0)
                out[i, j] = torch.softmax(w, 0).T @ rows[1]
        return out.view(case["batch"], -1, d), lse.view(case["batch"], -1)
    r = case["rotary"]
    pair = torch.arange(r // 2, device=DEV)
    angle = s["positions"].double().T[:, (pair * case["axes"] // (r // 2))] * ROPE_BASE ** (
        -2.0 * pair.double() / r)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None, :]

    def spun(x):
        y = x.double()
        if case["interleaved"]:
            z = torch.complex(y[..., 0:r:2], y[..., 1:r:2]) * turn
            z = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(y[..., :r // 2], y[..., r // 2:r]) * turn
            z = torch.cat([z.real, z.imag], -1)
        return torch.cat([z, y[..., r:]], -1)

    pool = s["pool"].double()
    k, v = spun(s["k"]), s["v"].double()
    if "scale" in s:
        k, v = ((x / s["scale"][0].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX) for x in (k, v))
    at = s["at"].long()
    for side, x in ((0, k), (1, v)):
        for j in range(case["kv_heads"]):
            page = s["table"][s["slots"].long(), 0, side, j, at // case["page"]].long()
            pool[page, at % case["page"]] = x[:, j]
    return spun(s["q"]), pool


# ---------------------------------------------------------------- work

def work(case):
    op, d, size = case["op"], case["head_dim"], _bytes(case)
    if op == "attend":
        h, hq = case["kv_heads"], case["kv_heads"] * case["group"]
        seen = sum(n - a for n, a in zip(_lens(case), _begins(case)))
        pages = sum(-(-n // case["page"]) - a // case["page"]
                    for n, a in zip(_lens(case), _begins(case)))
        return {"bytes": seen * h * 2 * d * size + pages * 2 * h * 4
                + case["batch"] * hq * (4 * d + 4) + 8 * case["batch"],
                "flops": 4.0 * seen * hq * d}
    if op == "append":
        n, h = case["tokens"], case["kv_heads"]
        hq, r = h * case["group"], case["rotary"]
        return {"bytes": n * (hq * d * 4 + 2 * h * d * (2 + size) + 8 + 4 * case["axes"]),
                "flops": n * (hq + h) * 3.0 * r}
    page = case["page"] * d * size
    if op == "fork":
        rows, lens = case["rows"], _fork_lens(case)
        tb = case["page"]
        tails = [n % tb for n in lens]
        read = sum(tails[:min(case["parents"], case["children"])])
        entries = sum(-(-(n + case["extra"]) // tb) for n in lens)
        # tails read once for each parent and written for each child; the parents' entries read,
        # the children's read and written; a count for each page that is taken or given back
        return {"bytes": rows * ((read + sum(tails)) * d * size + 4.0 * 5 * entries), "flops": 0.0}
    if op == "compact":
        n = case["seqs"] * case["rows"] * case["blocks"]
        pages = int(n / case["live"]) + 1
        live = n - (case["seqs"] // 2) * case["rows"] * (case["blocks"] // 2)
        moved = live * (1.0 - live / pages)
        return {"bytes": moved * 2 * page + 8.0 * (n + pages), "flops": 0.0}
    return {"bytes": case["pages"] * (2.0 * page + 8), "flops": 0.0}
