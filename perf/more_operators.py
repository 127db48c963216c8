"""What is measured of attention of more than one new token over a paged KV cache, and of
differential attention over one.

A cache is a pool of pages, each page_tokens x head_dim scalars of one (layer,
key/value, head, token block), and a table of page numbers [sequence][layer][2]
[head][block], -1 where there is no page.  The new tokens of sequence i are rows
starts[i] .. starts[i + 1] - 1 of q and the last ones of its lens[i] tokens; a token at
place p sees the tokens t <= p (all of the sequence where `causal` is false), with a window
those above p - window.  Differential attention takes a head's keys and queries as two
halves, each with a softmax of its own; the second one's result times a learned number
per head is subtracted from the first's, and the difference may be normalised (root mean
square, a weight per channel).  Shapes are those of the synthetic caches (28 x 8 x 4096 x 128,
64 x 8 x 8192 x 128, 36 x 8 x 16384 x 128 as e4m3, 64 x 8 x 32768 x 128).
"""
import math

import torch

own = False  # True: the framework's operators; False: their plain form

DEV = "cuda"
E4M3_MAX = 448.0
EPS = 1e-5


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the tiny cache's shape (2 heads x 300 tokens x 64), three new tokens: latency
        dict(name="chunk-tiny", op="chunk", dtype="bf16", batch=1, layers=2, kv_heads=2, group=4,
             head_dim=64, page=128, max_len=300, max_new=3, window=0, causal=True, empty=0),
        # a small model checks 5 drafted tokens of each of 24 ragged sequences
        dict(name="chunk-draft-0.6b", op="chunk", dtype="bf16", batch=24, layers=1, kv_heads=8,
             group=2, head_dim=128, page=256, max_len=4096, max_new=5, window=0, causal=True,
             empty=2),
        # a small model's whole prompt
        dict(name="chunk-prompt-0.6b", op="chunk", dtype="bf16", batch=1, layers=1, kv_heads=8,
             group=2, head_dim=128, page=256, max_len=4096, max_new=4096, window=0, causal=True,
             empty=0),
        # a large model goes on from a decoded prefix: 2048 tokens on top of 6144
        dict(name="chunk-prefix-32b", op="chunk", dtype="bf16", batch=1, layers=1, kv_heads=8,
             group=8, head_dim=128, page=256, max_len=8192, max_new=2048, window=0, causal=True,
             empty=0),
        # turns of a conversation: ragged chunks on ragged FP8 caches
        dict(name="chunk-turns-e4m3", op="chunk", dtype="e4m3", batch=8, layers=1, kv_heads=8,
             group=4, head_dim=128, page=256, max_len=8190, max_new=333, window=0, causal=True,
             empty=1),
        # 9 tokens on one long FP8 sequence: few rows, a long axis
        dict(name="chunk-long-e4m3", op="chunk", dtype="e4m3", batch=1, layers=1, kv_heads=8,
             group=8, head_dim=128, page=128, max_len=131071, max_new=9, window=0, causal=True,
             empty=0),
        # wide heads with a sliding window, small pages
        dict(name="chunk-window-256", op="chunk", dtype="bf16", batch=2, layers=1, kv_heads=4,
             group=2, head_dim=256, page=16, max_len=6001, max_new=3001, window=1024, causal=True,
             empty=0),
        # differential attention, one new token on the tiny cache's shape: latency
        dict(name="diff-tiny", op="diff", dtype="bf16", batch=1, layers=2, kv_heads=2, group=2,
             head_dim=64, page=128, max_len=300, max_new=0, window=0, causal=True, empty=0,
             norm=True),
        # its decode step: ragged sequences
        dict(name="diff-step", op="diff", dtype="bf16", batch=32, layers=1, kv_heads=8, group=4,
             head_dim=128, page=256, max_len=8192, max_new=0, window=0, causal=True, empty=1,
             norm=True),
        # the same over FP8 caches
        dict(name="diff-step-e4m3", op="diff", dtype="e4m3", batch=32, layers=1, kv_heads=8,
             group=4, head_dim=128, page=256, max_len=16384, max_new=0, window=0, causal=True,
             empty=0, norm=False),
        # its prompt
        dict(name="diff-prompt", op="diff", dtype="bf16", batch=1, layers=1, kv_heads=8, group=2,
             head_dim=128, page=256, max_len=4096, max_new=4096, window=0, causal=True, empty=0,
             norm=True),
        # ragged chunks on FP8 caches
        dict(name="diff-turns-e4m3", op="diff", dtype="e4m3", batch=5, layers=1, kv_heads=8,
             group=4, head_dim=128, page=128, max_len=4001, max_new=500, window=0, causal=True,
             empty=0, norm=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "diff"])
    dtype = rng.choice(["bf16", "e4m3"])
    size = 2 if dtype == "bf16" else 1
    while True:
        c = dict(op=op, dtype=dtype, batch=_log(rng, 1, 64), layers=rng.choice([1, 2]),
                 kv_heads=rng.choice([1, 2, 4, 8]), group=rng.choice([1, 2, 3, 4, 5, 8, 12, 16]),
                 head_dim=rng.choice([64, 96, 128, 128, 128, 256]),
                 page=rng.choice([16, 33, 64, 128, 128, 256, 256]), max_len=_log(rng, 1, 131072),
                 window=0, causal=rng.random() < 0.9, empty=0)
        c["max_new"] = min(c["max_len"], _log(rng, 1, 4096))
        if op == "diff":
            c["norm"] = rng.random() < 0.5
            if rng.random() < 0.4:
                c["max_new"] = 0
        if rng.random() < 0.3:
            c["window"] = _log(rng, 1, 8192)
        if c["batch"] > 2 and rng.random() < 0.3:
            c["empty"] = 1
        scores = c["batch"] * max(1, c["max_new"]) * c["kv_heads"] * c["group"] * c["max_len"]
        if (c["batch"] * c["layers"] * c["kv_heads"] * c["head_dim"] * c["max_len"] * 2 * size
                <= 5 << 28 and scores <= 1 << 30
                and scores * c["head_dim"] <= (7 << 34 if op == "chunk" else 9 << 33)):
            return c


def _bytes(case):
    return 2 if case["dtype"] == "bf16" else 1


def _spread(i, n):
    """A number for sequence i: n for the first, the others spread over (1/4, 1] of n."""
    return n if i == 0 else max(1, int(n * (0.25 + 0.75 * math.modf(i * 0.6180339887)[0])))


def _lens(case):
    """Lengths of the sequences: the longest first, `empty` at the end without a token."""
    b = case["batch"]
    lens = [_spread(i, case["max_len"]) for i in range(b)]
    for i in range(case["empty"]):
        lens[b - 1 - i] = 0
    return lens


def _news(case):
    """New tokens of each sequence: with max_new 0 one each, of the one-token form."""
    if not case["max_new"]:
        return [1] * case["batch"]
    return [min(_spread(3 * i, case["max_new"]), n) for i, n in enumerate(_lens(case))]


def _seen(case):
    """For each sequence: tokens seen by at least one of its rows, (token, row) pairs."""
    res = []
    w = case["window"]
    for n, new in zip(_lens(case), _news(case)):
        if not n or not new:
            res.append((0, 0, 0))
            continue
        first = n - new if case["max_new"] else n - 1          # place of the first new token
        lo = max(0, first - w + 1) if w else 0
        pairs = 0
        for p in range(first, n):
            a = max(0, p - w + 1) if w else 0
            pairs += (p + 1 if case["causal"] else n) - a
        res.append((lo, n - lo, pairs))
    return res


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _rand(shape, g):
    return torch.randn(shape, generator=g, device=DEV)


def _pool(case, pages, g):
    """Page contents: normal values, every channel with a scale of its own and a few of them
    five times that, as in key-value caches; e4m3 codes span the type's range."""
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


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    d, tb, b = case["head_dim"], case["page"], case["batch"]
    layers, h = case["layers"], case["kv_heads"]
    lens, news = _lens(case), _news(case)
    blocks = max(1, -(-max(lens) // tb))
    need = [-(-n // tb) for n in lens]
    have = torch.arange(blocks, device=DEV) < _ints(need)[:, None]
    have = have[:, None, None, None, :].expand(b, layers, 2, h, blocks)
    pages = max(1, int(sum(need)) * layers * 2 * h)
    s["pool"] = _pool(case, pages, g)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    # slot i of the table holds the sequence of length lens[i]
    s["table"] = torch.full((b, layers, 2, h, blocks), -1, dtype=torch.int32, device=DEV)
    s["table"][have] = order[:int(sum(need)) * layers * 2 * h]
    s["refs"] = torch.ones(pages, dtype=torch.int32, device=DEV)
    if case["dtype"] == "e4m3":
        s["scale"] = torch.exp(0.3 * _rand((layers, h), g)) / 8.0
    slots = torch.randperm(b, generator=g, device=DEV).tolist()
    s["slots"] = _ints(slots)
    s["lens"] = _ints([lens[i] for i in slots])
    starts = [0]
    for i in slots:
        starts.append(starts[-1] + news[i])
    s["starts"] = _ints(starts)
    s["max_new"] = max(news)
    s["q"] = (0.5 * _rand((starts[-1], h * case["group"], d), g)).to(torch.bfloat16)
    s["layer"], s["max_len"] = layers - 1, max(lens)
    if case["op"] == "diff":
        s["lam"] = 0.2 + 0.6 * torch.rand(h * case["group"], generator=g, device=DEV)
        s["norm"] = 0.2 + 0.8 * torch.rand(d, generator=g, device=DEV) if case["norm"] else None
    if own:
        import lossless_kv_cache_fixed_gb300 as P
        s["cache"] = P.PagedCache(P.SKV_BF16 if case["dtype"] == "bf16" else P.SKV_E4M3, layers, h,
                                  d, tb, pool=_codes(s["pool"]), table=s["table"], refs=s["refs"],
                                  scale=s.get("scale"))
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    s, case = state, state["case"]
    if own:
        more = dict(window=case["window"], causal=case["causal"], lse=True)
        if case["op"] == "chunk":
            return s["cache"].attend_chunk(s["layer"], s["slots"], s["lens"], s["starts"], s["q"],
                                           s["max_len"], **more)
        return s["cache"].attend_diff(s["layer"], s["slots"], s["lens"], s["q"], s["lam"],
                                      s["max_len"], starts=s["starts"] if case["max_new"] else None,
                                      norm=s["norm"], eps=EPS, **more)
    k, v, q, seen, row = _padded(s, case)
    if case["op"] == "chunk":
        o, lse = _softmax_plain(s, q, k, v, seen, case["head_dim"])
        return o.flatten(2, 3)[row].to(torch.bfloat16), lse.flatten(2, 3)[row]
    half = case["head_dim"] // 2
    o, lse1 = _softmax_plain(s, q[..., :half], k[..., :half], v, seen, half)
    o2, lse2 = _softmax_plain(s, q[..., half:], k[..., half:], v, seen, half)
    o = o.flatten(2, 3)[row] - s["lam"][:, None] * o2.flatten(2, 3)[row]
    if s["norm"] is not None:
        o = o / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS) * s["norm"]
    lse = torch.stack([lse1.flatten(2, 3)[row], lse2.flatten(2, 3)[row]], -1)
    return o.to(torch.bfloat16), lse


def _padded(s, case):
    """Keys and values [batch, heads, tokens, d], queries [batch, new, heads, group, d], what each
    row sees [batch, new, tokens], and each new token's place (sequence, row) in the padded form."""
    b, h, d = case["batch"], case["kv_heads"], case["head_dim"]
    page = s["table"][s["slots"].long(), s["layer"]].clamp(min=0).long()   # [b, 2, h, blocks]
    kv = s["pool"][page].view(b, 2, h, -1, d)
    k, v = kv[:, 0].float(), kv[:, 1].float()
    del kv
    first = s["starts"][:-1, None]
    news = s["starts"][1:, None] - first
    j = torch.arange(s["max_new"], device=DEV)
    q = s["q"].float()[(first + j).clamp(max=s["q"].shape[0] - 1).long()]
    q = q.view(b, -1, h, case["group"], d)
    t = torch.arange(k.shape[2], device=DEV)
    at = (s["lens"][:, None] - news + j)[:, :, None]           # places of the new tokens
    seen = (t < s["lens"][:, None, None]) & (j < news)[:, :, None]
    if case["causal"]:
        seen = seen & (t <= at)
    if case["window"]:
        seen = seen & (t > at - case["window"])
    token = torch.arange(s["q"].shape[0], device=DEV)
    of = torch.searchsorted(s["starts"], token, right=True) - 1
    return k, v, q, seen, (of, token - s["starts"][of])


def _softmax_plain(s, q, k, v, seen, d):
    """[batch, new, heads, group, channels] and the log of the sums of exponentials."""
    b, new, h, g, _ = q.shape
    x = q.permute(0, 2, 1, 3, 4).reshape(b, h, new * g, -1) @ k.transpose(2, 3)
    x = (x / math.sqrt(d)).view(b, h, new, g, -1)
    if "scale" in s:
        x = x * s["scale"][s["layer"]][:, None, None, None]
    x = torch.where(seen[:, None, :, None, :], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m0)
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, h, new * g, -1) @ v).view(b, h, new, g, -1) / torch.where(total == 0, 1.0, total)
    if "scale" in s:
        o = o * s["scale"][s["layer"]][:, None, None, None]
    lse = (m0 + torch.log(total))[..., 0]
    return o.permute(0, 2, 1, 3, 4), lse.permute(0, 2, 1, 3)


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    if sum(p for _, _, p in _seen(case)) * case["kv_heads"] * case["group"] * case["head_dim"] > 1 << 40:
        return None
    s = prepare(case, seed)
    d, h, group, w = case["head_dim"], case["kv_heads"], case["group"], case["window"]
    n, maps = s["q"].shape[0], 2 if case["op"] == "diff" else 1
    width = d // maps
    scale = s["scale"][s["layer"]].double() if "scale" in s else torch.ones(h, device=DEV).double()
    out = torch.zeros(n, h, group, d, dtype=torch.float64, device=DEV)
    lse = torch.full((n, h, group, maps), -math.inf, dtype=torch.float64, device=DEV)
    lens, starts = s["lens"].tolist(), s["starts"].tolist()
    for i, slot in enumerate(s["slots"].tolist()):
        a, z, total = starts[i], starts[i + 1], lens[i]
        if total == 0 or z == a:
            continue
        for j in range(h):
            rows = [s["pool"][s["table"][slot, s["layer"], side, j, :-(-total // case["page"])].long()]
                    .double().reshape(-1, d)[:total] * scale[j] for side in (0, 1)]
            for c in range(a, z, 512):                         # rows at once
                e = min(z, c + 512)
                at = total - (z - torch.arange(c, e, device=DEV))
                t = torch.arange(total, device=DEV)
                hide = torch.zeros(e - c, total, dtype=torch.bool, device=DEV)
                if case["causal"]:
                    hide |= t > at[:, None]
                if w:
                    hide |= t <= at[:, None] - w
                for m in range(maps):
                    part = slice(m * width, (m + 1) * width)
                    x = torch.einsum("ngd,td->gnt", s["q"][c:e, j * group:(j + 1) * group, part].double(),
                                     rows[0][:, part]) / math.sqrt(width)
                    x.masked_fill_(hide, -math.inf)
                    lse[c:e, j, :, m] = torch.logsumexp(x, -1).T
                    y = (torch.softmax(x, -1) @ rows[1]).transpose(0, 1)
                    lam = s["lam"][j * group:(j + 1) * group].double()[:, None] if m else None
                    out[c:e, j] += -lam * y if m else y
    out, lse = out.view(n, -1, d), lse.view(n, h * group, maps)
    if maps == 1:
        return out, lse[..., 0]
    if s["norm"] is not None:
        out = out * torch.rsqrt(out.square().mean(-1, keepdim=True) + EPS) * s["norm"].double()
    return out, lse


# ---------------------------------------------------------------- work

def work(case):
    d, h, page = case["head_dim"], case["kv_heads"], case["page"]
    hq = h * case["group"]
    maps = 2 if case["op"] == "diff" else 1
    seen = _seen(case)
    tokens = sum(n for _, n, _ in seen)
    pages = sum(-(-(lo + n) // page) - lo // page for lo, n, _ in seen)
    rows = sum(_news(case))
    return {"bytes": tokens * h * 2 * d * _bytes(case) + pages * 2 * h * 4
            + rows * hq * (4 * d + 4 * maps) + 12 * case["batch"],
            "flops": (2.0 + 2.0 * maps) * d * hq * sum(p for _, _, p in seen)}
