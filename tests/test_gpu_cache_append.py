"""The append of new tokens against float64: the turned queries, the rows of the pages,
everything else of the pool untouched.

Tolerances: the angle is formed in fp64 and its sine and cosine are fp32 values within
2^-22, the rotation is two products and a sum in fp32, so before the last rounding a
value is off by at most 2^-20 (|a| + |b|); then bf16 (2^-8) or e4m3 (2^-4, and half of
its smallest step, 2^-10, in code units)."""
import math

import numpy as np
import pytest
import torch

from cache_helpers import ints, skv, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def turned(x, rot, pos, freqs, axis, inter):
    """x [n, heads, d] float64 turned, and |a| + |b| of each channel's pair."""
    x = x.double().cpu()
    y, m = x.clone(), x.abs()
    half = rot // 2
    if half:
        ang = pos.double().cpu()[axis.cpu().long()].T[:, None, :] * freqs.cpu()
        c, s = torch.cos(ang), torch.sin(ang)
        i = torch.arange(half)
        ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + half)
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
        m[..., ia] = m[..., ib] = a.abs() + b.abs()
    return y, m


def near(got, ref, mag, dtype, scale=None):
    if dtype == 0:
        tol = 2.0 ** -8 * ref.abs() + 2.0 ** -20 * mag
    else:
        s = scale
        ref, mag = ref / s, mag / s
        tol = 2.0 ** -4 * ref.abs() + 2.0 ** -10 + 2.0 ** -19 * mag
        over = ref.abs() >= 448
        assert torch.all(got[over].abs() >= 448 * (1 - 2.0 ** -4))
        ref = ref.clamp(-448, 448)
    assert torch.all((got - ref).abs() <= tol), ((got - ref).abs() / tol).max()


CASES = [
    # dtype, n, heads, q_heads, d, rotary, tb, axes, interleaved, start
    (0, 1, 1, 1, 16, 16, 16, 1, False, 0),
    (0, 3, 2, 6, 64, 64, 5, 1, False, 7),
    (0, 3, 2, 6, 64, 64, 5, 1, True, 7),
    (1, 3, 2, 6, 64, 32, 16, 3, False, 0),
    (1, 130, 1, 3, 96, 96, 33, 3, True, 1000000),
    (0, 37, 8, 16, 128, 128, 256, 3, False, 3),
    (0, 5, 3, 0, 128, 64, 1, 4, False, 0),            # no queries
    (1, 9, 2, 2, 128, 0, 128, 1, False, 0),           # no rotation
    (0, 2, 1, 5, 24, 16, 7, 2, False, 0),             # 16 + 8 channels
    (0, 2000, 2, 4, 64, 64, 64, 2, True, 70000),      # four tokens a block
]


@pytest.mark.parametrize("dtype,n,heads,hq,d,rot,tb,axes,inter,start", CASES)
def test_append_matches_float64(dtype, n, heads, hq, d, rot, tb, axes, inter, start):
    P = skv()
    g = torch.Generator(device="cuda").manual_seed(n + d)
    layers, seqs = 2, 3
    blocks = -(-(n + 9) // tb)
    pages = seqs * layers * 2 * heads * blocks + 3
    scale = torch.rand(layers, heads, generator=g, device="cuda") * 0.02 + 0.005 if dtype else None
    c = P.PagedCache(dtype, layers, heads, d, tb, pages, seqs, blocks, scale=scale)
    c.pool.copy_(torch.randint(0, 100, c.pool.shape, generator=g, device="cuda"))
    c.table.copy_(torch.randperm(pages, generator=g, device="cuda")[:c.table.numel()].view_as(c.table))
    c.refs[c.table.flatten().long()] = 1
    # tokens of sequences 2 and 0, in a strided projection output
    slots = ints([2 if i < n - n // 3 else 0 for i in range(n)])
    at = ints([i % (n - n // 3) + 4 for i in range(n)])
    qkv = torch.randn(n, hq + 2 * heads + 1, d, generator=g, device="cuda").bfloat16()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + heads], qkv[:, hq + heads:hq + 2 * heads]
    rope = pos = None
    axis = torch.zeros(rot // 2, dtype=torch.uint8, device="cuda")
    freqs = torch.ones(rot // 2, dtype=torch.float64, device="cuda")
    if rot:
        freqs = 10000.0 ** (-torch.arange(rot // 2, device="cuda").double() * 2 / rot)
        axis = torch.randint(0, axes, (rot // 2,), generator=g, device="cuda").to(torch.uint8)
        rope = P.Rope(freqs, axis if axes > 1 else None, axes, inter)
        pos = start + torch.randint(-5, 50000, (axes, n), generator=g, device="cuda").int()
    want = c.pool.clone()
    out = c.append(1, slots, at, q if hq else None, k, v, rope, pos)
    c.status()
    if hq:
        ref, mag = turned(q, rot, pos, freqs, axis, inter)
        assert out.shape == (n, hq, d) and out.dtype == torch.bfloat16
        near(out.double().cpu(), ref, mag, 0)
    else:
        assert out is None
    kr, km = turned(k, rot, pos, freqs, axis, inter)
    vr, vm = v.double().cpu(), v.double().abs().cpu()
    page = c.table[slots.long(), 1][torch.arange(n), :, :, (at // tb).long()].long()  # [n, 2, heads]
    row = (at % tb).long()
    got = values(c.pool, dtype)
    for side, ref, mag in ((0, kr, km), (1, vr, vm)):
        for h in range(heads):
            x = got[page[:, side, h], row].cpu()
            s = scale[1, h].double().cpu() if dtype else None
            near(x, ref[:, h], mag[:, h], dtype, s)
            if dtype == 0 and side == 1:
                assert torch.equal(x, ref[:, h])
            want[page[:, side, h], row] = c.pool[page[:, side, h], row]
    assert torch.equal(want, c.pool)                   # nothing else was written


def test_in_place_and_any_strides():
    P = skv()
    c = P.PagedCache(P.SKV_BF16, 1, 2, 64, 16, 16, 2, 2)
    c.reserve(ints([0]), ints([0]), ints([9]))
    q = torch.randn(9, 4, 64, device="cuda").bfloat16()
    kv = torch.randn(2, 64 + 16, 9, 2, device="cuda").bfloat16().permute(0, 2, 3, 1).contiguous()
    k, v = kv[0][..., :64], kv[1][..., 8:72]            # rows of 80 channels, an 8-channel offset
    rope = P.Rope(torch.linspace(0.1, 1, 32, dtype=torch.float64, device="cuda"))
    pos = torch.arange(9, device="cuda").int()[None]
    args = (0, ints([0] * 9), ints(range(9)))
    want = c.append(*args, q, k, v, rope, pos)
    got = q.clone()
    assert c.append(*args, got, k, v, rope, pos, q_out=got) is got
    c.status()
    assert torch.equal(want, got)
    p = c.table[0, 0, 1, :, 0].long()
    assert torch.equal(c.pool[p, :9].view(torch.bfloat16), v.permute(1, 0, 2))
    # heads before tokens
    c2 = P.PagedCache(P.SKV_BF16, 1, 2, 64, 16, 16, 2, 2)
    c2.reserve(ints([0]), ints([0]), ints([9]))
    t = lambda x: x.permute(1, 0, 2).contiguous().permute(1, 0, 2)  # noqa: E731
    assert torch.equal(c2.append(*args, t(q), t(k), t(v), rope, pos), want)
    for side in (0, 1):
        assert torch.equal(c.pool[c.table[0, 0, side, :, 0].long(), :9],
                           c2.pool[c2.table[0, 0, side, :, 0].long(), :9])


def test_angles_of_far_positions():
    """Positions up to 2^31 - 1 at freq 1 stay exact: (1, 0) turns to (cos, sin)."""
    P = skv()
    c = P.PagedCache(P.SKV_BF16, 1, 1, 16, 16, 4, 1, 1)
    c.reserve(ints([0]), ints([0]), ints([6]))
    pos = ints([[0, 1, 1 << 20, (1 << 24) + 1, 2 ** 31 - 1, -(2 ** 31)]])
    x = torch.zeros(6, 1, 16, device="cuda").bfloat16()
    x[..., :8] = 1
    f = torch.linspace(0.25, 1, 8, dtype=torch.float64, device="cuda")
    got = c.append(0, ints([0] * 6), ints(range(6)), x, x, x, P.Rope(f), pos).double().cpu()
    ang = pos[0].double().cpu()[:, None] * f.cpu()
    ref = torch.cat([torch.cos(ang), torch.sin(ang)], 1)
    # 2^31 * 2^-53 relative is 2^-22 radians of the reference's own angle
    assert torch.all((got[:, 0] - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -20)


def test_specials():
    P = skv()
    for dtype in (0, 1):
        c = P.PagedCache(dtype, 1, 1, 16, 4, 4, 1, 1)
        c.reserve(ints([0]), ints([0]), ints([2]))
        x = torch.full((2, 1, 16), 3.0, device="cuda").bfloat16()
        x[0, 0, :4] = torch.tensor([math.nan, math.inf, -math.inf, 60000.0])
        c.append(0, ints([0, 0]), ints([0, 1]), x, x, x)
        c.status()
        for side in (0, 1):
            v = values(c.pool[int(c.table[0, 0, side, 0, 0])], dtype).cpu()
            assert math.isnan(v[0, 0]) and torch.all(v[0, 4:] == 3) and torch.all(v[1] == 3)
            top = [math.inf, -math.inf, float(torch.tensor(60000.0).bfloat16())]
            assert v[0, 1:4].tolist() == (top if dtype == 0 else [448, -448, 448])


def test_padding_and_bad_places():
    P = skv()
    c = P.PagedCache(P.SKV_BF16, 1, 2, 64, 16, 64, 3, 2)
    c.reserve(ints([0]), ints([0]), ints([16]))
    c.fork(ints([0]), ints([1]), ints([16]))            # shares its pages with slot 0
    c.status()
    c.pool.zero_()
    x = torch.ones(1, 2, 64, device="cuda").bfloat16()
    q = c.append(0, ints([-1]), ints([5]), x, x, x)      # padding: no error
    c.status()
    assert torch.equal(q, x) and not c.pool.any()
    for slot, at in ((3, 0), (0, -1), (0, 32), (0, 16), (2, 0), (0, 3), (1, 3)):
        q = c.append(0, ints([slot]), ints([at]), x, x, x)
        with pytest.raises(P.SkvError):
            c.status()
        assert torch.equal(q, x) and not c.pool.any()
    c.free(ints([1]))
    c.append(0, ints([0]), ints([3]), x, x, x)           # its own again
    c.status()
    assert int(c.pool.count_nonzero()) == 4 * 64
    bad = P.Rope(torch.ones(32, dtype=torch.float64, device="cuda"),
                 torch.full((32,), 2, dtype=torch.uint8, device="cuda"), axes=2)
    q = c.append(0, ints([0]), ints([3]), x, x, x, bad, ints([[1], [1]]))
    with pytest.raises(P.SkvError):
        c.status()
    assert torch.equal(q, x)                             # not turned


def test_no_tokens_and_another_stream():
    P = skv()
    c = P.PagedCache(P.SKV_BF16, 1, 2, 64, 16, 64, 3, 2)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    e = torch.empty(0, 2, 64, device="cuda").bfloat16()
    assert c.append(0, none, none, e, e, e).shape == (0, 2, 64)
    c.reserve(ints([0]), ints([0]), ints([16]))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x = torch.randn(3, 2, 64, device="cuda").bfloat16()
    s.wait_stream(torch.cuda.current_stream())
    q = c.append(0, ints([0] * 3), ints(range(3)), x, x, x, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(q, x)
    assert torch.equal(c.pool[c.table[0, 0, 0, :, 0].long(), :3].view(torch.bfloat16),
                       x.permute(1, 0, 2))
