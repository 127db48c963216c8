"""How precisely the weights of differential chunks meet the values: two maps that attend to the same
tokens nearly cancel, and what their weights are off by does not."""
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


@pytest.mark.parametrize("d", [16, 64, 80, 96, 128, 192, 256])
@pytest.mark.parametrize("n,new", [(150, 60), (300, 40), (1000, 300), (9000, 40), (2500, None)])
@pytest.mark.parametrize("lam", [0.8, 1.0, -0.5])
def test_maps_that_attend_to_the_same_tokens(d, n, new, lam):
    """bf16 weights in two parts: 2^-16 of each (2^-18 for what keeps the rest above 0), the scores' and
    sums' roundings as in chunk_helpers, and half a step of the result."""
    c = filled(0, 1, 1, d, 64, 1, n)
    pool = c.pool.view(torch.bfloat16)
    rows = new or 1
    q = queries(rows, 2, d).abs() + 0.05
    q = q.bfloat16()
    for t in (n // 7, n // 3):                               # keys along the queries of both maps
        pool[int(c.table[0, 0, 0, 0, t // 64]), t % 64] = 0.5
    out, lse = c.attend_diff(0, ints([0]), ints([n]), q, torch.full((2,), lam, device="cuda"), n,
                             starts=None if new is None else ints([0, new]), lse=True)
    c.status()
    k, v = rows_of(c, 0, 0, 0, 0, n)
    ok = seen(n - rows + torch.arange(rows, device="cuda"), n, 0, 0, True)
    f = torch.tensor(lam).float().item()
    for h in (0, 1):
        ref, tol = 0.0, 0.0
        for m, by in ((0, 1.0), (1, f)):
            part = slice(m * d // 2, (m + 1) * d // 2)
            scale = (d // 2) ** -0.5
            o, rl, _, e = one_map(0, q[:, h, part].double(), k[:, part], v, ok, scale)
            assert torch.all((lse[:, h, m].double() - rl).abs() <= e)
            w = torch.softmax((q[:, h, part].double() @ k[:, part].T * scale).masked_fill(~ok, -math.inf), 1)
            ref = ref + (o if m == 0 else -by * o)
            tol = tol + abs(by) * (2.0 ** -16 + 2.0 ** -18 + 2 * e[:, None]) * (w @ v.abs())
        tol = tol + 2.0 ** -22 * ref.abs()
        off = (out[:, h].double() - ref).abs()
        assert torch.all(off <= tol + 2.0 ** -8 * (ref.abs() + tol)), (h, float((off / (tol + 2.0 ** -8 * ref.abs())).max()))


@pytest.mark.parametrize("d", [64, 80, 256])
@pytest.mark.parametrize("n,new", [(150, 60), (3000, 20), (3000, 300)])
def test_growing_scores(d, n, new):
    """Scores that grow along the rows by far more than the slack of the running maximum, plain and
    times large and small numbers, in bf16 and within the same bound."""
    c = filled(0, 1, 1, d, 16, 1, n)
    pool = c.pool.view(torch.bfloat16)
    f = torch.linspace(0.01, 2.0, n, device="cuda")
    t = torch.arange(n, device="cuda")
    rows = c.table[0, 0, 0, 0, t // 16].long()
    pool[rows, t % 16] = (pool[rows, t % 16].float() * f[:, None]).bfloat16()
    q0 = queries(new, 2, d, 2).float()
    k, v = rows_of(c, 0, 0, 0, 0, n)
    ok = seen(n - new + torch.arange(new, device="cuda"), n, 0, 0, True)
    for mul, scale in ((8.0, None), (1e-6, None), (0.0, None), (1.0, -0.3), (1e4, 1e-5), (64.0, None)):
        q = (q0 * mul).bfloat16()
        out, lse = c.attend_diff(0, ints([0]), ints([n]), q, torch.full((2,), 0.7, device="cuda"), n,
                                 starts=ints([0, new]), scale=scale, lse=True)
        c.status()
        sc = (d // 2) ** -0.5 if scale is None else scale
        by = torch.tensor(0.7).item()
        for h in (0, 1):
            ref, tol = 0.0, 0.0
            for m in (0, 1):
                part = slice(m * d // 2, (m + 1) * d // 2)
                o, rl, _, e = one_map(0, q[:, h, part].double(), k[:, part], v, ok, sc)
                assert torch.all((lse[:, h, m].double() - rl).abs() <= e + 2.0 ** -22 * rl.abs())
                w = torch.softmax((q[:, h, part].double() @ k[:, part].T * sc).masked_fill(~ok, -math.inf), 1)
                ref = ref + (o if m == 0 else -by * o)
                tol = tol + (1.0 if m == 0 else by) * (2.0 ** -16 + 2.0 ** -18 + 2 * e[:, None]) * (w @ v.abs())
            tol = tol + 2.0 ** -22 * ref.abs() + 1e-30
            off = (out[:, h].double() - ref).abs()
            assert torch.all(off <= tol + 2.0 ** -8 * (ref.abs() + tol)), (h, mul)


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 80, 128, 256])
@pytest.mark.parametrize("n,new", [(600, 4), (600, 90), (5000, 90), (600, None)])
def test_scores_that_get_huge_next_to_rows_whose_are(dtype, d, n, new):
    """Of two heads, neighbours in a warp, one has huge scores from the first token on, the other from
    token 400 on, which takes all of the first map's weight: with lambda 0 its result is that token's
    value, whatever the other head holds."""
    c = filled(dtype, 1, 1, d, 64, 1, n, scaled=False)
    pool = c.pool.view(torch.bfloat16) if dtype == 0 else c.pool
    t = torch.arange(n, device="cuda")
    rows = c.table[0, 0, 0, 0, t // 64].long()
    pool[rows, t % 64] = 0
    pool[rows, t % 64, 0] = 1.0 if dtype == 0 else 0x38                  # 1
    pool[rows[400], 400 % 64, 1] = 2.0 ** 14 if dtype == 0 else 0x7E     # 448
    m = new or 1
    q = torch.zeros(m, 2, d, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(6)
    q[:, 0, 0] = 2.0 ** 25
    q[:, 1, 1] = 2.0 ** 26 * (1 + 63 / 64 * torch.rand(m, generator=g, device="cuda")) * (1 if dtype == 0 else 2.0 ** 4)
    q = q.bfloat16()
    more = dict(starts=None if new is None else ints([0, new]), lse=True)
    lam = torch.zeros(2, device="cuda")
    out, lse = c.attend_diff(0, ints([0]), ints([n]), q, lam, n, **more)
    k, v = rows_of(c, dtype, 0, 0, 0, n)
    assert torch.equal(out[:, 1].double(), v[400].expand(m, d))
    want = q[:, 1, 1].double() * k[400, 1] * (d // 2) ** -0.5
    assert torch.all((lse[:, 1, 0].double() - want).abs() <= 2.0 ** -21 * want)
    calm = q.clone()
    calm[:, 0, 0] = 1.0
    o, l = c.attend_diff(0, ints([0]), ints([n]), calm, lam, n, **more)
    assert torch.equal(o[:, 1], out[:, 1]) and torch.equal(l[:, 1], lse[:, 1])
    c.status()
