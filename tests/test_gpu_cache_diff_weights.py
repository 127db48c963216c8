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
