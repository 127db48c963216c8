"""Windows over caches whose pages before the window are gone."""
import pytest
import torch

from cache_helpers import check_attend, ints
from test_gpu_cache_attend import filled

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tb", [1, 5, 16, 24, 33, 64])
def test_pages_before_the_window_may_be_missing(dtype, d, tb):
    """What lies outside the range has no effect: no error, and the same bits."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    begins = [16, 48, 47, 49, 33, 150, 0, 199, 64]
    lens = [150, 200, 90, 49, 150, 151, 77, 200, 64]
    c = filled(dtype, 1, 2, d, tb, len(lens), 200, seed=tb)
    g = torch.Generator(device="cuda").manual_seed(tb)
    q = torch.randn(len(lens), 4, d, generator=g, device="cuda").bfloat16()
    args = (0, ints(range(len(lens))), ints(lens), q, 200)
    out, lse = c.attend(*args, begins=ints(begins), lse=True)
    c.status()
    check_attend(c, dtype, 0, range(len(lens)), begins, lens, q, d ** -0.5, out, lse)
    for s, (a, n) in enumerate(zip(begins, lens)):
        c.table[s, ..., :a // tb] = -1
        c.table[s, ..., -(-n // tb):] = -1
    o2, l2 = c.attend(*args, begins=ints(begins), lse=True)
    c.status()
    assert torch.equal(out, o2) and torch.equal(lse, l2)
