"""Shapes at the edge of what a launch takes."""
import pytest
import torch

from cache_helpers import ints, skv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("heads", list(range(3052, 3073, 2)) + [4000, 8192])
def test_append_of_thousands_of_heads(dtype, heads):
    """A block's rows take 16 bytes of shared memory each: around the 48 KB that a launch has
    without asking, of which the kernel's own variables take their part."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    P = skv()
    c = P.PagedCache(dtype, 1, 1, 16, 4, 4, 1, 1)
    c.reserve(ints([0]), ints([0]), ints([1]))
    q = torch.randn(1, heads - 2, 16, device="cuda").bfloat16()
    x = torch.ones(1, 1, 16, device="cuda").bfloat16()
    rope = P.Rope(torch.zeros(8, dtype=torch.float64, device="cuda"))
    out = c.append(0, ints([0]), ints([0]), q, x, x, rope, ints([[7]]))
    c.status()
    assert torch.equal(out, q)                        # angle 0
