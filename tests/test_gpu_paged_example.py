"""The example that codes a cache, decodes it into pages and goes on decoding there."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

EXAMPLES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


@pytest.mark.parametrize("args", [[], ["--e4m3", "--tokens", "512", "--steps", "2"],
                                  ["--tokens", "255", "--steps", "3", "--branches", "1"]],
                         ids=["bf16", "e4m3-full-blocks", "across-a-block"])
def test_paged_decode(args, capsys):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if EXAMPLES not in sys.path:
        sys.path.insert(0, EXAMPLES)
    import lossless_kv_cache_fixed_gb300 as P
    P.build()
    import paged_decode
    paged_decode.main(args)
    assert "one more step" in capsys.readouterr().out
