"""A CUDA error that a call of the paged cache reports is not reported again by the coder."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# status() waits for its stream, which a capture refuses on the host.
CHILD = """
import sys
sys.path[:0] = [%r, %r]
import torch
import lossless_kv_cache_fixed_gb300 as P
import paged_decode, synth
spec = synth.WORKLOADS["qwen3-0.6b-e4m3"].scaled(name="errors", L=1, H=1, T=256, calib_draws=1)
w, kv, mu, codec, host = paged_decode.coded_prompt(spec)
cache = P.PagedCache(P.SKV_BF16, 1, 1, 64, 16, num_pages=8, max_seqs=1, max_blocks=1)
torch.cuda.synchronize()
graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.stream(stream):
    graph.capture_begin()
    try:
        cache.status()
        print("no error")
    except P.SkvError as e:
        print("refused", e.status)
    try:
        graph.capture_end()
    except RuntimeError:
        pass
torch.cuda.synchronize()
buf, nbytes = codec.encode(kv, mu)
print("encoded", nbytes == host.numel(), flush=True)
"""


def test_a_reported_error_does_not_stay():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", CHILD % (ROOT, os.path.join(ROOT, "examples"))],
                       capture_output=True, text=True, timeout=120)
    assert "refused -6" in r.stdout and "encoded True" in r.stdout, (r.stdout, r.stderr[-2000:])
