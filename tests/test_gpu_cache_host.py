"""Host threads and host memory around the paged cache's calls."""
import threading

import pytest
import torch

from cache_helpers import ints, skv
from test_gpu_cache_attend import filled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def test_threads_that_attend_on_one_stream():
    """Rows that are cut and joined: two kernels a call, with parts in the stream's workspace."""
    c = filled(0, 2, 2, 128, 64, 2, 3000)
    g = torch.Generator(device="cuda").manual_seed(4)
    q = [torch.randn(2, 8, 128, generator=g, device="cuda").bfloat16() for _ in range(4)]
    lens = [ints(v) for v in ([3000, 10], [77, 2999], [2500, 2500], [3000, 3000])]
    slots = ints([0, 1])
    want = [c.attend(i % 2, slots, lens[i], q[i], 3000, lse=True) for i in range(4)]
    got = [[] for _ in range(4)]
    torch.cuda.synchronize()

    def work(i):
        for _ in range(200):
            got[i].append(c.attend(i % 2, slots, lens[i], q[i], 3000, lse=True))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    c.status()
    for i in range(4):
        assert len(got[i]) == 200
        for o, l in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


@pytest.mark.parametrize("other", [False, True], ids=["current", "another-stream"])
def test_a_dropped_pinned_pool(other):
    """The caller drops the host pool while its copy waits behind other work; memory of the
    same size that it asks for next is not the pool's."""
    P = skv()
    c = P.PagedCache(P.SKV_BF16, 1, 1, 64, 16, 8, 1, 1)
    stream = torch.cuda.Stream() if other else torch.cuda.current_stream()
    data = torch.randint(-2 ** 15, 2 ** 15, (4, 16, 64), dtype=torch.int16)
    src, dst = ints([0, 1, 2, 3]), ints([4, 5, 6, 7])
    for _ in range(5):
        c.pool.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            torch.cuda._sleep(20_000_000)
        host = data.pin_memory()
        c.copy_pages(src, dst, src_pool=host, stream=stream if other else None)
        del host
        after = [torch.zeros(4, 16, 64, dtype=torch.int16).pin_memory() for _ in range(3)]
        torch.cuda.synchronize()
        c.status()
        assert torch.equal(c.pool[4:].cpu(), data)
        assert all(not t.any() for t in after)


# One thread captures a graph (in torch's default mode, which forbids calls that wait or ask
# for events in every thread), another copies pages to host memory meanwhile.
CAPTURE = """
import sys, threading
sys.path[:0] = [%r]
import torch
import lossless_kv_cache_fixed_gb300 as P
c = P.PagedCache(P.SKV_BF16, 1, 1, 64, 16, num_pages=8, max_seqs=1, max_blocks=1)
c.pool.copy_(torch.arange(c.pool.numel(), device="cuda").view_as(c.pool) %% 30000)
ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
src, dst = ints(3, 4), ints(0, 1)
hosts = [torch.zeros(2, 16, 64, dtype=torch.int16).pin_memory() for _ in range(5)]
side, stream = torch.cuda.Stream(), torch.cuda.Stream()
c.copy_pages(src, dst, dst_pool=hosts[0], stream=side)
x = torch.ones(1000, device="cuda")
torch.cuda.synchronize()
go, done, errors = threading.Event(), threading.Event(), []
def work():
    go.wait()
    try:
        for h in hosts[1:]:
            c.copy_pages(src, dst, dst_pool=h, stream=side)
    except Exception as e:
        errors.append(e)
    done.set()
t = threading.Thread(target=work); t.start()
graph = torch.cuda.CUDAGraph()
with torch.cuda.stream(stream):
    graph.capture_begin()
    x.add_(1)
    go.set(); done.wait()
    x.add_(1)
    graph.capture_end()
t.join()
graph.replay()
torch.cuda.synchronize()
print("captured", float(x[0]) == 3.0, errors, all(torch.equal(h, c.pool[3:5].cpu()) for h in hosts),
      flush=True)
"""


def test_host_copies_while_another_thread_captures():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CAPTURE % root], capture_output=True, text=True,
                       timeout=120)
    assert "captured True [] True" in r.stdout, (r.stdout, r.stderr[-2000:])
