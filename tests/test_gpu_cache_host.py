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
