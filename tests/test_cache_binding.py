"""What PagedCache does on the host around the calls of the library, without a GPU: its
tensors lie in host memory and the library is a stand-in that records its calls."""
import threading
import time

import pytest
import torch

D, TB, HEADS = 64, 16, 2


@pytest.fixture(scope="module")
def P():
    import lossless_kv_cache_fixed_gb300 as P
    P.build()
    return P


class Device(torch.Tensor):
    """A host tensor that PagedCache takes for one on its device."""
    is_cuda = property(lambda self: True)


class Library:
    """Stands in for the library: records the arguments of each call and how many calls are
    inside at once; every call takes a while, as one with several launches does."""

    def __init__(self, seconds=0.0):
        self.seconds, self.calls = seconds, []
        self.inside = self.most = 0
        self.guard = threading.Lock()

    def __getattr__(self, name):
        def call(*args):
            with self.guard:
                self.inside += 1
                self.most = max(self.most, self.inside)
                self.calls.append((name, args))
            time.sleep(self.seconds)
            with self.guard:
                self.inside -= 1
            return 0
        return call


def host_cache(P, library, pages=8):
    pool = torch.zeros(pages, TB, D, dtype=torch.int16).as_subclass(Device)
    table = torch.full((2, 1, 2, HEADS, 2), -1, dtype=torch.int32)
    c = P.PagedCache(P.SKV_BF16, 1, HEADS, D, TB, pool=pool, table=table,
                     refs=torch.zeros(pages, dtype=torch.int32))
    c._lib = library
    c._index = -1                                   # what get_device() says of host tensors
    c._current_device, c._raw_stream = (lambda: -1), (lambda index: 5)
    c._capturing = lambda: False
    c._empty = lambda shape, strides, dtype: torch.empty_strided(shape, strides, dtype=dtype)
    c._attend_bytes = {4: 4096}
    return c


def ints(*v):
    return torch.tensor(v, dtype=torch.int32)


def test_threads_on_one_stream_do_not_mix_their_launches(P):
    """A call of several launches hands data from one to the next in the stream's workspace,
    so no other call on it may be enqueued in between, from whichever thread."""
    library = Library(0.02)
    c = host_cache(P, library)
    q = torch.zeros(1, 4, D, dtype=torch.bfloat16)
    calls = [lambda: c.attend(0, ints(0), ints(1), q, 8), lambda: c.attend(0, ints(1), ints(3), q, 8),
             lambda: c.reserve(ints(0), ints(0), ints(4)), lambda: c.fork(ints(0), ints(1), ints(4)),
             lambda: c.compact(), lambda: c.free(ints(1)), lambda: c.clear()]
    threads = [threading.Thread(target=f) for f in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert sorted(n for n, _ in library.calls) == sorted(
        ["skv_cache_attend"] * 2 + ["skv_cache_" + n for n in ("reserve", "fork", "compact", "free",
                                                              "init")])
    assert library.most == 1


@pytest.mark.parametrize("side", ["src_pool", "dst_pool"])
def test_a_pool_without_pages_is_not_the_caches_own(P, side):
    """The library takes a null pool for the cache's own, and an empty tensor's address is
    null: such a pool is refused, not written to or read from in another's place."""
    library = Library()
    c = host_cache(P, library)
    none = torch.empty(0, TB, D, dtype=torch.int16)
    assert none.data_ptr() == 0
    with pytest.raises(P.SkvError):
        c.copy_pages(ints(1), ints(2), **{side: none})
    assert not library.calls


class Copies(torch.utils._python_dispatch.TorchDispatchMode):
    """Records torch's own copies: where from, and how many calls the library had had by then."""

    def __init__(self, library):
        super().__init__()
        self.library, self.seen = library, []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        if func is torch.ops.aten.copy_.default:
            last = (args + ((kwargs or {}).get("non_blocking", False),))[2]
            self.seen.append((args[1].untyped_storage().data_ptr(), last, len(self.library.calls)))
        return func(*args, **(kwargs or {}))


@pytest.mark.parametrize("side", ["src_pool", "dst_pool"])
def test_a_pinned_pool_lives_until_its_copy_is_done(P, side):
    """A kernel reads or writes the pool after the call has returned, and the caller may have
    dropped it by then: torch's allocator learns of it from a copy behind the kernel."""
    library = Library()
    c = host_cache(P, library)
    pool = torch.zeros(4, TB, D, dtype=torch.int16)
    with Copies(library) as copies:
        c.copy_pages(ints(1), ints(2), **{side: pool})
        assert copies.seen == [(pool.data_ptr(), True, 1)]
        # not for device pools, nor while a graph is captured
        c.copy_pages(ints(1), ints(2))
        c.copy_pages(ints(1), ints(2), **{side: pool.clone().as_subclass(Device)})
        c._capturing = lambda: True
        copies.seen.clear()
        c.copy_pages(ints(1), ints(2), **{side: pool})
        assert not copies.seen


def test_strides_of_dimensions_of_one_do_not_matter(P):
    """One token, or one head: torch keeps any stride there, and no address depends on it."""
    library = Library()
    c = host_cache(P, library)
    q = torch.zeros(4, D, 1, dtype=torch.bfloat16).permute(2, 0, 1)      # one token
    assert q.is_contiguous() and q.stride(0) == 1
    c.attend(0, ints(0), ints(1), q, 8)
    (name, args), = library.calls
    assert name == "skv_cache_attend" and args[7] % 8 == 0 and args[8] == D
    kv = torch.zeros(HEADS, D, 1, dtype=torch.bfloat16).permute(2, 0, 1)
    c.append(0, ints(0), ints(0), q, kv, kv)
    wide = torch.zeros(3, D, 5, dtype=torch.bfloat16)
    one = torch.as_strided(wide, (3, 1, D), (D, 3, 1))                   # one query head of three tokens
    kv = torch.zeros(3, HEADS, D, dtype=torch.bfloat16)
    c.append(0, ints(0, 0, 0), ints(0, 1, 2), one, kv, kv)
    for _, args in library.calls[1:]:
        t = args[3]._obj
        assert all(getattr(t, f) % 8 == 0 for f, _ in P.SkvTokens._fields_ if "stride" in f)
    assert library.calls[2][1][3]._obj.q_stride == D
