"""The paged cache's C ABI without a GPU: what the host can see is refused before any
device work (every pointer here is a made-up number, so a launch would fail otherwise)."""
import pytest


@pytest.fixture(scope="module")
def P():
    import lossless_kv_cache_fixed_gb300 as P
    P.build()
    return P


A = 1 << 20  # an aligned address that nothing lies at


def cache(P, **kw):
    v = dict(dtype=P.SKV_BF16, layers=2, heads=2, head_dim=64, page_tokens=16, max_seqs=4,
             max_blocks=8, flags=0, num_pages=64, pool=A, table=A, refs=A, status=A, scale=None)
    v.update(kw)
    return P.SkvCache(*(v[f] for f, _ in P.SkvCache._fields_))


BAD_CACHES = [dict(dtype=2), dict(flags=1), dict(layers=0), dict(heads=-1), dict(head_dim=60),
              dict(head_dim=0), dict(page_tokens=0), dict(max_seqs=0), dict(max_blocks=0),
              dict(num_pages=0), dict(num_pages=0xFFFFFFFF), dict(pool=None), dict(pool=A + 8),
              dict(table=None), dict(table=A + 2), dict(refs=None), dict(status=None),
              dict(scale=A),                               # e4m3 only
              dict(dtype=1, head_dim=72),                  # e4m3 rows of whole 16 bytes
              dict(page_tokens=1 << 28),                   # page bytes past 31 bits
              dict(layers=1 << 15, heads=1 << 14, max_blocks=4)]


@pytest.mark.parametrize("kw", BAD_CACHES, ids=lambda kw: ",".join("%s=%s" % i for i in kw.items()))
def test_every_call_refuses_a_bad_cache(P, kw):
    c = cache(P, **kw)
    t = P.SkvTokens(A, A, A, 64, 64, 64, 64, 64, 64)
    assert P.skv_cache_workspace_bytes(c, 1) == 0
    assert P.skv_cache_attend_workspace_bytes(c, 1, 2) == 0
    for rc in (P.skv_cache_init(c, None), P.skv_cache_status(c, None),
               P.skv_cache_reserve(c, A, A, A, 1, A, 1 << 30, None),
               P.skv_cache_fork(c, A, A, A, 1, A, 1 << 30, None),
               P.skv_cache_free(c, A, 1, None),
               P.skv_cache_compact(c, None, None, A, 1 << 30, None),
               P.skv_cache_copy_pages(c, None, 0, A, None, 0, A, 1, None),
               P.skv_cache_append(c, 0, None, t, A, A, None, 1, 2, A, None),
               P.skv_cache_attend(c, 0, A, A, None, 1, A, 128, 64, 2, 0.1, 10, A, None, A, 1 << 30,
                                  None)):
        assert rc == P.SKV_ERR_ARG


def test_page_calls_refuse_bad_arguments(P):
    c = cache(P)
    ws = P.skv_cache_workspace_bytes(c, 3)
    assert ws > 0 and ws % 256 == 0
    assert P.skv_cache_workspace_bytes(c, -1) == 0 and P.skv_cache_workspace_bytes(c, 65536) == 0
    for call in (P.skv_cache_reserve, P.skv_cache_fork):
        for args in ((None, A, A, 3, A, ws), (A, None, A, 3, A, ws), (A, A, None, 3, A, ws),
                     (A + 2, A, A, 3, A, ws), (A, A, A, -1, A, ws), (A, A, A, 65536, A, 1 << 30),
                     (A, A, A, 3, None, ws), (A, A, A, 3, A + 64, ws)):
            assert call(c, *args, None) == P.SKV_ERR_ARG, args
        assert call(c, A, A, A, 3, A, ws - 1, None) == P.SKV_ERR_CAPACITY
        assert call(c, A, A, A, 0, A, ws, None) == P.SKV_OK        # nothing to do
    assert P.skv_cache_free(c, None, 1, None) == P.SKV_ERR_ARG
    assert P.skv_cache_free(c, A, -1, None) == P.SKV_ERR_ARG
    assert P.skv_cache_free(c, None, 0, None) == P.SKV_OK
    ws0 = P.skv_cache_workspace_bytes(c, 0)
    for t, r in ((A + 64, None), (None, A + 64), (A + 2, A + 64), (A, A + 64), (A + 64, A)):
        assert P.skv_cache_compact(c, t, r, A, ws0, None) == P.SKV_ERR_ARG, (t, r)
    assert P.skv_cache_compact(c, None, None, A, ws0 - 1, None) == P.SKV_ERR_CAPACITY
    for args in ((None, 0, None, None, 0, A, 1), (None, 0, A, None, 0, None, 1),
                 (A + 8, 4, A, None, 0, A, 1), (None, 0, A, A + 8, 4, A, 1),
                 (None, 0, A, None, 0, A, -1)):
        assert P.skv_cache_copy_pages(c, *args, None) == P.SKV_ERR_ARG, args
    assert P.skv_cache_copy_pages(c, None, 0, None, None, 0, None, 0, None) == P.SKV_OK


def test_append_refuses_bad_arguments(P):
    c = cache(P)
    good = dict(q=A, k=A, v=A, q_stride=256, q_head_stride=64, k_stride=256, k_head_stride=64,
                v_stride=256, v_head_stride=64)
    rope = P.SkvRope(64, 1, 0, 0, A, None)

    def call(layer=0, r=rope, slots=A, at=A, pos=A, n=2, hq=4, out=A, **kw):
        t = P.SkvTokens(*({**good, **kw}[f] for f, _ in P.SkvTokens._fields_))
        return P.skv_cache_append(c, layer, r, t, slots, at, pos, n, hq, out, None)

    for kw in (dict(layer=2), dict(layer=-1), dict(n=-1), dict(hq=-1), dict(slots=None),
               dict(at=None), dict(pos=None), dict(out=None), dict(out=A + 8), dict(q=None),
               dict(k=None), dict(v=A + 2), dict(q_stride=252), dict(q_head_stride=4),
               dict(k_stride=1), dict(k_head_stride=63), dict(v_stride=7), dict(v_head_stride=2),
               dict(at=A + 2)):
        assert call(**kw) == P.SKV_ERR_ARG, kw
    for r in (P.SkvRope(24, 1, 0, 0, A, None), P.SkvRope(80, 1, 0, 0, A, None),
              P.SkvRope(-16, 1, 0, 0, A, None), P.SkvRope(64, 0, 0, 0, A, None),
              P.SkvRope(64, 5, 0, 0, A, None), P.SkvRope(64, 1, 2, 0, A, None),
              P.SkvRope(64, 1, 0, 1, A, None), P.SkvRope(64, 1, 0, 0, None, None),
              P.SkvRope(64, 1, 0, 0, A + 4, None)):
        assert call(r=r) == P.SKV_ERR_ARG, [getattr(r, f) for f, _ in r._fields_]
    assert call(n=0, slots=None, at=None, pos=None) == P.SKV_OK


def test_attend_refuses_bad_arguments(P):
    c = cache(P)

    def call(c=c, layer=0, slots=A, lens=A, begins=None, batch=1, q=A, qs=256, qhs=64, hq=4,
             max_len=10, out=A, lse=None, ws=A, wsb=1 << 30):
        return P.skv_cache_attend(c, layer, slots, lens, begins, batch, q, qs, qhs, hq, 0.125,
                                  max_len, out, lse, ws, wsb, None)

    for kw in (dict(layer=2), dict(layer=-1), dict(batch=-1), dict(hq=0), dict(hq=3), dict(hq=-2),
               dict(max_len=-1), dict(max_len=2 ** 31 - 1), dict(slots=None), dict(lens=None),
               dict(q=None), dict(out=None), dict(q=A + 8), dict(out=A + 2), dict(lse=A + 2),
               dict(begins=A + 1), dict(qs=12), dict(qhs=60), dict(ws=None), dict(ws=A + 16),
               dict(batch=1 << 30, hq=4), dict(c=cache(P, head_dim=264), qhs=264)):
        assert call(**kw) == P.SKV_ERR_ARG, kw
    assert call(batch=0, slots=None, lens=None, q=None, out=None, ws=None) == P.SKV_OK


def test_python_wrappers_refuse_bad_tensors(P):
    torch = pytest.importorskip("torch")
    f = torch.ones(32, dtype=torch.float64)
    with pytest.raises(P.SkvError):
        P.Rope(f.float())
    with pytest.raises(P.SkvError):
        P.Rope(f, torch.zeros(32))
    with pytest.raises(P.SkvError):
        P.Rope(f, axes=5)
    with pytest.raises(P.SkvError):
        P.Rope(torch.ones(12, dtype=torch.float64))
    pool = torch.zeros(8, 16, 64, dtype=torch.int16)
    table = torch.full((2, 1, 2, 2, 2), -1, dtype=torch.int32)
    refs = torch.zeros(8, dtype=torch.int32)
    for kw in (dict(pool=pool.float()), dict(pool=pool[:, ::2]), dict(table=table.long()),
               dict(table=table[..., :1]), dict(refs=refs[:4]), dict(refs=None),
               dict(scale=torch.ones(1, 2)), {}):            # {}: not on a GPU
        args = dict(pool=pool, table=table, refs=refs)
        args.update(kw)
        with pytest.raises(P.SkvError):
            P.PagedCache(P.SKV_BF16, 1, 2, 64, 16, **args)
    with pytest.raises(P.SkvError):
        P.PagedCache(P.SKV_BF16, 1, 2, 64, 16, num_pages=8, device="cpu")
