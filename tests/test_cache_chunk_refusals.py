"""Attention of chunks and differential attention without a GPU: what the host can see is
refused before any device work (every pointer of the C calls is a made-up number)."""
import pytest

from test_cache_binding import D, Library, host_cache, ints
from test_cache_refusals import A, BAD_CACHES, cache


@pytest.fixture(scope="module")
def P():
    import lossless_kv_cache_fixed_gb300 as P
    P.build()
    return P


def call(P, diff, c=None, layer=0, batch=2, tokens=5, max_len=10, window=0, flags=0, reserved=0,
         slots=A, lens=A, begins=None, starts=A, q=A, qs=256, qhs=64, hq=4, scale=0.125, out=A,
         lse=None, ws=A, wsb=1 << 40, lam=A, norm=None, eps=1e-5, diff_reserved=0):
    c = cache(P) if c is None else c
    k = P.SkvChunk(batch, tokens, max_len, window, flags, reserved, slots, lens, begins, starts)
    if diff:
        d = P.SkvDiff(lam, norm, eps, diff_reserved)
        return P.skv_cache_attend_diff(c, layer, k, d, q, qs, qhs, hq, scale, out, lse, ws, wsb, None)
    return P.skv_cache_attend_chunk(c, layer, k, q, qs, qhs, hq, scale, out, lse, ws, wsb, None)


@pytest.mark.parametrize("kw", BAD_CACHES, ids=lambda kw: ",".join("%s=%s" % i for i in kw.items()))
def test_bad_caches(P, kw):
    c = cache(P, **kw)
    assert P.skv_cache_attend_chunk_workspace_bytes(c, 2) == 0
    for diff in (False, True):
        assert call(P, diff, c) == P.SKV_ERR_ARG


@pytest.mark.parametrize("diff", [False, True])
def test_bad_arguments(P, diff):
    for kw in (dict(layer=2), dict(layer=-1), dict(batch=-1), dict(tokens=-1), dict(hq=0), dict(hq=3),
               dict(hq=-2), dict(max_len=-1), dict(max_len=2 ** 31 - 1), dict(window=-1),
               dict(flags=2), dict(reserved=1), dict(slots=None), dict(lens=None), dict(q=None),
               dict(out=None), dict(q=A + 8), dict(out=A + 2), dict(lse=A + 2), dict(begins=A + 1),
               dict(starts=A + 2), dict(starts=None), dict(qs=12), dict(qhs=60), dict(ws=None),
               dict(ws=A + 16), dict(tokens=1 << 30), dict(batch=1 << 30, max_len=1 << 20),
               dict(tokens=1 << 28, max_len=1 << 20),
               dict(c=cache(P, head_dim=264), qhs=264)):
        assert call(P, diff, **kw) == P.SKV_ERR_ARG, kw
    for kw in (dict(tokens=0), dict(batch=0)):                 # nothing to do
        assert call(P, diff, slots=None, lens=None, q=None, out=None, ws=None, **kw) == P.SKV_OK


def test_bad_arguments_of_differential_attention(P):
    for kw in (dict(lam=None), dict(lam=A + 2), dict(norm=A + 1), dict(eps=-1.0),
               dict(eps=float("nan")), dict(diff_reserved=1), dict(c=cache(P, head_dim=72), qhs=72)):
        assert call(P, True, **kw) == P.SKV_ERR_ARG, kw


def test_the_binding_refuses_bad_tensors(P):
    torch = pytest.importorskip("torch")
    library = Library()
    c = host_cache(P, library)
    c._chunk_bytes = {4: 4096}
    q = torch.zeros(5, 4, D, dtype=torch.bfloat16)
    two, starts, lam = ints(0, 1), ints(0, 3, 5), torch.zeros(4)
    good = dict(slots=two, lens=two, starts=starts, q=q, max_len=8)
    for kw in (dict(slots=two.long()), dict(lens=ints(1)), dict(starts=ints(0, 3)), dict(starts=None),
               dict(q=q.float()), dict(q=q[:, :, :32]), dict(begins=ints(0)),
               dict(out=q.float()), dict(out=q[:4]), dict(out=q.transpose(0, 1))):
        with pytest.raises(P.SkvError):
            c.attend_chunk(0, **{**good, **kw})
    good["lam"] = lam
    for kw in (dict(lam=lam[:3]), dict(lam=lam.double()), dict(norm=torch.zeros(D - 1)),
               dict(norm=torch.zeros(D).bfloat16()), dict(starts=None), dict(q=q.float()),
               dict(lens=ints(1)), dict(out=q[:4])):
        with pytest.raises(P.SkvError):
            c.attend_diff(0, **{**good, **kw})
    assert not library.calls
    c.attend_chunk(0, two, two, starts, q, 8)
    c.attend_diff(0, two, two, q, lam, 8, starts=starts, norm=torch.zeros(D))
    c.attend_diff(0, two, two, q[:2], lam, 8)
    assert [n for n, _ in library.calls] == ["skv_cache_attend_chunk"] + ["skv_cache_attend_diff"] * 2


def test_strides_of_dimensions_of_one(P):
    import torch
    library = Library()
    c = host_cache(P, library)
    c._chunk_bytes = {4: 4096}
    q = torch.zeros(4, D, 1, dtype=torch.bfloat16).permute(2, 0, 1)      # one token
    c.attend_chunk(0, ints(0), ints(1), ints(0, 1), q, 8)
    c.attend_diff(0, ints(0), ints(1), q, torch.zeros(4), 8)
    assert [(a[4] if "chunk" in n else a[5]) % 8 for n, a in library.calls] == [0, 0]
