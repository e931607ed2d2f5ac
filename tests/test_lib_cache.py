"""Host-side refusals of the prompt and cache calls (CPU: every call here fails its
checks, or has nothing to do, before it reaches a CUDA API)."""
import ctypes

import pytest
import torch

import block_diffusion_speculative_attn_gb300 as bdsa

A = 0x100000  # never dereferenced
M = 0x10000000  # apart from everything else


@pytest.fixture(scope="module")
def L():
    from block_diffusion_speculative_attn_gb300 import build
    build.build()
    return bdsa.lib()


def _chunk(L, **kw):
    a = dict(q=A, qs=1024, k=A, v=A, bt=A, mp=4, np=8, sl=A, cu=A, bs=2, T=10, Hq=8, Hkv=2,
             D=128, ps=16, scale=0.1, mb=1, out=M, lse=2 * M, ws=3 * M, wsb=1 << 40, sms=152)
    a.update(kw)
    return L.bdsa_chunk_attn_paged(a["q"], a["qs"], a["k"], a["v"], a["bt"], a["mp"], a["np"],
                                   a["sl"], a["cu"], a["bs"], a["T"], a["Hq"], a["Hkv"], a["D"],
                                   a["ps"], a["scale"], a["mb"], a["out"], a["lse"], a["ws"],
                                   a["wsb"], a["sms"], None, None)


def test_chunk_refusals(L):
    assert _chunk(L, bs=0) == 0 and _chunk(L, T=0) == 0
    for kw in (dict(bs=-1), dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=7), dict(mp=0),
               dict(np=0), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(mb=0), dict(qs=1023), dict(q=None), dict(k=None), dict(v=None), dict(bt=None),
               dict(sl=None), dict(cu=None), dict(out=None)):
        assert _chunk(L, **kw) == 1, kw
    for kw in (dict(D=96), dict(D=256), dict(Hq=258, qs=258 * 128), dict(ps=4), dict(ps=24),
               dict(np=1 << 28), dict(mb=(1 << 30) + 1), dict(T=2 ** 31 - 1), dict(qs=1 << 30)):
        assert _chunk(L, **kw) == 2, kw
    for kw in (dict(q=A + 8), dict(k=A + 8), dict(v=A + 8), dict(out=M + 8), dict(lse=2 * M + 2),
               dict(ws=3 * M + 128), dict(qs=1028)):
        assert _chunk(L, **kw) == 3, kw
    need = L.bdsa_chunk_attn_workspace_bytes(128, 152)
    assert need > 0 and L.bdsa_chunk_attn_workspace_bytes(96, 152) == 0
    assert _chunk(L, ws=None) == 4 and _chunk(L, wsb=need - 1) == 4
    # outputs over inputs or one another
    for kw in (dict(out=A), dict(lse=A + 1024), dict(ws=A), dict(lse=M + 16), dict(ws=M),
               dict(out=M, q=M + 2 * 9 * 1024), dict(ws=2 * M)):
        assert _chunk(L, **kw) == 1, kw


def _write(L, **kw):
    a = dict(k=A, ks=4096, v=A + 2048, vs=4096, sm=A, T=10, kc=M, vc=2 * M, rb=2048, ns=100)
    a.update(kw)
    return L.bdsa_cache_write(a["k"], a["ks"], a["v"], a["vs"], a["sm"], a["T"], a["kc"], a["vc"],
                              a["rb"], a["ns"], None, None)


def test_write_refusals(L):
    assert _write(L, T=0) == 0
    for kw in (dict(T=-1), dict(rb=0), dict(ns=0), dict(ks=2032), dict(vs=0), dict(k=None),
               dict(v=None), dict(sm=None), dict(kc=None), dict(vc=None), dict(vc=M + 1024),
               dict(kc=A), dict(vc=A + 4096 * 9)):
        assert _write(L, **kw) == 1, kw
    assert _write(L, rb=(1 << 20) + 16, ks=1 << 21, vs=1 << 21) == 2
    assert _write(L, ns=1 << 31) == 2 and _write(L, ks=1 << 31) == 2
    for kw in (dict(rb=2040), dict(ks=4104), dict(vs=4104), dict(k=A + 8), dict(v=A + 8),
               dict(kc=M + 8), dict(vc=2 * M + 8)):
        assert _write(L, **kw) == 3, kw


def _fork(L, **kw):
    n = iter(range(1, 20))
    a = dict(par=A, keep=A, bt=A, own=A, mp=4, np=8, bi=2, bo=3, ps=16, ring=next(n) * M, st=A,
             bto=next(n) * M, owno=next(n) * M, sh=next(n) * M, sto=next(n) * M, cs=next(n) * M,
             cd=next(n) * M, cl=next(n) * M, ws=next(n) * M, wsb=1 << 30)
    a.update(kw)
    return L.bdsa_cache_fork(*(a[k] for k in ("par", "keep", "bt", "own", "mp", "np", "bi", "bo",
                                              "ps", "ring", "st", "bto", "owno", "sh", "sto", "cs",
                                              "cd", "cl", "ws", "wsb")), None, None)


def test_fork_refusals(L):
    for kw in (dict(bi=-1), dict(bo=-1), dict(ps=0), dict(mp=0), dict(np=0), dict(ring=None),
               dict(st=None), dict(sto=None), dict(bt=None), dict(own=None), dict(par=None),
               dict(keep=None), dict(bto=None), dict(owno=None), dict(sh=None), dict(cs=None),
               dict(cd=None), dict(cl=None)):
        assert _fork(L, **kw) == 1, kw
    for kw in (dict(bi=16385), dict(bo=16385), dict(np=1 << 28), dict(bi=16384, mp=1 << 17)):
        assert _fork(L, **kw) == 2, kw
    assert _fork(L, ws=9 * M + 16) == 3
    need = L.bdsa_cache_fork_workspace_bytes(2, 3, 8)
    assert need > 0 and L.bdsa_cache_fork_workspace_bytes(-1, 3, 8) == 0
    assert _fork(L, ws=None) == 4 and _fork(L, wsb=need - 1) == 4
    for kw in (dict(bto=A), dict(owno=A), dict(sto=A), dict(ring=A), dict(cs=7 * M), dict(ws=A),
               dict(sh=3 * M + 8)):
        assert _fork(L, **kw) == 1, kw


def _list(*ptrs):
    return (ctypes.c_void_p * len(ptrs))(*ptrs)


def _copy(L, **kw):
    a = dict(c=_list(M, 2 * M), n=2, rb=2048, ps=16, np=8, s=A, d=A, l=A, e=5)
    a.update(kw)
    return L.bdsa_cache_copy(a["c"], a["n"], a["rb"], a["ps"], a["np"], a["s"], a["d"], a["l"],
                             a["e"], None, None)


def _compact(L, **kw):
    a = dict(c=_list(M, 2 * M), n=2, rb=2048, ps=16, np=8, bt=A, mp=4, sl=A, p=A, w=7, bs=3)
    a.update(kw)
    return L.bdsa_cache_compact(a["c"], a["n"], a["rb"], a["ps"], a["np"], a["bt"], a["mp"],
                                a["sl"], a["p"], a["w"], a["bs"], None, None)


def test_cache_list_refusals(L):
    assert _copy(L, e=0) == 0 and _copy(L, c=None, n=0) == 0
    assert _compact(L, bs=0) == 0 and _compact(L, w=0) == 0 and _compact(L, c=None, n=0) == 0
    for call in (_copy, _compact):
        for kw in (dict(n=-1), dict(rb=0), dict(ps=0), dict(np=0), dict(c=None),
                   dict(c=_list(M, None)), dict(c=_list(M, M)),
                   dict(c=_list(M, M + 2048 * 16 * 8 - 16)), dict(c=_list(2 * M, A))):
            assert call(L, **kw) == 1, (call, kw)
        many = _list(*[M * (i + 1) for i in range(1025)])
        assert call(L, c=many, n=1025) == 2 and call(L, rb=(1 << 20) + 16) == 2
        assert call(L, np=1 << 28) == 2
        assert call(L, rb=2040) == 3 and call(L, c=_list(M + 8, 2 * M)) == 3
    for kw in (dict(e=-1), dict(s=None), dict(d=None), dict(l=None)):
        assert _copy(L, **kw) == 1, kw
    for kw in (dict(bs=-1), dict(w=-1), dict(mp=0), dict(bt=None), dict(sl=None), dict(p=None)):
        assert _compact(L, **kw) == 1, kw


def test_binding_refuses_cpu_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: bdsa.chunk_attn_paged(x, x, x, i.view(2, 2), i, i, page_size=2, scale=1.0),
                 lambda: bdsa.cache_write(x, x, i, x, x),
                 lambda: bdsa.cache_fork(i, i, i.view(2, 2), i, i, i, page_size=2),
                 lambda: bdsa.cache_copy([x], i, i, i, page_size=2),
                 lambda: bdsa.cache_compact([x], i.view(2, 2), i, i.view(2, 2), page_size=2)):
        with pytest.raises(ValueError):
            call()
