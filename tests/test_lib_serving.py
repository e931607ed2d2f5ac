"""Host-side refusals of the serving operators (CPU: every call here fails its
checks, or has nothing to do, before it reaches a CUDA API)."""
import ctypes

import pytest
import torch

import block_diffusion_speculative_attn_gb300 as bdsa

A = 0x100000  # never dereferenced


@pytest.fixture(scope="module")
def L():
    from block_diffusion_speculative_attn_gb300 import build
    build.build()
    return bdsa.lib()


def _table(L, **kw):
    a = dict(seq=A, new=A + 0x1000, own=A + 0x2000, shared=None, bt=A, mp=4, np=8, bs=2, ps=16,
             ring=A, state=A, own_out=A + 0x3000, state_out=A + 0x4000, cu=A, slot=A, pos=A,
             mt=10)
    a.update(kw)
    return L.bdsa_block_table_update(a["seq"], a["new"], a["own"], a["shared"], a["bt"], a["mp"],
                                     a["np"], a["bs"], a["ps"], a["ring"], a["state"],
                                     a["own_out"], a["state_out"], a["cu"], a["slot"], a["pos"],
                                     a["mt"], None, None)


def test_table_refusals(L):
    assert _table(L, bs=-1) == 1
    assert _table(L, ps=0) == 1
    assert _table(L, mp=0) == 1
    assert _table(L, np=0) == 1
    assert _table(L, mt=-1) == 1
    for name in ("seq", "new", "own", "bt", "ring", "state", "own_out", "state_out", "cu"):
        assert _table(L, **{name: None}) == 1, name
    assert _table(L, own_out=A + 0x2000) == 1        # in place: read while written
    assert _table(L, own_out=A + 0x2004) == 1        # overlapping
    assert _table(L, state_out=A + 4) == 1
    assert _table(L, bs=16385) == 2
    assert _table(L, np=1 << 28, ps=16) == 2         # slots past int32
    assert _table(L, mt=1 << 31) == 2
    assert _table(L, slot=A + 2) == 3


def _sample(L, **kw):
    a = dict(l=A, dt=0, lsr=8000, lsi=1000, u=A, T=A, k=A, p=A, m=A, bs=4, B=8, V=1000, tok=A,
             pr=A, psr=8000, psi=1000, sms=152)
    a.update(kw)
    return L.bdsa_token_sample(a["l"], a["dt"], a["lsr"], a["lsi"], a["u"], a["T"], a["k"],
                               a["p"], a["m"], a["bs"], a["B"], a["V"], a["tok"], a["pr"],
                               a["psr"], a["psi"], a["sms"], None, None)


def test_sample_refusals(L):
    assert _sample(L, bs=0) == 0
    assert _sample(L, bs=-1) == 1
    assert _sample(L, B=0) == 1
    assert _sample(L, V=0) == 1
    assert _sample(L, dt=3) == 1
    assert _sample(L, dt=-1) == 1
    assert _sample(L, lsi=-1) == 1
    assert _sample(L, l=None) == 1
    assert _sample(L, u=None) == 1                   # tokens need uniforms
    assert _sample(L, tok=None, pr=None) == 1
    assert _sample(L, psi=999) == 1                  # rows of probs overlap
    assert _sample(L, psr=7999) == 1
    assert _sample(L, psr=1000, psi=1000) == 1
    assert _sample(L, psr=0) == 1
    assert _sample(L, V=(1 << 21) + 1, psi=1 << 22, psr=1 << 26) == 2
    assert _sample(L, bs=1 << 24, psr=0, bt=0) in (1, 2)
    assert _sample(L, l=A + 2) == 3
    assert _sample(L, l=A + 1, dt=1) == 3
    assert _sample(L, pr=A + 2) == 3


def _prefix(L, **kw):
    a = dict(q=A, k=A, v=A, bt=A, mp=40, np=80, sl=A, go=A, pl=A, ng=2, mc=100, bs=2, B=8, Hq=8,
             Hkv=2, D=128, ps=16, scale=0.1, mode=1, out=A, lse=None, ws=None, wsb=0, sms=152)
    a.update(kw)
    return L.bdsa_block_attn_paged_prefix(a["q"], a["k"], a["v"], a["bt"], a["mp"], a["np"],
                                          a["sl"], a["go"], a["pl"], a["ng"], a["mc"], a["bs"],
                                          a["B"], a["Hq"], a["Hkv"], a["D"], a["ps"], a["scale"],
                                          a["mode"], a["out"], a["lse"], a["ws"], a["wsb"],
                                          a["sms"], None, None)


def test_prefix_refusals(L):
    assert _prefix(L, bs=0) == 0
    assert _prefix(L, go=None) == 1
    assert _prefix(L, pl=None) == 1
    assert _prefix(L, ng=0) == 1
    assert _prefix(L, ng=3) == 1                     # more groups than requests
    assert _prefix(L, mode=2) == 1                   # no trees
    assert _prefix(L, q=None) == 1
    assert _prefix(L, scale=0.0) == 1
    assert _prefix(L, D=96) == 2
    assert _prefix(L, Hq=64, Hkv=2) == 2             # G * B > 128
    assert _prefix(L, ps=24) == 2
    assert _prefix(L, out=A + 2) == 3


def test_outputs_apart_from_inputs_and_one_another(L):
    M = 1 << 24
    ins = dict(zip(("seq", "new", "own", "shared", "state"), range(M, 6 * M, M)))
    outs = dict(zip(("bt", "ring", "own_out", "state_out", "cu", "slot", "pos"),
                    range(6 * M, 13 * M, M)))
    for o in outs:
        for i in list(ins) + [x for x in outs if x != o]:
            a = {**ins, **outs, "bs": 32, "np": 64, "mt": 64}
            a[o] = a[i] + 4
            assert _table(L, **a) == 1, (o, i)
    ins = dict(zip(("l", "u", "T", "k", "p", "m"), range(M, 7 * M, M)))
    outs = dict(tok=7 * M, pr=8 * M)
    for o in outs:
        for i in list(ins) + [x for x in outs if x != o]:
            a = {**ins, **outs}
            a[o] = a[i] + 4
            assert _sample(L, **a) == 1, (o, i)
    a = {**ins, **outs, "l": 8 * M - 4 * 32000 + 16}  # the last logit row meets probs
    assert _sample(L, **a) == 1
    assert _sample(L, **{**a, "l": 8 * M + 4 * 32000 - 16}) == 1
    M = 1 << 32
    ins = dict(zip(("q", "k", "v", "bt", "sl", "go", "pl"), range(M, 8 * M, M)))
    outs = dict(out=8 * M, lse=9 * M, ws=10 * M, wsb=1 << 30)
    for o in ("out", "lse", "ws"):
        for i in list(ins) + [x for x in ("out", "lse", "ws") if x != o]:
            a = {**ins, **outs}
            a[o] = a[i]
            assert _prefix(L, **a) == 1, (o, i)


def test_prefix_workspace(L):
    f = L.bdsa_block_attn_prefix_workspace_bytes
    al = lambda x: (x + 255) // 256 * 256
    bs, B, Hq, Hkv, D, ng, sms = 32, 16, 32, 8, 128, 3, 152
    rows, slots = bs * B * Hq, 256 * sms
    want = L.bdsa_block_attn_workspace_bytes(bs, B, Hq, Hkv, D, 4096, sms)
    want += al(4) + 2 * al(4 * rows) + al(4 * slots) + al(4 * rows * D) + \
        al(4 * slots * D)
    assert f(bs, B, Hq, Hkv, D, 4096, ng, sms) == want
    assert f(bs, B, Hq, Hkv, D, 4096, 0, sms) == 0


def test_python_checks_need_no_gpu():
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        bdsa.block_table_update(i, i, i, i.view(2, 2), i, i[:2], page_size=4, total_tokens=4)
    with pytest.raises(ValueError):
        bdsa.token_sample(torch.zeros(1, 1, 8), torch.zeros(1, 1))
