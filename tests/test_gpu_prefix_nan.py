"""A NaN among a row's keys, values or its query reaches the row's output in the
shared-prefix call: keys and values of the prefix, of the request, of the block, in
calls whose units are cut and whole."""
import numpy as np
import pytest
import torch

import block_diffusion_speculative_attn_gb300 as bdsa  # noqa: F401
from block_diffusion_speculative_attn_gb300 import workloads as wl
from gpu_helpers import ATTN_MAX_ABS
from test_gpu_attn_prefix import Case

pytestmark = pytest.mark.gpu
NAN = float("nan")


def slot(c, r, t):
    return int(c.table[r, t // c.ps]) * c.ps + t % c.ps


def expect(c, reqs, head, base, mode, sms, first=0, cols=slice(None)):
    """Rows [first, B) of the KV head's query heads in reqs are NaN in cols; every
    other output is the one without the NaN."""
    G = c.Hq // c.Hkv
    nan = np.zeros((c.bs, c.B, c.Hq, c.D), bool)
    for r in reqs:
        nan[r, first:, head * G:(head + 1) * G, cols] = True
    out, lse, st = c.run(mode, sms=sms)
    o = out.float().cpu().numpy().reshape(nan.shape)
    assert st == 0
    assert (np.isnan(o) == nan).all(), (sms, int(np.isnan(o).sum()), int(nan.sum()))
    assert np.abs((o - base.reshape(nan.shape))[~nan]).max() <= ATTN_MAX_ABS
    rows = nan.any(-1)
    if cols == slice(None):                      # the scores: the row has no sum
        assert (np.isnan(lse.cpu().numpy().reshape(rows.shape)) == rows).all()


def make(D=128, B=8):
    # requests 1 and 3 have one visible own key in VERIFY's first row
    return Case([3, 2], [1408, 640], [700, 0, 33, 0, 300], B, 8, 2, D, 64, seed=21)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sms", [1, 5, 0])
def test_a_shared_key(D, sms):
    for t in (0, 200, 1407):
        c = make(D)
        base = c.want(wl.VERIFY)[0]
        c.k[slot(c, 0, t), 1, 5] = NAN
        expect(c, [0, 1, 2], 1, base, wl.VERIFY, sms)


@pytest.mark.parametrize("B", [8, 32])
@pytest.mark.parametrize("sms", [1, 5, 0])
@pytest.mark.parametrize("mode", [wl.DRAFT, wl.VERIFY])
def test_an_own_key(mode, sms, B):
    base = make(B=B).want(mode)[0]
    for r, t in ((0, 1408), (0, 1700), (0, 2107), (2, 1408 + 32), (4, 700)):
        c = make(B=B)
        c.k[slot(c, r, t), 0, 127] = NAN
        expect(c, [r], 0, base, mode, sms)
    # a block's key: in VERIFY the rows from its own on
    for r, i in ((0, 3), (1, 0), (3, 0), (3, 7), (4, 7)):
        c = make(B=B)
        c.k[slot(c, r, int(c.seq[r]) + i), 1, 0] = NAN
        expect(c, [r], 1, base, mode, sms, first=i if mode == wl.VERIFY else 0)


@pytest.mark.parametrize("sms", [1, 0])
def test_values(sms):
    """A NaN value: its column alone."""
    base = make().want(wl.DRAFT)[0]
    c = make()
    c.v[slot(c, 3, 130), 1, 77] = NAN
    expect(c, [3, 4], 1, base, wl.DRAFT, sms, cols=slice(77, 78))
    c = make()
    c.v[slot(c, 0, 1900), 1, 3] = NAN
    expect(c, [0], 1, base, wl.DRAFT, sms, cols=slice(3, 4))


@pytest.mark.parametrize("sms", [1, 0])
def test_a_query(sms):
    c = make()
    base = c.want(wl.VERIFY)[0]
    c.q.view(c.bs, c.B, c.Hq, c.D)[2, :, 4:, 9] = NAN
    expect(c, [2], 1, base, wl.VERIFY, sms)


def test_infinite_keys():
    """A score of +inf has no softmax, as in the plain call; one of -inf no weight."""
    for where in (300, 1900):
        c = make()
        q = c.q.view(c.bs, c.B, c.Hq, c.D)
        q[..., 0] = q[..., 0].abs() + 1
        base = c.want(wl.VERIFY)[0]
        c.k[slot(c, 0, where), 0, 0] = float("inf")
        expect(c, [0, 1, 2] if where < 1408 else [0], 0, base, wl.VERIFY, 0)
        c.k[slot(c, 0, where), 0, 0] = -float("inf")
        ref, _ = c.want(wl.VERIFY)
        out, _, st = c.run(wl.VERIFY)
        assert st == 0
        assert np.abs(out.float().cpu().numpy().reshape(ref.shape) - ref).max() <= ATTN_MAX_ABS


def test_repeats_itself():
    """The same inputs, the same bits, whatever the workspace held."""
    c = make()
    d = c.dev()
    ws = torch.empty(bdsa.block_attn_prefix_workspace_bytes(c.bs, c.B, c.Hq, c.Hkv, c.D, 4096, 2),
                     dtype=torch.uint8, device="cuda")
    first = None
    for fill in (0, 0xff, 0x5a, 0x7f):
        ws.fill_(fill)
        out, lse, st = c.run(wl.VERIFY, d, workspace=ws)
        got = (out.view(torch.int16).clone(), lse.view(torch.int32).clone())
        first = first or got
        assert st == 0 and torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
