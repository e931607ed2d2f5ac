"""Draws of bdsa_token_sample without filters from rows that one logit leads by 20
to 40 nats, where most weights are below the unit the sums are kept in.

A token drawn has at least half a unit of weight (the row's scale is 2^E, the
power of two above its largest weight, a unit 2^-41 of it).  The draw's target is
met to within what the sums are exact to: half a unit a logit, and 2^-30 of the
total for the weights' own rounding.  Where the target falls between two tokens
that have half a unit, into the share of those that have less, either neighbour is
right."""
import numpy as np
import pytest
import torch

import block_diffusion_speculative_attn_gb300 as bdsa

pytestmark = pytest.mark.gpu
DEV = "cuda"
US = [0.0, -3.0, 2.0 ** -24, 2.0 ** -22, 0.5, 1 - 2.0 ** -24, 1.0, float("nan")]


def allowed(l, T, u):
    """Whether token t may be drawn with uniform u, [V] bool, for one row in fp64."""
    y = l * np.log2(np.e) / T
    E = np.floor(y.max()) + 1
    units = np.exp2(y - E + 41)
    edge = 1e-4                       # of the weight: rows round y by far less
    sure, maybe = units > 0.5 * (1 + edge), units > 0.5 * (1 - edge)
    c = np.cumsum(units)
    total = c[-1]
    u = 0.0 if not u > 0 else min(u, 1.0)
    goal = u * total
    tol = 0.5 * len(l) + 1 + 2.0 ** -30 * total
    lo, hi = c - units, c
    hit = maybe & (lo - tol <= goal) & (goal <= hi + tol)
    if (sure & (lo + tol < goal) & (goal < hi - tol)).any():
        return hit
    at = np.flatnonzero(maybe)
    before, after = at[hi[at] <= goal], at[lo[at] >= goal]
    hit[before[-1:]] = True
    hit[after[:1]] = True
    return hit


def check(l, T=None, us=US, probs=False, seed=0):
    """Every u on the row l (fp32, bf16 or fp16 [V])."""
    n, V = len(us), l.shape[0]
    rows = l.to(DEV).expand(1, n, V)
    u = torch.tensor(us, dtype=torch.float32, device=DEV).view(1, n)
    tokens = torch.full((1, n), -7, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    t = None if T is None else torch.tensor([T], dtype=torch.float32, device=DEV)
    bdsa.token_sample(rows, u, temperature=t, tokens=tokens, want_probs=probs,
                      dev_status=status)
    got = tokens[0].cpu().numpy()
    row = l.double().numpy()
    T = 1.0 if T is None else float(np.float32(T))
    assert status.item() == 0
    for k in range(n):
        assert 0 <= got[k] < V, (us[k], got[k])
        ok = allowed(row, T, float(np.float32(us[k])))
        assert ok[got[k]], (us[k], got[k], np.flatnonzero(ok)[:4])
    return got


@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("V", [5003, 151936, 1 << 21])
@pytest.mark.parametrize("where", ["first", "middle", "last", "last but one"])
def test_one_logit_leads(V, where, probs):
    x = {"first": 0, "middle": V // 2, "last": V - 1, "last but one": V - 2}[where]
    for gap in (20, 26, 28, 28.6, 29, 29.5, 30, 31, 32, 33, 34, 36, 40, 90):
        l = torch.zeros(V)
        l[x] = gap
        got = check(l, probs=probs)
        if gap >= 29:                 # the rest has less than half a unit each
            assert (got == x).all(), gap


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [0.05, 0.7, 3.0])
def test_leaders_over_noise(dtype, T):
    """One to three leaders, their gaps in l / T, and noise below them."""
    rng = np.random.default_rng(int(T * 100))
    for V in (4096, 40001, 151936):
        for gap in (27.0, 30.0, 33.0):
            for leaders in (1, 2, 3):
                l = torch.from_numpy(rng.normal(size=V).astype(np.float32) * T * 0.7)
                l[torch.from_numpy(rng.choice(V, leaders, replace=False))] = gap * T
                us = US + rng.random(4).astype(np.float32).tolist()
                check(l.to(dtype), T, us)


def test_masked_in_front():
    """The first logits masked: the first pass's scale is not the row's."""
    V = 151936
    for front in (-float("inf"), -1e4):
        for gap in (28.0, 30.0, 34.0):
            l = torch.zeros(V)
            l[:70000] = front
            l[140000] = gap
            check(l)
            check(l, probs=True)
