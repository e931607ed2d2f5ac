"""bdsa_chunk_attn_paged against the fp64 oracle with the fp32 part of the error bound
taken from each case's inputs; offsets past 2^31; how far a NaN in a value reaches.

Bound.  S is the largest sum_d |q_d k_d| * scale of a case, n its longest row of keys.
A score is D products, exact in fp32, and D sums, each off by at most a step (2^-23)
of a partial sum below S; the scale, the product with it and the subtraction of the
maximum round it (each at most 2^-24 of a value below 2 S, twice for the maximum): in
all at most e = S (D 2^-23 + 8 * 2^-24).  A weight is off by that, by its exponential
and by those that rescale it (2^-22 each, at most one a key tile); the sums of the
weights and of their products with the values by n steps, n * 2^-23; the logarithm, its
product with ln 2 and the joins by 2^-20 + 2^-22 |lse|.  So
  |lse| error <= E = e + n 2^-23 + (n / 128 + 2) 2^-22 + 2^-20 + 2^-22 |lse|
and out, whose weights are off by E above and below the line, by 2 E weight beside the
two roundings to bf16 (the weights, and out: 2^-8 each, as in test_gpu_chunk_attn)."""
import numpy as np
import pytest
import torch

import block_diffusion_speculative_attn_gb300 as bdsa
from test_gpu_chunk_attn import DEV, SHAPES, Case

pytestmark = pytest.mark.gpu


def check(c, **kw):
    out, lse = c.run(**kw)
    ref, ref_lse, weight = c.want()
    q, k = c.q.double().abs().numpy(), c.k.double().abs().numpy()
    S = 0.0
    for r in range(c.bs):
        t = np.arange(c.ctx[r] + c.new[r])
        kk = k[c.table[r, t // c.ps].astype(np.int64) * c.ps + t % c.ps]
        for h in range(c.Hkv):
            G = c.Hq // c.Hkv
            rows = q[c.cu[r]:c.cu[r + 1], h * G:(h + 1) * G].reshape(-1, c.D)
            S = max(S, (rows @ kk[:, h].T).max(initial=0.0) * c.scale)
    n = int((c.ctx + c.new).max())
    fixed = S * (c.D * 2.0 ** -23 + 8 * 2.0 ** -24) + n * 2.0 ** -23 + \
        (n / 128 + 2) * 2.0 ** -22 + 2.0 ** -20
    E = fixed + 2.0 ** -22 * np.abs(ref_lse)
    assert (np.abs(lse - ref_lse) <= E).all(), (np.abs(lse - ref_lse).max(), E.min())
    tol = 2.0 ** -8 * (np.abs(ref) + weight) * (1 + 2.0 ** -8) + \
        2 * E[:, :, None] * (1 + E[:, :, None]) * weight
    assert (np.abs(out - ref) <= tol).all(), (np.abs(out - ref) - tol).max()
    assert int(c.status) == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("spread", [1e-3, 1.0, 5.0, 30.0])
@pytest.mark.parametrize("mb", [1, 32])
def test_bound_of_the_inputs(spread, mb, D):
    check(Case([200, 3, 64], [300, 900, 0], Hq=8, Hkv=2, D=D, mb=mb, spread=spread, seed=31))


@pytest.mark.parametrize("shape", [i for i, (new, _) in enumerate(SHAPES) if sum(new)])
@pytest.mark.parametrize("sms", [0, 3])
def test_bound_of_the_shapes(shape, sms):
    check(Case(*SHAPES[shape], Hq=8, Hkv=2, D=128, ps=16, seed=32 + shape), sms=sms)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("heads,npt", [((4, 2), 64), ((16, 2), 16), ((2, 2), 128)])
def test_how_far_a_value_reaches(heads, npt, bad):
    """A value of token 300's of request 0, KV head 1: its log-sum-exps, the other
    heads and the other request do not see it; nor do tokens whose row tile (npt tokens)
    ends before key 256, where its 128-key tile starts.  Those from 300 on do."""
    c = Case([400, 9], [0, 500], *heads, D=64, ps=16, seed=33)
    clean, clean_lse = c.run()
    c.v[int(c.table[0, 300 // 16]) * 16 + 300 % 16, 1] = bad
    out, lse = c.run()
    assert (lse == clean_lse).all() and int(c.status) == 0
    G = heads[0] // heads[1]
    assert (out[:, :G] == clean[:, :G]).all()
    assert (out[400:] == clean[400:]).all()
    before = 256 // npt * npt
    assert (out[:before] == clean[:before]).all()
    assert not np.isfinite(out[300:400, G:]).any()


def test_caches_past_2_31_bytes():
    """Pages whose byte offsets need more than 32 bits (2.5 GB a cache)."""
    Hkv, D, ps, pages = 8, 128, 16, 76000
    small = Case([40, 1], [90, 700], Hq=16, Hkv=Hkv, D=D, ps=ps, seed=34)
    used = small.k.shape[0] // ps
    at = np.random.default_rng(34).permutation(pages - 66001)[:used] + 66000
    at[:2] = 0, pages - 1
    big = []
    for x in (small.k, small.v):
        t = torch.zeros((pages * ps, Hkv, D), dtype=torch.bfloat16, device=DEV)
        t.view(pages, ps, Hkv, D)[torch.from_numpy(at).to(DEV)] = x.to(DEV).view(used, ps, Hkv, D)
        big.append(t)
    assert pages * ps * Hkv * D * 2 > 2 ** 31
    d = small.dev()
    d["k"], d["v"] = big
    d["table"] = torch.from_numpy(np.where(small.table >= 0, at[small.table], -1)
                                  .astype(np.int32)).to(DEV)
    a, b = small.run(d), small.run()
    assert (a[0] == b[0]).all() and (a[1] == b[1]).all()
    small.check(b)


def test_outputs_past_2_31_elements():
    """600000 requests of one token and one key: out is that key's value."""
    n, Hq, Hkv, D, ps, pages = 600_000, 32, 8, 128, 8, 1000
    g = torch.Generator(device=DEV).manual_seed(35)
    q = torch.randn((n, Hq, D), generator=g, device=DEV, dtype=torch.bfloat16)
    k = torch.randn((pages * ps, Hkv, D), generator=g, device=DEV, dtype=torch.bfloat16)
    v = torch.randn((pages * ps, Hkv, D), generator=g, device=DEV, dtype=torch.bfloat16)
    table = torch.randint(pages, (n, 1), generator=g, device=DEV, dtype=torch.int32)
    cu = torch.arange(n + 1, device=DEV, dtype=torch.int32)
    st = torch.zeros(1, device=DEV, dtype=torch.int32)
    assert q.numel() > 2 ** 31
    out = bdsa.chunk_attn_paged(q, k, v, table, torch.zeros_like(cu[:n]), cu, page_size=ps,
                                scale=0.1, dev_status=st)
    # (one weight of 1: its rounding to bf16 and out's, half a step each)
    for r in range(0, n, 50000):
        rows = slice(r, r + 50000)
        want = v[table[rows, 0].long() * ps].repeat_interleave(Hq // Hkv, 1)
        diff = (out[rows].float() - want.float()).abs()
        assert bool((diff <= 2.0 ** -7 * want.float().abs()).all())
    assert int(st) == 0


def test_copy_and_compact_past_2_31_bytes():
    ps, pages, row = 16, 80000, (8, 128)
    cache = torch.zeros((pages * ps, *row), dtype=torch.bfloat16, device=DEV)
    assert cache.numel() * 2 > 2 ** 31
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    g = torch.Generator().manual_seed(36)
    x = torch.randn((ps, *row), generator=g).to(torch.bfloat16).to(DEV)
    p = cache.view(pages, ps, *row)
    p[1], p[pages - 2] = x, -x
    bdsa.cache_copy([cache], i32([1, pages - 2]), i32([pages - 1, 2]), i32([ps, 5]), page_size=ps)
    assert torch.equal(p[pages - 1], x) and torch.equal(p[2, :5], -x[:5])
    assert not p[2, 5:].any() and int((p != 0).flatten(1).any(1).sum()) == 4
    # rows 3, 17, 31 of a region that starts at position 5
    table = i32([[pages - 1, 0, pages - 2]])
    before = p[pages - 2].clone()
    bdsa.cache_compact([cache], table, i32([5]), i32([[3, 17, 31, -1]]), page_size=ps)
    assert torch.equal(p[pages - 1, 5], x[8]) and not p[pages - 1, 6].any()
    assert torch.equal(p[pages - 1, 7], before[4]) and torch.equal(p[pages - 1, 8:], x[8:])
    assert torch.equal(p[pages - 1, :5], x[:5]) and torch.equal(p[pages - 2], before)
