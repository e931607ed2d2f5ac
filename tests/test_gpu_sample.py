"""GPU parity of bdsa_token_sample against the fp64 oracle.

Tolerance of a probability, relative: the weight's, the scale's and the
product's rounding (2^-24 each; the exponential's 2^-30 is within the 0.1), and
the fixed-point sum (V / 2 units of 2^-41 against a sum of at least 1/2).  Tokens and kept
sets are equal except on rows the oracle marks as within 1e-9 of a border."""
import numpy as np
import pytest
import torch

import block_diffusion_speculative_attn_gb300 as bdsa
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rtol(V):
    return 3.1 * 2.0 ** -24 + V * 2.0 ** -42 + 2.0 ** -37


def run(l, u=None, probs=True, status=None, **kw):
    to = lambda a, d: None if a is None else torch.as_tensor(np.asarray(a), dtype=d, device=DEV)
    types = dict(temperature=torch.float32, top_k=torch.int32, top_p=torch.float32,
                 min_p=torch.float32)
    kw = {k: to(v, types[k]) for k, v in kw.items()}
    t, p = bdsa.token_sample(l, to(u, torch.float32), want_probs=probs, dev_status=status, **kw)
    return (None if t is None else t.cpu().numpy(), None if p is None else p.cpu().numpy())


def check(l, u, got_t, got_p, **kw):
    kw = {k: None if v is None else np.asarray(v, np.int32 if k == "top_k" else np.float32)
          for k, v in kw.items()}
    t, p, near = oracle.token_sample(l.double().cpu().numpy(),
                                     None if u is None else np.asarray(u, np.float32), **kw)
    ok = ~near
    assert ok.any()
    if got_t is not None:
        assert (got_t[ok] == t[ok]).all()
    if got_p is not None:
        # the kept sets (a kept weight below fp32's range may come out as zero)
        assert not (got_p[ok][p[ok] == 0] > 0).any() and (got_p[ok][p[ok] > 1e-36] > 0).all()
        err = np.abs(got_p[ok] - p[ok])
        assert (err <= rtol(l.shape[-1]) * p[ok] + 1e-37).all(), \
            float((err / (p[ok] + 1e-37)).max())
    return near


FILTERS = {
    "none": dict(),
    "temperature": dict(temperature=True),
    "top_k": dict(top_k=True),
    "top_p": dict(top_p=True),
    "min_p": dict(min_p=True),
    "k_p": dict(temperature=True, top_k=True, top_p=True),
    "all": dict(temperature=True, top_k=True, top_p=True, min_p=True),
}


def params(rng, bs, V, which):
    make = dict(temperature=lambda: rng.uniform(0.3, 2.0, bs).astype(np.float32),
                top_k=lambda: rng.integers(1, max(2, min(V, 120)), bs).astype(np.int32),
                top_p=lambda: rng.uniform(0.2, 0.999, bs).astype(np.float32),
                min_p=lambda: rng.uniform(0.001, 0.3, bs).astype(np.float32))
    return {k: make[k]() for k in which}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [1, 2, 31, 33, 1000, 5003, 40001])
@pytest.mark.parametrize("which", list(FILTERS))
def test_matches_oracle(dtype, V, which):
    rng = np.random.default_rng(V * 7 + len(which))
    bs, B = 3, 4
    l = torch.from_numpy(rng.normal(size=(bs, B, V)).astype(np.float32) * 3).to(DEV).to(dtype)
    u = rng.random((bs, B), dtype=np.float32)
    kw = params(rng, bs, V, FILTERS[which])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    t, p = run(l, u, status=status, **kw)
    check(l, u, t, p, **kw)
    t2, _ = run(l, u, probs=False, **kw)     # the same tokens without the distribution
    assert (t2 == t).all()
    _, p2 = run(l, None, **kw)               # the same distribution without the tokens
    assert (p2 == p).all()
    assert status.item() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("std", [0.05, 1.0, 3.0, 30.0])
def test_vocabulary_rows(dtype, std):
    """Full-size rows, flat to peaked, every filter."""
    rng = np.random.default_rng(int(std * 100))
    bs, B, V = 7, 2, 151936
    l = torch.from_numpy(rng.normal(size=(bs, B, V)).astype(np.float32) * std).to(DEV).to(dtype)
    u = rng.random((bs, B), dtype=np.float32)
    for which in FILTERS:
        kw = params(rng, bs, V, FILTERS[which])
        t, p = run(l, u, **kw)
        check(l, u, t, p, **kw)


@pytest.mark.parametrize("V,dtype", [(1 << 21, torch.float32), (1 << 21, torch.bfloat16),
                                     (600011, torch.float32)])
def test_vocabularies_past_shared_memory(V, dtype):
    rng = np.random.default_rng(9)
    l = torch.from_numpy(rng.normal(size=(2, 1, V)).astype(np.float32) * 3).to(DEV).to(dtype)
    u = rng.random((2, 1), dtype=np.float32)
    for which in ("none", "all", "top_p"):
        kw = params(rng, 2, V, FILTERS[which])
        t, p = run(l, u, **kw)
        check(l, u, t, p, **kw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [7, 4096, 151936])
def test_ties_everywhere(dtype, V):
    """All logits equal: every cut falls inside one run of ties and takes the
    lowest indices; sums are exact."""
    l = torch.full((1, 1, V), 0.75, device=DEV, dtype=dtype)
    for k in (1, 3, V // 2, V):
        t, p = run(l, [[0.999999]], top_k=[k])
        n = k if 0 < k < V else V
        assert (p[0, 0] > 0).sum() == n and (p[0, 0, :n] > 0).all()
        assert t[0, 0] == min(n - 1, int(np.floor(np.float64(np.float32(0.999999)) * n)))
    t, p = run(l, [[0.0]], top_p=[0.5])
    n = -(-V // 2)
    assert (p[0, 0, :n] > 0).all() and not (p[0, 0, n:] > 0).any() and t[0, 0] == 0
    t, p = run(l, [[0.5]], min_p=[1.0])
    assert (p[0, 0] > 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [1031, 20011, 100003])
@pytest.mark.parametrize("kind", ["smooth", "steps", "one_leads", "two_levels", "masked"])
def test_flat_nucleus(dtype, V, kind):
    """top-p alone on rows whose nucleus is thousands of tokens: the cut in a thin
    place, inside a long run of ties, just behind a token that holds most of the
    weight, and between two values."""
    rng = np.random.default_rng(V + len(kind))
    bs, B = 6, 3
    l = rng.normal(size=(bs, B, V)).astype(np.float32)
    if kind == "steps":
        l = np.round(l * 2) / 2
    elif kind == "one_leads":
        l[..., V // 3] = np.log(V) + 2.0
    elif kind == "two_levels":
        l = np.where(rng.random((bs, B, V)) < 0.3, 1.0, 0.0).astype(np.float32)
    elif kind == "masked":
        l[rng.random((bs, B, V)) < 0.5] = -np.inf
        l[rng.random((bs, B, V)) < 0.1] = np.nan
    l = torch.from_numpy(l).to(DEV).to(dtype)
    u = rng.random((bs, B), dtype=np.float32)
    u[0] = 0.0
    u[1] = 1 - 2.0 ** -24
    for tp in ([0.95, 0.9, 0.5, 0.1, 0.99, 0.998], [0.9998, 0.99995, 1e-6, 0.3, 0.7, 0.97]):
        kw = dict(top_p=np.array(tp, np.float32),
                  temperature=rng.uniform(0.7, 2.0, bs).astype(np.float32))
        t, p = run(l, u, **kw)
        check(l, u, t, p, **kw)
        t2, _ = run(l, u, probs=False, **kw)
        assert (t2 == t).all()


def test_two_valued_rows_cut_inside_each_run():
    V = 3001
    base = torch.zeros(V, device=DEV)
    base[1::3] = np.log(2.0)
    l = base.view(1, 1, V).bfloat16()
    hi = np.flatnonzero(l[0, 0].float().cpu().numpy() > 0)
    lo = np.flatnonzero(l[0, 0].float().cpu().numpy() == 0)
    for k in (1, len(hi) - 1, len(hi), len(hi) + 1, V - 1):
        _, p = run(l, top_k=[k])
        want = np.sort(np.concatenate([hi, lo])[:k])
        assert (np.flatnonzero(p[0, 0]) == want).all()


@pytest.mark.parametrize("V", [40, 5003, 151936])
def test_masked_infinite_and_nan_logits(V):
    rng = np.random.default_rng(V)
    l = rng.normal(size=(6, 1, V)).astype(np.float32)
    l[0, 0, rng.random(V) < 0.7] = -np.inf
    l[1, 0, rng.random(V) < 0.5] = np.nan
    l[2, 0, :] = -np.inf                       # nothing left
    l[3, 0, [V // 3, V // 2]] = np.inf
    l[4, 0, :] = np.finfo(np.float32).min      # the type's lowest value everywhere
    l[5, 0, :] = np.finfo(np.float32).min
    l[5, 0, V - 2] = 1.0
    u = rng.random((6, 1), dtype=np.float32)
    for which in ("none", "all", "top_p", "top_k"):
        kw = params(rng, 6, V, FILTERS[which])
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        lt = torch.from_numpy(l).to(DEV)
        t, p = run(lt, u, status=status, **kw)
        check(lt, u, t, p, **kw)
        assert t[2, 0] == -1 and not p[2].any() and status.item() == 16


def test_signed_zeros_are_equal():
    l = torch.tensor([[[-0.0, 0.0, -0.0, -1.0]]], device=DEV)
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        _, p = run(l.to(dt), top_k=[2])
        assert (np.flatnonzero(p[0, 0]) == [0, 1]).all()


def test_greedy_and_extreme_parameters():
    rng = np.random.default_rng(1)
    V = 5003
    l = torch.from_numpy(np.round(rng.normal(size=(9, 2, V)) * 2).astype(np.float32)).to(DEV)
    u = rng.random((9, 2), dtype=np.float32)
    T = np.array([0.0, 1e-30, 1e-38, 1e30, 3e38, -1.0, np.nan, np.inf, 0.0], np.float32)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    t, p = run(l, u, status=status, temperature=T)
    check(l, u, t, p, temperature=T)
    first = l.cpu().numpy().argmax(-1)
    assert (t[[0, 8]] == first[[0, 8]]).all() and (t[5:8] == -1).all() and status.item() == 16
    kw = dict(top_k=np.array([-3, 0, 1, V - 1, V, V + 5, 2 ** 31 - 1, 2, 2], np.int32),
              top_p=np.array([-1, 0, 1, 2, np.nan, 1e-40, 1 - 2 ** -24, 0.5, 1], np.float32),
              min_p=np.array([-1, 0, 1, 2, np.nan, 1e-30, 0.999, 1e-4, 0], np.float32))
    for name, v in kw.items():
        t, p = run(l, u, **{name: v})
        v2 = np.where(np.isnan(v), 1.0 if name == "top_p" else 0.0, v) if name != "top_k" else v
        check(l, u, t, p, **{name: v2})
    t, _ = run(l, np.full((9, 2), np.nan))
    t0, _ = run(l, np.zeros((9, 2)))
    assert (t == t0).all()
    t, _ = run(l, np.full((9, 2), 7.0))
    assert (t == V - 1).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_strided_and_odd_rows(dtype):
    """Rows that start on any element, of a larger buffer; probs into a strided
    buffer whose other elements stay as they were."""
    rng = np.random.default_rng(2)
    bs, B, V = 3, 5, 4099
    for off in (0, 1, 3, 7):
        big = torch.from_numpy(rng.normal(size=(bs, B, V + 9)).astype(np.float32) * 3)
        big = big.to(DEV).to(dtype)
        l = big[:, :, off:off + V]
        pbuf = torch.full((B, bs, V + 4), -5.0, device=DEV)
        pv = pbuf.transpose(0, 1)[:, :, 1:1 + V]
        u = rng.random((bs, B), dtype=np.float32)
        kp = rng.uniform(0.3, 0.95, bs).astype(np.float32)
        t, p = bdsa.token_sample(l, torch.from_numpy(u).to(DEV), probs=pv,
                                 top_p=torch.from_numpy(kp).to(DEV))
        check(l, u, t.cpu().numpy(), p.cpu().numpy(), top_p=kp)
        assert (pbuf[:, :, 0] == -5).all() and (pbuf[:, :, V + 1:] == -5).all()


def test_broadcast_logits():
    """Stride-0 rows: one row of logits drawn from many times."""
    rng = np.random.default_rng(4)
    row = torch.from_numpy(rng.normal(size=(1, 1, 3000)).astype(np.float32)).to(DEV)
    l = row.expand(4, 50, 3000)
    u = rng.random((4, 50), dtype=np.float32)
    t, _ = run(l, u, probs=False)
    check(l, u, t, None)


def test_draws_follow_the_distribution():
    rng = np.random.default_rng(6)
    V, n = 50, 200000
    row = torch.from_numpy(rng.normal(size=(1, 1, V)).astype(np.float32)).to(DEV)
    t, _ = run(row.expand(1, n, V), rng.random((1, n), dtype=np.float32), probs=False,
               top_k=[20], temperature=[1.3])
    _, p, _ = oracle.token_sample(row.double().cpu().numpy(), None, np.array([1.3], np.float32),
                                  np.array([20]))
    got = np.bincount(t[0], minlength=V)
    want = p[0, 0] * n
    assert (got[want == 0] == 0).all()
    k = want > 0
    chi2 = ((got[k] - want[k]) ** 2 / want[k]).sum()
    assert chi2 < 19 + 6 * np.sqrt(2 * 19)


def test_graph_replay_and_streams():
    rng = np.random.default_rng(8)
    bs, B, V = 5, 3, 20001
    mk = lambda: torch.from_numpy(rng.normal(size=(bs, B, V)).astype(np.float32) * 3).to(DEV)
    l, u = mk(), torch.rand(bs, B, device=DEV)
    tp = torch.full((bs,), 0.9, device=DEV)
    probs = torch.empty(bs, B, V, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        t0, _ = bdsa.token_sample(l, u, top_p=tp, probs=probs)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t1, _ = bdsa.token_sample(l, u, top_p=tp, probs=probs)
    for _ in range(2):
        l.copy_(mk())
        u.uniform_()
        g.replay()
        torch.cuda.synchronize()
        check(l, u.cpu().numpy(), t1.cpu().numpy(), probs.cpu().numpy(),
              top_p=np.full(bs, 0.9, np.float32))


def test_refusals():
    l = torch.zeros(2, 3, 8, device=DEV)
    u = torch.zeros(2, 3, device=DEV)
    with pytest.raises(ValueError):
        bdsa.token_sample(l)                                  # nothing wanted
    with pytest.raises(TypeError):
        bdsa.token_sample(l.double(), u)
    with pytest.raises(ValueError):
        bdsa.token_sample(l.transpose(1, 2), torch.zeros(2, 8, device=DEV))
    with pytest.raises(ValueError):
        bdsa.token_sample(l, u[:, :2].contiguous())
    with pytest.raises(ValueError):
        bdsa.token_sample(l, u, temperature=torch.ones(3, device=DEV))
    with pytest.raises(TypeError):
        bdsa.token_sample(l, u, top_k=torch.ones(2, device=DEV))
    with pytest.raises(bdsa.BdsaError):
        bdsa.token_sample(l, probs=torch.zeros(1, 1, 8, device=DEV).expand(2, 3, 8))
    t, p = bdsa.token_sample(l[:0], u[:0], want_probs=True)
    assert t.shape == (0, 3) and p.shape == (0, 3, 8)
