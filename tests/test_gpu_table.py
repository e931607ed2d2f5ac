"""GPU parity of bdsa_block_table_update against the oracle (integers, equal)."""
import numpy as np
import pytest
import torch

import block_diffusion_speculative_attn_gb300 as bdsa
import oracle
from block_diffusion_speculative_attn_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)


def pool_state(rng, bs, ps, max_pages, have_hi, spare):
    """Requests with scattered pages, the rest of the pool in the ring."""
    lens = rng.integers(0, have_hi + 1, bs)
    owned = np.minimum((lens + ps - 1) // ps + rng.integers(0, 2, bs), max_pages)
    pool = int(owned.sum()) + spare
    perm = rng.permutation(pool)
    table = np.full((bs, max_pages), -1)
    cols = np.arange(max_pages)
    table[cols[None] < owned[:, None]] = perm[:int(owned.sum())]
    head = int(rng.integers(0, pool))
    ring = np.full(pool, -1)
    ring[(head + np.arange(spare)) % pool] = perm[int(owned.sum()):]
    return lens, owned, table, ring, np.array([head, spare])


def both(seq, new, owned, table, ring, state, ps, cap, shared=None):
    want = oracle.block_table_update(seq, new, owned, table, ring, state, ps, cap, shared)
    t, f = dev(table), dev(ring)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = dict(owned=dev(np.zeros(len(seq))), free_state=dev(np.zeros(2)),
               cu_tokens=dev(np.zeros(len(seq) + 1)), slot_map=dev(np.full(cap, -7)),
               positions=dev(np.full(cap, -7)))
    o = bdsa.block_table_update(dev(seq), dev(new), dev(owned), t, f, dev(state), page_size=ps,
                                total_tokens=cap, shared=None if shared is None else dev(shared),
                                out=out, dev_status=st)
    got = dict(o, block_table=t, free_pages=f)
    for k, v in got.items():
        assert (v.cpu().numpy() == want[k]).all(), k
    assert (st.item() == 16) == (want["n_bad"] > 0)
    return want


@pytest.mark.parametrize("ps", [1, 3, 8, 16, 64])
@pytest.mark.parametrize("bs", [1, 2, 33, 600, 1537])
@pytest.mark.parametrize("what", ["decode", "step", "chunk", "none"])
def test_grow(ps, bs, what):
    rng = np.random.default_rng(ps * 1000 + bs)
    max_pages = 300 // ps + 40
    lens, owned, table, ring, state = pool_state(rng, bs, ps, max_pages, 200, 60 * bs + 5)
    new = {"decode": np.ones(bs, int), "step": np.full(bs, 17), "chunk": rng.integers(0, 60, bs),
           "none": np.zeros(bs, int)}[what]
    lens = np.minimum(lens, owned * ps)
    both(lens, new, owned, table, ring, state, ps, int(new.sum()))


@pytest.mark.parametrize("bs", [5, 700])
def test_release_grow_and_shared_together(bs):
    rng = np.random.default_rng(bs)
    ps, max_pages = 4, 64
    lens, owned, table, ring, state = pool_state(rng, bs, ps, max_pages, 200, 20 * bs)
    done = rng.random(bs) < 0.4
    lens = np.where(done, 0, lens)
    new = np.where(done, 0, rng.integers(0, 30, bs))
    shared = np.where(rng.random(bs) < 0.5, rng.integers(0, 6, bs), 0)
    w = both(lens, new, owned, table, ring, state, ps, int(new.sum()) + 13, shared)
    assert w["n_bad"] == 0 and w["free_state"][1] != state[1]


def test_shortage_and_short_maps():
    rng = np.random.default_rng(0)
    bs, ps = 40, 4
    lens, owned, table, ring, state = pool_state(rng, bs, ps, 32, 60, 25)
    new = rng.integers(0, 20, bs)
    assert both(lens, new, owned, table, ring, state, ps, int(new.sum()))["n_bad"] > 0
    assert both(lens, new, owned, table, ring, state, ps, 7)["n_bad"] > 0   # maps cut short
    both(lens, new, owned, table, ring, state, ps, 0)


def test_bad_requests_and_states():
    rng = np.random.default_rng(1)
    bs, ps, mp = 9, 4, 16
    lens, owned, table, ring, state = pool_state(rng, bs, ps, mp, 40, 50)
    new = rng.integers(1, 9, bs)
    for name, r, v in (("lens", 2, -1), ("new", 3, -5), ("owned", 4, -1), ("owned", 5, mp + 1),
                       ("new", 6, 1000), ("lens", 7, 2 ** 31 - 1)):
        a = dict(lens=lens.copy(), new=new.copy(), owned=owned.copy())
        a[name][r] = v
        w = both(a["lens"], a["new"], a["owned"], table, ring, state, ps,
                 int(np.maximum(a["new"], 0).sum()))
        assert w["n_bad"] > 0
    both(lens, new, owned, table, ring, state, ps, 99, shared=np.array([0, -1] + [0] * 7))
    for s in ([-1, 5], [len(ring), 5], [0, len(ring) + 1], [0, -1]):
        both(lens, new, owned, table, ring, np.array(s), ps, 99)
    bad_ring = ring.copy()
    bad_ring[(state[0] + 1) % len(ring)] = len(ring) + 3
    both(lens, new, owned, table, bad_ring, state, ps, 99)
    bad_table = table.copy()
    bad_table[0, 0] = 10 ** 6
    both(np.minimum(lens, 1), new, owned, bad_table, ring, state, ps, 99)
    # bookkeeping that adds up to more pages than the pool: nothing is pushed
    both(np.zeros(bs, int), np.zeros(bs, int), owned, table, ring, np.array([0, len(ring)]), ps, 1)


def test_largest_batch_and_empty_batch():
    rng = np.random.default_rng(2)
    bs, ps = 16384, 16
    lens = rng.integers(0, 64, bs)
    owned = (lens + ps - 1) // ps
    new = rng.integers(0, 3, bs)
    pool = int(owned.sum()) + bs
    perm = rng.permutation(pool)
    table = np.full((bs, 6), -1)
    table[np.arange(6)[None] < owned[:, None]] = perm[:int(owned.sum())]
    ring = np.full(pool, -1)
    ring[:bs] = perm[int(owned.sum()):]
    both(lens, new, owned, table, ring, np.array([0, bs]), ps, int(new.sum()))
    e = torch.zeros(0, dtype=torch.int32, device=DEV)
    o = bdsa.block_table_update(e, e, e, torch.zeros((0, 4), dtype=torch.int32, device=DEV),
                                dev(np.arange(8)), dev([3, 2]), page_size=4, total_tokens=0)
    assert o["free_state"].tolist() == [3, 2] and o["cu_tokens"].tolist() == [0]


def test_rounds_of_serving_conserve_pages():
    """Two hundred rounds on the device alone, ping-ponging the state; the pages
    held and free are a permutation of the pool at the end, and the last slots
    are prepare_block's."""
    rng = np.random.default_rng(3)
    bs, ps, mp, pool = 24, 8, 40, 900
    table, ring = dev(np.full((bs, mp), -1)), dev(rng.permutation(pool))
    owned, state = dev(np.zeros(bs)), dev([0, pool])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens = np.zeros(bs, int)
    for _ in range(200):
        lens = np.where((rng.random(bs) < 0.1) | (lens > 250), 0, lens)
        new = np.full(bs, 16)
        o = bdsa.block_table_update(dev(lens), dev(new), owned, table, ring, state, page_size=ps,
                                    total_tokens=bs * 16, dev_status=status)
        owned, state = o["owned"], o["free_state"]
        ids, pos, loc = bdsa.prepare_block(dev(np.zeros(bs)), dev(lens), table, pool, 16, ps, 0,
                                           dev_status=status)
        assert (o["slot_map"].view(bs, 16) == loc).all()
        assert (o["positions"].view(bs, 16) == pos).all()
        lens = lens + rng.integers(1, 17, bs)
    assert status.item() == 0
    t, ow, f, st = (x.cpu().numpy() for x in (table, owned, ring, state))
    held = np.concatenate([t[r, :ow[r]] for r in range(bs)])
    free = f[(st[0] + np.arange(st[1])) % pool]
    assert sorted(np.concatenate([held, free]).tolist()) == list(range(pool))


def test_unaligned_maps_and_graph():
    rng = np.random.default_rng(4)
    bs, ps = 50, 16
    lens, owned, table, ring, state = pool_state(rng, bs, ps, 16, 100, 200)
    new = rng.integers(0, 9, bs)
    n = int(new.sum())
    want = oracle.block_table_update(lens, new, owned, table, ring, state, ps, n)
    out = dict(owned=dev(np.zeros(bs)), free_state=dev(np.zeros(2)),
               cu_tokens=dev(np.zeros(bs + 1)), slot_map=dev(np.zeros(n + 1))[1:],
               positions=dev(np.zeros(n + 1))[1:])
    t, f = dev(table), dev(ring)
    a = (dev(lens), dev(new), dev(owned), t, f, dev(state))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        bdsa.block_table_update(*a, page_size=ps, total_tokens=n, out=out)
    for _ in range(2):  # nothing is released, so the replay repeats itself
        g.replay()
        torch.cuda.synchronize()
        for k in ("owned", "free_state", "cu_tokens", "slot_map", "positions"):
            assert (out[k].cpu().numpy() == want[k]).all()
        assert (t.cpu().numpy() == want["block_table"]).all()


def test_refusals():
    i = torch.zeros(4, dtype=torch.int32, device=DEV)
    bt = torch.zeros((4, 3), dtype=torch.int32, device=DEV)
    ok = dict(page_size=4, total_tokens=4)
    with pytest.raises(ValueError):
        bdsa.block_table_update(i[:3], i, i, bt, i, i[:2], **ok)
    with pytest.raises(TypeError):
        bdsa.block_table_update(i.float(), i, i, bt, i, i[:2], **ok)
    with pytest.raises(ValueError):
        bdsa.block_table_update(i, i, i, bt, i, i[:3], **ok)
    with pytest.raises(bdsa.BdsaError):
        bdsa.block_table_update(i, i, i, bt, i, i[:2], page_size=0, total_tokens=4)
    own = torch.zeros(4, dtype=torch.int32, device=DEV)
    out = bdsa.block_table_update(i, i, own, bt, dev(np.arange(4)), dev([0, 4]), **ok)
    with pytest.raises(bdsa.BdsaError):   # in place
        bdsa.block_table_update(i, i, out["owned"], bt, dev(np.arange(4)), dev([0, 4]), out=out,
                                **ok)
