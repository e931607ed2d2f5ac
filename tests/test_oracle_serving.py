"""Pins of the serving operators' oracles: cases worked by hand, and properties
that do not go through the oracle's own arithmetic."""
import numpy as np
import pytest

import oracle


def sample(l, u=None, **kw):
    l = np.asarray(l, np.float64)[None, None]
    kw = {k: np.asarray([v]) for k, v in kw.items()}
    t, p, near = oracle.token_sample(l, None if u is None else np.full((1, 1), u), **kw)
    return int(t[0, 0]), p[0, 0], bool(near[0, 0])


# weights 4 : 2 : 1 : 1 at indices 2, 0, 1, 3
L4 = np.log([2.0, 1.0, 4.0, 1.0])


@pytest.mark.parametrize("kw,want", [
    (dict(), [2, 1, 4, 1]),
    (dict(top_k=1), [0, 0, 4, 0]),
    (dict(top_k=3), [2, 1, 4, 0]),              # the tie at weight 1 goes to the lower index
    (dict(top_k=0), [2, 1, 4, 1]),              # off
    (dict(top_k=9), [2, 1, 4, 1]),
    (dict(top_p=0.49), [0, 0, 4, 0]),           # 4/8 reaches 0.49
    (dict(top_p=0.51), [2, 0, 4, 0]),
    (dict(top_p=0.8), [2, 1, 4, 0]),
    (dict(top_p=0.0), [0, 0, 4, 0]),
    (dict(top_p=1.0), [2, 1, 4, 1]),
    (dict(top_k=2, top_p=0.6), [0, 0, 4, 0]),   # 4/6 of the first two reaches 0.6
    (dict(min_p=0.3), [2, 0, 4, 0]),
    (dict(min_p=2.0), [0, 0, 4, 0]),            # the first of the order always stays
    (dict(temperature=0.5), [4, 1, 16, 1]),
    (dict(temperature=0.0), [0, 0, 1, 0]),
])
def test_filters_by_hand(kw, want):
    _, p, _ = sample(L4, **kw)
    np.testing.assert_allclose(p, np.asarray(want) / np.sum(want), rtol=1e-12)


@pytest.mark.parametrize("u,tok", [(0.0, 0), (0.24, 0), (0.26, 1), (0.374, 1), (0.376, 2),
                                   (0.874, 2), (0.876, 3), (0.999, 3)])
def test_draw_is_inverse_cdf_in_index_order(u, tok):
    assert sample(L4, u)[0] == tok


def test_masked_rows_and_values():
    inf, nan = np.inf, np.nan
    t, p, _ = sample([-inf, nan, 0.0, 0.0], 0.6)
    assert t == 3 and p.tolist() == [0, 0, 0.5, 0.5]
    t, p, _ = sample([-inf, nan], 0.6)
    assert t == -1 and not p.any()
    t, p, _ = sample([0.0, inf, 3.0, inf], 0.4)
    assert t == 1 and p.tolist() == [0, 0.5, 0, 0.5]
    for T in (-1.0, nan, inf):
        t, p, _ = sample([0.0, 1.0], 0.4, temperature=T)
        assert t == -1 and not p.any()
    assert sample([1.0, 3.0, 3.0], 0.9, temperature=0.0)[0] == 1


def test_kept_sets_are_nested_prefixes():
    rng = np.random.default_rng(5)
    l = rng.normal(size=200) * 2
    full = sample(l)[1]
    for k in (1, 7, 50):
        p = sample(l, top_k=k)[1]
        assert (p > 0).sum() == k and full[p > 0].min() >= full[p == 0].max()
    last = 0
    for tp in (0.1, 0.5, 0.9, 0.99):
        p = sample(l, top_p=tp)[1]
        n = int((p > 0).sum())
        assert full[p > 0].sum() >= tp and np.sort(full[p > 0])[1:].sum() < tp
        assert n >= last
        last = n


def test_table_by_hand():
    # ps 4; request 0 grows by one page, 1 shrinks to nothing, 2 keeps its
    # shared page, 3 needs nothing new
    table = np.array([[7, -1, -1], [3, 5, -1], [6, 2, -1], [1, -1, -1]])
    ring = np.array([9, -1, -1, -1, -1, -1, 4, 0, 8, 10, 11])   # head 6: 4, 0, 8, 10, 11, 9
    o = oracle.block_table_update([4, 0, 0, 1], [3, 0, 0, 2], [1, 2, 2, 1], table, ring, [6, 6], 4,
                                  8, shared=[0, 0, 1, 0])
    assert o["block_table"].tolist() == [[7, 4, -1], [-1, -1, -1], [6, -1, -1], [1, -1, -1]]
    assert o["owned"].tolist() == [2, 0, 1, 1]
    assert o["free_state"].tolist() == [7, 8]
    # behind 9 (cell 0): 3, 5, 2
    assert o["free_pages"].tolist()[:4] == [9, 3, 5, 2]
    assert o["cu_tokens"].tolist() == [0, 3, 3, 3, 5]
    assert o["slot_map"].tolist() == [16, 17, 18, 5, 6, -7, -7, -7]
    assert o["positions"].tolist() == [4, 5, 6, 1, 2, -7, -7, -7]
    assert o["n_bad"] == 0


def test_table_shortage_is_first_come_first_served():
    table = np.full((3, 4), -1)
    o = oracle.block_table_update([0, 0, 0], [2, 3, 1], [0, 0, 0], table, np.arange(4), [0, 4], 1,
                                  6)
    assert o["owned"].tolist() == [2, 0, 0]     # 3 do not fit the 2 left; request 2 waits too
    assert o["free_state"].tolist() == [2, 2]
    assert o["slot_map"].tolist() == [0, 1, -1, -1, -1, -1] and o["n_bad"] > 0


def test_table_conserves_pages():
    rng = np.random.default_rng(3)
    pool, bs, ps = 400, 12, 8
    table, owned = np.full((bs, 64), -1), np.zeros(bs, int)
    ring, state = rng.permutation(pool), [0, pool]
    lens = np.zeros(bs, int)
    for _ in range(60):
        new = rng.integers(0, 40, bs)
        lens = np.where(rng.random(bs) < 0.2, 0, lens)
        o = oracle.block_table_update(lens, new, owned, table, ring, state, ps, 1000)
        table, ring, owned, state = (o[k] for k in ("block_table", "free_pages", "owned",
                                                    "free_state"))
        lens = np.minimum(lens + new, owned * ps)
        held = np.concatenate([table[r, :owned[r]] for r in range(bs)])
        free = ring[(state[0] + np.arange(state[1])) % pool]
        assert sorted(np.concatenate([held, free]).tolist()) == list(range(pool))
