"""GPU parity of the cache calls (write, fork, copy, compact) with their oracles.
They move bytes and whole numbers, so every comparison is exact."""
import numpy as np
import pytest
import torch

import block_diffusion_speculative_attn_gb300 as bdsa
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy()


def rand(shape, seed, dtype=torch.int16):
    """Any bit patterns, NaN among them."""
    g = torch.Generator().manual_seed(seed)
    e = torch.empty((), dtype=dtype).element_size() // 2
    x = torch.randint(-2 ** 15, 2 ** 15, (*shape[:-1], shape[-1] * e), generator=g)
    return x.to(torch.int16).view(dtype).to(DEV)


# ------------------------------------------------------------------ write
@pytest.mark.parametrize("T", [1, 2, 3, 5, 31, 257, 2100])
@pytest.mark.parametrize("H,D,dtype", [(1, 8, torch.bfloat16), (8, 128, torch.bfloat16),
                                       (3, 64, torch.float16), (5, 128, torch.float32),
                                       (9, 128, torch.float32)])
def test_write(T, H, D, dtype):
    slots = T + 37
    wide = rand((T, 4 * H + 1, D), T, dtype)
    k, v = rand((slots, H, D), T + 1, dtype), rand((slots, H, D), T + 2, dtype)
    at = np.random.default_rng(T).permutation(slots)[:T]
    at[::4] = -1
    kn, vn = wide[:, H:2 * H], wide[:, 3 * H:4 * H]
    want_k, want_v = k.clone(), v.clone()
    for t, s in enumerate(at):
        if s >= 0:
            want_k[s], want_v[s] = kn[t], vn[t]
    st = status()
    bdsa.cache_write(kn, vn, i32(at), k, v, dev_status=st)
    assert (bits(k) == bits(want_k)).all() and (bits(v) == bits(want_v)).all()
    assert int(st) == 0


def test_write_slots_outside_the_cache():
    k, v = rand((10, 2, 64), 1), rand((10, 2, 64), 2)
    kn, vn = rand((4, 2, 64), 3), rand((4, 2, 64), 4)
    want_k, want_v, st = k.clone(), v.clone(), status()
    want_k[9], want_v[9] = kn[2], vn[2]
    bdsa.cache_write(kn, vn, i32([10, -2, 9, 2 ** 31 - 1]), k, v, dev_status=st)
    assert (bits(k) == bits(want_k)).all() and (bits(v) == bits(want_v)).all()
    assert int(st) == 16


def test_write_past_2_31_bytes():
    """Slots whose byte offsets need more than 32 bits."""
    slots, H, D = 1_200_000, 8, 128
    k = torch.zeros((slots, H, D), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros((slots, H, D), dtype=torch.bfloat16, device=DEV)
    kn, vn = rand((3, H, D), 5, torch.bfloat16), rand((3, H, D), 6, torch.bfloat16)
    at = [slots - 1, 0, 1_100_000]
    bdsa.cache_write(kn, vn, i32(at), k, v)
    assert (bits(k[at]) == bits(kn)).all() and (bits(v[at]) == bits(vn)).all()
    assert int((k != 0).any(-1).any(-1).sum()) == 3


# ------------------------------------------------------------------ fork
class Fork:
    """Tables whose rows hold scattered pages, some pages held by several rows."""

    def __init__(self, bs, rows, width, ps, seed, free=None, share=0.5, empty=0.1):
        rng = np.random.default_rng(seed)
        self.ps = ps
        self.owned = rng.integers(0, width + 1, bs)
        self.table = np.full((bs, width), -1, np.int64)
        page = 0
        for r in range(bs):
            n0 = 0
            if r and rng.random() < share:  # some leading pages of an earlier row
                s = int(rng.integers(0, r))
                n0 = int(min(self.owned[r], rng.integers(0, self.owned[s] + 1)))
                self.table[r, :n0] = self.table[s, :n0]
            n = self.owned[r] - n0
            self.table[r, n0:self.owned[r]] = page + np.arange(n)
            page += n
        free = rows if free is None else free
        self.pool = page + free + int(rng.integers(1, 5))
        ids = rng.permutation(self.pool)
        self.table = np.where(self.table >= 0, ids[np.maximum(self.table, 0)], -1)
        self.head = int(rng.integers(0, self.pool))
        self.ring = np.full(self.pool, -7)
        self.ring[(self.head + np.arange(free)) % self.pool] = ids[page:page + free]
        self.state = [self.head, free]
        self.parent = rng.integers(0, max(bs, 1), rows)
        self.parent[rng.random(rows) < empty] = -1
        cap = self.owned[self.parent] * ps if bs else np.zeros(rows, np.int64)
        self.keep = (rng.random(rows) * (cap + 1)).astype(np.int64)
        whole = rng.random(rows) < 0.3
        self.keep[whole] = self.keep[whole] // ps * ps

    def run(self, **kw):
        self.ring_dev, self.status = i32(self.ring), status()
        out = bdsa.cache_fork(i32(self.parent), i32(self.keep), i32(self.table), i32(self.owned),
                              self.ring_dev, i32(self.state), page_size=self.ps,
                              dev_status=self.status, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, out=None, bad=False):
        out = out or self.run()
        want = oracle.cache_fork(self.parent, self.keep, self.table, self.owned, self.ring,
                                 self.state, self.ps)
        for key in bdsa.FORK_KEYS:
            assert (out[key].cpu().numpy() == want[key]).all(), key
        assert (self.ring_dev.cpu().numpy() == want["free_pages"]).all()
        assert (int(self.status) == 16) == bad == (want["n_bad"] > 0)
        return out


@pytest.mark.parametrize("bs,rows,width", [(1, 1, 1), (1, 7, 3), (5, 5, 1), (8, 64, 9),
                                           (33, 17, 40), (300, 500, 70), (1000, 3, 5),
                                           (3, 1500, 65), (0, 4, 2), (6, 0, 4)])
@pytest.mark.parametrize("ps", [1, 7, 16, 64])
def test_fork(bs, rows, width, ps):
    # (of no rows, every parent is outside)
    Fork(bs, rows, width, ps, bs * 7 + rows + ps).check(bad=bs == 0)


def test_fork_large():
    f = Fork(4096, 5000, 130, 16, 1, share=0.8)
    f.check()


def test_fork_long_rows():
    """Rows in several parts."""
    Fork(9, 13, 1000, 16, 1, share=0.7).check()
    Fork(3, 40, 8192, 16, 2, share=0.9).check()


@pytest.mark.parametrize("pool", [1, 40000])
def test_fork_of_no_rows_at_all(pool):
    f = Fork(0, 0, 3, 16, 1)
    f.pool, f.ring, f.state = pool, np.arange(pool), [0, 1]
    out = f.check()
    assert out["free_state"].tolist() == [0, 1]


def test_fork_is_the_identity_for_rows_of_their_own():
    f = Fork(40, 40, 6, 16, 2, share=0.0)
    f.parent, f.keep = np.arange(40), f.owned * 16 - (f.owned > 0)
    out = f.check()
    assert (out["block_table"].cpu().numpy() == f.table).all()
    assert int((out["copy_len"] != 0).sum()) == 0 and int(out["shared"].sum()) == 0
    assert out["free_state"].tolist() == f.state


def test_fork_frees_every_page_once():
    f = Fork(50, 50, 20, 8, 3, share=0.9)
    f.parent[:] = -1
    out = f.check()
    used = len(np.unique(f.table[f.table >= 0]))
    assert int(out["free_state"][1]) == f.state[1] + used


@pytest.mark.parametrize("free", [0, 1, 5])
def test_fork_when_the_ring_runs_out(free):
    f = Fork(10, 60, 8, 16, 4, free=free, empty=0.0)
    f.keep = np.maximum(f.keep, 1) // 16 * 16 + 1
    f.keep = np.minimum(f.keep, f.owned[f.parent] * 16)
    f.check(bad=True)


def test_fork_bad_arguments_in_the_data():
    f = Fork(12, 30, 8, 16, 5)
    f.parent[3], f.parent[4], f.keep[5], f.keep[6] = 12, -2, -1, 2 ** 31 - 1
    f.parent[6] = 0
    f.check(bad=True)
    f = Fork(12, 30, 8, 16, 6)
    f.owned[2], f.owned[7] = 9, -3
    f.keep = np.minimum(f.keep, 16)
    f.check(bad=True)
    f = Fork(12, 30, 8, 16, 7)
    f.table[np.arange(12), f.owned // 2] = np.where(f.owned > 0, f.pool + 3, -1)
    f.check(bad=True)
    for state in ([-1, 3], [10 ** 6, 3], [0, 10 ** 6], [0, -1]):
        f = Fork(12, 30, 8, 16, 8)
        f.state = state
        f.check(bad=True)
    f = Fork(12, 30, 8, 16, 9)  # more free pages than the table leaves
    f.state[1] = f.pool
    f.ring[:] = np.arange(f.pool)
    f.parent[:] = -1
    f.check(bad=True)
    f = Fork(12, 30, 8, 16, 10)  # ring cells outside the pool
    f.ring[:] = -5
    f.check(bad=True)


def test_fork_the_same_page_twice_in_a_row():
    f = Fork(6, 12, 8, 16, 11, share=0.0)
    f.owned[:] = 8
    f.table[:, :] = f.table[0, 0] if f.table[0, 0] >= 0 else 0
    f.keep = np.full(12, 100)
    f.parent = np.arange(12) % 6
    f.check()


def test_fork_repeats_itself_and_reuses_outputs():
    f = Fork(60, 80, 12, 16, 12, share=0.7)
    a = f.run()
    ring = f.ring_dev.clone()
    ws = torch.full((bdsa.cache_fork_workspace_bytes(60, 80, f.pool),), 255, dtype=torch.uint8,
                    device=DEV)
    b = f.run(out={k: torch.full_like(v, 99) for k, v in a.items()}, workspace=ws)
    assert all(torch.equal(a[k], b[k]) for k in a) and torch.equal(ring, f.ring_dev)


# ------------------------------------------------------------------ copy
@pytest.mark.parametrize("n,C,H,D,ps,dtype", [(1, 1, 1, 8, 1, torch.int16),
                                              (7, 3, 2, 64, 16, torch.bfloat16),
                                              (40, 10, 8, 128, 64, torch.bfloat16),
                                              (5, 2, 3, 40, 24, torch.float32),
                                              (3, 300, 1, 64, 8, torch.float16),
                                              (2, 1, 16, 256, 1024, torch.float32)])
def test_copy(n, C, H, D, ps, dtype):
    pages = 2 * n + 3
    rng = np.random.default_rng(n)
    ids = rng.permutation(pages)
    src, dst, ln = ids[:n].copy(), ids[n:2 * n], rng.integers(0, ps + 1, n)
    src[n // 2:] = src[0]             # one page to several
    ln[0] = ps
    caches = rand((C, pages * ps, H, D), n, dtype)
    want = caches.clone().view(C, pages, ps, H, D)
    for s, d, m in zip(src, dst, ln):
        want[:, d, :m] = want[:, s, :m]
    st = status()
    bdsa.cache_copy(caches, i32(src), i32(dst), i32(ln), page_size=ps, dev_status=st)
    assert (bits(caches) == bits(want.view_as(caches))).all() and int(st) == 0
    # the same as separate tensors, skipped entries among them
    parts = [c.clone() for c in rand((C, pages * ps, H, D), n, dtype)]
    src2, dst2, ln2 = (np.concatenate([a, b]) for a, b in
                       ((src, [-1, -1, 0]), (dst, [-1, -1, 1]), (ln, [0, 5, 0])))
    bdsa.cache_copy(parts, i32(src2), i32(dst2), i32(ln2), page_size=ps, dev_status=st)
    assert (bits(torch.stack(parts)) == bits(caches)).all() and int(st) == 0


def test_copy_bad_entries():
    caches = rand((2, 80, 2, 64), 1)
    want = caches.clone()
    want[:, 16:32] = want[:, 48:64]
    st = status()
    bdsa.cache_copy(caches, i32([5, -1, 0, 3, 0, 0]), i32([0, 2, 5, 1, 2, 2]),
                    i32([4, 4, 4, 16, 17, -1]), page_size=16, dev_status=st)
    assert (bits(caches) == bits(want)).all() and int(st) == 16


# ------------------------------------------------------------------ compact
def paths(rng, bs, width, nodes, full=False):
    path = np.full((bs, width), -1)
    for r in range(bs):
        m = width if full else int(rng.integers(0, min(width, nodes) + 1))
        path[r, :m] = np.sort(rng.choice(nodes, m, replace=False))
    return path


@pytest.mark.parametrize("bs,C,H,D,ps,width,nodes", [
    (1, 1, 1, 8, 1, 1, 5), (4, 3, 2, 64, 16, 16, 16), (9, 10, 8, 128, 64, 481, 481),
    (3, 2, 3, 40, 24, 600, 3001), (2, 280, 1, 64, 8, 12, 60), (1, 1, 16, 128, 32, 3000, 3001),
    (40, 1, 1, 64, 7, 90, 100)])
def test_compact(bs, C, H, D, ps, width, nodes):
    rng = np.random.default_rng(bs * width)
    path = paths(rng, bs, width, nodes)
    ctx = rng.integers(0, 70, bs)
    need = (ctx + nodes + ps - 1) // ps
    ids = rng.permutation(int(need.sum()) + 1)
    table = np.full((bs, int(need.max()) + 1), -1)
    table[np.arange(table.shape[1])[None] < need[:, None]] = ids[:-1]
    caches = rand((C, len(ids) * ps, H, D), bs, torch.bfloat16)
    before, st = bits(caches), status()
    bdsa.cache_compact(caches, i32(table), i32(ctx), i32(path), page_size=ps, dev_status=st)
    after = bits(caches)
    for c in range(C):
        want, bad = oracle.cache_compact(before[c], table, ctx, path, ps)
        assert (after[c] == want).all() and bad == 0
    assert int(st) == 0


def test_compact_refuses_whole_requests():
    rng = np.random.default_rng(1)
    bs, ps, nodes = 9, 8, 40
    table = rng.permutation(bs * 8).reshape(bs, 8)
    ctx = np.full(bs, 20)
    path = np.full((bs, 6), -1)
    path[:, :5] = [0, 3, 4, 20, 39]
    path[1, 2] = 3                    # twice
    path[2, 1:3] = [5, 4]             # descending
    path[3, 0] = -2                   # below the region
    path[4, 4] = 44                   # position 64 of a row that holds 64
    table[5, 7] = bs * 8              # a source page outside the pool
    table[6, 2] = -1                  # a destination page
    ctx[7] = -1
    cache = rand((bs * 8 * ps, 2, 64), 2)
    before, st = bits(cache), status()
    bdsa.cache_compact([cache], i32(table), i32(ctx), i32(path), page_size=ps, dev_status=st)
    want, bad = oracle.cache_compact(before, table, ctx, path, ps)
    assert bad == 7 and int(st) == 16 and (bits(cache) == want).all()
    assert (want != before).any()


def test_compact_rows_that_lie_behind_the_kept_ones():
    """First tokens and a window of the last ones: several CTAs share a request."""
    bs, ps, n = 3, 16, 900
    keep = [4 + 200, 3, 4 + 440]
    path = np.full((bs, max(keep)), -1)
    for r, m in enumerate(keep):
        path[r, :m] = np.concatenate([np.arange(min(4, m)), n - max(m - 4, 0) +
                                      np.arange(max(m - 4, 0))])[:m]
    table = np.random.default_rng(3).permutation(bs * 57).reshape(bs, 57)
    caches = rand((3, bs * 57 * ps, 2, 64), 4, torch.bfloat16)
    before, st = bits(caches), status()
    for _ in range(2):  # (the rows that move stay where they were: the same again)
        bdsa.cache_compact(caches, i32(table), i32(np.zeros(bs)), i32(path), page_size=ps,
                           dev_status=st)
        for c in range(3):
            want, bad = oracle.cache_compact(before[c], table, np.zeros(bs), path, ps)
            assert bad == 0 and (bits(caches)[c] == want).all()
    assert int(st) == 0


def test_lists_longer_than_a_grid():
    n = 70001
    cache = rand((1, 2 * n, 1, 8), 5)
    want = cache.clone()
    want[0, n:] = want[0, :n]
    ids = torch.arange(n, dtype=torch.int32, device=DEV)
    bdsa.cache_copy(cache, ids, ids + n, torch.ones_like(ids), page_size=1)
    assert (bits(cache) == bits(want)).all()
    # a request each: row 1 of its two moves to row 0
    path = torch.ones((n, 1), dtype=torch.int32, device=DEV)
    table = torch.stack([ids, ids + n], 1).contiguous()
    want[0, :n] = want[0, n:]
    cache[0, n:] += 1
    want[0, :n], want[0, n:] = cache[0, n:], cache[0, n:]
    bdsa.cache_compact(cache, table, torch.zeros_like(ids), path, page_size=1)
    assert (bits(cache) == bits(want)).all()


@pytest.mark.parametrize("rows", [20, 700])
def test_fork_captured(rows):
    """As one cluster and as four grids."""
    f = Fork(rows, rows, 60, 16, 30, share=0.8)
    want = f.check()
    ring, parts = i32(f.ring), [i32(x) for x in (f.parent, f.keep, f.table, f.owned, f.state)]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        out = bdsa.cache_fork(parts[0], parts[1], parts[2], parts[3], ring, parts[4],
                              page_size=16)
    for _ in range(3):
        ring.copy_(i32(f.ring))
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], want[k]) for k in out) and torch.equal(ring, f.ring_dev)


# ------------------------------------------------------------------ together
def serving_step(caches, s, ps, x):
    """Prompts written and attended, forked into samples, extended by one token: the
    calls as one program makes them."""
    n = x["lens"].shape[0]
    t = bdsa.block_table_update(s["zero"], x["lens"], s["zero"], s["table"], s["ring"], s["state"],
                                page_size=ps, total_tokens=x["qkv"].shape[0])
    Hq, Hkv = x["Hq"], x["Hkv"]
    k, v = caches[0], caches[1]
    bdsa.cache_write(x["qkv"][:, Hq:Hq + Hkv], x["qkv"][:, Hq + Hkv:], t["slot_map"], k, v)
    o1 = bdsa.chunk_attn_paged(x["qkv"][:, :Hq], k, v, s["table"], s["zero"], t["cu_tokens"],
                               page_size=ps, scale=0.125)
    owned = torch.zeros_like(x["owned_rows"])
    owned[:n] = t["owned"]
    wide = torch.full((owned.numel(), s["table"].shape[1]), -1, dtype=torch.int32, device=DEV)
    wide[:n] = s["table"]
    f = bdsa.cache_fork(x["parent"], x["keep"], wide, owned, s["ring"], t["free_state"],
                        page_size=ps)
    bdsa.cache_copy(caches, f["copy_src"], f["copy_dst"], f["copy_len"], page_size=ps)
    u = bdsa.block_table_update(x["keep"], x["ones"], f["owned"], f["block_table"], s["ring"],
                                f["free_state"], page_size=ps, total_tokens=x["one"].shape[0],
                                shared=f["shared"])
    bdsa.cache_write(x["one"][:, Hq:Hq + Hkv], x["one"][:, Hq + Hkv:], u["slot_map"], k, v)
    o2 = bdsa.chunk_attn_paged(x["one"][:, :Hq], k, v, f["block_table"], x["keep"],
                               u["cu_tokens"], page_size=ps, scale=0.125)
    return o1, o2, f["block_table"], u["owned"], u["free_state"]


@pytest.mark.parametrize("ps", [8, 64])
def test_prompts_forked_and_extended(ps):
    """Every sample attends its prompt's keys and its own token's, whoever shares the
    pages; eager and captured."""
    Hq, Hkv, D, per = 8, 2, 64, 3
    lens = np.array([5, 64, 130, 1, 77])
    n, rows, T = len(lens), per * len(lens), int(lens.sum())
    width, pool = 160 // ps + 2, 100
    g = torch.Generator().manual_seed(1)
    bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    x = dict(Hq=Hq, Hkv=Hkv, lens=i32(lens), qkv=bf(T, Hq + 2 * Hkv, D),
             one=bf(rows, Hq + 2 * Hkv, D), parent=i32(np.arange(rows) % n),
             keep=i32(np.tile(lens, per)), ones=i32(np.ones(rows)), owned_rows=i32(np.zeros(rows)))
    caches = torch.full((2, pool * ps, Hkv, D), float("nan"), dtype=torch.bfloat16, device=DEV)

    def fresh():
        return dict(zero=i32(np.zeros(n)), table=i32(np.full((n, width), -1)),
                    ring=i32(np.random.default_rng(2).permutation(pool)), state=i32([0, pool]))

    s = fresh()
    o1, o2, table, owned, state = serving_step(caches, s, ps, x)
    torch.cuda.synchronize()
    used = torch.unique(table[table >= 0]).numel()
    assert int(state[1]) == pool - used
    cu = np.concatenate([[0], np.cumsum(lens)])
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    for r in range(n):
        at = slice(cu[r], cu[r + 1])
        q, k, v = (f64(x["qkv"][at, a:b]) for a, b in ((0, Hq), (Hq, Hq + Hkv),
                                                      (Hq + Hkv, Hq + 2 * Hkv)))
        one = np.arange(-(-int(lens[r]) // 8))[None]
        pad = lambda a: np.concatenate([a, np.zeros((-len(a) % 8, *a.shape[1:]))])  # noqa: E731
        ref, _, w = oracle.chunk_attn(q, pad(k), pad(v), one, [0], [0, len(q)], 8, 0.125)
        assert (np.abs(f64(o1[at]) - ref) <= 2.0 ** -8 * (np.abs(ref) + w) + 2.0 ** -11 * w).all()
        for j in range(r, rows, n):
            row = f64(x["one"][j])[None]
            ks = pad(np.concatenate([k, row[:, Hq:Hq + Hkv]]))
            vs = pad(np.concatenate([v, row[:, Hq + Hkv:]]))
            ref, _, w = oracle.chunk_attn(row[:, :Hq], ks, vs, np.arange(len(ks) // 8)[None],
                                          [len(k)], [0, 1], 8, 0.125)
            assert (np.abs(f64(o2[j])[None] - ref) <=
                    2.0 ** -8 * (np.abs(ref) + w) + 2.0 ** -11 * w).all()
    # captured, replayed on the start's state
    s2 = fresh()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        got = serving_step(caches, s2, ps, x)
    for _ in range(2):
        for k, t in fresh().items():
            s2[k].copy_(t)
        caches.fill_(float("nan"))
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, (o1, o2, table, owned, state)):
        assert torch.equal(a, b)


def test_accepted_path_compacted_after_a_tree():
    """tree_accept's path as it comes: the next step reads the kept rows in order."""
    rng = np.random.default_rng(5)
    bs, nodes, ps, V = 6, 40, 16, 50
    parent = np.full((bs, nodes), -1)
    for i in range(1, nodes):
        parent[:, i] = rng.integers(max(0, i - 6), i, bs)
    ids = np.tile(np.arange(nodes), (bs, 1))
    p = np.zeros((bs, nodes, V), np.float32)  # every node draws the token of its last child
    for r in range(bs):
        for i in range(nodes):
            kids = np.flatnonzero(parent[r] == i)
            p[r, i, kids[-1] if len(kids) else V - 1] = 1.0
    ctx = rng.integers(0, 40, bs)
    acc = bdsa.tree_accept(i32(ids), i32(parent), torch.from_numpy(p).to(DEV), None, i32(ctx))
    table = rng.permutation(bs * 6).reshape(bs, 6)
    caches = rand((4, bs * 6 * ps, 2, 64), 3, torch.bfloat16)
    before, st = bits(caches), status()
    bdsa.cache_compact(caches, i32(table), i32(ctx), acc["path"], page_size=ps, dev_status=st)
    path = acc["path"].cpu().numpy()
    assert int((path >= 0).sum(1).max()) > 2 and int(st) == 0
    for c in range(4):
        want, bad = oracle.cache_compact(before[c], table, ctx, path, ps)
        assert bad == 0 and (bits(caches)[c] == want).all()


def test_another_stream():
    f = Fork(20, 30, 8, 16, 20)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        out = f.run()
    f.check(out)
