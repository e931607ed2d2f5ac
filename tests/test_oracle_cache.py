"""Pins of the oracles of the prompt and cache calls (CPU)."""
import numpy as np
import pytest
import torch

import oracle
from block_diffusion_speculative_attn_gb300 import workloads as wl


@pytest.mark.parametrize("mode,mb", [(wl.VERIFY, 1), (wl.DRAFT, 1 << 20)])
def test_chunk_attn_of_blocks_is_block_attention(mode, mb):
    cfg = wl.config("tiny")
    inp = wl.make_attn_inputs(cfg, device="cpu")
    ref, ref_lse = oracle.block_attn(wl.bf16_bits(inp.q), wl.bf16_bits(inp.k_cache),
                                     wl.bf16_bits(inp.v_cache), inp.block_table, inp.seq_lens,
                                     cfg.B, cfg.Hq, cfg.Hkv, cfg.D, cfg.page_size, inp.scale,
                                     mode, num_pages=inp.num_pages)
    cu = np.arange(cfg.bs + 1) * cfg.B
    out, lse, weight = oracle.chunk_attn(inp.q.double().numpy(), inp.k_cache.double().numpy(),
                                         inp.v_cache.double().numpy(), inp.block_table,
                                         inp.seq_lens, cu, cfg.page_size, inp.scale, mb)
    # (that oracle accumulates in fp64 too and hands out fp64 or fp32)
    assert np.abs(out - ref).max() < 1e-6 and np.abs(lse - ref_lse).max() < 1e-5
    assert (weight >= np.abs(out) - 1e-12).all()


def test_chunk_attn_blocks_against_torch():
    rng = np.random.default_rng(0)
    L, n, mb, D, ps = 13, 21, 8, 16, 8
    table = rng.permutation(5)[None]
    q, k, v = rng.normal(size=(n, 2, D)), rng.normal(size=(40, 1, D)), rng.normal(size=(40, 1, D))
    out, lse, _ = oracle.chunk_attn(q, k, v, table, [L], [0, n], ps, 0.3, mb)
    slots = table[0, np.arange(L + n) // ps] * ps + np.arange(L + n) % ps
    pos = torch.arange(L, L + n)
    mask = torch.arange(L + n)[None] < torch.clamp((pos // mb + 1) * mb, max=L + n)[:, None]
    t = lambda a: torch.from_numpy(a)[None].transpose(1, 2)  # noqa: E731
    ref = torch.nn.functional.scaled_dot_product_attention(
        t(q), t(k[slots]).expand(1, 2, -1, -1), t(v[slots]).expand(1, 2, -1, -1), attn_mask=mask,
        scale=0.3)
    assert np.abs(out - ref[0].transpose(0, 1).numpy()).max() < 1e-12


def test_fork_by_hand():
    # row 0: 2.5 pages [4, 1, 6], row 1 shares page 4 and has [4, 2]; 4 tokens a page
    out = oracle.cache_fork(parent=[0, 0, 1, -1, 1], keep_lens=[10, 10, 8, 3, 6],
                            block_table=[[4, 1, 6, 5], [4, 2, -1, -1]], owned=[4, 2],
                            free_pages=[9, 7, 0, 3, 8, 9, 9, 9, 9, 9], free_state=[1, 4],
                            page_size=4)
    assert out["block_table"].tolist() == [[4, 1, 6, -1], [4, 1, 7, -1], [4, 2, -1, -1],
                                           [-1] * 4, [4, 0, -1, -1]]
    assert out["owned"].tolist() == [3, 3, 2, 0, 2]
    assert out["shared"].tolist() == [2, 2, 1, 0, 1]
    assert out["copy_src"].tolist() == [-1, 6, -1, -1, 2]
    assert out["copy_dst"].tolist() == [-1, 7, -1, -1, 0]
    assert out["copy_len"].tolist() == [0, 2, 0, 0, 2]
    # page 5, reserved past row 0's tokens, goes back behind the tail
    assert out["free_state"].tolist() == [3, 3] and out["free_pages"][5] == 5
    assert out["n_bad"] == 0


def test_fork_keeps_every_page_once():
    """Pages in use and pages free partition the pool before and after, and every
    row reads its parent's tokens."""
    rng = np.random.default_rng(3)
    for _ in range(50):
        ps, bs = int(rng.integers(1, 9)), 6
        owned = rng.integers(0, 6, bs)
        pool = int(owned.sum()) + 25
        ids = rng.permutation(pool)
        table = np.full((bs, 6), -1)
        table[np.arange(6)[None] < owned[:, None]] = ids[:owned.sum()]
        head = int(rng.integers(0, pool))
        ring = np.full(pool, -1)
        ring[(head + np.arange(25)) % pool] = ids[owned.sum():]
        parent = rng.integers(-1, bs, 20)
        keep = [int(rng.integers(0, owned[p] * ps + 1)) if p >= 0 else 0 for p in parent]
        out = oracle.cache_fork(parent, keep, table, owned, ring, [head, 25], ps)
        h, c = out["free_state"]
        free = out["free_pages"][(h + np.arange(c)) % pool]
        held = np.unique(out["block_table"][out["block_table"] >= 0])
        assert sorted([*free, *held]) == list(range(pool))
        token = {(int(table[p, j]), o): (p, j * ps + o) for p in range(bs)
                 for j in range(owned[p]) for o in range(ps)}
        for s, d, n in zip(out["copy_src"], out["copy_dst"], out["copy_len"]):
            for o in range(n):
                token[int(d), o] = token[int(s), o]
        writers = {}
        for r, (p, t) in enumerate(zip(parent, keep)):
            row = out["block_table"][r]
            assert [token[int(row[x // ps]), x % ps] for x in range(t)] == \
                [(p, x) for x in range(t)]
            if t % ps:
                assert writers.setdefault(int(row[t // ps]), r) == r
                assert (out["block_table"] == row[t // ps]).sum() == 1


def test_compact_by_hand():
    cache = np.arange(24).reshape(12, 2)
    table = np.array([[2, 0], [1, -1]])  # 4 slots a page
    out, bad = oracle.cache_compact(cache, table, [1, 0], [[0, 2, 5, -1], [2, 1, -1, -1]], 4)
    # request 0: positions 1, 3, 6 (slots 9, 11, 2) to 1, 2, 3 (slots 9, 10, 11)
    want = cache.copy()
    want[10], want[11] = cache[11], cache[2]
    assert (out == want).all() and bad == 1
