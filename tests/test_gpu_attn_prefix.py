"""GPU parity of bdsa_block_attn_paged_prefix (groups of requests that share a
prefix) against the fp64 block-attention oracle, which knows no prefix: it reads
every request's keys through the request's own row.

Tolerances are the block attention's (bf16 inputs, P rounded to bf16, fp32
elsewhere); the join of prefix and rest adds fp32 roundings only."""
import numpy as np
import pytest
import torch

import block_diffusion_speculative_attn_gb300 as bdsa
import oracle
from block_diffusion_speculative_attn_gb300 import workloads as wl
from gpu_helpers import assert_attn_close

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Case:
    """Requests in groups; the shared pages stand in every row, the rest of each
    row is the request's own.  Slots nobody references hold NaN."""

    def __init__(self, groups, prefixes, own, B, Hq, Hkv, D, ps, seed=0, max_pages=None,
                 spread=1.0):
        rng = np.random.default_rng(seed)
        self.B, self.Hq, self.Hkv, self.D, self.ps = B, Hq, Hkv, D, ps
        self.bs = bs = int(np.sum(groups))
        self.offs = np.concatenate([[0], np.cumsum(groups)]).astype(np.int32)
        self.prefix = np.asarray(prefixes, np.int32)
        gid = np.repeat(np.arange(len(groups)), groups)
        own = np.broadcast_to(np.asarray(own), (bs,))
        self.seq = (self.prefix[gid] + own).astype(np.int32)
        need = (self.seq + B + ps - 1) // ps
        shared = self.prefix // ps                  # whole pages shared
        total = int(shared.sum() + (need - shared[gid]).sum()) + 2
        perm = rng.permutation(total).astype(np.int32)
        width = max_pages or int(need.max()) + 1
        self.table = np.full((bs, width), -1, np.int32)
        at = 0
        for g in range(len(groups)):
            ids = perm[at:at + shared[g]]
            at += int(shared[g])
            self.table[self.offs[g]:self.offs[g + 1], :shared[g]] = ids
        for r in range(bs):
            n0, n = int(shared[gid[r]]), int(need[r])
            self.table[r, n0:n] = perm[at:at + n - n0]
            at += n - n0
        self.num_pages = total
        g = torch.Generator().manual_seed(seed + 1)
        bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)
        self.q, self.k, self.v = (bf(bs * B, Hq, D) * spread, bf(total * ps, Hkv, D),
                                  bf(total * ps, Hkv, D))
        # a prefix that ends inside a page: the page is a copy in each row
        for gi in range(len(groups)):
            part = int(self.prefix[gi] - shared[gi] * ps)
            if part:
                r0 = int(self.offs[gi])
                src = int(self.table[r0, shared[gi]]) * ps
                for r in range(r0 + 1, int(self.offs[gi + 1])):
                    dst = int(self.table[r, shared[gi]]) * ps
                    self.k[dst:dst + part] = self.k[src:src + part]
                    self.v[dst:dst + part] = self.v[src:src + part]
        used = np.zeros(total * ps, bool)
        for r in range(bs):
            t = np.arange(self.seq[r] + B)
            used[self.table[r, t // ps].astype(np.int64) * ps + t % ps] = True
        free = torch.from_numpy(~used)
        self.k[free] = float("nan")
        self.v[free] = float("nan")
        self.scale = 1.0 / np.sqrt(D)

    def dev(self):
        self.d = {n: getattr(self, n).to(DEV) for n in ("q", "k", "v")}
        for n in ("table", "seq", "offs", "prefix"):
            self.d[n] = torch.from_numpy(getattr(self, n)).to(DEV)
        return self.d

    def run(self, mode, d=None, **kw):
        d = d or self.dev()
        lse = torch.full((self.bs * self.B, self.Hq), float("nan"), device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = bdsa.block_attn_paged(d["q"], d["k"], d["v"], d["table"], d["seq"], B=self.B,
                                    page_size=self.ps, scale=self.scale, mode=mode,
                                    max_ctx_len=int(self.seq.max()), num_pages=self.num_pages,
                                    lse=lse, dev_status=status, group_offsets=d["offs"],
                                    prefix_lens=d["prefix"], **kw)
        torch.cuda.synchronize()
        return out, lse, int(status.item())

    def want(self, mode):
        return oracle.block_attn(wl.bf16_bits(self.q), wl.bf16_bits(self.k), wl.bf16_bits(self.v),
                                 self.table, self.seq, self.B, self.Hq, self.Hkv, self.D, self.ps,
                                 self.scale, mode, num_pages=self.num_pages, nthreads=16)

    def check(self, modes=(wl.DRAFT, wl.VERIFY), **kw):
        for mode in modes:
            out, lse, st = self.run(mode, **kw)
            assert st == 0
            ref, rlse = self.want(mode)
            assert_attn_close(out, ref, lse, rlse, f"mode {mode}")


# one small tile-exact case first, then the shapes
def test_smallest():
    Case([2], [128], 8, 8, 2, 1, 64, 16).check()


def test_smallest_d128():
    Case([2], [128], 8, 8, 4, 1, 128, 16).check()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv", [(1, 2, 2), (1, 32, 8), (8, 8, 2), (16, 32, 8), (32, 16, 4),
                                      (16, 64, 8), (5, 6, 2), (3, 35, 5), (64, 4, 2), (1, 128, 1)])
def test_heads_and_blocks(D, B, Hq, Hkv):
    Case([5, 1, 3], [700, 300, 1000], np.arange(1, 10) * 17, B, Hq, Hkv, D, 16, seed=B).check()


@pytest.mark.parametrize("ps", [8, 16, 32, 64, 128, 256, 1024])
def test_page_sizes_and_odd_prefixes(ps):
    Case([3, 2, 4], [1027, 128, 129], [0, 5, 200, 1, 0, 300, 64, 127, 3], 4, 8, 2, 128, ps,
         seed=ps).check()


@pytest.mark.parametrize("prefix", [0, 1, 127, 128, 255, 256, 5000])
def test_prefix_lengths(prefix):
    Case([4], [prefix], [0, 1, 129, 64], 8, 8, 2, 64, 16, seed=prefix).check()


def test_many_units_a_cta():
    """More units than CTAs: whole units, cut units and unit switches in a CTA."""
    rng = np.random.default_rng(0)
    n = rng.integers(1, 6, 40)
    Case(n, rng.integers(0, 900, 40), 20, 8, 32, 8, 128, 32, seed=3).check()


def test_one_unit_over_many_ctas():
    Case([2], [40000], 10, 8, 2, 1, 128, 64, seed=4).check((wl.VERIFY,))


def test_rows_past_two_tiles():
    """A group whose rows fill several 256-row units of each head."""
    Case([40], [640], np.arange(40), 16, 8, 2, 64, 16, seed=5).check()


def test_groups_of_one_equal_the_plain_call():
    """Groups of one request: the join only regroups the sums of the plain call."""
    c = Case([1] * 7, [0, 128, 300, 513, 1024, 90, 777], 33, 16, 8, 2, 128, 16, seed=6)
    c.check()


def test_peaked_scores():
    """Large scores (running-max rescales in the prefix and in the join)."""
    c = Case([4, 2], [1500, 600], 40, 8, 8, 2, 128, 16, seed=7, spread=12.0)
    for mode in (wl.DRAFT, wl.VERIFY):
        out, lse, st = c.run(mode)
        ref, rlse = c.want(mode)
        # P = e^(s - m) carries the relative error of an fp32 score, 2^-22 |s|
        # with |s| < 80 here, on top of the bf16 roundings (2^-9 of |v| < 5)
        g = out.float().cpu().numpy().reshape(ref.shape)
        assert np.abs(g - ref).max() < 5 * (2 ** -8 + 80 * 2.0 ** -22) and st == 0
        assert np.abs(lse.cpu().numpy().reshape(rlse.shape) - rlse).max() < 1e-3


def test_grids():
    c = Case([6, 3], [900, 2000], 77, 16, 16, 4, 128, 32, seed=8)
    for sms in (1, 2, 7, 64, 152, 4096):
        c.check((wl.VERIFY,), sms=sms)


def test_only_the_first_row_holds_the_shared_pages():
    c = Case([4], [512], 30, 8, 8, 2, 128, 64, seed=9)
    ref, rlse = c.want(wl.VERIFY)
    c.table[1:, :8] = 10 ** 6
    out, lse, st = c.run(wl.VERIFY)
    assert st == 0
    assert_attn_close(out, ref, lse, rlse)


def test_bad_requests_get_zeros():
    def rows(c, reqs):
        return np.concatenate([np.arange(r * c.B, (r + 1) * c.B) for r in reqs])

    def expect(c, bad):
        good = [r for r in range(c.bs) if r not in bad]
        out, lse, st = c.run(wl.DRAFT)
        assert st == 16
        o, l = out.float().cpu().numpy(), lse.cpu().numpy()
        assert (o[rows(c, bad)] == 0).all() and (l[rows(c, bad)] == -np.inf).all()
        if good:
            assert np.abs(o[rows(c, good)] - base[rows(c, good)]).max() < 1e-2

    make = lambda: Case([3, 2], [700, 256], 30, 8, 8, 2, 128, 64, seed=10)
    base = make().want(wl.DRAFT)[0].reshape(40, 8, 128)
    c = make()
    c.prefix[1] = -5
    expect(c, [3, 4])
    c = make()
    c.prefix[0] = 731                   # longer than its requests
    expect(c, [0, 1, 2])
    c = make()
    c.prefix[0] = 2 ** 31 - 1
    expect(c, [0, 1, 2])
    c = make()
    c.table[0, 3] = c.num_pages         # a shared page outside the pool
    expect(c, [0, 1, 2])
    c = make()
    c.table[0, 3] = -1
    expect(c, [0, 1, 2])
    c = make()
    c.table[4, 4] = -7                  # an own page
    expect(c, [4])
    for offs in ([0, 3, 4], [1, 3, 5], [0, 6, 5], [0, 3, 9], [-1, 3, 5], [0, -2, 5]):
        c = make()
        c.offs = np.asarray(offs, np.int32)
        expect(c, [0, 1, 2, 3, 4])


def test_two_calls_at_once():
    """Two streams, a workspace each."""
    a = Case([3, 2], [700, 2560], 30, 8, 8, 2, 128, 64, seed=14)
    b = Case([9], [1280], np.arange(9) * 9, 16, 32, 8, 128, 16, seed=15)
    da, db = a.dev(), b.dev()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for c, d, s in ((a, da, sa), (b, db, sb)):
            with torch.cuda.stream(s):
                lse = torch.empty((c.bs * c.B, c.Hq), device=DEV)
                o = bdsa.block_attn_paged(d["q"], d["k"], d["v"], d["table"], d["seq"], B=c.B,
                                          page_size=c.ps, scale=c.scale, mode=wl.VERIFY,
                                          max_ctx_len=4096, num_pages=c.num_pages, lse=lse,
                                          group_offsets=d["offs"], prefix_lens=d["prefix"])
                outs.append((c, o, lse))
    torch.cuda.synchronize()
    want = {c: c.want(wl.VERIFY) for c in (a, b)}
    for c, o, lse in outs:
        assert_attn_close(o, want[c][0], lse, want[c][1])


def test_workspace_reuse_graph_and_stream():
    """One dirty workspace across calls of different shapes, a side stream, and a
    replayed graph whose inputs change."""
    a = Case([3, 2], [700, 256], 30, 8, 8, 2, 128, 64, seed=11)
    b = Case([9], [1280], np.arange(9) * 9, 16, 32, 8, 64, 16, seed=12)
    n = max(bdsa.block_attn_prefix_workspace_bytes(c.bs, c.B, c.Hq, c.Hkv, c.D, 4096,
                                                   len(c.prefix)) for c in (a, b))
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    for c in (a, b, a, b):
        d = c.dev()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            out, lse, st = c.run(wl.VERIFY, d, workspace=ws)
        ref, rlse = c.want(wl.VERIFY)
        assert_attn_close(out, ref, lse, rlse)
    d = a.dev()
    out = torch.empty_like(d["q"])
    lse = torch.empty((a.bs * a.B, a.Hq), device=DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bdsa.block_attn_paged(d["q"], d["k"], d["v"], d["table"], d["seq"], B=a.B,
                              page_size=a.ps, scale=a.scale, mode=wl.VERIFY, max_ctx_len=4096,
                              num_pages=a.num_pages, out=out, lse=lse, workspace=ws,
                              group_offsets=d["offs"], prefix_lens=d["prefix"])
    for s in range(3):
        a.q = torch.randn(a.q.shape, generator=torch.Generator().manual_seed(s)).bfloat16()
        d["q"].copy_(a.q)
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        ref, rlse = a.want(wl.VERIFY)
        assert_attn_close(out, ref, lse, rlse)


def test_refusals():
    c = Case([2], [128], 8, 8, 2, 1, 64, 16)
    d = c.dev()
    kw = dict(B=8, page_size=16, scale=0.1, mode=1, max_ctx_len=200, num_pages=c.num_pages)
    args = (d["q"], d["k"], d["v"], d["table"], d["seq"])
    with pytest.raises(ValueError):
        bdsa.block_attn_paged(*args, group_offsets=d["offs"], **kw)
    with pytest.raises(ValueError):
        bdsa.block_attn_paged(*args, group_offsets=d["prefix"], prefix_lens=d["prefix"], **kw)
    with pytest.raises(TypeError):
        bdsa.block_attn_paged(*args, group_offsets=d["offs"].long(), prefix_lens=d["prefix"], **kw)
    with pytest.raises(ValueError):
        bdsa.block_attn_paged(*args, group_offsets=d["offs"], prefix_lens=d["prefix"],
                              tree_mask=torch.zeros(16, dtype=torch.int64, device=DEV), **kw)
    with pytest.raises(bdsa.BdsaError):   # more groups than requests
        bdsa.block_attn_paged(*args, group_offsets=torch.zeros(4, dtype=torch.int32, device=DEV),
                              prefix_lens=torch.zeros(3, dtype=torch.int32, device=DEV), **kw)
    with pytest.raises(bdsa.BdsaError):   # workspace too small
        bdsa.block_attn_paged(*args, group_offsets=d["offs"], prefix_lens=d["prefix"],
                              workspace=torch.empty(256, dtype=torch.uint8, device=DEV), **kw)
    with pytest.raises(ValueError):
        bdsa.block_attn_paged(d["q"][:8].contiguous(), *args[1:], group_offsets=d["offs"],
                              prefix_lens=d["prefix"], **kw)
