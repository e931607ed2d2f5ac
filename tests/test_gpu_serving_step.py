"""The serving operators together, as a speculative step uses them: pages for the
next block, the block's ids and slots, a draft pass and a verify pass behind
shared prefixes, sampled drafts, filtered targets, acceptance, and the pages
behind the committed tokens given back.

Each operator's outputs are checked against its oracle on the inputs it got in
the step.  The tolerances are those of the operators' own tests: attention
1e-2 / 1e-3 / 1e-3 (bf16 inputs, P rounded to bf16), a probability 3.1 x 2^-24
plus V units of 2^-42 relative, everything else equal (rows the oracles mark as
within 1e-9 of a border aside)."""
import numpy as np
import pytest
import torch

import block_diffusion_speculative_attn_gb300 as bdsa
import oracle
from block_diffusion_speculative_attn_gb300 import workloads as wl
from gpu_helpers import assert_attn_close

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Engine:
    """A toy model (random maps, one layer) and the state of a batch in groups
    with shared prompts."""

    def __init__(self, groups, prompts, B, Hq, Hkv, D, V, ps, seed):
        rng = np.random.default_rng(seed)
        self.B, self.Hq, self.Hkv, self.D, self.V, self.ps = B, Hq, Hkv, D, V, ps
        self.bs = bs = int(np.sum(groups))
        gid = np.repeat(np.arange(len(groups)), groups)
        pre_pages = np.asarray(prompts) // ps
        self.prefix = (pre_pages * ps).astype(np.int32)
        own_len = rng.integers(0, 3 * ps, bs)
        seq = self.prefix[gid] + own_len
        have = -(-seq // ps)
        self.max_pages = int(have.max()) + 8
        spare = bs * 4
        total = int(pre_pages.sum() + (have - pre_pages[gid]).sum()) + spare
        perm = rng.permutation(total).astype(np.int32)
        table = np.full((bs, self.max_pages), -1, np.int32)
        at = 0
        offs = np.concatenate([[0], np.cumsum(groups)])
        for g in range(len(groups)):
            table[offs[g]:offs[g + 1], :pre_pages[g]] = perm[at:at + pre_pages[g]]
            at += int(pre_pages[g])
        for r in range(bs):
            n0, n = int(pre_pages[gid[r]]), int(have[r])
            table[r, n0:n] = perm[at:at + n - n0]
            at += n - n0
        ring = np.full(total, -1, np.int32)
        head = total - 3                                # the ring wraps at once
        ring[(head + np.arange(spare)) % total] = perm[at:]
        self.pages, self.max_ctx = total, self.max_pages * ps - B
        i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(DEV)
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s, k=1.0: (torch.randn(s, generator=g) * k).to(DEV)
        E = 64
        self.w = dict(emb=rnd(V, E), q=rnd(E, Hq * D, k=0.12), k=rnd(E, Hkv * D, k=0.12),
                      v=rnd(E, Hkv * D, k=0.12), o=rnd(Hq * D, V, k=0.5), pos=rnd(4096, E, k=0.3))
        self.offs, self.prefix_lens = i32(offs), i32(self.prefix)
        self.shared = i32(pre_pages[gid])
        self.params = dict(temperature=torch.linspace(0.7, 1.3, bs, device=DEV),
                           top_k=i32(rng.integers(5, 60, bs)),
                           top_p=torch.linspace(0.8, 0.99, bs, device=DEV))
        self.state = dict(seq=i32(seq), owned=i32(have), table=i32(table), ring=i32(ring),
                          free=i32([head, spare]), last=i32(rng.integers(1, V, bs)),
                          k=rnd(total * ps, Hkv, D).to(torch.bfloat16),
                          v=rnd(total * ps, Hkv, D).to(torch.bfloat16))
        self.block = i32(np.full(bs, B))
        self.none = i32(np.zeros(bs))
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def uniforms(self, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        return torch.rand((3, self.bs, self.B), generator=g, device=DEV)

    def forward(self, s, seq, ids, positions, slots, mode, log):
        x = self.w["emb"][ids.reshape(-1).long()]
        x = x + self.w["pos"][positions.reshape(-1).long() % 4096]
        head = lambda n, h: (x @ self.w[n]).view(-1, h, self.D).to(torch.bfloat16)
        q = head("q", self.Hq)
        s["k"].index_copy_(0, slots.long(), head("k", self.Hkv))
        s["v"].index_copy_(0, slots.long(), head("v", self.Hkv))
        lse = torch.empty((self.bs * self.B, self.Hq), device=DEV)
        a = bdsa.block_attn_paged(q, s["k"], s["v"], s["table"], seq, B=self.B,
                                  page_size=self.ps, scale=self.D ** -0.5, mode=mode,
                                  max_ctx_len=self.max_ctx, lse=lse, dev_status=self.status,
                                  group_offsets=self.offs, prefix_lens=self.prefix_lens)
        if log is not None:
            log.append(("attn", dict(q=q, k=s["k"].clone(), v=s["v"].clone(),
                                     table=s["table"].clone(), seq=seq.clone(), mode=mode),
                        dict(out=a, lse=lse)))
        return (a.reshape(self.bs, self.B, -1).float() @ self.w["o"])

    def table(self, s, seq, new, total, log):
        before = {k: s[k].clone() for k in ("table", "ring", "owned", "free")}
        o = bdsa.block_table_update(seq, new, s["owned"], s["table"], s["ring"], s["free"],
                                    page_size=self.ps, total_tokens=total, shared=self.shared,
                                    dev_status=self.status)
        s["owned"], s["free"] = o["owned"], o["free_state"]
        if log is not None:
            log.append(("table", dict(before, seq=seq.clone(), new=new.clone(), total=total),
                        dict(o, table=s["table"].clone(), ring=s["ring"].clone())))
        return o

    def step(self, s, u, log=None):
        """One draft / verify / accept step of every request; s is updated."""
        B, V = self.B, self.V
        maps = self.table(s, s["seq"], self.block, self.bs * B, log)
        ids, positions, slots = bdsa.prepare_block(s["last"], s["seq"], s["table"], self.pages, B,
                                                   self.ps, 0, dev_status=self.status)
        if log is not None:
            log.append(("slots", dict(slots=slots, positions=positions), maps))
        draft = self.forward(s, s["seq"], ids, positions, maps["slot_map"], wl.DRAFT, log)
        tokens, q = bdsa.token_sample(draft[:, 1:], u[0][:, 1:].contiguous(),
                                      temperature=self.params["temperature"], want_probs=True,
                                      dev_status=self.status)
        ids[:, 1:] = tokens
        target = self.forward(s, s["seq"], ids, positions, maps["slot_map"], wl.VERIFY, log)
        _, p = bdsa.token_sample(target, want_probs=True, dev_status=self.status, **self.params)
        args = dict(u_acc=u[1][:, 1:].contiguous(), u_samp=u[2][:, 0].contiguous())
        acc = bdsa.spec_accept(ids, p, q, args["u_acc"], args["u_samp"], s["seq"],
                               dev_status=self.status)
        if log is not None:
            one = dict(temperature=self.params["temperature"])
            log.append(("sample", dict(l=draft[:, 1:], u=u[0][:, 1:], **one),
                        dict(t=tokens, p=q)))
            log.append(("sample", dict(l=target, u=None, **self.params), dict(t=None, p=p)))
            log.append(("accept", dict(ids=ids, p=p, q=q, seq=s["seq"], **args), acc))
        s["seq"], s["last"] = acc["new_seq_lens"], acc["bonus_id"]
        self.table(s, s["seq"], self.none, 0, log)
        return acc

    # ---------------------------------------------------------- the oracles
    def check(self, log):
        n = lambda t: None if t is None else t.cpu().numpy()
        for what, a, got in log:
            if what == "table":
                want = oracle.block_table_update(n(a["seq"]), n(a["new"]), n(a["owned"]),
                                                 n(a["table"]), n(a["ring"]), n(a["free"]), self.ps,
                                                 a["total"], n(self.shared))
                assert want["n_bad"] == 0
                for k, w in (("table", "block_table"), ("ring", "free_pages"), ("owned", "owned"),
                             ("free_state", "free_state"), ("cu_tokens", "cu_tokens"),
                             ("slot_map", "slot_map"), ("positions", "positions")):
                    assert (n(got[k]) == want[w]).all(), k
            elif what == "slots":  # two ways to the same slots
                assert (n(a["slots"]).reshape(-1) == n(got["slot_map"])).all()
                assert (n(a["positions"]).reshape(-1) == n(got["positions"])).all()
            elif what == "attn":
                bits = lambda t: wl.bf16_bits(t.cpu())
                ref, rlse = oracle.block_attn(bits(a["q"]), bits(a["k"]), bits(a["v"]),
                                              n(a["table"]), n(a["seq"]), self.B, self.Hq,
                                              self.Hkv, self.D, self.ps, self.D ** -0.5,
                                              a["mode"], num_pages=self.pages, nthreads=16)
                assert_attn_close(got["out"], ref, got["lse"], rlse, f"mode {a['mode']}")
            elif what == "sample":
                kw = {k: n(v) for k, v in a.items() if k not in ("l", "u")}
                t, p, near = oracle.token_sample(n(a["l"].double()), n(a["u"]), **kw)
                ok = ~near
                if got["t"] is not None:
                    assert (n(got["t"])[ok] == t[ok]).all()
                err = np.abs(n(got["p"])[ok] - p[ok])
                assert (err <= (3.1 * 2.0 ** -24 + self.V * 2.0 ** -42 + 2.0 ** -37) * p[ok]
                        + 1e-37).all()
            else:
                want = oracle.spec_accept(n(a["ids"]), n(a["p"]), n(a["q"]), n(a["u_acc"]),
                                          n(a["u_samp"]), n(a["seq"]))
                ok = (want["flags"] & 2) == 0
                for k in ("accept_len", "commit_len", "bonus_id", "new_seq_lens"):
                    assert (n(got[k])[ok] == want[k][ok]).all(), k
        assert self.status.item() == 0

    def check_pages(self, s):
        """Every page is in one place: shared, owned by one request, or free."""
        n = lambda t: t.cpu().numpy()
        table, owned, shared, ring = n(s["table"]), n(s["owned"]), n(self.shared), n(s["ring"])
        head, count = n(s["free"])
        own = [table[r, shared[r]:owned[r]] for r in range(self.bs)]
        common = [table[int(o), :shared[int(o)]] for o in n(self.offs)[:-1]]
        free = [ring[(head + np.arange(count)) % len(ring)]]
        assert (np.sort(np.concatenate(own + common + free)) == np.arange(self.pages)).all()
        for r in range(self.bs):
            assert (table[r, owned[r]:] == -1).all()


@pytest.mark.parametrize("groups,prompts,B,Hq,Hkv,D,V,ps", [
    ([3, 1], [300, 140], 8, 4, 2, 64, 1009, 16),
    ([5, 2, 4], [1024, 0, 517], 16, 8, 2, 128, 5003, 32),
    ([9], [260], 4, 8, 1, 128, 40001, 8),
])
def test_steps(groups, prompts, B, Hq, Hkv, D, V, ps):
    e = Engine(groups, prompts, B, Hq, Hkv, D, V, ps, seed=V)
    e.check_pages(e.state)
    committed = 0
    for i in range(3):
        log = []
        acc = e.step(e.state, e.uniforms(i), log)
        e.check(log)
        e.check_pages(e.state)
        committed += int(acc["commit_len"].sum())
    assert committed >= 3 * e.bs


def test_step_in_a_graph():
    """The whole step captured once and replayed over changing state."""
    e = Engine([4, 2], [400, 200], 8, 8, 2, 128, 3001, 16, seed=11)
    static = {k: v.clone() for k, v in e.state.items()}
    u = e.uniforms(0)
    keep = {k: v.clone() for k, v in static.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        e.step(dict(static), u)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    after = dict(static)
    with torch.cuda.graph(g):
        e.step(after, u)
    state = {k: v.clone() for k, v in keep.items()}
    for i in range(3):
        for k, v in static.items():
            v.copy_(state[k])
        u.copy_(e.uniforms(20 + i))
        g.replay()
        log = []
        want = {k: v.clone() for k, v in state.items()}
        e.step(want, u.clone(), log)
        e.check(log)
        for k in static:
            assert torch.equal(after[k], want[k]), k
        state = {k: v.clone() for k, v in after.items()}
    e.check_pages(state)
