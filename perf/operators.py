"""The serving operators around the draft/verify step, as measured work.

Three operators, each with the plain form of its definition and the framework's
call:

  sample  logits [bs, B, V] -> the distribution p that the acceptance calls
          read (temperature, top-k, top-p, min-p) and a token drawn from given
          uniforms
  attn    block attention of a batch whose requests share a long prefix, the
          prefix attended once for each group of requests
  table   block tables grown from request lengths out of a ring of free pages,
          with the slot and the position of every new token

`listed()` names the cases, `draw(rng)` makes one more of the same ranges,
`prepare` makes a program's state, `run` is one pass, `exact` the definition in
64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DRAFT, VERIFY = 0, 1
_DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one small draft block in full precision with every filter set: a
        # call whose cost is its latency
        dict(name="sample_tiny", op="sample", bs=2, B=8, V=1000, dtype="fp32", std=2.0,
             filters="all", probs=True),
        # tokens of one decode step for a batch of chats: nucleus sampling, odd
        # vocabulary (rows that start on odd elements), no distribution wanted
        dict(name="sample_decode", op="sample", bs=61, B=1, V=100003, dtype="fp16", std=3.0,
             filters="top_p", probs=False),
        # draft pass: the 15 mask slots of each request drawn at a temperature,
        # their full distributions kept as q for the acceptance
        dict(name="sample_draft", op="sample", bs=32, B=15, V=151936, dtype="bf16", std=3.0,
             filters="temperature", probs=True),
        # verify pass: every slot's filtered distribution as p for the
        # acceptance, and a token of each
        dict(name="sample_verify", op="sample", bs=32, B=16, V=151936, dtype="fp32", std=3.0,
             filters="all", probs=True),
        # the smallest step with a shared prefix: two requests, one KV head
        dict(name="attn_tiny", op="attn", bs=2, Hq=2, Hkv=1, D=64, B=8, ps=16, mode=VERIFY,
             groups=1, prefix_lo=128, prefix_hi=128, own_lo=8, own_hi=96),
        # single-token decode of 64 requests behind one system prompt
        dict(name="attn_decode", op="attn", bs=64, Hq=32, Hkv=8, D=128, B=1, ps=16, mode=VERIFY,
             groups=1, prefix_lo=2048, prefix_hi=2048, own_lo=1, own_hi=512),
        # verify pass of 32 requests behind one few-shot prompt
        dict(name="attn_verify", op="attn", bs=32, Hq=32, Hkv=8, D=128, B=16, ps=64, mode=VERIFY,
             groups=1, prefix_lo=4096, prefix_hi=4096, own_lo=64, own_hi=1024),
        # draft pass (bidirectional blocks) of 64 requests in 8 ragged groups
        dict(name="attn_draft", op="attn", bs=64, Hq=16, Hkv=4, D=128, B=32, ps=32, mode=DRAFT,
             groups=8, prefix_lo=512, prefix_hi=8192, own_lo=1, own_hi=700),
        # verify pass of 8 questions about one long document
        dict(name="attn_long", op="attn", bs=8, Hq=64, Hkv=8, D=128, B=16, ps=64, mode=VERIFY,
             groups=1, prefix_lo=131072, prefix_hi=131072, own_lo=16, own_hi=2048),
        # one draft/verify step of 32 requests: room for 16 more tokens each
        dict(name="table_step", op="table", bs=32, ps=64, have_lo=1024, have_hi=4096,
             new_lo=16, new_hi=16),
        # one decode step of a large batch with small pages
        dict(name="table_decode", op="table", bs=4093, ps=16, have_lo=1, have_hi=2048,
             new_lo=1, new_hi=1),
        # admission of 1024 prompts
        dict(name="table_admit", op="table", bs=1024, ps=16, have_lo=0, have_hi=0,
             new_lo=1, new_hi=4096),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "attn", "table"])
    if op == "sample":
        V = min(_logu(rng, 500, 152000), 151936)
        B = rng.choice([1, 1, 7, 8, 15, 16])
        rows = _logu(rng, 1, 512)
        return dict(op=op, bs=max(1, rows // B), B=B, V=V,
                    dtype=rng.choice(["fp32", "bf16", "fp16"]), std=rng.choice([2.0, 3.0]),
                    filters=rng.choice(["temperature", "top_k", "top_p", "min_p", "all"]),
                    probs=rng.random() < 0.6)
    if op == "attn":
        Hq, Hkv = rng.choice([(2, 1), (16, 4), (32, 8), (64, 8), (24, 8)])
        G = Hq // Hkv
        B = rng.choice([b for b in (1, 3, 8, 16, 32) if G * b <= 128])
        D = rng.choice([64, 128, 128])
        ps = rng.choice([8, 16, 32, 64, 128])
        bs = _logu(rng, 2, 64)
        # at most the rows x keys of the largest listed case
        cap = 8 * 16 * 64 * 131072 // (bs * B * Hq)
        hi = _logu(rng, 256, min(32768, max(512, cap // 2)))
        return dict(op=op, bs=bs, Hq=Hq, Hkv=Hkv, D=D, B=B, ps=ps,
                    mode=rng.choice([DRAFT, VERIFY]), groups=rng.randint(1, max(1, bs // 4)),
                    prefix_lo=max(1, hi // 4), prefix_hi=hi, own_lo=1,
                    own_hi=_logu(rng, 16, 1024))
    bs = _logu(rng, 1, 4096)
    ps = rng.choice([8, 16, 32, 64])
    kind = rng.choice(["step", "admit"])
    if kind == "step":
        n = rng.choice([1, 8, 16, 17])
        return dict(op=op, bs=bs, ps=ps, have_lo=1, have_hi=_logu(rng, 16, 4096),
                    new_lo=n, new_hi=n)
    return dict(op=op, bs=bs, ps=ps, have_lo=0, have_hi=0,
                new_lo=1, new_hi=max(1, min(_logu(rng, 16, 4096), 2000000 // bs)))


# ------------------------------------------------------------------ sample
def _sample_inputs(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 11)
    bs, B, V = c["bs"], c["B"], c["V"]
    lg = torch.randn((bs, B, V), generator=g, device="cuda", dtype=torch.float32)
    # a few strong candidates over a wide bulk, as a language model's head gives
    lg.mul_(c["std"])
    hot = torch.randint(0, V // 4, (bs, B, 4), generator=g, device="cuda") + \
        torch.arange(4, device="cuda") * (V // 4)
    lg.scatter_add_(2, hot, 6.0 + 3.0 * torch.rand((bs, B, 4), generator=g, device="cuda"))
    lg = lg.to(_DTYPES[c["dtype"]])
    rnd = lambda *s: torch.rand(s, generator=g, device="cuda", dtype=torch.float32)
    f = c["filters"]
    p = dict(temperature=None, top_k=None, top_p=None, min_p=None)
    if f in ("temperature", "all", "top_p", "min_p"):
        p["temperature"] = 0.6 + 0.7 * rnd(bs)
    if f in ("top_k", "all"):
        p["top_k"] = torch.randint(20, 101, (bs,), generator=g, device="cuda").to(torch.int32)
    if f in ("top_p", "all"):
        p["top_p"] = 0.8 + 0.19 * rnd(bs)
    if f in ("min_p", "all"):
        p["min_p"] = 0.01 + 0.09 * rnd(bs)
    return lg, rnd(bs, B), p


def _sample_plain(st):
    """Sort each row, cut the sorted order three times, put the rest back."""
    lg, u, p = st["logits"], st["u"], st["params"]
    bs, B, V = lg.shape
    col = lambda t, d: (torch.full((bs,), d, device=lg.device, dtype=torch.float64)
                        if t is None else t.double())[:, None, None]
    sv, si = torch.sort(lg.float(), dim=-1, descending=True, stable=True)
    z = sv.double()
    w = torch.exp((z - z[..., :1]) / col(p["temperature"], 1.0))
    rank = torch.arange(V, device=lg.device)
    keep = torch.ones_like(w, dtype=torch.bool)
    if p["top_k"] is not None:
        keep &= rank < p["top_k"][:, None, None]
    if p["top_p"] is not None:
        wk = torch.where(keep, w, 0.0)
        before = torch.cumsum(wk, -1) - wk
        keep &= before < col(p["top_p"], 1.0) * wk.sum(-1, keepdim=True)
    if p["min_p"] is not None:
        keep &= w >= col(p["min_p"], 0.0)
    keep[..., 0] = True
    w = torch.zeros_like(w).scatter_(-1, si, torch.where(keep, w, 0.0))
    cum = torch.cumsum(w, -1)
    S = cum[..., -1:]
    tok = (cum > u.double()[..., None] * S).to(torch.int8).argmax(-1).to(torch.int32)
    return {"tokens": tok, "probs": (w / S).float()} if st["probs"] else {"tokens": tok}


def _sample_own(st):
    import block_diffusion_speculative_attn_gb300 as bdsa
    p = st["params"]
    tok, pr = bdsa.token_sample(st["logits"], st["u"], temperature=p["temperature"],
                                top_k=p["top_k"], top_p=p["top_p"], min_p=p["min_p"],
                                want_probs=st["probs"])
    return {"tokens": tok, "probs": pr} if st["probs"] else {"tokens": tok}


def _sample_exact(c, seed):
    """Row by row: the cut as a rank below the kept count of a lexicographic order."""
    lg, u, p = _sample_inputs(c, seed)
    bs, B, V = lg.shape
    tokens = np.zeros((bs, B), np.int32)
    probs = torch.zeros((bs, B, V), dtype=torch.float64, device=lg.device) if c["probs"] else None
    host = {k: None if t is None else t.double().tolist() for k, t in p.items()}
    for r in range(bs):
        T = 1.0 if host["temperature"] is None else host["temperature"][r]
        for i in range(B):
            x = lg[r, i].to(torch.float64)
            lp = torch.log_softmax(x / T, 0)
            order = torch.argsort(x, descending=True, stable=True)
            n = V
            if host["top_k"] is not None:
                n = min(n, int(host["top_k"][r]))
            mass = torch.exp(lp[order[:n]])
            if host["top_p"] is not None:
                c0 = torch.cumsum(mass / mass.sum(), 0)
                n = min(n, 1 + int((c0[:-1] < host["top_p"][r]).sum()))
            if host["min_p"] is not None:
                n = min(n, int((mass >= host["min_p"][r] * mass[0]).sum()))
            kept, _ = torch.sort(order[:max(n, 1)])
            pk = torch.softmax(x[kept] / T, 0)
            cdf = torch.cumsum(pk, 0)
            k = torch.searchsorted(cdf, u[r, i].double().reshape(1) * cdf[-1:], right=True)
            tokens[r, i] = int(kept[min(int(k), kept.numel() - 1)])
            if probs is not None:
                probs[r, i, kept] = pk
    tok = torch.from_numpy(tokens).cuda()
    return {"tokens": tok, "probs": probs} if c["probs"] else {"tokens": tok}


# ------------------------------------------------------------------ attn
def _attn_inputs(c, seed):
    rng = np.random.Generator(np.random.PCG64(seed * 104729 + 5))
    bs, B, ps, ng = c["bs"], c["B"], c["ps"], min(c["groups"], c["bs"])
    cuts = np.sort(rng.choice(np.arange(1, bs), ng - 1, replace=False)) if ng > 1 else []
    offs = np.concatenate([[0], cuts, [bs]]).astype(np.int32)
    pre_pages = (rng.integers(c["prefix_lo"], c["prefix_hi"] + 1, ng) + ps - 1) // ps
    own_lens = rng.integers(c["own_lo"], c["own_hi"] + 1, bs)
    gid = np.repeat(np.arange(ng), np.diff(offs))
    seq = pre_pages[gid] * ps + own_lens
    need = (seq + B + ps - 1) // ps
    total = int(pre_pages.sum() + (need - pre_pages[gid]).sum())
    perm = rng.permutation(total).astype(np.int32)
    table = np.full((bs, int(need.max())), -1, np.int32)
    at = 0
    for g in range(ng):
        ids = perm[at:at + pre_pages[g]]
        at += int(pre_pages[g])
        table[offs[g]:offs[g + 1], :pre_pages[g]] = ids
    for r in range(bs):
        n0, n = int(pre_pages[gid[r]]), int(need[r])
        table[r, n0:n] = perm[at:at + n - n0]
        at += n - n0
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    bf = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    return dict(q=bf(bs * B, c["Hq"], c["D"]), k=bf(total * ps, c["Hkv"], c["D"]),
                v=bf(total * ps, c["Hkv"], c["D"]), table=torch.from_numpy(table).cuda(),
                seq=torch.from_numpy(seq.astype(np.int32)).cuda(), lens=seq.tolist(),
                offs=torch.from_numpy(offs).cuda(),
                pre=torch.from_numpy((pre_pages * ps).astype(np.int32)).cuda(), pages=total,
                pre_host=(pre_pages * ps).tolist(), gid=gid.tolist())


def _attn_plain(st):
    """Each request over all of its keys."""
    c = st["case"]
    bs, B, ps, Hq, Hkv, D = (c[k] for k in ("bs", "B", "ps", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(D)
    dev = st["q"].device
    out = torch.empty((bs * B, Hq, D), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((bs * B, Hq), dtype=torch.float32, device=dev)
    for r in range(bs):
        n = st["lens"][r] + B
        t = torch.arange(n, device=dev)
        slots = st["table"][r][t // ps].long() * ps + t % ps
        k = st["k"][slots].float().permute(1, 2, 0)                      # Hkv, D, n
        v = st["v"][slots].float().permute(1, 0, 2)                      # Hkv, n, D
        q = st["q"][r * B:(r + 1) * B].float().view(B, Hkv, G, D)
        s = torch.matmul(q.permute(1, 0, 2, 3).reshape(Hkv, B * G, D), k) * scale
        if c["mode"] == VERIFY:
            i = torch.arange(B, device=dev).repeat_interleave(G)
            s = torch.where(t[None, :] <= st["lens"][r] + i[:, None], s, float("-inf"))
        m = s.amax(-1, keepdim=True)
        e = torch.exp(s - m)
        l = e.sum(-1, keepdim=True)
        o = torch.matmul(e, v) / l
        out[r * B:(r + 1) * B] = o.view(Hkv, B, G, D).permute(1, 0, 2, 3).reshape(B, Hq, D)
        lse[r * B:(r + 1) * B] = (m + torch.log(l)).view(Hkv, B, G).permute(1, 0, 2).reshape(B, Hq)
    return {"out": out, "lse": lse}


def _attn_own(st):
    import block_diffusion_speculative_attn_gb300 as bdsa
    c = st["case"]
    lse = torch.empty((c["bs"] * c["B"], c["Hq"]), dtype=torch.float32, device=st["q"].device)
    out = bdsa.block_attn_paged(st["q"], st["k"], st["v"], st["table"], st["seq"], B=c["B"],
                                page_size=c["ps"], scale=1.0 / math.sqrt(c["D"]), mode=c["mode"],
                                max_ctx_len=st["max_ctx"], num_pages=st["pages"], lse=lse,
                                workspace=st["workspace"], group_offsets=st["offs"],
                                prefix_lens=st["pre"])
    return {"out": out, "lse": lse}


def _attn_exact(c, seed):
    """Head by head over each group's stacked queries, prefix and rest joined by
    their log-sum-exp."""
    a = _attn_inputs(c, seed)
    bs, B, ps, Hq, Hkv, D = (c[k] for k in ("bs", "B", "ps", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    if bs * B * Hq * max(a["lens"]) * D * 4 > 5e12:
        return None
    dev = a["q"].device
    out = torch.empty((bs * B, Hq, D), dtype=torch.float64, device=dev)
    lse = torch.empty((bs * B, Hq), dtype=torch.float64, device=dev)
    offs = a["offs"].tolist()

    def part(rows, h, slots, mask=None):
        q = a["q"][rows, h * G:(h + 1) * G].double().reshape(-1, D) * D ** -0.5
        s = q @ a["k"][slots, h].double().T
        if mask is not None:
            s.masked_fill_(mask.repeat_interleave(G, 0), float("-inf"))
        ls = torch.logsumexp(s, -1)
        return torch.softmax(s, -1) @ a["v"][slots, h].double(), ls

    def slots_of(r, lo, hi):
        pages = a["table"][r].long()[:, None] * ps + torch.arange(ps, device=dev)
        return pages.reshape(-1)[lo:hi]

    for g in range(len(offs) - 1):
        P = a["pre_host"][g]
        grows = slice(offs[g] * B, offs[g + 1] * B)
        for h in range(Hkv):
            op, lp = part(grows, h, slots_of(offs[g], 0, P))
            for r in range(offs[g], offs[g + 1]):
                L = a["lens"][r]
                mask = None
                if c["mode"] == VERIFY:
                    mask = torch.arange(P, L + B, device=dev)[None] > \
                        L + torch.arange(B, device=dev)[:, None]
                rows = slice(r * B, (r + 1) * B)
                o, ls = part(rows, h, slots_of(r, P, L + B), mask)
                mine = slice((r - offs[g]) * B * G, (r - offs[g] + 1) * B * G)
                tot = torch.logaddexp(ls, lp[mine])
                o = o * torch.exp(ls - tot)[:, None] + \
                    op[mine] * torch.exp(lp[mine] - tot)[:, None]
                out[rows, h * G:(h + 1) * G] = o.view(B, G, D)
                lse[rows, h * G:(h + 1) * G] = tot.view(B, G)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ table
def _table_inputs(c, seed):
    """A pool in the middle of its life: owned pages scattered, the free ones in
    a ring that starts anywhere."""
    bs, ps = c["bs"], c["ps"]
    # the lengths are one draw of the case, dealt out in another order for each seed, so
    # that the number of new tokens is the case's
    fix = np.random.Generator(np.random.PCG64(bs * 31 + ps))
    rng = np.random.Generator(np.random.PCG64(seed * 7919 + 17))
    have = rng.permutation(fix.integers(c["have_lo"], c["have_hi"] + 1, bs))
    new = rng.permutation(fix.integers(c["new_lo"], c["new_hi"] + 1, bs))
    owned = (have + ps - 1) // ps
    need = (have + new + ps - 1) // ps
    pool = int(need.sum()) + int(rng.integers(1, 2 * bs + 2))
    width = (c["have_hi"] + c["new_hi"]) // ps + 2
    perm = rng.permutation(pool).astype(np.int32)
    table = np.full((bs, width), -1, np.int32)
    cols = np.arange(table.shape[1])
    table[cols[None] < owned[:, None]] = perm[:int(owned.sum())]
    free = perm[int(owned.sum()):]
    head = int(rng.integers(0, pool))
    ring = np.full(pool, -1, np.int32)
    ring[(head + np.arange(len(free))) % pool] = free
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
    return dict(seq=dev(have), new=dev(new), owned=dev(owned), table=dev(table), ring=dev(ring),
                state=dev([head, len(free)]), total=int(new.sum()))


def _table_plain(st):
    seq, new, owned = st["seq"].long(), st["new"].long(), st["owned"].long()
    table, ring, ps = st["table"], st["ring"].long(), st["case"]["ps"]
    pool = ring.numel()
    need = (seq + new + ps - 1) // ps
    grow = torch.clamp(need - owned, min=0)
    ends = torch.cumsum(grow, 0)
    col = torch.arange(table.shape[1], device=table.device)[None]
    pos = (st["state"][0].long() + (ends - grow)[:, None] + col - owned[:, None]) % pool
    fresh = (col >= owned[:, None]) & (col < need[:, None])
    table.copy_(torch.where(fresh, ring[pos], table.long()))
    cu = torch.zeros(seq.numel() + 1, dtype=torch.int64, device=table.device)
    cu[1:] = torch.cumsum(new, 0)
    t = torch.arange(st["total"], device=table.device)
    r = torch.searchsorted(cu, t, right=True) - 1
    p = seq[r] + t - cu[r]
    slot = table[r, p // ps].long() * ps + p % ps
    state = torch.stack([(st["state"][0].long() + ends[-1]) % pool,
                         st["state"][1].long() - ends[-1]])
    i32 = lambda x: x.to(torch.int32)
    return {"table": table, "owned": i32(torch.maximum(need, owned)), "state": i32(state),
            "cu": i32(cu), "slots": i32(slot), "positions": i32(p)}


def _table_own(st):
    import block_diffusion_speculative_attn_gb300 as bdsa
    o = bdsa.block_table_update(st["seq"], st["new"], st["owned"], st["table"], st["ring"],
                                st["state"], page_size=st["case"]["ps"],
                                total_tokens=st["total"])
    return {"table": st["table"], "owned": o["owned"], "state": o["free_state"],
            "cu": o["cu_tokens"], "slots": o["slot_map"], "positions": o["positions"]}


def _table_exact(c, seed):
    a = _table_inputs(c, seed)
    n = {k: v.cpu().numpy().astype(np.int64) for k, v in a.items() if torch.is_tensor(v)}
    ps, pool = c["ps"], len(n["ring"])
    head, count = (int(x) for x in n["state"])
    table, owned, cu, slots, poss = n["table"], n["owned"].copy(), [0], [], []
    for r in range(c["bs"]):
        want = -(-(n["seq"][r] + n["new"][r]) // ps)
        for j in range(owned[r], want):
            table[r, j] = n["ring"][head]
            head, count = (head + 1) % pool, count - 1
        owned[r] = max(owned[r], want)
        p = np.arange(n["seq"][r], n["seq"][r] + n["new"][r])
        slots.append(table[r, p // ps] * ps + p % ps)
        poss.append(p)
        cu.append(cu[-1] + len(p))
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()
    return {"table": dev(table), "owned": dev(owned), "state": dev([head, count]), "cu": dev(cu),
            "slots": dev(np.concatenate(slots)), "positions": dev(np.concatenate(poss))}


# ------------------------------------------------------------------ entry points
def prepare(case, seed):
    if case["op"] == "sample":
        lg, u, p = _sample_inputs(case, seed)
        return dict(case=case, logits=lg, u=u, params=p, probs=case["probs"])
    if case["op"] == "attn":
        st = dict(case=case, **_attn_inputs(case, seed))
        st["max_ctx"] = max(st["lens"])
        if own:
            import block_diffusion_speculative_attn_gb300 as bdsa
            n = bdsa.block_attn_prefix_workspace_bytes(
                case["bs"], case["B"], case["Hq"], case["Hkv"], case["D"], st["max_ctx"],
                len(st["pre_host"]))
            st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        return st
    return dict(case=case, **_table_inputs(case, seed))


_RUN = {"sample": (_sample_plain, _sample_own), "attn": (_attn_plain, _attn_own),
        "table": (_table_plain, _table_own)}


def run(state):
    return _RUN[state["case"]["op"]][1 if own else 0](state)


def exact(case, seed):
    if case["op"] == "sample":
        return _sample_exact(case, seed)
    if case["op"] == "attn":
        return _attn_exact(case, seed)
    return _table_exact(case, seed)


def work(case):
    """Bytes: each input read and each output written once.  Operations of the
    sampling: one exponential's worth (8) a logit; of the attention: both
    products over every visible key."""
    if case["op"] == "sample":
        n = case["bs"] * case["B"] * case["V"]
        e = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": n * (e + (4 if case["probs"] else 0)) + case["bs"] * case["B"] * 8,
                "flops": 8 * n}
    mid = lambda k: (case[k + "_lo"] + case[k + "_hi"]) / 2
    if case["op"] == "attn":
        rows = case["bs"] * case["B"] * case["Hq"]
        keys = mid("prefix") + mid("own") + case["B"]
        kv = 2 * 2 * case["Hkv"] * case["D"] * (
            min(case["groups"], case["bs"]) * mid("prefix") +
            case["bs"] * (mid("own") + case["B"]))
        return {"bytes": int(kv + rows * (4 * case["D"] + 4)),
                "flops": int(4 * rows * keys * case["D"])}
    tokens = case["bs"] * mid("new")
    pages = case["bs"] * mid("new") / case["ps"]
    return {"bytes": int(8 * tokens + 8 * pages + 20 * case["bs"]), "flops": int(4 * tokens)}
