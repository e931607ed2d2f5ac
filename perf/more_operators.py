"""Operators of a serving cache as measured work: prompts attended in chunks, and
the pages of the cache they live in.

Four kinds of cases, each with the plain form of its definition and the
framework's calls:

  attn     attention of a ragged batch of new tokens (chunks of prompts, single
           tokens) over a paged cache, token-causal or causal by blocks
  write    the new tokens' keys and values, as the projection leaves them, into
           their cache slots
  fork     rows of the block table continued from rows of the old one (beams
           reordered, prompts forked into samples, finished rows freed), full
           pages shared, partial last pages copied in every layer's caches
  compact  kept rows of a request moved to the front of their region in every
           layer's caches (a tree's accepted path, a window behind its sinks)

`listed()` names the cases, `draw(rng)` makes one more of the same ranges,
`prepare` makes a program's state, `run` is one pass, `exact` the definition in
64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_BIG = 1 << 40


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # two short chats in a small model: a call whose cost is its latency
        dict(name="attn_tiny", op="attn", bs=2, Hq=2, Hkv=1, D=64, ps=16, block=1, ones=0,
             new_lo=1, new_hi=8, ctx_lo=0, ctx_hi=96),
        # one decode step of 64 chats of any length: single tokens
        dict(name="attn_tokens", op="attn", bs=64, Hq=32, Hkv=8, D=128, ps=16, block=1, ones=64,
             new_lo=1, new_hi=1, ctx_lo=512, ctx_hi=8192),
        # continuous batching: 44 chats decode while four prompts get a chunk each
        dict(name="attn_mixed", op="attn", bs=48, Hq=16, Hkv=4, D=128, ps=32, block=1, ones=44,
             new_lo=128, new_hi=512, ctx_lo=256, ctx_hi=4096),
        # admission of 24 ragged prompts
        dict(name="attn_prompts", op="attn", bs=24, Hq=32, Hkv=8, D=128, ps=64, block=1, ones=0,
             new_lo=17, new_hi=2048, ctx_lo=0, ctx_hi=0),
        # prompts of a block-diffusion model: blocks of 32 see themselves whole
        dict(name="attn_blocks", op="attn", bs=8, Hq=16, Hkv=4, D=128, ps=32, block=32, ones=0,
             new_lo=512, new_hi=1024, ctx_lo=1024, ctx_hi=8192),
        # the last chunk of a long document's prompt
        dict(name="attn_long", op="attn", bs=1, Hq=32, Hkv=8, D=128, ps=64, block=1, ones=0,
             new_lo=4096, new_hi=4096, ctx_lo=28672, ctx_hi=28672),
        # a verify step's keys and values in one layer
        dict(name="write_step", op="write", T=512, Hq=32, Hkv=8, D=128, ps=64, pages=1024),
        # a ragged chunk of prompts in one layer
        dict(name="write_prompts", op="write", T=49157, Hq=32, Hkv=8, D=128, ps=16, pages=4096),
        # a step of beam search: 8 prompts with 8 beams, in a small drafter's layers
        dict(name="fork_beams", op="fork", kind="beams", groups=8, width=8, ps=16, layers=5,
             Hkv=8, D=128, len_lo=200, len_hi=1500),
        # 32 prompts answered 8 times each, forked after their prefill
        dict(name="fork_samples", op="fork", kind="samples", groups=32, width=8, ps=64, layers=16,
             Hkv=8, D=128, len_lo=100, len_hi=1500),
        # a verified tree of 481 nodes: its accepted path stays
        dict(name="compact_tree", op="compact", kind="tree", bs=32, ps=64, layers=16, Hkv=8,
             D=128, nodes=481, keep_lo=1, keep_hi=16, ctx_lo=64, ctx_hi=512),
        # long chats cut to their first tokens and a window of their last ones
        dict(name="compact_window", op="compact", kind="window", bs=16, ps=16, layers=8, Hkv=8,
             D=128, nodes=4001, keep_lo=700, keep_hi=1300, ctx_lo=0, ctx_hi=0),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "write", "fork", "compact"])
    if op == "attn":
        Hq, Hkv = rng.choice([(2, 1), (16, 4), (32, 8), (24, 8), (16, 16), (12, 1)])
        bs = _logu(rng, 1, 96)
        kind = rng.choice(["tokens", "mixed", "prompts", "chunks"])
        ones = {"tokens": bs, "mixed": bs - max(1, bs // 12)}.get(kind, 0)
        # at most half of the rows x keys of the largest listed case
        cap = 32 * 4096 * 16384 // Hq
        many = max(1, bs - ones)
        if kind == "tokens":
            new_hi, ctx_hi = 1, _logu(rng, 64, max(65, min(16384, cap // bs)))
        elif kind == "prompts":
            new_hi, ctx_hi = _logu(rng, 16, max(17, min(4096, int(math.sqrt(cap / many))))), 0
        else:
            new_hi = _logu(rng, 16, max(17, min(2048, int(math.sqrt(cap / many)) // 2)))
            ctx_hi = _logu(rng, 16, max(17, min(16384, cap // (many * new_hi + bs))))
        return dict(op=op, bs=bs, Hq=Hq, Hkv=Hkv, D=rng.choice([64, 128, 128]),
                    ps=rng.choice([8, 16, 32, 64, 128]), block=rng.choice([1, 1, 1, 8, 32, 100]),
                    ones=ones, new_lo=min(new_hi, rng.choice([1, 7, 16])), new_hi=new_hi,
                    ctx_lo=ctx_hi // 8, ctx_hi=ctx_hi)
    Hkv, D, ps = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([8, 16, 32, 64, 128])
    if op == "write":
        T = _logu(rng, 1, 49157)
        return dict(op=op, T=T, Hq=Hkv * rng.choice([1, 3, 4, 8]), Hkv=Hkv, D=D, ps=ps,
                    pages=T // ps + _logu(rng, 1, 400))
    if op == "fork":
        kind = rng.choice(["beams", "samples"])
        groups, width = _logu(rng, 1, 32), rng.choice([2, 3, 4, 8])
        return dict(op=op, kind=kind, groups=groups, width=width, ps=ps,
                    layers=_logu(rng, 1, 16), Hkv=Hkv, D=D, len_lo=rng.choice([1, 40, 100]),
                    len_hi=_logu(rng, 101, 1500))
    kind = rng.choice(["tree", "window"])
    if kind == "tree":
        nodes = _logu(rng, 40, 481)
        return dict(op=op, kind=kind, bs=_logu(rng, 1, 32), ps=ps, layers=_logu(rng, 1, 16),
                    Hkv=Hkv, D=D, nodes=nodes, keep_lo=1, keep_hi=rng.randint(2, 16),
                    ctx_lo=0, ctx_hi=_logu(rng, 16, 500))
    nodes = _logu(rng, 200, 4001)
    return dict(op=op, kind=kind, bs=_logu(rng, 1, 16), ps=ps, layers=_logu(rng, 1, 8), Hkv=Hkv,
                D=D, nodes=nodes, keep_lo=nodes // 8, keep_hi=nodes // 3, ctx_lo=0, ctx_hi=0)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _gen(seed, k):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + k)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


# ------------------------------------------------------------------ attn
def _attn_lens(c):
    """New tokens and context of every request: one draw of the case."""
    fix = np.random.Generator(np.random.PCG64(c["bs"] * 31 + c["new_hi"] * 7 + c["ctx_hi"]))
    new = np.ones(c["bs"], np.int64)
    many = c["bs"] - c["ones"]
    new[:many] = fix.integers(c["new_lo"], c["new_hi"] + 1, many)
    return new, fix.integers(c["ctx_lo"], c["ctx_hi"] + 1, c["bs"])


def _attn_inputs(c, seed):
    rng = np.random.Generator(np.random.PCG64(seed * 104729 + 5))
    new, ctx = _attn_lens(c)
    deal = rng.permutation(c["bs"])  # another order of the same lengths
    new, ctx = new[deal], ctx[deal]
    ps = c["ps"]
    need = (new + ctx + ps - 1) // ps
    total = int(need.sum()) + 3
    perm = rng.permutation(total).astype(np.int32)
    width = int(need.max()) + 1
    table = np.full((c["bs"], width), -1, np.int32)
    table[np.arange(width)[None] < need[:, None]] = perm[:int(need.sum())]
    g = _gen(seed, 13)
    cu = np.concatenate([[0], np.cumsum(new)])
    return dict(qkv=_randn(g, int(cu[-1]), c["Hq"] + 2 * c["Hkv"], c["D"]),
                k=_randn(g, total * ps, c["Hkv"], c["D"]),
                v=_randn(g, total * ps, c["Hkv"], c["D"]), table=_dev(table), seq=_dev(ctx),
                cu=_dev(cu), new=new.tolist(), ctx=ctx.tolist(), starts=cu.tolist())


def _attn_groups(c, a):
    """Requests of like lengths together, so that padding them to the longest
    wastes little: their numbers and the padded sizes."""
    order = sorted(range(c["bs"]), key=lambda r: (-a["new"][r], -a["ctx"][r]))
    groups, cur, n, m = [], [], 0, 0
    for r in order:
        n2, m2 = max(n, a["new"][r]), max(m, a["ctx"][r] + a["new"][r])
        if cur and ((len(cur) + 1) * n2 * m2 * c["Hq"] > 1 << 29 or 2 * a["new"][r] < n2):
            groups.append((torch.tensor(cur, device="cuda"), n, m))
            cur, n2, m2 = [], a["new"][r], a["ctx"][r] + a["new"][r]
        cur.append(r)
        n, m = n2, m2
    groups.append((torch.tensor(cur, device="cuda"), n, m))
    return groups


def _attn_plain(st):
    """Padded groups of requests: all scores, the mask, a softmax, the sums."""
    c, dev = st["case"], st["qkv"].device
    Hq, Hkv, D, ps, blk = (c[k] for k in ("Hq", "Hkv", "D", "ps", "block"))
    T, G = st["qkv"].shape[0], Hq // Hkv
    out = torch.empty((T + 1, Hq, D), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((T + 1, Hq), dtype=torch.float32, device=dev)
    for rows, n, m in st["groups"]:
        R = rows.numel()
        i, t = torch.arange(n, device=dev), torch.arange(m, device=dev)
        L = st["seq"][rows].long()[:, None]
        first = st["cu"][rows].long()[:, None]
        count = st["cu"][rows + 1].long()[:, None] - first
        tok = torch.where(i < count, first + i, T)
        seen = torch.minimum(L + count, ((L + i) // blk + 1) * blk)           # R, n
        page = st["table"][rows][:, t // ps].long().clamp(min=0)
        slot = page * ps + t % ps                                              # R, m
        k = st["k"][slot].float().permute(0, 2, 3, 1)                          # R, Hkv, D, m
        v = st["v"][slot].float().permute(0, 2, 1, 3)                          # R, Hkv, m, D
        q = st["qkv"][tok.clamp(max=T - 1), :Hq].float().view(R, n, Hkv, G, D)
        s = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(R, Hkv, n * G, D), k)
        s.mul_(1.0 / math.sqrt(D))
        hide = t[None, None, :] >= seen[:, :, None]                            # R, n, m
        s.view(R, Hkv, n, G, m).masked_fill_(hide[:, None, :, None, :], float("-inf"))
        top = s.amax(-1, keepdim=True)
        s.sub_(top).exp_()
        l = s.sum(-1, keepdim=True)
        o = torch.matmul(s, v) / l
        out[tok] = o.view(R, Hkv, n, G, D).permute(0, 2, 1, 3, 4).reshape(R, n, Hq, D).bfloat16()
        lse[tok] = (top + torch.log(l)).view(R, Hkv, n, G).permute(0, 2, 1, 3).reshape(R, n, Hq)
    return {"out": out[:T], "lse": lse[:T]}


def _attn_own(st):
    import block_diffusion_speculative_attn_gb300 as bdsa
    c, qkv = st["case"], st["qkv"]
    lse = torch.empty((qkv.shape[0], c["Hq"]), dtype=torch.float32, device=qkv.device)
    out = bdsa.chunk_attn_paged(qkv[:, :c["Hq"]], st["k"], st["v"], st["table"], st["seq"],
                                st["cu"], page_size=c["ps"], scale=1.0 / math.sqrt(c["D"]),
                                mask_block=c["block"], lse=lse)
    return {"out": out, "lse": lse}


def _attn_exact(c, seed):
    """Request by request and head by head, the softmax as exp(s - logsumexp)."""
    a = _attn_inputs(c, seed)
    if _attn_work(c)["flops"] > 5e12:
        return None
    Hq, Hkv, D, ps, blk = (c[k] for k in ("Hq", "Hkv", "D", "ps", "block"))
    G, dev, T = Hq // Hkv, a["qkv"].device, a["qkv"].shape[0]
    out = torch.empty((T, Hq, D), dtype=torch.float64, device=dev)
    lse = torch.empty((T, Hq), dtype=torch.float64, device=dev)
    for r in range(c["bs"]):
        L, n, at = a["ctx"][r], a["new"][r], a["starts"][r]
        pages = a["table"][r].long()[:-(-(L + n) // ps), None] * ps
        slots = (pages + torch.arange(ps, device=dev)).reshape(-1)[:L + n]
        pos = torch.arange(L, L + n, device=dev)
        last = (pos - pos % blk + blk - 1).clamp(max=L + n - 1)
        bias = torch.zeros((n, L + n), dtype=torch.float64, device=dev)
        bias[torch.arange(L + n, device=dev)[None] > last[:, None]] = float("-inf")
        for j in range(Hq):
            s = a["qkv"][at:at + n, j].double() @ a["k"][slots, j // G].double().T
            s = s * (D ** -0.5) + bias
            ls = torch.logsumexp(s, 1)
            out[at:at + n, j] = torch.exp(s - ls[:, None]) @ a["v"][slots, j // G].double()
            lse[at:at + n, j] = ls
    return {"out": out, "lse": lse}


def _attn_work(c):
    new, ctx = _attn_lens(c)
    pairs = float((new * ctx + new * (new + 1) / 2).sum())
    kv = 2 * 2 * c["Hkv"] * c["D"] * float((new + ctx).sum())
    return {"bytes": int(kv + new.sum() * c["Hq"] * (4 * c["D"] + 4)),
            "flops": int(4 * c["Hq"] * c["D"] * pairs)}


# ------------------------------------------------------------------ write
def _write_inputs(c, seed):
    rng = np.random.Generator(np.random.PCG64(seed * 104729 + 7))
    ps, T = c["ps"], c["T"]
    pages = rng.permutation(c["pages"])[:-(-T // ps)]
    slots = (pages[:, None] * ps + np.arange(ps)).reshape(-1)[:T]
    g = _gen(seed, 17)
    shape = (c["pages"] * ps, c["Hkv"], c["D"])
    return dict(qkv=_randn(g, T, c["Hq"] + 2 * c["Hkv"], c["D"]), slots=_dev(slots),
                k=_randn(g, *shape), v=_randn(g, *shape))


def _write_plain(st):
    Hq, Hkv = st["case"]["Hq"], st["case"]["Hkv"]
    at = st["slots"].long()
    st["k"][at] = st["qkv"][:, Hq:Hq + Hkv]
    st["v"][at] = st["qkv"][:, Hq + Hkv:]
    return {"k": st["k"], "v": st["v"]}


def _write_own(st):
    import block_diffusion_speculative_attn_gb300 as bdsa
    Hq, Hkv = st["case"]["Hq"], st["case"]["Hkv"]
    bdsa.cache_write(st["qkv"][:, Hq:Hq + Hkv], st["qkv"][:, Hq + Hkv:], st["slots"], st["k"],
                     st["v"])
    return {"k": st["k"], "v": st["v"]}


def _write_exact(c, seed):
    a = _write_inputs(c, seed)
    source = torch.full((a["k"].shape[0],), -1, dtype=torch.int64, device="cuda")
    source.scatter_(0, a["slots"].long(), torch.arange(c["T"], device="cuda"))
    hit = (source >= 0)[:, None, None]
    new = a["qkv"].index_select(0, source.clamp(min=0))
    return {"k": torch.where(hit, new[:, c["Hq"]:c["Hq"] + c["Hkv"]], a["k"]),
            "v": torch.where(hit, new[:, c["Hq"] + c["Hkv"]:], a["v"])}


# ------------------------------------------------------------------ fork
def _fork_inputs(c, seed):
    """A block table before the fork, the rows to make of it, and a free ring that
    starts anywhere."""
    P, w, ps = c["groups"], c["width"], c["ps"]
    fix = np.random.Generator(np.random.PCG64(P * 31 + w * 7 + ps))
    rng = np.random.Generator(np.random.PCG64(seed * 104729 + 11))
    # (lengths, reserved pages and the pool are the case's, whatever the seed)
    lens = rng.permutation(fix.integers(c["len_lo"], c["len_hi"] + 1, P))
    extra = rng.permutation(fix.integers(0, 2, P))
    rows, W = P * w, int(lens.max()) // ps + 3
    page, table, owned = 0, np.full((rows, W), -1, np.int64), np.zeros(rows, np.int64)
    parent, keep = np.zeros(rows, np.int64), np.zeros(rows, np.int64)
    for g in range(P):
        need = -(-int(lens[g]) // ps)
        if c["kind"] == "beams":
            # row g * w + b; the beams part ways in the last two of their pages, some
            # beams live on several times, one group in eight is done
            for j in range(need):
                ways = 1 if j < need - 2 else max(1, w // 2) if j < need - 1 else w
                table[g * w:(g + 1) * w, j] = page + np.arange(w) * ways // w
                page += ways
            at = slice(g * w, (g + 1) * w)
            owned[at] = need
            parent[at] = g * w + rng.integers(0, w, w) if g % 8 != 7 else -1
            keep[at] = lens[g] if g % 8 != 7 else 0
        else:
            # rows below P are the prompts, the others are empty; a prompt may
            # have a page more than its tokens need
            owned[g] = need + int(extra[g])
            table[g, :owned[g]] = page + np.arange(owned[g])
            page += int(owned[g])
            parent[g::P] = g
            keep[g::P] = lens[g]
    pool = page + rows + int(fix.integers(1, 9))
    ids = rng.permutation(pool)
    table = np.where(table >= 0, ids[np.maximum(table, 0)], -1)
    head = int(rng.integers(0, pool))
    ring = np.full(pool, -1, np.int64)
    free = ids[page:]
    ring[(head + np.arange(len(free))) % pool] = free
    caches = _randn(_gen(seed, 19), 2 * c["layers"], pool * ps, c["Hkv"], c["D"])
    return dict(table=_dev(table), owned=_dev(owned), parent=_dev(parent), keep=_dev(keep),
                ring=_dev(ring), state=_dev([head, len(free)]), caches=caches)


def _fork_plain(st):
    """Reference counts by scattered sums, the choices as masks over the table."""
    ps, dev = st["case"]["ps"], st["table"].device
    table, ring, n_pages = st["table"].long(), st["ring"].long(), st["ring"].numel()
    parent, head, count = st["parent"].long(), st["state"][0].long(), st["state"][1].long()
    rows, W = parent.numel(), table.shape[1]
    col, row = torch.arange(W, device=dev), torch.arange(rows, device=dev)
    none = n_pages  # a page number for entries without a page
    live = col < st["owned"].long()[:, None]
    page = torch.where(live, table, none)
    flat = torch.arange(table.numel(), device=dev)
    first = torch.full((n_pages + 1,), _BIG, device=dev).scatter_reduce(
        0, page.reshape(-1), flat, "amin")
    n = torch.where(parent >= 0, st["keep"].long(), 0)
    whole, tail = n // ps, n % ps
    new = table[parent.clamp(min=0)]
    kept = torch.where(col < whole[:, None], new, none)
    refs = torch.zeros(n_pages + 1, dtype=torch.int64, device=dev).scatter_add(
        0, kept.reshape(-1), torch.ones_like(kept).reshape(-1))
    last = torch.where(tail > 0, new.gather(1, whole.clamp(max=W - 1)[:, None])[:, 0], none)
    heir = torch.full((n_pages + 1,), _BIG, device=dev).scatter_reduce(0, last, row, "amin")
    copy = (tail > 0) & ((refs[last] > 0) | (heir[last] != row))
    refs = refs.scatter_add(0, torch.where((tail > 0) & ~copy, last, none), torch.ones_like(row))
    refs[none] = 0
    fresh = ring[(head + torch.cumsum(copy, 0) - copy.long()) % n_pages]
    end = torch.where(copy, fresh, last)
    table_out = torch.where(col < whole[:, None], new, torch.where(
        (col == whole[:, None]) & (tail > 0)[:, None], end[:, None], -1))
    gone = (live & (refs[page] == 0)).reshape(-1) & (first[page.reshape(-1)] == flat)
    cell = torch.where(gone, (head + count + torch.cumsum(gone, 0) - 1) % n_pages, n_pages)
    st["ring"].copy_(torch.cat([ring, ring[:1]]).scatter_(0, cell, table.reshape(-1))[:n_pages])
    twice = (table_out >= 0) & (refs[table_out.clamp(min=0)] > 1)
    state = torch.stack([(head + copy.sum()) % n_pages, count - copy.sum() + gone.sum()])
    # rows of the pages that are copied; the others copy a row of theirs, or of the
    # first page in use, onto itself
    j = torch.arange(ps, device=dev)
    moves = copy[:, None] & (j < tail[:, None])
    page0 = torch.where(copy, last, table[0, 0])
    src = page0[:, None] * ps + j
    dst = torch.where(moves, fresh[:, None] * ps + j, src)
    caches = st["caches"]
    caches[:, dst.reshape(-1)] = caches[:, src.reshape(-1)]
    i32 = lambda x: x.to(torch.int32)  # noqa: E731
    return {"table": i32(table_out), "owned": i32(whole + (tail > 0)),
            "shared": i32(torch.where(twice, col + 1, 0).amax(1)), "state": i32(state),
            "ring": st["ring"], "copy_src": i32(torch.where(copy, last, -1)),
            "copy_dst": i32(torch.where(copy, fresh, -1)),
            "copy_len": i32(torch.where(copy, tail, 0)), "caches": caches}


def _fork_own(st):
    import block_diffusion_speculative_attn_gb300 as bdsa
    ps = st["case"]["ps"]
    f = bdsa.cache_fork(st["parent"], st["keep"], st["table"], st["owned"], st["ring"],
                        st["state"], page_size=ps)
    bdsa.cache_copy(st["caches"], f["copy_src"], f["copy_dst"], f["copy_len"], page_size=ps)
    return {"table": f["block_table"], "owned": f["owned"], "shared": f["shared"],
            "state": f["free_state"], "ring": st["ring"], "copy_src": f["copy_src"],
            "copy_dst": f["copy_dst"], "copy_len": f["copy_len"], "caches": st["caches"]}


def _fork_exact(c, seed):
    """Row by row, with a list of users for every page."""
    a = _fork_inputs(c, seed)
    n = {k: v.cpu().numpy().astype(np.int64) for k, v in a.items() if k != "caches"}
    ps, pool, rows = c["ps"], len(n["ring"]), len(n["parent"])
    table = np.full_like(n["table"], -1)
    owned, shared = np.zeros(rows, np.int64), np.zeros(rows, np.int64)
    whole_users, part_users, users = {}, {}, {}
    for r in range(rows):
        p, t = n["parent"][r], n["keep"][r]
        if p < 0:
            continue
        table[r, :t // ps] = n["table"][p, :t // ps]
        owned[r] = -(-t // ps)
        for x in table[r, :t // ps]:
            whole_users.setdefault(x, []).append(r)
        if t % ps:
            part_users.setdefault(n["table"][p, t // ps], []).append(r)
    head, count = (int(x) for x in n["state"])
    src, dst, ln = (np.full(rows, x, np.int64) for x in (-1, -1, 0))
    caches = a["caches"].clone()
    for r in range(rows):
        t = n["keep"][r]
        if n["parent"][r] < 0 or t % ps == 0:
            continue
        x = n["table"][n["parent"][r], t // ps]
        if x in whole_users or part_users[x][0] != r:
            src[r], dst[r], ln[r] = x, n["ring"][head], t % ps
            caches[:, dst[r] * ps:dst[r] * ps + ln[r]] = \
                a["caches"][:, x * ps:x * ps + ln[r]]
            head, count, x = (head + 1) % pool, count - 1, dst[r]
        table[r, t // ps] = x
    for r in range(rows):
        for x in table[r, :owned[r]]:
            users.setdefault(x, []).append(r)
    for r in range(rows):
        for j in range(owned[r]):
            if len(users[table[r, j]]) > 1:
                shared[r] = j + 1
    ring = n["ring"].copy()
    seen = set(users)
    for r in range(n["table"].shape[0]):
        for x in n["table"][r, :n["owned"][r]]:
            if x not in seen:
                seen.add(x)
                ring[(head + count) % pool] = x
                count += 1
    return {"table": _dev(table), "owned": _dev(owned), "shared": _dev(shared),
            "state": _dev([head, count]), "ring": _dev(ring), "copy_src": _dev(src),
            "copy_dst": _dev(dst), "copy_len": _dev(ln), "caches": caches}


def _fork_work(c):
    P, w, ps = c["groups"], c["width"], c["ps"]
    lens = np.random.Generator(np.random.PCG64(P * 31 + w * 7 + ps)).integers(
        c["len_lo"], c["len_hi"] + 1, P)
    # of w picks among w beams, w (1 - 1/w)^w are not a first one
    copies = w - 1 if c["kind"] == "samples" else w * (1 - 1 / w) ** w * (P - P // 8) / P
    moved = 2 * float((lens % ps).sum()) * copies
    ids = float((-(-lens // ps)).sum()) * (w if c["kind"] == "beams" else 1) + \
        float((-(-lens // ps)).sum()) * w
    return {"bytes": int(moved * c["layers"] * 2 * c["Hkv"] * c["D"] * 2 + 4 * ids + 40 * P * w),
            "flops": 0}


# ------------------------------------------------------------------ compact
def _keep_lens(c):
    fix = np.random.Generator(np.random.PCG64(c["bs"] * 31 + c["nodes"]))
    return fix.integers(c["keep_lo"], c["keep_hi"] + 1, c["bs"])


def _compact_inputs(c, seed):
    """Kept rows behind the place that they move to, so that a second pass moves
    the same rows again."""
    rng = np.random.Generator(np.random.PCG64(seed * 104729 + 17))
    bs, ps, nodes = c["bs"], c["ps"], c["nodes"]
    keep = rng.permutation(_keep_lens(c))
    path = np.full((bs, nodes if c["kind"] == "tree" else int(keep.max())), -1, np.int64)
    for r, m in enumerate(keep):
        if c["kind"] == "tree":
            path[r, 0] = 0
            path[r, 1:m] = m + np.sort(rng.choice(nodes - m, m - 1, replace=False))
        else:
            sinks = min(4, int(m))
            path[r, :sinks] = np.arange(sinks)
            path[r, sinks:m] = nodes - (m - sinks) + np.arange(m - sinks)
    ctx = rng.permutation(np.random.Generator(np.random.PCG64(bs)).integers(
        c["ctx_lo"], c["ctx_hi"] + 1, bs))
    need = (ctx + nodes + ps - 1) // ps
    total = int(need.sum()) + 2
    table = np.full((bs, int(need.max()) + 1), -1, np.int64)
    table[np.arange(table.shape[1])[None] < need[:, None]] = \
        rng.permutation(total)[:int(need.sum())]
    caches = _randn(_gen(seed, 23), 2 * c["layers"], total * ps, c["Hkv"], c["D"])
    return dict(path=_dev(path), seq=_dev(ctx), table=_dev(table), caches=caches)


def _compact_plain(st):
    ps, path, caches = st["case"]["ps"], st["path"].long(), st["caches"]
    place = torch.arange(path.shape[1], device=path.device).expand_as(path)
    L = st["seq"].long()[:, None]
    # (entries past the path move the first kept row, which stays where it is)
    old = L + torch.where(path >= 0, path, path[:, :1])
    new = L + torch.where(path >= 0, place, path[:, :1])
    slot = lambda t: st["table"].long().gather(1, t // ps) * ps + t % ps  # noqa: E731
    caches[:, slot(new).reshape(-1)] = caches[:, slot(old).reshape(-1)]
    return {"caches": caches}


def _compact_own(st):
    import block_diffusion_speculative_attn_gb300 as bdsa
    bdsa.cache_compact(st["caches"], st["table"], st["seq"], st["path"],
                       page_size=st["case"]["ps"])
    return {"caches": st["caches"]}


def _compact_exact(c, seed):
    a = _compact_inputs(c, seed)
    caches, ps = a["caches"].clone(), c["ps"]
    path, table, seq = (a[k].cpu().numpy() for k in ("path", "table", "seq"))
    for r in range(c["bs"]):
        where = lambda t: torch.from_numpy(  # noqa: E731
            table[r, t // ps].astype(np.int64) * ps + t % ps).cuda()
        kept = path[r][path[r] >= 0]
        rows = a["caches"].index_select(1, where(seq[r] + kept))
        caches.index_copy_(1, where(seq[r] + np.arange(len(kept))), rows)
    return {"caches": caches}


# ------------------------------------------------------------------ entry points
def prepare(case, seed):
    if case["op"] == "attn":
        a = _attn_inputs(case, seed)
        return dict(case=case, groups=_attn_groups(case, a), **a)
    make = {"write": _write_inputs, "fork": _fork_inputs, "compact": _compact_inputs}
    return dict(case=case, **make[case["op"]](case, seed))


_RUN = {"attn": (_attn_plain, _attn_own), "write": (_write_plain, _write_own),
        "fork": (_fork_plain, _fork_own), "compact": (_compact_plain, _compact_own)}


def run(state):
    return _RUN[state["case"]["op"]][1 if own else 0](state)


def exact(case, seed):
    return {"attn": _attn_exact, "write": _write_exact, "fork": _fork_exact,
            "compact": _compact_exact}[case["op"]](case, seed)


def work(case):
    """Bytes: each input read and each output written once (of caches, the rows that
    move).  Operations of the attention: both products over every token's causal
    keys."""
    if case["op"] == "attn":
        return _attn_work(case)
    if case["op"] == "write":
        return {"bytes": case["T"] * (8 * case["Hkv"] * case["D"] + 4), "flops": 0}
    if case["op"] == "fork":
        return _fork_work(case)
    stay = 1 if case["kind"] == "tree" else 4  # rows that are in their place already
    rows = float(np.maximum(_keep_lens(case) - stay, 0).sum())
    return {"bytes": int(rows * (case["layers"] * 8 * case["Hkv"] * case["D"] + 4)) + 8,
            "flops": 0}
