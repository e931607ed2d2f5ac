"""GPU parity of bdsa_chunk_attn_paged (ragged new tokens over the paged cache)
against the fp64 oracle.

Tolerance, row by row.  The kernel rounds each weight p to bf16 (half a step:
2^-8 of it) before the PV product, so out moves by at most 2^-8 sum p|v| / sum p
(`weight`), and rounds out itself once (2^-8 |out|).  What fp32 adds (scores of up
to 128 products, exponentials, sums, joins) is below 2^-12 of the weight.  The
log-sum-exp has no such rounding: a score's error is at most D 2^-24 sum |q k| scale,
under 1e-4 for these inputs."""
import numpy as np
import pytest
import torch

import block_diffusion_speculative_attn_gb300 as bdsa
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Case:
    """Ragged requests; cache slots that nobody's keys are in hold NaN."""

    def __init__(self, new, ctx, Hq=4, Hkv=2, D=64, ps=16, mb=1, seed=0, spread=1.0, width=None,
                 room=0):
        rng = np.random.default_rng(seed)
        self.new, self.ctx = np.asarray(new), np.asarray(ctx, np.int64)
        self.bs, self.Hq, self.Hkv, self.D, self.ps, self.mb = len(new), Hq, Hkv, D, ps, mb
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.T = int(self.cu[-1]) + room
        need = (self.new + np.maximum(self.ctx, 0) + ps - 1) // ps
        total = int(need.sum()) + 2
        perm = rng.permutation(total).astype(np.int32)
        self.table = np.full((self.bs, width or int(need.max()) + 1), -1, np.int32)
        at = 0
        for r in range(self.bs):
            self.table[r, :need[r]] = perm[at:at + need[r]]
            at += int(need[r])
        g = torch.Generator().manual_seed(seed + 1)
        bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
        self.q = bf(self.T, Hq, D) * spread
        self.k, self.v = bf(total * ps, Hkv, D), bf(total * ps, Hkv, D)
        used = np.zeros(total * ps, bool)
        for r in range(self.bs):
            t = np.arange(self.ctx[r] + self.new[r])
            used[self.table[r, t // ps].astype(np.int64) * ps + t % ps] = True
        self.k[torch.from_numpy(~used)] = float("nan")
        self.v[torch.from_numpy(~used)] = float("nan")
        self.scale = 1.0 / np.sqrt(D)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def dev(self):
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)  # noqa: E731
        return dict(q=self.q.to(DEV), k=self.k.to(DEV), v=self.v.to(DEV), table=i32(self.table),
                    ctx=i32(self.ctx), cu=i32(self.cu))

    def run(self, d=None, **kw):
        d = d or self.dev()
        lse = torch.full((self.T, self.Hq), 7.0, dtype=torch.float32, device=DEV)
        out = torch.full((self.T, self.Hq, self.D), 7.0, dtype=torch.bfloat16, device=DEV)
        bdsa.chunk_attn_paged(d["q"], d["k"], d["v"], d["table"], d["ctx"], d["cu"],
                              page_size=self.ps, scale=self.scale, mask_block=self.mb, out=out,
                              lse=lse, dev_status=self.status, **kw)
        torch.cuda.synchronize()
        return out.double().cpu().numpy(), lse.double().cpu().numpy()

    def want(self):
        return oracle.chunk_attn(self.q.double().numpy(), self.k.double().numpy(),
                                 self.v.double().numpy(), self.table, self.ctx, self.cu, self.ps,
                                 self.scale, self.mb)

    def check(self, got=None, status=0, **kw):
        out, lse = got or self.run(**kw)
        ref, ref_lse, weight = self.want()
        mine = ~np.isnan(ref_lse[:, 0])
        assert (out[~mine] == 7.0).all() and (lse[~mine] == 7.0).all()
        tol = 2.0 ** -8 * (np.abs(ref) + weight) + 2.0 ** -12 * weight
        err = np.abs(out[mine] - ref[mine])
        assert (err <= tol[mine] * (1 + 2.0 ** -8)).all(), np.nanmax(err - tol[mine])
        dead = np.isneginf(ref_lse[mine])
        assert (np.isneginf(lse[mine]) == dead).all()
        assert np.abs(lse[mine][~dead] - ref_lse[mine][~dead]).max(initial=0.0) < 1e-3
        assert int(self.status) == status


SHAPES = [
    # new, ctx
    ([1], [0]),
    ([1], [1]),
    ([5, 1, 0, 3], [0, 40, 9, 17]),
    ([1] * 9, [0, 1, 15, 16, 127, 128, 129, 400, 31]),
    ([127, 128, 129], [0, 0, 0]),
    ([300], [0]),
    ([1, 200, 0, 1, 64], [500, 77, 3, 0, 129]),
    ([33, 2], [700, 254]),
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [(4, 2), (2, 2), (6, 2), (16, 1), (7, 1), (8, 1)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_ragged(shape, heads, D):
    new, ctx = SHAPES[shape]
    Case(new, ctx, *heads, D=D, ps=[8, 16, 32, 64, 128][shape % 5], seed=shape).check()


@pytest.mark.parametrize("sms", [1, 2, 3, 29, 700])
@pytest.mark.parametrize("mb", [1, 32])
def test_cuts(sms, mb):
    """The same result, however many CTAs cut the work."""
    Case([1, 90, 300, 1], [1500, 700, 256, 4000], Hq=8, Hkv=2, D=128, ps=32, mb=mb,
         seed=3).check(sms=sms)


@pytest.mark.parametrize("mb", [2, 7, 8, 32, 100, 128, 129, 1000, 1 << 30])
@pytest.mark.parametrize("D", [64, 128])
def test_blocks(mb, D):
    Case([37, 1, 260, 128], [0, 63, 130, 31], Hq=4, Hkv=1, D=D, ps=16, mb=mb, seed=mb % 97).check()


@pytest.mark.parametrize("G", [1, 3, 5, 12, 48, 64, 100, 128])
def test_group_sizes(G):
    Case([70, 1, 9], [60, 300, 0], Hq=2 * G, Hkv=2, D=64, ps=8, seed=G).check()


@pytest.mark.parametrize("spread", [30.0, 1e-3])
def test_score_ranges(spread):
    Case([200, 3], [300, 900], spread=spread, D=128, seed=11).check()


def test_rows_behind_the_last_sequence_stay():
    c = Case([5, 40, 0], [3, 100, 7], D=128, room=37)
    c.q[45:] = float("nan")
    c.check()


def test_nothing_to_do():
    Case([0, 0], [5, 0], room=4).check()


def test_strided_queries():
    """q as a slice of a fused projection, heads dense, any row pitch."""
    c = Case([70, 1, 130], [20, 500, 0], Hq=8, Hkv=2, D=128, ps=64, seed=5)
    d = c.dev()
    wide = torch.full((c.T, 8 + 5, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, 2:10] = d["q"]
    d["q"] = wide[:, 2:10]
    c.check(c.run(d))


@pytest.mark.parametrize("bad", [-1, 10 ** 6])
@pytest.mark.parametrize("sms", [0, 700])
def test_bad_pages(bad, sms):
    """Rows that see a key on the page get zeros, the others their attention."""
    c = Case([200, 150, 1], [70, 600, 900], Hq=8, Hkv=2, D=128, ps=16, seed=7)
    c.table[0, 150 // 16] = bad       # seen from position 144 on
    c.table[2, 3] = bad
    c.check(status=16, sms=sms)


def test_bad_lengths():
    c = Case([20, 30, 1, 25], [40, 10, 70, 33], D=128, ps=16, seed=8, width=6)
    c.ctx[1] = -1
    c.ctx[3] = 96                     # 96 + 25 keys, the row holds 96
    c.check(status=16)
    c = Case([3, 4], [0, 0])
    c.ctx[0] = 2 ** 31 - 2
    c.check(status=16)


@pytest.mark.parametrize("cu", [[0, 9, 5, 20], [1, 5, 9, 20], [0, 5, 9, 24], [-3, 5, 9, 20]])
def test_bad_offsets_write_nothing(cu):
    c = Case([5, 4, 11], [3, 2, 9])
    c.cu = np.array(cu, np.int32)
    out, lse = c.run()
    assert (out == 7.0).all() and (lse == 7.0).all() and int(c.status) == 16


def test_nan_scores_reach_their_rows_alone():
    c = Case([60, 5], [100, 3], Hq=4, Hkv=2, D=128, seed=9)
    c.q[7, 1] = float("nan")
    slot = int(c.table[0, 130 // 16]) * 16 + 130 % 16
    c.k[slot, 1] = float("nan")       # key 130 of request 0, KV head 1 (heads 2, 3)
    out, lse = c.run()
    nan = np.zeros((65, 4), bool)
    nan[7, 1] = True
    nan[30:60, 2:] = True             # positions 130 .. 159
    assert (np.isnan(lse) == nan).all()
    assert (np.isnan(out) == nan[:, :, None]).all()


def test_infinite_scores():
    """Keys whose scores are -inf carry no weight; a row of nothing else is empty."""
    c = Case([4], [60], Hq=2, Hkv=1, D=64, seed=10)
    c.q[:] = c.q.abs() + 0.5
    t = np.arange(64)
    slots = torch.from_numpy(c.table[0, t // 16].astype(np.int64) * 16 + t % 16)
    c.k[slots[:50]] = float("-inf")
    out, lse = c.run()
    k = c.k.clone()
    q, kk, vv = c.q.double(), k[slots[50:]].double(), c.v[slots[50:]].double()
    for i in range(4):
        s = torch.einsum("hd,kd->hk", q[i], kk[:11 + i, 0]) * c.scale
        ref = torch.softmax(s, 1) @ vv[:11 + i, 0]
        w = torch.softmax(s, 1) @ vv[:11 + i, 0].abs()
        assert (np.abs(out[i] - ref.numpy()) <=
                (2.0 ** -8 * (ref.abs() + w) + 2.0 ** -11 * w).numpy()).all()
        assert np.abs(lse[i] - torch.logsumexp(s, 1).numpy()).max() < 1e-3
    c.k[slots] = float("-inf")
    out, lse = c.run()
    assert (out == 0).all() and np.isneginf(lse).all() and int(c.status) == 0


def test_two_calls_share_a_workspace_and_repeat_to_the_bit():
    a = Case([300, 1, 40], [1000, 3000, 5], Hq=8, Hkv=2, D=128, ps=32, seed=12)
    b = Case([1] * 20, [2500] * 20, Hq=8, Hkv=2, D=128, ps=32, seed=13)
    ws = torch.empty(bdsa.chunk_attn_workspace_bytes(128), dtype=torch.uint8, device=DEV)
    ra = a.run(workspace=ws)
    rb = b.run(workspace=ws)
    a.check(ra)
    b.check(rb)
    for c, r in ((a, ra), (b, rb)):
        again = c.run(workspace=ws.fill_(255))
        assert (again[0] == r[0]).all() and (again[1] == r[1]).all()


def test_captured_and_replayed_on_another_stream():
    c = Case([130, 1, 7], [300, 2000, 0], Hq=8, Hkv=2, D=128, ps=16, seed=14)
    d = c.dev()
    first = c.run(d)
    lse = torch.zeros((c.T, c.Hq), dtype=torch.float32, device=DEV)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        out = bdsa.chunk_attn_paged(d["q"], d["k"], d["v"], d["table"], d["ctx"], d["cu"],
                                    page_size=c.ps, scale=c.scale, lse=lse)
    for _ in range(3):
        out.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert (out.double().cpu().numpy() == first[0]).all()
    assert (lse.double().cpu().numpy() == first[1]).all()
    # other lengths in the same buffers
    c.ctx = np.array([250, 1970, 40])
    c.new = np.array([100, 37, 1])
    c.cu = np.array([0, 100, 137, 138], np.int32)
    d["ctx"].copy_(torch.from_numpy(c.ctx.astype(np.int32)))
    d["cu"].copy_(torch.from_numpy(c.cu))
    pages = (c.table >= 0).sum(1) * 16
    c.table[2, :3] = c.table[0, :3]
    d["table"].copy_(torch.from_numpy(c.table))
    assert (c.ctx[:2] + c.new[:2] <= pages[:2]).all()
    # (positions that the first lengths did not reach hold NaN)
    for n in ("k", "v"):
        x = torch.nan_to_num(getattr(c, n), nan=0.25)
        setattr(c, n, x)
        d[n].copy_(x)
    out.fill_(7.0)
    lse.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    c.check((out.double().cpu().numpy(), lse.double().cpu().numpy()))


def test_matches_block_attention():
    """Requests of B new tokens each: the block call's VERIFY and DRAFT masks."""
    for mb, mode in ((1, bdsa.VERIFY), (1 << 20, bdsa.DRAFT)):
        c = Case([16] * 5, [100, 0, 513, 64, 31], Hq=8, Hkv=2, D=128, ps=16, mb=mb, seed=15)
        d = c.dev()
        out, lse = c.run(d)
        lse2 = torch.empty((80, 8), dtype=torch.float32, device=DEV)
        out2 = bdsa.block_attn_paged(d["q"], d["k"], d["v"], d["table"], d["ctx"], B=16,
                                     page_size=16, scale=c.scale, mode=mode, max_ctx_len=600,
                                     lse=lse2)
        weight = c.want()[2]
        tol = 2 * 2.0 ** -8 * (np.abs(out) + weight) + 2.0 ** -10 * weight
        assert (np.abs(out - out2.double().cpu().numpy()) <= tol).all()
        assert np.abs(lse - lse2.double().cpu().numpy()).max() < 1e-3


@pytest.mark.parametrize("ps", [256, 1024])
@pytest.mark.parametrize("bad", [False, True])
def test_pages_of_several_tiles(ps, bad):
    c = Case([300, 1, 40], [900, 2100, 0], Hq=4, Hkv=2, D=64, ps=ps, seed=21)
    if bad:  # keys [ps, 2 ps) of request 0: its first tokens do not reach them at ps 1024
        c.table[0, 1] = -3
    c.check(status=16 if bad else 0)
    c.status.zero_()
    c.check(status=16 if bad else 0, sms=40)


def test_many_requests():
    rng = np.random.default_rng(22)
    new = rng.integers(0, 3, 1100)
    Case(new, rng.integers(0, 90, 1100), Hq=2, Hkv=1, D=64, ps=8, seed=22).check()


@pytest.mark.parametrize("heads", [(64, 64), (40, 8), (128, 1)])
def test_many_heads(heads):
    Case([40, 1], [200, 65], *heads, D=128, ps=32, seed=23).check()


@pytest.mark.parametrize("sms", [0, 30])
def test_output_at_any_16_bytes(sms):
    c = Case([70, 1, 3], [400, 900, 0], Hq=4, Hkv=2, D=128, ps=16, seed=24)
    d = c.dev()
    first = c.run(d, sms=sms)
    flat = torch.full((c.T * 4 * 128 + 16,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = flat[8:8 + c.T * 4 * 128].view(c.T, 4, 128)
    assert out.data_ptr() % 32 == 16
    bdsa.chunk_attn_paged(d["q"], d["k"], d["v"], d["table"], d["ctx"], d["cu"], page_size=16,
                          scale=c.scale, out=out, sms=sms)
    assert (out.double().cpu().numpy() == first[0]).all()
    assert (flat[:8] == 7.0).all() and (flat[8 + c.T * 4 * 128:] == 7.0).all()


def test_two_streams_at_once():
    cases = [Case([200, 1, 1], [900, 3000, 70], Hq=8, Hkv=2, D=128, ps=16, seed=s)
             for s in (25, 26)]
    devs = [c.dev() for c in cases]
    alone = [c.run(d) for c, d in zip(cases, devs)]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = []
    torch.cuda.synchronize()
    for _ in range(5):
        for c, d, s in zip(cases, devs, streams):
            with torch.cuda.stream(s):
                outs.append(bdsa.chunk_attn_paged(d["q"], d["k"], d["v"], d["table"], d["ctx"],
                                                  d["cu"], page_size=16, scale=c.scale))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert (o.double().cpu().numpy() == alone[i % 2][0]).all()
