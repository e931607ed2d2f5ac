// chunk_attn.cu -- attention of a ragged batch of new tokens over the paged cache
// they were written to, for sm_103a.
//
// Request r has L_r keys in the cache before its n_r new tokens, whose own keys
// follow them.  Token i at position p = L + i sees the keys below
//   lim(i) = min(L + n, (p / mb + 1) mb)        (mb = 1: p + 1, token-causal)
//   o_i = sum_{t < lim(i)} e^{s_it - m_i} v_t / sum_{t < lim(i)} e^{s_it - m_i}.
//
// Shape of the work: the (token, head of the group) rows of one (request, KV head)
// are cut into tiles of npt whole tokens (at most 128 rows), two tiles to a pair.  A
// unit is a pair over its keys, in 128-key tiles.  Units are ordered (request, KV
// head, pair) and charged kUnitCost keys and those that they see; persistent CTAs
// take equal ranges of that cost, so single tokens, prompts of any lengths and one
// long document split alike over the GPU without a list of units.  All sums over a
// request's pairs are closed forms, so a CTA finds its range by one scan of the
// requests and a search.  A unit cut between CTAs leaves fp32 partials (o / l and
// the log2-sum-exp of each row), which a second kernel joins.
//
// Inside a CTA (12 warps): warps 0-3 and 4-7 are the softmax of the two row tiles,
// one thread a row; then a K producer (also Q), a V producer and an MMA issuer for
// each row tile.  A row tile's S (128 columns of TMEM) is read by its softmax, which
// writes P as bf16 over it; PV takes P from TMEM.  The two tiles alternate on the
// tensor cores and share every K and V tile in shared memory.  A row tile whose rows
// see no key of the unit's last tiles sits those out.  O is rescaled in TMEM only
// when a row's max grows by 2^8.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <limits.h>

#include "attn_common.cuh"
#include "attn_tmem.cuh"
#include "bdsa_device.cuh"
#include "bdsa_internal.h"
#include "cache_internal.h"

namespace bdsa {
namespace {

constexpr int kRows = 128;      // query rows of a tile
constexpr int kUnitCost = 256;  // keys a unit switch is charged (a Q load, an epilogue)
constexpr int kMinCost = 768;   // a CTA takes at least this cost

// The unit that a CTA left cut after its first piece.
struct Cut {
    int valid, tok0, ntok, h, nt, S;
    long long cu, span, Wc;  // the unit's first cost and its cost, the whole call's
};

struct ChunkParams {
    const int32_t *block_table, *seq_lens, *cu;
    uint16_t *out;
    float *lse;
    Cut *cut;                  // [CTAs]
    float *slot_lse, *slot_o;  // [CTAs * 2, 256], [.., D]
    int32_t *dev_status;
    int bs, T, max_pages, num_pages, Hq, Hkv, G, npt, mb, log2_ps, box_rows;
    float scale_log2;
};

// A request's lengths and the costs of its units.
struct Req {
    int L, n, tok, P;  // context, new tokens, the first one's row, pairs
    bool bad;          // lengths that the table row cannot hold: its rows become zero
    int pstar;         // pairs whose keys are not clipped at L + n
    long long head;    // cost of a KV head's pairs
};

__device__ __forceinline__ Req load_req(const ChunkParams &p, int r) {
    Req q;
    const int c0 = __ldg(p.cu + r), c1 = __ldg(p.cu + r + 1);
    q.tok = c0;
    q.n = c1 - c0;
    q.L = __ldg(p.seq_lens + r);
    const long long room = (long long)p.max_pages << p.log2_ps;
    q.bad = q.L < 0 || (long long)q.L + q.n > min(room, (long long)INT_MAX - 2 * kBN);
    if (q.bad) q.L = 0;
    const int w = 2 * p.npt;
    q.P = (q.n + w - 1) / w;
    q.pstar = q.n >= p.mb ? (q.n - p.mb) / w : 0;
    const long long ps = q.pstar;
    q.head = (long long)q.P * (kUnitCost + q.L) + w * (ps * (ps + 1) / 2) + ps * (p.mb - 1) +
             (q.P - ps) * q.n;
    return q;
}

// Cost of the pairs before pair x of a KV head: pair y costs kUnitCost + L +
// min(n, (y + 1) w + mb - 1).
__device__ __forceinline__ long long pairs_before(const ChunkParams &p, const Req &q, int x) {
    const long long w = 2 * p.npt, a = min(x, q.pstar);
    return (long long)x * (kUnitCost + q.L) + w * (a * (a + 1) / 2) + a * (p.mb - 1) +
           (x - a) * q.n;
}

// Keys that token i of the request sees.
__device__ __forceinline__ int limit_of(const ChunkParams &p, int L, int n, int i) {
    const uint32_t pos = (uint32_t)(L + i), mb = (uint32_t)p.mb;
    return mb == 1u ? (int)pos + 1 : (int)min((uint32_t)(L + n), (pos / mb + 1u) * mb);
}

// A run of one unit's key tiles inside a CTA's range.
struct Piece {
    int r, L, n;          // request, its context and new tokens
    int i0, tok0, ntok;   // the pair's first token: in the request, its row; tokens left
    int h, a, e, nt;      // KV head, tiles [a, e) of nt
    bool bad;
    long long cu, span;   // the unit's first cost and its cost
};

__device__ __forceinline__ int tile_at(long long x, long long span, int nt) {
    return x >= span ? nt : x <= kUnitCost ? 0 : min(nt, (int)((x - kUnitCost) >> 7));
}

// Walks the pieces of a cost range.
struct Walk {
    int r;
    long long base;  // cost before request r
    long long c;     // next cost
    Req q;
    __device__ bool next(const ChunkParams &p, long long c1, Piece &pc) {
        while (c < c1) {
            const long long cost = q.head * p.Hkv;
            if (c >= base + cost) {
                if (++r >= p.bs) return false;
                base += cost;
                q = load_req(p, r);
                continue;
            }
            const long long rel = c - base;
            const int h = (int)(rel / q.head);
            const long long in = rel - h * q.head;
            int lo = 0, hi = q.P;  // the pair: pairs_before(lo) <= in < pairs_before(hi)
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (pairs_before(p, q, mid) <= in) lo = mid;
                else hi = mid;
            }
            const int w = 2 * p.npt;
            pc.cu = base + h * q.head + pairs_before(p, q, lo);
            pc.span = kUnitCost + q.L +
                      min((long long)q.n, (lo + 1LL) * w + p.mb - 1);
            const long long from = c - pc.cu, to = min(c1 - pc.cu, pc.span);
            c = pc.cu + to;
            pc.i0 = lo * w;
            pc.ntok = q.n - pc.i0;
            const int last = limit_of(p, q.L, q.n, pc.i0 + min(pc.ntok, w) - 1);
            pc.nt = (last + kBN - 1) / kBN;
            pc.a = tile_at(from, pc.span, pc.nt);
            pc.e = tile_at(to, pc.span, pc.nt);
            if (pc.a >= pc.e) continue;
            pc.r = r;
            pc.L = q.L;
            pc.n = q.n;
            pc.bad = q.bad;
            pc.h = h;
            pc.tok0 = q.tok + pc.i0;
            return true;
        }
        return false;
    }
};

// Key tiles of the piece that row tile t takes part in (0: none of its tokens
// sees one, or it has no tokens).
__device__ __forceinline__ int tiles_of(const ChunkParams &p, const Piece &pc, int t) {
    const int k = min(pc.ntok - t * p.npt, p.npt);
    if (k <= 0) return 0;
    const int lim = limit_of(p, pc.L, pc.n, pc.i0 + t * p.npt + k - 1);
    return max(0, min(pc.e, (lim + kBN - 1) / kBN) - pc.a);
}

template <int D>
struct CCfg {
    static constexpr int DH = D / 64;           // 128-byte slabs of a row
    static constexpr int kSlab = kRows * 128;   // one slab of a 128-row tile
    static constexpr int kTile = DH * kSlab;    // a Q, K or V tile
    // K is held until both tiles' S, V until both tiles' PV, about a tile longer
    static constexpr int NK = D == 128 ? 2 : 4, NV = D == 128 ? 3 : 4;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = 2 * kTile;
    static constexpr int kOffV = kOffK + NK * kTile;
    static constexpr int kOffBar = kOffV + NV * kTile;
    // barriers
    static constexpr int QF = 0;         // 2: Q tile loaded
    static constexpr int QE = QF + 2;    // 2: its last S of the piece done
    static constexpr int KF = QE + 2;
    static constexpr int KE = KF + NK;
    static constexpr int VF = KE + NK;
    static constexpr int VE = VF + NV;
    static constexpr int SF = VE + NV;   // 2: S of a row tile written (PV before it done)
    static constexpr int PF = SF + 2;    // 2 x 2: half of P written (and O rescaled)
    static constexpr int OF = PF + 4;    // 2: last PV of the piece done
    static constexpr int OE = OF + 2;    // 2: O read by the epilogue
    static constexpr int DR = OE + 2;    // 2: drain
    static constexpr int TK = DR + 2;    // 2: the other row tile's exponentials are done
    static constexpr int kNumBars = TK + 2;
    static constexpr int kOffMisc = kOffBar + 8 * kNumBars;
    static constexpr int kMisc = 256;
    static constexpr int kSmem = kOffMisc + kMisc + 1024;
    static constexpr int kProdK = 8, kMma0 = 9, kProdV = 10;  // (kMma1 = 11)
    static constexpr int kThreads = 12 * 32;
    // Registers a thread: 168 at launch (12 warps of 65536 / 384), moved from
    // the producers' warpgroup to the softmax ones, whose 128 scores a thread
    // spill otherwise: 256 * 208 + 128 * 80 <= 384 * 168.
    static constexpr int kSoftmaxRegs = 208, kProducerRegs = 80;
    static_assert(256 * kSoftmaxRegs + 128 * kProducerRegs <= kThreads * 168, "register split");
};

struct CSched {
    uint32_t tmem;
    int abort, r0, S;
    long long wsum[12];
    long long c0, c1, base, Wc;
};
static_assert(sizeof(CSched) <= 256, "the schedule state has 256 bytes");

template <int D>
__global__ void __launch_bounds__(CCfg<D>::kThreads, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const ChunkParams prm) {
    using C = CCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (sbase - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto bar = [&](int i) -> uint32_t { return sbase + C::kOffBar + 8u * (uint32_t)i; };
    CSched *sch = reinterpret_cast<CSched *>(smem + C::kOffMisc);
    volatile int *abort_flag = &sch->abort;
    // TMEM columns: S of row tile t at 128 t (P over its first 64), O at 256 + 128 t
    constexpr uint32_t kS = 0, kO = 256;

    if (warp == C::kMma0) {
        tmem_alloc(smem_u32(&sch->tmem), 512);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(C::QF + t), 1);
            mbar_init(bar(C::QE + t), 1);
            mbar_init(bar(C::SF + t), 1);
            mbar_init(bar(C::PF + 2 * t), 4);
            mbar_init(bar(C::PF + 2 * t + 1), 4);
            mbar_init(bar(C::OF + t), 1);
            mbar_init(bar(C::OE + t), 4);
            mbar_init(bar(C::DR + t), 1);
            mbar_init(bar(C::TK + t), 4);
        }
        for (int k = 0; k < C::NK; ++k) {
            mbar_init(bar(C::KF + k), 1);
            mbar_init(bar(C::KE + k), 2);
        }
        for (int k = 0; k < C::NV; ++k) {
            mbar_init(bar(C::VF + k), 1);
            mbar_init(bar(C::VE + k), 2);
        }
        *abort_flag = 0;
        fence_mbarrier_init();
    }
    if (warp == C::kProdK && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
    }
    if (warp == C::kProdV && lane == 0) tma_prefetch_desc(&tm_v);
    // rows of a tile past its whole tokens stay zero
    const int rows = prm.G * prm.npt;
    for (int idx = tid; idx < 2 * C::DH * (kRows - rows) * 8; idx += C::kThreads) {
        const int u = idx & 7, pad = kRows - rows;
        const int m = rows + (idx >> 3) % pad, slab = (idx >> 3) / pad;
        st_shared_v4(sbase + C::kOffQ + slab * C::kSlab + m * 128 + u * 16, 0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sch->tmem;

    // ---- everything before this call on the stream has finished
    grid_dependency_wait();
    grid_launch_dependents();

    // ---- schedule: a scan of the requests' costs
    {
        const int bs = prm.bs;
        const int per = (bs + C::kThreads - 1) / C::kThreads;
        const int i0 = min(bs, tid * per), i1 = min(bs, i0 + per);
        // offsets that do not run up from 0 to at most T: no row is anybody's
        bool wrong = false;
        for (int r = i0; r < i1; ++r) {
            const int o0 = __ldg(prm.cu + r), o1 = __ldg(prm.cu + r + 1);
            wrong |= o1 < o0 || (r == 0 && o0 != 0) || (r == bs - 1 && o1 > prm.T);
        }
        wrong = __syncthreads_or(wrong);
        long long sum = 0;
        if (!wrong)
            for (int r = i0; r < i1; ++r) sum += load_req(prm, r).head * prm.Hkv;
        long long inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += t;
        }
        if (lane == 31) sch->wsum[warp] = inc;
        __syncthreads();
        long long wex = 0, Wc = 0;
        for (int w = 0; w < C::kThreads / 32; ++w) {
            if (w < warp) wex += sch->wsum[w];
            Wc += sch->wsum[w];
        }
        const long long S = max(1LL, min((long long)gridDim.x, Wc / kMinCost));
        const long long b = blockIdx.x;
        const long long c0 = b < S ? b * Wc / S : Wc, c1 = b < S ? (b + 1) * Wc / S : Wc;
        long long at = wex + inc - sum;
        if (at <= c0 && c0 < at + sum) {
            for (int r = i0; r < i1; ++r) {
                const long long cost = load_req(prm, r).head * prm.Hkv;
                if (at <= c0 && c0 < at + cost) {
                    sch->r0 = r;
                    sch->base = at;
                }
                at += cost;
            }
        }
        if (tid == 0) {
            sch->c0 = c0;
            sch->c1 = c1;
            sch->S = (int)S;
            sch->Wc = Wc;
            prm.cut[blockIdx.x].valid = 0;
            if (wrong && blockIdx.x == 0) report_status(prm.dev_status, BDSA_DEVICE_OUT_OF_RANGE);
        }
        __syncthreads();
    }
    const long long c1 = sch->c1;
    Walk walk;
    walk.c = sch->c0;
    if (walk.c < c1) {
        walk.r = sch->r0;
        walk.base = sch->base;
        walk.q = load_req(prm, walk.r);
    }
    Piece pc;

    // (each warpgroup's split inside its own branch: code they share is compiled
    // for the smaller count)
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kProducerRegs));
        if (warp == C::kProdK || warp == C::kProdV) {
            // ------------------------------------------------ TMA producers
            if (lane == 0) {
                const bool is_k = warp == C::kProdK;
                const int NR = is_k ? C::NK : C::NV, FULL = is_k ? C::KF : C::VF;
                const int EMPTY = is_k ? C::KE : C::VE;
                const uint32_t dst0 = sbase + (is_k ? C::kOffK : C::kOffV);
                const void *tmap = is_k ? (const void *)&tm_k : (const void *)&tm_v;
                const int rows_box = prm.box_rows;
                const int nbox = kBN / rows_box;
                const int ps = 1 << prm.log2_ps;
                // keys without a page of the pool read as zeros: a row past the
                // cache's last is filled by the load
                const int outside = prm.num_pages << prm.log2_ps;
                int st = 0;
                uint32_t ph = 1;
                long g = 0;
                int kq[2] = {0, 0};  // pieces each row tile took part in
                bool ok = true;
                while (ok && walk.next(prm, c1, pc)) {
                    if (is_k) {
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (!ok || tiles_of(prm, pc, t) == 0) continue;
                            if (kq[t] > 0)
                                ok = mbar_wait(bar(C::QE + t), (kq[t] - 1) & 1, abort_flag,
                                               prm.dev_status);
                            if (!ok) break;
                            mbar_arrive_expect_tx(bar(C::QF + t), (uint32_t)(rows * D * 2));
                            for (int c = 0; c < C::DH; ++c)
                                tma_load_4d(sbase + C::kOffQ + t * C::kTile + c * C::kSlab, &tm_q,
                                            c * 64, 0, pc.h, pc.tok0 + t * prm.npt,
                                            bar(C::QF + t));
                            ++kq[t];
                        }
                        if (!ok) break;
                    }
                    const int32_t *bt = prm.block_table + (long)pc.r * prm.max_pages;
                    const int n_keys = pc.L + pc.n;
                    for (int j = pc.a; j < pc.e; ++j, ++g) {
                        const int t0 = j * kBN;
                        int32_t slot[kMaxBoxes];
#pragma unroll
                        for (int bx = 0; bx < kMaxBoxes; ++bx) {
                            if (bx >= nbox) break;
                            const int t = t0 + bx * rows_box;
                            const int page = t >> prm.log2_ps;
                            const int32_t id = t < n_keys && !pc.bad ? __ldg(bt + page) : -1;
                            slot[bx] = id >= 0 && id < prm.num_pages ? id * ps + (t & (ps - 1))
                                                                     : outside;
                        }
                        ok = mbar_wait(bar(EMPTY + st), ph, abort_flag, prm.dev_status);
                        if (!ok) break;
                        mbar_arrive_expect_tx(bar(FULL + st), (uint32_t)C::kTile);
#pragma unroll
                        for (int bx = 0; bx < kMaxBoxes; ++bx) {
                            if (bx >= nbox) break;
                            for (int c = 0; c < C::DH; ++c)
                                tma_load_2d(dst0 + st * C::kTile + c * C::kSlab +
                                                bx * rows_box * 128,
                                            tmap, pc.h * D + c * 64, slot[bx], bar(FULL + st));
                        }
                        if (++st == NR) {
                            st = 0;
                            ph ^= 1;
                        }
                    }
                }
                // Drain: the last load issued into each buffer has landed.
                if (is_k)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        if (kq[t] > 0) mbar_wait_drain(bar(C::QF + t), (kq[t] - 1) & 1);
                for (long i = max(0L, g - NR); i < g; ++i)
                    mbar_wait_drain(bar(FULL + (int)(i % NR)), (uint32_t)((i / NR) & 1));
            }
        } else {
            // ------------------------------------------------ MMA issuers, one a row tile
            // The whole warp walks the schedule and one elected lane issues: an
            // MMA takes its descriptors from uniform registers, which only code
            // that the warp runs together keeps them in.
            const int t = warp == C::kMma0 ? 0 : 1;
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0) + t * 128;
            const bool leader = elect_one();
            constexpr uint32_t idesc_qk = idesc_bf16_f32(kRows, kBN, 0, 0);
            constexpr uint32_t idesc_pv = idesc_bf16_f32(kRows, D, 0, 1);
            uint32_t gt = 0, kt = 0;  // S tiles and pieces of this row tile
            bool ok = true;
            auto wait = [&](int i, uint32_t parity) {
                ok = ok && mbar_wait(bar(i), parity & 1, abort_flag, prm.dev_status);
                ok = __all_sync(0xffffffffu, ok);
            };
            auto commit = [&](int i) {
                if (leader) umma_commit(bar(i));
            };
            // descriptors of the first operand tiles; another tile, or K step, is an
            // addition to the address field
            const uint64_t dq = smem_desc_sw128(sbase + C::kOffQ + t * C::kTile, 16, 1024);
            const uint64_t dk = smem_desc_sw128(sbase + C::kOffK, 16, 1024);
            const uint64_t dv = smem_desc_sw128(sbase + C::kOffV, C::kSlab, 1024);
            auto issue_s = [&](int ks) {
                const uint64_t k = dk + (uint32_t)(ks * (C::kTile >> 4));
                if (!leader) return;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * C::kSlab + (kk & 3) * 32) >> 4;
                    umma_bf16(tm + kS, dq + off, k + off, idesc_qk, kk > 0 ? 1u : 0u);
                }
                umma_commit(bar(C::SF + t));
            };
            auto issue_pv = [&](int vs, int part, bool first) {  // keys 64 part ..
                const uint64_t v = dv + (uint32_t)(vs * (C::kTile >> 4));
                if (!leader) return;
#pragma unroll
                for (int k4 = 0; k4 < 4; ++k4) {
                    const int kk = part * 4 + k4;
                    umma_bf16_ts(tm + kO, tm + kS + kk * 8, v + (uint32_t)(kk * 128), idesc_pv,
                                 (first && k4 == 0) ? 0u : 1u);
                }
            };
            // ring positions and their phases
            int ks = 0, vs = 0;
            uint32_t kph = 0, vph = 0;
            auto next_k = [&] {
                commit(C::KE + ks);
                if (++ks == C::NK) {
                    ks = 0;
                    kph ^= 1;
                }
            };
            auto next_v = [&] {
                commit(C::VE + vs);
                if (++vs == C::NV) {
                    vs = 0;
                    vph ^= 1;
                }
            };
            while (ok && walk.next(prm, c1, pc)) {
                const int n = tiles_of(prm, pc, t), all = pc.e - pc.a;
                if (n > 0) {
                    // the first S
                    wait(C::KF + ks, kph);
                    wait(C::QF + t, kt);
                    if (!ok) break;
                    tc_fence_after();
                    issue_s(ks);
                    if (n == 1) commit(C::QE + t);
                    next_k();
                    for (int j = 0; j < n; ++j) {
                        const bool more = j + 1 < n;
                        wait(C::VF + vs, vph);
                        if (j == 0 && kt > 0) wait(C::OE + t, kt - 1);
                        wait(C::PF + 2 * t, gt);
                        if (!ok) break;
                        tc_fence_after();
                        issue_pv(vs, 0, j == 0);
                        if (more) wait(C::KF + ks, kph);
                        wait(C::PF + 2 * t + 1, gt);
                        if (!ok) break;
                        ++gt;
                        tc_fence_after();
                        issue_pv(vs, 1, false);
                        if (more) {
                            issue_s(ks);
                            if (j + 2 == n) commit(C::QE + t);
                            next_v();
                            next_k();
                        } else {
                            commit(C::OF + t);
                            next_v();
                        }
                    }
                    ++kt;
                }
                // its share of the releases of tiles that its rows do not see
                for (int j = n; ok && j < all; ++j) {
                    wait(C::KF + ks, kph);
                    if (ok) next_k();
                    wait(C::VF + vs, vph);
                    if (ok) next_v();
                }
            }
            commit(C::DR + t);
            mbar_wait_drain(bar(C::DR + t), 0);
        }
    } else {
        // ------------------------------------------------ softmax + epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
        const int t = warp >> 2;                       // row tile
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lane_base + kS + t * 128;
        const uint32_t o_addr = tmem + lane_base + kO + t * 128;
        const float sl2 = prm.scale_log2;
        const int node = row / prm.G;                  // token within the tile
        uint32_t gs = 0, k = 0;
        uint32_t turn = 0;  // tiles that both row tiles took
        int vs0 = 0;        // V ring position and phase of the piece's first tile
        uint32_t vph0 = 0;
        bool ok = true;
        while (ok && walk.next(prm, c1, pc)) {
            const int n = tiles_of(prm, pc, t);
            const int nboth = t == 0 ? (prm.npt < pc.ntok ? n : 0)
                                     : (n > 0 ? tiles_of(prm, pc, 0) : 0);
            const int all = pc.e - pc.a, n_keys = pc.L + pc.n;
            const bool whole = pc.a == 0 && pc.e == pc.nt;
            const int token = t * prm.npt + node;
            const bool real = row < rows && token < pc.ntok;
            // keys this row sees (rows that are nobody's: all, nothing to mask)
            const int lim = real ? limit_of(prm, pc.L, pc.n, pc.i0 + token) : INT_MAX;
            // the piece's first key without a page of the pool
            int bad_key = pc.bad ? 0 : INT_MAX;
            if (n > 0 && !pc.bad) {
                const int p0 = (pc.a * kBN) >> prm.log2_ps;
                const int p1 = (min((pc.a + n) * kBN, n_keys) - 1) >> prm.log2_ps;
                const int32_t *bt = prm.block_table + (long)pc.r * prm.max_pages;
#pragma unroll 4
                for (int pg = p0 + lane; pg <= p1; pg += 32) {
                    const int32_t id = __ldg(bt + pg);
                    if (id < 0 || id >= prm.num_pages) bad_key = min(bad_key, pg << prm.log2_ps);
                }
                bad_key = __reduce_min_sync(0xffffffffu, bad_key);
            }
            float m_used = -INFINITY;
            uint64_t lacc[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
            for (int j = 0; j < n; ++j, ++gs) {
                const int t0 = (pc.a + j) * kBN;
                ok = mbar_wait(bar(C::SF + t), gs & 1, abort_flag, prm.dev_status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                float sv[128];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_ld32(s_addr + c * 32, *reinterpret_cast<float(*)[32]>(&sv[c * 32]));
                tmem_wait_ld();
                const int nvis = lim - t0;
                if (__any_sync(0xffffffffu, nvis < kBN)) {
#pragma unroll
                    for (int c = 0; c < 128; ++c) sv[c] = c < nvis ? sv[c] : -INFINITY;
                }
                float mx[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) mx[c] = sv[c];
#pragma unroll
                for (int c = 8; c < 128; c += 2)
                    mx[(c >> 1) & 7] = max3f(mx[(c >> 1) & 7], sv[c], sv[c + 1]);
                const float m_new = fmaxf(max3f(max3f(mx[0], mx[1], mx[2]), mx[3], mx[4]),
                                          max3f(mx[5], mx[6], mx[7])) *
                                    sl2;
                float alpha = 1.f;
                bool resc = false;
                if (m_new > m_used + kRescaleLog2) {
                    alpha = ex2_approx(m_used - m_new);
                    m_used = m_new;
                    resc = true;
                }
                if (__any_sync(0xffffffffu, resc)) {
                    const uint64_t a2 = f2_pack(alpha, alpha);
                    lacc[0] = f2_mul(lacc[0], a2);
                    lacc[1] = f2_mul(lacc[1], a2);
                    // (S of this tile was issued after PV of the last one, and
                    // its barrier covers both: O is complete)
                    if (j > 0) {
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            float ov[32];
                            tmem_ld32(o_addr + c * 32, ov);
                            tmem_wait_ld();
#pragma unroll
                            for (int q = 0; q < 32; ++q) ov[q] *= alpha;
                            tmem_st32(o_addr + c * 32, ov);
                        }
                    }
                }
                // V rows past the request's last key are whatever the page holds,
                // and 0 * NaN is NaN: they become zeros before PV reads them
                // (each row tile before its own PV; both write the same zeros)
                if (t0 + kBN > n_keys) {
                    const int vi = vs0 + j;  // (tiles of this piece: at most ..)
                    const int vs = vi % C::NV;
                    ok = mbar_wait(bar(C::VF + vs), (vph0 + (uint32_t)(vi / C::NV)) & 1,
                                   abort_flag, prm.dev_status);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const int first = n_keys - t0;
                    for (int idx = row; idx < C::DH * 8 * (kBN - first); idx += kRows) {
                        const int u = idx & 7, rr = idx >> 3;
                        const int slab = rr >= kBN - first ? 1 : 0;
                        const int m = first + rr - slab * (kBN - first);
                        st_shared_v4(sbase + C::kOffV + vs * C::kTile + slab * C::kSlab + m * 128 +
                                         u * 16,
                                     0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                // The row tiles' exponentials in turn: at the same time each takes
                // twice as long (the special function unit is shared), and then
                // both row tiles' MMAs come at once and nothing overlaps.
                const bool both = j < nboth;
                if (both && (t == 1 || turn > 0)) {
                    ok = mbar_wait(bar(C::TK + t), (t == 1 ? turn : turn - 1) & 1, abort_flag,
                                   prm.dev_status);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                }
                const float neg_m = m_used == -INFINITY ? 0.f : -m_used;
                const uint64_t sc2 = f2_pack(sl2, sl2), nm2 = f2_pack(neg_m, neg_m);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        const float2 xv = f2_unpack(
                            f2_fma(f2_pack(sv[c * 32 + 2 * q], sv[c * 32 + 2 * q + 1]), sc2, nm2));
                        const float p0 = ex2_approx(xv.x), p1 = ex2_approx(xv.y);
                        pk[q] = pack_bf16x2(p0, p1);
                        lacc[q & 1] = f2_add(lacc[q & 1], f2_pack(p0, p1));
                    }
                    tmem_st16(s_addr + c * 16, pk);
                    if (c & 1) {  // half of P: its PV may start
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(C::PF + 2 * t + (c >> 1)));
                    }
                }
                if (both) {
                    if (lane == 0) mbar_arrive(bar(C::TK + 1 - t));
                    ++turn;
                }
            }
            if (!ok) break;
            vs0 += all;
            vph0 += (uint32_t)(vs0 / C::NV);
            vs0 %= C::NV;
            // ---- end of the piece: o / l and the log2-sum-exp
            if (n > 0) {
                ok = mbar_wait(bar(C::OF + t), k & 1, abort_flag, prm.dev_status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                ++k;
            }
            const float2 la = f2_unpack(lacc[0]), lb = f2_unpack(lacc[1]);
            const float l = (la.x + la.y) + (lb.x + lb.y);
            const bool hit = bad_key < lim;
            const float inv = l > 0.f ? 1.f / l : isnan(l) ? l : 0.f;
            const float l2 = l > 0.f ? m_used + log2f(l) : isnan(l) ? l : -INFINITY;
            if (whole) {
                const long at = (long)(pc.tok0 + token) * prm.Hq + (long)pc.h * prm.G +
                                row % prm.G;
                uint16_t *po = prm.out + at * D;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    float ov[32];
                    tmem_ld32(o_addr + c * 32, ov);
                    tmem_wait_ld();
                    if (!real) continue;
                    uint32_t pk[16];
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        pk[q] = hit ? 0u : pack_bf16x2(ov[2 * q] * inv, ov[2 * q + 1] * inv);
                    // (out rows are 16-byte aligned)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        *reinterpret_cast<uint4 *>(po + c * 32 + 8 * v) =
                            make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2], pk[4 * v + 3]);
                }
                if (real && prm.lse != nullptr) prm.lse[at] = hit ? -INFINITY : l2 * kLn2;
            } else {
                const long dst =
                    ((long)blockIdx.x * 2 + (pc.a == 0 ? 1 : 0)) * 2 * kRows + t * kRows + row;
                float *po = prm.slot_o + dst * D;
                if (n > 0) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        float ov[32];
                        tmem_ld32(o_addr + c * 32, ov);
                        tmem_wait_ld();
                        if (!real) continue;
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            st_global_v8(po + c * 32 + 8 * v, __float_as_uint(ov[8 * v] * inv),
                                         __float_as_uint(ov[8 * v + 1] * inv),
                                         __float_as_uint(ov[8 * v + 2] * inv),
                                         __float_as_uint(ov[8 * v + 3] * inv),
                                         __float_as_uint(ov[8 * v + 4] * inv),
                                         __float_as_uint(ov[8 * v + 5] * inv),
                                         __float_as_uint(ov[8 * v + 6] * inv),
                                         __float_as_uint(ov[8 * v + 7] * inv));
                    }
                }
                // +inf marks a row that sees a key without a page; a NaN score leaves NaN
                if (real) prm.slot_lse[dst] = hit ? INFINITY : l2;
                if (tid == 0 && pc.a == 0) {
                    Cut d;
                    d.valid = 1;
                    d.tok0 = pc.tok0;
                    d.ntok = pc.ntok;
                    d.h = pc.h;
                    d.nt = pc.nt;
                    d.S = sch->S;
                    d.cu = pc.cu;
                    d.span = pc.span;
                    d.Wc = sch->Wc;
                    prm.cut[blockIdx.x] = d;
                }
            }
            if (n > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::OE + t));
            }
            if (hit && real) report_status(prm.dev_status, BDSA_DEVICE_OUT_OF_RANGE);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == C::kMma0) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the pieces of the unit that CTA blockIdx.x cut: 32 of its rows a CTA, 8
// threads a row.
constexpr int kJoinRows = 32, kJoinThreads = 8 * kJoinRows;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) chunk_join_kernel(const ChunkParams prm) {
    grid_dependency_wait();
    grid_launch_dependents();
    const Cut d = prm.cut[blockIdx.x];
    if (!d.valid) return;
    const int sub = threadIdx.x & 7, lane = threadIdx.x & 31;
    const int row = blockIdx.y * kJoinRows + (threadIdx.x >> 3);
    const int t = row / kRows, rr = row % kRows, token = t * prm.npt + rr / prm.G;
    const bool real = rr < prm.G * prm.npt && token < d.ntok;
    if (__syncthreads_or(real) == 0) return;
    // the unit's last piece: the first CTA whose range reaches its last tile
    const int b = blockIdx.x;
    int np = 0;
    for (int k0 = 1; np == 0 && b + k0 < d.S; k0 += 32) {
        const int k = k0 + lane;
        const long long end = (long long)(b + k + 1) * d.Wc / d.S;
        const bool done = b + k >= d.S - 1 || tile_at(end - d.cu, d.span, d.nt) >= d.nt;
        const uint32_t m = __ballot_sync(0xffffffffu, done);
        if (m != 0) np = k0 + __ffs(m);  // pieces: this CTA's and those up to that one
    }
    auto slot = [&](int i) { return ((long)(b + i) * 2 + (i == 0 ? 1 : 0)) * 2 * kRows + row; };
    float mx = -INFINITY;
    bool hit = false, nan = false;
    for (int i = sub; i < np; i += 8) {
        const float v = real ? __ldcg(prm.slot_lse + slot(i)) : -INFINITY;
        hit |= v == INFINITY;
        nan |= isnan(v);
        mx = fmaxf(mx, v);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        hit |= __shfl_xor_sync(0xffffffffu, (int)hit, o) != 0;
        nan |= __shfl_xor_sync(0xffffffffu, (int)nan, o) != 0;
    }
    if (!real) return;
    constexpr int W = D / 8;  // values a thread
    float acc[W], sum = 0.f;
#pragma unroll
    for (int c = 0; c < W; ++c) acc[c] = 0.f;
    if (!hit && !nan && mx > -INFINITY) {
#pragma unroll 2
        for (int i = 0; i < np; ++i) {
            const float v = __ldcg(prm.slot_lse + slot(i));
            if (v == -INFINITY) continue;  // (its o may not have been written)
            const float w = ex2_approx(v - mx);
            const float *po = prm.slot_o + slot(i) * D + sub * W;
            float ov[W];
#pragma unroll
            for (int c = 0; c < W; c += 8) ld_cg_v8(po + c, ov + c);
            sum += w;
#pragma unroll
            for (int c = 0; c < W; ++c) acc[c] = fmaf(w, ov[c], acc[c]);
        }
    }
    const float inv = nan ? NAN : sum > 0.f ? 1.f / sum : 0.f;
    const long at = (long)(d.tok0 + token) * prm.Hq + (long)d.h * prm.G + rr % prm.G;
    uint16_t *po = prm.out + at * D + sub * W;
#pragma unroll
    for (int c = 0; c < W; c += 8) {
        uint32_t pk[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            pk[q] = hit ? 0u : pack_bf16x2(acc[c + 2 * q] * inv, acc[c + 2 * q + 1] * inv);
        *reinterpret_cast<uint4 *>(po + c) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
    }
    if (prm.lse != nullptr && sub == 0)
        prm.lse[at] = hit ? -INFINITY : nan ? NAN : sum > 0.f ? (mx + log2f(sum)) * kLn2
                                                              : -INFINITY;
}

template <int D>
int launch_chunk(const ChunkArgs &a, cudaStream_t stream) {
    using C = CCfg<D>;
    static_assert(C::kSmem <= 227 * 1024, "shared memory of one CTA");
    EncodeTiledFn enc = encode_fn();
    if (enc == nullptr) return BDSA_CUDA_ERROR;
    const int G = a.Hq / a.Hkv, npt = kRows / G;
    CUtensorMap tq, tk, tv;
    {
        // q as (d, head of the group, KV head, token); a box is one row tile
        cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)G, (cuuint64_t)a.Hkv, (cuuint64_t)a.T};
        cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)G * D * 2,
                                 (cuuint64_t)a.q_stride * 2};
        cuuint32_t box[4] = {64, (cuuint32_t)G, 1, (cuuint32_t)npt};
        cuuint32_t es[4] = {1, 1, 1, 1};
        if (enc(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t *>(a.q), dims,
                strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) !=
            CUDA_SUCCESS)
            return BDSA_CUDA_ERROR;
    }
    const int box_rows = a.page_size < kBN ? a.page_size : kBN;
    for (int which = 0; which < 2; ++which) {
        cuuint64_t dims[2] = {(cuuint64_t)a.Hkv * D, (cuuint64_t)a.num_pages * a.page_size};
        cuuint64_t strides[1] = {(cuuint64_t)a.Hkv * D * 2};
        cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
        cuuint32_t es[2] = {1, 1};
        if (enc(which == 0 ? &tk : &tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                const_cast<uint16_t *>(which == 0 ? a.k_cache : a.v_cache), dims, strides, box,
                es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) !=
            CUDA_SUCCESS)
            return BDSA_CUDA_ERROR;
    }
    const ChunkPlan plan = chunk_plan(D, a.ctas);
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    ChunkParams p;
    p.block_table = a.block_table;
    p.seq_lens = a.seq_lens;
    p.cu = a.cu_tokens;
    p.out = a.out;
    p.lse = a.lse;
    p.cut = reinterpret_cast<Cut *>(ws);
    p.slot_lse = reinterpret_cast<float *>(ws + plan.off_lse);
    p.slot_o = reinterpret_cast<float *>(ws + plan.off_o);
    p.dev_status = a.dev_status;
    p.bs = a.bs;
    p.T = a.T;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = G;
    p.npt = npt;
    p.mb = a.mask_block;
    int lg = 0;
    while ((1 << lg) < a.page_size) ++lg;
    p.log2_ps = lg;
    p.box_rows = box_rows;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    if (cudaFuncSetAttribute(chunk_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmem) != cudaSuccess)
        return BDSA_CUDA_ERROR;
    if (launch_pdl(chunk_attn_kernel<D>, dim3(a.ctas), dim3(C::kThreads), (size_t)C::kSmem, stream,
                   tq, tk, tv, p) != cudaSuccess)
        return BDSA_CUDA_ERROR;
    return launch_pdl(chunk_join_kernel<D>, dim3(a.ctas, 2 * kRows / kJoinRows),
                      dim3(kJoinThreads), 0, stream, p) == cudaSuccess
               ? BDSA_OK
               : BDSA_CUDA_ERROR;
}

}  // namespace

int chunk_ctas(int num_sms) { return num_sms < 1 ? 1 : num_sms > 1024 ? 1024 : num_sms; }

ChunkPlan chunk_plan(int D, int ctas) {
    ChunkPlan p;
    p.off_lse = align256(sizeof(Cut) * (size_t)ctas);
    p.off_o = align256(p.off_lse + (size_t)ctas * 4 * kRows * sizeof(float));
    p.workspace = p.off_o + (size_t)ctas * 4 * kRows * D * sizeof(float);
    return p;
}

int launch_chunk_attn(const ChunkArgs &a, cudaStream_t stream) {
    return a.D == 128 ? launch_chunk<128>(a, stream) : launch_chunk<64>(a, stream);
}

}  // namespace bdsa
