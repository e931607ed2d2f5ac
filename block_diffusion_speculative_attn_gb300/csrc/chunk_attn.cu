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
// head, pair) and charged for a switch and the keys that they see; persistent CTAs
// take equal ranges of that cost, so single tokens, prompts of any lengths and one
// long document split alike over the GPU without a list of units.  All sums over a
// request's pairs are closed forms, so a CTA finds its range by one scan of the
// requests and a search.  A unit cut between CTAs leaves fp32 partials (o / l and
// the log2-sum-exp of each row), which a second kernel joins.
//
// Inside a CTA (12 warps): warps 0-3 and 4-7 are the softmax of the two row tiles,
// one thread a row; then a K producer (also Q), which alone walks the CTA's range and
// hands each piece on in shared memory, a V producer and an MMA issuer for each row
// tile.  A row tile's S (128 columns of TMEM) is read by its softmax, which
// writes P as bf16 over it; PV takes P from TMEM.  The two tiles alternate on the
// tensor cores and share every K and V tile in shared memory.  A row tile whose rows
// see no key of the unit's last tiles sits those out; where a pair has tokens for one
// row tile alone, both take its rows, each over every other key tile.  O is rescaled in
// TMEM only when a row's max grows by 2^8.
//
// What bounds it (us a call, launches in a graph):
//   64 single tokens over 512-8192 keys of 8 KV heads, pages of 16    191-195  HBM: 1.23 GB
//     at 0.93-0.95 of the copy rate (one row tile over all key tiles: 283)
//   24 prompts of 17-2048 tokens, 32 heads                            340-355  1.0 PFLOP/s;
//     161 key tiles a CTA of 1.55 us and 26 pieces of about 3 us
//   8 x 512-1024 tokens in blocks of 32 behind 1024-8192, 16 heads    241-252  1.31-1.37
//     PFLOP/s
//   4096 tokens behind 28672, 32 heads           1410 cool, 1440-1515 call after call at
//     the power limit: 1.36-1.46 PFLOP/s (0.71-0.76 of the measured rate)
//   44 single tokens and 4 chunks of 128-512 tokens, 16 heads          59
// A pair's key tile costs 2970 cycles against 2048 of MMAs: a row tile's chain of S, its
// maximum, the exponentials, P, PV and the next S is longer than the other tile's MMAs.
// Call after call the GPU is at its power limit besides (1.37 kW; the long chunk at 1650
// MHz, the blocks at 1810, the prompts at 1950); the chain is the larger part: a clock of
// the long chunk does 0.73 of what one of the library's product does at the same limit.
// A unit costs about 3 us besides: instructions that run once a unit come from far
// (with code of 127 KB instead of 79 the prompts took 574 us, not 349), and O has to leave
// TMEM before the next unit's PV.
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
// The cost of a unit: a key counts kPairKey where both row tiles have tokens, kOneKey
// where one has (a tile of those is 1.5 and 1.0-1.1 us), a switch kUnitCost (a Q load,
// an epilogue: 2 tiles of a pair).  With one weight the mixed batch above took 70 us:
// its CTAs ended between 45 and 68.
constexpr int kPairKey = 3, kOneKey = 2;
constexpr int kUnitCost = 768;
// A CTA takes at least this cost, two units of one tile: then a CTA whose whole share lies
// in one unit has tiles of it (4 at least), as the join takes for granted.  Calls of few
// short units run on fewer CTAs than they have units, one behind the other (2 requests
// of 8 tokens and one KV head: both on one CTA, 3-4 us each); other values were not
// measured.
constexpr int kMinCost = 2304;

// The unit that a CTA left cut after its first piece.
struct Cut {
    int valid, tok0, ntok, h, nt, S, key;
    long long cu, span;  // the unit's first cost and its cost
    long long each;      // the CTAs' shares
    int rem;
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
    int wide;                  // out is 32-byte aligned
};

// A request's lengths and the costs of its units.
struct Req {
    int L, n, tok, P;  // context, new tokens, the first one's row, pairs
    bool bad;          // lengths that the table row cannot hold: its rows become zero
    bool off;          // its offsets are not within q
    int pstar;         // pairs whose keys are not clipped at L + n
    int last;          // cost of a key in the last pair
    long long head;    // cost of a KV head's pairs
};

// Cost of the pairs before pair x < P of a KV head: pair y sees L + min(n, (y + 1) w +
// mb - 1) keys at most.
__device__ __forceinline__ long long pairs_before(const ChunkParams &p, const Req &q, int x) {
    const long long w = 2 * p.npt, a = min(x, q.pstar);
    return x * (kUnitCost + (long long)kPairKey * q.L) +
           kPairKey * (w * (a * (a + 1) / 2) + a * (p.mb - 1) + (x - a) * q.n);
}

__device__ __forceinline__ Req load_req(const ChunkParams &p, int r) {
    Req q;
    const int c0 = __ldg(p.cu + r), c1 = __ldg(p.cu + r + 1);
    q.L = __ldg(p.seq_lens + r);
    q.tok = c0;
    // (offsets that no row can have: the whole call does nothing then)
    q.off = c0 < 0 || c1 < c0 || c1 > p.T || (r == 0 && c0 != 0);
    q.n = q.off ? 0 : c1 - c0;
    const long long room = (long long)p.max_pages << p.log2_ps;
    q.bad = q.L < 0 || (long long)q.L + q.n > min(room, (long long)INT_MAX - 2 * kBN);
    if (q.bad) q.L = 0;
    const int w = 2 * p.npt;
    q.P = (q.n + w - 1) / w;
    q.pstar = q.n >= p.mb ? (q.n - p.mb) / w : 0;
    q.last = q.n - (q.P - 1) * w <= p.npt ? kOneKey : kPairKey;
    q.head = q.P > 0 ? pairs_before(p, q, q.P - 1) + kUnitCost + q.last * ((long long)q.L + q.n)
                     : 0;
    return q;
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
    int key;              // the cost of one of its keys
};

// The unit's first tile that is not before cost x: whole tiles, to the nearest.
__device__ __forceinline__ int tile_at(long long x, long long span, int nt, int key) {
    if (x >= span) return nt;
    if (x <= kUnitCost) return 0;
    const uint64_t k = (uint64_t)(x - kUnitCost);
    return min(nt, (int)(key == kPairKey ? (k + 64 * kPairKey) / (128 * kPairKey)
                                         : (k + 64 * kOneKey) / (128 * kOneKey)));
}

// a / b for 0 <= a, 0 < b: a 64-bit division is a long subroutine here.
__device__ __forceinline__ long long divide(long long a, long long b) {
    return ((uint64_t)(a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// Where CTA b's share of the cost starts: equal shares, the first rem one longer.
struct Shares {
    long long each;
    int rem;
    __device__ long long start(int b) const { return b * each + min(b, rem); }
};

// Walks the pieces of a cost range: one search for the first unit, then unit by unit.
struct Walk {
    int r, h, x;      // request, KV head, pair
    long long cu, c;  // the unit's first cost, the next cost
    Req q;
    __device__ void start(const ChunkParams &p, int r0, const Req &req, long long base) {
        r = r0;
        q = req;
        const long long rel = c - base;
        h = (int)divide(rel, q.head);
        const long long in = rel - h * q.head;
        int lo = 0, hi = q.P;  // pairs_before(lo) <= in < pairs_before(hi)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pairs_before(p, q, mid) <= in) lo = mid;
            else hi = mid;
        }
        x = lo;
        cu = base + h * q.head + pairs_before(p, q, lo);
    }
    __device__ bool next(const ChunkParams &p, long long c1, Piece &pc) {
        while (c < c1) {
            while (x >= q.P) {
                x = 0;
                if (++h < p.Hkv && q.P > 0) break;
                h = 0;
                if (++r >= p.bs) return false;
                q = load_req(p, r);
            }
            const int w = 2 * p.npt;
            pc.cu = cu;
            pc.key = x == q.P - 1 ? q.last : kPairKey;
            pc.span = kUnitCost + pc.key * (q.L + min((long long)q.n, (x + 1LL) * w + p.mb - 1));
            const long long from = c - cu, to = min(c1 - cu, pc.span);
            c = cu + to;
            pc.i0 = x * w;
            pc.ntok = q.n - pc.i0;
            if (to == pc.span) {
                cu += pc.span;
                ++x;
            }
            const int last = limit_of(p, q.L, q.n, pc.i0 + min(pc.ntok, w) - 1);
            pc.nt = (last + kBN - 1) / kBN;
            pc.a = tile_at(from, pc.span, pc.nt, pc.key);
            pc.e = tile_at(to, pc.span, pc.nt, pc.key);
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

// A piece as the K producer hands it to the other roles (in shared memory).  A pair
// whose tokens fit one row tile is split: the two row tiles take the same rows over
// every other key tile each, so that one's MMAs run beside the other's softmax, and
// join their halves in the end.
struct Work {
    int n[2];          // key tiles that each row tile takes
    int all, a;        // the piece's tiles, the first one (all = 0: no more pieces)
    int split, nboth;  // a split pair; first tiles that both row tiles take
    int whole;         // the unit's only piece
    int r, L, n_new, i0, tok0, ntok, h;
    int bad;           // (the request's lengths mean nothing)
    int bad_key;       // the piece's first key without a page, ready with BK
};
static_assert(sizeof(Work) == 64, "");

__device__ __forceinline__ void fill_work(const ChunkParams &p, const Piece &pc, Work *w) {
    const int n0 = tiles_of(p, pc, 0), n1 = tiles_of(p, pc, 1);
    const bool split = pc.ntok <= p.npt && n0 > 1;
    w->n[0] = split ? (n0 + 1) / 2 : n0;
    w->n[1] = split ? n0 / 2 : n1;
    w->all = pc.e - pc.a;
    w->a = pc.a;
    w->split = split;
    w->nboth = min(n0, n1);
    w->whole = pc.a == 0 && pc.e == pc.nt;
    w->r = pc.r;
    w->L = pc.L;
    w->n_new = pc.n;
    w->i0 = pc.i0;
    w->tok0 = pc.tok0;
    w->ntok = pc.ntok;
    w->h = pc.h;
    w->bad = pc.bad;
}

// mbar_wait with the part behind the first try in one place (the instruction caches hold
// the code of all roles); where many registers are live, mbar_wait itself.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int *abort,
                                     int32_t *dev_status) {
    return mbar_wait(bar, parity, abort, dev_status);
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort,
                                         int32_t *dev_status) {
    return mbar_try_wait(bar, parity) || wait_on(bar, parity, abort, dev_status);
}

// 16 consecutive columns of the thread's lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(r[k]);
}

__device__ __forceinline__ float rcp_approx(float x) {  // 1 ulp
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2_approx(float x) {  // 2^-22
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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
    static constexpr int MG = TK + 2;    // row tile 1's half of a split pair is done
    static constexpr int NW = 4;         // pieces handed on
    static constexpr int WF = MG + 1;    // NW: a piece is handed on
    static constexpr int WE = WF + NW;   // NW: every role is done with it
    static constexpr int BK = WE + NW;   // NW: its bad_key is there
    static constexpr int kNumBars = BK + NW;
    static constexpr int kOffHalf = (kOffBar + 8 * kNumBars + 15) / 16 * 16;
    static constexpr int kOffWork = kOffHalf + 8 * kRows;  // (its rows' m and l)
    static constexpr int kOffMisc = kOffWork + 64 * NW;
    static constexpr int kSmem = kOffMisc + 256 + 1024;
    static constexpr int kProdK = 8, kMma0 = 9, kProdV = 10;  // (kMma1 = 11)
    static constexpr int kThreads = 12 * 32;
};

struct CSched {
    uint32_t tmem;
    int abort, r0, S;
    long long wsum[12];
    long long c0, c1, base;
    Shares sh;
    Req req;               // request r0's
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
        mbar_init(bar(C::MG), 4);
        for (int k = 0; k < C::NW; ++k) {
            mbar_init(bar(C::WF + k), 1);
            mbar_init(bar(C::WE + k), 11);  // V producer, 2 MMA issuers, 8 softmax warps
            mbar_init(bar(C::BK + k), 1);
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
        long long sum = 0;
        Req mine;  // the thread's last request
        for (int r = i0; r < i1; ++r) {
            mine = load_req(prm, r);
            wrong |= mine.off;
            sum += mine.head * prm.Hkv;
        }
        long long inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += t;
        }
        if (lane == 31) sch->wsum[warp] = inc;
        wrong = __syncthreads_or(wrong);
        long long wex = 0, Wc = 0;
        for (int w = 0; w < C::kThreads / 32; ++w) {
            if (w < warp) wex += sch->wsum[w];
            Wc += sch->wsum[w];
        }
        if (wrong) Wc = 0;
        const int S = (int)max(1LL, min((long long)gridDim.x, Wc / kMinCost));
        Shares sh;
        sh.each = divide(Wc, S);
        sh.rem = (int)(Wc - sh.each * S);
        const int b = blockIdx.x;
        const long long c0 = b < S ? sh.start(b) : Wc, c1 = b < S ? sh.start(b + 1) : Wc;
        long long at = wex + inc - sum;
        if (c0 < c1 && at <= c0 && c0 < at + sum) {
            for (int r = i0; r < i1; ++r) {
                if (per > 1) mine = load_req(prm, r);
                const long long cost = mine.head * prm.Hkv;
                if (at <= c0 && c0 < at + cost) {
                    sch->r0 = r;
                    sch->base = at;
                    sch->req = mine;
                }
                at += cost;
            }
        }
        if (tid == 0) {
            sch->c0 = c0;
            sch->c1 = c1;
            sch->S = S;
            sch->sh = sh;
            prm.cut[blockIdx.x].valid = 0;
            if (wrong && blockIdx.x == 0) report_status(prm.dev_status, BDSA_DEVICE_OUT_OF_RANGE);
        }
        __syncthreads();
    }
    Work *works = reinterpret_cast<Work *>(smem + C::kOffWork);

    if (warp >= 8) {
        if (warp == C::kProdK || warp == C::kProdV) {
            // ------------------------------------------------ TMA producers; K's walks
            // (lane b loads box b of a tile)
            const bool is_k = warp == C::kProdK;
            const int NR = is_k ? C::NK : C::NV, FULL = is_k ? C::KF : C::VF;
            const int EMPTY = is_k ? C::KE : C::VE;
            const uint32_t dst0 = sbase + (is_k ? C::kOffK : C::kOffV) +
                                  (uint32_t)(lane * prm.box_rows * 128);
            const void *tmap = is_k ? (const void *)&tm_k : (const void *)&tm_v;
            const bool loads = lane * prm.box_rows < kBN;
            const int ps = 1 << prm.log2_ps;
            // keys without a page of the pool read as zeros: a row past the
            // cache's last is filled by the load
            const int outside = prm.num_pages << prm.log2_ps;
            const long long c1 = sch->c1;
            Walk walk;
            walk.c = sch->c0;
            if (is_k && walk.c < c1) walk.start(prm, sch->r0, sch->req, sch->base);
            int st = 0;
            uint32_t ph = 1;
            long g = 0;
            int kq[2] = {0, 0};  // pieces each row tile took part in
            bool ok = true;
            auto wait = [&](int i, uint32_t parity) {
                ok = ok && wait_bar(bar(i), parity & 1, abort_flag, prm.dev_status);
                ok = __all_sync(0xffffffffu, ok);
                return ok;
            };
            for (uint32_t k = 0;; ++k) {
                const int ws = k % C::NW;
                volatile Work *w = works + ws;
                if (is_k) {
                    if (k >= C::NW && !wait(C::WE + ws, k / C::NW - 1)) break;
                    Piece pc;
                    const bool more = walk.next(prm, c1, pc);
                    if (lane == 0) {
                        if (more) fill_work(prm, pc, works + ws);
                        else w->all = 0;
                        if (more && pc.a == 0 && pc.e < pc.nt) {  // the unit goes on elsewhere
                            Cut d;
                            d.valid = 1;
                            d.tok0 = pc.tok0;
                            d.ntok = pc.ntok;
                            d.h = pc.h;
                            d.nt = pc.nt;
                            d.S = sch->S;
                            d.key = pc.key;
                            d.cu = pc.cu;
                            d.span = pc.span;
                            d.each = sch->sh.each;
                            d.rem = sch->sh.rem;
                            prm.cut[blockIdx.x] = d;
                        }
                        mbar_arrive(bar(C::WF + ws));
                    }
                    __syncwarp();
                } else if (!wait(C::WF + ws, k / C::NW)) {
                    break;
                }
                const int all = w->all, a0 = w->a;
                if (all == 0) break;
                const int32_t *bt = prm.block_table + (long)w->r * prm.max_pages;
                const int n_keys = w->bad ? 0 : w->L + w->n_new;
                const int col = w->h * D;
                int bad_key = w->bad ? 0 : INT_MAX;
                for (int j = 0; j < all; ++j) {
                    const int t = (a0 + j) * kBN + lane * prm.box_rows;
                    const bool mine = loads && t < n_keys;
                    const int id = mine ? __ldg(bt + (t >> prm.log2_ps)) : -1;
                    const bool in = id >= 0 && id < prm.num_pages;
                    const int slot = in ? id * ps + (t & (ps - 1)) : outside;
                    if (mine && !in) bad_key = min(bad_key, t);
                    if (!wait(EMPTY + st, ph)) break;
                    if (lane == 0) mbar_arrive_expect_tx(bar(FULL + st), (uint32_t)C::kTile);
                    __syncwarp();
                    if (loads) {
#pragma unroll
                        for (int c = 0; c < C::DH; ++c)
                            tma_load_2d(dst0 + st * C::kTile + c * C::kSlab, tmap, col + c * 64,
                                        slot, bar(FULL + st));
                    }
                    ++g;
                    if (++st == NR) {
                        st = 0;
                        ph ^= 1;
                    }
                    if (is_k && j == 0) {  // (the first K tile needs no wait for Q)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            if (!ok || w->n[x] == 0) continue;
                            if (kq[x] > 0 && !wait(C::QE + x, kq[x] - 1)) continue;
                            if (lane == 0) {
                                mbar_arrive_expect_tx(bar(C::QF + x), (uint32_t)(rows * D * 2));
                                for (int c = 0; c < C::DH; ++c)
                                    tma_load_4d(sbase + C::kOffQ + x * C::kTile + c * C::kSlab,
                                                &tm_q, c * 64, 0, w->h,
                                                w->tok0 + (w->split ? 0 : x * prm.npt),
                                                bar(C::QF + x));
                            }
                            ++kq[x];
                        }
                        if (!ok) break;
                    }
                }
                if (!ok) break;
                if (is_k) {
                    bad_key = __reduce_min_sync(0xffffffffu, bad_key);
                    if (lane == 0) {
                        w->bad_key = bad_key;
                        mbar_arrive(bar(C::BK + ws));
                    }
                } else if (lane == 0) {
                    mbar_arrive(bar(C::WE + ws));
                }
                __syncwarp();
            }
            // Drain: the last load issued into each buffer has landed.
            if (lane == 0) {
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    if (is_k && kq[x] > 0) mbar_wait_drain(bar(C::QF + x), (kq[x] - 1) & 1);
                for (long i = max(0L, g - NR); i < g; ++i)
                    mbar_wait_drain(bar(FULL + (int)(i % NR)), (uint32_t)((i / NR) & 1));
            }
            __syncwarp();
        } else {
            // ------------------------------------------------ MMA issuers, one a row tile
            // The whole warp takes each piece and one elected lane issues: an
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
                ok = ok && wait_bar(bar(i), parity & 1, abort_flag, prm.dev_status);
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
                                 (first && part == 0 && k4 == 0) ? 0u : 1u);
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
            // a tile that this row tile does not take: only its release
            auto pass_k = [&] {
                wait(C::KF + ks, kph);
                if (!ok) return;
                if (leader) mbar_arrive(bar(C::KE + ks));
                if (++ks == C::NK) {
                    ks = 0;
                    kph ^= 1;
                }
            };
            auto pass_v = [&] {
                wait(C::VF + vs, vph);
                if (!ok) return;
                if (leader) mbar_arrive(bar(C::VE + vs));
                if (++vs == C::NV) {
                    vs = 0;
                    vph ^= 1;
                }
            };
            for (uint32_t k = 0;; ++k) {
                const int ws = k % C::NW;
                wait(C::WF + ws, k / C::NW);
                if (!ok) break;
                const int n = works[ws].n[t], all = works[ws].all;
                const bool split = works[ws].split != 0;
                if (all == 0) break;
                __syncwarp();
                if (leader) mbar_arrive(bar(C::WE + ws));
                const int first = split ? t : 0;
                if (n > 0) {
                    if (first) pass_k();
                    // step j: PV of tile j (none at -1), then S of tile j + 1
#pragma unroll 1
                    for (int j = -1; j < n; ++j) {
                        const bool more = j + 1 < n;
                        if (j >= 0) {
                            wait(C::VF + vs, vph);
                            if (j == 0 && kt > 0) wait(C::OE + t, kt - 1);
                        }
#pragma unroll 1
                        for (int part = 0; part < 2; ++part) {
                            if (j >= 0) {
                                wait(C::PF + 2 * t + part, gt);
                                if (!ok) break;
                                tc_fence_after();
                                issue_pv(vs, part, j == 0);
                            }
                            if (part == 0 && more) {
                                if (split && j >= 0) pass_k();
                                wait(C::KF + ks, kph);
                                if (j < 0) wait(C::QF + t, kt);
                            }
                        }
                        if (!ok) break;
                        if (more) {
                            tc_fence_after();
                            issue_s(ks);
                            if (j + 2 == n) commit(C::QE + t);
                        } else {
                            commit(C::OF + t);
                        }
                        if (j >= 0) {
                            next_v();
                            ++gt;
                        }
                        if (more) {
                            next_k();
                            if (split && (t == 1 || j >= 0)) pass_v();
                        }
                    }
                    ++kt;
                }
                // (K before V, tile by tile: the rings move together)
                const int past = n > 0 ? first + (n - 1) * (split ? 2 : 1) + 1 : 0;
                for (int j = past; ok && j < all; ++j) {
                    pass_k();
                    pass_v();
                }
                if (!ok) break;
            }
            commit(C::DR + t);
            mbar_wait_drain(bar(C::DR + t), 0);
        }
    } else {
        // ------------------------------------------------ softmax + epilogue
        const int t = warp >> 2;                       // row tile
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lane_base + kS + t * 128;
        const uint32_t o_addr = tmem + lane_base + kO + t * 128;
        const float sl2 = prm.scale_log2;
        uint32_t gs = 0, k = 0;
        uint32_t turn = 0;  // tiles that both row tiles took
        uint32_t halves = 0;  // split pairs
        int vs0 = 0;        // V ring position and phase of the piece's first tile
        uint32_t vph0 = 0;
        float2 *half = reinterpret_cast<float2 *>(smem + C::kOffHalf);
        bool ok = true;
        for (uint32_t piece = 0;; ++piece) {
            const int ws = piece % C::NW;
            ok = wait_bar(bar(C::WF + ws), (piece / C::NW) & 1, abort_flag, prm.dev_status);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || works[ws].all == 0) break;
            // (read where it is used: kept in registers across the tiles it costs spills)
            const volatile Work &w = works[ws];
            const int n = w.n[t], n_keys = w.L + w.n_new, nboth = w.nboth;
            const bool split = w.split != 0;
            // keys this row sees (rows that are nobody's: all, nothing to mask)
            int lim = INT_MAX;
            if (row < rows) {
                const int token = (split ? 0 : t * prm.npt) + row / prm.G;
                if (token < w.ntok) lim = limit_of(prm, w.L, w.n_new, w.i0 + token);
            }
            int vi = vs0 + (split ? t : 0);                      // the tile's place in the ring
            int t0 = (w.a + (split ? t : 0)) * kBN;              // its first key
            const int step = split ? 2 : 1;
            float m_used = -INFINITY;
            uint64_t lacc[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
            for (int j = 0; j < n; ++j, ++gs, vi += step, t0 += step * kBN) {
                ok = mbar_wait(bar(C::SF + t), gs & 1, abort_flag, prm.dev_status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                // ---- scores of keys that a row does not see become -inf
                const int nvis = lim - t0;
                if (__builtin_expect(__any_sync(0xffffffffu, nvis < kBN), 0)) {
#pragma unroll 1
                    for (int b = 0; b < kBN; b += 32) {
                        if (!__any_sync(0xffffffffu, nvis < b + 32)) continue;
                        float sv[32];
                        tmem_ld32(s_addr + b, sv);
                        tmem_wait_ld();
                        const int left = nvis - b;
#pragma unroll
                        for (int c = 0; c < 32; ++c) sv[c] = c < left ? sv[c] : -INFINITY;
                        tmem_st32(s_addr + b, sv);
                    }
                    tmem_wait_st();
                }
                // ---- the maximum (S is read twice: 128 scores a thread held over both
                // passes are half of its registers, and code of four times the size)
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int b = 0; b < kBN; b += 64) {
                    float sv[64];
                    tmem_ld32(s_addr + b, *reinterpret_cast<float(*)[32]>(&sv[0]));
                    tmem_ld32(s_addr + b + 32, *reinterpret_cast<float(*)[32]>(&sv[32]));
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 64; c += 2)
                        mx[(c >> 1) & 3] = max3f(mx[(c >> 1) & 3], sv[c], sv[c + 1]);
                }
                const float m_new = fmaxf(max3f(mx[0], mx[1], mx[2]), mx[3]) * sl2;
                float alpha = 1.f;
                bool resc = false;
                if (m_new > m_used + kRescaleLog2) {
                    alpha = ex2_approx(m_used - m_new);
                    m_used = m_new;
                    resc = true;
                }
                if (__builtin_expect(__any_sync(0xffffffffu, resc), 0)) {
                    const uint64_t a2 = f2_pack(alpha, alpha);
                    lacc[0] = f2_mul(lacc[0], a2);
                    lacc[1] = f2_mul(lacc[1], a2);
                    // (S of this tile was issued after PV of the last one, and
                    // its barrier covers both: O is complete)
                    if (j > 0) {
#pragma unroll 1
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
                if (__builtin_expect(t0 + kBN > n_keys, 0)) {
                    const int vs = vi % C::NV;
                    ok = mbar_wait(bar(C::VF + vs), (vph0 + (uint32_t)(vi / C::NV)) & 1,
                                   abort_flag, prm.dev_status);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const int valid = n_keys - t0;
                    for (int idx = row; idx < C::DH * 8 * (kBN - valid); idx += kRows) {
                        const int u = idx & 7, rr = idx >> 3;
                        const int slab = rr >= kBN - valid ? 1 : 0;
                        const int m = valid + rr - slab * (kBN - valid);
                        st_shared_v4(sbase + C::kOffV + vs * C::kTile + slab * C::kSlab + m * 128 +
                                         u * 16,
                                     0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                // (the next 32 scores are on their way while these become P)
                float sv[2][32];
                tmem_ld32(s_addr, sv[0]);
                // The row tiles' exponentials in turn: at the same time each takes about
                // twice as long, and then both row tiles' MMAs come at once and nothing
                // overlaps (the prompts 418 us instead of 353; with the turn handed on
                // after a quarter, a half, three quarters of them 393, 382, 375).
                const bool both = j < nboth;
                if (both && (t == 1 || turn > 0)) {
                    ok = mbar_wait(bar(C::TK + t), (t == 1 ? turn : turn - 1) & 1, abort_flag,
                                   prm.dev_status);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                }
                const float neg_m = m_used == -INFINITY ? 0.f : -m_used;
                const uint64_t sc2 = f2_pack(sl2, sl2), nm2 = f2_pack(neg_m, neg_m);
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t pk[16];
                        tmem_wait_ld();
                        if (h + c < 2) tmem_ld32(s_addr + h * 64 + c * 32 + 32, sv[1 - c]);
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            const float2 xv = f2_unpack(
                                f2_fma(f2_pack(sv[c][2 * q], sv[c][2 * q + 1]), sc2, nm2));
                            const float p0 = ex2_approx(xv.x), p1 = ex2_approx(xv.y);
                            pk[q] = pack_bf16x2(p0, p1);
                            lacc[q & 1] = f2_add(lacc[q & 1], f2_pack(p0, p1));
                        }
                        tmem_st16(s_addr + h * 32 + c * 16, pk);
                    }
                    // half of P: its PV may start
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::PF + 2 * t + h));
                }
                if (both) {
                    if (lane == 0) mbar_arrive(bar(C::TK + 1 - t));
                    ++turn;
                }
            }
            if (!ok) break;
            vs0 += w.all;
            vph0 += (uint32_t)(vs0 / C::NV);
            vs0 %= C::NV;
            // ---- end of the piece: o / l and the log2-sum-exp
            if (n > 0) {
                ok = wait_bar(bar(C::OF + t), k & 1, abort_flag, prm.dev_status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                ++k;
            }
            const float2 la = f2_unpack(lacc[0]), lb = f2_unpack(lacc[1]);
            float l = (la.x + la.y) + (lb.x + lb.y);
            float w0 = 1.f, w1 = 0.f;  // weights of the halves of a split pair
            if (split) {
                if (t == 1) {  // its half stays in TMEM for row tile 0
                    half[row] = make_float2(m_used, l);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(C::MG));
                        mbar_arrive(bar(C::WE + ws));
                    }
                    continue;
                }
                ok = wait_bar(bar(C::MG), halves & 1, abort_flag, prm.dev_status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                ++halves;
                const float2 o = half[row];
                const float mm = fmaxf(m_used, o.x);
                w0 = m_used == -INFINITY ? 0.f : ex2_approx(m_used - mm);
                w1 = o.x == -INFINITY ? 0.f : ex2_approx(o.x - mm);
                l = l * w0 + o.y * w1;
                m_used = mm;
            }
            ok = wait_bar(bar(C::BK + ws), (piece / C::NW) & 1, abort_flag, prm.dev_status);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const bool hit = w.bad_key < lim;
            const float inv = l > 0.f ? rcp_approx(l) : isnan(l) ? l : 0.f;
            const float l2 = l > 0.f ? m_used + lg2_approx(l) : isnan(l) ? l : -INFINITY;
            w0 = hit ? 0.f : w0 * inv;
            w1 = hit ? 0.f : w1 * inv;
            const int token = (split ? 0 : t * prm.npt) + row / prm.G;
            const bool real = lim != INT_MAX, whole = w.whole != 0;
            const long at = (long)(w.tok0 + token) * prm.Hq + (long)w.h * prm.G + row % prm.G;
            const long dst =
                ((long)blockIdx.x * 2 + (w.a == 0 ? 1 : 0)) * 2 * kRows + t * kRows + row;
            float *ps = prm.slot_o + dst * D;
            uint16_t *po = prm.out + at * D;
#pragma unroll 1
            for (int c = 0; n > 0 && c < D; c += 16) {
                float ov[16];
                tmem_ld16(o_addr + c, ov);
                if (split) {
                    float o1[16];
                    tmem_ld16(o_addr + 128 + c, o1);
                    tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < 16; ++q) ov[q] = ov[q] * w0 + o1[q] * w1;
                } else {
                    tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < 16; ++q) ov[q] *= w0;
                }
                if (!real) continue;
                if (whole) {
                    uint32_t pk[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        pk[q] = hit ? 0u : pack_bf16x2(ov[2 * q], ov[2 * q + 1]);
                    if (prm.wide) {  // a whole sector
                        st_global_v8(po + c, pk[0], pk[1], pk[2], pk[3], pk[4], pk[5], pk[6],
                                     pk[7]);
                    } else {
                        *reinterpret_cast<uint4 *>(po + c) =
                            make_uint4(pk[0], pk[1], pk[2], pk[3]);
                        *reinterpret_cast<uint4 *>(po + c + 8) =
                            make_uint4(pk[4], pk[5], pk[6], pk[7]);
                    }
                } else {
#pragma unroll
                    for (int v = 0; v < 16; v += 8)
                        st_global_v8(ps + c + v, __float_as_uint(ov[v]),
                                     __float_as_uint(ov[v + 1]), __float_as_uint(ov[v + 2]),
                                     __float_as_uint(ov[v + 3]), __float_as_uint(ov[v + 4]),
                                     __float_as_uint(ov[v + 5]), __float_as_uint(ov[v + 6]),
                                     __float_as_uint(ov[v + 7]));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (n > 0) mbar_arrive(bar(C::OE + t));
                if (split) mbar_arrive(bar(C::OE + 1));
                mbar_arrive(bar(C::WE + ws));
            }
            if (real) {
                // +inf marks a row of a partial that sees a key without a page; a NaN
                // score leaves NaN
                if (!whole) prm.slot_lse[dst] = hit ? INFINITY : l2;
                else if (prm.lse != nullptr) prm.lse[at] = hit ? -INFINITY : l2 * kLn2;
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
        const long long end = Shares{d.each, d.rem}.start(b + k + 1);
        const bool done = b + k >= d.S - 1 || tile_at(end - d.cu, d.span, d.nt, d.key) >= d.nt;
        const uint32_t m = __ballot_sync(0xffffffffu, done);
        if (m != 0) np = k0 + __ffs(m);  // pieces: this CTA's and those up to that one
    }
    auto slot = [&](int i) { return ((long)(b + i) * 2 + (i == 0 ? 1 : 0)) * 2 * kRows + row; };
    // lane `sub` of a row reads the log2-sum-exps of pieces sub, sub + 8, ..
    auto lse_of = [&](int i) {
        return real && i < np ? __ldcg(prm.slot_lse + slot(i)) : -INFINITY;
    };
    const float first = lse_of(sub);
    float mx = -INFINITY;
    bool hit = false, nan = false;
    for (int i = sub; i < np; i += 8) {
        const float v = i == sub ? first : lse_of(i);
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
    constexpr int W = D / 8;  // values a thread
    float acc[W], sum = 0.f;
#pragma unroll
    for (int c = 0; c < W; ++c) acc[c] = 0.f;
    const bool some = real && !hit && !nan && mx > -INFINITY;
    for (int i0 = 0; i0 < np; i0 += 8) {
        const float v = i0 == 0 ? first : lse_of(i0 + sub);
        const float wv = some && v > -INFINITY ? ex2_approx(v - mx) : 0.f;
#pragma unroll 4
        for (int j = 0; j < min(8, np - i0); ++j) {
            const float w = __shfl_sync(0xffffffffu, wv, (lane & ~7) + j);
            if (w == 0.f) continue;  // (its o may not have been written)
            const float *po = prm.slot_o + slot(i0 + j) * D + sub * W;
            float ov[W];
#pragma unroll
            for (int c = 0; c < W; c += 8) ld_cg_v8(po + c, ov + c);
            sum += w;
#pragma unroll
            for (int c = 0; c < W; ++c) acc[c] = fmaf(w, ov[c], acc[c]);
        }
    }
    if (!real) return;
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
    p.wide = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
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
