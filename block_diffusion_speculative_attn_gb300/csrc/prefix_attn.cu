// prefix_attn.cu -- attention of a group's stacked query rows over the prefix
// its requests share, for sm_103a.
//
// For every group, KV head and query row the softmax is cut at key P' (a whole
// number of 128-key tiles):
//   softmax over [0, L + B) = join of  (o1, lse1) over [0, P')   this kernel
//                             and      (o2, lse2) over [P', ..)  block_attn.cu
// with o = (o1 e^{lse1 - m} + o2 e^{lse2 - m}) / (e^{lse1 - m} + e^{lse2 - m}).
// The keys below P' are the same for the whole group and visible to every row,
// so the rows of all its requests form one tall matrix per KV head and the
// prefix is one unmasked attention over it: K and V are read once for the group
// instead of once a request, and the work turns from memory bound to tensor
// bound.
//
// Shape of the work (attn_prefix.cuh): a unit is 256 rows (two 128-row tiles)
// of one (group, KV head) over all P' / 128 key tiles; units are concatenated
// and persistent CTAs take equal cost ranges.  A piece leaves its rows' o / l
// and log2-sum-exp in fp32.
//
// A team of two CTAs takes two units' rows over the same keys, each loading every
// tile for itself: they are at the same keys at about the same time, so that those
// come from HBM once a team.
//
// Inside a CTA (12 warps): warps 0-3 and 4-7 are the softmax of the two row
// tiles, one thread a row; then a K producer (also Q), a V producer and an MMA
// issuer for each row tile (one issuer for both spent more time on its waits,
// commits and descriptors than the tensor cores on the MMAs).  A row tile's S
// (128 columns of TMEM) is read by its softmax, which
// writes P as bf16 over it; PV takes P from TMEM.  The two tiles alternate on
// the tensor cores -- while one tile's PV and next S run (1024 cycles at D =
// 128), the other's softmax runs on the ALUs -- and share every K and V tile in
// shared memory.  O is rescaled in TMEM only when a row's max grows by 2^8.
//
// Measured, with the block kernel behind it: 8 verify requests of 16 tokens and 64
// heads over 131072 shared keys 362 us for 554 GFLOP when the GPU is cool, 368-392 us
// call after call, 1.41-1.53 PFLOP/s (0.74 to 0.80 of the measured bf16 rate), a key
// tile of a pair every 1.6 us: a row tile's chain of S, its maximum, the
// exponentials and P is longer than the other tile's MMAs.  32 requests of 16 tokens
// and 32 heads over 4096 keys 69 us (every key attended by every request itself: 86
// us), 64 single tokens over 2048 keys 63 us (119): there the start, a piece's end
// and the block kernel's short units count.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <limits.h>

#include "attn_common.cuh"
#include "attn_prefix.cuh"
#include "bdsa_device.cuh"
#include "bdsa_internal.h"

namespace bdsa {
namespace {

template <int D>
struct PCfg {
    static constexpr int DH = D / 64;                 // 128-byte slabs of a row
    static constexpr int kSlab = kPrefixRows * 128;   // one slab of a 128-row tile
    static constexpr int kTile = DH * kSlab;          // a Q, K or V tile
    // K is held until both tiles' S, V until both tiles' PV, about a tile
    // longer
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
    static constexpr int kSmem = kOffMisc + 448 + 1024;
    // a K producer (also Q), an MMA issuer for each row tile, a V producer
    static constexpr int kProdK = 8, kMma0 = 9, kProdV = 10;  // (kMma1 = 11)
    static constexpr int kThreads = 12 * 32;
    // Registers a thread: 168 at launch (12 warps of 65536 / 384), moved from
    // the producers' warpgroup to the softmax ones, whose 128 scores a thread
    // spill otherwise: 256 * 208 + 128 * 80 <= 384 * 168.
    static constexpr int kSoftmaxRegs = 208, kProducerRegs = 80;
    static_assert(256 * kSoftmaxRegs + 128 * kProducerRegs <= kThreads * 168, "register split");
};

struct PSched {
    uint32_t tmem;
    int abort;
    long long wsum[12], wsum2[2][12];
    int T, member, S;      // CTAs a team, this one's place, teams
    long long Wc;
    long long c0, c1;      // this CTA's cost range
    long long gbase;       // cost offset of the group holding c0
    int g0;
};
static_assert(sizeof(PSched) <= 448, "the schedule state has 448 bytes");

struct PParams {
    PrefixParams x;
    const int32_t *block_table;
    int32_t *dev_status;
    int max_pages, num_pages, B, Hq, Hkv, G, log2_ps, box_rows;
    float scale_log2;
};

// A run of one unit's key tiles inside a CTA's range.
struct PPiece {
    int r0, tok0, ntok;   // the group's first request; this unit's first token, tokens left
    int h, a, e, nt;      // KV head, tiles [a, e) of nt
    long long last;       // the cost of the unit's last tile
};

// Walks the pieces of a cost range, group by group.
struct PWalk {
    int g;
    long long base;       // cost offset of group g
    int r0, tokens, nt, units;
    int T, member;
    long long c;          // next cost
    __device__ void load(const PParams &p) {
        group_shape(p.x, g, p.B, r0, tokens, nt);
        units = group_units(p.x, tokens, T);
    }
    // The next piece, or false at the end of the range.
    __device__ bool next(const PParams &p, long long c1, PPiece &pc) {
        while (c < c1) {
            const long long span = kPrefixUnitCost + nt;
            const long long gcost = nt > 0 ? span * p.Hkv * units : 0;
            if (c >= base + gcost) {
                if (++g >= p.x.ng) return false;
                base += gcost;
                load(p);
                continue;
            }
            const long long u = (c - base) / span;
            const long long cu = base + u * span, lo = c - cu, hi = min(c1 - cu, span);
            c = cu + hi;
            const int a = (int)max(0LL, lo - kPrefixUnitCost);
            const int e = (int)max(0LL, hi - kPrefixUnitCost);
            if (a >= e) continue;
            const int pair = (int)(u % units) * T + member;
            pc.h = (int)(u / units);
            pc.r0 = r0;
            pc.tok0 = r0 * p.B + pair * 2 * p.x.npt;
            pc.ntok = tokens - pair * 2 * p.x.npt;
            if (pc.ntok <= 0) continue;  // no tokens left for this member
            pc.a = a;
            pc.e = e;
            pc.nt = nt;
            pc.last = cu + span - 1;
            return true;
        }
        return false;
    }
};

// A (in TMEM, bf16 pairs) x B (shared memory).
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// One lane of the (converged) warp, always the same.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// 16 consecutive 32-bit columns of the thread's lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
        "r"(v[15])
        : "memory");
}

template <int D>
__global__ void __launch_bounds__(PCfg<D>::kThreads, 1)
    prefix_attn_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const PParams prm) {
    using C = PCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (sbase - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto bar = [&](int i) -> uint32_t { return sbase + C::kOffBar + 8u * (uint32_t)i; };
    PSched *sch = reinterpret_cast<PSched *>(smem + C::kOffMisc);
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
        }
        for (int k = 0; k < C::NK; ++k) {
            mbar_init(bar(C::KF + k), 1);
            mbar_init(bar(C::KE + k), 2);
        }
        for (int k = 0; k < C::NV; ++k) {
            mbar_init(bar(C::VF + k), 1);
            mbar_init(bar(C::VE + k), 2);
        }
        mbar_init(bar(C::DR), 1);
        mbar_init(bar(C::DR + 1), 1);
        mbar_init(bar(C::TK), 4);
        mbar_init(bar(C::TK + 1), 4);
        *abort_flag = 0;
        fence_mbarrier_init();
    }
    if (warp == C::kProdK && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
    }
    if (warp == C::kProdV && lane == 0) tma_prefetch_desc(&tm_v);
    // rows of a tile past its whole tokens stay zero
    const int rows = prm.G * prm.x.npt;
    for (int idx = tid; idx < 2 * C::DH * (kPrefixRows - rows) * 8; idx += C::kThreads) {
        const int u = idx & 7, pad = kPrefixRows - rows;
        const int m = rows + (idx >> 3) % pad, slab = (idx >> 3) / pad;
        st_shared_v4(sbase + C::kOffQ + slab * C::kSlab + m * 128 + u * 16, 0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sch->tmem;

    // ---- everything before this call on the stream has finished; the block
    // attention of this call may launch (it reads only inputs, and waits for
    // this grid before it reads the partials)
    grid_dependency_wait();
    grid_launch_dependents();

    // ---- schedule: a scan of the groups' costs
    {
        const int ng = prm.x.ng;
        const int per = (ng + C::kThreads - 1) / C::kThreads;
        const int i0 = min(ng, tid * per), i1 = min(ng, i0 + per);
        auto cost = [&](int g, int T) -> long long {
            int r0, tokens, nt;
            group_shape(prm.x, g, prm.B, r0, tokens, nt);
            return nt > 0 ? (long long)(kPrefixUnitCost + nt) * prm.Hkv *
                                group_units(prm.x, tokens, T)
                          : 0;
        };
        // offsets that do not run up from 0 to bs place nothing: no work, and
        // the block attention writes zeros
        bool wrong = false;
        long long sum2[2] = {0, 0};  // costs by teams of 1 and of 2
        for (int g = i0; g < i1; ++g) {
            sum2[0] += cost(g, 1);
            sum2[1] += cost(g, 2);
            const int o0 = __ldg(prm.x.group_offsets + g), o1 = __ldg(prm.x.group_offsets + g + 1);
            wrong |= o1 < o0 || (g == 0 && o0 != 0) || (g == ng - 1 && o1 != prm.x.bs);
        }
        wrong = __syncthreads_or(wrong);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            long long v = sum2[k];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == 0) sch->wsum2[k][warp] = v;
        }
        __syncthreads();
        long long c1s = 0, c2s = 0;
        for (int w = 0; w < C::kThreads / 32; ++w) {
            c1s += sch->wsum2[0][w];
            c2s += sch->wsum2[1][w];
        }
        // Teams of two unless the pairs they leave without a partner cost more
        // than 1/16 (131072 shared keys: 389 us, teams of one 428; 32 requests of 16
        // tokens behind 4096: 70 against 71.5; with 64 single tokens behind 2048 half
        // of the CTAs would be without work: 79 against 63).
        const int T = gridDim.x >= 2 && 2 * c2s <= c1s + c1s / 16 ? 2 : 1;
        const long long Wc = T == 2 ? c2s : c1s;
        long long sum = 0;
        for (int g = i0; g < i1; ++g) sum += cost(g, T);
        long long inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += t;
        }
        if (lane == 31) sch->wsum[warp] = inc;
        __syncthreads();
        long long wex = 0;
        for (int w = 0; w < warp; ++w) wex += sch->wsum[w];
        const long long S = max(1LL, min((long long)(gridDim.x / T), Wc / kPrefixMinCost));
        const long long b = blockIdx.x / T;
        const bool mine = b < S && !wrong;
        const long long c0 = mine ? prefix_range_start(b, Wc, S) : Wc;
        const long long c1 = mine ? prefix_range_start(b + 1, Wc, S) : Wc;
        long long at = wex + inc - sum;
        for (int g = i0; g < i1; ++g) {
            const long long cg = cost(g, T);
            if (at <= c0 && c0 < at + cg) {
                sch->g0 = g;
                sch->gbase = at;
            }
            at += cg;
        }
        if (tid == 0) {
            sch->c0 = c0;
            sch->c1 = c1;
            sch->T = T;
            sch->S = (int)S;
            sch->Wc = Wc;
            sch->member = blockIdx.x % T;
            if (blockIdx.x == 0) {
                prm.x.head[0] = wrong ? -1 : T;
                if (wrong) report_status(prm.dev_status, BDSA_DEVICE_OUT_OF_RANGE);
            }
        }
        __syncthreads();
    }
    const long long c1 = sch->c1;
    PWalk walk;
    walk.c = sch->c0;
    walk.T = sch->T;
    walk.member = sch->member;
    if (walk.c < c1) {
        walk.g = sch->g0;
        walk.base = sch->gbase;
        walk.load(prm);
    }
    PPiece pc;

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
                const long ps = 1L << prm.log2_ps;
                long g = 0;
                int kq[2] = {0, 0};  // pieces each row tile took part in
                bool ok = true;
                while (ok && walk.next(prm, c1, pc)) {
                    if (is_k) {
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (!ok || t * prm.x.npt >= pc.ntok) break;
                            if (kq[t] > 0)
                                ok = mbar_wait(bar(C::QE + t), (kq[t] - 1) & 1, abort_flag,
                                               prm.dev_status);
                            if (!ok) break;
                            mbar_arrive_expect_tx(bar(C::QF + t), (uint32_t)(rows * D * 2));
                            for (int c = 0; c < C::DH; ++c)
                                tma_load_4d(sbase + C::kOffQ + t * C::kTile + c * C::kSlab, &tm_q,
                                            c * 64, 0, pc.h, pc.tok0 + t * prm.x.npt,
                                            bar(C::QF + t));
                            ++kq[t];
                        }
                        if (!ok) break;
                    }
                    const int32_t *bt = prm.block_table + (long)pc.r0 * prm.max_pages;
                    for (int j = pc.a; j < pc.e; ++j, ++g) {
                        const long t0 = (long)j * kBN;
                        // pages past the row (reported by the softmax) load nothing
                        int32_t slot[kMaxBoxes];
#pragma unroll
                        for (int bx = 0; bx < kMaxBoxes; ++bx) {
                            if (bx >= nbox) break;
                            const long t = t0 + (long)bx * rows_box;
                            const long page = t >> prm.log2_ps;
                            const int32_t id = page < prm.max_pages ? __ldg(bt + page) : -1;
                            slot[bx] = id >= 0 && id < prm.num_pages
                                           ? (int32_t)(id * ps + (t & (ps - 1)))
                                           : 0;
                        }
                        const int st = (int)(g % NR);
                        ok = mbar_wait(bar(EMPTY + st), (uint32_t)(((g / NR) & 1) ^ 1), abort_flag,
                                       prm.dev_status);
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
            {
                const int t = warp == C::kMma0 ? 0 : 1;
                const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0) + t * 128;
                const bool leader = elect_one();
                constexpr uint32_t idesc_qk = idesc_bf16_f32(kPrefixRows, kBN, 0, 0);
                constexpr uint32_t idesc_pv = idesc_bf16_f32(kPrefixRows, D, 0, 1);
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
                    const int n = pc.e - pc.a;
                    if (t * prm.x.npt >= pc.ntok) {
                        // no tokens in this row tile: its share of the rings' releases
                        for (int j = 0; ok && j < n; ++j) {
                            wait(C::KF + ks, kph);
                            if (ok) next_k();
                            wait(C::VF + vs, vph);
                            if (ok) next_v();
                        }
                        continue;
                    }
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
                commit(C::DR + t);
                mbar_wait_drain(bar(C::DR + t), 0);
            }
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
        long gs = 0;
        int k = 0;
        uint32_t turn = 0;  // tiles that both row tiles took
        bool ok = true, first_piece = true;
        while (ok && walk.next(prm, c1, pc)) {
            const bool slot0 = first_piece && pc.a > 0;  // continues an earlier CTA's unit
            first_piece = false;
            if (t * prm.x.npt >= pc.ntok) continue;      // no tokens in this row tile
            // page ids of the piece: any outside the pool makes it a bad one
            bool bad = false;
            {
                const long p0 = ((long)pc.a * kBN) >> prm.log2_ps;
                const long p1 = ((long)pc.e * kBN - 1) >> prm.log2_ps;
                const int32_t *bt = prm.block_table + (long)pc.r0 * prm.max_pages;
                for (long p = p0 + lane; p <= p1; p += 32) {
                    const int32_t id = p < prm.max_pages ? __ldg(bt + p) : -1;
                    bad |= id < 0 || id >= prm.num_pages;
                }
                bad = __any_sync(0xffffffffu, bad);
            }
            const bool both = prm.x.npt < pc.ntok;       // both row tiles have tokens
            float m_used = -INFINITY;
            uint64_t lacc[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
            for (int j = pc.a; j < pc.e; ++j, ++gs) {
                ok = mbar_wait(bar(C::SF + t), (uint32_t)(gs & 1), abort_flag, prm.dev_status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                float sv[128];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_ld32(s_addr + c * 32, *reinterpret_cast<float(*)[32]>(&sv[c * 32]));
                tmem_wait_ld();
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
                    if (j > pc.a) {
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
                // The row tiles' exponentials in turn: at the same time each takes
                // twice as long (the special function unit is shared), and then
                // both row tiles' MMAs come at once and nothing overlaps.
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
            // ---- end of the piece: o / l and the log2-sum-exp
            const uint32_t team = blockIdx.x / sch->T;
            const uint32_t teams =
                team << 16 | (pc.e == pc.nt ? team
                                            : (uint32_t)prefix_team_of(pc.last, sch->Wc, sch->S));
            ok = mbar_wait(bar(C::OF + t), (uint32_t)(k & 1), abort_flag, prm.dev_status);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const float2 la = f2_unpack(lacc[0]), lb = f2_unpack(lacc[1]);
            const float l = (la.x + la.y) + (lb.x + lb.y);
            const float inv = l > 0.f ? 1.f / l : 0.f;
            const int token = t * prm.x.npt + node;
            const bool real = row < rows && token < pc.ntok;
            const long dst = slot0 ? (long)blockIdx.x * 2 * kPrefixRows + t * kPrefixRows + row
                                   : (long)(pc.tok0 + token) * prm.Hq + (long)pc.h * prm.G +
                                         row % prm.G;
            float *po = (slot0 ? prm.x.slot_o : prm.x.row_o) + dst * D;
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
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::OE + t));
            // a bad piece is marked by +inf; a NaN score leaves NaN
            if (real) {
                (slot0 ? prm.x.slot_lse : prm.x.row_lse)[dst] =
                    bad ? INFINITY : l > 0.f ? m_used + log2f(l) : isnan(l) ? l : -INFINITY;
                if (!slot0) prm.x.row_teams[dst] = teams;
            }
            if (bad && lane == 0) report_status(prm.dev_status, BDSA_DEVICE_OUT_OF_RANGE);
            ++k;
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

template <int D>
int launch_partials(const AttnArgs &a, const PrefixParams &x, int grid, cudaStream_t stream) {
    using C = PCfg<D>;
    static_assert(C::kSmem <= 227 * 1024, "shared memory of one CTA");
    EncodeTiledFn enc = encode_fn();
    if (enc == nullptr) return BDSA_CUDA_ERROR;
    const int G = a.Hq / a.Hkv;
    CUtensorMap tq, tk, tv;
    {
        // q as (d, head of the group, KV head, token); a box is one row tile
        cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)G, (cuuint64_t)a.Hkv,
                              (cuuint64_t)a.bs * a.B};
        cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)G * D * 2,
                                 (cuuint64_t)a.Hq * D * 2};
        cuuint32_t box[4] = {64, (cuuint32_t)G, 1, (cuuint32_t)x.npt};
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
    PParams p;
    p.x = x;
    p.block_table = a.block_table;
    p.dev_status = a.dev_status;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = G;
    int lg = 0;
    while ((1 << lg) < a.page_size) ++lg;
    p.log2_ps = lg;
    p.box_rows = box_rows;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    if (cudaFuncSetAttribute(prefix_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmem) != cudaSuccess)
        return BDSA_CUDA_ERROR;
    return launch_pdl(prefix_attn_kernel<D>, dim3(grid), dim3(C::kThreads),
                      (size_t)C::kSmem, stream, tq, tk, tv, p) == cudaSuccess
               ? BDSA_OK
               : BDSA_CUDA_ERROR;
}

}  // namespace

int launch_prefix_partials(const AttnArgs &a, const PrefixParams &x, int grid,
                           cudaStream_t stream) {
    return a.D == 128 ? launch_partials<128>(a, x, grid, stream)
                      : launch_partials<64>(a, x, grid, stream);
}

}  // namespace bdsa
