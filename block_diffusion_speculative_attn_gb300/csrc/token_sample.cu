// token_sample.cu -- logits to the distribution that the acceptance calls read,
// and a token drawn from it.
//
// For a row l of V logits with temperature T, top-k k, top-p p, min-p m:
//   w_i = exp((l_i - max l) / T);  order: value descending, index ascending
//   kept = the first n of the order, n = max(1, min(n_k, n_p, n_m)) with
//     n_k = k, n_p = the shortest prefix whose weight reaches p times the weight
//     of the first n_k, n_m = the weights >= m
//   probs_i = w_i / S on the kept indices, 0 elsewhere (S = their weight)
//   token   = the smallest kept index whose cumulative weight, in index order,
//             exceeds u * S (the draw rule of the acceptance calls)
//
// Arithmetic.  Every weight is held as a 64-bit integer in units of 2^-41 of
// the row's largest weight, from an exponential good to about 2^-39 (a table of
// 2^(j/128) and a short series on the float-float remainder).  Integer sums are
// exact in any order, so the partial sums of threads, warps and CTAs combine
// freely (shared-memory atomics among them) and a row gives the same answer
// however it is cut; a draw over 150 k tokens misses the exactly summed one
// about once in 10^7 rows, where fp32 weights would miss once in a thousand.
//
// Layout.  One thread-block cluster per row, its CTAs the vocabulary slices,
// each slice resident in shared memory: the logits are read from HBM once,
// every later pass runs on chip.  The cut is found by radix selection on the
// logits' ordered bit patterns: each level is a histogram (count and weight) of
// the keys in the current range over kBins bins, summed over the cluster
// through distributed shared memory; the bin that holds the cut becomes the
// next range, until it is a single key.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "bdsa_device.cuh"
#include "bdsa_internal.h"

namespace bdsa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 512;  // one a thread
constexpr int kMaxCluster = 8;
constexpr int kUnitLog2 = 41;  // a weight's unit is 2^-41 of the row's largest
constexpr uint32_t kAll = 0xffffffffu;

// ------------------------------------------------------------ 2^(j / 128)
// hi + lo: the factor as two floats; fix: in units of 2^-kUnitLog2.
struct ExpTable {
    float hi[128], lo[128];
    uint64_t fix[128];
};
constexpr double exp2_series(double x) {  // 2^x for 0 <= x < 1 (Taylor series of e^(x ln 2))
    const double y = x * 0.69314718055994530942;
    double term = 1.0, sum = 1.0;
    for (int n = 1; n < 30; ++n) {
        term *= y / n;
        sum += term;
    }
    return sum;
}
constexpr ExpTable make_exp_table() {
    ExpTable t{};
    for (int j = 0; j < 128; ++j) {
        const double v = exp2_series(j / 128.0);
        t.hi[j] = (float)v;
        t.lo[j] = (float)(v - (double)t.hi[j]);
        t.fix[j] = (uint64_t)(v * (double)(1ull << kUnitLog2) + 0.5);
    }
    return t;
}
__device__ const ExpTable g_exp_table = make_exp_table();

// log2(e) / T as two floats, and the row's largest logit.
struct RowScale {
    float lmax, ch, cl;
};

// w = 2^(c (l - lmax)): returns it in units of 2^-41 and, in wf, as a float.
// l - lmax is taken exactly (TwoSum), the product with c as hi + lo, the
// integer and 1/128 parts go to the shift and the table, and the remainder r,
// |r| <= 1/256, to 2^r - 1 = s + s^2/2 + s^3/6 + s^4/24, s = r ln 2.
__device__ __forceinline__ uint64_t weight(float l, const RowScale &rs, const ExpTable &tab,
                                           float &wf) {
    const float dh = l - rs.lmax;
    const float yh = dh * rs.ch;
    wf = 0.f;
    if (!(yh > -125.f)) return 0;  // below every unit and fp32's range (also -inf and NaN)
    const float bb = dh - l;
    const float dl = (l - (dh - bb)) - (rs.lmax + bb);
    const float yl = fmaf(dh, rs.ch, -yh) + fmaf(dh, rs.cl, dl * rs.ch);
    const float t = fmaf(yh, 128.f, 12582912.f);  // round to an integer
    const int k = __float_as_int(t) - 0x4B400000;
    const float r = fmaf(t - 12582912.f, -0.0078125f, yh);
    constexpr float kL2h = 0.693147182464599609375f, kL2l = -1.904654323148236017e-09f;
    const float sh = r * kL2h;
    const float sl = fmaf(r, kL2h, -sh) + fmaf(r, kL2l, yl * kL2h);
    const float q = fmaf(sh * sh, fmaf(sh, fmaf(sh, 0.041666667f, 0.16666667f), 0.5f), sh * sl);
    const float lo = sl + q;
    const int idx = k & 127, n = k >> 7;  // n <= 0
    const float th = tab.hi[idx], tl = tab.lo[idx];
    const float ph = th * sh;
    const float pl = fmaf(th, sh, -ph) + fmaf(th, lo, tl * sh);
    wf = (th + (ph + (pl + tl))) * __int_as_float((n + 127) << 23);  // n >= -126: normal
    // the correction ph + pl in units of 2^-41, from 2^-29 and 2^-38 steps
    // (|ph| < 5.5e-3 and |pl| < 1.5e-5 keep both below 2^22 steps, where adding
    // 1.5 * 2^23 rounds to an integer)
    const float m1 = fmaf(ph, 536870912.f, 12582912.f);
    const int i1 = __float_as_int(m1) - 0x4B400000;
    const float rem = fmaf(m1 - 12582912.f, -1.862645149230957e-09f, ph) + pl;
    const float m2 = fmaf(rem, 274877906944.f, 12582912.f);
    const int i2 = __float_as_int(m2) - 0x4B400000;
    const int64_t m = (int64_t)tab.fix[idx] + ((int64_t)i1 << 12) + ((int64_t)i2 << 3);
    const int s = -n;
    if (s == 0) return (uint64_t)m;
    if (s > kUnitLog2 + 2) return 0;
    return ((uint64_t)m + (1ull << (s - 1))) >> s;
}

// floor(x * v) and ceil(x * v) for a float 0 < x < 1 and an integer v < 2^63,
// exactly (128-bit product of the mantissa).
__device__ __forceinline__ uint64_t scaled(float x, uint64_t v, bool up) {
    const uint32_t b = __float_as_uint(x);
    const int e = (int)(b >> 23);
    const uint64_t m = e ? (uint64_t)((b & 0x7fffffu) | 0x800000u) : (uint64_t)(b & 0x7fffffu);
    const int sh = 150 - (e ? e : 1);  // x = m * 2^-sh, 24 <= sh <= 149
    const uint64_t lo = m * v, hi = __umul64hi(m, v);
    uint64_t q;
    bool rest;
    if (sh < 64) {
        q = (hi << (64 - sh)) | (lo >> sh);  // hi < 2^(87 - 64): no bits lost (sh >= 24)
        rest = (lo & ((1ull << sh) - 1)) != 0;
    } else if (sh == 64) {
        q = hi;
        rest = lo != 0;
    } else {
        q = sh < 128 ? hi >> (sh - 64) : 0;
        rest = lo != 0 || (sh < 128 ? (hi & ((1ull << (sh - 64)) - 1)) != 0 : hi != 0);
    }
    return q + (up && rest ? 1 : 0);
}

// ------------------------------------------------------------ logit types
// Raw bits, their value, and a key that orders like the value with NaN as the
// smallest (as -inf) and -0 equal to +0.
template <typename T>
struct Logit;
template <>
struct Logit<float> {
    using Raw = uint32_t;
    static constexpr Raw kNegInf = 0xff800000u;
    static __device__ __forceinline__ float value(Raw r) {
        const float v = __uint_as_float(r);
        return v == v ? v : -INFINITY;
    }
    static __device__ __forceinline__ uint32_t key(Raw r) {
        const uint32_t b = __float_as_uint(value(r) + 0.f);
        return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
    }
    static __device__ __forceinline__ Raw from_key(uint32_t k) {
        return k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu);
    }
};
// 16-bit types: the key is the 16-bit pattern's.
template <typename T>
struct Logit16 {
    using Raw = uint16_t;
    static __device__ __forceinline__ uint32_t key16(float v, Raw r, Raw neg_inf) {
        uint32_t b = v == v ? r : neg_inf;
        if (v == 0.f) b = 0;
        return (b ^ ((b >> 15) ? 0xffffu : 0x8000u)) & 0xffffu;
    }
    static __device__ __forceinline__ Raw from_key(uint32_t k) {
        return (Raw)(k ^ ((k >> 15) ? 0x8000u : 0xffffu));
    }
};
template <>
struct Logit<__nv_bfloat16> : Logit16<__nv_bfloat16> {
    static constexpr Raw kNegInf = 0xff80;
    static __device__ __forceinline__ float wide(Raw r) {
        return __uint_as_float((uint32_t)r << 16);
    }
    static __device__ __forceinline__ float value(Raw r) {
        const float v = wide(r);
        return v == v ? v : -INFINITY;
    }
    static __device__ __forceinline__ uint32_t key(Raw r) { return key16(wide(r), r, kNegInf); }
};
template <>
struct Logit<__half> : Logit16<__half> {
    static constexpr Raw kNegInf = 0xfc00;
    static __device__ __forceinline__ float wide(Raw r) { return __half2float(__ushort_as_half(r)); }
    static __device__ __forceinline__ float value(Raw r) {
        const float v = wide(r);
        return v == v ? v : -INFINITY;
    }
    static __device__ __forceinline__ uint32_t key(Raw r) { return key16(wide(r), r, kNegInf); }
};

// ------------------------------------------------------------ cluster
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
template <class T>
__device__ __forceinline__ const T *map_to_rank(const T *p, uint32_t rank) {
    uint64_t out;
    asm volatile("mapa.u64 %0, %1, %2;"
                 : "=l"(out)
                 : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
    return reinterpret_cast<const T *>(out);
}

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int o) {
    return __shfl_xor_sync(kAll, (unsigned long long)v, o);
}
__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += shfl_xor64(v, o);
    return v;
}
__device__ __forceinline__ uint64_t warp_scan64(uint64_t v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t t = __shfl_up_sync(kAll, (unsigned long long)v, o);
        if (lane >= o) v += t;
    }
    return v;
}

// ------------------------------------------------------------ shared state
struct Hist {
    uint32_t cnt[kBins];
    // weight = m0 + m1 2^14 + m2 2^28: a slice has at most 2^18 logits, so no
    // counter reaches 2^32
    uint32_t m0[kBins], m1[kBins], m2[kBins];
};

struct Shared {
    ExpTable tab;
    Hist hist[2];
    uint64_t scan_c[kWarps], scan_m[kWarps];
    uint64_t wsum[kWarps];        // kept weight of each warp's segment
    uint32_t wties[kWarps];       // cut-key elements of each warp's segment
    // cluster exchange: written by this CTA, read by all, one use each
    uint32_t x_max, x_min;
    uint64_t x_sum;
    uint32_t x_ties;
    // the bin a select level chose
    int bin;
    uint64_t bin_c, bin_m, bin_dc, bin_dm;
    uint32_t red[2][kWarps];
};

// A position in the row's order: every key above `key`, and the first `ties`
// elements (by index) that equal it.
struct Cut {
    uint32_t key;
    uint64_t ties;
};

// This thread's bin of a level: exclusive prefix and own count and weight.
struct Level {
    uint64_t c, m, dc, dm;
};

template <typename T, bool kResident>
struct Row {
    using L = Logit<T>;
    using Raw = typename L::Raw;
    const Raw *s;      // the slice: shared memory, or global memory
    const Raw *g;
    int n;             // elements of the slice
    bool inf;          // the row's maximum is +inf: +inf counts as 0, the rest as -inf
    __device__ __forceinline__ Raw raw(int i) const { return kResident ? s[i] : __ldg(g + i); }
    __device__ __forceinline__ float value(Raw r) const {
        const float v = L::value(r);
        return inf ? (v == INFINITY ? 0.f : -INFINITY) : v;
    }
};

// One histogram level over the keys in [klo, khi], bin 0 the highest keys.
// kMass: weights too.  Every thread of every CTA of the cluster ends with its
// bin's totals over the cluster.
template <bool kMass, class R>
__device__ Level level_hist(const R &row, Shared &sm, int buf, uint32_t klo, uint32_t khi,
                            int shift, const RowScale &rs, uint32_t ncta) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Hist &h = sm.hist[buf];
    h.cnt[tid] = h.m0[tid] = h.m1[tid] = h.m2[tid] = 0;
    __syncthreads();
    for (int i = tid; i < row.n; i += kThreads) {
        const auto raw = row.raw(i);
        const uint32_t key = R::L::key(raw);
        if (key < klo || key > khi) continue;
        const uint32_t b = (khi - key) >> shift;
        atomicAdd(&h.cnt[b], 1u);
        if (kMass) {
            float wf;
            const uint64_t w = weight(row.value(raw), rs, sm.tab, wf);
            const uint32_t l0 = (uint32_t)w & 0x3fffu, l1 = (uint32_t)(w >> 14) & 0x3fffu;
            const uint32_t l2 = (uint32_t)(w >> 28);
            if (l0) atomicAdd(&h.m0[b], l0);
            if (l1) atomicAdd(&h.m1[b], l1);
            if (l2) atomicAdd(&h.m2[b], l2);
        }
    }
    cluster_sync();
    Level lv{0, 0, 0, 0};
    for (uint32_t r = 0; r < ncta; ++r) {
        const Hist *o = map_to_rank(&h, r);
        lv.dc += o->cnt[tid];
        if (kMass)
            lv.dm += (uint64_t)o->m0[tid] + ((uint64_t)o->m1[tid] << 14) +
                     ((uint64_t)o->m2[tid] << 28);
    }
    uint64_t ic = warp_scan64(lv.dc, lane), im = kMass ? warp_scan64(lv.dm, lane) : 0;
    if (lane == 31) {
        sm.scan_c[warp] = ic;
        sm.scan_m[warp] = im;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        ic += sm.scan_c[w];
        im += sm.scan_m[w];
    }
    lv.c = ic - lv.dc;
    lv.m = im - lv.dm;
    __syncthreads();  // scan_c / scan_m may be written again
    return lv;
}

// Bins of a range [klo, khi]: the smallest shift that fits kBins.
__device__ __forceinline__ int range_shift(uint32_t klo, uint32_t khi) {
    const int bits = 32 - __clz(khi - klo);
    return max(0, bits - 9);
}

// The shortest prefix of the order with at least `target` elements (kMass
// false) or at least `target` weight (kMass true; 0 < target <= the row's
// weight).  `lv` is the level over [klo, khi].  above_m: the weight of the keys
// above the cut's.
template <bool kMass, class R>
__device__ Cut select_cut(const R &row, Shared &sm, int &buf, Level lv, uint32_t klo,
                          uint32_t khi, uint64_t target, const RowScale &rs, uint32_t ncta,
                          uint64_t &above_m, uint64_t &key_count) {
    int shift = range_shift(klo, khi);
    uint64_t base_c = 0, base_m = 0;
    for (;;) {
        const uint64_t e = kMass ? base_m + lv.m : base_c + lv.c;
        const uint64_t d = kMass ? lv.dm : lv.dc;
        if (threadIdx.x == 0) sm.bin = -1;
        __syncthreads();
        if (e < target && target <= e + d) {
            sm.bin = (int)threadIdx.x;
            sm.bin_c = lv.c;
            sm.bin_m = lv.m;
            sm.bin_dc = lv.dc;
            sm.bin_dm = lv.dm;
        }
        __syncthreads();
        const int b = sm.bin;
        if (b < 0) {  // (never: the target is within the range's total)
            above_m = base_m;
            key_count = 0;
            return Cut{0, 0};
        }
        base_c += sm.bin_c;
        base_m += sm.bin_m;
        const uint64_t dc = sm.bin_dc, dm = sm.bin_dm;
        __syncthreads();
        khi -= (uint32_t)b << shift;
        const uint32_t span = shift ? (1u << shift) - 1 : 0;
        klo = khi - klo > span ? khi - span : klo;
        if (shift == 0) {
            Cut c;
            c.key = khi;
            const uint64_t w = dm / dc;  // equal keys, equal weights
            c.ties = kMass ? (target - base_m + w - 1) / w : target - base_c;
            above_m = base_m;
            key_count = dc;
            return c;
        }
        buf ^= 1;
        shift = range_shift(klo, khi);
        lv = level_hist<true>(row, sm, buf, klo, khi, shift, rs, ncta);
    }
}

template <typename T, bool kResident>
__global__ void __launch_bounds__(kThreads, 2) token_sample_kernel(const SampleArgs a) {
    using R = Row<T, kResident>;
    using L = Logit<T>;
    using Raw = typename L::Raw;
    extern __shared__ __align__(16) uint8_t s_dyn[];
    __shared__ Shared sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ncta = (uint32_t)a.ncta, rank = ncta > 1 ? cluster_rank() : 0u;
    const long rowi = blockIdx.x / ncta;
    const int r = (int)(rowi / a.B), i = (int)(rowi % a.B);
    const Raw *grow = static_cast<const Raw *>(a.logits) + r * a.lsr + i * a.lsi;
    const int e0 = min(a.V, (int)rank * a.slice), e1 = min(a.V, e0 + a.slice);
    R row;
    row.g = grow + e0;
    row.n = e1 - e0;
    row.inf = false;

    // ---- this row's parameters
    float temp = a.temperature ? a.temperature[r] : 1.f;
    const int top_k = a.top_k ? a.top_k[r] : 0;
    const float top_p = a.top_p ? a.top_p[r] : 1.f;
    const float min_p = a.min_p ? a.min_p[r] : 0.f;
    const bool bad_temp = !(temp >= 0.f) || temp == INFINITY;
    const bool greedy = temp == 0.f;
    const bool one = greedy || min_p > 1.f;  // only the first of the order is kept

    for (int j = tid; j < 128; j += kThreads) {
        sm.tab.hi[j] = g_exp_table.hi[j];
        sm.tab.lo[j] = g_exp_table.lo[j];
        sm.tab.fix[j] = g_exp_table.fix[j];
    }
    // ---- the slice into shared memory, its largest key and smallest key above
    // -inf's.  The copy keeps the slice's offset from a 16-byte boundary.
    constexpr int kVec = 16 / (int)sizeof(Raw);
    const uint32_t kNegInf = L::key(L::kNegInf);
    uint32_t kmax = 0, kmin = 0xffffffffu;
    auto take = [&](Raw v) {
        const uint32_t k = L::key(v);
        kmax = max(kmax, k);
        if (k > kNegInf) kmin = min(kmin, k);
    };
    const int mis = (int)((reinterpret_cast<uintptr_t>(row.g) & 15) / sizeof(Raw));
    const int head = min(row.n, mis ? kVec - mis : 0);
    const int nvec = (row.n - head) / kVec, tail0 = head + nvec * kVec;
    Raw *dst = reinterpret_cast<Raw *>(s_dyn) + mis;
    row.s = dst;
    if (tid < head) {
        const Raw v = __ldg(row.g + tid);
        if (kResident) dst[tid] = v;
        take(v);
    }
    if (tid < row.n - tail0) {
        const Raw v = __ldg(row.g + tail0 + tid);
        if (kResident) dst[tail0 + tid] = v;
        take(v);
    }
    const uint4 *gv = reinterpret_cast<const uint4 *>(row.g + head);
    uint4 *sv = reinterpret_cast<uint4 *>(dst + head);
#pragma unroll 4
    for (int x = tid; x < nvec; x += kThreads) {
        const uint4 q = __ldg(gv + x);
        if (kResident) sv[x] = q;
        const Raw *e = reinterpret_cast<const Raw *>(&q);
#pragma unroll
        for (int k = 0; k < kVec; ++k) take(e[k]);
    }
    kmax = __reduce_max_sync(kAll, kmax);
    kmin = __reduce_min_sync(kAll, kmin);
    if (lane == 0) {
        sm.red[0][warp] = kmax;
        sm.red[1][warp] = kmin;
    }
    __syncthreads();
    if (warp == 0) {
        kmax = __reduce_max_sync(kAll, lane < kWarps ? sm.red[0][lane] : 0u);
        kmin = __reduce_min_sync(kAll, lane < kWarps ? sm.red[1][lane] : 0xffffffffu);
        if (lane == 0) {
            sm.x_max = kmax;
            sm.x_min = kmin;
        }
    }
    cluster_sync();
    kmax = 0;
    kmin = 0xffffffffu;
    for (uint32_t c = 0; c < ncta; ++c) {
        kmax = max(kmax, *map_to_rank(&sm.x_max, c));
        kmin = min(kmin, *map_to_rank(&sm.x_min, c));
    }
    float *prow = a.probs ? a.probs + r * a.psr + i * a.psi + e0 : nullptr;
    if (bad_temp || kmax <= kNegInf) {  // no distribution (uniform over the cluster)
        if (prow)
            for (int x = tid; x < row.n; x += kThreads) prow[x] = 0.f;
        if (rank == 0 && tid == 0) {
            if (a.tokens) a.tokens[rowi] = -1;
            report_status(a.dev_status, BDSA_DEVICE_OUT_OF_RANGE);
        }
        cluster_sync();  // x_max / x_min have been read everywhere
        return;
    }
    RowScale rs;
    rs.lmax = L::value(L::from_key(kmax));
    row.inf = rs.lmax == INFINITY;
    if (row.inf) rs.lmax = 0.f;
    {
        // temperatures below 1e-30 act as 1e-30 (greedy rows weigh every kept
        // logit alike: only one is kept)
        const double c = 1.4426950408889634 / (double)fmaxf(greedy ? 1.f : temp, 1e-30f);
        rs.ch = (float)c;
        rs.cl = (float)(c - (double)rs.ch);
    }
    if (row.inf) kmin = kmax;  // only the +inf logits have weight

    // ---- the cut
    Cut cut{0, ~0ull};  // everything
    uint64_t key_count = 0;  // elements with the cut's key
    const bool use_k = one || (top_k > 0 && top_k < a.V);
    const bool use_p = !one && top_p < 1.f;
    if (use_k || use_p) {
        int buf = 0;
        const Level lv = level_hist<true>(row, sm, buf, kmin, kmax, range_shift(kmin, kmax), rs, ncta);
        // totals of the range (the last thread's inclusive prefix)
        if (tid == kThreads - 1) {
            sm.bin_c = lv.c + lv.dc;
            sm.bin_m = lv.m + lv.dm;
        }
        __syncthreads();
        const uint64_t all_c = sm.bin_c, all_m = sm.bin_m;
        __syncthreads();
        uint64_t total = all_m, above = 0;
        const uint64_t k = one ? 1u : (uint64_t)top_k;
        if (use_k && k < all_c) {
            cut = select_cut<false>(row, sm, buf, lv, kmin, kmax, k, rs, ncta, above, key_count);
            float wf;
            total = above + cut.ties * weight(row.value(L::from_key(cut.key)), rs, sm.tab, wf);
        }
        if (use_p) {
            uint64_t target = top_p > 0.f ? scaled(top_p, total, true) : 1;
            if (target < 1) target = 1;
            uint64_t kc2 = 0;
            const Cut c2 = select_cut<true>(row, sm, buf, lv, kmin, kmax, target, rs, ncta, above, kc2);
            if (c2.key > cut.key || (c2.key == cut.key && c2.ties < cut.ties)) {
                cut = c2;
                key_count = kc2;
            }
        }
    }

    // ---- the cut's ties: the first cut.ties of key_count by index.  A warp
    // owns the contiguous segment [w0, w1) of the slice; tie_end: the warp's
    // elements with the cut's key are kept below this index.
    const int seg = ((row.n + kWarps - 1) / kWarps + 31) & ~31;
    const int w0 = min(row.n, warp * seg), w1 = min(row.n, w0 + seg);
    int tie_end = w1;
    if (cut.ties < key_count) {
        uint32_t mine = 0;
        for (int x = w0 + lane; x < w1; x += 32) mine += L::key(row.raw(x)) == cut.key;
        mine = __reduce_add_sync(kAll, mine);
        if (lane == 0) sm.wties[warp] = mine;
        __syncthreads();
        if (tid == 0) {
            uint32_t t = 0;
            for (int w = 0; w < kWarps; ++w) t += sm.wties[w];
            sm.x_ties = t;
        }
        cluster_sync();
        uint64_t before = 0;
        for (uint32_t c = 0; c < rank; ++c) before += *map_to_rank(&sm.x_ties, c);
        for (int w = 0; w < warp; ++w) before += sm.wties[w];
        const uint64_t left = cut.ties > before ? cut.ties - before : 0;  // this warp keeps
        if (left < mine) {
            tie_end = w0;
            uint32_t seen = 0;
            for (int x0 = w0; x0 < w1 && seen < left; x0 += 32) {
                const int x = x0 + lane;
                const unsigned m = __ballot_sync(kAll, x < w1 && L::key(row.raw(x)) == cut.key);
                const uint32_t n = __popc(m);
                if (seen + n >= left) {
                    // the (left - seen)-th set bit of m ends the kept ties
                    tie_end = x0 + (int)__fns(m, 0, (int)(left - seen)) + 1;
                }
                seen += n;
            }
        }
    }

    // ---- kept weight, the draw
    const bool use_m = min_p > 0.f;
    const uint64_t wmin = use_m ? (min_p >= 1.f ? 1ull << kUnitLog2
                                                : scaled(min_p, 1ull << kUnitLog2, true))
                                : 0;
    auto kept = [&](int x, Raw raw, float &wf) -> uint64_t {
        wf = 0.f;
        if (use_k || use_p) {
            const uint32_t key = L::key(raw);
            if (key < cut.key || (key == cut.key && x >= tie_end)) return 0;
        }
        const uint64_t w = weight(row.value(raw), rs, sm.tab, wf);
        if (w < wmin) {
            wf = 0.f;
            return 0;
        }
        return w;
    };
    uint64_t sum = 0;
    for (int x = w0 + lane; x < w1; x += 32) {
        float wf;
        sum += kept(x, row.raw(x), wf);
    }
    sum = warp_sum64(sum);
    if (lane == 0) sm.wsum[warp] = sum;
    __syncthreads();
    if (tid == 0) {
        uint64_t t = 0;
        for (int w = 0; w < kWarps; ++w) t += sm.wsum[w];
        sm.x_sum = t;
    }
    cluster_sync();
    uint64_t total = 0, before = 0;
    for (uint32_t c = 0; c < ncta; ++c) {
        const uint64_t t = *map_to_rank(&sm.x_sum, c);
        if (c < rank) before += t;
        total += t;
    }
    if (a.tokens) {
        const float u = a.u[rowi];
        // floor(u * total), below total; u outside [0, 1) is clamped
        uint64_t target = u > 0.f ? (u < 1.f ? scaled(u, total, false) : total - 1) : 0;
        for (int w = 0; w < warp; ++w) before += sm.wsum[w];
        if (before <= target && target < before + sum) {
            // this warp: lane sums over contiguous runs, the lane, the element
            const int run = seg / 32, x0 = min(w1, w0 + lane * run), x1 = min(w1, x0 + run);
            uint64_t ls = 0;
            float wf;
            for (int x = x0; x < x1; ++x) ls += kept(x, row.raw(x), wf);
            uint64_t c = before + warp_scan64(ls, lane) - ls;
            if (c <= target && target < c + ls) {
                int x = x0;
                for (;; ++x) {
                    c += kept(x, row.raw(x), wf);
                    if (c > target || x + 1 >= x1) break;
                }
                a.tokens[rowi] = e0 + x;
            }
        }
    }
    // ---- the distribution
    if (prow) {
        const float inv = (float)((double)(1ull << kUnitLog2) / (double)total);
        for (int x = w0 + lane; x < w1; x += 32) {  // (tie_end is the segment's)
            float wf;
            kept(x, row.raw(x), wf);
            prow[x] = wf * inv;
        }
    }
    cluster_sync();  // this CTA's shared memory has been read everywhere
}

template <typename T>
int launch_typed(const SampleArgs &in, int num_sms, cudaStream_t stream) {
    SampleArgs a = in;
    constexpr int kMaxSlice = 96 * 1024;  // bytes: two CTAs an SM
    const long bytes = (long)a.V * (long)sizeof(T);
    // CTAs a row: enough that a slice stays resident, and more while they
    // still spread the rows over the GPU (a slice of at least 4096 logits)
    const long rows = (long)a.bs * a.B;
    int ncta = 1;
    while (ncta < kMaxCluster &&
           ((bytes + ncta - 1) / ncta > kMaxSlice ||
            (rows * ncta * 2 <= 2 * num_sms && a.V / (2 * ncta) >= 4096)))
        ncta *= 2;
    a.ncta = ncta;
    a.slice = (int)((((long)a.V + ncta - 1) / ncta + 31) & ~31L);
    const size_t smem = (size_t)a.slice * sizeof(T) + 16;
    const bool resident = smem <= 200 * 1024;
    auto kernel = resident ? token_sample_kernel<T, true> : token_sample_kernel<T, false>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             resident ? (int)smem : 0) != cudaSuccess)
        return BDSA_CUDA_ERROR;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * ncta));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = resident ? smem : 0;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ncta;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? BDSA_OK : BDSA_CUDA_ERROR;
}

}  // namespace

int launch_token_sample(const SampleArgs &a, int dtype, int num_sms, cudaStream_t stream) {
    switch (dtype) {
        case BDSA_F32: return launch_typed<float>(a, num_sms, stream);
        case BDSA_BF16: return launch_typed<__nv_bfloat16>(a, num_sms, stream);
        case BDSA_F16: return launch_typed<__half>(a, num_sms, stream);
        default: return BDSA_INVALID_ARG;
    }
}

}  // namespace bdsa
