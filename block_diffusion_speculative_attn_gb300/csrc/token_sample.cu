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
// Arithmetic.  A weight is a float-float (hi + lo, good to about 2^-30 of
// itself) from a 16-entry table of 2^(j/16) and a short polynomial; sums are
// kept as 64-bit integers in units of 2^-41 of the row's largest weight.
// Integer sums are exact in any order, so the partial sums of threads, warps and
// CTAs combine freely (shared-memory atomics among them) and a row gives the
// same answer however it is cut.  fp32 weights would not do: over 150 k tokens
// their rounding moves one draw in about a thousand to a neighbouring token,
// against one in 10^5 here.
//
// Layout.  One thread-block cluster per row (of one CTA when there are rows
// enough), its CTAs the vocabulary slices.  Two kernels:
//   sample_full    no filter arrays: one pass for the weights (stored to probs as
//                  they are) and their sum, against a scale taken from the row's
//                  first logits; a second one, on lines still in L2, that divides
//                  by the sum.  Two CTAs a row keep the rows in flight within L2.
//   sample_cut     filters: the row is streamed once for the maxima of some
//                  thousand parts of it (and, with probs, zeros are stored); a
//                  pivot below which nothing can be kept comes from those maxima
//                  (the k-th largest of them is at most the k-th largest logit,
//                  and their weights bound the weight above a pivot from below);
//                  the few logits above it are sorted and cut exactly.
//                  A flat row's nucleus (top-p alone, more than kListMax
//                  candidates) is cut the same way in a window around the cut
//                  that one counting pass finds.  Otherwise (large k, long runs
//                  of ties, no active filter) radix selection on the logits'
//                  ordered bit patterns: each level is a histogram (count and
//                  weight) over the current key range, summed over the cluster
//                  through distributed shared memory; the bin that holds the cut
//                  becomes the next range, until it is a single key.  These
//                  passes read the row again, mostly from L2.
// Measured: sample_full, 480 bf16 rows of 151936 to probs and tokens, 167 us for
// 438 MB (2.6 TB/s): the exponentials' packed-fp32 instructions and then the
// second pass's trip through L2, one after the other in a CTA and only in part
// under the other CTA of the SM.  sample_cut, 512 fp32 rows of 151936, every filter,
// 120 us for 622 MB (5.2 TB/s, 0.77 of a plain copy's rate): the stream of the row
// and the zeros; two waves of CTAs, the second two thirds full.  61 fp16 rows of
// 100003, top-p over thousands, 63 us: three passes over resident slices and a
// dozen cluster-wide steps.  16 fp32 rows of 1000, 11 us: those steps alone.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <stddef.h>

#include "bdsa_device.cuh"
#include "bdsa_internal.h"

namespace bdsa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 512;         // one a thread of sample_cut
constexpr int kParts = 8;          // parts of a thread's share of a slice, a maximum each
constexpr int kMaxCluster = 8;
constexpr int kListMax = 1024;  // candidates the sorted list holds
constexpr int kWinBins = 2048;  // bins of a flat row's counts, four a thread
constexpr int kWinMax = 4;      // the window: at most so many bins on either side
constexpr uint32_t kAll = 0xffffffffu;

// ------------------------------------------------------------ 2^(j / 16)
// The factor as hi + lo.  Sixteen words of either lie in banks of their own, so a
// warp's lookups never conflict.
struct ExpTable {
    float hi[16], lo[16];
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
    for (int j = 0; j < 16; ++j) {
        const double v = exp2_series(j / 16.0);
        t.hi[j] = (float)v;
        t.lo[j] = (float)(v - (double)(float)v);
    }
    return t;
}
__device__ const ExpTable g_exp_table = make_exp_table();

// A row's weights are 2^(y - E), y = c l with c = log2(e) / T = ch + cl and E an
// integer above the largest y (so the largest weight is in [1/2, 1]): a plain
// product and an exponent, without the subtraction of the largest logit, whose
// rounding would have to be carried along.  Rows with |c lmax| >= 2^17 (very small
// temperatures) are `wide`: y = c (l - lmax), E = 0.
struct RowScale {
    float lmax, ch, cl;
    float ymin;        // weights with y <= ymin are zero (2^-124 of the scale)
    int E;
    uint32_t ebits;    // (127 - E) << 23, modulo 2^32
    bool wide;
    __device__ __forceinline__ void set_scale(int e) {
        E = e;
        ymin = (float)(e - 124);
        ebits = (uint32_t)(127 - e) << 23;
    }
};
__device__ __forceinline__ RowScale row_scale(float lmax, float temp) {
    // log2(e) / T as two floats by a corrected fp32 division (a double one costs
    // every thread of the CTA some twenty fp64 instructions, which this GPU runs
    // at 1/64 of the fp32 rate); temperatures below 1e-30 act as 1e-30
    constexpr float kL2e = 1.44269502162933349609375f, kL2el = 1.925963033500011e-08f;
    RowScale rs;
    const float t = fmaxf(temp, 1e-30f);
    rs.lmax = lmax;
    rs.ch = __fdiv_rn(kL2e, t);
    const float rest = fmaf(-rs.ch, t, kL2e) + kL2el;
    rs.cl = __fdiv_rn(rest, t);
    const float y = lmax * rs.ch;
    rs.wide = !(fabsf(y) < 131072.f);
    rs.set_scale(rs.wide ? 0 : (int)floorf(y) + 1);
    return rs;
}

// One lane value, or a packed pair, with the same operations.
struct V1 {
    float a;
};
struct V2 {
    uint64_t a;
};
__device__ __forceinline__ V1 operator+(V1 x, V1 y) { return {x.a + y.a}; }
__device__ __forceinline__ V1 operator*(V1 x, V1 y) { return {x.a * y.a}; }
__device__ __forceinline__ V1 vfma(V1 x, V1 y, V1 z) { return {fmaf(x.a, y.a, z.a)}; }
__device__ __forceinline__ V2 operator+(V2 x, V2 y) { return {f2_add(x.a, y.a)}; }
__device__ __forceinline__ V2 operator*(V2 x, V2 y) { return {f2_mul(x.a, y.a)}; }
__device__ __forceinline__ V2 vfma(V2 x, V2 y, V2 z) { return {f2_fma(x.a, y.a, z.a)}; }
template <class V>
__device__ __forceinline__ V splat(float x);
template <>
__device__ __forceinline__ V1 splat<V1>(float x) { return {x}; }
template <>
__device__ __forceinline__ V2 splat<V2>(float x) { return {f2_pack(x, x)}; }

// Table entry and power of two of k sixteenths, from t = k + 1.5 * 2^23: the
// float's low bits are k's, and 19 places up only k's own remain.
__device__ __forceinline__ uint32_t table_at(float t) { return __float_as_uint(t) & 15u; }
__device__ __forceinline__ float pow2_at(float t, uint32_t ebits) {
    return __uint_as_float(((__float_as_uint(t) << 19) & 0xff800000u) + ebits);
}
__device__ __forceinline__ void lookup(const ExpTable &tab, uint32_t ebits, V1 t, V1 &th, V1 &tl,
                                       V1 &sc) {
    th.a = tab.hi[table_at(t.a)];
    tl.a = tab.lo[table_at(t.a)];
    sc.a = pow2_at(t.a, ebits);
}
__device__ __forceinline__ void lookup(const ExpTable &tab, uint32_t ebits, V2 t, V2 &th, V2 &tl,
                                       V2 &sc) {
    const float2 u = f2_unpack(t.a);
    const uint32_t i0 = table_at(u.x), i1 = table_at(u.y);
    th.a = f2_pack(tab.hi[i0], tab.hi[i1]);
    tl.a = f2_pack(tab.lo[i0], tab.lo[i1]);
    sc.a = f2_pack(pow2_at(u.x, ebits), pow2_at(u.y, ebits));
}
// Zero where y <= ymin (and for -inf and NaN).
__device__ __forceinline__ void keep_above(V1 y, float ymin, V1 &h, V1 &l) {
    const bool ok = y.a > ymin;
    h.a = ok ? h.a : 0.f;
    l.a = ok ? l.a : 0.f;
}
__device__ __forceinline__ void keep_above(V2 y, float ymin, V2 &h, V2 &l) {
    const float2 v = f2_unpack(y.a);
    float2 a = f2_unpack(h.a), b = f2_unpack(l.a);
    if (!(v.x > ymin)) a.x = b.x = 0.f;
    if (!(v.y > ymin)) a.y = b.y = 0.f;
    h.a = f2_pack(a.x, a.y);
    l.a = f2_pack(b.x, b.y);
}

// The weight of l as wh + wl, |wl| <= ulp(wh) / 2.  y = yh + yl (kWide: of the
// difference to lmax, with its TwoSum error); y's sixteenths go to the table and
// the power of two, and the rest r of yh, |r| <= 1/32, with z = r + yl, to
//   2^z - 1 = r L + (yl L + z^2 (c2 + c3 z + c4 z^2 + c5 z^3)),  L = ln 2
// (as a float: its rounding, 2^-28 of itself, is 2^-33 of the weight).
template <class V, bool kWide>
__device__ __forceinline__ void weight_ff(V l, const RowScale &rs, const ExpTable &tab, V &wh,
                                          V &wl) {
    const V one_n = splat<V>(-1.f), ch = splat<V>(rs.ch);
    V yh, yl;
    if constexpr (kWide) {
        const V dh = l + splat<V>(-rs.lmax);
        const V bb = vfma(l, one_n, dh);
        const V dl =
            vfma(splat<V>(rs.lmax) + bb, one_n, vfma(vfma(bb, one_n, dh), one_n, l));
        yh = dh * ch;
        yl = vfma(dh, ch, yh * one_n);
        yl = vfma(dl, ch, vfma(dh, splat<V>(rs.cl), yl));
    } else {
        yh = l * ch;
        yl = vfma(l, splat<V>(rs.cl), vfma(l, ch, yh * one_n));
    }
    const V t = vfma(yh, splat<V>(16.f), splat<V>(12582912.f));  // round to an integer
    const V r = vfma(t + splat<V>(-12582912.f), splat<V>(-0.0625f), yh);  // exact
    const V z = r + yl;
    constexpr float kL = 0.693147182464599609375f;
    V h = vfma(z, splat<V>(1.3333558e-3f), splat<V>(9.6181291e-3f));
    h = vfma(z, h, splat<V>(5.5504109e-2f));
    h = vfma(z, h, splat<V>(2.40226507e-1f));
    const V lo = vfma(z * z, h, yl * splat<V>(kL));
    const V e = vfma(r, splat<V>(kL), lo);
    V th, tl, sc;
    lookup(tab, rs.ebits, t, th, tl, sc);
    const V b = vfma(th, e, tl);
    const V s = th + b;                                // Fast2Sum: s + (b - (s - th)) exactly
    const V q = vfma(vfma(th, one_n, s), one_n, b);
    wh = s * sc;
    wl = q * sc;
    keep_above(yh, rs.ymin, wh, wl);
}

// A weight's unit is 2^-41 of the row's scale.
constexpr float kUnits = 2199023255552.f;

// The weight in units of 2^-41 of the scale and, in wf, as a float.
__device__ __forceinline__ uint64_t weight(float l, const RowScale &rs, const ExpTable &tab,
                                           float &wf) {
    V1 wh, wl;
    if (rs.wide) weight_ff<V1, true>(V1{l}, rs, tab, wh, wl);
    else weight_ff<V1, false>(V1{l}, rs, tab, wh, wl);
    wf = wh.a;
    return (uint64_t)(__float2ll_rn(wh.a * kUnits) + (long long)__float2int_rn(wl.a * kUnits));
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
// A logit as fp32 (NaN as -inf), and the low bits of its ordered pattern that are
// the same for every value of the type and sign.
template <typename T>
struct Logit;
template <>
struct Logit<float> {
    using Raw = uint32_t;
    static constexpr int kKeyShift = 0;
    static __device__ __forceinline__ float wide(Raw r) { return __uint_as_float(r); }
};
template <>
struct Logit<__nv_bfloat16> {
    using Raw = uint16_t;
    static constexpr int kKeyShift = 16;
    static __device__ __forceinline__ float wide(Raw r) {
        return __uint_as_float((uint32_t)r << 16);
    }
};
template <>
struct Logit<__half> {
    using Raw = uint16_t;
    static constexpr int kKeyShift = 13;
    static __device__ __forceinline__ float wide(Raw r) {
        return __half2float(__ushort_as_half(r));
    }
};
__device__ __forceinline__ float clean(float v) { return fmaxf(v, -INFINITY); }
// Unsigned integers that order like the floats (no NaN; -0 as +0).
__device__ __forceinline__ uint32_t float_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_float(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

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
// The two halves of a barrier that only keeps a CTA's shared memory alive until
// the others have read it: arrive after the last read, wait before leaving.
__device__ __forceinline__ void cluster_reads_done() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_reads() {
    __syncwarp();
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

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, (unsigned long long)v, o);
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

// ------------------------------------------------------------ one CTA's sums
// Inclusive prefix sums of v over the CTA, in thread order.
__device__ __forceinline__ uint64_t block_scan64(uint64_t v, uint64_t *scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t t = warp_scan64(v, lane);
    if (lane == 31) scratch[warp] = t;
    __syncthreads();
    uint64_t before = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) before += w < warp ? scratch[w] : 0;
    __syncthreads();
    return before + t;
}

// What the draw needs: the weight of each warp's contiguous segment of the slice,
// and scratch.
struct DrawShared {
    uint64_t wsum[kWarps], scan[kWarps], step;
    uint64_t x_sum;  // the slice's weight, read by the cluster
    int last;
};

// Sets sum (each warp's segment weight, in every lane) up for the draw: total is
// the cluster's weight, before the weight in front of this slice.
__device__ __forceinline__ void share_sums(DrawShared &d, uint64_t sum, uint32_t ncta,
                                           uint32_t rank, uint64_t &total, uint64_t &before) {
    if ((threadIdx.x & 31) == 0) d.wsum[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        uint64_t t = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) t += d.wsum[w];
        d.x_sum = t;
    }
    cluster_sync();
    uint64_t x[kMaxCluster];
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) x[c] = c < ncta ? *map_to_rank(&d.x_sum, c) : 0;
    total = before = 0;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
        if (c < (int)rank) before += x[c];
        total += x[c];
    }
}

// The warp whose segment of this slice holds the target, or -1; before (the
// weight in front of the slice) becomes the weight in front of that segment.
// Uniform over the CTA.
__device__ __forceinline__ int warp_of_target(const DrawShared &d, uint64_t target,
                                              uint64_t &before) {
    if (target < before) return -1;
    for (int w = 0; w < kWarps; ++w) {
        if (target < before + d.wsum[w]) return w;
        before += d.wsum[w];
    }
    return -1;
}

// One step of the draw by the whole CTA: every thread brings the weights q[4] of
// four successive indices (their sum s4, the first at index idx) in thread
// order; before grows by the step's weight.  The thread that reaches the target
// writes its token; until then each step's last positive weight does.  True when
// the step has one, or the target was reached before it (uniform).
__device__ __forceinline__ bool draw_in_block(DrawShared &d, uint64_t target,
                                              uint64_t &before, const uint64_t (&q)[4],
                                              uint64_t s4, int idx, int32_t *token) {
    if (before > target) return true;  // (uniform)
    const int tid = threadIdx.x;
    if (tid == 0) d.last = -1;
    const uint64_t inc = block_scan64(s4, d.scan);
    if (s4) atomicMax(&d.last, tid);
    if (tid == kThreads - 1) d.step = inc;
    __syncthreads();
    const uint64_t step = d.step;
    const bool some = d.last >= 0;
    const bool hit = before + inc > target && before + inc - s4 <= target;
    const bool rest = before + step <= target && tid == d.last;
    if (hit || rest) {
        uint64_t c = before + inc - s4;
        int at = 0;
        for (int k = 0; k < 4; ++k) {
            if (q[k]) at = k;
            c += q[k];
            if (c > target) break;
        }
        *token = idx + at;
    }
    before += step;
    __syncthreads();
    return some;
}

// floor(u * total), below total; u outside [0, 1) is clamped.
__device__ __forceinline__ uint64_t draw_target(float u, uint64_t total) {
    return u > 0.f ? (u < 1.f ? scaled(u, total, false) : total - 1) : 0;
}

// 2^41 / total, rounded once (to within 2^-46).
__device__ __forceinline__ float inverse(uint64_t total) {
    const float hi = __ull2float_rz(total);  // hi <= total, both in units
    const float lo = __ull2float_rn(total - (uint64_t)hi);
    const float i0 = __fdiv_rn(kUnits, hi);
    // i0 + (kUnits - i0 (hi + lo)) / hi
    return i0 + __fdividef(fmaf(-i0, lo, fmaf(-i0, hi, kUnits)), hi);
}

// The logit as the weights see it when the row's largest is +inf: the +inf ones
// share the weight.
__device__ __forceinline__ float if_inf(float v) { return v == INFINITY ? 0.f : -INFINITY; }

// The running sum of one thread: weights of two packed lanes as 2^(y - E), floats
// with their remainders, for the row scale `rs` (E in rs.ebits and rs.ymin).
struct Running {
    V2 acc, low;
    __device__ __forceinline__ void clear() { acc = low = splat<V2>(0.f); }
    __device__ __forceinline__ void add(V2 h, V2 l) {  // TwoSum
        const V2 neg = splat<V2>(-1.f);
        const V2 t = acc + h;
        const V2 hh = vfma(acc, neg, t);
        const V2 err = vfma(vfma(hh, neg, t), neg, acc) + vfma(hh, neg, h);
        acc = t;
        low = low + (err + l);
    }
    // in units, of a scale 2^(to - from) as large
    __device__ __forceinline__ uint64_t units(int from, int to) const {
        const float2 a = f2_unpack(acc.a), b = f2_unpack(low.a);
        if (to - from > 126) return 0;
        const float f = kUnits * __int_as_float((127 + from - to) << 23);
        const long long v = __float2ll_rn(a.x * f) + __float2ll_rn(a.y * f) +
                            __float2ll_rn(b.x * f) + __float2ll_rn(b.y * f);
        return (uint64_t)max(v, 0ll);
    }
};

// How a slice splits into 16-byte vectors: element counts of the ragged ends.
struct Span {
    int head, nvec, tail;  // tail: the first element behind the vectors
};
template <typename Raw>
__device__ __forceinline__ Span span_of(const Raw *p, int len) {
    constexpr int kVec = 16 / (int)sizeof(Raw);
    const int mis = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(Raw));
    Span s;
    s.head = min(len, mis ? kVec - mis : 0);
    s.nvec = (len - s.head) / kVec;
    s.tail = s.head + s.nvec * kVec;
    return s;
}

// A warp's segment of a slice: vectors [v0, v1) of the slice's Span, and the
// ragged ends (the head with the first warp, the tail with the last).  Segments
// are in index order.
struct Segment {
    int v0, v1, head0, head1, tail0, tail1;  // elements [head0, head1), [tail0, tail1)
};
__device__ __forceinline__ Segment segment_of(const Span &sp, int len, int w) {
    const int per = (sp.nvec + kWarps - 1) / kWarps;
    Segment g;
    g.v0 = min(sp.nvec, w * per);
    g.v1 = min(sp.nvec, g.v0 + per);
    g.head0 = 0;
    g.head1 = w == 0 ? sp.head : 0;
    g.tail0 = sp.tail;
    g.tail1 = w == kWarps - 1 ? len : sp.tail;
    return g;
}

// kV = 4 or 8 floats, a 16- or 32-byte line piece a lane when aligned; kLast: not
// read again, so the first to leave L2.
template <int kV, bool kLast>
__device__ __forceinline__ void store_vec(float *p, const float (&w)[kV], bool aligned) {
    if (!aligned) {
#pragma unroll
        for (int k = 0; k < kV; ++k) p[k] = w[k];
    } else if constexpr (kV == 8 && kLast) {
        asm volatile(
            "st.global.L2::evict_first.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p),
            "f"(w[0]), "f"(w[1]), "f"(w[2]), "f"(w[3]), "f"(w[4]), "f"(w[5]), "f"(w[6]), "f"(w[7])
            : "memory");
    } else if constexpr (kV == 8) {
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p),
                     "f"(w[0]), "f"(w[1]), "f"(w[2]), "f"(w[3]), "f"(w[4]), "f"(w[5]), "f"(w[6]),
                     "f"(w[7])
                     : "memory");
    } else if constexpr (kLast) {
        __stcs(reinterpret_cast<float4 *>(p), make_float4(w[0], w[1], w[2], w[3]));
    } else {
        *reinterpret_cast<float4 *>(p) = make_float4(w[0], w[1], w[2], w[3]);
    }
}
template <int kV>
__device__ __forceinline__ void load_vec(const float *p, float (&w)[kV]) {
    if constexpr (kV == 8) {
        asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(w[0]), "=f"(w[1]), "=f"(w[2]), "=f"(w[3]), "=f"(w[4]), "=f"(w[5]),
                       "=f"(w[6]), "=f"(w[7])
                     : "l"(p)
                     : "memory");
    } else {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    }
}

// ============================================================ sample_full
struct FullShared {
    ExpTable tab;
    DrawShared draw;
    float red[kWarps];
    float x_max;  // read by the cluster
    int x_first;  // greedy rows: the slice's first largest logit; read by the cluster
};

template <typename T>
struct FullRow {
    using L = Logit<T>;
    using Raw = typename L::Raw;
    static constexpr int kVec = 16 / (int)sizeof(Raw);
    const Raw *g;
    int len;
    bool inf;
    __device__ __forceinline__ float value(Raw r) const {
        const float v = clean(L::wide(r));
        return inf ? if_inf(v) : v;
    }
};

// Weights and sum of a segment at a known scale, this lane's share in units (rows
// of very small temperatures, and rows with +inf logits).
template <typename T>
__device__ __noinline__ uint64_t sum_segment(const FullRow<T> &row, const Span &sp,
                                             const Segment &sg, const RowScale &rs,
                                             const ExpTable &tab, int lane) {
    uint64_t sum = 0;
    float wf;
    for (int x = sg.head0 + lane; x < sg.head1; x += 32)
        sum += weight(row.value(__ldg(row.g + x)), rs, tab, wf);
    for (int x = sp.head + sg.v0 * row.kVec + lane; x < sp.head + sg.v1 * row.kVec; x += 32)
        sum += weight(row.value(__ldg(row.g + x)), rs, tab, wf);
    for (int x = sg.tail0 + lane; x < sg.tail1; x += 32)
        sum += weight(row.value(__ldg(row.g + x)), rs, tab, wf);
    return sum;
}

// The first index of the row at or behind x1 whose weight is not zero in units, or
// else the last such below x0 (the row's largest has one).  By the whole CTA, the
// row g of V logits; logits far below half a unit are passed over by y alone (a leader
// at the end of a row of 151936, u = 0: 43 us a call, with every weight taken 109,
// with u = 0.5 12).
template <typename T>
__device__ __noinline__ int nearest_weight(const typename Logit<T>::Raw *g, int V, int x0, int x1,
                                           bool inf, const RowScale &rs, const ExpTable &tab,
                                           int *scratch) {
    using L = Logit<T>;
    constexpr int kEach = 16, kStep = kEach * kThreads;
    const int tid = threadIdx.x;
    // (half a unit is 2^-42 of the scale; the margin covers y's fp32 rounding)
    auto has = [&](float v) {
        const float y = rs.wide ? (v - rs.lmax) * rs.ch : v * rs.ch;
        float wf;
        return y > (float)rs.E - 42.25f && weight(v, rs, tab, wf) != 0;
    };
    // the thread's kEach logits at x, x + step, ..: the last k that has weight, or -1
    auto last_of = [&](int x, int step) {
        float v[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int e = x + k * step;
            v[k] = e >= 0 && e < V ? clean(L::wide(__ldg(g + e))) : -INFINITY;
        }
        int at = -1;
#pragma unroll
        for (int k = 0; k < kEach; ++k) at = has(inf ? if_inf(v[k]) : v[k]) ? k : at;
        return at;
    };
    for (int base = x1; base < V; base += kStep) {
        const int x = base + (kEach - 1) * kThreads + tid, k = last_of(x, -kThreads);
        if (!__syncthreads_or(k >= 0)) continue;
        if (tid == 0) *scratch = INT_MAX;
        __syncthreads();
        if (k >= 0) atomicMin(scratch, x - k * kThreads);
        __syncthreads();
        return *scratch;
    }
    for (int end = x0; end > 0; end -= kStep) {
        const int x = end - kStep + tid, k = last_of(x, kThreads);
        if (!__syncthreads_or(k >= 0)) continue;
        if (tid == 0) *scratch = -1;
        __syncthreads();
        if (k >= 0) atomicMax(scratch, x + k * kThreads);
        __syncthreads();
        return *scratch;
    }
    return -1;  // (never)
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_full_kernel(const SampleArgs a) {
    using L = Logit<T>;
    using Raw = typename L::Raw;
    constexpr int kVec = 16 / (int)sizeof(Raw);
    __shared__ FullShared sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ncta = (uint32_t)a.ncta, rank = ncta > 1 ? cluster_rank() : 0u;
    const long rowi = blockIdx.x / ncta;
    const int r = (int)(rowi / a.B), i = (int)(rowi % a.B);
    const int e0 = min(a.V, (int)rank * a.slice);
    FullRow<T> row;
    row.len = min(a.V, e0 + a.slice) - e0;
    row.g = static_cast<const Raw *>(a.logits) + r * a.lsr + i * a.lsi + e0;
    row.inf = false;
    const Span sp = span_of(row.g, row.len);
    const Segment sg = segment_of(sp, row.len, warp);
    const uint4 *gv = reinterpret_cast<const uint4 *>(row.g + sp.head);
    const float temp = a.temperature ? a.temperature[r] : 1.f;
    const bool bad_temp = !(temp >= 0.f) || temp == INFINITY, greedy = temp == 0.f;
    float *prow = a.probs ? a.probs + r * a.psr + i * a.psi + e0 : nullptr;
    if (tid < 16) {
        sm.tab.hi[tid] = g_exp_table.hi[tid];
        sm.tab.lo[tid] = g_exp_table.lo[tid];
    }
    __syncthreads();

    // ---- the scale of the first pass: that of the row's first logits, so at most
    // the row's own (a row whose first logits are masked takes 0)
    const Raw *row0 = row.g - e0;
    float first = -INFINITY;
    for (int x = 0; x < min(a.V, 4); ++x) first = fmaxf(first, L::wide(__ldg(row0 + x)));
    RowScale rs = row_scale(0.f, bad_temp || greedy ? 1.f : temp);
    const float y0 = first * rs.ch;
    const int E0 = fabsf(y0) < 131072.f ? (int)floorf(y0) + 1 : 0;
    rs.set_scale(E0);

    // ---- weights, their sum, the largest logit
    float mx = -INFINITY;
    Running run;
    run.clear();
    const bool vec = (reinterpret_cast<uintptr_t>(prow + sp.head) % (4 * kVec)) == 0;
    auto ragged = [&](int x0, int x1) {
        for (int x = x0 + lane; x < x1; x += 32) {
            const float v = L::wide(__ldg(row.g + x));
            mx = fmaxf(mx, v);
            V2 h, l;
            weight_ff<V2, false>(V2{f2_pack(v, -INFINITY)}, rs, sm.tab, h, l);
            run.add(h, l);
            if (prow) prow[x] = f2_unpack(h.a).x;
        }
    };
    ragged(sg.head0, sg.head1);
    {
        // two vectors a step, the next step's on their way meanwhile
        uint4 q[2], next[2];
        auto fetch = [&](int x, uint4 (&v)[2]) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (x + 32 * u < sg.v1) v[u] = __ldcs(gv + x + 32 * u);
        };
        fetch(sg.v0 + lane, q);
        for (int x = sg.v0 + lane; x < sg.v1; x += 64) {
            fetch(x + 64, next);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (x + 32 * u >= sg.v1) break;
                const Raw *e = reinterpret_cast<const Raw *>(&q[u]);
                float *out = prow + sp.head + (long)(x + 32 * u) * kVec;
                float w[kVec];
#pragma unroll
                for (int k = 0; k < kVec; k += 2) {
                    const float v0 = L::wide(e[k]), v1 = L::wide(e[k + 1]);
                    mx = max3f(mx, v0, v1);
                    V2 h, l;
                    weight_ff<V2, false>(V2{f2_pack(v0, v1)}, rs, sm.tab, h, l);
                    run.add(h, l);
                    const float2 f = f2_unpack(h.a);
                    w[k] = f.x;
                    w[k + 1] = f.y;
                }
                if (prow) store_vec<kVec, false>(out, w, vec);
            }
            q[0] = next[0];
            q[1] = next[1];
        }
    }
    ragged(sg.tail0, sg.tail1);

    // ---- the row's largest logit
    float rmx = mx;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) rmx = fmaxf(rmx, __shfl_xor_sync(kAll, rmx, o));
    if (lane == 0) sm.red[warp] = rmx;
    __syncthreads();
    rmx = sm.red[lane % kWarps];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) rmx = fmaxf(rmx, __shfl_xor_sync(kAll, rmx, o));
    if (ncta > 1) {
        if (tid == 0) sm.x_max = rmx;
        cluster_sync();
        if (lane < (int)ncta) rmx = *map_to_rank(&sm.x_max, lane);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) rmx = fmaxf(rmx, __shfl_xor_sync(kAll, rmx, o));
    }
    if (bad_temp || rmx == -INFINITY) {  // no distribution (uniform over the cluster)
        cluster_reads_done();
        if (prow)
            for (int x = tid; x < row.len; x += kThreads) prow[x] = 0.f;
        if (rank == 0 && tid == 0) {
            if (a.tokens) a.tokens[rowi] = -1;
            report_status(a.dev_status, BDSA_DEVICE_OUT_OF_RANGE);
        }
        cluster_wait_reads();
        return;
    }
    if (greedy) {  // the first largest logit alone
        if (tid == 0) sm.x_first = INT_MAX;
        __syncthreads();
        int first = INT_MAX;
        for (int x = tid; x < row.len && first == INT_MAX; x += kThreads)
            if (clean(L::wide(__ldg(row.g + x))) == rmx) first = e0 + x;
        first = __reduce_min_sync(kAll, first);
        if (lane == 0) atomicMin(&sm.x_first, first);
        cluster_sync();
        first = lane < (int)ncta ? *map_to_rank(&sm.x_first, lane) : INT_MAX;
        first = __reduce_min_sync(kAll, first);
        cluster_reads_done();
        if (prow)
            for (int x = tid; x < row.len; x += kThreads) prow[x] = e0 + x == first ? 1.f : 0.f;
        if (a.tokens && rank == 0 && tid == 0) a.tokens[rowi] = first;
        cluster_wait_reads();
        return;
    }
    row.inf = rmx == INFINITY;
    rs = row_scale(row.inf ? 0.f : rmx, temp);
    // the first pass holds unless its scale was far below the row's (its weights
    // may have left fp32's range) or above it, or the row needs the wide form
    const bool again = rs.wide || row.inf || rs.E < E0 || rs.E > E0 + 100;
    uint64_t sum = again ? sum_segment<T>(row, sp, sg, rs, sm.tab, lane) : run.units(E0, rs.E);
    sum = warp_sum64(sum);
    uint64_t total, before;
    share_sums(sm.draw, sum, ncta, rank, total, before);
    cluster_reads_done();

    // ---- the distribution (each lane has its own stores before it)
    if (prow) {
        const float inv = inverse(total);
        if (again) {
            auto one = [&](int x) {
                float wf;
                weight(row.value(__ldg(row.g + x)), rs, sm.tab, wf);
                prow[x] = wf * inv;
            };
            for (int x = sg.head0 + lane; x < sg.head1; x += 32) one(x);
            __syncwarp();
            for (int x = sp.head + sg.v0 * kVec + lane; x < sp.head + sg.v1 * kVec; x += 32) one(x);
            for (int x = sg.tail0 + lane; x < sg.tail1; x += 32) one(x);
        } else {
            // the stored weights are relative to E0
            const float f = __int_as_float((127 + E0 - rs.E) << 23);
            const V2 f2 = splat<V2>(f), i2 = splat<V2>(inv);
            for (int x = sg.head0 + lane; x < sg.head1; x += 32) prow[x] = prow[x] * f * inv;
            for (int x = sg.tail0 + lane; x < sg.tail1; x += 32) prow[x] = prow[x] * f * inv;
            if (vec) {
                constexpr int kU = 16 / kVec;
                for (int x = sg.v0 + lane; x < sg.v1; x += 32 * kU) {
                    float w[kU][kVec];
#pragma unroll
                    for (int u = 0; u < kU; ++u)
                        if (x + 32 * u < sg.v1)
                            load_vec<kVec>(prow + sp.head + (long)(x + 32 * u) * kVec, w[u]);
#pragma unroll
                    for (int u = 0; u < kU; ++u) {
                        if (x + 32 * u >= sg.v1) break;
#pragma unroll
                        for (int k = 0; k < kVec; k += 2) {
                            const float2 y =
                                f2_unpack((V2{f2_pack(w[u][k], w[u][k + 1])} * f2 * i2).a);
                            w[u][k] = y.x;
                            w[u][k + 1] = y.y;
                        }
                        store_vec<kVec, true>(prow + sp.head + (long)(x + 32 * u) * kVec, w[u],
                                              true);
                    }
                }
            } else {
                for (int v = sg.v0 + lane; v < sg.v1; v += 32)
                    for (int k = 0; k < kVec; ++k) {
                        float *o = prow + sp.head + (long)v * kVec + k;
                        *o = *o * f * inv;
                    }
            }
        }
    }
    // ---- the draw
    if (a.tokens) {
        const uint64_t target = draw_target(a.u[rowi], total);
        const int w = warp_of_target(sm.draw, target, before);
        if (w >= 0) {
            // in warp w's segment of this slice: its weights again, four positions a
            // thread.  Single weights round to units, the segment's sum as a whole: a
            // target past the rounded ones goes to the segment's last that is not
            // zero, and where all of them are zero (a logit leads by 29 nats and more)
            // to the row's next that is not, or the last.
            const Segment d = segment_of(sp, row.len, w);
            const int x0 = d.head1 > d.head0 ? 0 : sp.head + d.v0 * kVec;
            const int x1 = d.tail1 > d.tail0 ? row.len : sp.head + d.v1 * kVec;
            bool drawn = false;
            for (int base = x0; base < x1; base += 4 * kThreads) {
                const int x = base + 4 * tid;
                uint64_t q[4], s4 = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float wf;
                    q[k] = x + k < x1 ? weight(row.value(__ldg(row.g + x + k)), rs, sm.tab, wf) : 0;
                    s4 += q[k];
                }
                drawn |= draw_in_block(sm.draw, target, before, q, s4, e0 + x, a.tokens + rowi);
            }
            if (!drawn) {  // (uniform)
                const int x = nearest_weight<T>(row.g - e0, a.V, e0 + x0, e0 + x1, row.inf, rs,
                                                sm.tab, &sm.draw.last);
                if (tid == 0) a.tokens[rowi] = x;
            }
        }
    }
    cluster_wait_reads();
}

// ============================================================ sample_cut
struct Hist {
    uint32_t cnt[kBins];
    // weight = m0 + m1 2^14 + m2 2^28: a slice has at most 2^18 logits, so no
    // counter reaches 2^32
    uint32_t m0[kBins], m1[kBins], m2[kBins];
};
// Candidates of the list path: this CTA's, and the cluster's in sorted order
// (key descending, index ascending, as ~key << 32 | index) with their weights'
// prefix sums.
struct Lists {
    uint64_t own[kListMax];
    uint64_t a[kListMax], b[kListMax];
};

struct CutShared {
    ExpTable tab;
    union {
        Hist hist[2];
        Lists list;
    };
    uint32_t parts[kBins];        // pivot search: this CTA's part maxima by bin
    uint64_t scan[kWarps], scan_c[kWarps];
    DrawShared draw;
    uint32_t wties[kWarps];       // cut-key elements of each warp's segment
    uint64_t wextra[kWarps];      // kept weight of each warp's segment in the window
    uint32_t near[kWinMax + 1];   // elements so many bins from the window's middle
    uint32_t wbin[2 * kWinMax + 1][3];  // weights of the window's bins (as Hist's)
    float red[2][kWarps];
    uint32_t hit[kListMax];       // parts that reach the pivot: thread * kParts + part
    int n_hit, n_list, n_below, n_min, n_cut;
    // cluster exchange: written by this CTA, read by all, one use each
    float x_max, x_low;
    uint64_t x_all, x_above;
    uint32_t x_ties, x_min;
    // the bin a select level (or the pivot search) chose
    int bin;
    uint64_t bin_c, bin_m, bin_dc, bin_dm;
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

// This CTA's slice: in shared memory (kRes), or read from global memory again
// (mostly L2: it has been streamed).
template <typename T, bool kRes>
struct Row {
    using L = Logit<T>;
    const typename L::Raw *g;  // in global memory
    const typename L::Raw *s;  // kRes: the copy, as far from a 16-byte boundary
    int n;
    bool inf;  // the row's maximum is +inf
    __device__ __forceinline__ typename L::Raw raw(int x) const {
        return kRes ? s[x] : __ldg(g + x);
    }
    __device__ __forceinline__ uint4 vec(const uint4 *p) const { return kRes ? *p : __ldg(p); }
    __device__ __forceinline__ float at(int x) const {
        const float v = clean(L::wide(raw(x)));
        return inf ? if_inf(v) : v;
    }
    static __device__ __forceinline__ uint32_t key(float v) { return float_key(v) >> L::kKeyShift; }
    // a float of the type with this key
    static __device__ __forceinline__ float value(uint32_t key) {
        const float v = key_float(key << L::kKeyShift);
        return key >> (31 - L::kKeyShift) ? v : key_float((key << L::kKeyShift) |
                                                          ((1u << L::kKeyShift) - 1));
    }
};

// Runs body(x) for the positions x of [x0, x1) with pred(logit), one warp, in no
// particular order: each lane picks its positions of 32 * 32 first and the lanes
// then run their picks together, so that a warp's steps are the fullest lane's
// picks instead of every position with a picked neighbour.
template <class R, class P, class B>
__device__ __forceinline__ void for_selected(const R &row, int x0, int x1, int lane, P pred,
                                             B body) {
    for (int base = x0; base < x1; base += 1024) {
        uint32_t mask = 0;
        const int steps = min(32, (x1 - base + 31) / 32);
#pragma unroll 8
        for (int j = 0; j < steps; ++j) {
            const int x = base + 32 * j + lane;
            if (x < x1 && pred(row.at(x), x)) mask |= 1u << j;
        }
        while (mask) {
            const int j = __ffs(mask) - 1;
            mask &= mask - 1;
            body(base + 32 * j + lane);
        }
    }
    __syncwarp();
}

// One histogram level over the keys in [klo, khi], bin 0 the highest keys.  Every
// thread of every CTA of the cluster ends with its bin's totals over the cluster.
template <class R>
__device__ Level level_hist(const R &row, int w0, int w1, CutShared &sm, int buf, uint32_t klo,
                            uint32_t khi, int shift, const RowScale &rs, uint32_t ncta) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Hist &h = sm.hist[buf];
    h.cnt[tid] = h.m0[tid] = h.m1[tid] = h.m2[tid] = 0;
    __syncthreads();
    for_selected(
        row, w0, w1, lane,
        [&](float v, int) {
            const uint32_t key = R::key(v);
            return key >= klo && key <= khi;
        },
        [&](int x) {
            const float v = row.at(x);
            const uint32_t b = (khi - R::key(v)) >> shift;
            float wf;
            const uint64_t w = weight(v, rs, sm.tab, wf);
            const uint32_t l0 = (uint32_t)w & 0x3fffu, l1 = (uint32_t)(w >> 14) & 0x3fffu;
            const uint32_t l2 = (uint32_t)(w >> 28);
            atomicAdd(&h.cnt[b], 1u);
            if (l0) atomicAdd(&h.m0[b], l0);
            if (l1) atomicAdd(&h.m1[b], l1);
            if (l2) atomicAdd(&h.m2[b], l2);
        });
    cluster_sync();
    Level lv{0, 0, 0, 0};
    for (uint32_t r = 0; r < ncta; ++r) {
        const Hist *o = map_to_rank(&h, r);
        lv.dc += o->cnt[tid];
        lv.dm += (uint64_t)o->m0[tid] + ((uint64_t)o->m1[tid] << 14) + ((uint64_t)o->m2[tid] << 28);
    }
    uint64_t ic = warp_scan64(lv.dc, lane), im = warp_scan64(lv.dm, lane);
    if (lane == 31) {
        sm.scan_c[warp] = ic;
        sm.scan[warp] = im;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        ic += sm.scan_c[w];
        im += sm.scan[w];
    }
    lv.c = ic - lv.dc;
    lv.m = im - lv.dm;
    __syncthreads();  // scan_c / scan may be written again
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
// above the cut's; key_count: the elements with the cut's key.
template <bool kMass, class R>
__device__ Cut select_cut(const R &row, int w0, int w1, CutShared &sm, int &buf, Level lv,
                          uint32_t klo, uint32_t khi, uint64_t target, const RowScale &rs,
                          uint32_t ncta, uint64_t &above_m, uint64_t &key_count) {
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
        const uint64_t dc = sm.bin_dc, dm = sm.bin_dm;
        if (b < 0) {  // (never: the target is within the range's total)
            above_m = base_m;
            key_count = 0;
            return Cut{0, 0};
        }
        base_c += sm.bin_c;
        base_m += sm.bin_m;
        __syncthreads();
        khi -= (uint32_t)b << shift;
        const uint32_t span = shift ? (1u << shift) - 1 : 0;
        klo = khi - klo > span ? khi - span : klo;
        if (shift == 0) {
            Cut c;
            c.key = khi;
            const uint64_t w = kMass ? dm / dc : 0;  // equal keys, equal weights
            c.ties = kMass ? (target - base_m + w - 1) / w : target - base_c;
            above_m = base_m;
            key_count = dc;
            return c;
        }
        buf ^= 1;
        shift = range_shift(klo, khi);
        lv = level_hist(row, w0, w1, sm, buf, klo, khi, shift, rs, ncta);
    }
}

// Ascending bitonic sort of a[0, n) (n a power of two) by the whole CTA.
__device__ __forceinline__ void bitonic_sort(uint64_t *a, int n) {
    for (int k = 2; k <= n; k <<= 1) {
        for (int j = k >> 1; j > 0; j >>= 1) {
            for (int p = threadIdx.x; p < n / 2; p += kThreads) {
                const int i = ((p & ~(j - 1)) << 1) | (p & (j - 1)), q = i | j;
                const uint64_t x = a[i], y = a[q];
                if ((x > y) == ((i & k) == 0)) {
                    a[i] = y;
                    a[q] = x;
                }
            }
            __syncthreads();
        }
    }
}

// Threads an entry of a list of n <= kThreads gets when all entries are compared
// with all: a power of two, at most a warp.
__device__ __forceinline__ int list_parts(int n) {
    int p = 32;
    while (p > 1 && p * n > kThreads) p >>= 1;
    return p;
}

// Sorts the distinct keys a[0, n) ascending, n <= kListMax, room for a power of
// two; b is scratch of the same size.  Returns where the result is (a or b).
// Up to kThreads keys each find their rank by comparing with all the others (for
// the usual hundred or two a few dozen steps without a barrier: 16 rows of 1000 10.7
// us, by the network 13.4); more are sorted by a bitonic network.
__device__ __forceinline__ uint64_t *sort_list(uint64_t *a, uint64_t *b, int n) {
    const int tid = threadIdx.x;
    if (n <= kThreads) {
        const int parts = list_parts(n), x = tid / parts, part = tid % parts;
        const uint64_t key = x < n ? a[x] : 0;
        int rank = 0;
        if (x < n)
            for (int y = part; y < n; y += parts) rank += a[y] < key;
        for (int o = parts >> 1; o > 0; o >>= 1) rank += __shfl_xor_sync(kAll, rank, o);
        if (x < n && part == 0) b[rank] = key;
        __syncthreads();
        return b;
    }
    int np = 2;
    while (np < n) np <<= 1;
    for (int x = n + tid; x < np; x += kThreads) a[x] = ~0ull;
    __syncthreads();
    bitonic_sort(a, np);
    return a;
}

// Prefix sums of a[0, n), n <= kListMax, in place (two entries a thread).
__device__ __forceinline__ void scan_list(uint64_t *a, int n, uint64_t *scratch) {
    static_assert(kListMax == 2 * kThreads, "two entries a thread");
    const int i = 2 * threadIdx.x;
    const uint64_t x = i < n ? a[i] : 0, y = i + 1 < n ? a[i + 1] : 0;
    const uint64_t t = block_scan64(x + y, scratch);
    if (i < n) a[i] = t - y;
    if (i + 1 < n) a[i + 1] = t;
    __syncthreads();
}

// The CTAs' lists (n_list entries of list.own each) to list.a of every CTA, after
// a cluster_sync; returns their entries (past kListMax: nothing is copied).  The
// counts one a lane, then every entry of every list at once: a remote read takes
// most of a microsecond.
__device__ __forceinline__ int gather_lists(CutShared &sm, uint32_t ncta) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int m = lane < (int)ncta ? *map_to_rank(&sm.n_list, lane) : 0;
    int ends = min(m, kListMax + 1);
#pragma unroll
    for (int o = 1; o < kMaxCluster; o <<= 1) {
        const int t = __shfl_up_sync(kAll, ends, o);
        if (lane >= o) ends += t;
    }
    const int n = __shfl_sync(kAll, ends, kMaxCluster - 1);
    if (n > kListMax) return n;
    for (int x0 = warp * 32; x0 < n; x0 += kThreads) {
        const int x = x0 + lane;
        int c = 0, from = 0;
#pragma unroll
        for (int q = 0; q < kMaxCluster - 1; ++q) {
            const int e = __shfl_sync(kAll, ends, q);
            if (x >= e) {
                c = q + 1;
                from = e;
            }
        }
        if (x < n) sm.list.a[x] = map_to_rank(sm.list.own, c)[x - from];
    }
    return n;
}

// Runs body(logit, position) for this thread's share of the slice: vectors tid +
// kThreads j, and a position of each ragged end.
template <typename T, bool kRes, class B>
__device__ __forceinline__ void for_slice(const Row<T, kRes> &row, const Span &sp, B body) {
    using L = Logit<T>;
    using Raw = typename L::Raw;
    constexpr int kVec = 16 / (int)sizeof(Raw);
    const int tid = threadIdx.x;
    if (tid < sp.head) body(row.at(tid));
    if (tid < row.n - sp.tail) body(row.at(sp.tail + tid));
    const uint4 *gv = reinterpret_cast<const uint4 *>((kRes ? row.s : row.g) + sp.head);
    constexpr int kU = 4;
    for (int x = tid; x < sp.nvec; x += kU * kThreads) {
        uint4 q[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u)
            if (x + u * kThreads < sp.nvec) q[u] = row.vec(gv + x + u * kThreads);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (x + u * kThreads >= sp.nvec) break;
            const Raw *e = reinterpret_cast<const Raw *>(&q[u]);
#pragma unroll
            for (int k = 0; k < kVec; ++k) body(clean(L::wide(e[k])));
        }
    }
}

// The weight of the slice in units, this thread's share (every thread of the CTA).
template <typename T, bool kRes, bool kWide>
__device__ __forceinline__ uint64_t sum_stream(const Row<T, kRes> &row, const Span &sp,
                                               const RowScale &rs, const ExpTable &tab) {
    using L = Logit<T>;
    using Raw = typename L::Raw;
    constexpr int kVec = 16 / (int)sizeof(Raw);
    const int tid = threadIdx.x;
    Running run;
    run.clear();
    auto add = [&](float v0, float v1) {
        if (row.inf) {
            v0 = if_inf(v0);
            v1 = if_inf(v1);
        }
        V2 h, l;
        weight_ff<V2, kWide>(V2{f2_pack(v0, v1)}, rs, tab, h, l);
        run.add(h, l);
    };
    if (tid < sp.head) add(clean(L::wide(row.raw(tid))), -INFINITY);
    if (tid < row.n - sp.tail) add(clean(L::wide(row.raw(sp.tail + tid))), -INFINITY);
    const uint4 *gv = reinterpret_cast<const uint4 *>((kRes ? row.s : row.g) + sp.head);
    constexpr int kU = kRes ? 2 : 4;
    for (int x = tid; x < sp.nvec; x += kU * kThreads) {
        uint4 q[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u)
            if (x + u * kThreads < sp.nvec) q[u] = row.vec(gv + x + u * kThreads);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (x + u * kThreads >= sp.nvec) break;
            const Raw *e = reinterpret_cast<const Raw *>(&q[u]);
#pragma unroll
            for (int k = 0; k < kVec; k += 2) add(clean(L::wide(e[k])), clean(L::wide(e[k + 1])));
        }
    }
    return run.units(0, 0);
}

template <typename T, bool kRes>
__global__ void __launch_bounds__(kThreads, 2) sample_cut_kernel(const SampleArgs a) {
    using R = Row<T, kRes>;
    using L = Logit<T>;
    using Raw = typename L::Raw;
    constexpr int kVec = 16 / (int)sizeof(Raw);
    extern __shared__ __align__(16) uint8_t s_dyn[];
    __shared__ CutShared sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ncta = (uint32_t)a.ncta, rank = ncta > 1 ? cluster_rank() : 0u;
    const long rowi = blockIdx.x / ncta;
    const int r = (int)(rowi / a.B), i = (int)(rowi % a.B);
    const int e0 = min(a.V, (int)rank * a.slice);
    R row;
    row.n = min(a.V, e0 + a.slice) - e0;
    row.g = static_cast<const Raw *>(a.logits) + r * a.lsr + i * a.lsi + e0;
    row.inf = false;
    const Span sp = span_of(row.g, row.n);
    Raw *copy = reinterpret_cast<Raw *>(s_dyn) +
                (reinterpret_cast<uintptr_t>(row.g) & 15) / sizeof(Raw);
    row.s = copy;
    const uint4 *gv = reinterpret_cast<const uint4 *>(row.g + sp.head);

    // ---- this row's parameters
    const float temp = a.temperature ? a.temperature[r] : 1.f;
    const int top_k = a.top_k ? a.top_k[r] : 0;
    const float top_p = a.top_p ? a.top_p[r] : 1.f;
    const float min_p = a.min_p ? a.min_p[r] : 0.f;
    const bool bad_temp = !(temp >= 0.f) || temp == INFINITY;
    const bool one = temp == 0.f || min_p > 1.f;  // only the first of the order is kept
    const bool use_k = one || (top_k > 0 && top_k < a.V);
    const bool use_p = !one && top_p < 1.f;
    const bool use_m = !one && min_p > 0.f;
    float *prow = a.probs ? a.probs + r * a.psr + i * a.psi + e0 : nullptr;
    if (tid < 16) {
        sm.tab.hi[tid] = g_exp_table.hi[tid];
        sm.tab.lo[tid] = g_exp_table.lo[tid];
    }
    if (tid == 0) sm.n_hit = sm.n_list = sm.n_below = sm.n_min = 0;

    // ---- one pass: the largest logit of each of the thread's kParts parts (vector
    // tid + kThreads (part + kParts j), the ragged ends to part 0); zeros to probs
    float tm[kParts];
#pragma unroll
    for (int u = 0; u < kParts; ++u) tm[u] = -INFINITY;
    {
        const Span op = prow ? span_of(reinterpret_cast<const uint32_t *>(prow), row.n)
                             : Span{0, 0, 0};
        const int zeros = prow ? op.nvec : 0;
        float4 *zv = reinterpret_cast<float4 *>(prow + op.head);
        constexpr int kZ = kVec / 4;  // 16-byte stores to each 16-byte load
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int x0 = 0; x0 < sp.nvec; x0 += kParts * kThreads) {
            const int x = x0 + tid;
            uint4 q[kParts];
#pragma unroll
            for (int u = 0; u < kParts; ++u)
                if (x + u * kThreads < sp.nvec) q[u] = __ldg(gv + x + u * kThreads);
#pragma unroll
            for (int u = 0; u < kParts * kZ; ++u) {
                const int z = x0 * kZ + tid + u * kThreads;
                if (z < zeros) __stcs(zv + z, zero);
            }
#pragma unroll
            for (int u = 0; u < kParts; ++u) {
                if (x + u * kThreads >= sp.nvec) break;
                if (kRes) reinterpret_cast<uint4 *>(copy + sp.head)[x + u * kThreads] = q[u];
                const Raw *e = reinterpret_cast<const Raw *>(&q[u]);
#pragma unroll
                for (int k = 0; k < kVec; k += 2)  // (max.f32 passes over NaN)
                    tm[u] = max3f(tm[u], L::wide(e[k]), L::wide(e[k + 1]));
            }
        }
        auto ragged = [&](int x) {
            const Raw v = __ldg(row.g + x);
            if (kRes) copy[x] = v;
            tm[0] = fmaxf(tm[0], L::wide(v));
        };
        if (tid < sp.head) ragged(tid);
        if (tid < row.n - sp.tail) ragged(sp.tail + tid);
        if (prow) {  // what the loop above did not reach
            const int steps = (sp.nvec + kParts * kThreads - 1) / (kParts * kThreads);
            for (int z = steps * kParts * kThreads * kZ + tid; z < zeros; z += kThreads)
                __stcs(zv + z, zero);
            if (tid < op.head) prow[tid] = 0.f;
            if (tid < row.n - op.tail) prow[op.tail + tid] = 0.f;
        }
    }
    // the row's largest logit and its smallest part maximum
    float mx = -INFINITY, lowest = INFINITY;
#pragma unroll
    for (int u = 0; u < kParts; ++u) {
        mx = fmaxf(mx, tm[u]);
        if (tm[u] > -INFINITY) lowest = fminf(lowest, tm[u]);
    }
    auto reduce = [&](float &hi, float &lo, int from) {
#pragma unroll
        for (int o = from; o > 0; o >>= 1) {
            hi = fmaxf(hi, __shfl_xor_sync(kAll, hi, o));
            lo = fminf(lo, __shfl_xor_sync(kAll, lo, o));
        }
    };
    reduce(mx, lowest, 16);
    if (lane == 0) {
        sm.red[0][warp] = mx;
        sm.red[1][warp] = lowest;
    }
    __syncthreads();
    mx = sm.red[0][lane % kWarps];
    lowest = sm.red[1][lane % kWarps];
    reduce(mx, lowest, kWarps / 2);
    if (ncta > 1) {
        if (tid == 0) {
            sm.x_max = mx;
            sm.x_low = lowest;
        }
        cluster_sync();
        if (lane < (int)ncta) {
            mx = *map_to_rank(&sm.x_max, lane);
            lowest = *map_to_rank(&sm.x_low, lane);
        }
        reduce(mx, lowest, 16);
    }
    if (bad_temp || mx == -INFINITY) {  // no distribution (uniform over the cluster)
        cluster_reads_done();
        if (rank == 0 && tid == 0) {
            if (a.tokens) a.tokens[rowi] = -1;
            report_status(a.dev_status, BDSA_DEVICE_OUT_OF_RANGE);
        }
        cluster_wait_reads();
        return;
    }
    if (mx == INFINITY) {
        row.inf = true;
        mx = lowest = 0.f;
#pragma unroll
        for (int u = 0; u < kParts; ++u) tm[u] = if_inf(tm[u]);
    }
    const RowScale rs = row_scale(mx, temp == 0.f ? 1.f : temp);
    float wmax_f;
    const uint64_t wmax = weight(mx, rs, sm.tab, wmax_f);
    const float u01 = a.tokens ? a.u[rowi] : 0.f;
    const uint64_t wmin = use_m ? (min_p >= 1.f ? wmax : scaled(min_p, wmax, true)) : 0;
    const uint64_t want_k = one ? 1u : (uint64_t)top_k;

    // ================================================= the row's weight
    uint64_t all_sum = 0;  // (top-p without top-k)
    if (use_p && !use_k) {
        const uint64_t mine = rs.wide ? sum_stream<T, kRes, true>(row, sp, rs, sm.tab)
                                      : sum_stream<T, kRes, false>(row, sp, rs, sm.tab);
        const uint64_t t = warp_sum64(mine);
        if (lane == 0) sm.scan[warp] = t;
        __syncthreads();
        if (tid == 0) {
            uint64_t v = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += sm.scan[w];
            sm.x_all = v;
        }
        cluster_sync();
        uint64_t x[kMaxCluster];
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) x[c] = c < ncta ? *map_to_rank(&sm.x_all, c) : 0;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) all_sum += x[c];
    }

    // ================================================= filters, by a sorted list
    float pivot_k = -INFINITY;  // at least want_k logits are at or above it
    if (use_k || use_p || use_m) {
        // ---- pivot: nothing below it is kept
        float pivot = -INFINITY;
        bool list = true;
        bool guess = false;  // the pivot is where top-p's estimate ended
        // (top-p within top-k takes its share of all k, min-p's losers included)
        const bool by_m = use_m && !(use_k && use_p);
        if (by_m) {
            // w >= m iff l >= lmax + T ln m, less the rounding of both sides: the
            // logarithm's, 2^-21 absolute near m = 1, counts T times
            const float t = __logf(fminf(min_p, 1.f)) / (rs.ch * 0.693147181f);
            pivot = rs.lmax + t * (t < 0.f ? 1.0001f : 1.f) - 1e-4f * fabsf(rs.lmax) - 1e-5f -
                    1e-6f * temp;
        }
        if ((use_k || use_p) && a.V > kListMax / 4) {
            // A histogram of the part maxima over equal bins of [lowest, lmax],
            // from the top: the pivot is the lower end of the first bin where
            // want_k maxima are reached (want_k logits at least are then at or
            // above it), or where their weights -- taken at the bin's middle, an
            // estimate the exact cut checks -- reach top-p's goal.  A bin that
            // goes far past want_k is cut again.
            float lo = lowest, hi = rs.lmax;
            uint32_t above = 0;  // maxima above hi
            const uint32_t need = (uint32_t)min(want_k, (uint64_t)1 << 20);
            const float goal =
                1.002f * fminf(top_p, 1.f) * (float)all_sum * (524288.f / kUnits);
            for (int level = 0; level < 3; ++level) {
                const float scale = hi > lo ? (float)kBins / (hi - lo) : 0.f;
                sm.parts[tid] = 0;
                if (tid == 0) sm.bin = -1;
                __syncthreads();
#pragma unroll
                for (int u = 0; u < kParts; ++u)
                    if (tm[u] >= lo && tm[u] <= hi)
                        atomicAdd(sm.parts + min(kBins - 1, (int)((hi - tm[u]) * scale)), 1u);
                uint32_t n = 0;
                if (ncta > 1) {
                    cluster_sync();
                    uint32_t x[kMaxCluster];
#pragma unroll
                    for (int c = 0; c < kMaxCluster; ++c)
                        x[c] = c < ncta ? map_to_rank(sm.parts, c)[tid] : 0;
#pragma unroll
                    for (int c = 0; c < kMaxCluster; ++c) n += x[c];
                } else {
                    __syncthreads();
                    n = sm.parts[tid];
                }
                // counts in the low half, weights (units of 2^-19 of the scale,
                // 2^15 part maxima at most) in the high half
                uint64_t v = n;
                if (!use_k && n) {
                    float wf;
                    weight(hi - ((float)tid + 0.5f) * (hi - lo) * (1.f / kBins), rs, sm.tab, wf);
                    v += (uint64_t)((float)n * wf * 65536.f) << 32;
                }
                const uint64_t inc = block_scan64(v, sm.scan);
                const uint32_t upto = above + (uint32_t)inc;
                const float g16 = goal * 0.125f;
                const bool in = use_k ? upto >= need && upto - n < need
                                      : (float)(inc >> 32) >= g16 &&
                                            (float)((inc - v) >> 32) < g16;
                if (in) {
                    sm.bin = tid;
                    sm.bin_c = upto;
                    sm.bin_dc = n;
                }
                if (ncta > 1) cluster_sync();  // (parts have been read everywhere)
                else __syncthreads();
                const int bin = sm.bin;
                if (bin < 0) {  // too few maxima (a later level: the last pivot stands)
                    if (level == 0) lo = -INFINITY;
                    break;
                }
                // the bin's ends, both lowered by more than a rounding of the bin
                // number: every maximum counted is above lo, and none is counted
                // again when the bin is cut (one may be left out, which only
                // lowers the pivot)
                const uint32_t got = (uint32_t)sm.bin_c, in_bin = (uint32_t)sm.bin_dc;
                const float step = (hi - lo) * (1.f / kBins);
                const float eps = 4e-7f * (fabsf(hi) + fabsf(lo) + (hi - lo));
                const float nhi = hi - (float)bin * step - eps;
                lo = fmaxf(lo, hi - (float)(bin + 1) * step - eps);
                __syncthreads();
                if (!use_k || got <= need + need / 4 + 64 || in_bin < 32 || nhi <= lo) break;
                above = got - in_bin;
                hi = nhi;
            }
            if (use_k) pivot_k = lo;
            guess = !use_k && lo > pivot;
            if (lo > -INFINITY) pivot = fmaxf(pivot, lo);
            else list = by_m || a.V <= kListMax;
            // (every maximum at or above the pivot brings a candidate at least)
            if (lo > -INFINITY && (uint32_t)sm.bin_c > kListMax && !by_m) list = false;
        }
        // ---- candidates of the slice: the parts that reach the pivot, then their
        // logits, a warp a part
        if (list) {
#pragma unroll
            for (int u = 0; u < kParts; ++u) {
                if (tm[u] < pivot || tm[u] == -INFINITY) continue;
                const int at = atomicAdd(&sm.n_hit, 1);
                if (at < kListMax) sm.hit[at] = (uint32_t)(tid * kParts + u);
            }
            __syncthreads();
            const int hits = sm.n_hit;
            auto offer = [&](float v, int x) {
                if (row.inf) v = if_inf(v);
                if (v < pivot || v == -INFINITY) return;
                const int at = atomicAdd(&sm.n_list, 1);
                if (at < kListMax)
                    sm.list.own[at] = (uint64_t)~float_key(v) << 32 | (uint32_t)(e0 + x);
            };
            if (hits <= kListMax) {
                for (int h = warp; h < hits; h += kWarps) {
                    const int owner = (int)(sm.hit[h] / kParts), part = (int)(sm.hit[h] % kParts);
                    // element e of the part: vector owner + kThreads (part + kParts j)
                    for (int e = lane;; e += 32) {
                        const int j = e / kVec, x = owner + kThreads * (part + kParts * j);
                        if (x < sp.nvec) {
                            const int at = sp.head + x * kVec + e % kVec;
                            offer(clean(L::wide(row.raw(at))), at);
                        }
                        if (owner + kThreads * (part + kParts * ((e - lane + 32) / kVec)) >=
                            sp.nvec)
                            break;
                    }
                    if (part == 0 && lane == 0) {
                        if (owner < sp.head) offer(clean(L::wide(row.raw(owner))), owner);
                        if (owner < row.n - sp.tail)
                            offer(clean(L::wide(row.raw(sp.tail + owner))), sp.tail + owner);
                    }
                }
            } else if (tid == 0) {
                sm.n_list = kListMax + 1;
            }
        }
        cluster_sync();
        int n = 0;
        if (list) {
            n = gather_lists(sm, ncta);
            list = n <= kListMax && n > 0;
        }
        cluster_reads_done();  // (of the lists)
        // ---- the exact cut
        if (list) {  // (uniform over the cluster)
            __syncthreads();
            uint64_t *keys = sort_list(sm.list.a, sm.list.b, n);
            uint64_t *cum = keys == sm.list.a ? sm.list.b : sm.list.a;
            // (min-p: weights fall with the rank, so the first n_m pass)
            int nm = 0;
            for (int x = tid; x < n; x += kThreads) {
                float wf;
                const uint64_t w = weight(key_float(~(uint32_t)(keys[x] >> 32)), rs, sm.tab, wf);
                cum[x] = w;
                nm += w >= wmin;
            }
            __syncthreads();
            scan_list(cum, n, sm.scan);
            int nk = n;
            if (use_k) nk = (int)min((uint64_t)n, want_k);
            int keep = nk;
            if (use_p) {
                const uint64_t base = use_k ? cum[nk - 1] : all_sum;
                const uint64_t goal =
                    top_p > 0.f ? max((uint64_t)1, scaled(top_p, base, true)) : 1;
                // (the list may stop short of the goal: where the pivot is
                // min-p's, which then keeps no more than the list, or by the
                // estimate, which is caught below)
                int below = 0;
                for (int x = tid; x < nk; x += kThreads) below += cum[x] < goal;
                below = __reduce_add_sync(kAll, below);
                if (lane == 0 && below) atomicAdd(&sm.n_below, below);
            }
            if (use_m) {
                nm = __reduce_add_sync(kAll, nm);
                if (lane == 0 && nm) atomicAdd(&sm.n_min, nm);
            }
            if (use_p || use_m) {
                __syncthreads();
                if (use_p) keep = min(keep, sm.n_below + 1);
                if (use_m) keep = min(keep, sm.n_min);
                // all of the list is below the goal: it is the answer only if min-p
                // ends inside it, or set the pivot
                if (use_p && !use_k && sm.n_below == n &&
                    (!use_m || (guess && sm.n_min == n)))
                    list = false;
            }
            keep = max(keep, 1);
            if (list) {
                const uint64_t total = cum[keep - 1];
                if (prow) {
                    // the kept ones of this slice (over the zeros of the first pass)
                    const float inv = inverse(total);
                    for (int x = tid; x < keep; x += kThreads) {
                        const uint64_t sv = keys[x];
                        const int e = (int)(uint32_t)sv - e0;
                        if (e < 0 || e >= row.n) continue;
                        float wf;
                        weight(key_float(~(uint32_t)(sv >> 32)), rs, sm.tab, wf);
                        prow[e] = wf * inv;
                    }
                }
                if (a.tokens && rank == 0) {
                    const uint64_t target = draw_target(u01, total);
                    auto own = [&](int x) { return cum[x] - (x ? cum[x - 1] : 0); };
                    if (keep <= kThreads) {
                        // each kept one adds up the weights of indices up to its own
                        const int parts = list_parts(keep), x = tid / parts, part = tid % parts;
                        const uint32_t idx = x < keep ? (uint32_t)keys[x] : 0u;
                        uint64_t c = 0;
                        if (x < keep)
                            for (int y = part; y < keep; y += parts)
                                if ((uint32_t)keys[y] <= idx) c += own(y);
                        for (int o = parts >> 1; o > 0; o >>= 1)
                            c += __shfl_xor_sync(kAll, (unsigned long long)c, o);
                        if (x < keep && part == 0 && c > target && c - own(x) <= target)
                            a.tokens[rowi] = (int)idx;
                    } else {
                        // in index order: index << 32 | rank, sorted and summed
                        __syncthreads();
                        for (int x = tid; x < kListMax; x += kThreads)
                            keys[x] = x < keep ? keys[x] << 32 | (uint32_t)x : ~0ull;
                        __syncthreads();
                        bitonic_sort(keys, kListMax);
                        uint64_t w[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int x = 2 * tid + k;
                            w[k] = x < keep ? own((int)(uint32_t)keys[x]) : 0;
                        }
                        const uint64_t t = block_scan64(w[0] + w[1], sm.scan);
                        const uint64_t t0 = t - w[1];
                        if (t0 > target && t0 - w[0] <= target)
                            a.tokens[rowi] = (int)(keys[2 * tid] >> 32);
                        if (t > target && t0 <= target)
                            a.tokens[rowi] = (int)(keys[2 * tid + 1] >> 32);
                    }
                }
                cluster_wait_reads();
                return;
            }
        }
        __syncthreads();
        cluster_wait_reads();  // the lists have been read everywhere: histograms may follow
    }

    // top-p alone: a logit below which the cut cannot be, the one whose weight V
    // times makes the share that may be left out (margins cover the fp32
    // roundings); -inf when there is none
    float low_p = -INFINITY;
    if (use_p && !use_k && all_sum > 0 && top_p < 0.9999f) {
        const float share = (1.f - fmaxf(top_p, 0.f)) * (float)all_sum /
                            (kUnits * (float)a.V * wmax_f);
        if (share > 0.f)
            low_p = rs.lmax + (__logf(share) - 0.01f) / (rs.ch * 0.693147181f) -
                    1e-4f * fabsf(rs.lmax) - 1e-5f;
    }

    // ================================================= a flat row's nucleus
    // The logits above low_p are counted in equal bins, with their places in the
    // bins (in 256ths) added up; each bin's count times the weight of its mean logit
    // says in which bin the cut is, to a fraction of a bin.  (The bins' middles
    // would not do: when one logit holds most of the weight, half a bin of it is
    // more than the few per cent behind the cut.)  One pass then adds up the exact
    // weight above a window of a few bins around it and lists the window's logits;
    // their bins' weights, and a sort of the cut's own bin, give the cut exactly.
    // (If the cut is outside the window, or the window holds too many, by selection
    // below.  61 rows of 100003 fp16 logits with thousands kept: 63 us; by selection
    // alone 118.)
    if (low_p > -INFINITY && low_p < rs.lmax && !use_m && !row.inf && !rs.wide) {
        const float hi = rs.lmax, scale = (float)kWinBins / (hi - low_p);
        uint32_t *win = reinterpret_cast<uint32_t *>(sm.list.a), *place = win + kWinBins;
        static_assert(kWinBins == 4 * kThreads && sizeof(sm.list.a) == 4 * kWinBins &&
                          offsetof(Lists, b) == offsetof(Lists, a) + sizeof(sm.list.a),
                      "counts and places over a and b");
#pragma unroll
        for (int k = 0; k < 8; ++k) win[tid + k * kThreads] = 0;
        if (tid < kWarps) sm.wextra[tid] = 0;
        if (tid <= kWinMax) sm.near[tid] = 0;
        if (tid < 3 * (2 * kWinMax + 1)) (&sm.wbin[0][0])[tid] = 0;
        if (tid == 0) {
            sm.n_list = sm.n_below = sm.n_cut = 0;
            sm.bin = -1;
        }
        __syncthreads();
        // (a logit's bin: monotone in the logit, and the same in either pass)
        for_slice(row, sp, [&](float v) {
            const float t = (hi - v) * scale;
            if (t < (float)kWinBins) {
                atomicAdd(win + (int)t, 1u);
                atomicAdd(place + (int)t, (uint32_t)((t - (float)(int)t) * 256.f));
            }
        });
        cluster_sync();
        uint32_t cnt[4] = {0, 0, 0, 0}, at[4] = {0, 0, 0, 0};
#pragma unroll
        for (int c0 = 0; c0 < kMaxCluster; c0 += 4) {
            uint4 x[4], y[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                x[c] = y[c] = make_uint4(0, 0, 0, 0);
                if (c0 + c < (int)ncta) {
                    x[c] = map_to_rank(reinterpret_cast<const uint4 *>(win), c0 + c)[tid];
                    y[c] = map_to_rank(reinterpret_cast<const uint4 *>(place), c0 + c)[tid];
                }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                cnt[0] += x[c].x;
                cnt[1] += x[c].y;
                cnt[2] += x[c].z;
                cnt[3] += x[c].w;
                at[0] += y[c].x;
                at[1] += y[c].y;
                at[2] += y[c].z;
                at[3] += y[c].w;
            }
        }
        const uint64_t goal = top_p > 0.f ? max((uint64_t)1, scaled(top_p, all_sum, true)) : 1;
        uint64_t est[4], mine = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float wf;
            const float mean = cnt[k] ? ((float)at[k] / (float)cnt[k] + 0.5f) * (1.f / 256.f) : 0.f;
            est[k] = cnt[k] * weight(hi - ((float)(4 * tid + k) + mean) / scale, rs, sm.tab, wf);
            mine += est[k];
        }
        uint64_t upto = block_scan64(mine, sm.scan) - mine;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (upto < goal && upto + est[k] >= goal) sm.bin = 4 * tid + k;
            upto += est[k];
        }
        __syncthreads();
        const int b = sm.bin;
        if (b >= 0) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int d = abs(4 * tid + k - b);
                if (d <= kWinMax && cnt[k]) atomicAdd(sm.near + d, cnt[k]);
            }
        }
        __syncthreads();
        // as wide as the list takes
        int d = -1;
        uint32_t in_win = 0;
        for (int q = 0; q <= kWinMax && b >= 0 && b + q < kWinBins; ++q) {
            in_win += sm.near[q];
            if (in_win > (uint32_t)kListMax) break;
            d = q;
        }
        bool found = d >= 0;
        if (found) {  // (uniform over the cluster)
            const float t0 = (float)(b - d), t1 = (float)(b + d + 1);
            const Segment sg = segment_of(sp, row.n, warp);
            Running run;
            run.clear();
            auto take = [&](float v, int at) {  // the logit, unless it is not above the window
                const float t = (hi - v) * scale;
                if (t < t0) return v;
                if (t < t1) {
                    const int n = atomicAdd(&sm.n_list, 1);
                    if (n < kListMax)
                        sm.list.own[n] = (uint64_t)~float_key(v) << 32 | (uint32_t)(e0 + at);
                }
                return -INFINITY;
            };
            auto add = [&](float v0, float v1) {
                V2 h, l;
                weight_ff<V2, false>(V2{f2_pack(v0, v1)}, rs, sm.tab, h, l);
                run.add(h, l);
            };
            for (int x = sg.head0 + lane; x < sg.head1; x += 32) add(take(row.at(x), x), -INFINITY);
            for (int x = sg.tail0 + lane; x < sg.tail1; x += 32) add(take(row.at(x), x), -INFINITY);
            const uint4 *sv = reinterpret_cast<const uint4 *>((kRes ? row.s : row.g) + sp.head);
            constexpr int kU = kRes ? 2 : 4;
            for (int x0 = sg.v0 + lane; x0 < sg.v1; x0 += 32 * kU) {
                uint4 q[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u)
                    if (x0 + 32 * u < sg.v1) q[u] = row.vec(sv + x0 + 32 * u);
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    if (x0 + 32 * u >= sg.v1) break;
                    const Raw *e = reinterpret_cast<const Raw *>(&q[u]);
                    const int at = sp.head + (x0 + 32 * u) * kVec;
#pragma unroll
                    for (int k = 0; k < kVec; k += 2)
                        add(take(clean(L::wide(e[k])), at + k),
                            take(clean(L::wide(e[k + 1])), at + k + 1));
                }
            }
            __syncwarp();
            uint64_t sum = warp_sum64(run.units(0, 0));
            if (lane == 0) sm.scan[warp] = sum;
            __syncthreads();
            if (tid == 0) {
                uint64_t v = 0;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) v += sm.scan[w];
                sm.x_above = v;
            }
            cluster_sync();
            uint64_t above = 0, xa[kMaxCluster];
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c)
                xa[c] = c < ncta ? *map_to_rank(&sm.x_above, c) : 0;
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c) above += xa[c];
            const int n = gather_lists(sm, ncta);
            __syncthreads();
            found = n > 0 && n <= kListMax && above < goal;
            if (found) {
                // the weights of the window's bins, then of the cut's bin one by one
                uint64_t key[2], w[2];
                int bin[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int x = tid + k * kThreads;
                    key[k] = x < n ? sm.list.a[x] : ~0ull;
                    const float v = key_float(~(uint32_t)(key[k] >> 32));
                    float wf;
                    w[k] = x < n ? weight(v, rs, sm.tab, wf) : 0;
                    bin[k] = x < n ? (int)((hi - v) * scale) - (b - d) : -1;
                    if (x < n) {
                        const uint32_t l0 = (uint32_t)w[k] & 0x3fffu;
                        const uint32_t l1 = (uint32_t)(w[k] >> 14) & 0x3fffu;
                        atomicAdd(&sm.wbin[bin[k]][0], l0);
                        atomicAdd(&sm.wbin[bin[k]][1], l1);
                        atomicAdd(&sm.wbin[bin[k]][2], (uint32_t)(w[k] >> 28));
                    }
                }
                __syncthreads();
                int cut = -1;
                for (int q = 0; q <= 2 * d; ++q) {
                    const uint64_t m = (uint64_t)sm.wbin[q][0] + ((uint64_t)sm.wbin[q][1] << 14) +
                                       ((uint64_t)sm.wbin[q][2] << 28);
                    if (above + m >= goal) {
                        cut = q;
                        break;
                    }
                    above += m;
                }
                found = cut >= 0;
                if (found) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (bin[k] == cut) sm.list.b[atomicAdd(&sm.n_cut, 1)] = key[k];
                    __syncthreads();
                    const int m = sm.n_cut;
                    uint64_t *keys = sort_list(sm.list.b, sm.list.a, m);
                    uint64_t *cum = keys == sm.list.a ? sm.list.b : sm.list.a;
                    for (int x = tid; x < m; x += kThreads) {
                        float wf;
                        cum[x] = weight(key_float(~(uint32_t)(keys[x] >> 32)), rs, sm.tab, wf);
                    }
                    __syncthreads();
                    scan_list(cum, m, sm.scan);
                    int below = 0;
                    for (int x = tid; x < m; x += kThreads) below += above + cum[x] < goal;
                    below = __reduce_add_sync(kAll, below);
                    if (lane == 0 && below) atomicAdd(&sm.n_below, below);
                    __syncthreads();
                    const uint64_t last = keys[sm.n_below];
                    // the kept ones of the window, to their warps' segments
                    const int per = (sp.nvec + kWarps - 1) / kWarps * kVec;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int e = (int)(uint32_t)key[k] - e0;
                        if (key[k] > last || e < 0 || e >= row.n) continue;
                        const int q = e < sp.head   ? 0
                                      : e >= sp.tail ? kWarps - 1
                                                     : (e - sp.head) / per;
                        atomicAdd((unsigned long long *)&sm.wextra[q], (unsigned long long)w[k]);
                    }
                    __syncthreads();
                    sum += sm.wextra[warp];
                    uint64_t total, before;
                    share_sums(sm.draw, sum, ncta, rank, total, before);
                    cluster_reads_done();
                    auto kept = [&](float v, int x) {
                        return ((uint64_t)~float_key(v) << 32 | (uint32_t)(e0 + x)) <= last;
                    };
                    if (a.tokens) {
                        const uint64_t target = draw_target(u01, total);
                        const int w = warp_of_target(sm.draw, target, before);
                        if (w >= 0) {
                            const Segment g = segment_of(sp, row.n, w);
                            const int x0 = g.head1 > g.head0 ? 0 : sp.head + g.v0 * kVec;
                            const int x1 = g.tail1 > g.tail0 ? row.n : sp.head + g.v1 * kVec;
                            for (int base = x0; base < x1; base += 4 * kThreads) {
                                const int x = base + 4 * tid;
                                uint64_t q[4], s4 = 0;
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const float v = x + k < x1 ? row.at(x + k) : -INFINITY;
                                    float wf;
                                    q[k] = x + k < x1 && kept(v, x + k) ? weight(v, rs, sm.tab, wf)
                                                                        : 0;
                                    s4 += q[k];
                                }
                                draw_in_block(sm.draw, target, before, q, s4, e0 + x,
                                              a.tokens + rowi);
                            }
                        }
                    }
                    if (prow) {  // over the zeros of the first pass
                        const float inv = inverse(total);
                        const int seg = ((row.n + kWarps - 1) / kWarps + 31) & ~31;
                        const int w0 = min(row.n, warp * seg), w1 = min(row.n, w0 + seg);
                        for_selected(row, w0, w1, lane, kept, [&](int x) {
                            float wf;
                            weight(row.at(x), rs, sm.tab, wf);
                            prow[x] = wf * inv;
                        });
                    }
                    cluster_wait_reads();
                    return;
                }
            }
        }
        cluster_sync();  // counts and lists have been read everywhere
    }

    // ================================================= any row, by selection
    const int seg = ((row.n + kWarps - 1) / kWarps + 31) & ~31;
    const int w0 = min(row.n, warp * seg), w1 = min(row.n, w0 + seg);
    Cut cut{0, ~0ull};       // everything
    uint64_t key_count = 0;  // elements with the cut's key
    if (use_k || use_p) {
        // The keys the cut can be among: from the pivot of top-k (want_k logits
        // are at or above it); for top-p alone from low_p; else from the smallest
        // logit.
        const uint32_t kmax = R::key(rs.lmax);
        uint32_t kmin = 0xffffffffu;
        if (pivot_k > -INFINITY) {
            kmin = R::key(pivot_k);
        } else if (low_p > -INFINITY) {
            kmin = min(kmax, R::key(low_p));
        }
        if (kmin == 0xffffffffu) {
            const uint32_t kinf = R::key(-INFINITY);
            kmin = kmax;
            for (int x = tid; x < row.n; x += kThreads) {
                const uint32_t k = R::key(row.at(x));
                if (k > kinf) kmin = min(kmin, k);
            }
            kmin = __reduce_min_sync(kAll, kmin);
            if (tid == 0) sm.x_min = kmax;
            __syncthreads();
            if (lane == 0) atomicMin(&sm.x_min, kmin);
            cluster_sync();
            for (uint32_t c = 0; c < ncta; ++c) kmin = min(kmin, *map_to_rank(&sm.x_min, c));
        }
        int buf = 0;
        const Level lv =
            level_hist(row, w0, w1, sm, buf, kmin, kmax, range_shift(kmin, kmax), rs, ncta);
        // totals of the range (the last thread's inclusive prefix)
        if (tid == kThreads - 1) {
            sm.bin_c = lv.c + lv.dc;
            sm.bin_m = lv.m + lv.dm;
        }
        __syncthreads();
        const uint64_t all_c = sm.bin_c, all_m = sm.bin_m;
        __syncthreads();
        uint64_t total = !use_k && all_sum > 0 ? all_sum : all_m, above = 0;
        if (use_k && want_k <= all_c) {
            cut = select_cut<false>(row, w0, w1, sm, buf, lv, kmin, kmax, want_k, rs, ncta, above,
                                    key_count);
            float wf;
            total = above + cut.ties * weight(R::value(cut.key), rs, sm.tab, wf);
        }
        if (use_p) {
            // (the range's own weights round one by one, the row's weight at
            // once: the goal stays within the range)
            uint64_t target = top_p > 0.f ? max((uint64_t)1, scaled(top_p, total, true)) : 1;
            target = min(target, all_m);
            uint64_t kc2 = 0;
            const Cut c2 = select_cut<true>(row, w0, w1, sm, buf, lv, kmin, kmax, target, rs, ncta,
                                            above, kc2);
            if (c2.key > cut.key || (c2.key == cut.key && c2.ties < cut.ties)) {
                cut = c2;
                key_count = kc2;
            }
        }
    }

    // ---- the cut's ties: the first cut.ties of key_count by index.  A warp
    // owns the contiguous segment [w0, w1) of the slice; tie_end: the warp's
    // elements with the cut's key are kept below this index.
    int tie_end = w1;
    if (cut.ties < key_count) {
        uint32_t mine = 0;
        for (int x = w0 + lane; x < w1; x += 32) mine += R::key(row.at(x)) == cut.key;
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
                const unsigned m = __ballot_sync(kAll, x < w1 && R::key(row.at(x)) == cut.key);
                const uint32_t n = __popc(m);
                // the (left - seen)-th set bit of m ends the kept ties
                if (seen + n >= left) tie_end = x0 + (int)__fns(m, 0, (int)(left - seen)) + 1;
                seen += n;
            }
        }
    }

    // ---- kept weight, the draw, the distribution
    auto in_cut_by = [&](float v, int x, int ends) {
        if (!(use_k || use_p)) return true;
        const uint32_t key = R::key(v);
        return key > cut.key || (key == cut.key && x < ends);
    };
    auto in_cut = [&](float v, int x) { return in_cut_by(v, x, tie_end); };
    auto kept = [&](int x, float &wf, int ends) -> uint64_t {
        const float v = row.at(x);
        wf = 0.f;
        if (!in_cut_by(v, x, ends)) return 0;
        const uint64_t w = weight(v, rs, sm.tab, wf);
        if (w < wmin) {
            wf = 0.f;
            return 0;
        }
        return w;
    };
    uint64_t sum = 0;
    for_selected(row, w0, w1, lane, in_cut, [&](int x) {
        float wf;
        sum += kept(x, wf, tie_end);
    });
    sum = warp_sum64(sum);
    uint64_t total, before;
    share_sums(sm.draw, sum, ncta, rank, total, before);
    cluster_reads_done();
    if (a.tokens) {
        const uint64_t target = draw_target(u01, total);
        const int w = warp_of_target(sm.draw, target, before);
        if (w >= 0) {  // the draw is in warp w's segment of this slice
            // (that warp's ties end where it says)
            if (warp == w && lane == 0) sm.bin = tie_end;
            __syncthreads();
            const int x0 = w * seg, x1 = min(row.n, x0 + seg), ends = sm.bin;
            for (int base = x0; base < x1; base += 4 * kThreads) {
                const int x = base + 4 * tid;
                uint64_t q[4], s4 = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float wf;
                    q[k] = x + k < x1 ? kept(x + k, wf, ends) : 0;
                    s4 += q[k];
                }
                draw_in_block(sm.draw, target, before, q, s4, e0 + x, a.tokens + rowi);
            }
        }
    }
    if (prow) {  // over the zeros of the first pass (tie_end is the segment's)
        const float inv = inverse(total);
        for_selected(row, w0, w1, lane, in_cut, [&](int x) {
            float wf;
            kept(x, wf, tie_end);
            prow[x] = wf * inv;
        });
    }
    cluster_wait_reads();
}

// Slices that stay in shared memory: two of them fit an SM (61 rows of 100003 fp16,
// four slices each: 63 us, read again from L2 65).
constexpr size_t kMaxResident = 72 * 1024;

template <typename K>
int launch_cluster(K *kernel, const SampleArgs &a, int threads, size_t smem, cudaStream_t stream) {
    // (the same limit in every call, so that host threads do not undo one another's)
    if (smem > 0 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kMaxResident) != cudaSuccess)
        return BDSA_CUDA_ERROR;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long)a.bs * a.B * a.ncta));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.ncta;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? BDSA_OK : BDSA_CUDA_ERROR;
}

template <typename T>
int launch_typed(const SampleArgs &in, int num_sms, cudaStream_t stream) {
    SampleArgs a = in;
    const long rows = (long)a.bs * a.B;
    auto set_slices = [&](int ncta) {
        a.ncta = ncta;
        a.slice = (int)((((long)a.V + ncta - 1) / ncta + 31) & ~31L);
    };
    // one CTA a row when there is a row for every SM, else slices of at least 4096
    // (512 fp32 rows of 151936, filtered: one CTA a row 120 us, two 137, four 168)
    int ncta = 1;
    while (ncta < kMaxCluster &&
           ((rows * ncta <= num_sms && a.V / (2 * ncta) >= 4096) || a.V > ncta * (1 << 18)))
        ncta *= 2;
    if (!a.top_k && !a.top_p && !a.min_p) {
        // (two CTAs a row, four to an SM pair: the rows in flight, as stored
        // weights, fit L2 up to V = 200 k; 480 bf16 rows of 151936 168 us, with one
        // CTA 198, three 181, four 186)
        if (ncta < 2 && a.probs && a.V >= 16384) ncta = 2;
        set_slices(ncta);
        return launch_cluster(sample_full_kernel<T>, a, kThreads, 0, stream);
    }
    set_slices(ncta);
    // small slices stay in shared memory for the later passes
    const size_t smem = (size_t)a.slice * sizeof(T) + 16;
    if (smem <= kMaxResident)
        return launch_cluster(sample_cut_kernel<T, true>, a, kThreads, smem, stream);
    return launch_cluster(sample_cut_kernel<T, false>, a, kThreads, 0, stream);
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
