// cache_rows.cu -- rows of the paged cache written, copied and moved.
//
// A row is one slot's keys (or values) of every KV head: row_bytes contiguous
// bytes, a page is page_size of them.  The three kernels move rows and compute
// nothing, so the bytes, each read and written once, bound them; every thread has
// several independent 16-byte loads in flight before its first store.
#include <cuda_runtime.h>
#include <limits.h>

#include "attn_common.cuh"
#include "bdsa_device.cuh"
#include "bdsa_internal.h"
#include "cache_internal.h"

namespace bdsa {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint4 ld_stream(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}
__device__ __forceinline__ void st_vec(uint8_t *p, uint4 v) {
    asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w)
                 : "memory");
}

// Lanes that share a row of `vecs` 16-byte pieces: a power of two, at most a CTA.
int lanes_of(int vecs) {
    int n = 1;
    while (n < vecs && n < kThreads) n *= 2;
    return n;
}

// ---------------------------------------------------------------- write
// Tokens are dealt to groups of `lanes` threads, kWriteRows at a time.
constexpr int kWriteRows = 4;

__global__ void __launch_bounds__(kThreads) cache_write_kernel(const WriteArgs a, int lanes) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int per = kThreads / lanes, vecs = a.row_bytes / 16;
    const int group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
    bool report = false;
    for (long long t0 = ((long long)blockIdx.x * per + group) * kWriteRows; t0 < a.T;
         t0 += (long long)gridDim.x * per * kWriteRows) {
        long long slot[kWriteRows];
#pragma unroll
        for (int k = 0; k < kWriteRows; ++k) {
            const int s = t0 + k < a.T ? __ldg(a.slot_map + t0 + k) : -1;
            report |= s < -1 || s >= a.num_slots;
            slot[k] = s >= 0 && s < a.num_slots ? s : -1;
        }
        for (int v = lane; v < vecs; v += lanes) {
            uint4 x[2][kWriteRows];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < kWriteRows; ++k)
                    if (slot[k] >= 0)
                        x[i][k] = ld_stream(a.src[i] + (t0 + k) * a.stride[i] + (long long)v * 16);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < kWriteRows; ++k)
                    if (slot[k] >= 0)
                        st_vec(a.cache[i] + slot[k] * a.row_bytes + (long long)v * 16, x[i][k]);
        }
    }
    if (report) report_status(a.dev_status, BDSA_DEVICE_OUT_OF_RANGE);
}

// ---------------------------------------------------------------- copy
// CTA (chunk, entry, cache): kCopyBytes of the entry's rows, which lie in a row.
constexpr int kCopyVecs = 8;                             // a thread
constexpr long long kCopyBytes = 16LL * kCopyVecs * kThreads;

__global__ void __launch_bounds__(kThreads)
    cache_copy_kernel(const CopyArgs a, const __grid_constant__ CacheList caches, int e0) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int e = e0 + blockIdx.y;
    const int len = __ldg(a.len + e), s = __ldg(a.src + e), d = __ldg(a.dst + e);
    if (len == 0 || (s == -1 && d == -1)) return;
    if (len < 0 || len > a.page_size || s < 0 || s >= a.num_pages || d < 0 || d >= a.num_pages) {
        if (threadIdx.x == 0) report_status(a.dev_status, BDSA_DEVICE_OUT_OF_RANGE);
        return;
    }
    const long long page = a.page_size * a.row_bytes, end = len * a.row_bytes;
    const uint8_t *from = caches.p[blockIdx.z] + s * page;
    uint8_t *to = caches.p[blockIdx.z] + d * page;
    for (long long at = blockIdx.x * kCopyBytes; at < end; at += gridDim.x * kCopyBytes) {
        uint4 x[kCopyVecs];
#pragma unroll
        for (int k = 0; k < kCopyVecs; ++k) {
            const long long o = at + (k * kThreads + threadIdx.x) * 16LL;
            if (o < end) x[k] = ld_stream(from + o);
        }
#pragma unroll
        for (int k = 0; k < kCopyVecs; ++k) {
            const long long o = at + (k * kThreads + threadIdx.x) * 16LL;
            if (o < end) st_vec(to + o, x[k]);
        }
    }
}

// ---------------------------------------------------------------- compact
// Kept row i, at position L + path[i], moves to L + i.  path runs up strictly, so
// path[i] >= i: a place is never behind a row that has yet to be read.  A thread owns
// 16 bytes of the row of one cache and reads kMoveRows rows before it writes them, so
// no two threads meet and none waits for another; where no row lies on another's
// place (all that move lie past the kept rows' region), several CTAs share a
// request's rows.  Where some do, one CTA a request and column of bytes is left: 4000
// rows of 16 caches without 100 of them take 557 us for one request (the bytes 38), 916
// for 16 (604).  The slots of 32 rows are looked up by the lanes of a warp, one each,
// and passed round.
constexpr int kMoveThreads = 128;
// Rows a thread has in flight and CTAs an SM that a call is cut into: 16 chats of 16
// caches, about 1000 kept rows each, 164 us (0.89 of the copy rate); with 8 CTAs 178,
// 16 rows and 8, 4, 1 CTAs 169, 182, 195; 32 short paths of 32 caches 8.6 us, with 16
// rows 9.8.
constexpr int kMoveRows = 8;
constexpr int kMoveCtas = 16;

__global__ void __launch_bounds__(kMoveThreads)
    cache_compact_kernel(const CompactArgs a, const __grid_constant__ CacheList caches,
                         int n_caches, int r0) {
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ int s_count;
    const int r = r0 + blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    const int32_t *path = a.path + (long long)r * a.width;
    const int32_t *bt = a.block_table + (long long)r * a.max_pages;
    const int L = __ldg(a.seq_lens + r);
    // ---- the kept rows' number: entries before the first -1
    if (tid == 0) s_count = a.width;
    __syncthreads();
    for (int i0 = 0; i0 < a.width; i0 += kMoveThreads) {
        const bool end = i0 + tid < a.width && __ldg(path + i0 + tid) == -1;
        if (end) atomicMin(&s_count, i0 + tid);
        if (__syncthreads_or(end)) break;
    }
    const int m = s_count;
    // ---- every row and every place on a page of the pool, else nothing moves
    const long long room = (long long)a.max_pages * a.page_size;
    const uint32_t ps = (uint32_t)a.page_size;
    auto in_pool = [&](int i) {
        const int id = __ldg(bt + ((uint32_t)L + (uint32_t)i) / ps);
        return id >= 0 && id < a.num_pages;
    };
    bool bad = false, near = false;
    for (int i = tid; i < m; i += kMoveThreads) {
        const int x = __ldg(path + i), before = i > 0 ? __ldg(path + i - 1) : -1;
        const bool ok = L >= 0 && x > before && x >= i && (long long)L + x < room;
        bad |= !ok || !in_pool(x) || !in_pool(i);
        near |= x > i && x < m;
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) report_status(a.dev_status, BDSA_DEVICE_OUT_OF_RANGE);
        return;
    }
    // the request's CTAs share its rows, unless a row lies on the place of another
    const bool alone = __syncthreads_or(near) != 0;
    const int part = blockIdx.z, parts = alone ? 1 : gridDim.z;
    if (alone && part > 0) return;
    // ---- the rows
    const int vecs = (int)(a.row_bytes / 16);
    const long long column = (long long)blockIdx.x * kMoveThreads + tid;
    const int c = (int)(column / vecs);
    const bool mine = c < n_caches;
    uint8_t *cache = caches.p[mine ? c : 0] + (column % vecs) * 16;
    auto slot_of = [&](int i) -> int {  // of position L + i
        const uint32_t p = (uint32_t)L + (uint32_t)i;
        return __ldg(bt + p / ps) * a.page_size + (int)(p % ps);
    };
    // the slots of row i and of its place (-1: there already, or no row)
    auto look_up = [&](int i) -> int2 {
        const int x = i < m ? __ldg(path + i) : i;
        return x == i ? make_int2(-1, 0) : make_int2(slot_of(x), slot_of(i));
    };
    const int step = parts * 32;
    int2 next = look_up(part * 32 + lane);
    for (int i0 = part * 32; i0 < m; i0 += step) {
        const int2 now = next;
        next = look_up(i0 + step + lane);
        if (!__any_sync(0xffffffffu, now.x >= 0)) continue;
#pragma unroll
        for (int b = 0; b < 32; b += kMoveRows) {
            uint4 x[kMoveRows];
#pragma unroll
            for (int k = 0; k < kMoveRows; ++k) {
                const int f = __shfl_sync(0xffffffffu, now.x, b + k);
                if (mine && f >= 0) x[k] = ld_stream(cache + f * a.row_bytes);
            }
#pragma unroll
            for (int k = 0; k < kMoveRows; ++k) {
                const int f = __shfl_sync(0xffffffffu, now.x, b + k);
                const int d = __shfl_sync(0xffffffffu, now.y, b + k);
                if (mine && f >= 0) st_vec(cache + d * a.row_bytes, x[k]);
            }
        }
    }
}

}  // namespace

int launch_cache_write(const WriteArgs &a, int num_sms, cudaStream_t stream) {
    const int lanes = lanes_of(a.row_bytes / 16);
    const int per = kThreads / lanes * kWriteRows;  // tokens a CTA takes at once
    const long long want = ((long long)a.T + per - 1) / per, most = 8LL * num_sms;
    const unsigned grid = (unsigned)(want < most ? want : most);
    return launch_pdl(cache_write_kernel, dim3(grid), dim3(kThreads), 0, stream, a, lanes) == cudaSuccess
               ? BDSA_OK
               : BDSA_CUDA_ERROR;
}

int launch_cache_copy(const CopyArgs &a, void *const *caches, int n_caches, cudaStream_t stream) {
    const long long page = a.page_size * a.row_bytes;
    const long long want = (page + kCopyBytes - 1) / kCopyBytes;
    const unsigned chunks = (unsigned)(want < 1024 ? want : 1024);
    for (int c0 = 0; c0 < n_caches; c0 += kCachesPerLaunch) {
        const int nc = n_caches - c0 < kCachesPerLaunch ? n_caches - c0 : kCachesPerLaunch;
        CacheList list = {};
        for (int i = 0; i < nc; ++i) list.p[i] = static_cast<uint8_t *>(caches[c0 + i]);
        for (int e0 = 0; e0 < a.n; e0 += 65535) {
            const unsigned ne = (unsigned)(a.n - e0 < 65535 ? a.n - e0 : 65535);
            if (launch_pdl(cache_copy_kernel, dim3(chunks, ne, nc), dim3(kThreads), 0, stream, a,
                           list, e0) != cudaSuccess)
                return BDSA_CUDA_ERROR;
        }
    }
    return BDSA_OK;
}

int launch_cache_compact(const CompactArgs &a, void *const *caches, int n_caches, int num_sms,
                         cudaStream_t stream) {
    const long long vecs = a.row_bytes / 16;
    for (int c0 = 0; c0 < n_caches; c0 += kCachesPerLaunch) {
        const int nc = n_caches - c0 < kCachesPerLaunch ? n_caches - c0 : kCachesPerLaunch;
        CacheList list = {};
        for (int i = 0; i < nc; ++i) list.p[i] = static_cast<uint8_t *>(caches[c0 + i]);
        const unsigned grid = (unsigned)((nc * vecs + kMoveThreads - 1) / kMoveThreads);
        // (each CTA checks the whole path: not more of them than fill the GPU)
        const long long ctas = (long long)grid * a.bs, rows32 = ((long long)a.width + 31) / 32;
        long long parts = kMoveCtas * num_sms / ctas;
        parts = parts < 1 ? 1 : parts < rows32 ? parts : rows32;
        for (int r0 = 0; r0 < a.bs; r0 += 65535) {
            const unsigned nr = (unsigned)(a.bs - r0 < 65535 ? a.bs - r0 : 65535);
            if (launch_pdl(cache_compact_kernel, dim3(grid, nr, (unsigned)parts),
                           dim3(kMoveThreads), 0, stream, a, list, nc, r0) != cudaSuccess)
                return BDSA_CUDA_ERROR;
        }
    }
    return BDSA_OK;
}

}  // namespace bdsa
