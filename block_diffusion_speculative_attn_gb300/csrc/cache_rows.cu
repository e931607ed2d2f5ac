// cache_rows.cu -- rows of the paged cache written, copied and moved.
//
// A row is one slot's keys (or values) of every KV head: row_bytes contiguous
// bytes, a page is page_size of them.  The three kernels move rows and compute
// nothing, so the bytes, each read and written once, bound them; every thread has
// several independent 16-byte loads in flight before its first store.
#include <cuda_runtime.h>
#include <limits.h>

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
// CTA (columns, request, cache).  Kept row i, at position L + path[i], moves to L + i.
// path runs up strictly, so path[i] >= i and a row's place never lies behind a row
// that has yet to be read by a later batch: a batch is read whole, then written.
constexpr int kMoveRows = 8;  // rows a thread has in flight

__global__ void __launch_bounds__(kThreads)
    cache_compact_kernel(const CompactArgs a, const __grid_constant__ CacheList caches, int r0,
                         int lanes, int cols) {
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ int s_count;
    const int r = r0 + blockIdx.y, tid = threadIdx.x;
    const int32_t *path = a.path + (long long)r * a.width;
    const int32_t *bt = a.block_table + (long long)r * a.max_pages;
    const int L = __ldg(a.seq_lens + r);
    // ---- the kept rows' number: entries before the first -1
    if (tid == 0) s_count = a.width;
    __syncthreads();
    int stop = a.width;
    for (int i = tid; i < a.width; i += kThreads)
        if (__ldg(path + i) == -1) {
            stop = i;
            break;
        }
    if (stop < a.width) atomicMin(&s_count, stop);
    __syncthreads();
    const int m = s_count;
    // ---- every row and every place on a page of the pool, else nothing moves
    const long long room = (long long)a.max_pages * a.page_size;
    auto slot_of = [&](int i) -> long long {  // of position L + i
        const uint32_t p = (uint32_t)L + (uint32_t)i, ps = (uint32_t)a.page_size;
        return (long long)__ldg(bt + p / ps) * a.page_size + p % ps;
    };
    auto in_pool = [&](int i) {
        const int id = __ldg(bt + ((uint32_t)L + (uint32_t)i) / (uint32_t)a.page_size);
        return id >= 0 && id < a.num_pages;
    };
    bool bad = false;
    for (int i = tid; i < m; i += kThreads) {
        const int x = __ldg(path + i), before = i > 0 ? __ldg(path + i - 1) : -1;
        const bool ok = L >= 0 && x > before && x >= i && (long long)L + x < room;
        bad |= !ok || !in_pool(x) || !in_pool(i);
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) report_status(a.dev_status, BDSA_DEVICE_OUT_OF_RANGE);
        return;
    }
    // ---- the rows, in batches of `per` * kMoveRows
    const int per = kThreads / lanes, group = tid / lanes, lane = tid % lanes;
    const int vecs = (int)(a.row_bytes / 16);
    const int v0 = blockIdx.x * cols, v1 = min(vecs, v0 + cols);
    uint8_t *cache = caches.p[blockIdx.z];
    for (int i0 = 0; i0 < m; i0 += per * kMoveRows) {
        for (int v = v0 + lane; v < v1 + lane; v += lanes) {  // (the same count for all)
            uint4 x[kMoveRows];
            long long to[kMoveRows];
#pragma unroll
            for (int k = 0; k < kMoveRows; ++k) {
                const int i = i0 + k * per + group;
                to[k] = -1;
                if (i >= m || v >= v1) continue;
                const int from = __ldg(path + i);
                if (from == i) continue;  // in its place already
                x[k] = ld_stream(cache + slot_of(from) * a.row_bytes + v * 16LL);
                to[k] = slot_of(i) * a.row_bytes + v * 16LL;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kMoveRows; ++k)
                if (to[k] >= 0) st_vec(cache + to[k], x[k]);
        }
        // (a later batch reads no place of this one: its rows are at or behind
        // their own places, which follow this batch's)
    }
}

template <typename K, typename... A>
cudaError_t launch(K kernel, dim3 grid, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

int launch_cache_write(const WriteArgs &a, int num_sms, cudaStream_t stream) {
    const int lanes = lanes_of(a.row_bytes / 16);
    const int per = kThreads / lanes * kWriteRows;  // tokens a CTA takes at once
    const long long want = ((long long)a.T + per - 1) / per, most = 8LL * num_sms;
    const unsigned grid = (unsigned)(want < most ? want : most);
    return launch(cache_write_kernel, dim3(grid), stream, a, lanes) == cudaSuccess
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
            if (launch(cache_copy_kernel, dim3(chunks, ne, nc), stream, a, list, e0) !=
                cudaSuccess)
                return BDSA_CUDA_ERROR;
        }
    }
    return BDSA_OK;
}

int launch_cache_compact(const CompactArgs &a, void *const *caches, int n_caches, int num_sms,
                         cudaStream_t stream) {
    const int vecs = (int)(a.row_bytes / 16);
    for (int c0 = 0; c0 < n_caches; c0 += kCachesPerLaunch) {
        const int nc = n_caches - c0 < kCachesPerLaunch ? n_caches - c0 : kCachesPerLaunch;
        CacheList list = {};
        for (int i = 0; i < nc; ++i) list.p[i] = static_cast<uint8_t *>(caches[c0 + i]);
        // a row's columns are split while there are fewer CTAs than fill the GPU
        int cols = vecs;
        while (cols > 8 && (long long)a.bs * nc * ((vecs + cols - 1) / cols) < 4LL * num_sms)
            cols = (cols + 1) / 2;
        const int lanes = lanes_of(cols);
        for (int r0 = 0; r0 < a.bs; r0 += 65535) {
            const unsigned nr = (unsigned)(a.bs - r0 < 65535 ? a.bs - r0 : 65535);
            if (launch(cache_compact_kernel, dim3((vecs + cols - 1) / cols, nr, nc), stream, a,
                       list, r0, lanes, cols) != cudaSuccess)
                return BDSA_CUDA_ERROR;
        }
    }
    return BDSA_OK;
}

}  // namespace bdsa
