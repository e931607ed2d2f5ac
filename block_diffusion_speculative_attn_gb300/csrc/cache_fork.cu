// cache_fork.cu -- rows of the block table continued from rows of an old one.
//
// New row r holds the first t_r = keep[r] tokens of old row parent[r]: its first
// floor(t_r / ps) pages, whole, are shared with whoever else continues them; its
// partial last page can have one writer only, so the first row that ends in it keeps
// it if no row holds it whole, and every other row gets a fresh page and an entry in
// the list of copies.  Old pages that no new row holds go back to the ring.
//
// Who holds a page is counted, not remembered: each call scatters over the pool, for
// every page, its first entry in the old table (atomic min), the new rows that hold
// it whole (atomic add) and the first that ends in it (atomic min).  The results of
// those do not depend on their order, so neither do the tables or the ring.  Four
// steps, with a warp for each part of a row (kPart entries at most, a whole row where
// there are many rows; 16 rows of 8192 pages by whole rows 506 us, in parts 22):
//   clear   the scattered arrays
//   mark    the three scatters
//   count   pages that each old row gives back, new rows that need a fresh page
//   write   the new table, the copies, the ring (every CTA sums the counts itself)
#include <cuda_runtime.h>
#include <limits.h>

#include "attn_common.cuh"
#include "bdsa_device.cuh"
#include "bdsa_internal.h"
#include "cache_internal.h"

namespace bdsa {
namespace {

constexpr uint32_t kNone = 0xFFFFFFFFu;
constexpr int kForkThreads = 512, kForkCtas = 16;
// Table entries and pages, and parts of rows, up to which one cluster takes the call (a
// launch instead of four, about 10 us of the host's time): 64 rows of 64 pages 11.4 us
// in one cluster, 11.8 in four grids; 256 rows 16 and 12, 512 rows 26 and 13, 2048 rows
// of 128 pages 114 and 27.  Its 256 warps take the parts in turns, however short: 256
// rows of 4 pages (512 parts) 12.6 and 10.4, 1024 rows of 1 page 30 and 14, 10000 rows
// 263 and 44.
constexpr long long kClusterWork = 1 << 15;
constexpr long long kClusterParts = 1024;
// Entries of a warp's part of a row at most; more where a table's parts would be more
// than kMaxParts.
constexpr int kPart = 128, kMaxParts = BDSA_TABLE_MAX_REQUESTS;

// The part of the work that a warp takes.
struct Share {
    long long warp, warps;  // this warp of how many
    int lane;
};
__device__ __forceinline__ Share share() {
    const int per = blockDim.x / 32;
    return {(long long)blockIdx.x * per + threadIdx.x / 32, (long long)gridDim.x * per,
            (int)threadIdx.x % 32};
}

// Pages of an old row (0: owned pages that mean nothing).
__device__ __forceinline__ int owned_pages(const ForkArgs &a, int r, bool &bad) {
    const int n = __ldg(a.owned + r);
    bad = n < 0 || n > a.max_pages;
    return bad ? 0 : n;
}

// What a new row keeps.
struct Kept {
    const int32_t *row;  // the parent's
    int whole, tail;     // pages it holds whole, tokens in the last one
    bool bad;            // a parent or a length that means nothing: the row is empty
};
__device__ __forceinline__ Kept kept_of(const ForkArgs &a, int r) {
    Kept k{a.block_table, 0, 0, false};
    const int p = __ldg(a.parent + r);
    if (p == -1) return k;
    k.bad = p < -1 || p >= a.bs_in;
    if (k.bad) return k;
    bool wrong;
    const int own = owned_pages(a, p, wrong), t = __ldg(a.keep + r);
    k.bad = wrong || t < 0 || (long long)t > (long long)own * a.page_size;
    if (k.bad) return k;
    k.row = a.block_table + (long long)p * a.max_pages;
    k.whole = t / a.page_size;
    k.tail = t % a.page_size;
    return k;
}
__device__ __forceinline__ bool in_pool(const ForkArgs &a, int id) {
    return id >= 0 && id < a.num_pages;
}

__device__ void step_clear(const ForkArgs &a) {
    const long long n = (long long)gridDim.x * blockDim.x;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < a.num_pages; i += n) {
        a.first[i] = kNone;
        a.heir[i] = kNone;
        a.refs[i] = 0;
    }
}

// A warp's part of a row: the row and its entries [lo, hi).
struct Part {
    int r, lo, hi;
    bool old, first;  // a row of the old table; the row's first part
};
__device__ __forceinline__ long long parts_of(const ForkArgs &a) {
    return (long long)a.bs_in * a.parts_in + (long long)a.bs_out * a.parts_out;
}
__device__ __forceinline__ Part part_at(const ForkArgs &a, long long x) {
    const long long in = (long long)a.bs_in * a.parts_in;
    Part p;
    p.old = x < in;
    const int y = (int)(p.old ? x : x - in), n = p.old ? a.parts_in : a.parts_out;
    const int len = p.old ? a.len_in : a.len_out;
    p.r = y / n;
    p.lo = (y - p.r * n) * len;
    p.hi = min(a.max_pages, p.lo + len);
    p.first = p.lo == 0;
    return p;
}

__device__ void step_mark(const ForkArgs &a) {
    const Share s = share();
    for (long long x = s.warp, n = parts_of(a); x < n; x += s.warps) {
        const Part p = part_at(a, x);
        if (p.old) {
            bool bad;
            const int hi = min(p.hi, owned_pages(a, p.r, bad));
            const long long at = (long long)p.r * a.max_pages;
            for (int j = p.lo + s.lane; j < hi; j += 32) {
                const int id = __ldg(a.block_table + at + j);
                if (in_pool(a, id)) atomicMin(a.first + id, (uint32_t)(at + j));
            }
        } else {
            const Kept k = kept_of(a, p.r);
            for (int j = p.lo + s.lane; j < min(p.hi, k.whole); j += 32) {
                const int id = __ldg(k.row + j);
                if (in_pool(a, id)) atomicAdd(a.refs + id, 1);
            }
            if (p.first && s.lane == 0 && k.tail > 0) {
                const int id = __ldg(k.row + k.whole);
                if (in_pool(a, id)) atomicMin(a.heir + id, (uint32_t)p.r);
            }
        }
    }
}

// The new row gets a fresh page for its last tokens (id: the old one).
__device__ __forceinline__ bool needs_copy(const ForkArgs &a, const Kept &k, int r, int &id) {
    id = k.tail > 0 ? __ldg(k.row + k.whole) : -1;
    return in_pool(a, id) && (__ldcg(a.refs + id) > 0 || __ldcg(a.heir + id) != (uint32_t)r);
}
// Entry `at` of the old table is the first of a page that nobody holds any more.
__device__ __forceinline__ bool is_gone(const ForkArgs &a, long long at) {
    const int id = __ldg(a.block_table + at);
    return in_pool(a, id) && __ldcg(a.first + id) == (uint32_t)at && __ldcg(a.refs + id) == 0 &&
           __ldcg(a.heir + id) == kNone;
}

__device__ void step_count(const ForkArgs &a) {
    const Share s = share();
    for (long long x = s.warp, n = parts_of(a); x < n; x += s.warps) {
        const Part p = part_at(a, x);
        if (p.old) {
            bool bad;
            const int hi = min(p.hi, owned_pages(a, p.r, bad));
            int c = 0;
            for (int j = p.lo + s.lane; j < hi; j += 32)
                c += is_gone(a, (long long)p.r * a.max_pages + j);
            c = __reduce_add_sync(0xffffffffu, c);
            if (s.lane == 0) a.gone[x] = c;
        } else if (p.first && s.lane == 0) {
            int id;
            a.copies[p.r] = needs_copy(a, kept_of(a, p.r), p.r, id);
            a.shared_out[p.r] = 0;
        }
    }
}

// Exclusive prefix sums of v[0, n) into the CTA's out[0, n], the total in out[n].
__device__ void scan_rows(const int32_t *v, int n, int *out) {
    __shared__ int s_w[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x / 32;
    for (int i = tid; i < n; i += blockDim.x) out[i] = __ldcg(v + i);
    // (an odd number of rows in a row a thread: no bank conflicts)
    const int per = ((n + (int)blockDim.x - 1) / (int)blockDim.x) | 1;
    const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
    __syncthreads();
    int sum = 0;
    for (int i = i0; i < i1; ++i) sum += out[i];
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
    }
    if (lane == 31) s_w[warp] = inc;
    __syncthreads();
    int before = inc - sum, all = 0;
    for (int w = 0; w < nw; ++w) {
        if (w < warp) before += s_w[w];
        all += s_w[w];
    }
    for (int i = i0; i < i1; ++i) {
        const int c = out[i];
        out[i] = before;
        before += c;
    }
    if (tid == 0) out[n] = all;
    __syncthreads();
}

__device__ void step_write(const ForkArgs &a) {
    extern __shared__ int s_rows[];
    int *s_copies = s_rows, *s_gone = s_rows + a.bs_out + 1;
    scan_rows(a.copies, a.bs_out, s_copies);
    scan_rows(a.gone, a.bs_in * a.parts_in, s_gone);
    const Share s = share();
    const uint32_t np = (uint32_t)a.num_pages;
    const int head_in = __ldg(a.free_state), count_in = __ldg(a.free_state + 1);
    const bool state_ok =
        head_in >= 0 && head_in < a.num_pages && count_in >= 0 && count_in <= a.num_pages;
    const uint32_t head = state_ok ? (uint32_t)head_in : 0u;
    const int count = state_ok ? count_in : 0;
    const int want = s_copies[a.bs_out], gone = s_gone[a.bs_in * a.parts_in];
    const int popped = min(want, count);
    // more pages in use and free than the pool has: nothing goes back
    const bool push = state_ok && (long long)count + gone <= a.num_pages;
    bool report = false;
    if (s.warp == 0 && s.lane == 0) {
        a.free_state_out[0] =
            state_ok ? (int)(((uint64_t)head + (uint64_t)popped) % np) : head_in;
        a.free_state_out[1] = state_ok ? count - popped + (push ? gone : 0) : count_in;
        report = !push || popped < want;
    }
    for (long long x = s.warp, all = parts_of(a); x < all; x += s.warps) {
        const Part p = part_at(a, x);
        const int r = p.r;
        if (p.old) {
            // ---- pages that go back, in the order of their entries
            bool bad;
            const int hi = min(p.hi, owned_pages(a, r, bad));
            report |= bad;
            int at = s_gone[x];
            for (int j0 = p.lo; j0 < hi; j0 += 32) {
                const int j = j0 + s.lane;
                const long long e = (long long)r * a.max_pages + j;
                const bool g = j < hi && is_gone(a, e);
                report |= j < hi && !in_pool(a, __ldg(a.block_table + e));
                const uint32_t m = __ballot_sync(0xffffffffu, g);
                if (g && push) {
                    const uint64_t k = (uint64_t)(at + __popc(m & ((1u << s.lane) - 1)));
                    a.free_pages[((uint64_t)head + (uint64_t)count + k) % np] =
                        __ldg(a.block_table + e);
                }
                at += __popc(m);
            }
            continue;
        }
        // ---- a new row
        const Kept k = kept_of(a, r);
        int old;
        const bool copy = needs_copy(a, k, r, old);
        int end = old, fresh = -1;  // its last page; a fresh one
        bool have = k.tail > 0;
        if (copy) {
            const int at = s_copies[r];
            have = at < popped;
            if (have) {
                uint64_t cell = (uint64_t)head + (uint64_t)at;
                if (cell >= np) cell -= np;
                fresh = __ldcg(a.free_pages + cell);
                if (!in_pool(a, fresh)) fresh = -1;
                report |= fresh < 0;
            }
            end = fresh;
        } else if (have && !in_pool(a, old)) {
            end = -1;
            report = true;
        }
        report |= k.bad;
        int shared = 0;
        int32_t *out = a.block_table_out + (long long)r * a.max_pages;
        for (int j = p.lo + s.lane; j < p.hi; j += 32) {
            int id = -1;
            if (j < k.whole) {
                id = __ldg(k.row + j);
                if (in_pool(a, id)) {
                    if (__ldcg(a.refs + id) > 1) shared = j + 1;
                } else {
                    id = -1;
                    report = true;
                }
            } else if (j == k.whole && have) {
                id = end;
            }
            out[j] = id;
        }
        shared = __reduce_max_sync(0xffffffffu, shared);
        if (s.lane == 0) {
            if (shared > 0) atomicMax(a.shared_out + r, shared);
            if (p.first) {
                a.owned_out[r] = k.whole + (have ? 1 : 0);
                a.copy_src[r] = fresh >= 0 ? old : -1;
                a.copy_dst[r] = fresh;
                a.copy_len[r] = fresh >= 0 ? k.tail : 0;
            }
        }
    }
    if (report) report_status(a.dev_status, BDSA_DEVICE_OUT_OF_RANGE);
}

// Everything before is done and seen by every CTA of the cluster.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One cluster does all steps: a launch instead of four.
__global__ void __launch_bounds__(kForkThreads) fork_cluster_kernel(const ForkArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    step_clear(a);
    cluster_sync();
    step_mark(a);
    cluster_sync();
    step_count(a);
    cluster_sync();
    step_write(a);
}

// The steps as grids, for tables that one cluster would be long about.
__global__ void __launch_bounds__(kForkThreads) fork_clear_kernel(const ForkArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    step_clear(a);
}
__global__ void __launch_bounds__(kForkThreads) fork_mark_kernel(const ForkArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    step_mark(a);
}
__global__ void __launch_bounds__(kForkThreads) fork_count_kernel(const ForkArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    step_count(a);
}
__global__ void __launch_bounds__(kForkThreads) fork_write_kernel(const ForkArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    step_write(a);
}

// The rows' parts: as many as kPart asks for, if a table has no more than kMaxParts then.
int parts_of_row(int bs, int max_pages) {
    const int by_len = (max_pages + kPart - 1) / kPart, most = kMaxParts / (bs > 0 ? bs : 1);
    return by_len < most ? by_len : most < 1 ? 1 : most;
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

size_t fork_workspace_bytes(int bs_in, int bs_out, int num_pages) {
    return 3 * up256(4 * (size_t)num_pages) + up256(4 * (size_t)kMaxParts) +
           up256(4 * (size_t)bs_out);
}

int launch_cache_fork(ForkArgs a, void *workspace, cudaStream_t stream) {
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const size_t pages = up256(4 * (size_t)a.num_pages);
    a.first = reinterpret_cast<uint32_t *>(ws);
    a.heir = reinterpret_cast<uint32_t *>(ws + pages);
    a.refs = reinterpret_cast<int32_t *>(ws + 2 * pages);
    a.gone = reinterpret_cast<int32_t *>(ws + 3 * pages);
    a.copies = reinterpret_cast<int32_t *>(ws + 3 * pages + up256(4 * (size_t)kMaxParts));
    a.parts_in = parts_of_row(a.bs_in, a.max_pages);
    a.parts_out = parts_of_row(a.bs_out, a.max_pages);
    a.len_in = (a.max_pages + a.parts_in - 1) / a.parts_in;
    a.len_out = (a.max_pages + a.parts_out - 1) / a.parts_out;
    const long long rows = (long long)a.bs_in + a.bs_out;
    const long long parts = (long long)a.bs_in * a.parts_in + (long long)a.bs_out * a.parts_out;
    const size_t smem = 4 * ((size_t)a.bs_in * a.parts_in + (size_t)a.bs_out + 2);
    if (parts <= kClusterParts && rows * a.max_pages + a.num_pages <= kClusterWork) {
        if (cudaFuncSetAttribute((const void *)fork_cluster_kernel,
                                 cudaFuncAttributeNonPortableClusterSizeAllowed,
                                 1) != cudaSuccess)
            return BDSA_CUDA_ERROR;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kForkCtas);
        cfg.blockDim = dim3(kForkThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kForkCtas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, fork_cluster_kernel, (const ForkArgs)a) == cudaSuccess
                   ? BDSA_OK
                   : BDSA_CUDA_ERROR;
    }
    // past the default 48 KB, on this device; the same limit in every call, so that
    // host threads do not undo one another's
    constexpr int kMost = 4 * (2 * BDSA_TABLE_MAX_REQUESTS + 2);
    if (smem > 44 * 1024 &&
        cudaFuncSetAttribute((const void *)fork_write_kernel,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kMost) != cudaSuccess)
        return BDSA_CUDA_ERROR;
    const unsigned warps = kForkThreads / 32;
    const unsigned by_part = (unsigned)(parts > 0 ? (parts + warps - 1) / warps : 1);
    const unsigned by_page =
        (unsigned)(((long long)a.num_pages + kForkThreads - 1) / kForkThreads);
    // (every CTA of the last step sums all counts: not many more than fill the GPU)
    const unsigned few = by_part < 608 ? by_part : 608;
    auto step = [&](void (*k)(const ForkArgs), unsigned grid, size_t bytes) {
        return launch_pdl(k, dim3(grid), dim3(kForkThreads), bytes, stream, a) == cudaSuccess;
    };
    const bool ok = step(fork_clear_kernel, by_page < 1024 ? by_page : 1024, 0) &&
                    step(fork_mark_kernel, by_part, 0) && step(fork_count_kernel, by_part, 0) &&
                    step(fork_write_kernel, few, smem);
    return ok ? BDSA_OK : BDSA_CUDA_ERROR;
}

}  // namespace bdsa
