// block_table.cu -- block tables and slot maps from request lengths, one launch.
//
// Request r holds owned_r pages and is to hold L_r + n_r tokens:
//   need_r = ceil((L_r + n_r) / ps)
//   grow_r = max(0, need_r - owned_r)                    pages popped
//   rel_r  = max(0, owned_r - max(need_r, shared_r))     pages pushed
// Free pages are a FIFO ring: pops come from the head in request order, pushes
// go behind the tail.  The pages a call pops and the cells it pushes into are
// disjoint (owned and free pages together are at most num_pages), so no thread
// reads what another writes and the whole update needs no grid-wide step.
//
// What bounds it: latency.  The bytes (a few ints a request and a page, 8 bytes
// a new token) are small, so the work is split so that nothing waits: every CTA
// scans all requests itself (the three prefix sums live in its shared memory)
// and then takes its share of the requests, the popped pages, the pushed pages
// and the tokens, each item finding its request by a binary search of the
// scanned offsets.  Measured (launches in a graph): 32 requests of 16 tokens 4.9 us,
// 4093 decode requests 8.7 us, 1024 prompts of 2.1 million tokens 18.6 us (17.9 MB).
#include <cuda_runtime.h>
#include <limits.h>

#include "bdsa_device.cuh"
#include "bdsa_internal.h"

namespace bdsa {
namespace {

constexpr int kTabThreads = 512;
constexpr int kTabWarps = kTabThreads / 32;

struct ReqPlan {
    int n, own, grow, rel;
    bool wrong;  // lengths or owned pages that mean nothing: its tokens have no slot
    bool bad;    // the row stays as it is
};

__device__ __forceinline__ ReqPlan plan_request(const TableArgs &a, int r) {
    ReqPlan q;
    const int L = a.seq_lens[r], n = a.new_lens[r], own = a.owned[r];
    const int sh = a.shared ? a.shared[r] : 0;
    q.n = max(n, 0);
    q.own = own;
    q.grow = q.rel = 0;
    const uint32_t tok = (uint32_t)L + (uint32_t)n, ps = (uint32_t)a.page_size;
    q.wrong = L < 0 || n < 0 || tok > (uint32_t)INT32_MAX || own < 0 || own > a.max_pages;
    q.bad = q.wrong || sh < 0;
    if (q.bad) return q;
    const uint32_t need = tok / ps + (tok % ps != 0);
    if (need > (uint32_t)a.max_pages) {
        q.bad = true;
        return q;
    }
    if ((int)need > own) q.grow = (int)need - own;
    else q.rel = max(0, own - max((int)need, min(sh, own)));
    return q;
}

// Last r in [0, bs) with off[r] <= x (off[0] = 0, off nondecreasing): the
// request that item x belongs to, when off[bs] > x.
__device__ __forceinline__ int find_request(const int *off, int bs, int x) {
    int lo = 0, hi = bs;  // off[lo] <= x < off[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Slots and positions of the new tokens, kGroup in a row a thread: four (one
// 16-byte store an array, and tokens of a request share its lookups) when every
// thread has some, one when they are few, so that no thread walks through four
// requests (4093 decode tokens 8.7 us, with four 11.5 us; 1024 prompts of 2.1
// million tokens 18.6 us, with one 35.6 us).  True when something is out of range.
struct TokenRange {
    uint32_t head;
    int popped;
    long gid, stride;
    long long T;  // tokens that have room
};
template <int kGroup>
__device__ __forceinline__ bool map_tokens(const TableArgs &a, const TokenRange &tr,
                                           const int *s_tok, const int *s_pop) {
    const int bs = a.bs;
    const uint32_t np = (uint32_t)a.num_pages;
    bool report = false;
    const uint32_t ps = (uint32_t)a.page_size;
    for (long t0 = tr.gid * kGroup; t0 < tr.T; t0 += tr.stride * kGroup) {
        int slot[kGroup], pos[kGroup];
        int r = find_request(s_tok, bs, (int)t0) - 1;
        int r_end = (int)t0;  // the first token of request r + 1
        int own = 0, base = 0, first = 0, in_page = 0, id = -1;
        uint32_t page = 0;
        bool bad = false, granted = false, fresh = true;
#pragma unroll
        for (int k = 0; k < kGroup; ++k) {
            slot[k] = pos[k] = -1;
            const long t = t0 + k;
            if (t >= tr.T) continue;
            if (t >= r_end) {  // the next request with a token here
                do {
                    ++r;
                    r_end = s_tok[r + 1];
                } while (t >= r_end && r + 1 < bs);
                const ReqPlan q = plan_request(a, r);
                bad = q.wrong;
                own = q.own;
                first = a.seq_lens[r];
                base = s_pop[r];
                granted = !q.bad && (long long)base + q.grow <= tr.popped;
                const uint32_t p = (uint32_t)first + (uint32_t)(t - s_tok[r]);
                page = p / ps;
                in_page = (int)(p % ps);
                fresh = true;
            } else if (++in_page == (int)ps) {
                in_page = 0;
                ++page;
                fresh = true;
            }
            if (fresh && !bad) {
                if (page < (uint32_t)own) {
                    id = a.block_table[(long)r * a.max_pages + page];
                } else if (granted) {
                    uint32_t cell = tr.head + (uint32_t)base + (page - (uint32_t)own);
                    if (cell >= np) cell -= np;
                    id = a.free_pages[cell];
                } else {
                    id = -1;
                }
                if (id < 0 || id >= a.num_pages) {
                    id = -1;
                    report = true;
                }
                fresh = false;
            }
            if (bad) continue;
            pos[k] = (int)((uint32_t)first + (uint32_t)(t - s_tok[r]));
            if (id >= 0) slot[k] = id * (int)ps + in_page;
        }
        if (kGroup == 4 && a.vec && t0 + kGroup <= tr.T) {
            if (a.slot_map)
                *reinterpret_cast<int4 *>(a.slot_map + t0) =
                    make_int4(slot[0], slot[1 % kGroup], slot[2 % kGroup], slot[3 % kGroup]);
            if (a.positions)
                *reinterpret_cast<int4 *>(a.positions + t0) =
                    make_int4(pos[0], pos[1 % kGroup], pos[2 % kGroup], pos[3 % kGroup]);
        } else {
#pragma unroll
            for (int k = 0; k < kGroup; ++k) {
                if (t0 + k >= tr.T) continue;
                if (a.slot_map) a.slot_map[t0 + k] = slot[k];
                if (a.positions) a.positions[t0 + k] = pos[k];
            }
        }
    }
    return report;
}

__global__ void __launch_bounds__(kTabThreads) block_table_kernel(const TableArgs a) {
    grid_launch_dependents();
    extern __shared__ int s_off[];  // tok, pop, rel: [bs + 1] each
    __shared__ long long s_w[3][kTabWarps];
    __shared__ int s_popped;
    const int bs = a.bs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int *s_tok = s_off, *s_pop = s_off + bs + 1, *s_rel = s_off + 2 * (bs + 1);
    const uint32_t np = (uint32_t)a.num_pages;
    const int head_in = a.free_state[0], count_in = a.free_state[1];
    const bool state_ok =
        head_in >= 0 && head_in < a.num_pages && count_in >= 0 && count_in <= a.num_pages;
    const uint32_t head = state_ok ? (uint32_t)head_in : 0u;
    const int count = state_ok ? count_in : 0;

    // ---- exclusive prefix sums of (tokens, pops, pushes) over the requests
    // (a thread's requests are an odd number in a row: no bank conflicts)
    for (int r = tid; r < bs; r += kTabThreads) {
        const ReqPlan q = plan_request(a, r);
        s_tok[r] = q.n;
        s_pop[r] = q.grow;
        s_rel[r] = q.rel;
    }
    const int per = ((bs + kTabThreads - 1) / kTabThreads) | 1;
    const int i0 = min(bs, tid * per), i1 = min(bs, i0 + per);
    __syncthreads();
    long long v[3] = {0, 0, 0};
    for (int r = i0; r < i1; ++r) {
        v[0] += s_tok[r];
        v[1] += s_pop[r];
        v[2] += s_rel[r];
    }
    long long inc[3] = {v[0], v[1], v[2]};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const long long t = __shfl_up_sync(0xffffffffu, inc[k], o);
            if (lane >= o) inc[k] += t;
        }
    }
    if (lane == 31) {
#pragma unroll
        for (int k = 0; k < 3; ++k) s_w[k][warp] = inc[k];
    }
    if (tid == 0) s_popped = 0;
    __syncthreads();
    long long tot[3] = {0, 0, 0};
#pragma unroll
    for (int w = 0; w < kTabWarps; ++w) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const long long t = s_w[k][w];
            if (w < warp) inc[k] += t;
            tot[k] += t;
        }
    }
    // offsets saturate at INT32_MAX (page counts and token counts that reach it
    // are past every limit checked below)
    long long at[3] = {inc[0] - v[0], inc[1] - v[1], inc[2] - v[2]};
    auto sat = [](long long x) { return (int)min(x, (long long)INT32_MAX); };
    int my_popped = 0;
    for (int r = i0; r < i1; ++r) {
        const int n = s_tok[r], grow = s_pop[r], rel = s_rel[r];
        s_tok[r] = sat(at[0]);
        s_pop[r] = sat(at[1]);
        s_rel[r] = sat(at[2]);
        at[0] += n;
        at[1] += grow;
        at[2] += rel;
        // pages are granted in request order up to the first request that
        // does not fit: the popped total is the largest prefix sum that fits
        if (at[1] <= count) my_popped = (int)at[1];
    }
    if (my_popped > 0) atomicMax(&s_popped, my_popped);
    if (tid == 0) {
        s_tok[bs] = sat(tot[0]);
        s_pop[bs] = sat(tot[1]);
        s_rel[bs] = sat(tot[2]);
    }
    __syncthreads();
    const int popped = s_popped;
    // more pages owned and free than the pool has: nothing is released
    const bool rel_ok = state_ok && (long long)count + tot[2] <= (long long)a.num_pages;
    const int pushed = rel_ok ? (int)tot[2] : 0;
    const long stride = (long)gridDim.x * kTabThreads;
    const long gid = (long)blockIdx.x * kTabThreads + tid;

    // ---- per request: the new owned count and the token offsets
    bool report = false;
    for (long r = gid; r <= bs; r += stride) {
        if (r == bs) {
            a.cu_tokens[bs] = s_tok[bs];
            a.free_state_out[0] =
                state_ok ? (int)(((uint64_t)head + (uint64_t)popped) % np) : head_in;
            a.free_state_out[1] = state_ok ? count - popped + pushed : count_in;
            report |= !rel_ok || tot[0] > INT32_MAX || (a.slot_map && tot[0] > a.max_tokens) ||
                      (a.positions && tot[0] > a.max_tokens);
            break;
        }
        const ReqPlan q = plan_request(a, (int)r);
        const bool granted = q.grow == 0 || s_pop[r] + (long long)q.grow <= popped;
        report |= q.bad || !granted;
        a.owned_out[r] = q.own + (granted ? q.grow : 0) - (rel_ok ? q.rel : 0);
        a.cu_tokens[r] = s_tok[r];
    }

    // ---- popped pages into the table
    for (long x = gid; x < popped; x += stride) {
        const int r = find_request(s_pop, bs, (int)x);
        uint32_t cell = head + (uint32_t)x;
        if (cell >= np) cell -= np;
        int id = a.free_pages[cell];
        if (id < 0 || id >= a.num_pages) {
            id = -1;
            report = true;
        }
        a.block_table[(long)r * a.max_pages + a.owned[r] + ((int)x - s_pop[r])] = id;
    }

    // ---- released pages onto the ring
    for (long x = gid; x < pushed; x += stride) {
        const int r = find_request(s_rel, bs, (int)x);
        const int rel_r = s_rel[r + 1] - s_rel[r];
        int *entry =
            a.block_table + (long)r * a.max_pages + (a.owned[r] - rel_r) + ((int)x - s_rel[r]);
        const int id = *entry;
        *entry = -1;
        report |= id < 0 || id >= a.num_pages;
        a.free_pages[((uint64_t)head + (uint64_t)count + (uint64_t)x) % np] = id;
    }

    // ---- slots and positions of the new tokens
    const TokenRange tr{head, popped, gid, stride,
                        min(tot[0], (long long)min(a.max_tokens, (int64_t)INT32_MAX))};
    report |= tr.T > stride ? map_tokens<4>(a, tr, s_tok, s_pop)
                            : map_tokens<1>(a, tr, s_tok, s_pop);
    if (report) report_status(a.dev_status, BDSA_DEVICE_OUT_OF_RANGE);
}

}  // namespace

int launch_block_table(const TableArgs &a, int num_sms, cudaStream_t stream) {
    const size_t smem = (size_t)3 * (a.bs + 1) * sizeof(int);
    // past the default 48 KB of shared memory (static and dynamic together), on
    // this device; the same limit in every call, so that host threads do not undo
    // one another's
    constexpr int kMost = 3 * (BDSA_TABLE_MAX_REQUESTS + 1) * (int)sizeof(int);
    if (smem > 44 * 1024 &&
        cudaFuncSetAttribute(block_table_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMost) != cudaSuccess)
        return BDSA_CUDA_ERROR;
    // Every CTA repeats the scan, so no more of them than the items fill: one
    // a 4096 tokens (two rounds of a CTA's threads) or 512 requests (a CTA for every
    // SM is 0.2 us faster on 32 and 4093 decode requests, and takes the whole GPU).
    const long by_tok = (a.max_tokens + 4095) / 4096, by_req = ((long)a.bs + 511) / 512;
    long grid = by_tok > by_req ? by_tok : by_req;
    if (grid > num_sms) grid = num_sms;
    if (grid < 1) grid = 1;
    block_table_kernel<<<(unsigned)grid, kTabThreads, smem, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? BDSA_OK : BDSA_CUDA_ERROR;
}

}  // namespace bdsa
