// cache_api.cu -- the extern "C" boundary of the prompt and cache calls (declared
// in include/bdsa.h): host-side argument checks, workspace sizing and dispatch to
// the kernel launchers.  No call allocates device memory.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>

#include "../../include/bdsa.h"
#include "bdsa_internal.h"
#include "cache_internal.h"
#include "host_checks.h"

namespace {

constexpr int64_t kMaxRowBytes = 1 << 20;

// The checks of a list of caches of num_pages pages each; `ins` are lists that the
// call reads while it writes the caches.
int32_t check_caches(void *const *caches, int32_t n, int64_t row_bytes, int32_t page_size,
                     int32_t num_pages, std::initializer_list<Range> ins) {
    if (n < 0 || row_bytes < 1 || page_size < 1 || num_pages < 1) return BDSA_INVALID_ARG;
    if (n > BDSA_MAX_CACHES || row_bytes > kMaxRowBytes ||
        (int64_t)num_pages * page_size > INT32_MAX)
        return BDSA_UNSUPPORTED;
    if (n == 0) return BDSA_OK;
    if (!caches) return BDSA_INVALID_ARG;
    if (row_bytes % 16 != 0) return BDSA_MISALIGNED;
    const int64_t bytes = row_bytes * page_size * num_pages;
    uintptr_t at[BDSA_MAX_CACHES];
    for (int i = 0; i < n; ++i) {
        if (!caches[i]) return BDSA_INVALID_ARG;
        if (!aligned(caches[i], 16)) return BDSA_MISALIGNED;
        for (const Range &r : ins)
            if (meet({caches[i], bytes}, r)) return BDSA_INVALID_ARG;
        at[i] = reinterpret_cast<uintptr_t>(caches[i]);
    }
    std::sort(at, at + n);
    for (int i = 1; i < n; ++i)
        if (at[i] - at[i - 1] < (uintptr_t)bytes) return BDSA_INVALID_ARG;
    return BDSA_OK;
}

}  // namespace

extern "C" {

size_t bdsa_chunk_attn_workspace_bytes(int32_t D, int32_t num_sms) {
    if (D != 64 && D != 128) return 0;
    return bdsa::chunk_plan(D, bdsa::chunk_ctas(bdsa::device_num_sms(num_sms))).workspace;
}

int32_t bdsa_chunk_attn_paged(const bdsa_bf16 *q, int64_t q_stride, const bdsa_bf16 *k_cache,
                              const bdsa_bf16 *v_cache, const int32_t *block_table,
                              int32_t max_pages_per_req, int32_t num_pages,
                              const int32_t *seq_lens, const int32_t *cu_tokens, int32_t bs,
                              int32_t T, int32_t Hq, int32_t Hkv, int32_t D, int32_t page_size,
                              float softmax_scale, int32_t mask_block, bdsa_bf16 *out, float *lse,
                              void *workspace, size_t workspace_bytes, int32_t num_sms,
                              int32_t *dev_status, void *stream) {
    if (bs < 0 || T < 0 || Hq < 1 || Hkv < 1 || max_pages_per_req < 1 || num_pages < 1 ||
        !isfinite(softmax_scale) || !(softmax_scale > 0.f) || mask_block < 1 || Hq % Hkv != 0)
        return BDSA_INVALID_ARG;
    if (D != 64 && D != 128) return BDSA_UNSUPPORTED;
    if (Hq / Hkv > 128 || page_size < 8 || (page_size & (page_size - 1)) != 0 ||
        mask_block > (1 << 30) || (int64_t)num_pages * page_size > INT32_MAX ||
        T > INT32_MAX - 256)
        return BDSA_UNSUPPORTED;
    if (bs == 0 || T == 0) return BDSA_OK;
    if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !cu_tokens || !out)
        return BDSA_INVALID_ARG;
    const int64_t token = (int64_t)Hq * D;
    if (q_stride < token) return BDSA_INVALID_ARG;
    if (q_stride % 8 != 0 || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 256))
        return BDSA_MISALIGNED;
    if (q_stride >= (1LL << 30)) return BDSA_UNSUPPORTED;
    const int ctas = bdsa::chunk_ctas(bdsa::device_num_sms(num_sms));
    const size_t need = bdsa::chunk_plan(D, ctas).workspace;
    if (!workspace || workspace_bytes < need) return BDSA_WORKSPACE_TOO_SMALL;
    const int64_t cache = 2LL * num_pages * page_size * Hkv * D;
    if (!apart({{out, 2LL * T * token}, {lse, 4LL * T * Hq}, {workspace, (int64_t)need}},
               {{q, 2 * ((T - 1) * q_stride + token)},
                {k_cache, cache},
                {v_cache, cache},
                {block_table, 4LL * bs * max_pages_per_req},
                {seq_lens, 4LL * bs},
                {cu_tokens, 4LL * bs + 4}}))
        return BDSA_INVALID_ARG;
    bdsa::ChunkArgs a;
    a.q = reinterpret_cast<const uint16_t *>(q);
    a.q_stride = q_stride;
    a.k_cache = reinterpret_cast<const uint16_t *>(k_cache);
    a.v_cache = reinterpret_cast<const uint16_t *>(v_cache);
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.cu_tokens = cu_tokens;
    a.T = T;
    a.max_pages = max_pages_per_req;
    a.num_pages = num_pages;
    a.bs = bs;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = D;
    a.page_size = page_size;
    a.mask_block = mask_block;
    a.scale = softmax_scale;
    a.out = reinterpret_cast<uint16_t *>(out);
    a.lse = lse;
    a.workspace = workspace;
    a.ctas = ctas;
    a.dev_status = dev_status;
    return bdsa::launch_chunk_attn(a, static_cast<cudaStream_t>(stream));
}

int32_t bdsa_cache_write(const void *k_new, int64_t k_stride, const void *v_new,
                         int64_t v_stride, const int32_t *slot_map, int32_t T, void *k_cache,
                         void *v_cache, int32_t row_bytes, int64_t num_slots,
                         int32_t *dev_status, void *stream) {
    if (T < 0 || row_bytes < 1 || num_slots < 1 || k_stride < row_bytes || v_stride < row_bytes)
        return BDSA_INVALID_ARG;
    if (row_bytes > kMaxRowBytes || num_slots > INT32_MAX || k_stride > INT32_MAX ||
        v_stride > INT32_MAX)
        return BDSA_UNSUPPORTED;
    if (T == 0) return BDSA_OK;
    if (!k_new || !v_new || !slot_map || !k_cache || !v_cache) return BDSA_INVALID_ARG;
    if (row_bytes % 16 != 0 || k_stride % 16 != 0 || v_stride % 16 != 0 || !aligned(k_new, 16) ||
        !aligned(v_new, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
        return BDSA_MISALIGNED;
    const int64_t cache = num_slots * row_bytes;
    if (!apart({{k_cache, cache}, {v_cache, cache}},
               {{k_new, (T - 1) * k_stride + row_bytes},
                {v_new, (T - 1) * v_stride + row_bytes},
                {slot_map, 4LL * T}}))
        return BDSA_INVALID_ARG;
    bdsa::WriteArgs a;
    a.src[0] = static_cast<const uint8_t *>(k_new);
    a.src[1] = static_cast<const uint8_t *>(v_new);
    a.stride[0] = k_stride;
    a.stride[1] = v_stride;
    a.cache[0] = static_cast<uint8_t *>(k_cache);
    a.cache[1] = static_cast<uint8_t *>(v_cache);
    a.slot_map = slot_map;
    a.num_slots = num_slots;
    a.T = T;
    a.row_bytes = row_bytes;
    a.dev_status = dev_status;
    return bdsa::launch_cache_write(a, bdsa::device_num_sms(0),
                                    static_cast<cudaStream_t>(stream));
}

size_t bdsa_cache_fork_workspace_bytes(int32_t bs_in, int32_t bs_out, int32_t num_pages) {
    if (bs_in < 0 || bs_out < 0 || num_pages < 1) return 0;
    return bdsa::fork_workspace_bytes(bs_in, bs_out, num_pages);
}

int32_t bdsa_cache_fork(const int32_t *parent, const int32_t *keep_lens,
                        const int32_t *block_table, const int32_t *owned,
                        int32_t max_pages_per_req, int32_t num_pages, int32_t bs_in,
                        int32_t bs_out, int32_t page_size, int32_t *free_pages,
                        const int32_t *free_state, int32_t *block_table_out, int32_t *owned_out,
                        int32_t *shared_out, int32_t *free_state_out, int32_t *copy_src,
                        int32_t *copy_dst, int32_t *copy_len, void *workspace,
                        size_t workspace_bytes, int32_t *dev_status, void *stream) {
    if (bs_in < 0 || bs_out < 0 || page_size < 1 || max_pages_per_req < 1 || num_pages < 1)
        return BDSA_INVALID_ARG;
    if (bs_in > BDSA_TABLE_MAX_REQUESTS || bs_out > BDSA_TABLE_MAX_REQUESTS ||
        (int64_t)bs_in * max_pages_per_req > INT32_MAX ||
        (int64_t)num_pages * page_size > INT32_MAX)
        return BDSA_UNSUPPORTED;
    if (!free_pages || !free_state || !free_state_out) return BDSA_INVALID_ARG;
    if (bs_in > 0 && (!block_table || !owned)) return BDSA_INVALID_ARG;
    if (bs_out > 0 && (!parent || !keep_lens || !block_table_out || !owned_out || !shared_out ||
                       !copy_src || !copy_dst || !copy_len))
        return BDSA_INVALID_ARG;
    if (!aligned(workspace, 256)) return BDSA_MISALIGNED;
    const size_t need = bdsa::fork_workspace_bytes(bs_in, bs_out, num_pages);
    if (!workspace || workspace_bytes < need) return BDSA_WORKSPACE_TOO_SMALL;
    const int64_t in = 4LL * bs_in, out = 4LL * bs_out;
    if (!apart({{free_pages, 4LL * num_pages},
                {block_table_out, out * max_pages_per_req},
                {owned_out, out},
                {shared_out, out},
                {free_state_out, 8},
                {copy_src, out},
                {copy_dst, out},
                {copy_len, out},
                {workspace, (int64_t)need}},
               {{parent, out},
                {keep_lens, out},
                {block_table, in * max_pages_per_req},
                {owned, in},
                {free_state, 8}}))
        return BDSA_INVALID_ARG;
    bdsa::ForkArgs a = {};
    a.parent = parent;
    a.keep = keep_lens;
    a.block_table = block_table;
    a.owned = owned;
    a.free_pages = free_pages;
    a.free_state = free_state;
    a.block_table_out = block_table_out;
    a.owned_out = owned_out;
    a.shared_out = shared_out;
    a.free_state_out = free_state_out;
    a.copy_src = copy_src;
    a.copy_dst = copy_dst;
    a.copy_len = copy_len;
    a.max_pages = max_pages_per_req;
    a.num_pages = num_pages;
    a.bs_in = bs_in;
    a.bs_out = bs_out;
    a.page_size = page_size;
    a.dev_status = dev_status;
    return bdsa::launch_cache_fork(a, workspace, static_cast<cudaStream_t>(stream));
}

int32_t bdsa_cache_copy(void *const *caches, int32_t n_caches, int64_t row_bytes,
                        int32_t page_size, int32_t num_pages, const int32_t *copy_src,
                        const int32_t *copy_dst, const int32_t *copy_len, int32_t n,
                        int32_t *dev_status, void *stream) {
    if (n < 0) return BDSA_INVALID_ARG;
    if (n > 0 && (!copy_src || !copy_dst || !copy_len)) return BDSA_INVALID_ARG;
    const int64_t list = 4LL * n;
    const int32_t st = check_caches(caches, n_caches, row_bytes, page_size, num_pages,
                                    {{copy_src, list}, {copy_dst, list}, {copy_len, list}});
    if (st != BDSA_OK || n == 0 || n_caches == 0) return st;
    bdsa::CopyArgs a;
    a.src = copy_src;
    a.dst = copy_dst;
    a.len = copy_len;
    a.row_bytes = row_bytes;
    a.n = n;
    a.page_size = page_size;
    a.num_pages = num_pages;
    a.dev_status = dev_status;
    return bdsa::launch_cache_copy(a, caches, n_caches, static_cast<cudaStream_t>(stream));
}

int32_t bdsa_cache_compact(void *const *caches, int32_t n_caches, int64_t row_bytes,
                           int32_t page_size, int32_t num_pages, const int32_t *block_table,
                           int32_t max_pages_per_req, const int32_t *seq_lens,
                           const int32_t *path, int32_t width, int32_t bs, int32_t *dev_status,
                           void *stream) {
    if (bs < 0 || width < 0 || max_pages_per_req < 1) return BDSA_INVALID_ARG;
    if (bs > 0 && (!block_table || !seq_lens || (width > 0 && !path))) return BDSA_INVALID_ARG;
    const int32_t st = check_caches(caches, n_caches, row_bytes, page_size, num_pages,
                                    {{block_table, 4LL * bs * max_pages_per_req},
                                     {seq_lens, 4LL * bs},
                                     {path, 4LL * bs * width}});
    if (st != BDSA_OK || bs == 0 || width == 0 || n_caches == 0) return st;
    bdsa::CompactArgs a;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.path = path;
    a.row_bytes = row_bytes;
    a.bs = bs;
    a.width = width;
    a.max_pages = max_pages_per_req;
    a.page_size = page_size;
    a.num_pages = num_pages;
    a.dev_status = dev_status;
    return bdsa::launch_cache_compact(a, caches, n_caches, bdsa::device_num_sms(0),
                                      static_cast<cudaStream_t>(stream));
}

}  // extern "C"
