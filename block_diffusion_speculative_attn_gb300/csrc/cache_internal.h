// cache_internal.h -- host-side launch interfaces of the prompt and cache calls
// (attention of chunks over the paged cache, cache writes, forks and moves),
// shared between the C ABI and the kernel translation units.  Not installed.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace bdsa {

// ---------------------------------------------------------------- chunk attention
struct ChunkArgs {
    const uint16_t *q;                 // token t at q + t * q_stride
    const uint16_t *k_cache, *v_cache;
    const int32_t *block_table, *seq_lens, *cu_tokens;
    int64_t q_stride;
    int T, max_pages, num_pages, bs, Hq, Hkv, D, page_size, mask_block;
    float scale;
    uint16_t *out;                     // [T, Hq, D]
    float *lse;                        // [T, Hq], or null
    void *workspace;
    int ctas;                          // persistent CTAs
    int32_t *dev_status;
};

// Two partials of 256 query rows a CTA, and a note on the unit that it cut.
struct ChunkPlan {
    size_t off_lse, off_o, workspace;
};
ChunkPlan chunk_plan(int D, int ctas);
int chunk_ctas(int num_sms);  // CTAs of a call for this many SMs
int launch_chunk_attn(const ChunkArgs &a, cudaStream_t stream);

// ---------------------------------------------------------------- cache rows
struct WriteArgs {
    const uint8_t *src[2];       // K and V of token t at src[i] + t * stride[i]
    int64_t stride[2];           // bytes
    uint8_t *cache[2];           // [num_slots, row_bytes]
    const int32_t *slot_map;     // [T]
    int64_t num_slots;
    int T, row_bytes;
    int32_t *dev_status;
};
int launch_cache_write(const WriteArgs &a, int num_sms, cudaStream_t stream);

// The caches of one launch, by value in its parameters.
constexpr int kCachesPerLaunch = 256;
struct CacheList {
    uint8_t *p[kCachesPerLaunch];
};

struct CopyArgs {
    const int32_t *src, *dst, *len;  // [n]: pages, rows
    int64_t row_bytes;
    int n, page_size, num_pages;
    int32_t *dev_status;
};
int launch_cache_copy(const CopyArgs &a, void *const *caches, int n_caches, cudaStream_t stream);

struct CompactArgs {
    const int32_t *block_table, *seq_lens;  // [bs, max_pages], [bs]
    const int32_t *path;                    // [bs, width]
    int64_t row_bytes;
    int bs, width, max_pages, page_size, num_pages;
    int32_t *dev_status;
};
int launch_cache_compact(const CompactArgs &a, void *const *caches, int n_caches, int num_sms,
                         cudaStream_t stream);

// ---------------------------------------------------------------- fork
struct ForkArgs {
    const int32_t *parent, *keep;            // [bs_out]
    const int32_t *block_table, *owned;      // [bs_in, max_pages], [bs_in]
    int32_t *free_pages;                     // ring of num_pages cells
    const int32_t *free_state;               // {head, count}
    int32_t *block_table_out;                // [bs_out, max_pages]
    int32_t *owned_out, *shared_out, *free_state_out;
    int32_t *copy_src, *copy_dst, *copy_len; // [bs_out]
    int max_pages, num_pages, bs_in, bs_out, page_size;
    int parts_in, len_in, parts_out, len_out;  // parts of a row, entries of a part
    // workspace
    uint32_t *first, *heir;  // [num_pages]: first old entry, first row that it ends
    int32_t *refs;           // [num_pages]: new rows that hold it whole
    int32_t *copies, *gone;  // [bs_out], [bs_in * parts_in]: pages popped, pushed
    int32_t *dev_status;
};
size_t fork_workspace_bytes(int bs_in, int bs_out, int num_pages);
int launch_cache_fork(ForkArgs a, void *workspace, cudaStream_t stream);

}  // namespace bdsa
