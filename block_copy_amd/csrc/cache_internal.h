// cache_internal.h -- what the host checks of the cache operators
// (cache.cpp) hand to their kernels (cache_kernels.hip, attention.hip).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "kvcache.h"
#include "paging.h"

namespace kvc {

struct RopeArgs {
    const int32_t *positions;
    const double *freq;
    const void *q, *k;
    void *q_out, *k_out;
    int64_t q_st, q_sh, k_st, k_sh;       // token and head strides, in elements
    int64_t qo_st, qo_sh, ko_st, ko_sh;
    uint32_t tokens, q_heads, heads;      // heads = q_heads + k_heads
    uint32_t head_dim, rot_dim;
    uint32_t interleaved;
    uint32_t block_tokens;                // tokens of one workgroup
    float factor, sign;
};

struct RowArgs {   // kvcache_write and kvcache_read
    void *pages[2];            // keys, values
    float *scale[2];
    int64_t p_page[2], p_head[2], p_place[2];
    int64_t s_page[2], s_head[2], s_place[2];
    void *rows[2];
    int64_t r_token[2], r_head[2];
    const int64_t *slots;
    uint32_t *status;
    uint32_t num_slots;
    uint32_t tokens, head_dim;
    Divider page_size, kv_heads;
};

struct AttentionArgs {
    const void *q;
    void *out;
    float *lse;
    int64_t q_st, q_sh, o_st, o_sh, l_st, l_sh;
    const void *k, *v;
    const float *k_scale, *v_scale;
    int64_t k_head, v_head, ks_head, vs_head;               // in elements
    uint32_t k_page, k_place, v_page, v_place;              // in pieces of 8 elements
    uint32_t ks_page, ks_place, vs_page, vs_place;          // in elements
    const int32_t *table;
    int64_t table_stride;
    const int32_t *q_starts, *context_lens;
    uint32_t *status;
    float *part_o, *part_ml;   // [split][token][head][head_dim], [split][token][head][2]
    uint32_t num_pages, total_q, max_q_len, max_context;
    uint32_t q_heads, kv_heads, head_dim;
    uint32_t full;             // head_dim is 64, 128 or 256, and 8-bit rows can be read 16 codes at once
    uint32_t tiles, splits, split_keys;
    int32_t window;
    float scale_log2;          // |scale| * log2(e), or 1 where scale is 0
    uint32_t q_keep, q_flip;   // masks of q's words: scale's zero and sign
    Divider page_size, group;
};

// How one call is laid out over the grid; depends on host values alone.
struct AttentionShape {
    uint32_t single;           // the kernel for at most 16 rows a (sequence, key/value head)
    uint32_t tiles, splits, split_keys;
    uint64_t workspace_bytes;
};

// One kernel whose only argument is `a`.  (The launch's own result, not the
// thread's last error, which may be an earlier call's.)
template <class A>
hipError_t launch(void (*kernel)(const A), uint32_t grid_x, uint32_t grid_y, uint32_t threads, const A &a,
                  hipStream_t stream)
{
    void *args[] = {const_cast<A *>(&a)};
    return hipLaunchKernel(reinterpret_cast<const void *>(kernel), dim3(grid_x, grid_y), dim3(threads), args, 0,
                           stream);
}

hipError_t launch_rope(const RopeArgs &a, uint32_t dtype, bool wide, hipStream_t stream);
hipError_t launch_write(const RowArgs &a, uint32_t dtype, uint32_t format, bool wide, hipStream_t stream);
hipError_t launch_read(const RowArgs &a, uint32_t dtype, uint32_t format, bool wide, hipStream_t stream);
AttentionShape attention_shape(uint32_t num_seqs, uint32_t total_q, uint32_t q_heads, uint32_t kv_heads,
                               uint32_t head_dim, uint32_t max_q_len, uint32_t max_context,
                               uint32_t window);
hipError_t launch_attention(const AttentionArgs &a, const AttentionShape &shape, uint32_t num_seqs,
                            uint32_t dtype, uint32_t format, hipStream_t stream);

}  // namespace kvc
