/*
 * kvcache.h -- C ABI of the operators around a paged key/value cache on AMD
 * Instinct MI355X (gfx950): rotary positions, writing new tokens into pages
 * (as they are or quantised to 8 bits), reading tokens back, and attention of
 * new tokens over the pages.  Same library as kvcopy.h (libkvcopy.so); the
 * pages are the blocks that kvcopy_batch moves between host and device.
 *
 * Conventions shared by every entry point:
 *   - Every function that can fail returns KVCOPY_OK (0) or a negative
 *     KVCOPY_E* code (kvcopy_strerror, kvcopy_last_hip_error).  Nothing
 *     aborts, throws or prints.
 *   - Invalid arguments are rejected before anything is enqueued.  Work is
 *     enqueued on `stream` of the current device; no call allocates,
 *     synchronises or keeps a pointer, so a HIP graph can capture any of
 *     them.  Calls on several streams are independent as long as they share
 *     no output and no workspace.
 *   - Structures start with struct_size = sizeof(the structure).
 *   - Pointers are device addresses.  Strides count elements, not bytes; the
 *     innermost dimension (head_dim) is contiguous.  The stride of a dimension
 *     of extent 1 is ignored.
 *   - What lives in device memory cannot be checked on the host: the kernels
 *     bound every page number, slot, row range and length themselves, never
 *     access memory outside the arrays described, and, if `status` is given,
 *     OR a KVCACHE_BAD_* bit into it (the caller clears it).
 */
#ifndef KVCACHE_H
#define KVCACHE_H

#include <stdint.h>
#include <hip/hip_runtime_api.h> /* hipStream_t only */

#include "kvcopy.h" /* status codes */

#ifdef __cplusplus
extern "C" {
#endif

/* Element types.  Rows (q, k, v, out) are BF16 or FP16, and FP32 in
 * kvcache_rope and as the output of kvcache_read; pages are BF16, FP16, FP8
 * (OCP e4m3: finite, largest 448) or INT8 (symmetric, -127..127). */
enum {
    KVCACHE_BF16 = 0,
    KVCACHE_FP16 = 1,
    KVCACHE_FP32 = 2,
    KVCACHE_FP8 = 3,
    KVCACHE_INT8 = 4
};

/* Bits of the status word. */
#define KVCACHE_BAD_PAGE 1u   /* a page number outside 0 .. num_pages - 1: its tokens read as zeros */
#define KVCACHE_BAD_SLOT 2u   /* a slot beyond the pages: not written, read as zeros */
#define KVCACHE_BAD_LENGTH 4u /* a sequence longer than max_q_len or max_context, or q_starts out of order or range */

#define KVCACHE_MAX_HEAD_DIM 512u           /* kvcache_write, kvcache_read, kvcache_rope */
#define KVCACHE_MAX_ATTENTION_HEAD_DIM 256u /* kvcache_attention */

/* [tokens, heads, head_dim]: element (t, h, d) is at data + t * token_stride
 * + h * head_stride + d. */
typedef struct kvcache_rows {
    void *data;
    int64_t token_stride;
    int64_t head_stride;
} kvcache_rows_t;

/* Keys and values in pages.  Element (page, head, place, d) of the keys is at
 * k + page * k_stride[0] + head * k_stride[1] + place * k_stride[2] + d, so
 * either order of heads and places is described.  FP8 and INT8 pages have one
 * float scale per (page, head, place), at k_scale with strides ks_stride; the
 * value of a code is code * scale.  num_pages * page_size < 2^31; offsets are
 * 64-bit. */
typedef struct kvcache_pages {
    uint32_t struct_size;
    uint32_t format;
    void *k, *v;
    float *k_scale, *v_scale; /* NULL unless FP8 or INT8 */
    int64_t k_stride[3], v_stride[3];
    int64_t ks_stride[3], vs_stride[3];
    uint64_t num_pages;
    uint32_t kv_heads, page_size, head_dim;
    uint32_t reserved;
} kvcache_pages_t;

/*
 * kvcache_rope_frequencies -- the angle per position, in radians and in 64
 * bits, of each of the rot_dim / 2 pairs: freq[i] = base^(-2 i / rot_dim),
 * scaled for contexts longer than a model was trained on.  Host only.
 *   KVCACHE_ROPE_PLAIN   as above
 *   KVCACHE_ROPE_LINEAR  freq / factor: positions interpolated
 *   KVCACHE_ROPE_BASE    base * factor^(rot_dim / (rot_dim - 2)): the slowest
 *                        pair slowed by factor, the fastest kept
 *   KVCACHE_ROPE_PARTS   by the number of turns a pair makes over `original`
 *                        positions: at least `high` turns, kept; at most
 *                        `low`, slowed by factor; between, blended linearly
 *                        in the number of turns
 * out: rot_dim / 2 doubles.  errors: KVCOPY_EINVAL (rot_dim odd, 0 or above
 * KVCACHE_MAX_HEAD_DIM; rot_dim 2 with BASE; base <= 1; factor < 1; original
 * 0, low < 0 or high <= low with PARTS; a value that is not finite; kind
 * unknown; out NULL).
 */
enum {
    KVCACHE_ROPE_PLAIN = 0,
    KVCACHE_ROPE_LINEAR = 1,
    KVCACHE_ROPE_BASE = 2,
    KVCACHE_ROPE_PARTS = 3
};
int kvcache_rope_frequencies(double *out, uint32_t rot_dim, double base, int kind, double factor,
                             uint32_t original, double low, double high);

/*
 * kvcache_rope -- turns pair i of the first rot_dim values of every head of q
 * and k by the angle position * freq[i] and multiplies it by `factor`:
 *     a' = factor * (a cos - b sin),   b' = factor * (b cos + a sin),
 * with (a, b) = values (i, i + rot_dim / 2), or (2 i, 2 i + 1) with
 * KVCACHE_ROPE_INTERLEAVED.  KVCACHE_ROPE_INVERSE turns the other way, which
 * is also the gradient of the forward form.  The other values are copied.
 * Angles are reduced to one turn in 64 bits, and cosines and sines of FP32 rows
 * are taken there; the products are in 32 bits and rounded once.
 *
 * q_out may be q, and k_out k, with the same strides (in place); any other
 * overlap is undefined.  k.data NULL: only q.  freq: rot_dim / 2 doubles in
 * device memory.  tokens 0 is a no-op.
 * errors: KVCOPY_EINVAL (struct_size; dtype not BF16, FP16 or FP32; a NULL
 * pointer; head_dim 0 or above KVCACHE_MAX_HEAD_DIM; rot_dim odd or above
 * head_dim; q_heads 0 or above 2^16; tokens >= 2^31; unknown flags; factor not
 * finite), KVCOPY_EALIGN (a pointer not aligned to its element), KVCOPY_EHIP.
 */
#define KVCACHE_ROPE_INTERLEAVED 1u
#define KVCACHE_ROPE_INVERSE 2u
typedef struct kvcache_rope {
    uint32_t struct_size;
    uint32_t dtype;
    uint32_t flags;
    float factor;
    const int32_t *positions; /* tokens; may be negative */
    const double *freq;
    uint64_t tokens;
    uint32_t head_dim, rot_dim, q_heads, k_heads;
    kvcache_rows_t q, k, q_out, k_out;
} kvcache_rope_t;
int kvcache_rope(const kvcache_rope_t *args, hipStream_t stream);

/*
 * kvcache_write -- writes row t of k and v (kv_heads heads each) to slot
 * slots[t] = page * page_size + place.  A negative slot leaves the token out.
 * No two tokens of a call may share a slot of 0 or more whose contents matter:
 * tokens are written in no order and a row in several stores, so that slot ends
 * with codes, scales, keys and values of either, mixed (no other slot is
 * affected; padding may go to one slot that nobody reads).  16-bit pages have
 * the rows' dtype and take them unchanged.  8-bit pages get, for each token
 * and head of k and of v, with amax the largest magnitude and Q = 448 (FP8) or
 * 127 (INT8),
 *     scale = amax / Q   and   code = the nearest code to x * Q / amax,
 * ties to even, the quotient taken exactly; zeros give scale 0 and codes 0.
 * A row that holds an infinity or a NaN gives scale NaN and codes 0: it reads
 * back as NaN.
 * errors: KVCOPY_EINVAL (struct_size; format or dtype unknown, 16-bit pages
 * of another dtype; NULL pointers; a zero size; head_dim above
 * KVCACHE_MAX_HEAD_DIM; kv_heads above 2^16; num_pages * page_size or tokens *
 * kv_heads >= 2^31), KVCOPY_EALIGN (a pointer not aligned to its element),
 * KVCOPY_EHIP.
 */
int kvcache_write(const kvcache_pages_t *pages, uint32_t dtype, const kvcache_rows_t *k,
                  const kvcache_rows_t *v, const int64_t *slots, uint64_t tokens,
                  uint32_t *status, hipStream_t stream);

/*
 * kvcache_read -- the reverse: row t of k_out and v_out (dtype BF16, FP16 or
 * FP32) gets the values at slots[t], code * scale in 32 bits, rounded once;
 * zeros for a negative slot.  16-bit pages are converted through 32 bits.
 * errors: as kvcache_write (any dtype with any format).
 */
int kvcache_read(const kvcache_pages_t *pages, uint32_t dtype, const kvcache_rows_t *k_out,
                 const kvcache_rows_t *v_out, const int64_t *slots, uint64_t tokens,
                 uint32_t *status, hipStream_t stream);

/*
 * kvcache_attention -- attention of new tokens over the paged cache, which
 * already holds them.  Sequence s has the query rows q_starts[s] ..
 * q_starts[s + 1] - 1 (q_starts[0] = 0, q_starts[num_seqs] = total_q) and
 * context_lens[s] tokens in the cache, token t in page
 * page_table[s * table_stride + t / page_size], place t % page_size.  Query r
 * of n stands at position p = context_len - n + r and sees the keys at
 * positions j <= p and, with window > 0, j > p - window:
 *     out = sum_j softmax_j(scale * q . k_j) v_j,   lse = log sum_j exp(scale * q . k_j).
 * Query head h reads key/value head h / (q_heads / kv_heads).  A row that sees
 * no key gives out 0 and lse -infinity.  Keys and values a row does not see
 * never reach it, whatever they hold (an infinity or a NaN among them); those
 * past context_len are not read, and page numbers past the last one used are
 * ignored.
 * One new token a sequence (a decode step), a few (a drafted continuation) and
 * long chunks go through the same call.
 *
 * Products are accumulated in 32 bits.  Softmax weights, multiplied with the
 * value's scale, are rounded before the second product: to fp16 where the pages
 * are FP16 (from 2^-21 of a row's largest weight down in steps of 2^-31 of it),
 * else to bf16.  For at most 16 rows a key/value head they are two such parts (22
 * bits in fp16, 16 in bf16), for FP16 rows over 8-bit pages always.  Their sum is
 * kept unrounded.  There are no atomics: the same call gives the same bits.
 *
 * max_q_len and max_context bound the lengths (they shape the launch; a longer
 * sequence sets KVCACHE_BAD_LENGTH, and what lies beyond the bound is neither
 * computed nor seen; rows of out that no sequence covers are undefined).  The
 * workspace, kvcache_attention_workspace_bytes of the same structures (it
 * depends on the sizes alone, and may be 0), is scratch for one call at a time.
 * errors: KVCOPY_EINVAL (struct_size; dtype not BF16 or FP16, or 16-bit pages
 * of another dtype; NULL pointers; head_dim 0 or above
 * KVCACHE_MAX_ATTENTION_HEAD_DIM; q_heads no multiple of kv_heads or above
 * 2^16; num_seqs above 65535; total_q, max_q_len * group, max_context >= 2^31
 * - 2^16; table_columns too few for max_context; window negative; scale above
 * 1e38 or NaN; a page or place stride negative, or 2^35 or more (a scale's:
 * 2^32); workspace too small; launch beyond the grid's limit), KVCOPY_EALIGN
 * (head_dim, a stride or an address of q, out or pages no multiple of 8
 * elements; workspace no multiple of 16 bytes), KVCOPY_EHIP.
 */
typedef struct kvcache_attention {
    uint32_t struct_size;
    uint32_t dtype;
    kvcache_rows_t q, out;
    float *lse;                               /* may be NULL */
    int64_t lse_token_stride, lse_head_stride;
    const int32_t *page_table;
    int64_t table_stride;
    const int32_t *q_starts;                  /* num_seqs + 1 */
    const int32_t *context_lens;              /* num_seqs */
    void *workspace;
    uint64_t workspace_bytes;
    uint32_t *status;                         /* may be NULL */
    uint32_t num_seqs, q_heads, table_columns, total_q;
    uint32_t max_q_len, max_context;
    int32_t window;                           /* 0: none */
    float scale;
} kvcache_attention_t;
uint64_t kvcache_attention_workspace_bytes(const kvcache_pages_t *pages,
                                           const kvcache_attention_t *args);
/* Whether kvcache_attention would take these sizes and pages: its checks of
 * everything but the other pointers, their strides and the workspace, for a
 * caller who sets up a call before its tensors are there. */
int kvcache_attention_check(const kvcache_pages_t *pages, const kvcache_attention_t *args);
int kvcache_attention(const kvcache_pages_t *pages, const kvcache_attention_t *args,
                      hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* KVCACHE_H */
