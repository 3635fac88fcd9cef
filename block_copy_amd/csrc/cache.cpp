// cache.cpp -- the C entry points of the cache operators (include/kvcache.h):
// argument checks, and the hand-over to the kernels.
#include <cmath>
#include <cstddef>

#include "cache_internal.h"
#include "kvcopy_internal.h"

namespace kvc {
namespace {

constexpr uint32_t kMaxHeads = 1u << 16;
constexpr double kPi = 3.14159265358979323846;
constexpr double kLog2E = 1.4426950408889634074;

uint32_t element_bytes(uint32_t type)
{
    return type == KVCACHE_FP32 ? 4 : type == KVCACHE_BF16 || type == KVCACHE_FP16 ? 2 : 1;
}

bool aligned(const void *p, uint64_t bytes)
{
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// Whether pieces of 8 elements of this array can be moved at once: 16 bytes
// (8 of 8-bit types) to an address.
bool pieces(const void *p, uint32_t type, int64_t s0, int64_t s1, int64_t s2 = 0)
{
    const uint32_t bytes = element_bytes(type) == 1 ? 8 : 16;
    return aligned(p, bytes) && s0 % 8 == 0 && s1 % 8 == 0 && s2 % 8 == 0;
}

// The stride of a dimension, as far as it matters: one of extent 1 is never
// stepped over, and the stride that a slice gives it may be anything.
int64_t step(int64_t stride, uint64_t extent)
{
    return extent > 1 ? stride : 0;
}

struct PageSteps {
    int64_t page, head, place;
    PageSteps(const kvcache_pages_t *p, const int64_t *stride)
        : page(step(stride[0], p->num_pages)), head(step(stride[1], p->kv_heads)), place(step(stride[2], p->page_size))
    {
    }
};

int check_pages(const kvcache_pages_t *p, uint32_t most)
{
    if (!p || p->struct_size != sizeof(*p))
        return KVCOPY_EINVAL;
    if (p->format != KVCACHE_BF16 && p->format != KVCACHE_FP16 && p->format != KVCACHE_FP8 &&
        p->format != KVCACHE_INT8)
        return KVCOPY_EINVAL;
    const bool coded = element_bytes(p->format) == 1;
    if (!p->k || !p->v || (coded && (!p->k_scale || !p->v_scale)))
        return KVCOPY_EINVAL;
    if (p->num_pages == 0 || p->kv_heads == 0 || p->page_size == 0 || p->head_dim == 0 ||
        p->head_dim > most || p->kv_heads > kMaxHeads)
        return KVCOPY_EINVAL;
    if (p->num_pages >= 1ull << 31 || p->num_pages * p->page_size >= 1ull << 31)
        return KVCOPY_EINVAL;
    const uint32_t bytes = element_bytes(p->format);
    if (!aligned(p->k, bytes) || !aligned(p->v, bytes) ||
        (coded && (!aligned(p->k_scale, 4) || !aligned(p->v_scale, 4))))
        return KVCOPY_EALIGN;
    return KVCOPY_OK;
}

bool rope_pieces(const kvcache_rows_t &r, const kvcache_rope_t *g, uint32_t heads)
{
    return pieces(r.data, g->dtype, step(r.token_stride, g->tokens), step(r.head_stride, heads));
}

// The checks and arguments that kvcache_write and kvcache_read share.
int row_args(const kvcache_pages_t *p, uint32_t dtype, const kvcache_rows_t *k, const kvcache_rows_t *v,
             const int64_t *slots, uint64_t tokens, uint32_t *status, RowArgs &a, bool &wide)
{
    const int rc = check_pages(p, KVCACHE_MAX_HEAD_DIM);
    if (rc != KVCOPY_OK)
        return rc;
    if (!k || !v || tokens >= 1ull << 31 || tokens * p->kv_heads >= 1ull << 31)
        return KVCOPY_EINVAL;
    if (tokens == 0)
        return KVCOPY_OK;
    if (!k->data || !v->data || !slots)
        return KVCOPY_EINVAL;
    const uint32_t bytes = element_bytes(dtype);
    if (!aligned(k->data, bytes) || !aligned(v->data, bytes) || !aligned(slots, 8) || !aligned(status, 4))
        return KVCOPY_EALIGN;
    const kvcache_rows_t *rows[2] = {k, v};
    void *pages[2] = {p->k, p->v};
    float *scale[2] = {p->k_scale, p->v_scale};
    const int64_t *ps[2] = {p->k_stride, p->v_stride}, *ss[2] = {p->ks_stride, p->vs_stride};
    wide = p->head_dim % 8 == 0;
    for (int i = 0; i < 2; ++i) {
        a.pages[i] = pages[i];
        a.scale[i] = scale[i];
        a.p_page[i] = ps[i][0];
        a.p_head[i] = ps[i][1];
        a.p_place[i] = ps[i][2];
        a.s_page[i] = ss[i][0];
        a.s_head[i] = ss[i][1];
        a.s_place[i] = ss[i][2];
        a.rows[i] = rows[i]->data;
        a.r_token[i] = rows[i]->token_stride;
        a.r_head[i] = rows[i]->head_stride;
        const PageSteps s(p, ps[i]);
        wide = wide && pieces(pages[i], p->format, s.page, s.head, s.place) &&
               pieces(rows[i]->data, dtype, step(rows[i]->token_stride, tokens), step(rows[i]->head_stride, p->kv_heads));
    }
    a.slots = slots;
    a.status = status;
    a.num_slots = (uint32_t)(p->num_pages * p->page_size);
    a.tokens = (uint32_t)tokens;
    a.head_dim = p->head_dim;
    a.page_size = make_divider(p->page_size);
    a.kv_heads = make_divider(p->kv_heads);
    return KVCOPY_OK;
}

// Checks of kvcache_attention that need no device pointer (its workspace's
// size needs only these).
int attention_sizes(const kvcache_pages_t *p, const kvcache_attention_t *g)
{
    const int rc = check_pages(p, KVCACHE_MAX_ATTENTION_HEAD_DIM);
    if (rc != KVCOPY_OK)
        return rc;
    if (!g || g->struct_size != sizeof(*g) || (g->dtype != KVCACHE_BF16 && g->dtype != KVCACHE_FP16))
        return KVCOPY_EINVAL;
    if (element_bytes(p->format) == 2 && p->format != g->dtype)
        return KVCOPY_EINVAL;
    if (g->q_heads == 0 || g->q_heads > kMaxHeads || g->q_heads % p->kv_heads != 0)
        return KVCOPY_EINVAL;
    // what the kernels hold in 32 bits: pieces of 8 elements, and scales
    const auto fits = [p](const int64_t *stride, int bits) {
        const PageSteps s(p, stride);
        return (uint64_t)s.page < 1ull << bits && (uint64_t)s.place < 1ull << bits;
    };
    if (!fits(p->k_stride, 35) || !fits(p->v_stride, 35) ||
        (element_bytes(p->format) == 1 && (!fits(p->ks_stride, 32) || !fits(p->vs_stride, 32))))
        return KVCOPY_EINVAL;
    const uint64_t group = g->q_heads / p->kv_heads, most = (1ull << 31) - (1ull << 16);
    if (g->num_seqs > 65535 || g->total_q * group >= most || g->max_q_len * group >= most ||
        g->max_context >= most || g->window < 0 || !(std::fabs((double)g->scale) <= 1e38))
        return KVCOPY_EINVAL;
    if ((uint64_t)g->table_columns * p->page_size < g->max_context)
        return KVCOPY_EINVAL;
    return KVCOPY_OK;
}

// How such a call is laid out, and whether its launches fit a grid of 2^32 threads.
int attention_layout(const kvcache_pages_t *p, const kvcache_attention_t *g, AttentionShape &shape)
{
    shape = attention_shape(g->num_seqs, g->total_q, g->q_heads, p->kv_heads, p->head_dim, g->max_q_len,
                            g->max_context, (uint32_t)g->window);
    if ((uint64_t)p->kv_heads * shape.splits * shape.tiles >= 1ull << 23)
        return KVCOPY_EINVAL;
    // splits are joined by a workgroup of 256 for up to every row
    if (shape.splits > 1 && (uint64_t)g->total_q * g->q_heads >= 1ull << 24)
        return KVCOPY_EINVAL;
    return KVCOPY_OK;
}

bool attention_aligned(const kvcache_pages_t *p)
{
    const PageSteps k(p, p->k_stride), v(p, p->v_stride);
    return p->head_dim % 8 == 0 && pieces(p->k, p->format, k.page, k.head, k.place) &&
           pieces(p->v, p->format, v.page, v.head, v.place);
}

bool no_rows(const kvcache_attention_t *g)
{
    return g->num_seqs == 0 || g->total_q == 0 || g->max_q_len == 0;
}

}  // namespace
}  // namespace kvc

using namespace kvc;

extern "C" int kvcache_rope_frequencies(double *out, uint32_t rot_dim, double base, int kind, double factor,
                                        uint32_t original, double low, double high)
{
    if (!out || rot_dim == 0 || rot_dim % 2 || rot_dim > KVCACHE_MAX_HEAD_DIM)
        return KVCOPY_EINVAL;
    if (!std::isfinite(base) || !(base > 1.0) || kind < KVCACHE_ROPE_PLAIN || kind > KVCACHE_ROPE_PARTS)
        return KVCOPY_EINVAL;
    if (kind != KVCACHE_ROPE_PLAIN && (!std::isfinite(factor) || factor < 1.0))
        return KVCOPY_EINVAL;
    if (kind == KVCACHE_ROPE_BASE) {
        if (rot_dim == 2)
            return KVCOPY_EINVAL;
        base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
        if (!std::isfinite(base))
            return KVCOPY_EINVAL;
    }
    if (kind == KVCACHE_ROPE_PARTS &&
        (original == 0 || !std::isfinite(low) || !std::isfinite(high) || low < 0.0 || high <= low))
        return KVCOPY_EINVAL;
    for (uint32_t i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (kind == KVCACHE_ROPE_LINEAR) {
            f /= factor;
        } else if (kind == KVCACHE_ROPE_PARTS) {
            const double turns = original * f / (2.0 * kPi);
            double keep = (turns - low) / (high - low);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f *= keep + (1.0 - keep) / factor;
        }
        out[i] = f;
    }
    return KVCOPY_OK;
}

extern "C" int kvcache_rope(const kvcache_rope_t *g, hipStream_t stream)
{
    if (!g || g->struct_size != sizeof(*g))
        return KVCOPY_EINVAL;
    if (g->dtype != KVCACHE_BF16 && g->dtype != KVCACHE_FP16 && g->dtype != KVCACHE_FP32)
        return KVCOPY_EINVAL;
    if (g->flags & ~(KVCACHE_ROPE_INTERLEAVED | KVCACHE_ROPE_INVERSE) || !std::isfinite(g->factor))
        return KVCOPY_EINVAL;
    if (g->head_dim == 0 || g->head_dim > KVCACHE_MAX_HEAD_DIM || g->rot_dim % 2 || g->rot_dim > g->head_dim)
        return KVCOPY_EINVAL;
    if (g->q_heads == 0 || g->q_heads > kMaxHeads || g->k_heads > kMaxHeads || g->tokens >= 1ull << 31)
        return KVCOPY_EINVAL;
    if (g->tokens == 0)
        return KVCOPY_OK;
    const bool has_k = g->k.data != nullptr;
    if (!g->q.data || !g->q_out.data || !g->positions || (g->rot_dim && !g->freq) ||
        (has_k && (!g->k_out.data || g->k_heads == 0)))
        return KVCOPY_EINVAL;
    const uint32_t bytes = element_bytes(g->dtype);
    if (!aligned(g->q.data, bytes) || !aligned(g->q_out.data, bytes) || !aligned(g->positions, 4) ||
        !aligned(g->freq, 8) || (has_k && (!aligned(g->k.data, bytes) || !aligned(g->k_out.data, bytes))))
        return KVCOPY_EALIGN;
    RopeArgs a = {};
    a.positions = g->positions;
    a.freq = g->freq;
    a.q = g->q.data;
    a.q_out = g->q_out.data;
    a.q_st = g->q.token_stride;
    a.q_sh = g->q.head_stride;
    a.qo_st = g->q_out.token_stride;
    a.qo_sh = g->q_out.head_stride;
    if (has_k) {
        a.k = g->k.data;
        a.k_out = g->k_out.data;
        a.k_st = g->k.token_stride;
        a.k_sh = g->k.head_stride;
        a.ko_st = g->k_out.token_stride;
        a.ko_sh = g->k_out.head_stride;
    }
    a.tokens = (uint32_t)g->tokens;
    a.q_heads = g->q_heads;
    a.heads = g->q_heads + (has_k ? g->k_heads : 0);
    a.head_dim = g->head_dim;
    a.rot_dim = g->rot_dim;
    a.interleaved = (g->flags & KVCACHE_ROPE_INTERLEAVED) != 0;
    a.factor = g->factor;
    a.sign = g->flags & KVCACHE_ROPE_INVERSE ? -1.0f : 1.0f;
    const bool wide = g->head_dim % 8 == 0 && g->rot_dim % (a.interleaved ? 8 : 16) == 0 &&
                      rope_pieces(g->q, g, g->q_heads) && rope_pieces(g->q_out, g, g->q_heads) &&
                      (!has_k || (rope_pieces(g->k, g, g->k_heads) && rope_pieces(g->k_out, g, g->k_heads)));
    const hipError_t e = launch_rope(a, g->dtype, wide, stream);
    return e == hipSuccess ? KVCOPY_OK : hip_fail(e);
}

extern "C" int kvcache_write(const kvcache_pages_t *pages, uint32_t dtype, const kvcache_rows_t *k,
                             const kvcache_rows_t *v, const int64_t *slots, uint64_t tokens,
                             uint32_t *status, hipStream_t stream)
{
    if (dtype != KVCACHE_BF16 && dtype != KVCACHE_FP16)
        return KVCOPY_EINVAL;
    RowArgs a = {};
    bool wide = false;
    const int rc = row_args(pages, dtype, k, v, slots, tokens, status, a, wide);
    if (rc != KVCOPY_OK)
        return rc;
    if (element_bytes(pages->format) == 2 && pages->format != dtype)
        return KVCOPY_EINVAL;
    if (tokens == 0)
        return KVCOPY_OK;
    const hipError_t e = launch_write(a, dtype, pages->format, wide, stream);
    return e == hipSuccess ? KVCOPY_OK : hip_fail(e);
}

extern "C" int kvcache_read(const kvcache_pages_t *pages, uint32_t dtype, const kvcache_rows_t *k_out,
                            const kvcache_rows_t *v_out, const int64_t *slots, uint64_t tokens,
                            uint32_t *status, hipStream_t stream)
{
    if (dtype != KVCACHE_BF16 && dtype != KVCACHE_FP16 && dtype != KVCACHE_FP32)
        return KVCOPY_EINVAL;
    RowArgs a = {};
    bool wide = false;
    const int rc = row_args(pages, dtype, k_out, v_out, slots, tokens, status, a, wide);
    if (rc != KVCOPY_OK || tokens == 0)
        return rc;
    const hipError_t e = launch_read(a, dtype, pages->format, wide, stream);
    return e == hipSuccess ? KVCOPY_OK : hip_fail(e);
}

extern "C" uint64_t kvcache_attention_workspace_bytes(const kvcache_pages_t *pages,
                                                      const kvcache_attention_t *args)
{
    if (attention_sizes(pages, args) != KVCOPY_OK)
        return 0;
    return attention_shape(args->num_seqs, args->total_q, args->q_heads, pages->kv_heads, pages->head_dim,
                           args->max_q_len, args->max_context, (uint32_t)args->window)
        .workspace_bytes;
}

extern "C" int kvcache_attention_check(const kvcache_pages_t *p, const kvcache_attention_t *g)
{
    int rc = attention_sizes(p, g);
    AttentionShape shape;
    if (rc == KVCOPY_OK && !no_rows(g))
        rc = attention_layout(p, g, shape);
    return rc != KVCOPY_OK ? rc : attention_aligned(p) ? KVCOPY_OK : KVCOPY_EALIGN;
}

extern "C" int kvcache_attention(const kvcache_pages_t *p, const kvcache_attention_t *g, hipStream_t stream)
{
    int rc = attention_sizes(p, g);
    if (rc != KVCOPY_OK)
        return rc;
    if (no_rows(g))
        return KVCOPY_OK;
    if (!g->q.data || !g->out.data || !g->q_starts || !g->context_lens || (g->max_context && !g->page_table))
        return KVCOPY_EINVAL;
    AttentionShape shape;
    rc = attention_layout(p, g, shape);
    if (rc != KVCOPY_OK)
        return rc;
    if (shape.workspace_bytes > g->workspace_bytes || (shape.workspace_bytes && !g->workspace))
        return KVCOPY_EINVAL;
    if (!attention_aligned(p) ||
        !pieces(g->q.data, g->dtype, step(g->q.token_stride, g->total_q), step(g->q.head_stride, g->q_heads)) ||
        !pieces(g->out.data, g->dtype, step(g->out.token_stride, g->total_q), step(g->out.head_stride, g->q_heads)) ||
        (shape.workspace_bytes && !aligned(g->workspace, 16)) || !aligned(g->lse, 4) || !aligned(g->status, 4) ||
        !aligned(g->page_table, 4) || !aligned(g->q_starts, 4) || !aligned(g->context_lens, 4))
        return KVCOPY_EALIGN;
    AttentionArgs a = {};
    a.q = g->q.data;
    a.out = g->out.data;
    a.lse = g->lse;
    a.q_st = g->q.token_stride;
    a.q_sh = g->q.head_stride;
    a.o_st = g->out.token_stride;
    a.o_sh = g->out.head_stride;
    a.l_st = g->lse_token_stride;
    a.l_sh = g->lse_head_stride;
    a.k = p->k;
    a.v = p->v;
    a.k_scale = p->k_scale;
    a.v_scale = p->v_scale;
    const PageSteps k(p, p->k_stride), v(p, p->v_stride), ks(p, p->ks_stride), vs(p, p->vs_stride);
    a.k_page = (uint32_t)(k.page / 8);
    a.k_head = k.head;
    a.k_place = (uint32_t)(k.place / 8);
    a.v_page = (uint32_t)(v.page / 8);
    a.v_head = v.head;
    a.v_place = (uint32_t)(v.place / 8);
    a.ks_page = (uint32_t)ks.page;
    a.ks_head = ks.head;
    a.ks_place = (uint32_t)ks.place;
    a.vs_page = (uint32_t)vs.page;
    a.vs_head = vs.head;
    a.vs_place = (uint32_t)vs.place;
    a.table = g->page_table;
    a.table_stride = g->table_stride;
    a.q_starts = g->q_starts;
    a.context_lens = g->context_lens;
    a.status = g->status;
    a.num_pages = (uint32_t)p->num_pages;
    a.total_q = g->total_q;
    a.max_q_len = g->max_q_len;
    a.max_context = g->max_context;
    a.q_heads = g->q_heads;
    a.kv_heads = p->kv_heads;
    a.head_dim = p->head_dim;
    a.full = p->head_dim == 64 || p->head_dim == 128 || p->head_dim == 256;
    if (element_bytes(p->format) == 1)
        a.full = a.full && aligned(p->k, 16) && aligned(p->v, 16) && k.page % 16 == 0 && k.head % 16 == 0 &&
                 k.place % 16 == 0 && v.page % 16 == 0 && v.head % 16 == 0 && v.place % 16 == 0;
    a.tiles = shape.tiles;
    a.splits = shape.splits;
    a.split_keys = shape.split_keys;
    a.window = g->window;
    a.scale_log2 = g->scale == 0.0f ? 1.0f : (float)(std::fabs((double)g->scale) * kLog2E);
    a.q_keep = g->scale == 0.0f ? 0 : ~0u;
    a.q_flip = g->scale < 0.0f ? 0x80008000u : 0;
    a.page_size = make_divider(p->page_size);
    a.group = make_divider(g->q_heads / p->kv_heads);
    if (shape.splits > 1) {
        a.part_o = (float *)g->workspace;
        a.part_ml = a.part_o + (uint64_t)shape.splits * g->total_q * g->q_heads * p->head_dim;
    }
    const hipError_t e = launch_attention(a, shape, g->num_seqs, g->dtype, p->format, stream);
    return e == hipSuccess ? KVCOPY_OK : hip_fail(e);
}
