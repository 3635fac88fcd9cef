// cache_kernels.hip -- rotary positions, and rows of keys and values written
// into cache pages and read back from them.  All three are bound by memory:
// every value is read once and written once, in 16-byte pieces where sizes
// and addresses allow it (`wide`), else element by element.
#include <hip/hip_runtime.h>

#include "cache_internal.h"
#include "cache_types.h"

namespace kvc {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kMaxBlocks = 1u << 22;

// ---- rotary positions -------------------------------------------------------
//
// a' = f (a cos t - b sin t), b' = f (b cos t + a sin t), t = position * freq.
// A workgroup takes block_tokens tokens: it first computes their cosines and
// sines, one pair a thread, into shared memory, and then turns all heads with
// them, so the angle (a product and a reduction to one turn in 64 bits, since
// a position of 2^20 has lost 2^-4 radians in 32) costs little beside the
// heads' traffic.  The rows are read past the caches (their last use: 64.2
// against 66.6 us for 16,384 tokens of 32 + 8 heads of 128 in bf16, 5.2 TB/s of
// reads and writes, where the runtime's copy reaches 5.0 to 5.2 and kvcopy's
// own, at its best shape, 6.2); the results, used next, go through them.

struct Turn {
    float c, s;
};

// Rows of 32 bits take their cosine and sine from 64 bits, rounded once: the
// part of a turn in 32 bits is off by up to 2^-23 radians, which 16-bit rows do
// not see (16,384 tokens of 32 + 8 heads of 128: 138 us, and 139 in 32 bits).
template <class T>
__device__ __forceinline__ Turn turn_of(int32_t position, double freq, float factor, float sign)
{
    const double turns = (double)position * (freq * 0.15915494309189533577);   // 1 / (2 pi)
    const double part = turns - __builtin_rint(turns);                         // -0.5 .. 0.5
    Turn t;
    if constexpr (__is_same(T, Fp32)) {
        double s, c;
        sincospi(2.0 * part, &s, &c);
        t.c = (float)(c * factor);
        t.s = (float)(s * (factor * sign));
    } else {
        sincospif(2.0f * (float)part, &t.s, &t.c);
        t.c *= factor;
        t.s *= factor * sign;
    }
    return t;
}

// The fused products are spelled out, and their results kept in 32 bits (the
// compiler would fuse the rounding to fp16 into some of them), so that every
// variant rounds alike.
__device__ __forceinline__ void rotate(float &a, float &b, Turn t)
{
    const float x = __builtin_fmaf(a, t.c, -(b * t.s));
    b = __builtin_fmaf(b, t.c, a * t.s);
    a = x;
    asm("" : "+v"(a), "+v"(b));
}

template <class T>
__device__ __forceinline__ const typename T::elem *rope_row(const RopeArgs &r, uint32_t token,
                                                            uint32_t head, typename T::elem *&out)
{
    typedef typename T::elem E;
    if (head < r.q_heads) {
        out = (E *)r.q_out + token * r.qo_st + head * r.qo_sh;
        return (const E *)r.q + token * r.q_st + head * r.q_sh;
    }
    head -= r.q_heads;
    out = (E *)r.k_out + token * r.ko_st + head * r.ko_sh;
    return (const E *)r.k + token * r.k_st + head * r.k_sh;
}

template <class T, bool Wide, bool Interleaved>
__global__ __launch_bounds__(kThreads) void kvcache_rope_kernel(const RopeArgs r)
{
    typedef typename T::elem E;
    typedef typename T::piece P;
    __shared__ Turn turns[kThreads];
    const uint32_t half = r.rot_dim / 2;
    for (uint64_t first = (uint64_t)blockIdx.x * r.block_tokens; first < r.tokens;
         first += (uint64_t)gridDim.x * r.block_tokens) {
        const uint32_t left = r.tokens - (uint32_t)first;
        const uint32_t n = left < r.block_tokens ? left : r.block_tokens;
        for (uint32_t i = threadIdx.x; i < n * half; i += kThreads)
            turns[i] = turn_of<T>(r.positions[first + i / half], r.freq[i % half], r.factor, r.sign);
        __syncthreads();
        if (Wide) {
            // an item is one piece of 8 values, or the two pieces of 8 pairs
            const uint32_t turned = Interleaved ? r.rot_dim / 8 : r.rot_dim / 16;
            const uint32_t items = turned + (r.head_dim - r.rot_dim) / 8;
            for (uint32_t i = threadIdx.x; i < n * r.heads * items; i += kThreads) {
                const uint32_t row = i / items, c = i - row * items, t = row / r.heads;
                E *out;
                const E *in = rope_row<T>(r, (uint32_t)first + t, row - t * r.heads, out);
                float x[8], y[8];
                if (c >= turned) {
                    const uint32_t at = r.rot_dim + (c - turned) * 8;
                    *(P *)(out + at) = load_once((const P *)(in + at));
                } else if (Interleaved) {
                    const Turn *w = turns + t * half + c * 4;
                    unpack8<T>(load_once((const P *)(in + c * 8)), x);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        rotate(x[2 * j], x[2 * j + 1], w[j]);
                    *(P *)(out + c * 8) = pack8<T>(x);
                } else {
                    const Turn *w = turns + t * half + c * 8;
                    unpack8<T>(load_once((const P *)(in + c * 8)), x);
                    unpack8<T>(load_once((const P *)(in + half + c * 8)), y);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        rotate(x[j], y[j], w[j]);
                    *(P *)(out + c * 8) = pack8<T>(x);
                    *(P *)(out + half + c * 8) = pack8<T>(y);
                }
            }
        } else {
            const uint32_t items = half + (r.head_dim - r.rot_dim);
            for (uint32_t i = threadIdx.x; i < n * r.heads * items; i += kThreads) {
                const uint32_t row = i / items, c = i - row * items, t = row / r.heads;
                E *out;
                const E *in = rope_row<T>(r, (uint32_t)first + t, row - t * r.heads, out);
                if (c >= half) {
                    out[half + c] = in[half + c];
                } else {
                    const uint32_t ia = Interleaved ? 2 * c : c, ib = Interleaved ? 2 * c + 1 : c + half;
                    float a = (float)in[ia], b = (float)in[ib];
                    rotate(a, b, turns[t * half + c]);
                    out[ia] = (E)a;
                    out[ib] = (E)b;
                }
            }
        }
        __syncthreads();   // the angles are overwritten next
    }
}

// ---- rows into pages --------------------------------------------------------

// What a row's largest magnitude makes of its quotients x * Q / amax.  The
// quotient has to be rounded to a code as if it were exact, and x = amax / 2
// lies on a border of int8 whatever amax is.  x * Q is exact in 32 bits (11 + 7
// bits at most), and a quotient that is not on a border is at least 2^-20 of
// itself away from one (x * Q and border * amax are whole multiples of one
// unit, of at most 20 bits).  One reciprocal, a product and one correction by
// the exact remainder give the quotient to 2^-23, and exactly where it is
// representable, as every border is.  `pre`, a power of two, keeps both sides
// away from the ends of the exponent range.
struct Quantiser {
    float scale, mul, div, inv;
    __device__ __forceinline__ Quantiser(float amax, float top, bool finite)
    {
        const float pre = amax < 0x1p-60f ? 0x1p64f : amax > 0x1p60f ? 0x1p-64f : 1.0f;
        scale = finite ? amax / top : __builtin_nanf("");
        mul = finite ? top * pre : 0.0f;
        div = finite && amax > 0.0f ? amax * pre : 1.0f;
        inv = __builtin_amdgcn_rcpf(div);
    }
    __device__ __forceinline__ float operator()(float x) const
    {
        const float n = x * mul;
        const float y = n * inv;
        return __builtin_fmaf(__builtin_fmaf(-y, div, n), inv, y);
    }
};

template <class T>
__device__ __forceinline__ float value_of(uint32_t bits)
{
    return (float)__builtin_bit_cast(typename T::elem, (uint16_t)bits);
}

// kvcache_write: `Lanes` lanes share a row of keys and the same row of values,
// a 16-byte piece each; a row's largest magnitude goes over them in log2(Lanes)
// exchanges.  Format void: the pages hold T itself.  Bound by memory: 32,768
// tokens of 8 heads of 128, bf16 to e4m3, in 40 us, 5.1 TB/s of reads and
// writes.
template <class T, class Format, int Lanes>
__global__ __launch_bounds__(kThreads) void kvcache_write_kernel(const RowArgs a)
{
    const uint32_t lane = threadIdx.x % Lanes;
    const uint64_t rows = (uint64_t)a.tokens * a.kv_heads.d;
    const bool in = lane * 8 < a.head_dim;
    for (uint64_t row = (uint64_t)blockIdx.x * (kThreads / Lanes) + threadIdx.x / Lanes; row < rows;
         row += (uint64_t)gridDim.x * (kThreads / Lanes)) {
        const uint32_t token = a.kv_heads.div((uint32_t)row), head = a.kv_heads.mod((uint32_t)row, token);
        const int32_t slot = checked_slot(a.slots[token], a.num_slots);
        u32x4 p[2] = {};
        if (in) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                p[i] = *(const u32x4 *)((const typename T::elem *)a.rows[i] + token * a.r_token[i] +
                                        head * a.r_head[i] + lane * 8);
        }
        if (slot == -2 && lane == 0)
            set_status(a.status, KVCACHE_BAD_SLOT);
        const uint32_t page = a.page_size.div(slot < 0 ? 0 : slot);
        const uint32_t place = a.page_size.mod(slot < 0 ? 0 : slot, page);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t at = page_offset(page, place, a.p_page[i], a.p_place[i]) +
                               head * a.p_head[i] + lane * 8;
            if constexpr (__is_same(Format, void)) {
                if (in && slot >= 0)
                    *(u32x4 *)((typename T::elem *)a.pages[i] + at) = p[i];
            } else {
                uint32_t m = max_halves(max_halves(p[i].x & 0x7fff7fffu, p[i].y & 0x7fff7fffu),
                                  max_halves(p[i].z & 0x7fff7fffu, p[i].w & 0x7fff7fffu));
#pragma unroll
                for (int x = 1; x < Lanes; x <<= 1)
                    m = max_halves(m, __shfl_xor(m, x, 64));
                m = (m >> 16) > (m & 0xffffu) ? m >> 16 : m & 0xffffu;
                const Quantiser quant(value_of<T>(m < T::kExponent ? m : 0), Format::kQ,
                                      m < T::kExponent);
                float x[8];
                unpack8<T>(p[i], x);
                u32x2 c;
                if (m < T::kExponent) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        x[j] = quant(x[j]);
                    c.x = Format::code4(x[0], x[1], x[2], x[3]);
                    c.y = Format::code4(x[4], x[5], x[6], x[7]);
                } else {
                    c = u32x2{0, 0};
                }
                if (in && slot >= 0)
                    *(u32x2 *)((uint8_t *)a.pages[i] + at) = c;
                if (lane == 0 && slot >= 0)
                    a.scale[i][page_offset(page, place, a.s_page[i], a.s_place[i]) + head * a.s_head[i]] =
                        quant.scale;
            }
        }
    }
}

// The same for rows of any size and address: a wavefront to a row, an element
// at a time.
template <class T, class Format>
__global__ __launch_bounds__(kThreads) void kvcache_write_any_kernel(const RowArgs a)
{
    const uint32_t lane = threadIdx.x & 63u;
    const uint64_t rows = (uint64_t)a.tokens * a.kv_heads.d;
    for (uint64_t row = (uint64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); row < rows;
         row += (uint64_t)gridDim.x * (kThreads / 64)) {
        const uint32_t token = a.kv_heads.div((uint32_t)row), head = a.kv_heads.mod((uint32_t)row, token);
        const int32_t slot = checked_slot(a.slots[token], a.num_slots);
        if (slot < 0) {
            if (slot == -2 && lane == 0)
                set_status(a.status, KVCACHE_BAD_SLOT);
            continue;   // the whole wavefront
        }
        const uint32_t page = a.page_size.div(slot), place = a.page_size.mod(slot, page);
        for (int i = 0; i < 2; ++i) {
            const uint16_t *in = (const uint16_t *)a.rows[i] + token * a.r_token[i] + head * a.r_head[i];
            const int64_t at = page_offset(page, place, a.p_page[i], a.p_place[i]) + head * a.p_head[i];
            if constexpr (__is_same(Format, void)) {
                for (uint32_t d = lane; d < a.head_dim; d += 64)
                    ((uint16_t *)a.pages[i])[at + d] = in[d];
            } else {
                uint32_t m = 0;
                for (uint32_t d = lane; d < a.head_dim; d += 64) {
                    const uint32_t x = in[d] & 0x7fffu;
                    m = m > x ? m : x;
                }
                for (int x = 1; x < 64; x <<= 1) {
                    const uint32_t o = __shfl_xor(m, x, 64);
                    m = m > o ? m : o;
                }
                const Quantiser quant(value_of<T>(m < T::kExponent ? m : 0), Format::kQ,
                                      m < T::kExponent);
                for (uint32_t d = lane; d < a.head_dim; d += 64) {
                    const float y = m < T::kExponent ? quant(value_of<T>(in[d])) : 0.0f;
                    ((uint8_t *)a.pages[i])[at + d] = (uint8_t)Format::code4(y, 0.0f, 0.0f, 0.0f);
                }
                if (lane == 0)
                    a.scale[i][page_offset(page, place, a.s_page[i], a.s_place[i]) + head * a.s_head[i]] =
                        quant.scale;
            }
        }
    }
}

// ---- rows back from pages ---------------------------------------------------

// kvcache_read: lanes share rows as in kvcache_write.  Both sides pass the
// caches by: the rows are read back in bulk, for a connector or another
// process (65,536 tokens of 8 heads of 128, int8 to bf16: 75.8 us, against
// 84.7 us without).  S: what the pages hold; T: the output's type.
template <class S>
struct IsCode {
    static constexpr bool value = __is_same(S, Fp8) || __is_same(S, Int8);
};

template <class S, class T, int Lanes>
__global__ __launch_bounds__(kThreads) void kvcache_read_kernel(const RowArgs a)
{
    const uint32_t lane = threadIdx.x % Lanes;
    const uint64_t rows = (uint64_t)a.tokens * a.kv_heads.d;
    if (lane * 8 >= a.head_dim)
        return;
    for (uint64_t row = (uint64_t)blockIdx.x * (kThreads / Lanes) + threadIdx.x / Lanes; row < rows;
         row += (uint64_t)gridDim.x * (kThreads / Lanes)) {
        const uint32_t token = a.kv_heads.div((uint32_t)row), head = a.kv_heads.mod((uint32_t)row, token);
        const int32_t slot = checked_slot(a.slots[token], a.num_slots);
        if (slot == -2 && lane == 0)
            set_status(a.status, KVCACHE_BAD_SLOT);
        const uint32_t page = a.page_size.div(slot < 0 ? 0 : slot);
        const uint32_t place = a.page_size.mod(slot < 0 ? 0 : slot, page);
        typename T::piece out[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t at = page_offset(page, place, a.p_page[i], a.p_place[i]) +
                               head * a.p_head[i] + lane * 8;
            float x[8] = {};
            if constexpr (IsCode<S>::value) {
                if (slot >= 0) {
                    const u32x2 c = load_once((const u32x2 *)((const uint8_t *)a.pages[i] + at));
                    const float scale = a.scale[i][page_offset(page, place, a.s_page[i], a.s_place[i]) +
                                                   head * a.s_head[i]];
                    S::value4(c.x, x);
                    S::value4(c.y, x + 4);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        x[j] *= scale;
                }
                out[i] = pack8<T>(x);
            } else if constexpr (__is_same(S, T)) {
                out[i] = slot >= 0 ? load_once((const u32x4 *)((const typename S::elem *)a.pages[i] + at)) : u32x4{};
            } else {
                if (slot >= 0)
                    unpack8<S>(load_once((const u32x4 *)((const typename S::elem *)a.pages[i] + at)), x);
                out[i] = pack8<T>(x);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            store_once((typename T::piece *)((typename T::elem *)a.rows[i] + token * a.r_token[i] +
                                             head * a.r_head[i] + lane * 8), out[i]);
    }
}

template <class S, class T>
__global__ __launch_bounds__(kThreads) void kvcache_read_any_kernel(const RowArgs a)
{
    const uint32_t lane = threadIdx.x & 63u;
    const uint64_t rows = (uint64_t)a.tokens * a.kv_heads.d;
    for (uint64_t row = (uint64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); row < rows;
         row += (uint64_t)gridDim.x * (kThreads / 64)) {
        const uint32_t token = a.kv_heads.div((uint32_t)row), head = a.kv_heads.mod((uint32_t)row, token);
        const int32_t slot = checked_slot(a.slots[token], a.num_slots);
        if (slot == -2 && lane == 0)
            set_status(a.status, KVCACHE_BAD_SLOT);
        const uint32_t page = a.page_size.div(slot < 0 ? 0 : slot);
        const uint32_t place = a.page_size.mod(slot < 0 ? 0 : slot, page);
        for (int i = 0; i < 2; ++i) {
            typename T::elem *out = (typename T::elem *)a.rows[i] + token * a.r_token[i] + head * a.r_head[i];
            const int64_t at = page_offset(page, place, a.p_page[i], a.p_place[i]) + head * a.p_head[i];
            float scale = 1.0f;
            if constexpr (IsCode<S>::value) {
                if (slot >= 0)
                    scale = a.scale[i][page_offset(page, place, a.s_page[i], a.s_place[i]) + head * a.s_head[i]];
            }
            for (uint32_t d = lane; d < a.head_dim; d += 64) {
                float x = 0.0f;
                if (slot >= 0) {
                    if constexpr (IsCode<S>::value) {
                        float four[4];
                        S::value4(((const uint8_t *)a.pages[i])[at + d], four);
                        x = four[0] * scale;
                    } else {
                        x = (float)((const typename S::elem *)a.pages[i])[at + d];
                    }
                }
                out[d] = (typename T::elem)x;
            }
        }
    }
}

// ---- launches ---------------------------------------------------------------

uint32_t blocks_for(uint64_t items, uint32_t per_block)
{
    const uint64_t b = (items + per_block - 1) / per_block;
    return (uint32_t)(b < kMaxBlocks ? b : kMaxBlocks);
}

template <class T>
hipError_t rope_pick(const RopeArgs &a, bool wide, uint32_t blocks, hipStream_t s)
{
    if (wide && a.interleaved)
        return launch(kvcache_rope_kernel<T, true, true>, blocks, 1, kThreads, a, s);
    if (wide)
        return launch(kvcache_rope_kernel<T, true, false>, blocks, 1, kThreads, a, s);
    if (a.interleaved)
        return launch(kvcache_rope_kernel<T, false, true>, blocks, 1, kThreads, a, s);
    return launch(kvcache_rope_kernel<T, false, false>, blocks, 1, kThreads, a, s);
}

template <class T, class Format>
hipError_t write_pick(const RowArgs &a, bool wide, hipStream_t s)
{
    const uint64_t rows = (uint64_t)a.tokens * a.kv_heads.d;
    const auto go = [&](void (*kernel)(const RowArgs), uint32_t lanes) {
        return launch(kernel, blocks_for(rows, kThreads / lanes), 1, kThreads, a, s);
    };
    if (!wide)
        return go(kvcache_write_any_kernel<T, Format>, 64);
    if (a.head_dim <= 64)
        return go(kvcache_write_kernel<T, Format, 8>, 8);
    if (a.head_dim <= 128)
        return go(kvcache_write_kernel<T, Format, 16>, 16);
    if (a.head_dim <= 256)
        return go(kvcache_write_kernel<T, Format, 32>, 32);
    return go(kvcache_write_kernel<T, Format, 64>, 64);
}

template <class S, class T>
hipError_t read_pick(const RowArgs &a, bool wide, hipStream_t s)
{
    const uint64_t rows = (uint64_t)a.tokens * a.kv_heads.d;
    const auto go = [&](void (*kernel)(const RowArgs), uint32_t lanes) {
        return launch(kernel, blocks_for(rows, kThreads / lanes), 1, kThreads, a, s);
    };
    if (!wide)
        return go(kvcache_read_any_kernel<S, T>, 64);
    if (a.head_dim <= 64)
        return go(kvcache_read_kernel<S, T, 8>, 8);
    if (a.head_dim <= 128)
        return go(kvcache_read_kernel<S, T, 16>, 16);
    if (a.head_dim <= 256)
        return go(kvcache_read_kernel<S, T, 32>, 32);
    return go(kvcache_read_kernel<S, T, 64>, 64);
}

template <class S>
hipError_t read_type(const RowArgs &a, uint32_t dtype, bool wide, hipStream_t s)
{
    if (dtype == KVCACHE_BF16)
        return read_pick<S, Bf16>(a, wide, s);
    if (dtype == KVCACHE_FP16)
        return read_pick<S, Fp16>(a, wide, s);
    return read_pick<S, Fp32>(a, wide, s);
}

template <class T>
hipError_t write_format(const RowArgs &a, uint32_t format, bool wide, hipStream_t s)
{
    if (format == KVCACHE_FP8)
        return write_pick<T, Fp8>(a, wide, s);
    if (format == KVCACHE_INT8)
        return write_pick<T, Int8>(a, wide, s);
    return write_pick<T, void>(a, wide, s);
}

}  // namespace

hipError_t launch_rope(const RopeArgs &args, uint32_t dtype, bool wide, hipStream_t stream)
{
    RopeArgs a = args;
    const uint32_t half = a.rot_dim / 2;
    // Angles of up to 256 pairs fit a workgroup; few tokens are spread over the CUs instead.
    const uint32_t most = half ? kThreads / half : 1;
    const uint32_t spread = (a.tokens + 511) / 512;
    a.block_tokens = most < spread ? most : spread;
    // a workgroup's items are counted in 32 bits
    while (a.block_tokens > 1 && (uint64_t)a.block_tokens * a.heads * a.head_dim >= 1ull << 30)
        a.block_tokens /= 2;
    const uint32_t blocks = blocks_for(a.tokens, a.block_tokens);
    if (dtype == KVCACHE_BF16)
        return rope_pick<Bf16>(a, wide, blocks, stream);
    if (dtype == KVCACHE_FP16)
        return rope_pick<Fp16>(a, wide, blocks, stream);
    return rope_pick<Fp32>(a, wide, blocks, stream);
}

hipError_t launch_write(const RowArgs &a, uint32_t dtype, uint32_t format, bool wide, hipStream_t stream)
{
    if (dtype == KVCACHE_BF16)
        return write_format<Bf16>(a, format, wide, stream);
    return write_format<Fp16>(a, format, wide, stream);
}

hipError_t launch_read(const RowArgs &a, uint32_t dtype, uint32_t format, bool wide, hipStream_t stream)
{
    if (format == KVCACHE_FP8)
        return read_type<Fp8>(a, dtype, wide, stream);
    if (format == KVCACHE_INT8)
        return read_type<Int8>(a, dtype, wide, stream);
    if (format == KVCACHE_BF16)
        return read_type<Bf16>(a, dtype, wide, stream);
    return read_type<Fp16>(a, dtype, wide, stream);
}

}  // namespace kvc
