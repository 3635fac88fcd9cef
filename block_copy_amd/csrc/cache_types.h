// cache_types.h -- element types of the cache kernels: pieces of 8 values,
// their conversion from and to 32 bits, and the 8-bit formats.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kvc {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// A row type: its element, a pair, and eight of them in 16 bytes.
struct Bf16 {
    typedef __bf16 elem;
    typedef bf16x2 pair;
    typedef bf16x8 eight;
    typedef u32x4 piece;
    // exponent all ones, in both halves of a word
    static constexpr uint32_t kExponent = 0x7f80u;
    static __device__ __forceinline__ f32x16 mfma32(eight a, eight b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x4 mfma16(eight a, eight b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
struct Fp16 {
    typedef _Float16 elem;
    typedef f16x2 pair;
    typedef f16x8 eight;
    typedef u32x4 piece;
    static constexpr uint32_t kExponent = 0x7c00u;
    static __device__ __forceinline__ f32x16 mfma32(eight a, eight b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x4 mfma16(eight a, eight b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};
struct Fp32 {
    typedef float elem;
    struct piece {
        f32x4 lo, hi;
    };
};

// Two floats as a pair of 16-bit values, rounded to nearest even.
template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    f32x2 f;
    f.x = a;
    f.y = b;
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, typename T::pair));
}

template <class T>
__device__ __forceinline__ void unpack8(const u32x4 p, float *f)
{
    const typename T::eight e = __builtin_bit_cast(typename T::eight, p);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = (float)e[i];
}
template <class T>
__device__ __forceinline__ void unpack8(const Fp32::piece p, float *f)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[i] = p.lo[i];
        f[4 + i] = p.hi[i];
    }
}

template <class T>
__device__ __forceinline__ typename T::piece pack8(const float *f)
{
    u32x4 p;
    p.x = pack2<T>(f[0], f[1]);
    p.y = pack2<T>(f[2], f[3]);
    p.z = pack2<T>(f[4], f[5]);
    p.w = pack2<T>(f[6], f[7]);
    return p;
}
template <>
__device__ __forceinline__ Fp32::piece pack8<Fp32>(const float *f)
{
    Fp32::piece p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        p.lo[i] = f[i];
        p.hi[i] = f[4 + i];
    }
    return p;
}

// The 8-bit formats.  q: the largest code's value.
struct Fp8 {
    static constexpr float kQ = 448.0f;
    static __device__ __forceinline__ uint32_t code4(float a, float b, float c, float d)
    {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
        return (uint32_t)w;
    }
    static __device__ __forceinline__ void value4(uint32_t w, float *f)
    {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
        f[0] = lo.x;
        f[1] = lo.y;
        f[2] = hi.x;
        f[3] = hi.y;
    }
};
struct Int8 {
    static constexpr float kQ = 127.0f;
    static __device__ __forceinline__ uint32_t code4(float a, float b, float c, float d)
    {
        const int x = (int)__builtin_rintf(a), y = (int)__builtin_rintf(b);
        const int z = (int)__builtin_rintf(c), w = (int)__builtin_rintf(d);
        return (uint32_t)(x & 255) | (uint32_t)(y & 255) << 8 | (uint32_t)(z & 255) << 16 |
               (uint32_t)w << 24;
    }
    static __device__ __forceinline__ void value4(uint32_t w, float *f)
    {
        f[0] = (float)(int8_t)(w & 255);
        f[1] = (float)(int8_t)(w >> 8 & 255);
        f[2] = (float)(int8_t)(w >> 16 & 255);
        f[3] = (float)(int8_t)(w >> 24);
    }
};

// Eight codes as eight 16-bit values: exact in both types (an int8 code needs
// 7 bits, an e4m3 code 4 bits and exponents -9 .. 8).
template <class T, class F>
struct Widen;
template <class T>
struct Widen<T, Int8> {
    static __device__ __forceinline__ u32x4 eight(u32x2 c)
    {
        float f[8];
        Int8::value4(c.x, f);
        Int8::value4(c.y, f + 4);
        return pack8<T>(f);
    }
};
template <>
struct Widen<Bf16, Fp8> {
    static __device__ __forceinline__ u32x4 eight(u32x2 c)
    {
        u32x4 p;
        p.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.x, 1.0f, false));
        p.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.x, 1.0f, true));
        p.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.y, 1.0f, false));
        p.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.y, 1.0f, true));
        return p;
    }
};
template <>
struct Widen<Fp16, Fp8> {
    static __device__ __forceinline__ u32x4 eight(u32x2 c)
    {
        u32x4 p;
        p.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c.x, 1.0f, false));
        p.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c.x, 1.0f, true));
        p.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c.y, 1.0f, false));
        p.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c.y, 1.0f, true));
        return p;
    }
};

// The larger of each half of two words, as unsigned 16-bit numbers: without
// their signs, 16-bit floats order like their bits (NaN above infinity).
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b)
{
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                  __builtin_bit_cast(u16x2, b)));
}

// A piece past the caches' usual order: for data that is not used again soon.
template <class P>
__device__ __forceinline__ P load_once(const P *p)
{
    return __builtin_nontemporal_load(p);
}
__device__ __forceinline__ Fp32::piece load_once(const Fp32::piece *p)
{
    Fp32::piece r;
    r.lo = __builtin_nontemporal_load(&p->lo);
    r.hi = __builtin_nontemporal_load(&p->hi);
    return r;
}
__device__ __forceinline__ void store_once(u32x4 *to, u32x4 p)
{
    __builtin_nontemporal_store(p, to);
}
__device__ __forceinline__ void store_once(Fp32::piece *to, const Fp32::piece &p)
{
    __builtin_nontemporal_store(p.lo, &to->lo);
    __builtin_nontemporal_store(p.hi, &to->hi);
}

__device__ __forceinline__ void set_status(uint32_t *status, uint32_t bit)
{
    if (status)
        atomicOr(status, bit);
}

}  // namespace kvc
