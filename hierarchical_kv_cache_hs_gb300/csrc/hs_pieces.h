// What the elementwise operators share: 16-byte pieces as floats, and the quotient that
// e4m3 values are rounded from.
#pragma once

#include "hs_ops.h"

__device__ __forceinline__ float nan_max(float a, float b)  // keeps a NaN
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

template <typename T> struct Piece;  // 16 bytes of T as floats
template <> struct Piece<float> {
    static constexpr int n = 4;
    static __device__ void unpack(const uint4& v, float* f)
    {
        f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
    }
    static __device__ uint4 pack(const float* f)
    {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <> struct Piece<__nv_bfloat16> {
    static constexpr int n = 8;
    static __device__ void unpack(const uint4& v, float* f)
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    static __device__ uint4 pack(const float* f)
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Piece<__half> {
    static constexpr int n = 8;
    static __device__ void unpack(const uint4& v, float* f)
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = p.x, f[2 * i + 1] = p.y;
        }
    }
    static __device__ uint4 pack(const float* f)
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 p = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// y / scale, rounded once.  The scale's reciprocal serves its whole group: the product with it is corrected by
// its own remainder, which one fused operation gives exactly (P. Markstein, "Computation of elementary functions
// on the IBM RISC System/6000 processor", 1990).  65,536 cache rows take 31.4 us so, 8192 x 4096 with a residual
// 39.3; 41.2 and 45.3 with a division for each value; 30.9 and 39.2 with the product alone, which leaves values
// beside a border of e4m3 on its other side (5 in 10,000 of bf16 values in groups of 16).  inv 0: a scale that is
// 0 or no ordinary number.
__device__ __forceinline__ float inverse(float scale) { return scale > 1e-30f && scale < 1e30f ? 1.f / scale : 0.f; }
__device__ __forceinline__ float quotient(float y, float scale, float inv)
{
    const float q = y * inv;
    return fmaf(fmaf(-q, scale, y), inv, q);
}
__device__ __forceinline__ void quotients(float& y0, float& y1, float scale, float inv)  // of two, in paired operations
{
    asm("{\n\t.reg .b64 y, q, s, i;\n\tmov.b64 y, {%0, %1};\n\tmov.b64 s, {%2, %2};\n\tmov.b64 i, {%3, %3};\n\t"
        "mul.rn.f32x2 q, y, i;\n\tfma.rn.f32x2 y, q, s, y;\n\tfma.rn.f32x2 q, y, i, q;\n\tmov.b64 {%0, %1}, q;\n\t}"
        : "+f"(y0), "+f"(y1)
        : "f"(-scale), "f"(inv));
}
__device__ __forceinline__ float divided(float y, float scale, float inv)
{
    return inv != 0.f ? quotient(y, scale, inv) : y / (scale == 0.f ? 1.f : scale);
}

// Two 16-bit values as floats, the low half first.
template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t v)
{
    if constexpr (HsType<T>::is_bf16)
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    else
        return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// Two products in one instruction.
__device__ __forceinline__ void mul2(float& a0, float& a1, float b0, float b1)
{
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "f"(b0), "f"(b1));
}

// 32 bytes at once where they are aligned so.
__device__ __forceinline__ void load32(const void* p, bool whole, uint4 (&v)[2])
{
    if (whole) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x), "=r"(v[1].y), "=r"(v[1].z), "=r"(v[1].w)
                     : "l"(p));
    } else {
        v[0] = static_cast<const uint4*>(p)[0];
        v[1] = static_cast<const uint4*>(p)[1];
    }
}
__device__ __forceinline__ void store32(void* p, bool whole, const uint4& a, const uint4& b)
{
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y),
                     "r"(b.z), "r"(b.w)
                     : "memory");
    } else {
        static_cast<uint4*>(p)[0] = a;
        static_cast<uint4*>(p)[1] = b;
    }
}

// Threads of a cache row, 16 channels each: wide pieces of the row in either form, and of its values.
constexpr int kRowThreads = HS_ROW_DIM / 16;
