// The rotation of channels by a token's position: its angle, sine and cosine.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

// A frequency (radians a position) in turns a position, modulo 1, as a fixed-point number of 64 fractional bits:
// its 24-bit significand times 2^64 / 2 pi, shifted by its exponent.  Off by less than 2^-63 below 2^1, and twice
// that for each further power of two.
struct HsTurn {
    uint64_t turns;
    bool finite;
};
__device__ __forceinline__ HsTurn hs_turn(float freq)
{
    const uint32_t bits = __float_as_uint(freq);
    const int ex = (int)(bits >> 23 & 255);
    const uint64_t m = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);  // freq = m * 2^(ex - 150), a subnormal with ex 1
    constexpr uint64_t kTurn = 0x28BE60DB9391054Aull;               // 2^64 / 2 pi
    const uint64_t low = m * (uint32_t)kTurn, high = m * (uint32_t)(kTurn >> 32) + (low >> 32);
    const int down = 150 - (ex ? ex : 1);  // (high * 2^32 + low's last 32 bits) >> down, modulo 2^64
    uint64_t turns;
    if (down <= 0)
        turns = down <= -64 ? 0 : (m * kTurn) << -down;
    else if (down < 32)
        turns = (high << (32 - down)) | ((uint32_t)low >> down);
    else
        turns = down - 32 < 64 ? high >> (down - 32) : 0;
    return {bits >> 31 ? 0 - turns : turns, ex != 255};
}

__device__ __forceinline__ float2 fma2(const float2& a, const float2& b, const float2& c)  // two operations in one instruction
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// cos and sin of position * freq.  Only the fraction of a turn counts, so the product is taken in integers modulo
// 2^64 (of which the upper half is kept): exact to 2^-32 of a turn for frequencies of 1 and less at any int32
// position, where the fp32 product alone is off by 2^-7 radians at position 131,072.  In 64-bit floats the products
// of 65,536 tokens' 32 pairs would take longer than their rows' way through memory: this chip has few such units.
// The integer also gives the nearest quarter of a turn exactly, and t = what is left in eighths, in [-1, 1]; then
//   sin(a t) = 2 J1(a) T1(t) - 2 J3(a) T3(t) + ...,  cos(a t) = J0(a) - 2 J2(a) T2(t) + ...,  a = pi / 4
// (the Jacobi-Anger series: Bessel functions and Chebyshev polynomials), cut at t^7 and t^8 and gathered by powers: off
// by less than a step of fp32 (5e-8 and 1e-8 of the value) before the evaluation's own roundings, which add two.  The
// library's sincospif does the reduction again: 32.6 us against 34.1 where sines count most (65,536 tokens x 2 heads),
// 24.3 against 24.5 for 65,536 rows.
// A frequency that is not finite gives NaN.
__device__ __forceinline__ float2 hs_rotation(int position, const HsTurn& f)
{
    const uint32_t angle = (uint32_t)((f.turns * (uint64_t)(int64_t)position) >> 32);
    const uint32_t quarter = angle + (1u << 29);  // in its upper 2 bits
    const float t = (float)(int32_t)(angle << 2) * 0x1p-31f, z = t * t;
    const float2 z2 = make_float2(z, z);
    float2 p = make_float2(-3.5877150e-5f, fmaf(3.5298042e-6f, z, -3.2593860e-4f));  // sin(a t) / t, cos(a t)
    p = fma2(p, z2, make_float2(2.4898718e-3f, 1.5854325e-2f));
    p = fma2(p, z2, make_float2(-8.0745367e-2f, -3.0842514e-1f));
    p = fma2(p, z2, make_float2(7.8539815e-1f, 1.0f));
    p.x *= t;
    const bool odd = quarter >> 30 & 1;
    const uint32_t c = __float_as_uint(odd ? p.x : p.y), s = __float_as_uint(odd ? p.y : p.x);
    float2 r = make_float2(__uint_as_float(c ^ ((quarter + (1u << 30)) & 0x80000000u)), __uint_as_float(s ^ (quarter & 0x80000000u)));
    if (!f.finite) r.x = r.y = __int_as_float(0x7fffffff);
    return r;
}
