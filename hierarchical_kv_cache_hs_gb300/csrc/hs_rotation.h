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

// cos and sin of position * freq.  Only the fraction of a turn counts, so the product is taken in integers modulo
// 2^64 (of which the upper half is kept): exact to 2^-32 of a turn for frequencies of 1 and less at any int32
// position, where the fp32 product alone is off by 2^-7 radians at position 131,072.  In 64-bit floats the products
// of 65,536 tokens' 32 pairs would take longer than their rows' way through memory: this chip has few such units.
// A frequency that is not finite gives NaN.
__device__ __forceinline__ float2 hs_rotation(int position, const HsTurn& f)
{
    const uint64_t angle = f.turns * (uint64_t)(int64_t)position;
    const float half_turns = (float)(int32_t)(angle >> 32) * 0x1p-31f;  // [-1, 1]
    float2 r;
    sincospif(half_turns, &r.y, &r.x);
    if (!f.finite) r.x = r.y = __int_as_float(0x7fffffff);
    return r;
}
