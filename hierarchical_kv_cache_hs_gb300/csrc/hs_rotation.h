// The rotation of channels by a token's position: its angle, sine and cosine.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

// cos and sin of position * freq (radians).  The angle in turns is position * freq / 2 pi, and only its fraction
// counts, so it is taken in integers modulo 2^64: freq / 2 pi as a fixed-point number of 64 fractional bits (freq's
// 24-bit significand times 2^64 / 2 pi, shifted by its exponent; off by less than 2^-63 below 2^1, and by a bit more
// for each further power of two, 2^-48 of a turn at 2^16), then its product with the position.  That is exact to
// 2^-32 of a turn for frequencies of 1 and less at any int32 position; the fp32 product alone is off by 2^-7 radians
// at position 131,072.  In 64-bit floats the products of 65,536 tokens' 32 pairs would take longer than the rows'
// way through memory (this chip has few such units); the integer steps are about 15 a pair.  A frequency that is
// not finite gives NaN.
__device__ __forceinline__ float2 hs_rotation(int position, float freq)
{
    const uint32_t bits = __float_as_uint(freq);
    const int ex = (int)(bits >> 23 & 255);
    const uint64_t m = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);  // freq = m * 2^(ex - 150), a subnormal with ex 1
    // m * 2^64 / 2 pi as hi * 2^32 + lo, then times 2^(ex - 150)
    constexpr uint64_t kTurn = 0x28BE60DB9391054Aull;  // 2^64 / 2 pi
    const uint64_t low = m * (uint32_t)kTurn, high = m * (uint32_t)(kTurn >> 32) + (low >> 32);
    const int down = 150 - (ex ? ex : 1);              // at least -104
    uint64_t turns;                                    // (high * 2^32 + low's last 32 bits) >> down, modulo 2^64
    if (down <= 0)
        turns = down <= -64 ? 0 : (m * kTurn) << -down;
    else if (down < 32)
        turns = (high << (32 - down)) | ((uint32_t)low >> down);
    else
        turns = down - 32 < 64 ? high >> (down - 32) : 0;
    if (bits >> 31) turns = 0 - turns;
    const uint64_t angle = turns * (uint64_t)(int64_t)position;
    const float half_turns = (float)(int32_t)(angle >> 32) * 0x1p-31f;  // [-1, 1]
    float2 r;
    sincospif(half_turns, &r.y, &r.x);
    if (ex == 255) r.x = r.y = __int_as_float(0x7fffffff);
    return r;
}
