// rotary.cuh -- angles of rotary positions (internal to libgdn_decode.so).
#pragma once

#include <cstdint>

namespace gdn {

// A frequency in turns a position, as a 64-bit fraction of a turn: f / (2 pi) mod 1 times 2^64, by integer arithmetic
// (fp64 runs at two operations a clock and SM). With f = m 2^(E - 63), 2^63 <= m < 2^64, and C = 2^66 / (2 pi), the high
// half h of m C gives f / (2 pi) = h 2^(E - 65).
__device__ __forceinline__ uint64_t rotary_turns(double f)
{
    const uint64_t bits = (uint64_t)__double_as_longlong(f);
    const int e = (int)(bits >> 52) & 0x7FF;
    if (e == 0) return 0;                                          // zero (or below 2^-1022)
    const uint64_t m = ((bits & 0xFFFFFFFFFFFFFull) | 0x10000000000000ull) << 11;
    const uint64_t h = __umul64hi(m, 0xA2F9836E4E44152Aull);
    const int shift = e - 1023 - 1;                                // F = h 2^(E - 1) mod 2^64
    const uint64_t F = shift >= 64 || shift <= -64 ? 0 : shift >= 0 ? h << shift : h >> -shift;
    return (bits >> 63) ? 0 - F : F;
}

// cos and sin of position times frequency: the product modulo a turn is the product modulo 2^64, its top 32 bits
// the angle in [-1/2, 1/2) turns, which fp32 then rounds by up to 2^-25 half turns (9.4e-8 radians).
__device__ __forceinline__ void rotary_cos_sin(int position, uint64_t turns, float &c, float &s)
{
    const uint64_t phase = (uint64_t)(int64_t)position * turns;
    sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &s, &c);      // 2^-31: half turns
}

}  // namespace gdn
