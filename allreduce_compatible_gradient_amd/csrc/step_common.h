// step_common.h -- what the sources of libgq_step.so share: argument checks
// on the host; the 8-bit floating-point formats of include/gq_step.h on the
// device.
#pragma once

#include "gq_step.h"
#include "train_common.h"

namespace gqt {

// ---------------------------------------------------------------------------
// Host

constexpr int64_t kMaxSide = (int64_t)1 << 22;
constexpr int64_t kMaxRows = (int64_t)1 << 31;
constexpr int64_t kMaxBlocks = (int64_t)1 << 27; // of 128: a launch has fewer than 2^32 threads

inline int64_t blocks_of(int64_t d) { return (d + 127) / 128; }
inline int64_t fp8_pitch(int64_t d) { return 128 * blocks_of(d); }
inline int64_t exp_pitch(int64_t rows) { return (rows + 15) / 16 * 16; }

// ---------------------------------------------------------------------------
// Device

// max over a row of 16 lanes
__device__ __forceinline__ uint32_t row16_max(uint32_t m)
{
    m = quad_max(m);
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x141, 0xF, 0xF, true)); // half mirror
    return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x140, 0xF, 0xF, true)); // mirror
}

__device__ __forceinline__ uint32_t abs_bits(const float (&v)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        m = max(m, __float_as_uint(v[k]) & 0x7FFFFFFFu);
    return m;
}

// A block's byte E + 127 from the bits m of its largest |x| = f 2^k, 1 <= f <
// 2: e4m3 reaches 448 = 1.75 2^8, so E = k - 8, one more where the fraction
// bits exceed those of 1.75.  The second moment's reach 61440 = 1.875 2^15.
__device__ __forceinline__ uint32_t e4m3_exponent(uint32_t m)
{
    return m < 0x7F800000u ? max((m + 0x1FFFFFu) >> 23, 18u) - 8u : 255u;
}
__device__ __forceinline__ uint32_t e5m3_exponent(uint32_t m)
{
    return m < 0x7F800000u ? max((m + 0x0FFFFFu) >> 23, 34u) - 15u : 255u;
}
constexpr uint32_t kHighestE4m3 = 247; // the byte where 256 2^E has no float
constexpr uint32_t kHighestE5m3 = 240; // and where 32768 2^E has none

// 2^-E of a byte (not 255); exact: 2^-120 to 2^117.
__device__ __forceinline__ float inverse_step(uint32_t e) { return bits_f32((254u - e) << 23); }

// Four e4m3 codes of t (|t| <= 448), to nearest with ties to even.
__device__ __forceinline__ uint32_t e4m3_nearest4(float a, float b, float c, float d)
{
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// The codes of eight values, to nearest.
__device__ __forceinline__ u32x2 e4m3_nearest8(const float (&v)[8], uint32_t e)
{
    const float inv = inverse_step(e);
    float t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        t[k] = v[k] * inv;
        if (e == kHighestE4m3)
            t[k] = fminf(fmaxf(t[k], -240.0f), 240.0f);
    }
    return u32x2{e4m3_nearest4(t[0], t[1], t[2], t[3]), e4m3_nearest4(t[4], t[5], t[6], t[7])};
}

// Random rounding of x >= 0 whose code is the leading bits of x 2^scale, which
// may be subnormal, above 20 that are rounded off: u enters above a half of
// their last place.  The code is byte 2 of the result.
__device__ __forceinline__ uint32_t random_code(float x, int scale, uint32_t u)
{
    return ((__float_as_uint(ldexpf(x, scale)) + 8u) >> 4) + u;
}

// Byte 2 of each of four, in their order.
__device__ __forceinline__ uint32_t third_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return perm(perm(d, c, 0x0C0C0602u), perm(b, a, 0x0C0C0602u), 0x05040100u);
}

// Bytes above `top` become it.  For the exponents whose upper numbers have no
// float, so hardly ever.
__device__ __forceinline__ uint32_t cap_bytes(uint32_t w, uint32_t top)
{
    uint32_t r = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        r |= min(w >> (8 * k) & 0xFFu, top) << (8 * k);
    return r;
}

// The codes of eight values at random, with their signs.
__device__ __forceinline__ u32x2 e4m3_random8(const float (&v)[8], uint32_t e, const uint4 &draw)
{
    const int scale = 7 - (int)e; // 2^-120 x 2^-E: the least normal number, 2^-6, becomes 2^-126
    u32x2 w;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t t[4], b[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            t[k] = random_code(fabsf(v[4 * h + k]), scale, half16(draw, 4 * h + k));
            b[k] = __float_as_uint(v[4 * h + k]);
        }
        w[h] = third_bytes(t[0], t[1], t[2], t[3]);
        if (e == kHighestE4m3)
            w[h] = cap_bytes(w[h], 0x77u);
        const uint32_t top = perm(perm(b[3], b[2], 0x0C0C0703u), perm(b[1], b[0], 0x0C0C0703u),
                                  0x05040100u);
        w[h] |= top & 0x80808080u;
    }
    return w;
}

// Those of eight second moments (v >= 0).
__device__ __forceinline__ u32x2 e5m3_random8(const float (&v)[8], uint32_t e, const uint4 &draw)
{
    const int scale = 16 - (int)e; // 2^-111 x 2^-E: 2^-15 becomes 2^-126
    u32x2 w;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t t[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            t[k] = random_code(v[4 * h + k], scale, half16(draw, 4 * h + k));
        w[h] = third_bytes(t[0], t[1], t[2], t[3]);
        if (e == kHighestE5m3)
            w[h] = cap_bytes(w[h], 0xF7u);
    }
    return w;
}

// The numbers that eight codes are, times their step.
__device__ __forceinline__ void e4m3_values(const u32x2 w, float step, float (&v)[8])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], false);
        const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], true);
        v[4 * h] = lo[0] * step;
        v[4 * h + 1] = lo[1] * step;
        v[4 * h + 2] = hi[0] * step;
        v[4 * h + 3] = hi[1] * step;
    }
}
// A second moment's code as a float 2^111 times smaller than its number: the
// leading bits, subnormal below c = 8.
__device__ __forceinline__ float e5m3_small(const u32x2 w, int k)
{
    return bits_f32((w[k >> 2] >> (8 * (k & 3)) & 0xFFu) << 20);
}
__device__ __forceinline__ void e5m3_values(const u32x2 w, float step, float (&v)[8])
{
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[k] = e5m3_small(w, k) * 0x1p111f * step;
}

} // namespace gqt
