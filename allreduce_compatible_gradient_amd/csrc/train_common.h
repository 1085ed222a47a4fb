// train_common.h -- what the sources of libgq_train.so share: argument
// checks and errors on the host; loads, stores, Philox and the 8-bit group
// format on the device.
#pragma once

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "gq_train.h"

namespace gqt {

// ---------------------------------------------------------------------------
// Host

// Sets the calling thread's error text and returns `status`.
__attribute__((visibility("hidden"), format(printf, 2, 3))) int32_t fail(int32_t status,
                                                                         const char *fmt, ...);
__attribute__((visibility("hidden"))) int32_t ok();
// GQ_OK, or GQ_ERR_DEVICE with the name of the kernel whose launch failed.
__attribute__((visibility("hidden"))) int32_t check_launch(const char *kernel);

// A copy's pointers and alignment, and its rounding where it is written.
__attribute__((visibility("hidden"))) int32_t check_act8(const char *name, const gqt_act8 *a,
                                                         int64_t rows, bool written);

#define GQT_TRY(expr)                      \
    do {                                   \
        const int32_t try_status = (expr); \
        if (try_status != GQ_OK)           \
            return try_status;             \
    } while (0)

constexpr int64_t kMaxGroups = (int64_t)1 << 29; // rows ceil(d / 32): 8-column chunks fit 31 bits

inline int64_t elem_bytes(int32_t dtype) { return dtype == GQ_IN_F32 ? 4 : 2; }
inline bool dtype_ok(int32_t dtype) { return dtype == GQ_IN_F32 || dtype == GQ_IN_BF16; }
inline bool aligned_to(const void *p, int64_t a) { return ((uintptr_t)p & (uintptr_t)(a - 1)) == 0; }
inline int64_t groups_of(int64_t d) { return (d + 31) / 32; }
inline int64_t align256(int64_t b) { return (b + 255) & ~(int64_t)255; }

// ---------------------------------------------------------------------------
// Device

using bf16 = __bf16;
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// Vectors at an element's own alignment: global memory takes wide accesses
// at any byte address on this part, so rows of odd length keep 16-byte loads.
typedef u32x4 u32x4_e2 __attribute__((aligned(2)));
typedef u32x4 u32x4_e4 __attribute__((aligned(4)));

__device__ __forceinline__ float bits_f32(uint32_t u) { return __uint_as_float(u); }

// Eight consecutive elements at p as floats; those from n on read as 0.
__device__ __forceinline__ void load8(const bf16 *p, int n, float (&v)[8])
{
    if (n >= 8) {
        const u32x4 w = *reinterpret_cast<const u32x4_e2 *>(p);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = bits_f32(w[k] << 16);
            v[2 * k + 1] = bits_f32(w[k] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = k < n ? (float)p[k] : 0.0f;
    }
}

__device__ __forceinline__ void load8(const float *p, int n, float (&v)[8])
{
    if (n >= 8) {
        const u32x4 a = *reinterpret_cast<const u32x4_e4 *>(p);
        const u32x4 b = *reinterpret_cast<const u32x4_e4 *>(p + 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = bits_f32(a[k]);
            v[4 + k] = bits_f32(b[k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = k < n ? p[k] : 0.0f;
    }
}

// Rounds v to T in place (the value that a later reader of the output sees)
// and stores the first n.
__device__ __forceinline__ void store8(bf16 *p, int n, float (&v)[8])
{
    bf16x8 h;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        h[k] = (bf16)v[k];
        v[k] = (float)h[k];
    }
    if (n >= 8) {
        *reinterpret_cast<u32x4_e2 *>(p) = __builtin_bit_cast(u32x4, h);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n)
                p[k] = h[k];
    }
}

__device__ __forceinline__ void store8(float *p, int n, float (&v)[8])
{
    if (n >= 8) {
        u32x4 a, b;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            a[k] = __float_as_uint(v[k]);
            b[k] = __float_as_uint(v[4 + k]);
        }
        *reinterpret_cast<u32x4_e4 *>(p) = a;
        *reinterpret_cast<u32x4_e4 *>(p + 4) = b;
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n)
                p[k] = v[k];
    }
}

// Philox4x32-10 (Salmon et al., SC'11); the same generator and key schedule
// as the gradient quantizer's.
__device__ __forceinline__ uint4 philox10(uint4 c, uint32_t k0, uint32_t k1)
{
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = (uint64_t)c.x * 0xD2511F53u;
        const uint64_t p1 = (uint64_t)c.z * 0xCD9E8D57u;
        // v_bitop3_b32 with truth table 0x96 is a three-input xor
        c = make_uint4(__builtin_amdgcn_bitop3_b32((uint32_t)(p1 >> 32), c.y, k0, 0x96),
                       (uint32_t)p1,
                       __builtin_amdgcn_bitop3_b32((uint32_t)(p0 >> 32), c.w, k1, 0x96),
                       (uint32_t)p0);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return c;
}

__device__ __forceinline__ uint32_t half16(const uint4 &w, int k)
{
    const uint32_t word = (k >> 1) == 0 ? w.x : (k >> 1) == 1 ? w.y : (k >> 1) == 2 ? w.z : w.w;
    return (k & 1) ? (word >> 16) : (word & 0xFFFFu);
}

// An 8-bit copy as the kernels see it.
enum { kKeepNone = 0, kKeepNearest = 1, kKeepRandom = 2 };
struct Act8 {
    int8_t *codes;
    uint8_t *exps;
    int64_t pitch;  // bytes of a row of codes
    int32_t groups; // bytes of a row of exps
    int32_t keep;
    uint32_t k0, k1;
};

inline Act8 act8_view(const gqt_act8 *a, int64_t d)
{
    Act8 v{nullptr, nullptr, 32 * groups_of(d), (int32_t)groups_of(d), kKeepNone, 0, 0};
    if (a) {
        v.codes = (int8_t *)a->codes;
        v.exps = (uint8_t *)a->exps;
        v.keep = a->rounding == GQT_ROUND_RANDOM ? kKeepRandom : kKeepNearest;
        v.k0 = (uint32_t)a->seed;
        v.k1 = (uint32_t)(a->seed >> 32);
    }
    return v;
}

// max over the four lanes of a quad
__device__ __forceinline__ uint32_t quad_max(uint32_t m)
{
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true)); // lane ^ 1
    return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true)); // lane ^ 2
}

// Writes the codes of the eight values at (row, col), col a multiple of 8;
// the four lanes of a quad hold one group's four parts, all of them active,
// and columns past d hold 0.  Scaling by a power of two is exact, so the
// rounding sees x itself.
__device__ __forceinline__ void keep8(const Act8 &a, int64_t row, int32_t col, const float (&v)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        m = max(m, __float_as_uint(v[k]) & 0x7FFFFFFFu);
    m = quad_max(m);
    if (col >= a.pitch)
        return;
    // a = f 2^k with 1 <= f < 2: E = k - 6, one more where f > 127/64, whose
    // fraction bits are 0x7E0000
    const bool finite = m < 0x7F800000u;
    const uint32_t e = finite ? max((m + 0x1FFFFu) >> 23, 7u) - 6u : 255u;
    const float inv = bits_f32((254u - (finite ? e : 127u)) << 23);
    const int top = e == 249u ? 63 : 127;
    int q[8];
    if (a.keep == kKeepNearest) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            q[k] = min(max((int)rintf(finite ? v[k] * inv : 0.0f), -top), top);
    } else {
        // S = floor(t 2^16) + (0xFFFF - h) for the high half h of u carries
        // into bit 16 exactly when h is below the high half of frac 2^32; a
        // tie leaves 16 ones and takes the low half, from the second draw.
        const uint32_t blk = (uint32_t)col >> 3, r0 = (uint32_t)row;
        const uint4 A = philox10(make_uint4(blk, 0u, r0, 0u), a.k0, a.k1);
        uint32_t S[8];
        bool tie = false;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float t = finite ? fabsf(v[k]) * inv : 0.0f;
            S[k] = (uint32_t)(t * 0x1p16f) + (0xFFFFu - half16(A, k));
            tie |= (S[k] & 0xFFFFu) == 0xFFFFu;
        }
        if (tie) {
            const uint4 B = philox10(make_uint4(blk, 0u, r0, 1u), a.k0, a.k1);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float t = finite ? fabsf(v[k]) * inv : 0.0f;
                const uint32_t F = (uint32_t)((t - floorf(t)) * 0x1p32f);
                if ((S[k] & 0xFFFFu) == 0xFFFFu && half16(B, k) < (F & 0xFFFFu))
                    S[k] += 1u;
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int mag = min((int)(S[k] >> 16), top);
            q[k] = __float_as_uint(v[k]) >> 31 ? -mag : mag;
        }
    }
    u32x2 w;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        w[h] = (uint32_t)(q[4 * h] & 0xFF) | (uint32_t)(q[4 * h + 1] & 0xFF) << 8 |
               (uint32_t)(q[4 * h + 2] & 0xFF) << 16 | (uint32_t)q[4 * h + 3] << 24;
    *reinterpret_cast<u32x2 *>(a.codes + row * a.pitch + col) = w;
    if ((col & 24) == 0)
        a.exps[row * a.groups + (col >> 5)] = (uint8_t)e;
}

// 2^E of an exponent byte; NaN for 255.
__device__ __forceinline__ float step_of(uint32_t e)
{
    return bits_f32(e == 255u ? 0x7FC00000u : e << 23);
}

// The eight values at (row, col), col a multiple of 8 and below the pitch.
__device__ __forceinline__ void restore8(const Act8 &a, int64_t row, int32_t col, float (&v)[8])
{
    const u32x2 w = *reinterpret_cast<const u32x2 *>(a.codes + row * a.pitch + col);
    const float step = step_of(a.exps[row * a.groups + (col >> 5)]);
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[k] = (float)((int)(w[k >> 2] << (24 - 8 * (k & 3))) >> 24) * step;
}

} // namespace gqt
