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

constexpr int64_t kMaxGroups = (int64_t)1 << 29;  // rows ceil(d / 32): 8-column chunks fit 31 bits
constexpr int64_t kMaxColumns = (int64_t)1 << 27; // a launch over columns stays below 2^32 threads

inline int64_t elem_bytes(int32_t dtype) { return dtype == GQ_IN_F32 ? 4 : 2; }
inline bool dtype_ok(int32_t dtype) { return dtype == GQ_IN_F32 || dtype == GQ_IN_BF16; }
inline bool aligned_to(const void *p, int64_t a) { return ((uintptr_t)p & (uintptr_t)(a - 1)) == 0; }
inline int64_t groups_of(int64_t d) { return (d + 31) / 32; }

// Division of a 31-bit number by an invariant one: q = n m >> s.
struct FastDiv {
    uint32_t d, m, s;
};
inline FastDiv fast_div(uint32_t d)
{
    FastDiv f{d, 0, 31};
    while (((uint64_t)1 << (f.s - 31)) < d)
        ++f.s;
    f.m = (uint32_t)((((uint64_t)1 << f.s) / d) + 1);
    return f;
}

// ---------------------------------------------------------------------------
// Device

__device__ __forceinline__ uint32_t divide(uint32_t n, const FastDiv &f)
{
    return (uint32_t)(((uint64_t)n * f.m) >> f.s);
}

using bf16 = __bf16;
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// Vectors at an element's own alignment: global memory takes wide accesses
// at any byte address on this part, so rows of odd length keep 16-byte loads.
typedef u32x4 u32x4_e2 __attribute__((aligned(2)));
typedef u32x4 u32x4_e4 __attribute__((aligned(4)));

__device__ __forceinline__ float bits_f32(uint32_t u) { return __uint_as_float(u); }

// Eight consecutive elements as loaded, and as floats.
template <typename T>
struct Raw8 {
    u32x4 w[sizeof(T) / 2];
};
__device__ __forceinline__ void load_words(const bf16 *p, Raw8<bf16> &r)
{
    r.w[0] = *reinterpret_cast<const u32x4_e2 *>(p);
}
__device__ __forceinline__ void load_words(const float *p, Raw8<float> &r)
{
    r.w[0] = *reinterpret_cast<const u32x4_e4 *>(p);
    r.w[1] = *reinterpret_cast<const u32x4_e4 *>(p + 4);
}
__device__ __forceinline__ void unpack(const Raw8<bf16> &r, float (&v)[8])
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[2 * k] = bits_f32(r.w[0][k] << 16);
        v[2 * k + 1] = bits_f32(r.w[0][k] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(const Raw8<float> &r, float (&v)[8])
{
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[k] = bits_f32(r.w[k / 4][k % 4]);
}

// One element towards the front, 0 behind.
__device__ __forceinline__ void shift_one(Raw8<bf16> &r)
{
#pragma unroll
    for (int k = 0; k < 3; ++k)
        r.w[0][k] = __builtin_amdgcn_alignbit(r.w[0][k + 1], r.w[0][k], 16);
    r.w[0][3] >>= 16;
}
__device__ __forceinline__ void shift_one(Raw8<float> &r)
{
#pragma unroll
    for (int k = 0; k < 7; ++k)
        r.w[k / 4][k % 4] = r.w[(k + 1) / 4][(k + 1) % 4];
    r.w[1][3] = 0;
}
__device__ __forceinline__ uint32_t bits_of(const bf16 *p) { return *(const uint16_t *)p; }
__device__ __forceinline__ uint32_t bits_of(const float *p) { return __float_as_uint(*p); }

// The eight columns from col on of a row of d, in two halves, so that a loop
// can load a row ahead: one unconditional load, which for the columns next
// to the row's end takes its last eight; then those moved into place, with 0
// past the end.
template <typename T>
__device__ __forceinline__ void load_ahead(const T *row, int32_t col, int32_t d, Raw8<T> &r)
{
    if (d >= 8) // uniform
        load_words(row + min(col, d - 8), r);
}
template <typename T>
__device__ __forceinline__ void settle(const T *row, int32_t col, int32_t d, Raw8<T> &r)
{
    constexpr int kPer = 4 / sizeof(T); // elements a word
    if (col + 8 <= d)
        return;
    if (d < 8) {
#pragma unroll
        for (int k = 0; k < 8 / kPer; ++k) {
            uint32_t w = 0;
#pragma unroll
            for (int h = 0; h < kPer; ++h)
                if (col + kPer * k + h < d)
                    w |= bits_of(row + col + kPer * k + h) << (16 * h);
            r.w[k / 4][k % 4] = w;
        }
        return;
    }
    for (int at = max(d - col, 0); at < 8; ++at)
        shift_one(r);
}
template <typename T>
__device__ __forceinline__ void load8(const T *row, int32_t col, int32_t d, float (&v)[8])
{
    Raw8<T> r;
    load_ahead(row, col, d, r);
    settle(row, col, d, r);
    unpack(r, v);
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

// An 8-bit copy as the kernels see it.  Eight columns are a chunk: chunk i of
// the whole copy has its codes at 8 i and its exponent at i / 4.
enum { kKeepNone = 0, kKeepNearest = 1, kKeepRandom = 2 };
struct Act8 {
    int8_t *codes;
    uint8_t *exps;
    int64_t pitch;  // bytes of a row of codes
    int32_t groups; // bytes of a row of exps
    int32_t keep;
    uint32_t k0, k1;

    __device__ __forceinline__ int64_t chunk(int64_t row, int32_t col) const
    {
        return row * (pitch >> 3) + (col >> 3);
    }
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

// perm: byte s of the result is byte sel[s] of (hi, lo), lo's being 0 to 3;
// 9 and 11 give lo's and hi's sign (the top bit of byte 3) eight times.
__device__ __forceinline__ uint32_t perm(uint32_t hi, uint32_t lo, uint32_t sel)
{
    return __builtin_amdgcn_perm(hi, lo, sel);
}

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b)
{
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                  __builtin_bit_cast(u16x2, b)));
}
__device__ __forceinline__ uint32_t pk_min_u16(uint32_t a, uint32_t b)
{
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(u16x2, a),
                                                                  __builtin_bit_cast(u16x2, b)));
}
__device__ __forceinline__ uint32_t pk_sub_u16(uint32_t a, uint32_t b)
{
    return __builtin_bit_cast(uint32_t,
                              (u16x2)(__builtin_bit_cast(u16x2, a) - __builtin_bit_cast(u16x2, b)));
}

// Writes the codes of the eight values at (row, col), col a multiple of 8 and
// `at` their chunk; the four lanes of a quad hold one group's four parts, all
// of them active, and columns past d hold 0.  Scaling by a power of two is
// exact, so the rounding sees x itself.
__device__ __forceinline__ void keep8(const Act8 &a, int64_t row, int32_t col, int64_t at,
                                      const float (&v)[8])
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
    const bool highest = e == 249u; // where 64 2^E has no float
    u32x2 w;
    if (a.keep == kKeepNearest) {
        // Adding 1.5 2^23 rounds the scaled value to an integer (ties to
        // even) and leaves it in the low byte.
        const float inv = bits_f32((254u - e) << 23);
        uint32_t q[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float f = fmaf(v[k], inv, 0x1.8p23f);
            if (highest)
                f = fminf(fmaxf(f, 0x1.8p23f - 63.0f), 0x1.8p23f + 63.0f);
            q[k] = __float_as_uint(f);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            w[h] = perm(perm(q[4 * h + 3], q[4 * h + 2], 0x0C0C0400u),
                        perm(q[4 * h + 1], q[4 * h], 0x0C0C0400u), 0x05040100u);
    } else {
        // S = floor(t 2^16) + (0xFFFF - h) for the high half h of u carries
        // into bit 16 exactly when h is below the high half of frac 2^32; a
        // tie leaves 16 ones and takes the low half, from the second draw.
        const uint32_t blk = (uint32_t)col >> 3, r0 = (uint32_t)row;
        const int scale = 127 - (int)e; // t = |x| 2^scale
        const uint4 A = philox10(make_uint4(blk, 0u, r0, 0u), a.k0, a.k1);
        const uint4 N = make_uint4(~A.x, ~A.y, ~A.z, ~A.w);
        uint32_t S[8], most = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            S[k] = (uint32_t)ldexpf(fabsf(v[k]), scale + 16) + half16(N, k);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            most = pk_max_u16(most, perm(S[2 * k + 1], S[2 * k], 0x05040100u));
        if ((most >> 16) == 0xFFFFu || (most & 0xFFFFu) == 0xFFFFu) {
            const uint4 B = philox10(make_uint4(blk, 0u, r0, 1u), a.k0, a.k1);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float t = ldexpf(fabsf(v[k]), scale);
                const uint32_t F = (uint32_t)((t - floorf(t)) * 0x1p32f);
                if ((S[k] & 0xFFFFu) == 0xFFFFu && half16(B, k) < (F & 0xFFFFu))
                    S[k] += 1u;
            }
        }
        // magnitudes in pairs of 16 bits, negated by xor and subtraction
        const uint32_t top = highest ? 63u * 0x10001u : 127u * 0x10001u;
        uint32_t q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t mag = pk_min_u16(perm(S[2 * k + 1], S[2 * k], 0x07060302u), top);
            const uint32_t sign =
                perm(__float_as_uint(v[2 * k + 1]), __float_as_uint(v[2 * k]), 0x0B0B0909u);
            q[k] = pk_sub_u16(mag ^ sign, sign);
        }
        w[0] = perm(q[1], q[0], 0x06040200u);
        w[1] = perm(q[3], q[2], 0x06040200u);
    }
    if (!finite)
        w = u32x2{0, 0};
    *reinterpret_cast<u32x2 *>(a.codes + 8 * at) = w;
    if ((col & 24) == 0)
        a.exps[at >> 2] = (uint8_t)e;
}

// 2^E of an exponent byte; NaN for 255.
__device__ __forceinline__ float step_of(uint32_t e)
{
    return bits_f32(e == 255u ? 0x7FC00000u : e << 23);
}

// The eight values of a chunk, as loaded and as floats.
struct RawAct8 {
    u32x2 w;
    uint32_t e;
};
__device__ __forceinline__ void load_act8(const Act8 &a, int64_t at, RawAct8 &r)
{
    r.w = *reinterpret_cast<const u32x2 *>(a.codes + 8 * at);
    r.e = a.exps[at >> 2];
}
__device__ __forceinline__ void unpack_act8(const RawAct8 &r, float (&v)[8])
{
    const float step = step_of(r.e);
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[k] = (float)((int)(r.w[k >> 2] << (24 - 8 * (k & 3))) >> 24) * step;
}
__device__ __forceinline__ void restore8(const Act8 &a, int64_t at, float (&v)[8])
{
    RawAct8 r;
    load_act8(a, at, r);
    unpack_act8(r, v);
}

} // namespace gqt
