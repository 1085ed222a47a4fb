// fp8.hip -- 8-bit floating-point copies with a scale for each block of 128,
// and the products of linear layers from them, on MI355X (gfx950):
// include/gq_step.h.
#include "step_common.h"

#include <algorithm>

namespace gqt {
namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------
// The row copy: sixteen lanes hold a block's 128 columns, a thread block 16
// rows, whose exponent bytes lie side by side.

constexpr int kRowBlocks = 4; // of a thread: as many loads in flight

template <typename T>
__global__ __launch_bounds__(kThreads) void k_fp8_rows(const T *__restrict__ x, int64_t rows,
                                                       int32_t d, int64_t ldx, int32_t random,
                                                       uint32_t k0, uint32_t k1, uint32_t across,
                                                       int64_t epitch, uint8_t *__restrict__ codes,
                                                       uint8_t *__restrict__ exps)
{
    const int64_t row = (int64_t)(blockIdx.x / across) * 16 + threadIdx.x / 16;
    if (row >= rows)
        return; // whole blocks of sixteen lanes
    const int32_t first = blockIdx.x % across * kRowBlocks * 128 + threadIdx.x % 16 * 8;
    const int32_t pitch = (d + 127) / 128 * 128;
    const T *const p = x + row * ldx;
    float v[kRowBlocks][8];
#pragma unroll
    for (int b = 0; b < kRowBlocks; ++b)
        if (first + 128 * b < pitch)
            load8(p, first + 128 * b, d, v[b]);
#pragma unroll
    for (int b = 0; b < kRowBlocks; ++b) {
        const int32_t col = first + 128 * b;
        if (col >= pitch)
            return;
        const uint32_t e = e4m3_exponent(row16_max(abs_bits(v[b])));
        u32x2 w = {0, 0};
        if (e != 255u) {
            if (random) {
                const uint4 draw =
                    philox10(make_uint4((uint32_t)col >> 3, 0u, (uint32_t)row, 0u), k0, k1);
                w = e4m3_random8(v[b], e, draw);
            } else {
                w = e4m3_nearest8(v[b], e);
            }
        }
        *reinterpret_cast<u32x2 *>(codes + row * pitch + col) = w;
        if ((threadIdx.x & 15) == 0)
            exps[(int64_t)(col >> 7) * epitch + row] = (uint8_t)e;
    }
}

// ---------------------------------------------------------------------------
// A weight's copy: a thread block has a square, a thread eight rows of eight
// columns, which it transposes in registers; the transposed codes go through
// LDS, so that they leave in whole lines too.

// Byte k of each of eight rows' eight bytes becomes row k.
__device__ __forceinline__ void transpose8(const u32x2 (&r)[8], u32x2 (&c)[8])
{
#pragma unroll
    for (int half = 0; half < 2; ++half)     // columns 4 half to 4 half + 3
#pragma unroll
        for (int quad = 0; quad < 2; ++quad) { // rows 4 quad to 4 quad + 3
            const uint32_t a = r[4 * quad][half], b = r[4 * quad + 1][half];
            const uint32_t p = r[4 * quad + 2][half], q = r[4 * quad + 3][half];
            const uint32_t ab01 = perm(b, a, 0x05010400u), ab23 = perm(b, a, 0x07030602u);
            const uint32_t pq01 = perm(q, p, 0x05010400u), pq23 = perm(q, p, 0x07030602u);
            c[4 * half][quad] = perm(pq01, ab01, 0x05040100u);
            c[4 * half + 1][quad] = perm(pq01, ab01, 0x07060302u);
            c[4 * half + 2][quad] = perm(pq23, ab23, 0x05040100u);
            c[4 * half + 3][quad] = perm(pq23, ab23, 0x07060302u);
        }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_fp8_weight(const T *__restrict__ w, int32_t n,
                                                         int32_t k, int64_t ldw, uint32_t across,
                                                         uint8_t *__restrict__ codes,
                                                         uint8_t *__restrict__ codes_t,
                                                         uint8_t *__restrict__ exps)
{
    constexpr int kPitch = 128 + 16;
    __shared__ uint32_t largest[kThreads / 64];
    __shared__ __align__(16) uint8_t lds[128 * kPitch];
    const int32_t n0 = blockIdx.x / across * 128, k0 = blockIdx.x % across * 128;
    const int tr = threadIdx.x / 16, tc = threadIdx.x % 16;
    const int32_t row0 = n0 + 8 * tr, col = k0 + 8 * tc;
    float v[8][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (row0 + i < n) {
            load8(w + (row0 + i) * ldw, col, k, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] = 0.0f;
        }
        m = max(m, abs_bits(v[i]));
    }
    m = row16_max(m);
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if ((threadIdx.x & 63) == 0)
        largest[threadIdx.x >> 6] = m;
    __syncthreads();
    m = max(max(largest[0], largest[1]), max(largest[2], largest[3]));
    const uint32_t e = e4m3_exponent(m);
    const int32_t pitch_k = (k + 127) / 128 * 128, pitch_n = (n + 127) / 128 * 128;
    u32x2 r[8], c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        r[i] = e != 255u ? e4m3_nearest8(v[i], e) : u32x2{0, 0};
        if (row0 + i < n)
            *reinterpret_cast<u32x2 *>(codes + (int64_t)(row0 + i) * pitch_k + col) = r[i];
    }
    if (threadIdx.x == 0)
        exps[blockIdx.x] = (uint8_t)e;
    if (!codes_t) // uniform
        return;
    transpose8(r, c);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        *reinterpret_cast<u32x2 *>(lds + (8 * tc + j) * kPitch + 8 * tr) = c[j];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) { // eight lanes a row of 128 bytes
        const int row = 32 * i + threadIdx.x / 8, at = threadIdx.x % 8 * 16;
        if (k0 + row < k)
            *reinterpret_cast<u32x4 *>(codes_t + (int64_t)(k0 + row) * pitch_n + n0 + at) =
                *reinterpret_cast<const u32x4 *>(lds + row * kPitch + at);
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_fp8_restore(const uint8_t *__restrict__ codes,
                                                          const uint8_t *__restrict__ exps,
                                                          uint32_t chunks, uint32_t per_row,
                                                          int32_t d, int32_t squares,
                                                          int64_t epitch, T *__restrict__ out)
{
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= chunks)
        return;
    const uint32_t row = i / per_row;
    const int32_t col = 8 * (i % per_row);
    const int64_t block = col >> 7;
    const uint8_t e = squares ? exps[(row >> 7) * epitch + block] : exps[block * epitch + row];
    const int64_t pitch = (d + 127) / 128 * 128;
    float v[8];
    e4m3_values(*reinterpret_cast<const u32x2 *>(codes + row * pitch + col), step_of(e), v);
    store8(out + (int64_t)row * d + col, d - col, v);
}

// ---------------------------------------------------------------------------
// Products
//
// An MFMA of 16 x 16 x 128 takes a whole block of the summed axis and the two
// copies' powers of two as its scales, so that scaling costs nothing.  Lane l
// gives 32 of the 128 values of row l % 16 of either operand; as both take
// the same 32, their order is free.  So is which of a tile's rows a row of a
// fragment stands for: with F fragments it is row F (l % 16) + i for fragment
// i, which puts a lane's exponent bytes, and its columns of y, side by side.

#define GQT_INLINE __attribute__((always_inline))

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef u32x2 u32x2_e2 __attribute__((aligned(2)));
typedef u32x2 u32x2_e4 __attribute__((aligned(4)));
typedef uint32_t u32_e2 __attribute__((aligned(2)));
typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));

struct Operand {
    const uint8_t *codes;
    const uint8_t *exps;
    int64_t pitch;  // bytes of a row of codes
};

// The weight's exponents of the columns' block b and the depth's block s.
struct Squares {
    const uint8_t *exps;
    int32_t by_cols, by_depth;
    __device__ __forceinline__ uint32_t at(int32_t b, int32_t s) const
    {
        return exps[(int64_t)b * by_cols + (int64_t)s * by_depth];
    }
};

__device__ __forceinline__ i32x8 load_fragment(const uint8_t *p)
{
    const u32x4 a = *reinterpret_cast<const u32x4 *>(p);
    const u32x4 b = *reinterpret_cast<const u32x4 *>(p + 16);
    i32x8 f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[k] = (int)a[k];
        f[4 + k] = (int)b[k];
    }
    return f;
}

// Eight of a fragment's values times their step in bf16, where they are exact.
__device__ __forceinline__ bf16x8 widen(const i32x8 &f, int part, float step)
{
    bf16x8 r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const bf16x2 lo =
            __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)f[2 * part + h], step, false);
        const bf16x2 hi =
            __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)f[2 * part + h], step, true);
        r[4 * h] = lo[0];
        r[4 * h + 1] = lo[1];
        r[4 * h + 2] = hi[0];
        r[4 * h + 3] = hi[1];
    }
    return r;
}

// N bytes from p on (N = 1, 2, 4 or 8).
template <int N>
__device__ __forceinline__ void load_bytes(const uint8_t *p, uint32_t (&b)[N])
{
    if constexpr (N == 8) {
        const u32x2 w = *reinterpret_cast<const u32x2 *>(p);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            b[k] = w[k >> 2] >> (8 * (k & 3)) & 0xFFu;
    } else if constexpr (N == 4) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            b[k] = w >> (8 * k) & 0xFFu;
    } else if constexpr (N == 2) {
        const uint32_t w = *reinterpret_cast<const uint16_t *>(p);
        b[0] = w & 0xFFu;
        b[1] = w >> 8;
    } else {
        b[0] = *p;
    }
}

// Row r's 32 columns from `col` on of x as its copy holds them, made here:
// lanes r, r + 16, r + 32 and r + 48 have the block's four parts.
template <typename T>
__device__ __forceinline__ i32x8 make_fragment(const T *p, int32_t row, int32_t col, int32_t d,
                                               int32_t random, uint32_t k0, uint32_t k1,
                                               uint32_t &e)
{
    float v[4][8];
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        load8(p, col + 8 * q, d, v[q]);
        m = max(m, abs_bits(v[q]));
    }
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    e = e4m3_exponent(m);
    i32x8 f = {};
    if (e == 255u)
        return f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        u32x2 w;
        if (random)
            w = e4m3_random8(v[q], e,
                             philox10(make_uint4(((uint32_t)col >> 3) + q, 0u, (uint32_t)row, 0u),
                                      k0, k1));
        else
            w = e4m3_nearest8(v[q], e);
        f[2 * q] = (int)w[0];
        f[2 * q + 1] = (int)w[1];
    }
    return f;
}

template <typename O>
__device__ __forceinline__ void store_one(O *p, float v) { *p = (O)v; }

__device__ __forceinline__ float bias_at(const void *bias, int32_t dtype, int32_t col)
{
    return dtype == GQ_IN_F32 ? ((const float *)bias)[col] : (float)((const bf16 *)bias)[col];
}

// What a call computes.
struct Product {
    int64_t m;
    int32_t cols, depth, blocks; // blocks: of the depth
    Operand w;
    Squares squares;
    const void *bias;
    int32_t bias_dtype;
    int32_t tiles_n; // tiles along the columns
    // x as its row copy
    Operand x;
    int64_t epitch;
    // or itself
    const void *raw;
    int64_t ldx;
    int32_t random;
    uint32_t k0, k1;
};

// A block has 16 FM rows and 16 FN columns of y; its waves take the depth's
// blocks in turn and add their sums in LDS.  Fragments come straight from
// memory.  MADE: x's copy is made on the way (FM = 1).
template <typename T, int FM, int FN, bool MADE>
__global__ __launch_bounds__(FM * FN >= 16 ? 512 : 1024) void k_product_split(const Product a, T *__restrict__ y)
{
    constexpr bool kExact = sizeof(T) == 4;
    extern __shared__ __align__(16) float sums[];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int32_t col0 = (int32_t)(blockIdx.x % a.tiles_n) * 16 * FN;
    const int64_t row0 = (int64_t)(blockIdx.x / a.tiles_n) * 16 * FM;
    const uint8_t *xp[FM], *wp[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
        xp[i] = MADE ? nullptr : a.x.codes + min(row0 + FM * r + i, a.m - 1) * a.x.pitch + 32 * g;
#pragma unroll
    for (int j = 0; j < FN; ++j)
        wp[j] = a.w.codes + (int64_t)min(col0 + FN * r + j, a.cols - 1) * a.w.pitch + 32 * g;
    const int64_t made_row = min(row0 + r, a.m - 1);
    const T *const raw = MADE ? (const T *)a.raw + made_row * a.ldx : nullptr;
    // a tile's last rows may have no bytes: they are not stored, and read others'
    const uint8_t *const ep = MADE ? nullptr : a.x.exps + min(row0 + FM * r, a.epitch - FM);
    f32x4 acc[FM][FN] = {};
    for (int32_t s = wave; s < a.blocks; s += waves) {
        i32x8 fx[FM], fw[FN];
        uint32_t ex[FM];
        if constexpr (MADE) {
            fx[0] = make_fragment(raw, (int32_t)made_row, 128 * s + 32 * g, a.depth, a.random,
                                  a.k0, a.k1, ex[0]);
        } else {
#pragma unroll
            for (int i = 0; i < FM; ++i)
                fx[i] = load_fragment(xp[i] + 128 * (int64_t)s);
            load_bytes<FM>(ep + s * a.epitch, ex);
        }
#pragma unroll
        for (int j = 0; j < FN; ++j)
            fw[j] = load_fragment(wp[j] + 128 * (int64_t)s);
        const uint32_t ew = a.squares.at(col0 >> 7, s);
        if constexpr (kExact) {
#pragma unroll
            for (int part = 0; part < 4; ++part) {
                bf16x8 bw[FN];
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    bw[j] = widen(fw[j], part, step_of(ew));
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    const bf16x8 bx = widen(fx[i], part, step_of(ex[i]));
#pragma unroll
                    for (int j = 0; j < FN; ++j)
                        acc[i][j] =
                            __builtin_amdgcn_mfma_f32_16x16x32_bf16(bx, bw[j], acc[i][j], 0, 0, 0);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        fx[i], fw[j], acc[i][j], 0, 0, 0, (int)ex[i], 0, (int)ew);
        }
    }
    // sums[wave][i][q][lane][j]
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                sums[((wave * FM + i) * 4 + q) * 64 * FN + lane * FN + j] = acc[i][j][q];
    __syncthreads();
    for (int at = threadIdx.x; at < FM * 4 * 64; at += blockDim.x) {
        const int l = at & 63, q = at >> 6 & 3, i = at >> 8;
        const int64_t row = row0 + FM * (4 * (l >> 4) + q) + i;
        const int32_t col = col0 + FN * (l & 15);
        if (row >= a.m)
            continue;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            float v = 0.0f;
            for (int w = 0; w < waves; ++w)
                v += sums[((w * FM + i) * 4 + q) * 64 * FN + l * FN + j];
            if (col + j < a.cols) {
                if (a.bias)
                    v += bias_at(a.bias, a.bias_dtype, col + j);
                store_one(y + row * a.cols + col + j, v);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// The tiled product: four waves hold 2 x 2 parts of a tile of y, each FM x FN
// fragments of 32 x 32 sums; steps of 128 columns of both operands come
// through LDS, written there by the loads themselves, and are multiplied in
// two halves (an MFMA of 32 x 32 x 64 takes 32 values a lane).
//
// With F fragments, row F (l % 32) + i of a wave's rows belongs to fragment i.
// Sixteen-byte pieces of a row of 128 are stored at their number xor that of
// the row (of its F) modulo 8, so that the lanes of a fragment's read, F rows
// apart, take turns at the banks.

typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int F>
struct Panel { // 64 F rows of an operand's step
    static constexpr int kRows = 64 * F, kBytes = kRows * 128, kLoads = 2 * F;

    // Where this lane's pieces of the wave's loads lie, as offsets from the
    // panel's first row; rows past the last are the last.
    static __device__ __forceinline__ void offsets(uint32_t (&at)[kLoads], int wave, int lane,
                                                   int64_t rows_left, int64_t pitch)
    {
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
            const int row = 8 * (kLoads * wave + q) + lane / 8;
            const int piece = (lane & 7) ^ (row / F & 7);
            at[q] = (uint32_t)(min((int64_t)row, rows_left - 1) * pitch) + 16 * piece;
        }
    }

    // Enqueues this wave's share of a step into `to`, its part of the panel.
    // In assembly, for the compiler makes every read of LDS wait for such
    // loads, into whichever panel they go; land() waits for them.
    static __device__ __forceinline__ void load(uint32_t to, const u32x4 &from,
                                                const uint32_t (&at)[kLoads], int32_t step)
    {
#pragma unroll
        for (int q = 0; q < kLoads; ++q)
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\t"
                         "buffer_load_dwordx4 %1, %2, %3 offen lds"
                         :
                         : "s"(to + 1024 * q), "v"(at[q]), "s"(from), "s"(128 * step)
                         : "memory", "m0");
    }

    // Half u of fragment i, `row` being the first of this lane's F rows.
    static __device__ __forceinline__ i32x8 fragment(const uint8_t *row, int u, int i, int lane)
    {
        const int piece = 4 * u + 2 * (lane >> 5), turn = lane & 7;
        const u32x4 a = *reinterpret_cast<const u32x4 *>(row + 128 * i + 16 * (piece ^ turn));
        const u32x4 b = *reinterpret_cast<const u32x4 *>(row + 128 * i + 16 * ((piece + 1) ^ turn));
        i32x8 f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[k] = (int)a[k];
            f[4 + k] = (int)b[k];
        }
        return f;
    }
};

// Waits until all this block's loads into LDS have landed and all its reads
// of LDS so far are done.
__device__ __forceinline__ void land()
{
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
}

// The descriptor of `rows` rows of `pitch` bytes from p on, 2^30 bytes at most.
__device__ __forceinline__ u32x4 rows_at(const uint8_t *p, int64_t rows, int64_t pitch)
{
    const uint64_t at = (uint64_t)p;
    return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)at),
                 (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(at >> 32)),
                 (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(rows * pitch)), 0x00020000u};
}

// Where block t of a grid of tiles works: each XCD takes a contiguous run,
// and runs go down groups of kGroup tiles before they go across, so that the
// blocks at work on an XCD share rows and columns in its L2.
constexpr int kGroup = 8;
__device__ __forceinline__ void tile_of(int32_t block, int32_t tiles_m, int32_t tiles_n,
                                        int32_t &tm, int32_t &tn)
{
    const int32_t total = tiles_m * tiles_n;
    const int32_t xcd = block % 8, q = total / 8, rem = total % 8;
    const int32_t t = xcd * q + min(xcd, rem) + block / 8;
    const int32_t wide = kGroup * tiles_n;
    const int32_t first = t / wide * kGroup, high = min(tiles_m - first, kGroup);
    tm = first + t % wide % high;
    tn = t % wide / high;
}

// N consecutive results of a row, of which `left` exist.
template <int N>
__device__ __forceinline__ void store_row(bf16 *p, const float (&v)[N], int32_t left)
{
    if (left >= N) {
        uint32_t w[N / 2];
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
            const bf16x2 h = {(bf16)v[2 * k], (bf16)v[2 * k + 1]};
            w[k] = __builtin_bit_cast(uint32_t, h);
        }
        if constexpr (N == 4)
            *reinterpret_cast<u32x2_e2 *>(p) = u32x2{w[0], w[1]};
        else
            *reinterpret_cast<u32_e2 *>(p) = w[0];
        return;
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (k < left)
            p[k] = (bf16)v[k];
}
template <int N>
__device__ __forceinline__ void store_row(float *p, const float (&v)[N], int32_t left)
{
    if (left >= N) {
        if constexpr (N == 4)
            *reinterpret_cast<u32x4_e4 *>(p) =
                u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3])};
        else
            *reinterpret_cast<u32x2_e4 *>(p) = u32x2{__float_as_uint(v[0]), __float_as_uint(v[1])};
        return;
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (k < left)
            p[k] = v[k];
}

template <typename T, int FM, int FN>
__global__ __launch_bounds__(kThreads, FM * FN >= 8 ? 1 : 2) void k_product_tile(
    const Product a, int32_t tiles_m, T *__restrict__ y)
{
    constexpr bool kExact = sizeof(T) == 4;
    constexpr int kX = Panel<FM>::kBytes, kW = Panel<FN>::kBytes, kTurns = 2 * FM;
    extern __shared__ __align__(1024) uint8_t lds[]; // two panels of x, two of w
    const int lane = threadIdx.x & 63, r = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    int32_t tm, tn;
    tile_of(blockIdx.x, tiles_m, a.tiles_n, tm, tn);
    const int64_t row0 = (int64_t)tm * 64 * FM;
    const int32_t col0 = tn * 64 * FN;
    const int64_t rows_left = a.m - row0, cols_left = a.cols - col0;

    uint32_t x_at[Panel<FM>::kLoads], w_at[Panel<FN>::kLoads];
    Panel<FM>::offsets(x_at, wave, lane, rows_left, a.x.pitch);
    Panel<FN>::offsets(w_at, wave, lane, cols_left, a.w.pitch);
    const u32x4 x_rsrc =
        rows_at(a.x.codes + row0 * a.x.pitch, min(rows_left, (int64_t)64 * FM), a.x.pitch);
    const u32x4 w_rsrc =
        rows_at(a.w.codes + col0 * a.w.pitch, min(cols_left, (int64_t)64 * FN), a.w.pitch);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_u8 *)lds;
    const uint32_t x_to = lds0 + wave * (kX / 4), w_to = lds0 + 2 * kX + wave * (kW / 4);
    const uint8_t *const xs = lds + (32 * FM * wm + FM * r) * 128;
    const uint8_t *const ws = lds + 2 * kX + (32 * FN * wn + FN * r) * 128;
    // rows past the last have no bytes of their own: they are not stored
    const uint8_t *const ep = a.x.exps + min(row0 + 32 * FM * wm + FM * r, a.epitch - FM);
    const int32_t w_block = min((col0 + 32 * FN * wn) >> 7, (a.cols - 1) >> 7);
    const int32_t last = a.blocks - 1;

    f32x16 acc[FM][FN] = {};
    // x's fragments in turn, w's of a step's first and second half
    i32x8 fx[3], fw[2][FN];
    uint32_t ex[FM], ew, next_ex[FM], next_ew;

    Panel<FM>::load(x_to, x_rsrc, x_at, 0);
    Panel<FN>::load(w_to, w_rsrc, w_at, 0);
    Panel<FM>::load(x_to + kX, x_rsrc, x_at, min(1, last));
    Panel<FN>::load(w_to + kW, w_rsrc, w_at, min(1, last));
    load_bytes<FM>(ep, ex);
    ew = a.squares.at(w_block, 0);
    land();
#pragma unroll
    for (int j = 0; j < FN; ++j)
        fw[0][j] = Panel<FN>::fragment(ws, 0, j, lane);
    fx[0] = Panel<FM>::fragment(xs, 0, 0, lane);

    for (int32_t s = 0; s <= last; ++s) {
        const uint8_t *const x_now = xs + (s & 1) * kX, *const x_next = xs + (~s & 1) * kX;
        const uint8_t *const w_now = ws + (s & 1) * kW, *const w_next = ws + (~s & 1) * kW;
        bf16x8 wide[kExact ? FN : 1][4];
        // Turn t multiplies fragment t % FM of half t / FM, while those of the
        // turns behind it are read.  Before the last two all of this step has
        // been read, and all of the next has landed; where this one lay goes
        // the one after.
#pragma unroll
        for (int t = 0; t < kTurns; ++t) {
            const int u = t / FM, i = t % FM;
            if (t == kTurns - 2) {
                land();
                if (s + 2 <= last) {
                    Panel<FM>::load(x_to + (s & 1) * kX, x_rsrc, x_at, s + 2);
                    Panel<FN>::load(w_to + (s & 1) * kW, w_rsrc, w_at, s + 2);
                }
            }
            if (t < kTurns - 3)
                fx[(t + 1) & 1] = Panel<FM>::fragment(x_now, (t + 1) / FM, (t + 1) % FM, lane);
            if (t == kTurns - 3) {
                fx[0] = Panel<FM>::fragment(x_now, 1, FM - 2, lane);
                fx[2] = Panel<FM>::fragment(x_now, 1, FM - 1, lane);
            }
            if (t == kTurns - 1)
                fx[0] = Panel<FM>::fragment(x_next, 0, 0, lane);
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                if (t == j * FM / FN)
                    fw[1][j] = Panel<FN>::fragment(w_now, 1, j, lane);
                if (t == kTurns - 2 + 2 * j / FN)
                    fw[0][j] = Panel<FN>::fragment(w_next, 0, j, lane);
            }
            if (t == 0) {
                const int32_t n = min(s + 1, last);
                load_bytes<FM>(ep + n * a.epitch, next_ex);
                next_ew = a.squares.at(w_block, n);
            }
            const i32x8 &x = fx[t == kTurns - 1 ? 2 : t & 1];
            if constexpr (kExact) {
                if (i == 0) {
#pragma unroll
                    for (int j = 0; j < FN; ++j)
#pragma unroll
                        for (int part = 0; part < 4; ++part)
                            wide[j][part] = widen(fw[u][j], part, step_of(ew));
                }
#pragma unroll
                for (int part = 0; part < 4; ++part) {
                    const bf16x8 bx = widen(x, part, step_of(ex[i]));
#pragma unroll
                    for (int j = 0; j < FN; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bx, wide[j][part],
                                                                            acc[i][j], 0, 0, 0);
                }
            } else {
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        x, fw[u][j], acc[i][j], 0, 0, 0, (int)ex[i], 0, (int)ew);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < FM; ++i)
            ex[i] = next_ex[i];
        ew = next_ew;
    }

    const int32_t col = col0 + 32 * FN * wn + FN * r;
    float bias[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j)
        bias[j] = a.bias && col + j < a.cols ? bias_at(a.bias, a.bias_dtype, col + j) : 0.0f;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            const int of = 8 * (q / 4) + 4 * (lane >> 5) + q % 4;
            const int64_t row = row0 + 32 * FM * wm + FM * of + i;
            float v[FN];
#pragma unroll
            for (int j = 0; j < FN; ++j)
                v[j] = acc[i][j][q] + bias[j];
            if (row < a.m)
                store_row<FN>(y + row * a.cols + col, v, a.cols - col);
        }
}

// ---------------------------------------------------------------------------
// host

int32_t check_sides(int32_t dtype, int64_t rows, int64_t d)
{
    if (!dtype_ok(dtype))
        return fail(GQ_ERR_ARG, "dtype %d is neither GQ_IN_F32 nor GQ_IN_BF16", dtype);
    if (rows < 0 || rows >= kMaxRows || d < 1 || d > kMaxSide)
        return fail(GQ_ERR_ARG, "%lld rows of %lld columns: below 2^31 and from 1 to 2^22",
                    (long long)rows, (long long)d);
    if (rows * blocks_of(d) >= kMaxRows)
        return fail(GQ_ERR_UNSUPPORTED, "%lld rows of %lld columns: 2^31 blocks or more",
                    (long long)rows, (long long)d);
    return GQ_OK;
}

int32_t check_matrix(const char *name, const void *p, int32_t dtype, int64_t rows)
{
    if (!p && rows > 0)
        return fail(GQ_ERR_NULL, "%s is NULL", name);
    if (!aligned_to(p, elem_bytes(dtype)))
        return fail(GQ_ERR_ALIGN, "%s is not aligned to its elements", name);
    return GQ_OK;
}

int32_t check_ld(const char *name, int64_t ld, int64_t d)
{
    if ((ld != 0 && ld < d) || ld > ((int64_t)1 << 40))
        return fail(GQ_ERR_ARG, "%s = %lld: 0 or at least %lld", name, (long long)ld,
                    (long long)d);
    return GQ_OK;
}

int32_t check_codes(const char *name, const void *p, bool needed)
{
    if (!p && needed)
        return fail(GQ_ERR_NULL, "%s is NULL", name);
    if (!aligned_to(p, 16))
        return fail(GQ_ERR_ALIGN, "%s is not 16-byte aligned", name);
    return GQ_OK;
}

int32_t check_rounding(int32_t rounding)
{
    return rounding == GQS_ROUND_NEAREST || rounding == GQS_ROUND_RANDOM
               ? GQ_OK
               : fail(GQ_ERR_ARG, "rounding %d", rounding);
}

int32_t launch_rows(const void *x, int32_t dtype, int64_t rows, int64_t d, int64_t ldx,
                    int32_t rounding, uint64_t seed, uint8_t *codes, uint8_t *exps, hipStream_t st)
{
    const uint32_t across = (uint32_t)((blocks_of(d) + kRowBlocks - 1) / kRowBlocks);
    const uint32_t grid = (uint32_t)((rows + 15) / 16) * across;
    const int32_t random = rounding == GQS_ROUND_RANDOM;
    const uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
    if (dtype == GQ_IN_F32)
        k_fp8_rows<float><<<grid, kThreads, 0, st>>>((const float *)x, rows, (int32_t)d, ldx,
                                                     random, k0, k1, across, exp_pitch(rows),
                                                     codes, exps);
    else
        k_fp8_rows<bf16><<<grid, kThreads, 0, st>>>((const bf16 *)x, rows, (int32_t)d, ldx, random,
                                                    k0, k1, across, exp_pitch(rows), codes, exps);
    return check_launch("k_fp8_rows");
}

// Lets a kernel have more than 64 KB of LDS.
template <typename K>
int32_t allow_lds(K *kernel, const char *name, uint32_t bytes)
{
    if (bytes <= 65536)
        return GQ_OK;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    return e == hipSuccess ? GQ_OK : fail(GQ_ERR_DEVICE, "%s: %s", name, hipGetErrorString(e));
}

template <typename T, int FM, int FN, bool MADE>
int32_t launch_split(Product a, T *y, hipStream_t st)
{
    a.tiles_n = (int32_t)((a.cols + 16 * FN - 1) / (16 * FN));
    const int64_t grid = (a.m + 16 * FM - 1) / (16 * FM) * a.tiles_n;
    const int waves = std::min(FM * FN >= 16 ? 8 : 16, std::max(1, (int)a.blocks));
    const uint32_t lds = (uint32_t)waves * FM * FN * 1024;
    if (grid >= ((int64_t)1 << 31) / (64 * 16))
        return fail(GQ_ERR_UNSUPPORTED, "%lld tiles", (long long)grid);
    GQT_TRY(allow_lds(&k_product_split<T, FM, FN, MADE>, "k_product_split", lds));
    k_product_split<T, FM, FN, MADE><<<(uint32_t)grid, 64 * waves, lds, st>>>(a, y);
    return check_launch("k_product_split");
}

template <typename T, int FM, int FN>
int32_t launch_tile(Product a, T *y, hipStream_t st)
{
    const int64_t tiles_m = (a.m + 64 * FM - 1) / (64 * FM);
    a.tiles_n = (a.cols + 64 * FN - 1) / (64 * FN);
    if (tiles_m * a.tiles_n >= ((int64_t)1 << 31) / kThreads)
        return fail(GQ_ERR_UNSUPPORTED, "%lld tiles", (long long)(tiles_m * a.tiles_n));
    constexpr uint32_t kLds = 2 * (Panel<FM>::kBytes + Panel<FN>::kBytes);
    GQT_TRY(allow_lds(&k_product_tile<T, FM, FN>, "k_product_tile", kLds));
    k_product_tile<T, FM, FN><<<(uint32_t)(tiles_m * a.tiles_n), kThreads, kLds, st>>>(
        a, (int32_t)tiles_m, y);
    return check_launch("k_product_tile");
}

template <typename T>
int32_t launch_product(const Product &a, void *y, hipStream_t st)
{
    T *const out = (T *)y;
    if (a.m <= 16)
        return a.raw ? launch_split<T, 1, 1, true>(a, out, st)
                     : launch_split<T, 1, 1, false>(a, out, st);
    if (a.m <= 32)
        return launch_split<T, 2, 1, false>(a, out, st);
    if (a.m <= 64)
        return launch_split<T, 4, 2, false>(a, out, st);
    const int64_t squares = ((a.m + 127) / 128) * ((a.cols + 127) / 128);
    if (squares >= 64) {
        if constexpr (sizeof(T) == 2)
            if (squares >= 1024)
                return launch_tile<T, 4, 4>(a, out, st);
        return launch_tile<T, 2, 2>(a, out, st);
    }
    return launch_split<T, 8, 2, false>(a, out, st);
}

int32_t check_product(int32_t dtype, int64_t m, int64_t cols, int64_t depth, const void *w_codes,
                      const void *w_exps, const void *bias, int32_t bias_dtype, const void *y)
{
    GQT_TRY(check_sides(dtype, m, depth));
    GQT_TRY(check_sides(dtype, m, cols));
    GQT_TRY(check_codes("w_codes", w_codes, true));
    if (!w_exps)
        return fail(GQ_ERR_NULL, "w_exps is NULL");
    if (bias && !dtype_ok(bias_dtype))
        return fail(GQ_ERR_ARG, "bias_dtype %d is neither GQ_IN_F32 nor GQ_IN_BF16", bias_dtype);
    if (bias && !aligned_to(bias, elem_bytes(bias_dtype)))
        return fail(GQ_ERR_ALIGN, "bias is not aligned to its elements");
    return check_matrix("y", y, dtype, m);
}

Product product_of(int64_t m, const void *w_codes, const void *w_exps, int64_t cols, int64_t depth,
                   int32_t transposed, const void *bias, int32_t bias_dtype)
{
    Product a{};
    a.m = m;
    a.cols = (int32_t)cols;
    a.depth = (int32_t)depth;
    a.blocks = (int32_t)blocks_of(depth);
    a.w = {(const uint8_t *)w_codes, nullptr, fp8_pitch(depth)};
    a.squares = transposed ? Squares{(const uint8_t *)w_exps, 1, (int32_t)blocks_of(cols)}
                           : Squares{(const uint8_t *)w_exps, (int32_t)blocks_of(depth), 1};
    a.bias = bias;
    a.bias_dtype = bias_dtype;
    return a;
}

// The sizes of a row copy in a workspace.
int64_t codes_bytes(int64_t m, int64_t depth) { return m * fp8_pitch(depth); }
int64_t exps_bytes(int64_t m, int64_t depth) { return blocks_of(depth) * exp_pitch(m); }
bool made_on_the_way(int64_t m) { return m <= 16; }

int32_t check_workspace(int64_t need, const void *workspace, int64_t workspace_bytes)
{
    if (need > 0 && !workspace)
        return fail(GQ_ERR_NULL, "workspace is NULL");
    if (workspace_bytes < need)
        return fail(GQ_ERR_WORKSPACE, "workspace of %lld bytes, %lld are needed",
                    (long long)workspace_bytes, (long long)need);
    return aligned_to(workspace, 16) ? GQ_OK
                                     : fail(GQ_ERR_ALIGN, "workspace is not 16-byte aligned");
}

int32_t run_product(const Product &a, void *y, int32_t dtype, hipStream_t st)
{
    return dtype == GQ_IN_F32 ? launch_product<float>(a, y, st) : launch_product<bf16>(a, y, st);
}

} // namespace
} // namespace gqt

using namespace gqt;

extern "C" {

int64_t gqs_fp8_blocks(int64_t d) { return d < 1 || d > kMaxSide ? -1 : blocks_of(d); }
int64_t gqs_fp8_pitch(int64_t d) { return d < 1 || d > kMaxSide ? -1 : fp8_pitch(d); }
int64_t gqs_fp8_exp_pitch(int64_t rows)
{
    return rows < 0 || rows >= kMaxRows ? -1 : exp_pitch(rows);
}

int32_t gqs_fp8_rows(const void *x, int32_t dtype, int64_t rows, int64_t d, int64_t ldx,
                     int32_t rounding, uint64_t seed, void *codes, void *exps, void *stream)
{
    GQT_TRY(check_sides(dtype, rows, d));
    GQT_TRY(check_matrix("x", x, dtype, rows));
    GQT_TRY(check_ld("ldx", ldx, d));
    GQT_TRY(check_rounding(rounding));
    GQT_TRY(check_codes("codes", codes, rows > 0));
    GQT_TRY(check_codes("exps", exps, rows > 0));
    if (rows == 0)
        return ok();
    return launch_rows(x, dtype, rows, d, ldx, rounding, seed, (uint8_t *)codes, (uint8_t *)exps,
                       (hipStream_t)stream);
}

int32_t gqs_fp8_weight(const void *w, int32_t dtype, int64_t n, int64_t k, int64_t ldw,
                       void *codes, void *codes_t, void *exps, void *stream)
{
    GQT_TRY(check_sides(dtype, n, k));
    if (n < 1 || n > kMaxSide)
        return fail(GQ_ERR_ARG, "n = %lld: from 1 to 2^22", (long long)n);
    GQT_TRY(check_matrix("w", w, dtype, n));
    GQT_TRY(check_ld("ldw", ldw, k));
    GQT_TRY(check_codes("codes", codes, true));
    GQT_TRY(check_codes("codes_t", codes_t, false));
    if (!exps)
        return fail(GQ_ERR_NULL, "exps is NULL");
    const uint32_t across = (uint32_t)blocks_of(k);
    const int64_t grid = blocks_of(n) * across;
    if (grid >= ((int64_t)1 << 23))
        return fail(GQ_ERR_UNSUPPORTED, "%lld squares: below 2^23", (long long)grid);
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == GQ_IN_F32)
        k_fp8_weight<float><<<(uint32_t)grid, kThreads, 0, st>>>(
            (const float *)w, (int32_t)n, (int32_t)k, ldw, across, (uint8_t *)codes,
            (uint8_t *)codes_t, (uint8_t *)exps);
    else
        k_fp8_weight<bf16><<<(uint32_t)grid, kThreads, 0, st>>>(
            (const bf16 *)w, (int32_t)n, (int32_t)k, ldw, across, (uint8_t *)codes,
            (uint8_t *)codes_t, (uint8_t *)exps);
    return check_launch("k_fp8_weight");
}

int32_t gqs_fp8_restore(const void *codes, const void *exps, int64_t rows, int64_t d,
                        int32_t squares, int32_t dtype, void *out, void *stream)
{
    GQT_TRY(check_sides(dtype, rows, d));
    if (rows * blocks_of(d) >= ((int64_t)1 << 27))
        return fail(GQ_ERR_UNSUPPORTED, "%lld rows of %lld columns: 2^27 blocks or more",
                    (long long)rows, (long long)d);
    GQT_TRY(check_codes("codes", codes, rows > 0));
    if (!exps && rows > 0)
        return fail(GQ_ERR_NULL, "exps is NULL");
    GQT_TRY(check_matrix("out", out, dtype, rows));
    if (rows == 0)
        return ok();
    const uint32_t per_row = (uint32_t)((d + 7) / 8), chunks = (uint32_t)rows * per_row;
    const uint32_t grid = (chunks + kThreads - 1) / kThreads;
    const int64_t epitch = squares ? blocks_of(d) : exp_pitch(rows);
    const uint8_t *c = (const uint8_t *)codes, *e = (const uint8_t *)exps;
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == GQ_IN_F32)
        k_fp8_restore<float><<<grid, kThreads, 0, st>>>(c, e, chunks, per_row, (int32_t)d, squares,
                                                        epitch, (float *)out);
    else
        k_fp8_restore<bf16><<<grid, kThreads, 0, st>>>(c, e, chunks, per_row, (int32_t)d, squares,
                                                       epitch, (bf16 *)out);
    return check_launch("k_fp8_restore");
}

int64_t gqs_fp8_product_workspace_bytes(int64_t m, int64_t cols, int64_t depth, int32_t dtype)
{
    if (check_sides(dtype, m, depth) != GQ_OK || check_sides(dtype, m, cols) != GQ_OK)
        return -1;
    return 0;
}

int32_t gqs_fp8_product(const void *x_codes, const void *x_exps, int64_t m, const void *w_codes,
                        const void *w_exps, int64_t cols, int64_t depth, int32_t transposed,
                        const void *bias, int32_t bias_dtype, void *y, int32_t dtype,
                        void *workspace, int64_t workspace_bytes, void *stream)
{
    GQT_TRY(check_product(dtype, m, cols, depth, w_codes, w_exps, bias, bias_dtype, y));
    GQT_TRY(check_codes("x_codes", x_codes, m > 0));
    GQT_TRY(check_codes("x_exps", x_exps, m > 0));
    GQT_TRY(check_workspace(gqs_fp8_product_workspace_bytes(m, cols, depth, dtype), workspace,
                            workspace_bytes));
    if (m == 0)
        return ok();
    Product a = product_of(m, w_codes, w_exps, cols, depth, transposed, bias, bias_dtype);
    a.x = {(const uint8_t *)x_codes, (const uint8_t *)x_exps, fp8_pitch(depth)};
    a.epitch = exp_pitch(m);
    return run_product(a, y, dtype, (hipStream_t)stream);
}

int64_t gqs_fp8_linear_workspace_bytes(int64_t m, int64_t cols, int64_t depth, int32_t dtype)
{
    const int64_t product = gqs_fp8_product_workspace_bytes(m, cols, depth, dtype);
    if (product < 0 || made_on_the_way(m))
        return product;
    return product + codes_bytes(m, depth) + exps_bytes(m, depth);
}

int32_t gqs_fp8_linear(const void *x, int32_t dtype, int64_t m, int64_t depth, int64_t ldx,
                       int32_t rounding, uint64_t seed, const void *w_codes, const void *w_exps,
                       int64_t cols, int32_t transposed, const void *bias, int32_t bias_dtype,
                       void *y, void *workspace, int64_t workspace_bytes, void *stream)
{
    GQT_TRY(check_product(dtype, m, cols, depth, w_codes, w_exps, bias, bias_dtype, y));
    GQT_TRY(check_matrix("x", x, dtype, m));
    GQT_TRY(check_ld("ldx", ldx, depth));
    GQT_TRY(check_rounding(rounding));
    GQT_TRY(check_workspace(gqs_fp8_linear_workspace_bytes(m, cols, depth, dtype), workspace,
                            workspace_bytes));
    if (m == 0)
        return ok();
    const hipStream_t st = (hipStream_t)stream;
    Product a = product_of(m, w_codes, w_exps, cols, depth, transposed, bias, bias_dtype);
    if (made_on_the_way(m)) {
        a.raw = x;
        a.ldx = ldx;
        a.random = rounding == GQS_ROUND_RANDOM;
        a.k0 = (uint32_t)seed;
        a.k1 = (uint32_t)(seed >> 32);
    } else {
        uint8_t *const codes = (uint8_t *)workspace, *const exps = codes + codes_bytes(m, depth);
        GQT_TRY(launch_rows(x, dtype, m, depth, ldx, rounding, seed, codes, exps, st));
        a.x = {codes, exps, fp8_pitch(depth)};
        a.epitch = exp_pitch(m);
    }
    return run_product(a, y, dtype, st);
}

} // extern "C"
