// fp8.hip -- 8-bit floating-point copies with a scale for each block of 128,
// and the products of linear layers from them, on MI355X (gfx950):
// include/gq_step.h.
#include "step_common.h"

#include <algorithm>

namespace gqt {
namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------
// The row copy: one pass, bound by memory.  Sixteen lanes hold a block's 128
// columns, eight each, so that its largest value takes three steps between
// lanes and one Philox call serves a lane's eight roundings; a thread block
// has 16 rows, whose exponent bytes lie side by side.  bf16 8192 x 4096 (101
// MB): 20 us, 5.0 TB/s, either rounding.

constexpr int kRowBlocks = 4; // of a thread: as many loads in flight

template <typename T>
__global__ __launch_bounds__(kThreads) void k_fp8_rows(const T *__restrict__ x, int64_t rows,
                                                       int32_t d, int64_t ldx, int32_t random,
                                                       uint32_t k0, uint32_t k1, FastDiv across,
                                                       int64_t epitch, uint8_t *__restrict__ codes,
                                                       uint8_t *__restrict__ exps)
{
    const uint32_t down = divide(blockIdx.x, across);
    const int64_t row = (int64_t)down * 16 + threadIdx.x / 16;
    if (row >= rows)
        return; // whole blocks of sixteen lanes
    const int32_t first =
        (blockIdx.x - down * across.d) * kRowBlocks * 128 + threadIdx.x % 16 * 8;
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
// A weight's copy, one pass over it, bound by memory.  A thread block has a
// square, a thread eight rows of eight columns, which it transposes in
// registers; the transposed codes go through LDS, so that they leave in whole
// lines too.  bf16 4096 x 4096 with both (67 MB): 15 us, 4.5 TB/s; the writes
// to LDS meet in banks, behind the memory's time.

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
                                                          uint32_t chunks, FastDiv per_row,
                                                          int32_t d, int32_t squares,
                                                          int64_t epitch, T *__restrict__ out)
{
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= chunks)
        return;
    const uint32_t row = divide(i, per_row);
    const int32_t col = 8 * (i - row * per_row.d);
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
// The scaled 8-bit MFMAs take the two copies' powers of two as their scales, so
// that scaling costs nothing.  Lanes give parts of a row of either operand; as
// both take the same parts, their order is free.  So is which of a tile's rows
// a row of a fragment stands for: with F fragments it is row F r + i for lane
// r of fragment i, which puts a lane's exponent bytes, and its columns of y,
// side by side.
//
// The 8-bit MFMAs cut off, in each group of eight products, what lies below
// 2^-13 of the largest's leading bit, and add the groups in fp32: a group can
// lose 7 2^-13 of its largest product.  Next to large products that cancel,
// that may be all of a result.  Of normal inputs it moves 2.5 % of the bf16
// results by a last place, and their error stays that of the rounding, 1.66e-3.
// Many rows take them for bf16 results all the same, at twice the rate.  For
// fp32 results, and for few rows, which the MFMAs do not bound, the codes are
// widened to bf16 times their steps, which is exact, and multiplied by bf16
// MFMAs, exact too.

#define GQT_INLINE __attribute__((always_inline))

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef u32x2 u32x2_e2 __attribute__((aligned(2)));
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

// N exponent bytes side by side.
template <int N>
struct Bytes;
template <>
struct Bytes<1> {
    uint8_t b;
    __device__ __forceinline__ uint32_t byte(int) const { return b; }
};
template <>
struct Bytes<2> {
    uint16_t b;
    __device__ __forceinline__ uint32_t byte(int i) const { return b >> (8 * i) & 0xFFu; }
};
template <>
struct Bytes<4> {
    uint32_t b;
    __device__ __forceinline__ uint32_t byte(int i) const { return b >> (8 * i) & 0xFFu; }
};
template <>
struct Bytes<8> {
    u32x2 b;
    __device__ __forceinline__ uint32_t byte(int i) const
    {
        return b[i >> 2] >> (8 * (i & 3)) & 0xFFu;
    }
};

// N of them, PART at once.
template <int N, int PART>
struct Parts {
    Bytes<PART> part[N / PART];
    __device__ __forceinline__ uint32_t byte(int i) const { return part[i / PART].byte(i % PART); }
};

typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) u32x2 lds_u32x2;

// Loads from memory to LDS: `to` and what follows it for the other lanes.  In
// assembly, for the compiler makes every read of LDS wait for such loads,
// wherever they go, and does not count others behind them: a wait of ours has
// to come before the reads.
// Lanes past the descriptor's end give zeros.
__device__ __forceinline__ void load_lds16(uint32_t to, const u32x4 &from, uint32_t at, uint32_t base)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :: "s"(to), "v"(at), "s"(from), "s"(base) : "memory");
}
__device__ __forceinline__ void load_lds4(uint32_t to, const u32x4 &from, uint32_t at, uint32_t base)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
                 :: "s"(to), "v"(at), "s"(from), "s"(base) : "memory");
}
__device__ __forceinline__ void load_lds1(uint32_t to, const u32x4 &from, uint32_t at, uint32_t base)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ubyte %1, %2, %3 offen lds"
                 :: "s"(to), "v"(at), "s"(from), "s"(base) : "memory");
}

__device__ __forceinline__ u32x4 descriptor(const uint8_t *p, uint32_t bytes)
{
    const uint64_t at = (uint64_t)p;
    return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)at),
                 (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(at >> 32)),
                 (uint32_t)__builtin_amdgcn_readfirstlane(bytes), 0x00020000u};
}

// How rows of 128 bytes lie in LDS.  It gives 256 bytes a cycle, sixteen lanes
// their sixteen bytes.  A lane's F rows lie in F lines of 128 bytes, for the
// second eight of sixteen lanes with neighbours changed about, and a row's
// sixteen-byte pieces at their number xor the lane's, so that the lanes of a
// fragment's read, F rows apart, find all banks.
template <int F>
struct Order { // what the lane of rows F r on does to its lines' and pieces' numbers
    static __device__ __forceinline__ int change(int r) { return F > 1 ? r >> 3 & 1 : 0; }
    static __device__ __forceinline__ int turn(int r) { return F > 1 ? r & 7 : r >> 1 & 7; }
};

// A block of 16 F rows of an operand, in a wave's own part of LDS.
template <int F>
struct Strip {
    static constexpr int kBytes = 16 * F * 128, kLoads = 2 * F;

    // Where the lane's pieces lie, from the first row on; rows from `rows` on
    // are the last.
    static __device__ __forceinline__ void offsets(uint32_t (&at)[kLoads], int lane, int32_t rows,
                                                   int64_t pitch)
    {
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
            const int line = 8 * q + lane / 8;
            const int row = line ^ Order<F>::change(line / F);
            const int piece = (lane & 7) ^ Order<F>::turn(line / F);
            at[q] = (uint32_t)(min(row, rows - 1) * pitch) + 16 * piece;
        }
    }
    static __device__ __forceinline__ void load(uint32_t to, const u32x4 &from,
                                                const uint32_t (&at)[kLoads], int32_t step)
    {
#pragma unroll
        for (int q = 0; q < kLoads; ++q)
            load_lds16(to + 1024 * q, from, at[q], 128 * step);
    }
    static __device__ __forceinline__ i32x8 fragment(uint32_t strip, int i, int lane)
    {
        const int r = lane & 15;
        const uint32_t at = strip + r * F * 128 + 128 * Order<F>::change(r) +
                            16 * (Order<F>::turn(r) ^ (lane >> 4 << 1));
        const uint32_t of = 128 * (i & 1), beyond = 128 * (i & ~1);
        const u32x4 a = *(const lds_u32x4 *)(uintptr_t)((at ^ of) + beyond);
        const u32x4 b = *(const lds_u32x4 *)(uintptr_t)((at ^ (of + 16)) + beyond);
        i32x8 f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[k] = (int)a[k];
            f[4 + k] = (int)b[k];
        }
        return f;
    }
};

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
    uint32_t tiles_m;                      // tiles along the rows
    FastDiv by_tiles, by_group, by_rest;   // all, those of kGroup rows, rows of the last group
    int32_t splits, steps;    // parts of the depth, and blocks of one
    float *parts;             // where they leave their sums [splits][m][cols]
    // x as its row copy
    Operand x;
    int64_t epitch;
    // or itself
    const void *raw;
    int64_t ldx;
    int32_t random;
    uint32_t k0, k1;
};

// Few rows: a block has 16 F rows and 16 columns of y, so that a weight of
// thousands of columns is read by all of the card, once for each 16 F rows.
// Its waves take the depth's blocks in turn, each through LDS of its own, where
// loads of whole lines put them (lanes that load fragments straight from
// memory, sixteen rows at once, take four times as long), and add their sums
// at the end.  MADE: x's copy is made on the way, sixteen lanes a row (F = 1):
// every block makes it again, which up to 16 rows costs less than a kernel of
// its own, about 2 us.  From bf16 rows 1 x 4096 x 1024 (rows, columns, depth)
// 3.6 us, 1 x 4096 x 4096 5.9 to 6.1, 16 x 1024 x 4096 8.6; from their copy 32 x
// 4096 x 4096 5.8, 64 x 4096 x 4096 7.8 (a weight of 17 MB, 2.1 to 2.9 TB/s:
// bound by latency, more than by its bytes), 96 x 4096 x 4096 9.1 to 10.7, bound
// by the rows, which every block takes from the L2 again.  With 8-bit MFMAs bf16
// results of 17 rows and more took 0.4 to 0.7 us less; two blocks at once for
// each wave 0.1 to 1 us more up to 16 rows.
template <typename T, int F, bool MADE>
__global__ __launch_bounds__(F > 2 ? 512 : 1024) void k_product_direct(const Product a,
                                                                       T *__restrict__ y)
{
    using X = Strip<F>;
    using W = Strip<1>;
    constexpr int kStep = X::kBytes + W::kBytes;
    extern __shared__ __align__(1024) uint8_t lds[];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const uint32_t tm = divide(blockIdx.x, a.by_tiles);
    const int32_t col0 = (int32_t)(blockIdx.x - tm * a.by_tiles.d) * 16;
    const int64_t row0 = (int64_t)tm * 16 * F;
    const int32_t rows = (int32_t)min(a.m - row0, (int64_t)16 * F), cols = min(a.cols - col0, 16);
    const uint32_t own = (uint32_t)(uintptr_t)(lds_u8 *)lds + wave * kStep;

    uint32_t w_at[W::kLoads], x_at[X::kLoads];
    W::offsets(w_at, lane, cols, a.w.pitch);
    const u32x4 w_from =
        descriptor(a.w.codes + col0 * a.w.pitch, (uint32_t)cols * (uint32_t)a.w.pitch);
    u32x4 x_from{};
    // Where the lane's exponents are, kPart together (a row copy has bytes for
    // whole 16s of rows, which kPart divides); rows past them are not stored.
    constexpr int kPart = F == 6 ? 2 : F;
    int32_t e_at[F / kPart];
    if constexpr (!MADE) {
        X::offsets(x_at, lane, rows, a.x.pitch);
        x_from = descriptor(a.x.codes + row0 * a.x.pitch, (uint32_t)rows * (uint32_t)a.x.pitch);
#pragma unroll
        for (int i = 0; i < F; i += kPart)
            e_at[i / kPart] = (int32_t)min(row0 + F * r + i, a.epitch - kPart);
    }
    f32x4 acc[F] = {};
    for (int32_t s = wave; s < a.blocks; s += waves) {
        Parts<F, kPart> ex;
        Raw8<T> raw[4];
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); // what lay there has been read
        W::load(own, w_from, w_at, s);
        if constexpr (MADE) {
#pragma unroll
            for (int i = 0; i < 4; ++i) // row 4 i + g
                if (4 * i < rows)
                    load_ahead((const T *)a.raw + min(row0 + 4 * i + g, a.m - 1) * a.ldx,
                               128 * s + 8 * r, a.depth, raw[i]);
        } else {
            X::load(own + W::kBytes, x_from, x_at, s);
            const uint8_t *const e = a.x.exps + s * a.epitch;
#pragma unroll
            for (int i = 0; i < F / kPart; ++i)
                ex.part[i] = *reinterpret_cast<const Bytes<kPart> *>(e + e_at[i]);
        }
        const uint32_t ew = a.squares.at(col0 >> 7, s);
        if constexpr (MADE) {
            uint32_t of_row = 0; // lane r: the exponent of row r
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (4 * i >= rows)
                    break;
                const int32_t row = 4 * i + g, col = 128 * s + 8 * r;
                float v[8];
                settle((const T *)a.raw + min(row0 + row, a.m - 1) * a.ldx, col, a.depth, raw[i]);
                unpack(raw[i], v);
                const uint32_t e = e4m3_exponent(row16_max(abs_bits(v)));
                u32x2 w = {0, 0};
                if (e != 255u)
                    w = a.random ? e4m3_random8(v, e,
                                                philox10(make_uint4((uint32_t)col >> 3, 0u,
                                                                    (uint32_t)(row0 + row), 0u),
                                                         a.k0, a.k1))
                                 : e4m3_nearest8(v, e);
                const uint32_t at =
                    own + W::kBytes + row * 128 + 16 * ((r >> 1) ^ Order<1>::turn(row)) + 8 * (r & 1);
                *(lds_u32x2 *)(uintptr_t)at = w;
                const uint32_t other = (uint32_t)__shfl((int)e, 16 * (r & 3));
                of_row = r >> 2 == i ? other : of_row;
            }
            ex.part[0].b = (uint8_t)of_row;
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        const i32x8 fw = W::fragment(own, 0, lane);
        bf16x8 wide[4];
#pragma unroll
        for (int part = 0; part < 4; ++part)
            wide[part] = widen(fw, part, step_of(ew));
#pragma unroll
        for (int i = 0; i < F; ++i) {
            const i32x8 fx = X::fragment(own + W::kBytes, i, lane);
#pragma unroll
            for (int part = 0; part < 4; ++part)
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    widen(fx, part, step_of(ex.byte(i))), wide[part], acc[i], 0, 0, 0);
        }
    }
    // sums[wave][i][q][lane], where the blocks were
    float *const sums = reinterpret_cast<float *>(lds);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            sums[((wave * F + i) * 4 + q) * 64 + lane] = acc[i][q];
    __syncthreads();
    for (int at = threadIdx.x; at < F * 4 * 64; at += blockDim.x) {
        const int l = at & 63, q = at >> 6 & 3, i = at >> 8;
        const int64_t row = row0 + F * (4 * (l >> 4) + q) + i;
        const int32_t col = col0 + (l & 15);
        if (row >= a.m || col >= a.cols)
            continue;
        float v = 0.0f;
        for (int w = 0; w < waves; ++w)
            v += sums[((w * F + i) * 4 + q) * 64 + l];
        if (a.bias)
            v += bias_at(a.bias, a.bias_dtype, col);
        store_one(y + row * a.cols + col, v);
    }
}

// ---------------------------------------------------------------------------
// The tiled product: WM x WN waves hold as many parts of a tile of y, each FM x
// FN fragments of 32 x 32 sums.  Steps of 128 columns of both operands come
// through LDS, written there by the loads themselves, STAGES - 1 steps ahead,
// and are multiplied in two halves (an MFMA of 32 x 32 x 64 takes 32 values a
// lane).  A block goes from tile to tile without a pause in its loads.
//
// With F fragments, row F (l % 32) + i of a wave's rows belongs to fragment i.
//
// The matrix cores bound it, then the L2: a CU takes 26 bytes a cycle from
// there, and a 256 x 256 tile's step of 64 KB its MFMAs' time over again, so
// that smaller tiles are bound by their loads.  bf16 8192 x 8192 x 8192: 413 us,
// 2660 TFLOP/s (without the loads 3250, the MFMAs alone 4190); 8192 x 4096 x
// 4096 110 us, 2500, where they are busy 62% of the time and 4.6 us go to a
// tile's beginning and end.  fp32 results: 214 us, 1285 TFLOP/s.

typedef float f32x16 __attribute__((ext_vector_type(16)));

// Until all but the last LEFT of this wave's loads have landed, and all waves
// are here with their reads of LDS done.
template <int LEFT>
__device__ __forceinline__ void land()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LEFT) : "memory");
}

template <int F, int ROWS, int WAVES>
struct Panel { // an operand's step
    static constexpr int kBytes = ROWS * 128, kLoads = ROWS / 8 / WAVES;

    // Where this lane's pieces of the wave's loads lie, from the first row on.
    static __device__ __forceinline__ void offsets(uint32_t (&at)[kLoads], int wave, int lane,
                                                   int64_t pitch)
    {
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
            const int line = 8 * (kLoads * wave + q) + lane / 8;
            const int row = line ^ Order<F>::change(line / F);
            const int piece = (lane & 7) ^ Order<F>::turn(line / F);
            at[q] = (uint32_t)(row * pitch) + 16 * piece;
        }
    }

    // Where this lane's F lines begin, with its turn: what to xor for a piece.
    static __device__ __forceinline__ uint32_t lines(int half, int lane)
    {
        const int r = lane & 31;
        return (32 * half + r) * F * 128 + 128 * Order<F>::change(r) +
               16 * (Order<F>::turn(r) ^ (lane >> 5 << 1));
    }

    // Half u of fragment i.
    static __device__ __forceinline__ i32x8 fragment(uint32_t at, int u, int i)
    {
        const uint32_t of = 128 * (i & 1) + 64 * u, beyond = 128 * (i & ~1);
        const u32x4 a = *(const lds_u32x4 *)(uintptr_t)((at ^ of) + beyond);
        const u32x4 b = *(const lds_u32x4 *)(uintptr_t)((at ^ (of + 16)) + beyond);
        i32x8 f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[k] = (int)a[k];
            f[4 + k] = (int)b[k];
        }
        return f;
    }
};

// What work item `number` of a grid is: a tile, and a part of the depth.  Each
// XCD takes a contiguous run, and runs go down groups of kGroup tiles before
// they go across, so that the blocks at work on an XCD share rows and columns
// in its L2.
struct Item {
    int32_t tm, tn, split, first, end; // blocks of the depth from first to end
};
constexpr int kGroup = 4;
__device__ __forceinline__ Item item_of(uint32_t number, const Product &a)
{
    const uint32_t tiles = a.by_tiles.d, total = tiles * a.splits, xcd = number % 8;
    const uint32_t at = xcd * (total / 8) + min(xcd, total % 8) + number / 8;
    Item w;
    w.split = (int32_t)divide(at, a.by_tiles);
    uint32_t t = at - w.split * tiles;
    const uint32_t group = divide(t, a.by_group), first = group * kGroup;
    t -= group * a.by_group.d;
    const uint32_t high = min(a.tiles_m - first, (uint32_t)kGroup);
    w.tn = (int32_t)(high == kGroup ? t / kGroup : divide(t, a.by_rest));
    w.tm = (int32_t)(first + t - w.tn * high);
    w.first = w.split * a.steps;
    w.end = min(w.first + a.steps, a.blocks);
    return w;
}

// N consecutive results at a byte of a buffer; those past its end are dropped.
constexpr uint32_t kNowhere = 0x80000000u; // past 64 rows of 2^24 bytes
template <typename O, int N>
__device__ __forceinline__ void store_buffer(__amdgpu_buffer_rsrc_t to, uint32_t at,
                                             const float (&v)[N])
{
    if constexpr (sizeof(O) == 4) {
        if constexpr (N == 4)
            __builtin_amdgcn_raw_buffer_store_b128(
                u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3])}, to, (int)at, 0, 0);
        else if constexpr (N == 2)
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(v[0]), __float_as_uint(v[1])},
                                                  to, (int)at, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[0]), to, (int)at, 0, 0);
    } else if constexpr (N == 1) {
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (bf16)v[0]), to, (int)at,
                                              0, 0);
    } else {
        uint32_t w[N / 2];
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
            const bf16x2 h = {(bf16)v[2 * k], (bf16)v[2 * k + 1]};
            w[k] = __builtin_bit_cast(uint32_t, h);
        }
        if constexpr (N == 4)
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{w[0], w[1]}, to, (int)at, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b32(w[0], to, (int)at, 0, 0);
    }
}

// What a tile's kernel needs of LDS: STAGES of both panels and of the exponent
// bytes, of rows first, then of squares, in words.
template <int WM, int WN, int FM, int FN, int STAGES>
struct Stages {
    static constexpr int kWaves = WM * WN, kRows = 32 * FM * WM, kCols = 32 * FN * WN;
    using X = Panel<FM, kRows, kWaves>;
    using W = Panel<FN, kCols, kWaves>;
    static constexpr int kPanels = X::kBytes + W::kBytes, kStage = kPanels + 512;
    static constexpr int kLoads = X::kLoads + W::kLoads; // of a wave, panels alone
    static constexpr uint32_t kLds = STAGES * kStage;
};

// FREE: turns at the end of a step that multiply what has been read already,
// while its panels are given to later loads, and OVER: the turns over which
// those go out (all at once they hold up the MFMAs behind them).
template <int WM, int WN, int FM, int FN, int STAGES, int FREE, int OVER>
struct Shape : Stages<WM, WN, FM, FN, STAGES> {
    static constexpr int kWM = WM, kWN = WN, kFM = FM, kFN = FN, kStages = STAGES;
    static constexpr int kFree = FREE, kOver = OVER;
    static constexpr int kBlocksPerCu = WM * WN == 4 && STAGES == 2 ? 2 : 1;
};

// O: what is stored, y's type, or float where the depth is split.
template <typename S, bool EXACT, typename O>
__global__ __launch_bounds__(64 * S::kWaves, S::kWaves *S::kBlocksPerCu / 4) void k_product_tile(
    const Product a, O *__restrict__ y)
{
    using X = typename S::X;
    using W = typename S::W;
    constexpr int WN = S::kWN, FM = S::kFM, FN = S::kFN, kTurns = 2 * FM, kFree = S::kFree;
    constexpr int kAhead = (S::kStages - 2) * S::kLoads; // may be in flight at a step's end
    extern __shared__ __align__(1024) uint8_t lds[];
    const int lane = threadIdx.x & 63, r = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int32_t total = a.by_tiles.d * a.splits;

    // What is loaded: a step of an item, and where it lies.
    uint32_t x_at[X::kLoads], w_at[W::kLoads];
    X::offsets(x_at, wave, lane, a.x.pitch);
    W::offsets(w_at, wave, lane, a.w.pitch);
    u32x4 x_from, w_from;
    const u32x4 xe_from = descriptor(a.x.exps, 0xFFFFFFFFu);
    const u32x4 we_from = descriptor(a.squares.exps, 0xFFFFFFFFu);
    uint32_t e_at; // wave 0: the rows' exponents, wave 1: the squares'
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_u8 *)lds;
    int32_t number_ahead = blockIdx.x, step_ahead, end_ahead; // below 2^31 + the grid
    uint32_t to = lds0; // the stage
    const auto aim = [&]() GQT_INLINE {
        const Item w = item_of(number_ahead, a);
        const int64_t row0 = (int64_t)w.tm * S::kRows;
        const int32_t col0 = w.tn * S::kCols;
        const uint32_t rows = (uint32_t)min(a.m - row0, (int64_t)S::kRows);
        const uint32_t cols = (uint32_t)min(a.cols - col0, S::kCols);
        x_from = descriptor(a.x.codes + row0 * a.x.pitch, rows * (uint32_t)a.x.pitch);
        w_from = descriptor(a.w.codes + col0 * a.w.pitch, cols * (uint32_t)a.w.pitch);
        // rows past the last have no bytes of their own: they are not stored
        e_at = wave == 0 ? (uint32_t)min(row0 + 4 * lane, a.epitch - 4)
                         : (uint32_t)(min((col0 >> 7) + lane, (a.cols - 1) >> 7) * a.squares.by_cols);
        step_ahead = w.first;
        end_ahead = w.end;
    };
    // Loads `first` to `end` of the step's S::kLoads; two of the waves have one
    // more.
    const auto load = [&](int first, int end) GQT_INLINE {
#pragma unroll
        for (int c = 0; c < S::kLoads; ++c) {
            if (c < first || c >= end)
                continue;
            if (c < X::kLoads)
                load_lds16(to + 1024 * (X::kLoads * wave + c), x_from, x_at[c], 128 * step_ahead);
            else
                load_lds16(to + X::kBytes + 1024 * (W::kLoads * wave + c - X::kLoads), w_from,
                           w_at[c - X::kLoads], 128 * step_ahead);
        }
    };
    const auto load_exponents = [&]() GQT_INLINE {
        if (wave == 0)
            load_lds4(to + S::kPanels, xe_from, e_at, (uint32_t)(step_ahead * a.epitch));
        else if (wave == 1)
            load_lds1(to + S::kPanels + 256, we_from, e_at, step_ahead * a.squares.by_depth);
    };
    const auto advance = [&]() GQT_INLINE {
        to = to == lds0 + (S::kStages - 1) * S::kStage ? lds0 : to + S::kStage;
        if (++step_ahead >= end_ahead) {
            number_ahead += gridDim.x;
            if (number_ahead < total) {
                aim();
            } else { // nothing is left: zeros that nobody reads
                x_from[2] = w_from[2] = 0;
                step_ahead = end_ahead = 0;
            }
        }
    };

    // What is read: the places of this lane's lines and bytes in a stage.
    const uint32_t xs = lds0 + X::lines(wm, lane), ws = lds0 + X::kBytes + W::lines(wn, lane);
    const uint8_t *const xe = lds + S::kPanels + 32 * FM * wm + FM * r;
    const uint8_t *const we = lds + S::kPanels + 256 + 4 * (32 * FN * wn >> 7);
    constexpr int kRing = kFree == 2 ? 3 : 2;
    i32x8 fx[kRing], fw[2][FN]; // x's fragments in turn, w's of the two halves
    Bytes<FM> ex;
    uint32_t ew;

    constexpr auto share = [](int turn) { // loads that have gone out before a turn
        return std::min(S::kLoads * turn / S::kOver, S::kLoads);
    };
    aim();
#pragma unroll
    for (int s = 0; s < S::kStages; ++s) {
        load_exponents();
        load(0, s < S::kStages - 1 ? S::kLoads : share(kFree));
        if (s < S::kStages - 1)
            advance();
    }
    land<kAhead + share(kFree)>();
#pragma unroll
    for (int j = 0; j < FN; ++j)
        fw[0][j] = W::fragment(ws, 0, j);
    fx[0] = X::fragment(xs, 0, 0);
    ex = *reinterpret_cast<const Bytes<FM> *>(xe);
    ew = *reinterpret_cast<const uint32_t *>(we);
    uint32_t now = 0; // the stage
    for (int32_t number = blockIdx.x; number < total; number += gridDim.x) {
        const Item w = item_of(number, a);
        f32x16 acc[FM][FN] = {};
        for (int32_t s = w.first; s < w.end; ++s) {
            const uint32_t next = now == (S::kStages - 1) * S::kStage ? 0 : now + S::kStage;
            Bytes<FM> next_ex;
            uint32_t next_ew;
            bf16x8 wide[EXACT ? FN : 1][4];
            // Turn t multiplies fragment t % FM of half t / FM, while those of
            // the turns behind it are read.  Before the last kFree all of this
            // step has been read, and all of the next has landed; where this
            // one lay goes the one kStages after.
#pragma unroll
            for (int t = 0; t < kTurns; ++t) {
                const int u = t / FM, i = t % FM, out = t - (kTurns - kFree);
                if (out == 0) {
                    land<kAhead>();
                    advance();
                    load_exponents();
                }
                load(share(out < 0 ? t + kFree : out), share(out < 0 ? t + kFree + 1 : out + 1));
                if (out < -1 || (kFree == 1 && out == -1))
                    fx[(t + 1) & 1] = X::fragment(xs + now, (t + 1) / FM, (t + 1) % FM);
                if (kFree == 2 && out == -1) {
                    fx[0] = X::fragment(xs + now, 1, FM - 2);
                    fx[kRing - 1] = X::fragment(xs + now, 1, FM - 1);
                }
                if (t == kTurns - 1) {
                    fx[0] = X::fragment(xs + next, 0, 0);
                    next_ex = *reinterpret_cast<const Bytes<FM> *>(xe + next);
                    next_ew = *reinterpret_cast<const uint32_t *>(we + next);
                }
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    if (t == j * FM / FN)
                        fw[1][j] = W::fragment(ws + now, 1, j);
                    if (out == kFree * j / FN)
                        fw[0][j] = W::fragment(ws + next, 0, j);
                }
                const i32x8 &x = fx[t == kTurns - 1 ? kRing - 1 : t & 1];
                if constexpr (EXACT) {
                    if (i == 0) {
#pragma unroll
                        for (int j = 0; j < FN; ++j)
#pragma unroll
                            for (int part = 0; part < 4; ++part)
                                wide[j][part] = widen(fw[u][j], part, step_of(ew));
                    }
#pragma unroll
                    for (int part = 0; part < 4; ++part) {
                        const bf16x8 bx = widen(x, part, step_of(ex.byte(i)));
#pragma unroll
                        for (int j = 0; j < FN; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                                bx, wide[j][part], acc[i][j], 0, 0, 0);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < FN; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                            x, fw[u][j], acc[i][j], 0, 0, 0, (int)ex.byte(i), 0, (int)ew);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            ex = next_ex;
            ew = next_ew;
            now = next;
        }

        const int32_t col = w.tn * S::kCols + 32 * FN * wn + FN * r;
        O *const out = y + (int64_t)w.split * a.m * a.cols; // split 0 unless O are partial sums
        float bias[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j)
            bias[j] = a.bias && col + j < a.cols ? bias_at(a.bias, a.bias_dtype, col + j) : 0.0f;
        // waits for them here: where no row is stored the next item's first
        // steps would, and for all their own loads with them
#pragma unroll
        for (int j = 0; j < FN; ++j)
            asm volatile("" : "+v"(bias[j]));
        // The wave's rows by a descriptor that ends with the last: what lies
        // past it, or is put there, is not stored.
        const int64_t row0 = (int64_t)w.tm * S::kRows + 32 * FM * wm;
        const uint32_t pitch = (uint32_t)a.cols * sizeof(O);
        const auto rows = __builtin_amdgcn_make_buffer_rsrc(
            out + row0 * a.cols, 0, (int)(max(min(a.m - row0, (int64_t)32 * FM), (int64_t)0) * pitch),
            0x00020000);
        const int32_t left = a.cols - col;
        const auto store = [&](auto to_row) GQT_INLINE {
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    float v[FN];
#pragma unroll
                    for (int j = 0; j < FN; ++j)
                        v[j] = acc[i][j][q] + bias[j];
                    to_row((FM * (8 * (q / 4) + q % 4) + i) * pitch, v);
                }
        };
        const uint32_t lane_at = FM * 4 * (lane >> 5) * pitch + (uint32_t)col * sizeof(O);
        const uint32_t whole = left >= FN ? lane_at : kNowhere;
        store([&](uint32_t row_at, const float (&v)[FN]) GQT_INLINE {
            store_buffer<O>(rows, whole + row_at, v);
        });
        if (FN > 1 && (w.tn + 1) * S::kCols > a.cols && a.cols % FN) // the last columns' rest
            store([&](uint32_t row_at, const float (&v)[FN]) GQT_INLINE {
#pragma unroll
                for (int j = 0; j < FN - 1; ++j) {
                    const float one[1] = {v[j]};
                    const uint32_t at = lane_at + j * (uint32_t)sizeof(O);
                    store_buffer<O>(rows, (left < FN && j < left ? at : kNowhere) + row_at, one);
                }
            });
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); // nothing may land in LDS after the end
}

// Adds the parts' sums of a row, in their order, and the bias: 2 to 4 us where
// the depth is split.
constexpr int kSumColumns = 4;
__device__ __forceinline__ void store_sums(bf16 *p, const float (&v)[kSumColumns])
{
    const bf16x2 lo = {(bf16)v[0], (bf16)v[1]}, hi = {(bf16)v[2], (bf16)v[3]};
    *reinterpret_cast<u32x2_e2 *>(p) =
        u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
}
__device__ __forceinline__ void store_sums(float *p, const float (&v)[kSumColumns])
{
    *reinterpret_cast<u32x4_e4 *>(p) = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]),
                                             __float_as_uint(v[2]), __float_as_uint(v[3])};
}
template <typename O>
__global__ __launch_bounds__(kThreads) void k_sum_splits(const Product a, O *__restrict__ y)
{
    const int32_t col = kSumColumns * (blockIdx.x * kThreads + threadIdx.x);
    const int64_t row = blockIdx.y;
    if (col >= a.cols)
        return;
    const float *p = a.parts + row * a.cols + col;
    float v[kSumColumns] = {};
    if (col + kSumColumns <= a.cols) {
        for (int z = 0; z < a.splits; ++z, p += a.m * a.cols) {
            const u32x4 w = *reinterpret_cast<const u32x4_e4 *>(p);
#pragma unroll
            for (int k = 0; k < kSumColumns; ++k)
                v[k] += bits_f32(w[k]);
        }
    } else {
        for (int z = 0; z < a.splits; ++z, p += a.m * a.cols)
#pragma unroll
            for (int k = 0; k < kSumColumns; ++k)
                if (col + k < a.cols)
                    v[k] += p[k];
    }
#pragma unroll
    for (int k = 0; k < kSumColumns; ++k)
        if (a.bias && col + k < a.cols)
            v[k] += bias_at(a.bias, a.bias_dtype, col + k);
    O *const out = y + row * a.cols + col;
    if (col + kSumColumns <= a.cols) {
        store_sums(out, v);
    } else {
#pragma unroll
        for (int k = 0; k < kSumColumns; ++k)
            if (col + k < a.cols)
                store_one(out + k, v[k]);
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
    if (rows * blocks_of(d) >= kMaxBlocks)
        return fail(GQ_ERR_UNSUPPORTED, "%lld rows of %lld columns: 2^27 blocks or more",
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
    const FastDiv across = fast_div((uint32_t)((blocks_of(d) + kRowBlocks - 1) / kRowBlocks));
    const uint32_t grid = (uint32_t)((rows + 15) / 16) * across.d;
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

template <typename T, int F, bool MADE>
int32_t launch_direct(Product a, T *y, hipStream_t st)
{
    a.by_tiles = fast_div((uint32_t)((a.cols + 15) / 16)); // of a row of them
    const int64_t grid = (a.m + 16 * F - 1) / (16 * F) * a.by_tiles.d;
    const int waves = std::min(F > 2 ? 8 : 16, a.blocks);
    const uint32_t lds = (uint32_t)(waves * (Strip<F>::kBytes + Strip<1>::kBytes));
    if (grid >= ((int64_t)1 << 31) / (64 * 16))
        return fail(GQ_ERR_UNSUPPORTED, "%lld tiles", (long long)grid);
    GQT_TRY(allow_lds(&k_product_direct<T, F, MADE>, "k_product_direct", lds));
    k_product_direct<T, F, MADE><<<(uint32_t)grid, 64 * waves, lds, st>>>(a, y);
    return check_launch("k_product_direct");
}

constexpr int kCUs = 256;

// What takes a product: fragments straight from memory, or tiles of a shape,
// with the depth in `splits` parts where that fills the card.
enum Way { kDirect, kRows64, kSquare128, kSquare128x2, kSquare256, kWide256, kWays };
struct Plan {
    Way way;
    int32_t splits;
    int64_t bytes; // of the workspace
};

using Rows64 = Shape<2, 4, 1, 1, 4, 1, 2>;
using Square128 = Shape<4, 2, 1, 2, 4, 1, 2>;
using Square128x2 = Shape<2, 2, 2, 2, 2, 1, 2>;
using Square256 = Shape<4, 2, 2, 4, 2, 2, 2>;
using Wide256 = Shape<4, 2, 2, 2, 3, 1, 2>;

// The measured microseconds of a way: a block of the depth, and a tile's
// beginning and end, while at most `at_once` tiles are at work.
struct Cost {
    int32_t rows, cols, at_once;
    float step, tile;
};
constexpr Cost kCosts[2][kWays] = {
    // exact products of fp32 results
    {{}, {64, 128, kCUs, 0.62f, 1.5f}, {128, 128, kCUs, 0.95f, 2.6f}, {}, {},
     {256, 128, kCUs, 1.57f, 4.1f}},
    // 8-bit products of bf16 ones
    {{}, {64, 128, kCUs, 0.34f, 1.1f}, {128, 128, kCUs, 0.55f, 1.2f},
     {128, 128, 2 * kCUs, 0.9f, 3.6f}, {256, 256, kCUs, 1.6f, 4.6f}, {}},
};
constexpr Cost kDirectCosts[4] = { // of 32, 64, 96 and 128 rows
    {32, 16, kCUs, 0.08f, 0.2f},
    {64, 16, kCUs, 0.13f, 0.2f},
    {96, 16, kCUs, 0.2f, 0.9f},
    {128, 16, kCUs, 0.24f, 1.7f}};

// What costs least: rounds of tiles, and, where the depth is split, a second
// kernel that adds up the parts.  Microseconds in a graph, the ways forced: bf16
// 4096 x 1024 x 1024 Rows64 11.3, Square128 9.2, Square128x2 10.7, Square256
// 17.7; 2048 x 4096 x 4096 53, 40, 36, 51; 8192 x 4096 x 1024 71, 51, 50, 38;
// 512 x 4096 x 4096 15.6, 20.9, 24.7, 29.  fp32 8192 x 4096 x 1024 Rows64 110,
// Square128 83, Wide256 70; 1024 x 4096 x 4096 46, 36, 42.  Directly and by the
// best tiles: bf16 64 x 4096 x 4096 7.8, 10.9; 128 x 4096 x 4096 11.5, 13.7
// (96 rows in a kernel for 96 10.7, in one for 128 0.8 to 2 more);
// 256 x 4096 x 4096 20.3, 13.9; 64 x 8192 x 8192 19.1, 17.5.
Plan plan_of(int64_t m, int64_t cols, int64_t depth, int32_t dtype)
{
    const int64_t blocks = blocks_of(depth);
    Plan best{kDirect, 1, 0};
    if (m <= 16)
        return best;
    const auto tiles_of = [&](const Cost &c) {
        return ((m + c.rows - 1) / c.rows) * ((cols + c.cols - 1) / c.cols);
    };
    const auto time = [&](const Cost &c, int64_t z, float step) {
        const int64_t rounds = (tiles_of(c) * z + c.at_once - 1) / c.at_once;
        const float sums = z > 1 ? 3.5f + (float)(z * m * cols) * 1.5e-6f : 0.0f;
        return (float)rounds * ((float)((blocks + z - 1) / z) * step + c.tile) + sums;
    };
    // few blocks of direct loads have more of the L2 each
    const Cost &direct = kDirectCosts[std::min<int64_t>((m - 1) / 32, 3)];
    const float full = std::min(1.0f, (float)tiles_of(direct) / (float)kCUs);
    float least = time(direct, 1, direct.step * (0.55f + 0.45f * full));
    for (int way = kRows64; way < kWays; ++way) {
        const Cost &c = kCosts[dtype == GQ_IN_BF16][way];
        if (!c.at_once)
            continue;
        for (int32_t z = 1; z <= 16 && z <= blocks; ++z) {
            if (z > 1 && tiles_of(c) * z > c.at_once)
                break;
            const float us = time(c, z, c.step);
            if (us < least) {
                least = us;
                best = {(Way)way, z, z > 1 ? 4 * z * m * cols : 0};
            }
        }
    }
    return best;
}

template <typename S, bool EXACT, typename O>
int32_t launch_tile(const Product &a, O *y, hipStream_t st)
{
    const int64_t items = (int64_t)a.by_tiles.d * a.splits;
    GQT_TRY(allow_lds(&k_product_tile<S, EXACT, O>, "k_product_tile", S::kLds));
    k_product_tile<S, EXACT, O>
        <<<(uint32_t)std::min<int64_t>(items, kCUs * S::kBlocksPerCu), 64 * S::kWaves, S::kLds,
           st>>>(a, y);
    return check_launch("k_product_tile");
}

template <typename S, typename T>
int32_t launch_tiles(Product a, T *y, hipStream_t st)
{
    constexpr bool kExact = sizeof(T) == 4;
    const int64_t tiles_m = (a.m + S::kRows - 1) / S::kRows;
    const int64_t tiles_n = (a.cols + S::kCols - 1) / S::kCols;
    if (tiles_m * tiles_n >= ((int64_t)1 << 31) - 2 * kCUs)
        return fail(GQ_ERR_UNSUPPORTED, "%lld tiles", (long long)(tiles_m * tiles_n));
    a.tiles_m = (uint32_t)tiles_m;
    a.by_tiles = fast_div((uint32_t)(tiles_m * tiles_n));
    a.by_group = fast_div((uint32_t)(kGroup * tiles_n));
    a.by_rest = fast_div((uint32_t)std::max<int64_t>(tiles_m % kGroup, 1));
    a.steps = (a.blocks + a.splits - 1) / a.splits;
    a.splits = (a.blocks + a.steps - 1) / a.steps; // none is empty
    if (a.splits == 1)
        return launch_tile<S, kExact, T>(a, y, st);
    Product part = a;
    part.bias = nullptr;
    GQT_TRY((launch_tile<S, kExact, float>(part, a.parts, st)));
    const uint32_t across = (uint32_t)((a.cols + kSumColumns * kThreads - 1) / (kSumColumns * kThreads));
    k_sum_splits<T><<<dim3(across, (uint32_t)a.m), kThreads, 0, st>>>(a, y);
    return check_launch("k_sum_splits");
}

template <typename T>
int32_t launch_product(const Product &a, Way way, void *y, hipStream_t st)
{
    T *const out = (T *)y;
    switch (way) {
    case kRows64:
        return launch_tiles<Rows64>(a, out, st);
    case kSquare128:
        return launch_tiles<Square128>(a, out, st);
    case kSquare128x2:
        if constexpr (sizeof(T) == 2)
            return launch_tiles<Square128x2>(a, out, st);
        break;
    case kSquare256:
        if constexpr (sizeof(T) == 2)
            return launch_tiles<Square256>(a, out, st);
        break;
    case kWide256:
        if constexpr (sizeof(T) == 4)
            return launch_tiles<Wide256>(a, out, st);
        break;
    default:
        break;
    }
    if (a.m <= 16)
        return a.raw ? launch_direct<T, 1, true>(a, out, st)
                     : launch_direct<T, 1, false>(a, out, st);
    if (a.m <= 32)
        return launch_direct<T, 2, false>(a, out, st);
    if (a.m <= 64)
        return launch_direct<T, 4, false>(a, out, st);
    if (a.m <= 96)
        return launch_direct<T, 6, false>(a, out, st);
    return launch_direct<T, 8, false>(a, out, st);
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
int64_t plan_bytes(const Plan &p) { return (p.bytes + 15) / 16 * 16; }
int64_t linear_bytes(const Plan &p, int64_t m, int64_t depth)
{
    return made_on_the_way(m) ? p.bytes
                              : plan_bytes(p) + codes_bytes(m, depth) + exps_bytes(m, depth);
}

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

// Runs it by its plan, whose workspace comes first.
int32_t run_product(Product a, const Plan &plan, void *y, int32_t dtype, void *workspace,
                    hipStream_t st)
{
    a.splits = plan.splits;
    a.parts = (float *)workspace;
    return dtype == GQ_IN_F32 ? launch_product<float>(a, plan.way, y, st)
                              : launch_product<bf16>(a, plan.way, y, st);
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
    GQT_TRY(check_codes("codes", codes, rows > 0));
    if (!exps && rows > 0)
        return fail(GQ_ERR_NULL, "exps is NULL");
    GQT_TRY(check_matrix("out", out, dtype, rows));
    if (rows == 0)
        return ok();
    const FastDiv per_row = fast_div((uint32_t)((d + 7) / 8));
    const uint32_t chunks = (uint32_t)rows * per_row.d;
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
    return plan_of(m, cols, depth, dtype).bytes;
}

int32_t gqs_fp8_product(const void *x_codes, const void *x_exps, int64_t m, const void *w_codes,
                        const void *w_exps, int64_t cols, int64_t depth, int32_t transposed,
                        const void *bias, int32_t bias_dtype, void *y, int32_t dtype,
                        void *workspace, int64_t workspace_bytes, void *stream)
{
    GQT_TRY(check_product(dtype, m, cols, depth, w_codes, w_exps, bias, bias_dtype, y));
    GQT_TRY(check_codes("x_codes", x_codes, m > 0));
    GQT_TRY(check_codes("x_exps", x_exps, m > 0));
    const Plan plan = plan_of(m, cols, depth, dtype);
    GQT_TRY(check_workspace(plan.bytes, workspace, workspace_bytes));
    if (m == 0)
        return ok();
    Product a = product_of(m, w_codes, w_exps, cols, depth, transposed, bias, bias_dtype);
    a.x = {(const uint8_t *)x_codes, (const uint8_t *)x_exps, fp8_pitch(depth)};
    a.epitch = exp_pitch(m);
    return run_product(a, plan, y, dtype, workspace, (hipStream_t)stream);
}

int64_t gqs_fp8_linear_workspace_bytes(int64_t m, int64_t cols, int64_t depth, int32_t dtype)
{
    if (check_sides(dtype, m, depth) != GQ_OK || check_sides(dtype, m, cols) != GQ_OK)
        return -1;
    return linear_bytes(plan_of(m, cols, depth, dtype), m, depth);
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
    const Plan plan = plan_of(m, cols, depth, dtype);
    GQT_TRY(check_workspace(linear_bytes(plan, m, depth), workspace, workspace_bytes));
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
        uint8_t *const codes = (uint8_t *)workspace + plan_bytes(plan);
        uint8_t *const exps = codes + codes_bytes(m, depth);
        GQT_TRY(launch_rows(x, dtype, m, depth, ldx, rounding, seed, codes, exps, st));
        a.x = {codes, exps, fp8_pitch(depth)};
        a.epitch = exp_pitch(m);
    }
    return run_product(a, plan, y, dtype, workspace, st);
}

} // extern "C"
