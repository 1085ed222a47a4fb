// weight_grad.hip -- dw = dy^T x and db of a linear layer on MI355X (gfx950),
// with x in the 8-bit format of include/gq_train.h.
//
// Both operands are stored with the summed axis (the tokens) outermost, and
// an MFMA fragment is eight tokens of one column.  No transposing through
// LDS is needed for that: a lane that loads eight columns of eight tokens
// holds, column by column, eight fragments' parts, and which of the 16 rows
// or columns of an MFMA stands for which column of the matrix is free.  So
// lane i of a row of 16 takes columns 8 i to 8 i + 7; fragment c is column
// 8 i + c, put together by four byte permutes of pairs of tokens (dy), or by
// the permutes that narrow the decoded codes to bf16 (x).  A code times its
// group's power of two is exact in bf16; an fp32 dy is the sum of three bf16
// parts (exact from 2^-110 on, where its last bit is bf16's last place, 2^-133)
// and takes three MFMAs.  All sums are fp32.
//
// What bounds it is the work around the MFMAs: a wave spends as long decoding
// codes, pairing tokens and waiting as multiplying.  8192 x 4096 x 1024 bf16
// (tokens, rows and columns of dw) takes 76 us a call, 910 TFLOP/s, with the
// matrix cores busy 36 % of the time (profiled); the library's product of bf16 operands,
// x restored before, takes 91 us.  fp32 8192 x 2048 x 2048: 184 us, 373
// TFLOP/s counting one product a value, three times that in MFMAs (library
// 457 us).
#include "train_common.h"

namespace gqt {
namespace {

constexpr int kTile = 128;  // output tile: 128 rows and 128 columns of dw
constexpr int kWaves = 4;   // one per SIMD: a wave's sums take half its registers
constexpr int kWaveM = 32;  // tokens of a wave in a step: the depth of one MFMA
constexpr int kThreads = 64 * kWaves;

#define GQT_INLINE __attribute__((always_inline))

typedef uint32_t u32_e1 __attribute__((aligned(1)));
typedef u32x2 u32x2_e2 __attribute__((aligned(2)));
typedef bf16 bf16x4 __attribute__((ext_vector_type(4)));

template <typename T>
constexpr int parts() { return sizeof(T) == 4 ? 3 : 1; }

// Eight tokens of eight columns of dy as loaded: token j in a[j].
template <typename T>
struct RawDy {
    u32x4 a[8][sizeof(T) / 2];
};
// and of x: codes, and for one of the tokens (lane i of 16: token i % 8) the
// exponents of the tile's four groups.  One load a lane: byte loads of each
// token's own exponent took longer than all the others together.
struct RawX {
    u32x2 b[8];
    uint32_t e;
};

__device__ __forceinline__ u32x4 load16(const bf16 *p)
{
    return *reinterpret_cast<const u32x4_e2 *>(p);
}
__device__ __forceinline__ u32x4 load16(const float *p)
{
    return *reinterpret_cast<const u32x4_e4 *>(p);
}
// the upper halves of a pair of words
__device__ __forceinline__ uint32_t upper_halves(uint32_t lo, uint32_t hi)
{
    return __builtin_amdgcn_perm(hi, lo, 0x07060302u);
}

__device__ __forceinline__ bf16x8 as_fragment(u32x4 w) { return __builtin_bit_cast(bf16x8, w); }

// Fragment c of dy in its bf16 parts.
__device__ __forceinline__ void dy_fragment(const RawDy<bf16> &l, int c, u32x4 (&part)[1])
{
#pragma unroll
    for (int h = 0; h < 4; ++h)
        part[0][h] = __builtin_amdgcn_perm(l.a[2 * h + 1][0][c / 2], l.a[2 * h][0][c / 2],
                                           c % 2 ? 0x07060302u : 0x05040100u);
}

// A float's leading 8, middle 8 and last 8 significant bits: truncated, so
// that each rest is exact.  Below 2^-110 the last part drops what lies under
// 2^-133; subnormal parts count in the MFMA as they are.  An inf stays in the
// first part alone; a NaN's rest is one too.
__device__ __forceinline__ void dy_fragment(const RawDy<float> &l, int c, u32x4 (&part)[3])
{
    uint32_t b[3][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float v = bits_f32(l.a[j][c / 4][c % 4]);
        b[0][j] = __float_as_uint(v);
        const float rest = v - bits_f32(b[0][j] & 0xFFFF0000u);
        const float r1 = __builtin_isinf(v) ? 0.0f : rest;
        b[1][j] = __float_as_uint(r1);
        b[2][j] = __float_as_uint(r1 - bits_f32(b[1][j] & 0xFFFF0000u));
    }
#pragma unroll
    for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int h = 0; h < 4; ++h)
            part[p][h] = upper_halves(b[p][2 * h], b[p][2 * h + 1]);
}

// Adds the eight tokens of each column to its sum.
__device__ __forceinline__ void add_tokens(const RawDy<bf16> &l, float (&sum)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            sum[2 * c] += bits_f32(l.a[j][0][c] << 16);
            sum[2 * c + 1] += bits_f32(l.a[j][0][c] & 0xFFFF0000u);
        }
}
__device__ __forceinline__ void add_tokens(const RawDy<float> &l, float (&sum)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int c = 0; c < 8; ++c)
            sum[c] += bits_f32(l.a[j][c / 4][c % 4]);
}

// The eight tokens' scales.  `up` moves the lane's own group's exponent to
// the top byte.  255 makes an infinity, which inf 0 + inf turns into the NaN
// it stands for.
struct Steps {
    float of[8];
};
__device__ __forceinline__ Steps steps_of(const RawX &l, uint32_t up)
{
    Steps s;
#define GQT_TOKEN(J) /* from lane J of each 16 */                                              \
    do {                                                                                       \
        const uint32_t e = (uint32_t)__builtin_amdgcn_mov_dpp((int)l.e, 0x150 + J, 0xF, 0xF,   \
                                                              true);                           \
        const float step = bits_f32(((e << up) >> 1) & 0x7F800000u);                           \
        s.of[J] = fmaf(step, 0.0f, step);                                                      \
    } while (0)
    GQT_TOKEN(0);
    GQT_TOKEN(1);
    GQT_TOKEN(2);
    GQT_TOKEN(3);
    GQT_TOKEN(4);
    GQT_TOKEN(5);
    GQT_TOKEN(6);
    GQT_TOKEN(7);
#undef GQT_TOKEN
    return s;
}

// Frees `from` for the next loads.  (Two buffers in turn would save the copy,
// but a loop of two steps has the compiler move the sums between registers.
// In assembly, so that it stays where it is.)
__device__ __forceinline__ void copy_codes(RawX &to, const RawX &from)
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            asm("v_mov_b32 %0, %1" : "=v"(to.b[j][h]) : "v"(from.b[j][h]));
}

// Byte B of w as a signed number, in one instruction (the compiler takes
// two).  w comes from memory and all of the result is written, so no
// forwarding hazard has to be known for it.
template <int B>
__device__ __forceinline__ float code_f32(uint32_t w)
{
    float f;
    if (B == 0)
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_0"
            : "=v"(f) : "v"(w));
    else if (B == 1)
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_1"
            : "=v"(f) : "v"(w));
    else if (B == 2)
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_2"
            : "=v"(f) : "v"(w));
    else
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_3"
            : "=v"(f) : "v"(w));
    return f;
}

// Fragment c of x: its code times its step, exact in bf16.
__device__ __forceinline__ u32x4 x_fragment(const RawX &l, const Steps &s, int c)
{
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t w = l.b[j][c / 4];
        f[j] = s.of[j] * (c % 4 == 0   ? code_f32<0>(w)
                          : c % 4 == 1 ? code_f32<1>(w)
                          : c % 4 == 2 ? code_f32<2>(w)
                                       : code_f32<3>(w));
    }
    u32x4 r;
#pragma unroll
    for (int h = 0; h < 4; ++h)
        r[h] = upper_halves(__float_as_uint(f[2 * h]), __float_as_uint(f[2 * h + 1]));
    return r;
}

__device__ __forceinline__ void decode(const RawX &l, uint32_t up, u32x4 (&f)[8])
{
    const Steps s = steps_of(l, up);
#pragma unroll
    for (int c = 0; c < 8; ++c)
        f[c] = x_fragment(l, s, c);
}

// Asks the scheduler for MFMAS times one MFMA and VALU vector instructions,
// and keeps what follows behind them: left alone it brings all the decoding
// forward and runs out of registers.
template <int MFMAS, int VALU>
__device__ __forceinline__ void interleave()
{
#pragma unroll
    for (int i = 0; i < MFMAS; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
}

constexpr int step_tokens(bool shared) { return shared ? kWaves * kWaveM : kWaveM; }

struct Tiles {
    int32_t n, k, total; // tiles along n and k, and blocks (times the splits)
};

// A wave holds a 128 x 128 tile of dw.  Either (SHARED) the four waves of a
// block have one tile, each takes 32 of a step's 128 tokens, and their sums
// are added at the end; or they have the four tiles of a 256 x 256 square and
// the same 32 tokens, which asks half as much of the L2 and ends without a
// word between them, but leaves fewer blocks.  Which, plan_of estimates; us a
// call for bf16, shared against squares: 8192 x 4096 x 4096 294, 262; 512 x
// 4096 x 4096 49, 37; 8192 x 4096 x 1024 76, 93; 1000 x 1001 x 777 18, 28.
// out: dw itself (one split of the tokens) or the split's fp32 partial.
//
// Rows of the tile past n, and columns past the codes' pitch, are not
// stored, so what they hold is free: every lane loads eight columns that
// exist.  The lane whose eight would end past n (n >= 8) takes the last eight
// of the row, and so computes some rows that its neighbour stores.
//
// db: the tiles that share a tile's columns of dy take turns at adding up
// its steps, so that none is slower than the others, and each leaves a
// partial; or (db_whole) the first of them adds up all.
template <typename T, typename O, bool SHARED>
__global__ __launch_bounds__(kThreads, 1) void k_weight_grad(
    const T *__restrict__ dy, int64_t m, int32_t n, int64_t lddy, Act8 x, int32_t k, int64_t chunk,
    Tiles tiles, O *__restrict__ dw, float *__restrict__ db_part, O *__restrict__ db_whole)
{
    constexpr int P = parts<T>(), kLoads = sizeof(T) / 2; // 16-byte loads of eight columns
    constexpr int kStepM = step_tokens(SHARED), kSide = SHARED ? 1 : 2;
    __shared__ __align__(16) float lds[SHARED ? kTile * kTile / 2 * kWaves : 1];
    // Blocks go to the 8 XCDs in turn; each XCD takes a contiguous run of
    // tiles, k fastest, so that its L2 holds the rows of dy they share.
    const int xcd = blockIdx.x % 8, q = tiles.total / 8, rem = tiles.total % 8;
    const int tile = xcd * q + min(xcd, rem) + blockIdx.x / 8;
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tk = tile % tiles.k * kSide + (SHARED ? 0 : wave % 2);
    const int tn = tile / tiles.k % tiles.n * kSide + (SHARED ? 0 : wave / 2);
    const int z = tile / tiles.k / tiles.n;
    const int n0 = tn * kTile, k0 = tk * kTile;
    const int64_t m_begin = (int64_t)z * chunk;
    const int64_t m_end = m_begin + chunk < m ? m_begin + chunk : m;
    const int wave_m = SHARED ? kWaveM * wave : 0; // the wave's tokens in a step

    // the first of the eight rows of dw (columns of dy) of MFMA row r
    const auto first_row = [&](int r) { return min(n0 + 8 * r, n - 8); };
    const int dy_col = first_row(i);
    const int x_col = k0 + 8 * i < x.pitch ? k0 + 8 * i : 0;
    // A load's address is a step's base and a lane's 32-bit offset to token j.
    // The offsets are made opaque at each use, or their widening to 64 bits
    // leaves the loop and every load adds two 64-bit numbers.
    uint32_t dy_at[8], b_at[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        dy_at[j] = ((4 * j + g) * (uint32_t)lddy + dy_col) * (uint32_t)sizeof(T);
        b_at[j] = (4 * j + g) * (uint32_t)x.pitch + x_col;
    }
    // The word of four exponents ends with the row at the latest (with fewer
    // than four groups it begins in the row before).
    const int e_col = min(k0 >> 5, x.groups - 4), e_token = 4 * (i % 8) + g;
    const uint32_t up = 24 - 8 * ((x_col >> 5) - e_col);
    int32_t e_at = e_token * x.groups + e_col;
    // Where the next step's tokens of this wave lie; the last step's again
    // past the end.
    const int64_t row0 = m_begin + wave_m;
    const char *dy_p = reinterpret_cast<const char *>(dy + row0 * lddy);
    const int8_t *codes_p = x.codes + row0 * x.pitch;
    const uint8_t *exps_p = x.exps + row0 * x.groups;
    const int64_t dy_step = kStepM * lddy * (int64_t)sizeof(T), codes_step = kStepM * x.pitch,
                  exps_step = (int64_t)kStepM * x.groups;
    // Part h of dy's token j: its eight columns, or the first or last four.
    const auto load_dy = [&](RawDy<T> &l, int j, int h) GQT_INLINE {
        asm volatile("" : "+v"(dy_at[j]));
        l.a[j][h] = load16(reinterpret_cast<const T *>(dy_p + 16 * h + dy_at[j]));
    };
    const auto load_codes = [&](RawX &l, int j) GQT_INLINE {
        asm volatile("" : "+v"(b_at[j]));
        l.b[j] = *reinterpret_cast<const u32x2 *>(codes_p + b_at[j]);
    };
    // A single step's tokens, which may have no row before them, are loaded
    // again for nothing.
    const auto load_exps = [&](RawX &l) GQT_INLINE {
        l.e = *reinterpret_cast<const u32_e1 *>(exps_p + e_at);
    };

    f32x4 acc[8][8] = {};
    float sum[8] = {};
    // rows c of dw by columns b of it
    const auto mfma = [&](u32x4 fy, u32x4 fx, int c, int b) GQT_INLINE {
        acc[c][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_fragment(fy), as_fragment(fx),
                                                            acc[c][b], 0, 0, 0);
    };

    // While step s is multiplied, dy of step s + 1 and x of step s + 2 are
    // loaded; past the last step the last one is loaded again.  Rows further
    // apart than a lane's offset reaches and tokens that do not fill a step
    // come last, one step at a time.
    const int steps = lddy < ((int64_t)1 << 24) ? (int)((m_end - m_begin) / kStepM) : 0;
    // the step whose tokens this tile adds up next, and the one after
    int next_sum = db_part ? tk : db_whole && tk == 0 ? 0 : -1;
    const int turn = db_part ? tiles.k * kSide : 1;
    RawDy<T> ry;
    RawX rx0, rx1;
    if (steps > 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
            for (int h = 0; h < kLoads; ++h)
                load_dy(ry, j, h);
            load_codes(rx0, j);
        }
        const int64_t first = row0 * x.groups + e_at, at = max(first, (int64_t)0);
        rx0.e = *reinterpret_cast<const u32_e1 *>(x.exps + at) << (8 * (at - first));
        if (steps == 1)
            e_at = max(e_at, 0);
        const auto advance_x = [&](bool more) GQT_INLINE {
            codes_p += more ? codes_step : 0;
            exps_p += more ? exps_step : 0;
        };
        advance_x(steps > 1);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            load_codes(rx1, j);
        load_exps(rx1);
        // before step s is multiplied
        const auto enter = [&](int s) GQT_INLINE {
            if (s == next_sum) {
                add_tokens(ry, sum);
                next_sum += turn;
            }
            dy_p += s + 1 < steps ? dy_step : 0;
            advance_x(s + 2 < steps);
        };
        if constexpr (P == 1) {
            // x outside: its fragment b + 1 is decoded while fragment b meets
            // the eight of dy, which stay in registers.
            Steps st = steps_of(rx0, up);
            u32x4 fx = x_fragment(rx0, st, 0);
            for (int s = 0; s < steps; ++s) {
                enter(s);
                u32x4 fy[8][1];
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    if (b == 7) {
                        st = steps_of(rx1, up);
                        copy_codes(rx0, rx1);
                    }
                    const u32x4 fx_next = x_fragment(rx0, st, (b + 1) % 8);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        if (b == 0)
                            dy_fragment(ry, c, fy[c]);
                        mfma(fy[c][0], fx, c, b);
                    }
                    fx = fx_next;
                    interleave<8, 3>();
                    if (b == 0)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            load_dy(ry, j, 0);
                    if (b == 7) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            load_codes(rx1, j);
                        load_exps(rx1);
                    }
                }
            }
        } else {
            // dy outside: the parts of its fragment c + 1 are made while
            // fragment c is multiplied, and so is x of the next step.  Four
            // columns of dy done with leave their registers to the next
            // step's.
            u32x4 fx[8], fx_next[8], part[P];
            decode(rx0, up, fx);
            dy_fragment(ry, 0, part);
            for (int s = 0; s < steps; ++s) {
                enter(s);
                const Steps st = steps_of(rx1, up);
                copy_codes(rx0, rx1);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    load_codes(rx1, j);
                load_exps(rx1);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    u32x4 part_next[P];
                    dy_fragment(ry, (c + 1) % 8, part_next);
                    fx_next[c] = x_fragment(rx0, st, c);
#pragma unroll
                    for (int p = 0; p < P; ++p)
#pragma unroll
                        for (int b = 0; b < 8; ++b)
                            mfma(part[p], fx[b], c, b);
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        part[p] = part_next[p];
                    interleave<8 * P, 4>();
                    if (c % 4 == 2)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            load_dy(ry, j, c / 4);
                }
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    fx[c] = fx_next[c];
            }
        }
    }
    // Any tokens: those past the end read as the last one with a dy of 0.
    for (int64_t m0 = m_begin + (int64_t)steps * kStepM; m0 < m_end; m0 += kStepM) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t want = m0 + wave_m + 4 * j + g;
            const int64_t row = want < m_end ? want : m_end - 1;
#pragma unroll
            for (int h = 0; h < kLoads; ++h) {
                ry.a[j][h] = load16(dy + row * lddy + dy_col + 8 / kLoads * h);
                if (want >= m_end)
                    ry.a[j][h] = u32x4{0, 0, 0, 0};
            }
            rx0.b[j] = *reinterpret_cast<const u32x2 *>(x.codes + row * x.pitch + x_col);
        }
        {
            const int64_t want = m0 + wave_m + e_token;
            const int64_t row = want < m_end ? want : m_end - 1;
            rx0.e = 0;
#pragma unroll
            for (int p = 0; p < 4; ++p)
                if (e_col + p >= 0)
                    rx0.e |= (uint32_t)x.exps[row * x.groups + e_col + p] << (8 * p);
        }
        if ((db_part || db_whole) && tk == 0)
            add_tokens(ry, sum);
        u32x4 fx[8];
        decode(rx0, up, fx);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            u32x4 part[P];
            dy_fragment(ry, c, part);
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int b = 0; b < 8; ++b)
                    mfma(part[p], fx[b], c, b);
        }
    }

    // acc[c][b] of lane (i, g): row first_row(4 g + e) + c, column 8 i + b.
    // Rows before 8 r belong to the neighbour.
    const int col = k0 + 8 * i;
    O *const out = dw + ((int64_t)z * n) * k + col;
    const auto put = [&](int e, int c, float (&v)[8]) GQT_INLINE {
        const int r = 4 * g + e, row = first_row(r) + c;
        if (row >= n0 + 8 * r && row < n && col < k)
            store8(out + (int64_t)row * k, k - col, v);
    };
    if constexpr (SHARED) {
        // Half of the c at a time, each wave leaves its sums in LDS and adds
        // up those of all four waves for one c.
        f32x4(*const part)[4][4][2][64] = reinterpret_cast<f32x4(*)[4][4][2][64]>(lds);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            __syncthreads();
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        f32x4 v;
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            v[w] = acc[4 * h + c][4 * b + w][e];
                        part[wave][c][e][b][lane] = v;
                    }
            __syncthreads();
#pragma unroll 1
            for (int e = 0; e < 4; ++e) {
                float v[8];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    f32x4 t = part[0][wave][e][b][lane];
#pragma unroll
                    for (int w = 1; w < kWaves; ++w)
                        t += part[w][wave][e][b][lane];
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        v[4 * b + w] = t[w];
                }
                put(e, 4 * h + wave, v);
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                float v[8];
#pragma unroll
                for (int b = 0; b < 8; ++b)
                    v[b] = acc[c][b][e];
                put(e, c, v);
            }
    }
    if (db_part || (db_whole && tk == 0)) {
        const auto put_db = [&](int row, float v) GQT_INLINE {
            if (db_part)
                db_part[((int64_t)z * tiles.k * kSide + tk) * n + row] = v;
            else
                db_whole[row] = (O)v;
        };
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            sum[c] += __shfl_xor(sum[c], 16);
            sum[c] += __shfl_xor(sum[c], 32);
        }
        if constexpr (SHARED) {
            __syncthreads();
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (g == 0)
                    lds[(wave * 16 + i) * 8 + c] = sum[c];
            __syncthreads();
            if (threadIdx.x < kTile) {
                const int t = threadIdx.x, row = first_row(t / 8) + t % 8;
                float v = 0.0f;
#pragma unroll
                for (int w = 0; w < kWaves; ++w)
                    v += lds[w * kTile + t];
                if (row >= n0 + t / 8 * 8 && row < n)
                    put_db(row, v);
            }
        } else if (g == 0) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int row = dy_col + c;
                if (row >= n0 + 8 * i && row < n)
                    put_db(row, sum[c]);
            }
        }
    }
}

// n < 8: too few rows of dw for a tile, whose lanes load eight columns of dy
// that exist.  A block's 16 lanes take 128 columns of x, its 16 rows of
// threads every 16th token, and one product a value is an ordinary fused
// multiply-add.  16384 x 4 x 1024 takes 27 to 38 us a call (two boxes), bound
// by waiting for its loads: plan_of cuts it as it cuts the large tiles, a block
// a CU, so that a SIMD has one wave, which loads nothing ahead (VALU in 14 % of
// the issue slots).  db comes from block 0.
template <typename T>
__global__ __launch_bounds__(256) void k_weight_grad_narrow(
    const T *__restrict__ dy, int64_t m, int32_t n, int64_t lddy, Act8 x, int32_t k, int64_t chunk,
    float *__restrict__ part, float *__restrict__ db_part)
{
    __shared__ float lds[16][16][9];
    const int i = threadIdx.x % 16, t = threadIdx.x / 16;
    const int col = blockIdx.x * kTile + 8 * i;
    const int64_t z = blockIdx.y, m_begin = z * chunk;
    const int64_t m_end = m_begin + chunk < m ? m_begin + chunk : m;
    float acc[7][8] = {}, sum[7] = {};
    for (int64_t row = m_begin + t; row < m_end; row += 16) {
        float v[8];
        if (col < k)
            restore8(x, x.chunk(row, col), v);
        else
#pragma unroll
            for (int b = 0; b < 8; ++b)
                v[b] = 0.0f;
#pragma unroll
        for (int c = 0; c < 7; ++c) {
            const float g = c < n ? (float)dy[row * lddy + c] : 0.0f;
            sum[c] += g;
#pragma unroll
            for (int b = 0; b < 8; ++b)
                acc[c][b] = fmaf(g, v[b], acc[c][b]);
        }
    }
#pragma unroll
    for (int c = 0; c < 7; ++c) {
        __syncthreads();
#pragma unroll
        for (int b = 0; b < 8; ++b)
            lds[t][i][b] = acc[c][b];
        lds[t][i][8] = sum[c];
        __syncthreads();
        if (c >= n)
            continue;
        for (int at = threadIdx.x; at < 16 * 9; at += 256) {
            const int b = at % 9, column = blockIdx.x * kTile + 8 * (at / 9) + b;
            float v = 0.0f;
            for (int w = 0; w < 16; ++w)
                v += lds[w][at / 9][b];
            if (b < 8 && column < k)
                part[(z * n + c) * k + column] = v;
            if (at == 8 && blockIdx.x == 0 && db_part)
                db_part[z * n + c] = v;
        }
    }
}

__device__ __forceinline__ void store4(float *p, int64_t left, const f32x4 &v)
{
    if (left >= 4)
        *reinterpret_cast<u32x4_e4 *>(p) = __builtin_bit_cast(u32x4, v);
    else
        for (int j = 0; j < left; ++j)
            p[j] = v[j];
}
__device__ __forceinline__ void store4(bf16 *p, int64_t left, const f32x4 &v)
{
    const bf16x4 h = {(bf16)v[0], (bf16)v[1], (bf16)v[2], (bf16)v[3]};
    if (left >= 4)
        *reinterpret_cast<u32x2_e2 *>(p) = __builtin_bit_cast(u32x2, h);
    else
        for (int j = 0; j < left; ++j)
            p[j] = h[j];
}

// Adds partials in a fixed order: `splits` of count values for dw (unless it
// is whole already), and `db_parts` of n for db, whose blocks come after
// dw's.  256 values a block, four a lane, and a quarter of the partials a
// wave, so that a long chain of few values has loads enough in flight (us a
// call, against a value a lane and all partials a wave: 100000 x 8 x 32 18 and
// 25, 16384 x 16 x 4096 32 and 43; at odd sizes up to 0.9 more, fp32 1000 x
// 1001 x 777 26.3 and 25.4).  Bound by its launch or by reading the partials:
// 4 of 1024 x 1024 in 6 us.
template <typename O>
__global__ __launch_bounds__(256) void k_sum_parts(const float *__restrict__ dw_part,
                                                   int32_t splits, int64_t count,
                                                   O *__restrict__ dw, uint32_t dw_blocks,
                                                   const float *__restrict__ db_part,
                                                   int32_t db_parts, int32_t n,
                                                   O *__restrict__ db)
{
    __shared__ f32x4 sums[3][64];
    const bool second = blockIdx.x >= dw_blocks;
    const float *const part = second ? db_part : dw_part;
    O *const out = second ? db : dw;
    const int64_t size = second ? n : count;
    const int32_t terms = second ? db_parts : splits;
    const int64_t first = blockIdx.x - (second ? dw_blocks : 0);
    const int64_t blocks = second ? gridDim.x - dw_blocks : dw_blocks;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int32_t from = (int32_t)((int64_t)terms * wave / 4);
    const int32_t to = (int32_t)((int64_t)terms * (wave + 1) / 4);
    for (int64_t base = first * 256; base < size; base += blocks * 256) {
        const int64_t i = base + 4 * lane, left = size - i;
        f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
        const float *p = part + from * size + i;
        if (left >= 4) {
#pragma unroll 4
            for (int32_t z = from; z < to; ++z, p += size)
                s += __builtin_bit_cast(f32x4, *reinterpret_cast<const u32x4_e4 *>(p));
        } else if (left > 0) {
            // the values there are, the last one repeated: a loop over them
            // inside that over the partials would wait for every load
            const int32_t j1 = left > 1 ? 1 : 0, j2 = left > 2 ? 2 : j1;
#pragma unroll 4
            for (int32_t z = from; z < to; ++z, p += size)
                s += f32x4{p[0], p[j1], p[j2], 0.0f};
        }
        __syncthreads(); // the last turn's sums are read
        if (wave)
            sums[wave - 1][lane] = s;
        __syncthreads();
        if (wave == 0) {
            s = ((s + sums[0][lane]) + sums[1][lane]) + sums[2][lane];
            store4(out + i, left, s);
        }
    }
}

// How the work is cut: tiles, and how often the tokens are split.
struct Plan {
    bool shared;
    bool whole_db; // db comes from the tiles themselves
    Tiles tiles;
    int32_t splits;
    int64_t chunk;
    int64_t dw_part, db_part, bytes; // partials: values of dw's, of db's, and the workspace
    int32_t db_parts;
};

// The cut with the least estimated time.  A CU holds one block, so blocks
// run in rounds of 256; a round takes a fixed time and that of its steps, and
// partials are written and read again at 4 TB/s with 3 us for their launch
// (all measured).  8192 x 4096 x 1056 (288 tiles, so two rounds of whole
// tokens) takes 105 us cut so; 8192 x 4096 x 1024 (256 tiles) takes 76.
Plan plan_of(int64_t m, int64_t n, int64_t k, int32_t dtype)
{
    Plan p{};
    if (m == 0) // no partials: sums of nothing
        return p;
    double best = 0.0;
    for (int shared = 0; shared < 2; ++shared) {
        const int64_t side = shared ? kTile : 2 * kTile, tokens = step_tokens(shared);
        const int64_t tn = (n + side - 1) / side, tk = (k + side - 1) / side;
        const int64_t steps = (m + tokens - 1) / tokens;
        const double round_us = shared ? 8.0 : 17.0;
        const double step_us = dtype == GQ_IN_F32 ? 2.4 : 1.0;
        if (n < 8 && !shared)
            continue;
        for (int64_t s = 1; s <= 256 && s <= steps; ++s) {
            const int64_t chunk = (steps + s - 1) / s, splits = (steps + chunk - 1) / chunk;
            const double rounds = (double)((tn * tk * splits + 255) / 256);
            double us = rounds * (round_us + step_us * (double)chunk);
            if (splits > 1)
                us += 3.0 + (double)splits * (double)n * (double)k * 8.0 / 4e6;
            if (p.splits == 0 || us < best) {
                best = us;
                p.shared = shared;
                p.splits = (int32_t)splits;
                p.chunk = chunk * tokens;
                // n k < 2^36: below 2^23 tiles, or few splits
                p.tiles = {(int32_t)tn, (int32_t)tk, (int32_t)(tn * tk * splits)};
            }
        }
    }
    // db straight from the tiles, where the first of a column does all its
    // steps, against partials and a second launch, us (bf16, fp32): 4096 x
    // 1024 over 128 tokens 11.1 and 12.9 against 14.0 and 15.5, over 1536 (12
    // steps) 25.4 and 44.1 against 26.8 and 46.7; 4096 x 4096 over 384 (12
    // steps of squares) 28.6 and 48.7 against 33.0 and 53.8.  What a step
    // adds eats the launch's 3 us by about 20 steps.
    p.whole_db = n >= 8 && p.splits == 1 && p.chunk <= 12 * step_tokens(p.shared);
    p.db_parts = p.whole_db ? 0 : n < 8 ? p.splits : p.splits * p.tiles.k * (p.shared ? 1 : 2);
    p.dw_part = p.splits > 1 || n < 8 ? p.splits * n * k : 0;
    p.db_part = p.db_parts * n;
    p.bytes = 4 * (p.dw_part + p.db_part);
    return p;
}

bool sizes_ok(int64_t m, int64_t n, int64_t k)
{
    return m >= 0 && m < ((int64_t)1 << 32) && n >= 1 && n < kMaxColumns && k >= 1 &&
           k < kMaxColumns && n * k < ((int64_t)1 << 36);
}

template <typename T, typename O>
int32_t launch(const void *dy, int64_t m, int32_t n, int64_t lddy, const Act8 &x, int32_t k,
               void *dw, void *db, float *ws, hipStream_t st)
{
    const Plan p = plan_of(m, n, k, sizeof(T) == 4 ? GQ_IN_F32 : GQ_IN_BF16);
    float *const db_part = db && !p.whole_db ? ws + p.dw_part : nullptr;
    O *const db_whole = p.whole_db ? (O *)db : nullptr;
    const T *const dyt = (const T *)dy;
    if (m == 0) {
        // nothing to launch before the sums
    } else if (n < 8) {
        k_weight_grad_narrow<T><<<dim3(p.tiles.k, p.splits), 256, 0, st>>>(
            dyt, m, n, lddy, x, k, p.chunk, ws, db_part);
        GQT_TRY(check_launch("k_weight_grad_narrow"));
    } else {
        const dim3 grid(p.tiles.total);
        if (p.dw_part && p.shared)
            k_weight_grad<T, float, true><<<grid, kThreads, 0, st>>>(
                dyt, m, n, lddy, x, k, p.chunk, p.tiles, ws, db_part, nullptr);
        else if (p.dw_part)
            k_weight_grad<T, float, false><<<grid, kThreads, 0, st>>>(
                dyt, m, n, lddy, x, k, p.chunk, p.tiles, ws, db_part, nullptr);
        else if (p.shared)
            k_weight_grad<T, O, true><<<grid, kThreads, 0, st>>>(
                dyt, m, n, lddy, x, k, p.chunk, p.tiles, (O *)dw, db_part, db_whole);
        else
            k_weight_grad<T, O, false><<<grid, kThreads, 0, st>>>(
                dyt, m, n, lddy, x, k, p.chunk, p.tiles, (O *)dw, db_part, db_whole);
        GQT_TRY(check_launch("k_weight_grad"));
    }
    const int64_t count = (int64_t)n * k;
    const auto blocks = [](int64_t size) { return size < 1 << 30 ? (size + 255) / 256 : 1 << 22; };
    const int64_t dw_blocks = p.dw_part || m == 0 ? blocks(count) : 0;
    const int64_t db_blocks = db && !p.whole_db ? blocks(n) : 0;
    if (dw_blocks + db_blocks == 0)
        return ok();
    k_sum_parts<O><<<dim3((uint32_t)(dw_blocks + db_blocks)), 256, 0, st>>>(
        ws, p.splits, count, (O *)dw, (uint32_t)dw_blocks, db_part, p.db_parts, n, (O *)db);
    return check_launch("k_sum_parts");
}

} // namespace
} // namespace gqt

using namespace gqt;

extern "C" {

int64_t gqt_weight_grad_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t dtype)
{
    if (!sizes_ok(m, n, k) || !dtype_ok(dtype))
        return -1;
    return plan_of(m, n, k, dtype).bytes;
}

int32_t gqt_weight_grad(const void *dy, int32_t dtype, int64_t m, int64_t n, int64_t lddy,
                        const gqt_act8 *x8, int64_t k, void *dw, void *db, int32_t wdtype,
                        void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!dtype_ok(dtype) || !dtype_ok(wdtype))
        return fail(GQ_ERR_ARG, "dtype %d or wdtype %d is neither GQ_IN_F32 nor GQ_IN_BF16", dtype,
                    wdtype);
    if (!sizes_ok(m, n, k))
        return fail(GQ_ERR_ARG, "m = %lld, n = %lld, k = %lld out of range", (long long)m,
                    (long long)n, (long long)k);
    if (m > 0 && groups_of(k) >= (kMaxGroups + m - 1) / m)
        return fail(GQ_ERR_UNSUPPORTED, "m = %lld of k = %lld: 2^29 groups of 32 or more",
                    (long long)m, (long long)k);
    if ((!dy && m > 0) || !dw)
        return fail(GQ_ERR_NULL, "dy or dw is NULL");
    if ((lddy != 0 && lddy < n) || lddy > ((int64_t)1 << 40))
        return fail(GQ_ERR_ARG, "lddy = %lld: 0 or at least %lld", (long long)lddy, (long long)n);
    if (!aligned_to(dy, elem_bytes(dtype)) || !aligned_to(dw, elem_bytes(wdtype)) ||
        !aligned_to(db, elem_bytes(wdtype)))
        return fail(GQ_ERR_ALIGN, "dy, dw or db is not aligned to its elements");
    if (!x8)
        return fail(GQ_ERR_NULL, "x8 is NULL");
    GQT_TRY(check_act8("x8", x8, m, false));
    const int64_t need = gqt_weight_grad_workspace_bytes(m, n, k, dtype);
    if (need > 0 && !workspace)
        return fail(GQ_ERR_NULL, "workspace is NULL");
    if (workspace_bytes < need)
        return fail(GQ_ERR_WORKSPACE, "workspace of %lld bytes, %lld are needed",
                    (long long)workspace_bytes, (long long)need);
    if (!aligned_to(workspace, 16))
        return fail(GQ_ERR_ALIGN, "workspace is not 16-byte aligned");
    const Act8 x = act8_view(x8, k);
    float *const ws = (float *)workspace;
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == GQ_IN_F32)
        return wdtype == GQ_IN_F32
                   ? launch<float, float>(dy, m, (int32_t)n, lddy, x, (int32_t)k, dw, db, ws, st)
                   : launch<float, bf16>(dy, m, (int32_t)n, lddy, x, (int32_t)k, dw, db, ws, st);
    return wdtype == GQ_IN_F32
               ? launch<bf16, float>(dy, m, (int32_t)n, lddy, x, (int32_t)k, dw, db, ws, st)
               : launch<bf16, bf16>(dy, m, (int32_t)n, lddy, x, (int32_t)k, dw, db, ws, st);
}

} // extern "C"
