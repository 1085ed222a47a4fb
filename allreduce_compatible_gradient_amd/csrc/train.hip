// train.hip -- layer norm, GELU and the 8-bit activation copies on MI355X
// (gfx950): the operators of include/gq_train.h that stream their matrices.
// Times in the comments are of the kernel alone unless they say "call"; for
// comparison a copy of 0.25 to 1 GiB runs at 5.0 to 5.4 TB/s here, and small
// matrices stay in the cache, where more is possible.
//
// Every kernel reads its inputs once and writes its outputs once, eight
// columns (one 16-byte bf16 load) per lane and step, so that four lanes hold
// one 32-column group of the 8-bit format and one Philox call serves a
// lane's eight roundings.
#include "train_common.h"

#include <stdarg.h>
#include <stdio.h>

namespace gqt {

thread_local char g_err[512];

int32_t fail(int32_t status, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return status;
}

int32_t ok()
{
    g_err[0] = 0;
    return GQ_OK;
}

int32_t check_launch(const char *kernel)
{
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return fail(GQ_ERR_DEVICE, "%s: %s", kernel, hipGetErrorString(e));
    return ok();
}

namespace {

// ---------------------------------------------------------------------------
// Layer norm
//
// TPR threads hold one row, C chunks of eight columns each (chunk c of lane t
// at column 8 (c TPR + t)), so the row is read once and its mean and the sum
// of squared deviations from it (no cancellation, whatever the mean) are
// taken in registers.  Rows beyond 16384 columns are
// read three times by k_layer_norm_long, from the cache after the first: bf16
// 4096 x 16384 takes 48 us a call in registers and 94 so, 8192 x 8192 49 and
// 127.  The shape goes by d alone, so that keeping a copy does not change y.
//
// Forward: mean = sum x / d, rstd = 1 / sqrt(sum (x - mean)^2 / d + eps), y =
// (x - mean) rstd w + b.  Bound by memory: 16384 x 4096 bf16 50 us (5.3 TB/s
// of one read and one write), 131072 x 64 9.6 us.  Copies take instructions:
// bf16 8191 x 2048 15 us without, 19 with one to nearest (VALU in 50 % of the
// issue slots), 25 with one at random (55 %), 36 with two at random (63 %;
// 32768 x 2048 89 %).  Between, neither memory (3.2 TB/s with one at random)
// nor VALU is full; a block has one row, whose two sums cost four barriers.

template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *lds)
{
#pragma unroll
    for (int o = 1; o < (TPR < 64 ? TPR : 64); o <<= 1)
        v += __shfl_xor(v, o);
    if (TPR > 64) {
        // one slot per wave; the leading barrier frees the previous sum's slots
        __syncthreads();
        if ((threadIdx.x & 63) == 0)
            lds[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w)
            v += lds[w];
    }
    return v;
}

// Eight columns of a weight or bias; `other` without one.
__device__ __forceinline__ void load_weight8(const void *w, int32_t wdtype, int32_t col, int32_t d,
                                             float other, float (&v)[8])
{
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[k] = other;
    if (!w || col >= d)
        return;
    if (wdtype == GQ_IN_F32)
        load8(static_cast<const float *>(w), col, d, v);
    else
        load8(static_cast<const bf16 *>(w), col, d, v);
}

template <int TPR>
constexpr int block_threads()
{
    return TPR > 256 ? TPR : 256;
}

// Which of the block's rows this thread works on; of a whole wave the same,
// which leaves what depends on the row alone (two of the random numbers'
// products) to the scalar unit.
template <int TPR>
__device__ __forceinline__ int row_slot()
{
    const int slot = threadIdx.x / TPR;
    return TPR >= 64 ? __builtin_amdgcn_readfirstlane(slot) : slot;
}

template <typename T, int TPR, int C, bool KEEP>
__global__ __launch_bounds__(block_threads<TPR>()) void k_layer_norm(
    const T *__restrict__ x, int64_t rows, int32_t d, int64_t ldx, const void *__restrict__ w,
    const void *__restrict__ b, int32_t wdtype, float eps, T *__restrict__ y,
    float *__restrict__ mean_out, float *__restrict__ rstd_out, Act8 keep_x, Act8 keep_y)
{
    constexpr int kRows = block_threads<TPR>() / TPR;
    __shared__ float lds[TPR > 64 ? TPR / 64 : 1];
    const int t = threadIdx.x % TPR;
    float wv[C][8], bv[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        load_weight8(w, wdtype, 8 * (c * TPR + t), d, 1.0f, wv[c]);
        load_weight8(b, wdtype, 8 * (c * TPR + t), d, 0.0f, bv[c]);
    }
    const float inv_d = 1.0f / (float)d;
    const int64_t stride = (int64_t)gridDim.x * kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + row_slot<TPR>();
    if (row >= rows)
        return; // whole rows of lanes leave, and only where no barrier follows (kRows > 1)
    Raw8<T> ahead[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
        load_ahead(x + row * ldx, 8 * (c * TPR + t), d, ahead[c]);
    for (; row < rows; row += stride) {
        float v[C][8];
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            settle(x + row * ldx, 8 * (c * TPR + t), d, ahead[c]);
            unpack(ahead[c], v[c]);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                s += v[c][k];
        }
        // the next row is loaded while this one is worked on
        if (row + stride < rows)
#pragma unroll
            for (int c = 0; c < C; ++c)
                load_ahead(x + (row + stride) * ldx, 8 * (c * TPR + t), d, ahead[c]);
        const float mean = row_sum<TPR>(s, lds) * inv_d;
        s = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = 8 * (c * TPR + t);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float u = v[c][k] - mean;
                s = fmaf(col + k < d ? u : 0.0f, u, s);
            }
        }
        const float rstd = 1.0f / sqrtf(row_sum<TPR>(s, lds) * inv_d + eps);
        if (t == 0) {
            if (mean_out)
                mean_out[row] = mean;
            if (rstd_out)
                rstd_out[row] = rstd;
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = 8 * (c * TPR + t);
            if (KEEP && keep_x.keep != kKeepNone)
                keep8(keep_x, row, col, keep_x.chunk(row, col), v[c]);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[c][k] = fmaf((v[c][k] - mean) * rstd, wv[c][k], bv[c][k]);
            if (col < d)
                store8(y + row * d + col, d - col, v[c]);
            if (KEEP && keep_y.keep != kKeepNone) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (col + k >= d)
                        v[c][k] = 0.0f;
                keep8(keep_y, row, col, keep_y.chunk(row, col), v[c]);
            }
        }
    }
}

constexpr int kLongThreads = 1024;

template <typename T>
__global__ __launch_bounds__(kLongThreads) void k_layer_norm_long(
    const T *__restrict__ x, int64_t rows, int32_t d, int64_t ldx, const void *__restrict__ w,
    const void *__restrict__ b, int32_t wdtype, float eps, T *__restrict__ y,
    float *__restrict__ mean_out, float *__restrict__ rstd_out, Act8 keep_x, Act8 keep_y)
{
    __shared__ float lds[kLongThreads / 64];
    // columns rounded up to whole groups, so that quads stay whole
    const int64_t cols = ((int64_t)d + 31) / 32 * 32;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const T *xr = x + row * ldx;
        float s = 0.0f;
        for (int64_t col = 8 * threadIdx.x; col < d; col += 8 * kLongThreads) {
            float v[8];
            load8(xr, (int32_t)col, d, v);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                s += v[k];
        }
        const float mean = row_sum<kLongThreads>(s, lds) / (float)d;
        s = 0.0f;
        for (int64_t col = 8 * threadIdx.x; col < d; col += 8 * kLongThreads) {
            float v[8];
            load8(xr, (int32_t)col, d, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float u = v[k] - mean;
                s = fmaf(col + k < d ? u : 0.0f, u, s);
            }
        }
        const float rstd = 1.0f / sqrtf(row_sum<kLongThreads>(s, lds) / (float)d + eps);
        if (threadIdx.x == 0) {
            if (mean_out)
                mean_out[row] = mean;
            if (rstd_out)
                rstd_out[row] = rstd;
        }
        for (int64_t col = 8 * threadIdx.x; col < cols; col += 8 * kLongThreads) {
            float v[8], wv[8], bv[8];
            const int n = (int)(d - col);
            load8(xr, (int32_t)col, d, v);
            load_weight8(w, wdtype, (int32_t)col, d, 1.0f, wv);
            load_weight8(b, wdtype, (int32_t)col, d, 0.0f, bv);
            if (keep_x.keep != kKeepNone)
                keep8(keep_x, row, (int32_t)col, keep_x.chunk(row, (int32_t)col), v);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = fmaf((v[k] - mean) * rstd, wv[k], bv[k]);
            if (n > 0)
                store8(y + row * d + col, n, v);
            if (keep_y.keep != kKeepNone) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k >= n)
                        v[k] = 0.0f;
                keep8(keep_y, row, (int32_t)col, keep_y.chunk(row, (int32_t)col), v);
            }
        }
    }
}

// Backward: with g = dy w and xh = (x - mean) rstd, dx = rstd (g - mean of g
// over the row - xh times that of g xh); dw and db are the sums over rows of
// dy xh and dy.  Each thread adds up its columns over its block's rows in a
// fixed order; partial[block][2][d] is reduced by k_sum_partials.  Bound by
// memory: 16384 x 4096 bf16 79 us (5.1 TB/s of dy, x and dx, before 25 MB of
// partials); 8191 x 2048 bf16 from the copy 22.5 us (3.8 TB/s).
template <typename T, int TPR, int C, bool ACT8>
__global__ __launch_bounds__(block_threads<TPR>()) void k_layer_norm_backward(
    const T *__restrict__ dy, int64_t rows, int32_t d, int64_t lddy, const T *__restrict__ x,
    int64_t ldx, Act8 x8, const float *__restrict__ mean_in, const float *__restrict__ rstd_in,
    const void *__restrict__ w, int32_t wdtype, T *__restrict__ dx, float *__restrict__ partial)
{
    constexpr int kRows = block_threads<TPR>() / TPR;
    // The next row's loads run ahead where a CU holds one block, so that no
    // other covers them (bf16 8192 x 8192: 80 us, without 104), and with one
    // chunk a thread where a row's loads are few (bf16 16384 x 2048 from the
    // copy: 41, without 43).  Two fp32 rows are enough in flight as they are
    // (32768 x 2048: 151 us, ahead 161), and with more chunks the registers
    // cost what the loads gain (bf16 87381 x 768 from the copy: 74, ahead 86).
    constexpr bool kAhead = TPR > 256 || (C == 1 && (sizeof(T) == 2 || ACT8));
    __shared__ float lds[TPR > 64 ? TPR / 64 : 1];
    __shared__ float sums[kRows > 1 ? kRows * TPR * C * 8 : 1];
    const int t = threadIdx.x % TPR, slot = row_slot<TPR>();
    float wv[C][8], aw[C][8], ab[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        load_weight8(w, wdtype, 8 * (c * TPR + t), d, 1.0f, wv[c]);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            aw[c][k] = ab[c][k] = 0.0f;
    }
    const float inv_d = 1.0f / (float)d;
    const int64_t stride = (int64_t)gridDim.x * kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + slot;
    Raw8<T> raw_g[C], raw_x[C];
    RawAct8 raw_x8[C];
    float mean = 0.0f, rstd = 0.0f;
    const auto load = [&](int64_t r) {
        mean = mean_in[r];
        rstd = rstd_in[r];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = 8 * (c * TPR + t);
            load_ahead(dy + r * lddy, col, d, raw_g[c]);
            if (ACT8)
                load_act8(x8, x8.chunk(r, col < d ? col : 0), raw_x8[c]);
            else
                load_ahead(x + r * ldx, col, d, raw_x[c]);
        }
    };
    if (kAhead && row < rows)
        load(row);
    for (; row < rows; row += stride) {
        if (!kAhead)
            load(row);
        float g[C][8], xh[C][8];
        float s1 = 0.0f, s2 = 0.0f;
        const float r_rstd = rstd, r_mean = mean;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = 8 * (c * TPR + t);
            settle(dy + row * lddy, col, d, raw_g[c]);
            unpack(raw_g[c], g[c]);
            if (ACT8) {
                unpack_act8(raw_x8[c], xh[c]);
            } else {
                settle(x + row * ldx, col, d, raw_x[c]);
                unpack(raw_x[c], xh[c]);
            }
        }
        if (kAhead && row + stride < rows)
            load(row + stride);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int n = d - 8 * (c * TPR + t);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                // columns past d contribute nothing, even where the
                // statistics or the copy's padding hold a NaN
                xh[c][k] = k < n ? (xh[c][k] - r_mean) * r_rstd : 0.0f;
                aw[c][k] = fmaf(g[c][k], xh[c][k], aw[c][k]);
                ab[c][k] += g[c][k];
                g[c][k] *= wv[c][k];
                s1 += g[c][k];
                s2 = fmaf(g[c][k], xh[c][k], s2);
            }
        }
        s1 = row_sum<TPR>(s1, lds) * inv_d;
        s2 = row_sum<TPR>(s2, lds) * inv_d;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = 8 * (c * TPR + t);
            if (col >= d)
                continue;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                g[c][k] = r_rstd * (g[c][k] - s1 - xh[c][k] * s2);
            store8(dx + row * d + col, d - col, g[c]);
        }
    }
    if (!partial)
        return;
    float *out = partial + (int64_t)blockIdx.x * 2 * d;
    if (kRows == 1) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = 8 * (c * TPR + t);
            if (col < d) {
                store8(out + col, d - col, aw[c]);
                store8(out + d + col, d - col, ab[c]);
            }
        }
        return;
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                sums[(slot * C + c) * TPR * 8 + 8 * t + k] = which ? ab[c][k] : aw[c][k];
        __syncthreads();
        for (int col = threadIdx.x; col < d; col += block_threads<TPR>()) {
            float s = 0.0f;
            for (int r = 0; r < kRows; ++r)
                s += sums[r * C * TPR * 8 + col];
            out[which * d + col] = s;
        }
    }
}

// Rows of more than 8192 columns, too long for registers: dx alone, from two
// readings of the row (8192 x 8192: 103 us a call in registers, 161 with this
// and the column sums below; fp32 155 and 301).
template <typename T, bool ACT8>
__global__ __launch_bounds__(kLongThreads) void k_layer_norm_backward_long(
    const T *__restrict__ dy, int64_t rows, int32_t d, int64_t lddy, const T *__restrict__ x,
    int64_t ldx, Act8 x8, const float *__restrict__ mean_in, const float *__restrict__ rstd_in,
    const void *__restrict__ w, int32_t wdtype, T *__restrict__ dx)
{
    __shared__ float lds[kLongThreads / 64];
    const float inv_d = 1.0f / (float)d;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const float mean = mean_in[row], rstd = rstd_in[row];
        float s1 = 0.0f, s2 = 0.0f;
        for (int pass = 0; pass < 2; ++pass) {
            for (int64_t col = 8 * threadIdx.x; col < d; col += 8 * kLongThreads) {
                const int n = (int)(d - col);
                float g[8], xh[8], wv[8];
                load8(dy + row * lddy, (int32_t)col, d, g);
                if (ACT8)
                    restore8(x8, x8.chunk(row, (int32_t)col), xh);
                else
                    load8(x + row * ldx, (int32_t)col, d, xh);
                load_weight8(w, wdtype, (int32_t)col, d, 1.0f, wv);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    xh[k] = k < n ? (xh[k] - mean) * rstd : 0.0f;
                    g[k] *= wv[k];
                }
                if (pass == 0) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        s1 += g[k];
                        s2 = fmaf(g[k], xh[k], s2);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        g[k] = rstd * (g[k] - s1 - xh[k] * s2);
                    store8(dx + row * d + col, n, g);
                }
            }
            if (pass == 0) {
                s1 = row_sum<kLongThreads>(s1, lds) * inv_d;
                s2 = row_sum<kLongThreads>(s2, lds) * inv_d;
            }
        }
    }
}

// and their partial sums for dw and db, 2048 columns a block along x, the rows
// dealt out along y: a second reading of dy and x (one kernel for both that
// added them up in memory row by row took 265 us a call at 5461 x 12288, the
// two take 160).
template <typename T, bool ACT8>
__global__ __launch_bounds__(256) void k_norm_column_sums(
    const T *__restrict__ dy, int64_t rows, int32_t d, int64_t lddy, const T *__restrict__ x,
    int64_t ldx, Act8 x8, const float *__restrict__ mean_in, const float *__restrict__ rstd_in,
    float *__restrict__ partial)
{
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (at >= d)
        return;
    const int32_t col = (int32_t)at;
    float aw[8] = {}, ab[8] = {};
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        const float mean = mean_in[row], rstd = rstd_in[row];
        float g[8], xh[8];
        load8(dy + row * lddy, col, d, g);
        if (ACT8)
            restore8(x8, x8.chunk(row, col), xh);
        else
            load8(x + row * ldx, col, d, xh);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            aw[k] = fmaf(g[k], (xh[k] - mean) * rstd, aw[k]);
            ab[k] += g[k];
        }
    }
    float *const out = partial + (int64_t)blockIdx.y * 2 * d + col;
    store8(out, d - col, aw);
    store8(out + d, d - col, ab);
}

// dw and db: the blocks' partial sums added in block order, a sixteenth of
// the blocks a wave, eight loads in flight (one at a time in one wave, the
// chain of loads took 62 us for 1024 blocks whatever d; now 5.5 us for 768 of
// d = 4096, 3.9 us for 1024 of d = 64).  64 columns a block along x, dw / db
// along y.
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(64 * kSumWaves) void k_sum_partials(
    const float *__restrict__ partial, int32_t blocks, int32_t d, void *__restrict__ dw,
    void *__restrict__ db, int32_t wdtype)
{
    __shared__ float part[kSumWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t col = (int64_t)blockIdx.x * 64 + lane;
    void *out = blockIdx.y ? db : dw;
    if (!out)
        return;
    float s = 0.0f;
    if (col < d) {
        const float *p = partial + (int64_t)blockIdx.y * d + col;
        const int lo = blocks * wave / kSumWaves, hi = blocks * (wave + 1) / kSumWaves;
        int i = lo;
        for (; i + 8 <= hi; i += 8) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = p[(int64_t)(i + j) * 2 * d];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s += v[j];
        }
        for (; i < hi; ++i)
            s += p[(int64_t)i * 2 * d];
    }
    part[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && col < d) {
        s = 0.0f;
#pragma unroll
        for (int w = 0; w < kSumWaves; ++w)
            s += part[w][lane];
        if (wdtype == GQ_IN_F32)
            static_cast<float *>(out)[col] = s;
        else
            static_cast<bf16 *>(out)[col] = (bf16)s;
    }
}

// ---------------------------------------------------------------------------
// Elementwise operators: one thread per 8 columns, rows padded to whole groups

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
__device__ __forceinline__ uint32_t divide(uint32_t n, const FastDiv &f)
{
    return (uint32_t)(((uint64_t)n * f.m) >> f.s);
}

// The chunk of this thread; chunks = rows * (4 G).
struct Chunk {
    int64_t row;
    int32_t col;
};
__device__ __forceinline__ Chunk chunk_at(uint32_t i, const FastDiv &per_row)
{
    const uint32_t row = divide(i, per_row);
    return {(int64_t)row, (int32_t)((i - row * per_row.d) * 8)};
}

constexpr int kThreads = 256;

// A copy of a matrix, 16384 x 4096 bf16: to nearest bound by memory, 35 to 39
// us (5.2 to 5.8 TB/s of 2 + 33/32 bytes a value; VALU in 46 % of the issue
// slots); at random 46 us (71 %).
template <typename T>
__global__ __launch_bounds__(kThreads) void k_act8_save(const T *__restrict__ x, uint32_t chunks,
                                                        FastDiv per_row, int32_t d, int64_t ldx,
                                                        Act8 out)
{
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= chunks)
        return;
    const Chunk c = chunk_at(i, per_row);
    float v[8];
    load8(x + c.row * ldx, c.col, d, v);
    keep8(out, c.row, c.col, i, v);
}

// The values again, exact in T: bound by memory, 16384 x 4096 to bf16 31 us
// (6.6 TB/s, much of it within the cache).
template <typename T>
__global__ __launch_bounds__(kThreads) void k_act8_restore(Act8 in, uint32_t chunks,
                                                           FastDiv per_row, int32_t d,
                                                           T *__restrict__ out)
{
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= chunks)
        return;
    const Chunk c = chunk_at(i, per_row);
    if (c.col >= d)
        return;
    float v[8];
    restore8(in, i, v);
    store8(out + c.row * d + c.col, d - c.col, v);
}

// Phi(-z) e^(z^2 / 2) for z >= 0, as t p(t) with t = 1 / (1 + 0.32 z) and p of
// degree 9 fitted (minimax, relative error 3.2e-8; 1.4e-7 evaluated in fp32)
// to the scaled complementary error function.  1 - erf would lose the tail.
__device__ __forceinline__ float scaled_tail(float z)
{
    const float t = __builtin_amdgcn_rcpf(fmaf(0.32f, z, 1.0f));
    float p = -0.021078171208500862f;
    p = fmaf(p, t, 0.09540726244449615f);
    p = fmaf(p, t, -0.1467074602842331f);
    p = fmaf(p, t, 0.06532800942659378f);
    p = fmaf(p, t, -0.009377559646964073f);
    p = fmaf(p, t, 0.05865396186709404f);
    p = fmaf(p, t, 0.0878290981054306f);
    p = fmaf(p, t, 0.11462236195802689f);
    p = fmaf(p, t, 0.12766094505786896f);
    p = fmaf(p, t, 0.12766152620315552f);
    return p * t;
}

constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhC = 0.79788456080286536f; // sqrt(2 / pi)
constexpr float kTanhA = 0.044715f;
constexpr float kTanh1 = 2 * 0.79788456080286536; // the tanh form's 2 u = kTanh1 h + kTanh3 h^3
constexpr float kTanh3 = 2 * 0.79788456080286536 * 0.044715;
constexpr float kLog2E = 1.4426950408889634f;

// 4^x for x <= 0, by squaring 2^x: the part's exponential flushes results
// below 2^-126, its square does not.
__device__ __forceinline__ float exp4(float x)
{
    const float half = __builtin_amdgcn_exp2f(x);
    return half * half;
}

// The exponentials of a T: bf16 by exp4, whose few more roundings are far
// below the result's; fp32 by one that is good to the last bit and takes the
// argument with the fewest roundings, which are the result's error in the
// tail.  bf16 would be bound by VALU issue with it (see k_gelu); fp32, bound by
// memory, takes as long (8192 x 4096: erf 43 us a call and 45 with exp4, tanh
// 46 and 44, with a random copy 53 and 52, backward 70 and 70) but for the erf
// form with two random copies (64 and 56).
//
// e^(-h^2 / 2)
template <typename T>
__device__ __forceinline__ float bell(float h)
{
    if (sizeof(T) == 4)
        return expf(-0.5f * h * h);
    return exp4(-0.25f * kLog2E * h * h);
}
// e^-|2u|, u = sqrt(2 / pi) (h + 0.044715 h^3)
template <typename T>
__device__ __forceinline__ float tanh_exp(float h)
{
    if (sizeof(T) == 4)
        return expf(-fabsf(h * fmaf(kTanh3 * h, h, kTanh1)));
    return exp4(-fabsf(h * fmaf(kLog2E * kTanhC * kTanhA * h, h, kLog2E * kTanhC)));
}

// The tanh form's logistic function s = s(2 u) and its complement 1 - s, both
// from e^-|2u|, so that neither is the difference of near numbers.
struct Gate {
    float s, c;
};
template <typename T>
__device__ __forceinline__ Gate tanh_gate(float h)
{
    const float e = tanh_exp<T>(h);
    const float big = __builtin_amdgcn_rcpf(1.0f + e);
    const float small = e * big;
    return h < 0.0f ? Gate{small, big} : Gate{big, small};
}

template <typename T, int FORM>
__device__ __forceinline__ float gelu(float h)
{
    if (FORM == GQT_GELU_TANH)
        return h * tanh_gate<T>(h).s;
    const float tail = scaled_tail(fabsf(h)) * bell<T>(h);
    return h * (h < 0.0f ? tail : 1.0f - tail);
}

template <typename T, int FORM>
__device__ __forceinline__ float gelu_slope(float h)
{
    if (FORM == GQT_GELU_TANH) {
        const Gate g = tanh_gate<T>(h);
        // s (1 - s) is 0 in fp32 long before |h| = 64, where h u' would go
        // on to overflow; a NaN comes through g
        const float c = fminf(fmaxf(h, -64.0f), 64.0f);
        const float u = kTanhC * fmaf(3.0f * kTanhA * c, c, 1.0f);
        return fmaf(2.0f * c * u, g.s * g.c, g.s);
    }
    const float e = bell<T>(h);
    const float tail = scaled_tail(fabsf(h)) * e;
    return fmaf(h * kInvSqrt2Pi, e, h < 0.0f ? tail : 1.0f - tail);
}

// GELU y = h Phi(h), or in the tanh form h s(2 u), and its gradient dy y'(h)
// with y' = Phi + h phi or s + 2 h s (1 - s) u'.  With an exponential good to
// the last bit both kernels were bound by VALU issue (0.98 instructions a CU
// and clock, 79 us for the step of 8192 x 4096 bf16 in the tanh form with a
// random copy of h); now the step takes 64 us, 5.3 TB/s of its 338 MB, at 0.81
// and 0.70.  More instructions are bound by their issue: the erf form takes 29
// us forward without a copy (0.71) and 41 with a random one (0.91), the tanh
// form with two 50 (0.87).
template <typename T, int FORM, bool KEEP>
__global__ __launch_bounds__(kThreads) void k_gelu(const T *__restrict__ h, uint32_t chunks,
                                                   FastDiv per_row, int32_t d, int64_t ldh,
                                                   T *__restrict__ y, Act8 keep_h, Act8 keep_y)
{
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= chunks)
        return;
    const Chunk c = chunk_at(i, per_row);
    const int n = d - c.col;
    float v[8];
    load8(h + c.row * ldh, c.col, d, v);
    if (KEEP && keep_h.keep != kKeepNone)
        keep8(keep_h, c.row, c.col, i, v);
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[k] = gelu<T, FORM>(v[k]);
    if (n > 0)
        store8(y + c.row * d + c.col, n, v); // columns past d: gelu(0) = 0
    if (KEEP && keep_y.keep != kKeepNone)
        keep8(keep_y, c.row, c.col, i, v);
}

template <typename T, int FORM, bool ACT8>
__global__ __launch_bounds__(kThreads) void k_gelu_backward(
    const T *__restrict__ dy, uint32_t chunks, FastDiv per_row, int32_t d, int64_t lddy,
    const T *__restrict__ h, int64_t ldh, Act8 h8, T *__restrict__ dh)
{
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= chunks)
        return;
    const Chunk c = chunk_at(i, per_row);
    const int n = d - c.col;
    if (n <= 0)
        return;
    float g[8], v[8];
    load8(dy + c.row * lddy, c.col, d, g);
    if (ACT8)
        restore8(h8, i, v);
    else
        load8(h + c.row * ldh, c.col, d, v);
#pragma unroll
    for (int k = 0; k < 8; ++k)
        g[k] *= gelu_slope<T, FORM>(v[k]);
    store8(dh + c.row * d + c.col, n, g);
}

// ---------------------------------------------------------------------------
// Argument checks

int32_t check_sizes(int32_t dtype, int64_t rows, int64_t d)
{
    if (!dtype_ok(dtype))
        return fail(GQ_ERR_ARG, "dtype %d is neither GQ_IN_F32 nor GQ_IN_BF16", dtype);
    if (rows < 0 || rows >= ((int64_t)1 << 32) || d < 1 || d >= kMaxColumns)
        return fail(GQ_ERR_ARG, "rows = %lld, d = %lld out of range", (long long)rows,
                    (long long)d);
    if (rows > 0 && groups_of(d) >= (kMaxGroups + rows - 1) / rows)
        return fail(GQ_ERR_UNSUPPORTED, "rows = %lld of d = %lld: 2^29 groups of 32 or more",
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
    if (ld != 0 && ld < d)
        return fail(GQ_ERR_ARG, "%s = %lld: 0 or at least %lld", name, (long long)ld,
                    (long long)d);
    if (ld > ((int64_t)1 << 40))
        return fail(GQ_ERR_ARG, "%s = %lld out of range", name, (long long)ld);
    return GQ_OK;
}

int32_t check_vector(const char *name, const void *p, int64_t align)
{
    if (!aligned_to(p, align))
        return fail(GQ_ERR_ALIGN, "%s is not aligned to its elements", name);
    return GQ_OK;
}

} // namespace

int32_t check_act8(const char *name, const gqt_act8 *a, int64_t rows, bool written)
{
    if (!a)
        return GQ_OK;
    if ((!a->codes || !a->exps) && rows > 0)
        return fail(GQ_ERR_NULL, "%s has no codes or no exps", name);
    if (!aligned_to(a->codes, 16))
        return fail(GQ_ERR_ALIGN, "the codes of %s are not 16-byte aligned", name);
    if (written && a->rounding != GQT_ROUND_NEAREST && a->rounding != GQT_ROUND_RANDOM)
        return fail(GQ_ERR_ARG, "%s: rounding %d", name, a->rounding);
    return GQ_OK;
}

namespace {

constexpr int kCUs = 256;

// Layer norm shapes: threads per row (whole waves from 64 on) and chunks a
// thread, so that few lanes are idle (at half of them d = 256 and 5120 ran at
// 3.4 and 2.7 TB/s; just past 512 and 2048 it is still so: bf16 64527 x 520
// forward runs at 3.1 TB/s, d = 768 at 4.8, 2056 at 3.8, 2304 at 4.1, 2560 at
// 4.6, 1024 and 4096 at 5.6), the gradient's sums do not spill, and registers
// leave room for waves (bf16 8191 x 2048 forward with a random copy: 25 us a call
// with 256 threads a row, 34 with one wave and four chunks).
#define GQT_BY_ROW_LENGTH(LAUNCH, LONG) \
    do {                                \
        if (d <= 32)                    \
            LAUNCH(4, 1);               \
        else if (d <= 64)               \
            LAUNCH(8, 1);               \
        else if (d <= 128)              \
            LAUNCH(16, 1);              \
        else if (d <= 256)              \
            LAUNCH(32, 1);              \
        else if (d <= 512)              \
            LAUNCH(64, 1);              \
        else if (d <= 1024)             \
            LAUNCH(64, 2);              \
        else if (d <= 1536)             \
            LAUNCH(64, 3);              \
        else if (d <= 2048)             \
            LAUNCH(256, 1);             \
        else if (d <= 4096)             \
            LAUNCH(256, 2);             \
        else if (d <= 6144)             \
            LAUNCH(256, 3);             \
        else                            \
            LONG();                     \
    } while (0)

// Rows that one block takes at a time.
int64_t rows_per_block(int64_t d)
{
    return d <= 32 ? 64 : d <= 64 ? 32 : d <= 128 ? 16 : d <= 256 ? 8 : d <= 1536 ? 4 : 1;
}

// Chunks of eight columns that a thread holds, in the shapes above.
int chunks_per_thread(int64_t d)
{
    if (d > 6144)
        return d <= 8192 ? 2 : 4;
    if (d > 4096 || (d > 1024 && d <= 1536))
        return 3;
    return d > 2048 || (d > 512 && d <= 1024) ? 2 : 1;
}

// Blocks of a layer norm launch.  Up to 8 turns each, as many as the
// registers let a CU hold at once, as a part of a round more costs a round:
// us a call for bf16 with a copy, against four turns and at least 8 a CU, 8192
// x 1024 14.5 and 17.2, 16384 x 1536 38.0 and 42.1, 4096 x 4096 25.3 and 27.2.
// Beyond, four turns with the weights in registers, so that late blocks even
// out: forward and backward of 16384 x 4096 131 us, with all that a CU holds
// 138; fp32 65536 x 2048 with a copy 226 and 244.
int64_t norm_blocks(int64_t rows, int64_t d, bool keep)
{
    const int64_t all = (rows + rows_per_block(d) - 1) / rows_per_block(d);
    const int c = chunks_per_thread(d);
    int64_t held = 8 * kCUs;
    if (d <= 16384)
        held = kCUs * (d > 6144 ? 2 : keep ? (c == 1 ? 5 : c == 2 ? 3 : 2)
                                           : (c == 1 ? 8 : c == 2 ? 5 : 4));
    if (all <= held)
        return all;
    return all <= 8 * held ? held : (all + 3) / 4;
}

constexpr int64_t kMostGradColumns = 8192; // beyond, dw and db have a kernel of their own

// Blocks that leave 2 d partial sums each.  As many as their registers let a
// CU hold at once: a part of a round more costs a round (bf16 calls: 16384 x
// 4096 83 us with 3 blocks a CU, 98 with 4; 10922 x 6144 84 with 2, 93 with
// 4; 65536 x 1024 80 with 3, 89 with 4).
int64_t grad_blocks(int64_t rows, int64_t d)
{
    const int64_t all = (rows + rows_per_block(d) - 1) / rows_per_block(d);
    int64_t most;
    if (d > kMostGradColumns) // that many rows of blocks of 2048 columns
        most = (4 * kCUs * 2048 + d - 1) / d;
    else if (d > 6144)
        most = kCUs;
    else
        most = kCUs * (5 - chunks_per_thread(d));
    return all < most ? all : most;
}

template <typename T>
int32_t launch_norm(const void *x, int64_t rows, int32_t d, int64_t ldx, const void *w,
                    const void *b, int32_t wdtype, float eps, void *y, float *mean, float *rstd,
                    const gqt_act8 *sx, const gqt_act8 *sy, hipStream_t st)
{
    const Act8 kx = act8_view(sx, d), ky = act8_view(sy, d);
    const T *xt = (const T *)x;
    T *yt = (T *)y;
    const bool keep = sx || sy;
    const dim3 grid((uint32_t)norm_blocks(rows, d, keep));
#define GQT_KERNEL(TPR, C, KEEP)                                                                 \
    k_layer_norm<T, TPR, C, KEEP><<<grid, block_threads<TPR>(), 0, st>>>(                \
        xt, rows, d, ldx, w, b, wdtype, eps, yt, mean, rstd, kx, ky)
#define GQT_LAUNCH(TPR, C)               \
    do {                                 \
        if (keep)                        \
            GQT_KERNEL(TPR, C, true);    \
        else                             \
            GQT_KERNEL(TPR, C, false);   \
    } while (0)
#define GQT_LONG()                                                                               \
    k_layer_norm_long<T><<<grid, kLongThreads, 0, st>>>(xt, rows, d, ldx, w, b, wdtype, eps, yt, \
                                                        mean, rstd, kx, ky)
#define GQT_LONGER()            \
    do {                        \
        if (d <= 8192)          \
            GQT_LAUNCH(512, 2); \
        else if (d <= 16384)    \
            GQT_LAUNCH(512, 4); \
        else                    \
            GQT_LONG();         \
    } while (0)
    GQT_BY_ROW_LENGTH(GQT_LAUNCH, GQT_LONGER);
#undef GQT_LONGER
#undef GQT_LAUNCH
#undef GQT_KERNEL
#undef GQT_LONG
    return check_launch("k_layer_norm");
}

template <typename T>
int32_t launch_norm_backward(const void *dy, int64_t rows, int32_t d, int64_t lddy, const void *x,
                             int64_t ldx, const gqt_act8 *x8, const float *mean,
                             const float *rstd, const void *w, int32_t wdtype, void *dx,
                             float *partial, hipStream_t st)
{
    const Act8 a = act8_view(x ? nullptr : x8, d);
    const int64_t blocks = grad_blocks(rows, d);
    const dim3 grid((uint32_t)blocks);
    const T *dyt = (const T *)dy, *xt = (const T *)x;
    T *dxt = (T *)dx;
#define GQT_KERNEL(TPR, C, ACT8)                                                                 \
    k_layer_norm_backward<T, TPR, C, ACT8><<<grid, block_threads<TPR>(), 0, st>>>(       \
        dyt, rows, d, lddy, xt, ldx, a, mean, rstd, w, wdtype, dxt, partial)
#define GQT_LAUNCH(TPR, C)               \
    do {                                 \
        if (x)                           \
            GQT_KERNEL(TPR, C, false);   \
        else                             \
            GQT_KERNEL(TPR, C, true);    \
    } while (0)
    if (d > kMostGradColumns) {
        const dim3 all((uint32_t)(rows < 2 * kCUs ? rows : 2 * kCUs));
        if (x)
            k_layer_norm_backward_long<T, false><<<all, kLongThreads, 0, st>>>(
                dyt, rows, d, lddy, xt, ldx, a, mean, rstd, w, wdtype, dxt);
        else
            k_layer_norm_backward_long<T, true><<<all, kLongThreads, 0, st>>>(
                dyt, rows, d, lddy, xt, ldx, a, mean, rstd, w, wdtype, dxt);
        GQT_TRY(check_launch("k_layer_norm_backward_long"));
        if (!partial)
            return ok();
        const dim3 parts((uint32_t)((d + 2047) / 2048), (uint32_t)blocks);
        if (x)
            k_norm_column_sums<T, false><<<parts, 256, 0, st>>>(dyt, rows, d, lddy, xt, ldx, a, mean,
                                                                rstd, partial);
        else
            k_norm_column_sums<T, true><<<parts, 256, 0, st>>>(dyt, rows, d, lddy, xt, ldx, a, mean,
                                                               rstd, partial);
        return check_launch("k_norm_column_sums");
    }
#define GQT_LONGER() GQT_LAUNCH(512, 2)
    GQT_BY_ROW_LENGTH(GQT_LAUNCH, GQT_LONGER);
#undef GQT_LONGER
#undef GQT_LAUNCH
#undef GQT_KERNEL
    return check_launch("k_layer_norm_backward");
}

inline dim3 chunk_grid(uint32_t chunks) { return dim3((chunks + kThreads - 1) / kThreads); }

} // namespace
} // namespace gqt

// ---------------------------------------------------------------------------
// C ABI

using namespace gqt;

extern "C" {

const char *gqt_last_error(void) { return g_err; }

int64_t gqt_act8_groups(int64_t d) { return d < 1 || d >= kMaxColumns ? -1 : groups_of(d); }

int64_t gqt_act8_code_pitch(int64_t d)
{
    return d < 1 || d >= kMaxColumns ? -1 : 32 * groups_of(d);
}

int32_t gqt_act8_save(const void *x, int32_t dtype, int64_t rows, int64_t d, int64_t ldx,
                      const gqt_act8 *out, void *stream)
{
    GQT_TRY(check_sizes(dtype, rows, d));
    GQT_TRY(check_matrix("x", x, dtype, rows));
    GQT_TRY(check_ld("ldx", ldx, d));
    if (!out)
        return fail(GQ_ERR_NULL, "out is NULL");
    GQT_TRY(check_act8("out", out, rows, true));
    if (rows == 0)
        return ok();
    const FastDiv per_row = fast_div((uint32_t)(4 * groups_of(d)));
    const uint32_t chunks = (uint32_t)rows * per_row.d;
    const Act8 a = act8_view(out, d);
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == GQ_IN_F32)
        k_act8_save<float><<<chunk_grid(chunks), kThreads, 0, st>>>((const float *)x, chunks,
                                                                    per_row, (int32_t)d, ldx, a);
    else
        k_act8_save<bf16><<<chunk_grid(chunks), kThreads, 0, st>>>((const bf16 *)x, chunks,
                                                                   per_row, (int32_t)d, ldx, a);
    return check_launch("k_act8_save");
}

int32_t gqt_act8_restore(const gqt_act8 *in, int64_t rows, int64_t d, int32_t dtype, void *out,
                         void *stream)
{
    GQT_TRY(check_sizes(dtype, rows, d));
    if (!in)
        return fail(GQ_ERR_NULL, "in is NULL");
    GQT_TRY(check_act8("in", in, rows, false));
    GQT_TRY(check_matrix("out", out, dtype, rows));
    if (rows == 0)
        return ok();
    const FastDiv per_row = fast_div((uint32_t)(4 * groups_of(d)));
    const uint32_t chunks = (uint32_t)rows * per_row.d;
    const Act8 a = act8_view(in, d);
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == GQ_IN_F32)
        k_act8_restore<float><<<chunk_grid(chunks), kThreads, 0, st>>>(a, chunks, per_row,
                                                                       (int32_t)d, (float *)out);
    else
        k_act8_restore<bf16><<<chunk_grid(chunks), kThreads, 0, st>>>(a, chunks, per_row,
                                                                      (int32_t)d, (bf16 *)out);
    return check_launch("k_act8_restore");
}

int32_t gqt_layer_norm(const void *x, int32_t dtype, int64_t rows, int64_t d, int64_t ldx,
                       const void *w, const void *b, int32_t wdtype, float eps, void *y,
                       float *mean, float *rstd, const gqt_act8 *save_x, const gqt_act8 *save_y,
                       void *stream)
{
    GQT_TRY(check_sizes(dtype, rows, d));
    GQT_TRY(check_matrix("x", x, dtype, rows));
    GQT_TRY(check_ld("ldx", ldx, d));
    if (!dtype_ok(wdtype))
        return fail(GQ_ERR_ARG, "wdtype %d is neither GQ_IN_F32 nor GQ_IN_BF16", wdtype);
    if (!(eps >= 0.0f) || isinf(eps))
        return fail(GQ_ERR_ARG, "eps must be finite and >= 0");
    GQT_TRY(check_matrix("y", y, dtype, rows));
    GQT_TRY(check_vector("w", w, elem_bytes(wdtype)));
    GQT_TRY(check_vector("b", b, elem_bytes(wdtype)));
    GQT_TRY(check_vector("mean", mean, 4));
    GQT_TRY(check_vector("rstd", rstd, 4));
    GQT_TRY(check_act8("save_x", save_x, rows, true));
    GQT_TRY(check_act8("save_y", save_y, rows, true));
    if (rows == 0)
        return ok();
    return dtype == GQ_IN_F32
               ? launch_norm<float>(x, rows, (int32_t)d, ldx, w, b, wdtype, eps, y, mean, rstd,
                                    save_x, save_y, (hipStream_t)stream)
               : launch_norm<bf16>(x, rows, (int32_t)d, ldx, w, b, wdtype, eps, y, mean, rstd,
                                   save_x, save_y, (hipStream_t)stream);
}

int64_t gqt_layer_norm_backward_workspace_bytes(int64_t rows, int64_t d)
{
    if (rows < 0 || rows >= ((int64_t)1 << 32) || d < 1 || d >= kMaxColumns)
        return -1;
    return 8 * d * grad_blocks(rows, d);
}

int32_t gqt_layer_norm_backward(const void *dy, int32_t dtype, int64_t rows, int64_t d,
                                int64_t lddy, const void *x, int64_t ldx, const gqt_act8 *x8,
                                const float *mean, const float *rstd, const void *w,
                                int32_t wdtype, void *dx, void *dw, void *db, void *workspace,
                                int64_t workspace_bytes, void *stream)
{
    GQT_TRY(check_sizes(dtype, rows, d));
    GQT_TRY(check_matrix("dy", dy, dtype, rows));
    GQT_TRY(check_ld("lddy", lddy, d));
    if (x) {
        GQT_TRY(check_matrix("x", x, dtype, rows));
        GQT_TRY(check_ld("ldx", ldx, d));
    } else if (!x8) {
        return fail(GQ_ERR_NULL, "x and x8 are both NULL");
    } else {
        GQT_TRY(check_act8("x8", x8, rows, false));
    }
    if (!dtype_ok(wdtype))
        return fail(GQ_ERR_ARG, "wdtype %d is neither GQ_IN_F32 nor GQ_IN_BF16", wdtype);
    if ((!mean || !rstd) && rows > 0)
        return fail(GQ_ERR_NULL, "mean or rstd is NULL");
    GQT_TRY(check_vector("mean", mean, 4));
    GQT_TRY(check_vector("rstd", rstd, 4));
    GQT_TRY(check_matrix("dx", dx, dtype, rows));
    GQT_TRY(check_vector("w", w, elem_bytes(wdtype)));
    GQT_TRY(check_vector("dw", dw, elem_bytes(wdtype)));
    GQT_TRY(check_vector("db", db, elem_bytes(wdtype)));
    const bool sums = dw || db;
    if (sums) {
        const int64_t need = gqt_layer_norm_backward_workspace_bytes(rows, d);
        if (!workspace && need > 0)
            return fail(GQ_ERR_NULL, "workspace is NULL");
        if (workspace_bytes < need)
            return fail(GQ_ERR_WORKSPACE, "workspace of %lld bytes, %lld are needed",
                        (long long)workspace_bytes, (long long)need);
        if (!aligned_to(workspace, 16))
            return fail(GQ_ERR_ALIGN, "workspace is not 16-byte aligned");
    }
    const hipStream_t st = (hipStream_t)stream;
    float *partial = sums ? (float *)workspace : nullptr;
    if (rows > 0)
        GQT_TRY(dtype == GQ_IN_F32
                    ? launch_norm_backward<float>(dy, rows, (int32_t)d, lddy, x, ldx, x8, mean,
                                                  rstd, w, wdtype, dx, partial, st)
                    : launch_norm_backward<bf16>(dy, rows, (int32_t)d, lddy, x, ldx, x8, mean,
                                                 rstd, w, wdtype, dx, partial, st));
    if (!sums)
        return ok();
    k_sum_partials<<<dim3((uint32_t)((d + 63) / 64), 2), 64 * kSumWaves, 0, st>>>(
        partial, (int32_t)grad_blocks(rows, d), (int32_t)d, dw, db, wdtype);
    return check_launch("k_sum_partials");
}

int32_t gqt_gelu(const void *h, int32_t dtype, int64_t rows, int64_t d, int64_t ldh, int32_t form,
                 void *y, const gqt_act8 *save_h, const gqt_act8 *save_y, void *stream)
{
    GQT_TRY(check_sizes(dtype, rows, d));
    GQT_TRY(check_matrix("h", h, dtype, rows));
    GQT_TRY(check_ld("ldh", ldh, d));
    if (form != GQT_GELU_ERF && form != GQT_GELU_TANH)
        return fail(GQ_ERR_ARG, "form %d", form);
    GQT_TRY(check_matrix("y", y, dtype, rows));
    GQT_TRY(check_act8("save_h", save_h, rows, true));
    GQT_TRY(check_act8("save_y", save_y, rows, true));
    if (rows == 0)
        return ok();
    const FastDiv per_row = fast_div((uint32_t)(4 * groups_of(d)));
    const uint32_t chunks = (uint32_t)rows * per_row.d;
    const Act8 kh = act8_view(save_h, d), ky = act8_view(save_y, d);
    const hipStream_t st = (hipStream_t)stream;
#define GQT_LAUNCH(T, FORM)                                                                      \
    do {                                                                                         \
        if (save_h || save_y)                                                                    \
            k_gelu<T, FORM, true><<<chunk_grid(chunks), kThreads, 0, st>>>(                      \
                (const T *)h, chunks, per_row, (int32_t)d, ldh, (T *)y, kh, ky);                 \
        else                                                                                     \
            k_gelu<T, FORM, false><<<chunk_grid(chunks), kThreads, 0, st>>>(                     \
                (const T *)h, chunks, per_row, (int32_t)d, ldh, (T *)y, kh, ky);                 \
    } while (0)
    if (dtype == GQ_IN_F32) {
        if (form == GQT_GELU_ERF)
            GQT_LAUNCH(float, GQT_GELU_ERF);
        else
            GQT_LAUNCH(float, GQT_GELU_TANH);
    } else if (form == GQT_GELU_ERF) {
        GQT_LAUNCH(bf16, GQT_GELU_ERF);
    } else {
        GQT_LAUNCH(bf16, GQT_GELU_TANH);
    }
#undef GQT_LAUNCH
    return check_launch("k_gelu");
}

int32_t gqt_gelu_backward(const void *dy, int32_t dtype, int64_t rows, int64_t d, int64_t lddy,
                          const void *h, int64_t ldh, const gqt_act8 *h8, int32_t form, void *dh,
                          void *stream)
{
    GQT_TRY(check_sizes(dtype, rows, d));
    GQT_TRY(check_matrix("dy", dy, dtype, rows));
    GQT_TRY(check_ld("lddy", lddy, d));
    if (h) {
        GQT_TRY(check_matrix("h", h, dtype, rows));
        GQT_TRY(check_ld("ldh", ldh, d));
    } else if (!h8) {
        return fail(GQ_ERR_NULL, "h and h8 are both NULL");
    } else {
        GQT_TRY(check_act8("h8", h8, rows, false));
    }
    if (form != GQT_GELU_ERF && form != GQT_GELU_TANH)
        return fail(GQ_ERR_ARG, "form %d", form);
    GQT_TRY(check_matrix("dh", dh, dtype, rows));
    if (rows == 0)
        return ok();
    const FastDiv per_row = fast_div((uint32_t)(4 * groups_of(d)));
    const uint32_t chunks = (uint32_t)rows * per_row.d;
    const Act8 a = act8_view(h ? nullptr : h8, d);
    const hipStream_t st = (hipStream_t)stream;
#define GQT_LAUNCH(T, FORM)                                                                      \
    do {                                                                                         \
        if (h)                                                                                   \
            k_gelu_backward<T, FORM, false><<<chunk_grid(chunks), kThreads, 0, st>>>(            \
                (const T *)dy, chunks, per_row, (int32_t)d, lddy, (const T *)h, ldh, a,          \
                (T *)dh);                                                                        \
        else                                                                                     \
            k_gelu_backward<T, FORM, true><<<chunk_grid(chunks), kThreads, 0, st>>>(             \
                (const T *)dy, chunks, per_row, (int32_t)d, lddy, nullptr, 0, a, (T *)dh);       \
    } while (0)
    if (dtype == GQ_IN_F32) {
        if (form == GQT_GELU_ERF)
            GQT_LAUNCH(float, GQT_GELU_ERF);
        else
            GQT_LAUNCH(float, GQT_GELU_TANH);
    } else if (form == GQT_GELU_ERF) {
        GQT_LAUNCH(bf16, GQT_GELU_ERF);
    } else {
        GQT_LAUNCH(bf16, GQT_GELU_TANH);
    }
#undef GQT_LAUNCH
    return check_launch("k_gelu_backward");
}

} // extern "C"
