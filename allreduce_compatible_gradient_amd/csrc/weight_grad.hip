// weight_grad.hip -- dw = dy^T x and db of a linear layer on MI355X (gfx950),
// with x in the 8-bit format of include/gq_train.h.
//
// Both operands are stored with the reduced axis (the tokens) outermost, so
// a wave's MFMA fragments, eight consecutive tokens of one column, are
// transposed reads of row-major LDS tiles (ds_read_b64_tr_b16).  A code times
// its group's power of two is exact in bf16, so the codes become bf16 on
// their way into LDS and one bf16 MFMA per tile serves a bf16 dy; an fp32 dy
// is the exact sum of three bf16 parts and takes three.  All sums are fp32.
#include "train_common.h"

namespace gqt {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kTileN = 128, kTileK = 128; // output tile: rows of dw, columns of dw
constexpr int kTileM = 32;                // tokens per step: the depth of one MFMA
constexpr int kWgThreads = 256;
// LDS rows of 128 bf16 lie 288 bytes apart: a transposed read takes 32 bytes
// of each of 16 rows, which then fall into all banks evenly.
constexpr int kRowBytes = 288;
constexpr int kTileBytes = kTileM * kRowBytes;

template <typename T>
constexpr int parts() { return sizeof(T) == 4 ? 3 : 1; }

// The bf16 parts of eight values of dy: themselves, or the leading 8, middle
// 8 and last 8 significant bits of each float (truncated, so that the rest
// is exact; an inf or NaN stays in the first part alone).
__device__ __forceinline__ void split(const float (&v)[8], u32x4 (&part)[1])
{
#pragma unroll
    for (int k = 0; k < 4; ++k)
        part[0][k] = __float_as_uint(v[2 * k]) >> 16 | (__float_as_uint(v[2 * k + 1]) & 0xFFFF0000u);
}

__device__ __forceinline__ void split(const float (&v)[8], u32x4 (&part)[3])
{
    uint32_t b[3][8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t u = __float_as_uint(v[k]);
        b[0][k] = u & 0xFFFF0000u;
        const float r1 = (u & 0x7F800000u) == 0x7F800000u ? 0.0f : v[k] - bits_f32(b[0][k]);
        b[1][k] = __float_as_uint(r1) & 0xFFFF0000u;
        b[2][k] = __float_as_uint(r1 - bits_f32(b[1][k]));
        if ((u & 0x7FFFFFFFu) > 0x7F800000u) // a NaN whose payload lies below the cut
            b[0][k] = 0x7FC00000u;
    }
#pragma unroll
    for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            part[p][k] = b[p][2 * k] >> 16 | (b[p][2 * k + 1] & 0xFFFF0000u);
}

__device__ __forceinline__ s16x8 read_fragment(const char *tile, int col)
{
    // lane l reads columns col + l % 16, tokens 4 (l / 16) + {0..3} and 16 more
    const int lane = threadIdx.x & 63;
    const char *p = tile + (lane >> 2) * kRowBytes + (col + (lane & 3) * 4) * 2;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 16 * kRowBytes));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// One block: the 128 x 128 tile (blockIdx.x over n, blockIdx.y over k) of
// the tokens [z chunk, (z + 1) chunk).  out: dw itself (one split) or the
// z-th fp32 partial.
template <typename T, typename O>
__global__ __launch_bounds__(kWgThreads) void k_weight_grad(
    const T *__restrict__ dy, int64_t m, int32_t n, int64_t lddy, Act8 x, int32_t k, int64_t chunk,
    O *__restrict__ dw, O *__restrict__ db)
{
    constexpr int P = parts<T>();
    __shared__ __align__(16) char lds[(P + 1) * kTileBytes];
    char *const lds_b = lds + P * kTileBytes;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int n0 = blockIdx.x * kTileN, k0 = blockIdx.y * kTileK;
    const int wn = (wave & 1) * 64, wk = (wave >> 1) * 64;
    const int64_t m_begin = (int64_t)blockIdx.z * chunk;
    const int64_t m_end = m_begin + chunk < m ? m_begin + chunk : m;
    const bool with_bias = db != nullptr && blockIdx.y == 0 && wk == 0;

    f32x4 acc[4][4] = {}, bias[4] = {};
    s16x8 ones;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        ones[j] = 0x3F80;

    for (int64_t m0 = m_begin; m0 < m_end; m0 += kTileM) {
        // dy: rows t / 16 and 16 more, eight columns
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = t / 16 + 16 * i, c = (t % 16) * 8;
            float v[8];
            const int left = m0 + r < m_end ? n - n0 - c : 0;
            load8(dy + (left > 0 ? (m0 + r) * lddy + n0 + c : 0), left, v);
            u32x4 part[P];
            split(v, part);
#pragma unroll
            for (int p = 0; p < P; ++p)
                *reinterpret_cast<u32x4 *>(lds + p * kTileBytes + r * kRowBytes + c * 2) = part[p];
        }
        // codes: row t / 8, sixteen columns (half a group)
        {
            const int r = t / 8, c = (t % 8) * 16;
            float v[2][8] = {};
            if (m0 + r < m_end && k0 + c < x.pitch) {
                restore8(x, m0 + r, k0 + c, v[0]);
                restore8(x, m0 + r, k0 + c + 8, v[1]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 part[1];
                split(v[h], part);
                *reinterpret_cast<u32x4 *>(lds_b + r * kRowBytes + (c + 8 * h) * 2) = part[0];
            }
        }
        __syncthreads();
        s16x8 fb[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            fb[j] = read_fragment(lds_b, wk + 16 * j);
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const s16x8 fa = read_fragment(lds + p * kTileBytes, wn + 16 * i);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, fa), __builtin_bit_cast(bf16x8, fb[j]),
                        acc[i][j], 0, 0, 0);
                if (with_bias)
                    bias[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, fa), __builtin_bit_cast(bf16x8, ones), bias[i],
                        0, 0, 0);
            }
        __syncthreads();
    }

    // lane l holds rows 4 (l / 16) + {0..3} of column l % 16
    O *const out = dw + (int64_t)blockIdx.z * n * k;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = n0 + wn + 16 * i + 4 * (lane >> 4) + r;
            if (row >= n)
                continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = k0 + wk + 16 * j + (lane & 15);
                if (col < k)
                    out[(int64_t)row * k + col] = (O)acc[i][j][r];
            }
            if (with_bias && (lane & 15) == 0)
                db[(int64_t)blockIdx.z * n + row] = (O)bias[i][r];
        }
}

// Adds `splits` partials in order: count values of dw (or db).
template <typename O>
__global__ __launch_bounds__(256) void k_sum_splits(const float *__restrict__ part, int32_t splits,
                                                    int64_t count, O *__restrict__ out)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= count)
        return;
    float s = 0.0f;
    for (int z = 0; z < splits; ++z)
        s += part[z * count + i];
    out[i] = (O)s;
}

// How the tokens are split: enough blocks for two per CU, chunks of at least
// 256 tokens.
struct Split {
    int32_t splits;
    int64_t chunk;
};
Split split_of(int64_t m, int64_t n, int64_t k)
{
    const int64_t tiles = ((n + kTileN - 1) / kTileN) * ((k + kTileK - 1) / kTileK);
    int64_t s = 512 / tiles;
    if (s > (m + 255) / 256)
        s = (m + 255) / 256;
    if (s < 1)
        s = 1;
    Split r;
    r.chunk = (m + s - 1) / s;
    r.chunk = (r.chunk + kTileM - 1) / kTileM * kTileM;
    if (r.chunk < kTileM)
        r.chunk = kTileM;
    r.splits = (int32_t)((m + r.chunk - 1) / r.chunk);
    if (r.splits < 1)
        r.splits = 1;
    return r;
}

bool sizes_ok(int64_t m, int64_t n, int64_t k)
{
    return m >= 0 && m < ((int64_t)1 << 32) && n >= 1 && n <= 0x7FFFFFFF - 255 && k >= 1 &&
           k <= 0x7FFFFFFF - 255 && k < (((int64_t)1 << 40) + n - 1) / n;
}

template <typename T>
int32_t launch(const void *dy, int64_t m, int32_t n, int64_t lddy, const Act8 &x, int32_t k,
               void *dw, void *db, int32_t wdtype, float *ws, hipStream_t st)
{
    const Split s = split_of(m, n, k);
    const dim3 grid((n + kTileN - 1) / kTileN, (k + kTileK - 1) / kTileK, s.splits);
    const T *dyt = (const T *)dy;
    if (s.splits == 1) {
        if (wdtype == GQ_IN_F32)
            k_weight_grad<T, float><<<grid, kWgThreads, 0, st>>>(dyt, m, n, lddy, x, k, s.chunk,
                                                                 (float *)dw, (float *)db);
        else
            k_weight_grad<T, bf16><<<grid, kWgThreads, 0, st>>>(dyt, m, n, lddy, x, k, s.chunk,
                                                                (bf16 *)dw, (bf16 *)db);
        return check_launch("k_weight_grad");
    }
    const int64_t count = (int64_t)n * k;
    float *const db_part = ws + s.splits * count;
    k_weight_grad<T, float><<<grid, kWgThreads, 0, st>>>(dyt, m, n, lddy, x, k, s.chunk, ws,
                                                         db ? db_part : nullptr);
    GQT_TRY(check_launch("k_weight_grad"));
    const auto blocks = [](int64_t c) { return dim3((uint32_t)((c + 255) / 256)); };
    if (wdtype == GQ_IN_F32) {
        k_sum_splits<float><<<blocks(count), 256, 0, st>>>(ws, s.splits, count, (float *)dw);
        if (db)
            k_sum_splits<float><<<blocks(n), 256, 0, st>>>(db_part, s.splits, n, (float *)db);
    } else {
        k_sum_splits<bf16><<<blocks(count), 256, 0, st>>>(ws, s.splits, count, (bf16 *)dw);
        if (db)
            k_sum_splits<bf16><<<blocks(n), 256, 0, st>>>(db_part, s.splits, n, (bf16 *)db);
    }
    return check_launch("k_sum_splits");
}

} // namespace
} // namespace gqt

using namespace gqt;

extern "C" {

int64_t gqt_weight_grad_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t dtype)
{
    if (!sizes_ok(m, n, k) || !dtype_ok(dtype))
        return -1;
    const Split s = split_of(m, n, k);
    return s.splits > 1 ? 4 * s.splits * (n * k + n) : 0;
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
    return dtype == GQ_IN_F32
               ? launch<float>(dy, m, (int32_t)n, lddy, x, (int32_t)k, dw, db, wdtype,
                               (float *)workspace, (hipStream_t)stream)
               : launch<bf16>(dy, m, (int32_t)n, lddy, x, (int32_t)k, dw, db, wdtype,
                              (float *)workspace, (hipStream_t)stream);
}

} // extern "C"
