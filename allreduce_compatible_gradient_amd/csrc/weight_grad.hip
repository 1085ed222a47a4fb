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
constexpr int kStepM = 64;                // tokens per step: 32 for each half of the waves
constexpr int kWgThreads = 512;
// LDS rows of 128 bf16 lie 288 bytes apart: a transposed read takes 32 bytes
// of each of 16 rows, which then fall into all banks evenly.
constexpr int kRowBytes = 288;
constexpr int kTileBytes = kStepM * kRowBytes;

template <typename T>
constexpr int parts() { return sizeof(T) == 4 ? 3 : 1; }

// One thread's share of a step as loaded: rows r and r + 32, eight columns.
template <typename T>
struct Loaded {
    u32x4 a[2][sizeof(T) / 2];
    u32x2 b[2];
    uint32_t e[2];
};

__device__ __forceinline__ void load_raw(const bf16 *p, u32x4 (&w)[1])
{
    w[0] = *reinterpret_cast<const u32x4_e2 *>(p);
}
__device__ __forceinline__ void load_raw(const float *p, u32x4 (&w)[2])
{
    w[0] = *reinterpret_cast<const u32x4_e4 *>(p);
    w[1] = *reinterpret_cast<const u32x4_e4 *>(p + 4);
}
// the first n elements, the others 0
__device__ __forceinline__ void load_raw_part(const bf16 *p, int n, u32x4 (&w)[1])
{
    const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        w[0][k] = 2 * k < n ? q[2 * k] : 0u;
        w[0][k] |= 2 * k + 1 < n ? (uint32_t)q[2 * k + 1] << 16 : 0u;
    }
}
__device__ __forceinline__ void load_raw_part(const float *p, int n, u32x4 (&w)[2])
{
    const uint32_t *q = reinterpret_cast<const uint32_t *>(p);
#pragma unroll
    for (int k = 0; k < 8; ++k)
        w[k / 4][k % 4] = k < n ? q[k] : 0u;
}

// The bf16 parts of eight values of dy: themselves, or the leading 8, middle
// 8 and last 8 significant bits of each float (truncated, so that the rest
// is exact; an inf or NaN stays in the first part alone).
__device__ __forceinline__ void split(const u32x4 (&w)[1], u32x4 (&part)[1]) { part[0] = w[0]; }

__device__ __forceinline__ void split(const u32x4 (&w)[2], u32x4 (&part)[3])
{
    uint32_t b[3][8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t u = w[k / 4][k % 4];
        b[0][k] = u & 0xFFFF0000u;
        const float r1 = (u & 0x7F800000u) == 0x7F800000u ? 0.0f : bits_f32(u) - bits_f32(b[0][k]);
        b[1][k] = __float_as_uint(r1) & 0xFFFF0000u;
        b[2][k] = __float_as_uint(r1 - bits_f32(b[1][k]));
        if ((u & 0x7FFFFFFFu) > 0x7F800000u) // a NaN whose payload lies below the cut
            b[0][k] = 0x7FC00000u;
    }
#pragma unroll
    for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int k = 0; k < 4; ++k) // the upper halves of a pair
            part[p][k] = __builtin_amdgcn_perm(b[p][2 * k + 1], b[p][2 * k], 0x07060302u);
}

// Eight codes as bf16.  A code + 128 is an unsigned byte, which one
// instruction makes a float; (code + 128) step - 128 step is exact.
__device__ __forceinline__ u32x4 decode8(u32x2 codes, uint32_t e)
{
    const float step = step_of(e), off = -128.0f * step;
    u32x4 r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t u = codes[h] ^ 0x80808080u;
        float f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            f[k] = fmaf((float)((u >> (8 * k)) & 0xFFu), step, off);
        r[2 * h] = __builtin_amdgcn_perm(__float_as_uint(f[1]), __float_as_uint(f[0]), 0x07060302u);
        r[2 * h + 1] =
            __builtin_amdgcn_perm(__float_as_uint(f[3]), __float_as_uint(f[2]), 0x07060302u);
    }
    return r;
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

struct Tiles {
    int32_t n, k, total; // tiles along n and k, and blocks (times the splits)
};

// One block: a 128 x 128 tile of dw over the tokens of one split.  Its two
// halves of four waves take 32 of each step's 64 tokens, a 64 x 64 quarter
// of the tile a wave, and are added at the end.  out: dw itself (one split)
// or the split's fp32 partial.  BIAS: the tile also sums dy's rows, as a
// product with ones.
//
// Columns of the tile past n or past the codes' pitch may hold anything:
// they reach only values of dw that are not stored.  So every lane loads
// eight columns that exist, and the lane whose eight would end past n loads
// the row's last eight and places them one by one.
template <typename T, typename O, bool BIAS>
__device__ __forceinline__ void weight_grad_tile(const T *__restrict__ dy, int32_t n, int64_t lddy,
                                                 const Act8 &x, int32_t k, int64_t m_begin,
                                                 int64_t m_end, int n0, int k0,
                                                 O *__restrict__ out, O *__restrict__ db,
                                                 char *lds)
{
    constexpr int P = parts<T>();
    constexpr int kBufBytes = (P + 1) * kTileBytes;
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int half = wave >> 2, wn = (wave & 1) * 64, wk = ((wave >> 1) & 1) * 64;
    const int r = t / 16, c = (t % 16) * 8;
    const int left = n - n0 - c;
    const bool odd = left > 0 && left < 8; // eight columns from n - 8, from column `from` of the tile
    const int from = n - 8 - n0;
    const int dy_col = n < 8 ? 0 : odd ? n - 8 : left > 0 ? n0 + c : 0;
    const int code_col = k0 + c < x.pitch ? k0 + c : 0;

    const auto load_dy = [&](Loaded<T> &l, int i, int64_t row) {
        const T *const p = dy + row * lddy + dy_col;
        if (n >= 8)
            load_raw(p, l.a[i]);
        else
            load_raw_part(p, n, l.a[i]);
    };
    const auto load_codes = [&](Loaded<T> &l, int i, int64_t row) {
        l.b[i] = *reinterpret_cast<const u32x2 *>(x.codes + row * x.pitch + code_col);
        l.e[i] = x.exps[row * x.groups + (code_col >> 5)];
    };
    const auto load = [&](Loaded<T> &l, int64_t m0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            load_dy(l, i, m0 + r + 32 * i);
            load_codes(l, i, m0 + r + 32 * i);
        }
    };
    // the last step: past the last token, that token again with a dy of 0
    const auto load_tail = [&](Loaded<T> &l, int64_t m0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t want = m0 + r + 32 * i, row = want < m_end ? want : m_end - 1;
            load_dy(l, i, row);
            load_codes(l, i, row);
            if (want >= m_end)
#pragma unroll
                for (size_t h = 0; h < sizeof(T) / 2; ++h)
                    l.a[i][h] = u32x4{0, 0, 0, 0};
        }
    };
    const auto store = [&](const Loaded<T> &l, char *buf) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            char *const at = buf + (r + 32 * i) * kRowBytes;
            u32x4 part[P];
            split(l.a[i], part);
            if (odd && n >= 8) {
#pragma unroll
                for (int p = 0; p < P; ++p)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (from + e >= 0)
                            *reinterpret_cast<uint16_t *>(at + p * kTileBytes + (from + e) * 2) =
                                (uint16_t)(part[p][e / 2] >> (16 * (e % 2)));
            } else {
#pragma unroll
                for (int p = 0; p < P; ++p)
                    *reinterpret_cast<u32x4 *>(at + p * kTileBytes + c * 2) = part[p];
            }
            *reinterpret_cast<u32x4 *>(at + P * kTileBytes + c * 2) = decode8(l.b[i], l.e[i]);
        }
    };

    f32x4 acc[4][4] = {}, bias[4] = {};
    s16x8 ones;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        ones[j] = 0x3F80;
    const auto multiply = [&](const char *buf) {
        const char *const a = buf + half * 32 * kRowBytes, *const b = a + P * kTileBytes;
        s16x8 fb[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            fb[j] = read_fragment(b, wk + 16 * j);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            s16x8 fa[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                fa[i] = read_fragment(a + p * kTileBytes, wn + 16 * i);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, fa[i]), __builtin_bit_cast(bf16x8, fb[j]),
                        acc[i][j], 0, 0, 0);
                if (BIAS)
                    bias[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, fa[i]), __builtin_bit_cast(bf16x8, ones),
                        bias[i], 0, 0, 0);
            }
        }
    };

    // Step s + 2 is loaded, step s multiplied, and step s + 1 (loaded a step
    // ago) decoded into the other buffer, which the barrier of step s - 1
    // freed.  Tokens that do not fill a step come last, on their own.
    const int steps = (int)((m_end - m_begin) / kStepM);
    Loaded<T> reg[2];
    const auto step = [&](int s, int i) {
        if (s + 2 < steps)
            load(reg[i], m_begin + (int64_t)(s + 2) * kStepM);
        multiply(lds + i * kBufBytes);
        if (s + 1 < steps)
            store(reg[1 - i], lds + (1 - i) * kBufBytes);
        __syncthreads();
    };
    if (steps > 0) {
        load(reg[0], m_begin);
        if (steps > 1)
            load(reg[1], m_begin + kStepM);
        store(reg[0], lds);
        __syncthreads();
    }
    for (int s = 0; s < steps; s += 2) {
        step(s, 0);
        if (s + 1 < steps)
            step(s + 1, 1);
    }
    if (m_begin + (int64_t)steps * kStepM < m_end) {
        load_tail(reg[0], m_begin + (int64_t)steps * kStepM);
        store(reg[0], lds);
        __syncthreads();
        multiply(lds);
        __syncthreads();
    }

    // The halves trade: each keeps two of the four rows of MFMA tiles and
    // gets the other half's sums of them.
    f32x4(*const trade)[4][2][5][64] = reinterpret_cast<f32x4(*)[4][2][5][64]>(lds);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f32x4(*const to)[64] = trade[half][wave & 3][i];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            to[j][lane] = half ? acc[i][j] : acc[2 + i][j];
        if (BIAS)
            to[4][lane] = half ? bias[i] : bias[2 + i];
    }
    __syncthreads();
    // lane l holds rows 4 (l / 16) + {0..3} of column l % 16
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f32x4(*const from)[64] = trade[1 - half][wave & 3][i];
        const int row0 = n0 + wn + 16 * (2 * half + i) + 4 * (lane >> 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f32x4 v = (half ? acc[2 + i][j] : acc[i][j]) + from[j][lane];
            const int col = k0 + wk + 16 * j + (lane & 15);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (row0 + e < n && col < k)
                    out[(int64_t)(row0 + e) * k + col] = (O)v[e];
        }
        if (BIAS && wk == 0) {
            const f32x4 v = (half ? bias[2 + i] : bias[i]) + from[4][lane];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (row0 + e < n && (lane & 15) == 0)
                    db[row0 + e] = (O)v[e];
        }
    }
}

template <typename T, typename O>
__global__ __launch_bounds__(kWgThreads) void k_weight_grad(
    const T *__restrict__ dy, int64_t m, int32_t n, int64_t lddy, Act8 x, int32_t k, int64_t chunk,
    Tiles tiles, O *__restrict__ dw, O *__restrict__ db)
{
    constexpr int kBufBytes = 2 * (parts<T>() + 1) * kTileBytes;
    constexpr int kTradeBytes = 2 * 4 * 2 * 5 * 64 * 16; // the halves' sums
    __shared__ __align__(16) char lds[kBufBytes > kTradeBytes ? kBufBytes : kTradeBytes];
    // Blocks go to the 8 XCDs in turn; each XCD takes a contiguous run of
    // tiles, k fastest, so that its L2 holds the rows of dy they share.
    const int xcd = blockIdx.x % 8, q = tiles.total / 8, rem = tiles.total % 8;
    const int tile = xcd * q + min(xcd, rem) + blockIdx.x / 8;
    const int tk = tile % tiles.k, tn = tile / tiles.k % tiles.n, z = tile / tiles.k / tiles.n;
    const int n0 = tn * kTileN, k0 = tk * kTileK;
    const int64_t m_begin = (int64_t)z * chunk;
    const int64_t m_end = m_begin + chunk < m ? m_begin + chunk : m;
    O *const out = dw + (int64_t)z * n * k;
    O *const out_b = db ? db + (int64_t)z * n : nullptr;
    if (out_b && tk == 0)
        weight_grad_tile<T, O, true>(dy, n, lddy, x, k, m_begin, m_end, n0, k0, out, out_b, lds);
    else
        weight_grad_tile<T, O, false>(dy, n, lddy, x, k, m_begin, m_end, n0, k0, out, out_b, lds);
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

// How the tokens are split: enough blocks for every CU, chunks of at least
// 256 tokens.
struct Split {
    int32_t splits;
    int64_t chunk;
};
Split split_of(int64_t m, int64_t n, int64_t k)
{
    const int64_t tiles = ((n + kTileN - 1) / kTileN) * ((k + kTileK - 1) / kTileK);
    int64_t s = 256 / tiles;
    if (s > (m + 255) / 256)
        s = (m + 255) / 256;
    if (s < 1)
        s = 1;
    Split r;
    r.chunk = (m + s - 1) / s;
    r.chunk = (r.chunk + kStepM - 1) / kStepM * kStepM;
    if (r.chunk < kStepM)
        r.chunk = kStepM;
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
    Tiles tiles{(n + kTileN - 1) / kTileN, (k + kTileK - 1) / kTileK, 0};
    tiles.total = tiles.n * tiles.k * s.splits; // n k < 2^40: below 2^26 tiles, split or not
    const dim3 grid((uint32_t)tiles.total);
    const T *dyt = (const T *)dy;
    if (s.splits == 1) {
        if (wdtype == GQ_IN_F32)
            k_weight_grad<T, float><<<grid, kWgThreads, 0, st>>>(dyt, m, n, lddy, x, k, s.chunk, tiles,
                                                                 (float *)dw, (float *)db);
        else
            k_weight_grad<T, bf16><<<grid, kWgThreads, 0, st>>>(dyt, m, n, lddy, x, k, s.chunk, tiles,
                                                                (bf16 *)dw, (bf16 *)db);
        return check_launch("k_weight_grad");
    }
    const int64_t count = (int64_t)n * k;
    float *const db_part = ws + s.splits * count;
    k_weight_grad<T, float><<<grid, kWgThreads, 0, st>>>(dyt, m, n, lddy, x, k, s.chunk, tiles, ws,
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
