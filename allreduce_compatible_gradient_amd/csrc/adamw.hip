// adamw.hip -- AdamW over many tensors at once, its moments in 32 or 8 bits,
// and the gradients' norm, on MI355X (gfx950): include/gq_step.h.
//
// A launch takes up to 64 tensors, whose addresses are kernel arguments: no
// table in device memory has to be written before it, or kept until it ran,
// and a captured graph holds them.  A block has a chunk of one tensor, eight
// elements a lane and step, so that sixteen lanes hold one 128-element block
// of the 8-bit formats and one Philox call serves a lane's eight roundings of
// one array.
#include "step_common.h"

#include <stdarg.h>
#include <stdio.h>

#include <algorithm>
#include <new>

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

constexpr int kThreads = 256;
constexpr int kTensors = 64;                     // of a launch: 3.9 KB of arguments
constexpr int64_t kStep = 8 * kThreads;          // elements of a block's step
constexpr int64_t kFew = kStep * 2048;           // elements in all that take one step a block
constexpr int64_t kMaxElements = (int64_t)1 << 34; // i / 8 is one word of the counter, and
                                                    // a launch has fewer than 2^32 threads

// Where a launch's tensors are; tensor j has the blocks from first[j] on.
struct Tensors {
    gqs_tensor t[kTensors];
    uint32_t first[kTensors + 1];
    int32_t count;
    uint32_t number; // of t[0] in the whole list
    int32_t chunk;   // elements of a block
};

// The tensor of this block: the last whose first block is not behind it.
__device__ __forceinline__ int tensor_of(const Tensors &a, uint32_t block)
{
    int lo = 0, hi = a.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (a.first[mid] <= block)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// What the step's number and rate come to; on the device where they are there.
struct Coefs {
    float decay; // 1 - lr weight_decay
    float size;  // lr / (1 - beta1^step)
    float root;  // 1 / sqrt(1 - beta2^step)
    uint32_t step;
};

__host__ __device__ inline Coefs coefs_of(double lr, double beta1, double beta2,
                                          double weight_decay, int64_t step)
{
    Coefs c;
    c.decay = (float)(1.0 - lr * weight_decay);
    c.size = (float)(lr / (1.0 - pow(beta1, (double)step)));
    c.root = (float)(1.0 / sqrt(1.0 - pow(beta2, (double)step)));
    c.step = (uint32_t)step;
    return c;
}

__global__ void k_coefs(double lr, const float *lr_device, double beta1, double beta2,
                        double weight_decay, int64_t step, const int64_t *step_device, Coefs *out)
{
    *out = coefs_of(lr_device ? (double)*lr_device : lr, beta1, beta2, weight_decay,
                    step_device ? *step_device : step);
}

struct Rates {
    float beta1, other1; // and 1 - beta1, rounded on its own
    float beta2, other2;
    float eps;
    uint32_t k0, k1;
    int32_t random; // a bf16 p
};

// Rounds to bf16 at random and stores the first n: u is added below its last
// place, and the upper halves are the result.  What is not finite stays as it
// is (a NaN whose bits are all ones would become 0).
__device__ __forceinline__ void store_random8(bf16 *p, int n, float (&v)[8], const uint4 &draw)
{
    float bad = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        bad = fmaf(v[k], 0.0f, bad); // NaN from an inf or NaN
    uint32_t t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
        t[k] = __float_as_uint(v[k]) + half16(draw, k);
    if (bad != bad || n < 8) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t b = __float_as_uint(v[k]);
            v[k] = (b & 0x7FFFFFFFu) < 0x7F800000u ? bits_f32(t[k] & 0xFFFF0000u) : v[k];
        }
        store8(p, n, v);
        return;
    }
    u32x4 w;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        w[k] = perm(t[2 * k + 1], t[2 * k], 0x07060302u);
    *reinterpret_cast<u32x4_e2 *>(p) = w;
}

// P, G: the parameter's and gradient's types; BITS of the moments.
//
// One pass, bound by memory: 12 + 16 bytes an fp32 element with its 32-bit
// moments, 6 + 16 a bf16 one, 6 + 4 with 8-bit moments.  33.6M fp32 elements
// 165 us, 5.7 TB/s; 201M of bf16 862, 5.1; 33.6M of bf16 with 8-bit moments 57
// us, 5.9, 201M 394, 5.1, where about 650 vector instructions for eight elements, more than
// half of them the three Philox calls, take nearly as long as the memory.  A
// block of 128 of the 8-bit moments is in registers when its new power of two
// is found, so neither is read twice.
template <typename P, typename G, int BITS>
__global__ __launch_bounds__(kThreads) void k_adamw(const Tensors a, Coefs by_value,
                                                    const Coefs *__restrict__ coefs, Rates r,
                                                    const float *__restrict__ scale)
{
    const int j = tensor_of(a, blockIdx.x);
    const gqs_tensor &t = a.t[j];
    const Coefs c = coefs ? *coefs : by_value;
    const float factor = scale ? *scale : 1.0f;
    const int64_t base = (int64_t)(blockIdx.x - a.first[j]) * a.chunk;
    const int32_t n = (int32_t)min(t.n - base, (int64_t)a.chunk);
    // whole 128-element blocks, for the codes past n
    const int32_t end = BITS == 8 ? (n + 127) / 128 * 128 : n;
    P *const p = (P *)t.p + base;
    const G *const g = (const G *)t.g + base;
    const uint32_t number = a.number + j;
    for (int32_t i = 8 * threadIdx.x; i < end; i += 8 * kThreads) {
        float pv[8], gv[8], m[8], v[8];
        float keep1 = r.beta1, keep2 = r.beta2; // of m and v as they are in registers
        uint32_t least = 0;                     // bits of what the root takes at least
        load8(p, i, n, pv);
        load8(g, i, n, gv);
        if constexpr (BITS == 8) {
            // The steps, powers of two, go into the factors.
            const int64_t at = base + i;
            const u32x2 wm = *reinterpret_cast<const u32x2 *>((const uint8_t *)t.m + at);
            const u32x2 wv = *reinterpret_cast<const u32x2 *>((const uint8_t *)t.v + at);
            const uint32_t em = ((const uint8_t *)t.m_exps)[at / 128];
            const uint32_t ev = ((const uint8_t *)t.v_exps)[at / 128];
            e4m3_values(wm, 1.0f, m);
            keep1 *= step_of(em);
            // The lowest step of v's block as it came: a v below it is mostly 0
            // there, while its m is now and then a whole lowest step, whose
            // quotient would have no bound.
            least = (max(ev, 18u) - 18u) << 23;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = e5m3_small(wv, k);
            if (ev <= 143u) { // 2^111 2^E has a float
                keep2 *= bits_f32((ev + 111u) << 23);
            } else {
                keep2 *= step_of(ev);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] *= 0x1p111f;
            }
        } else {
            load8((const float *)t.m + base, i, n, m);
            load8((const float *)t.v + base, i, n, v);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float gs = gv[k] * factor;
            m[k] = fmaf(keep1, m[k], r.other1 * gs);
            v[k] = fmaf(keep2, v[k], r.other2 * (gs * gs));
            // The 8-bit moments' roundings leave no time for a division and a
            // root to the last bit: a unit in the last place each.  The bits of
            // numbers from 0 on are in their order, a NaN's above all.
            const float under = bits_f32(max(__float_as_uint(v[k]), least));
            const float change =
                BITS == 8 ? m[k] * __builtin_amdgcn_rcpf(
                                       fmaf(__builtin_amdgcn_sqrtf(under), c.root, r.eps))
                          : m[k] / fmaf(sqrtf(v[k]), c.root, r.eps);
            pv[k] = fmaf(-c.size, change, pv[k] * c.decay);
        }
        const uint32_t eighth = (uint32_t)((base + i) >> 3);
        if (i < n) {
            if constexpr (sizeof(P) == 2) {
                if (r.random)
                    store_random8(p + i, n - i, pv,
                                  philox10(make_uint4(eighth, c.step, number, 2u), r.k0, r.k1));
                else
                    store8(p + i, n - i, pv);
            } else {
                store8(p + i, n - i, pv);
            }
        }
        if constexpr (BITS == 8) {
            const int64_t at = base + i;
            if (n - i < 8) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (i + k >= n)
                        m[k] = v[k] = 0.0f;
            }
            const uint32_t em = e4m3_exponent(row16_max(abs_bits(m)));
            const uint32_t ev = e5m3_exponent(row16_max(abs_bits(v)));
            u32x2 wm = {0, 0}, wv = {0, 0};
            if (em != 255u)
                wm = e4m3_random8(m, em, philox10(make_uint4(eighth, c.step, number, 0u), r.k0, r.k1));
            if (ev != 255u)
                wv = e5m3_random8(v, ev, philox10(make_uint4(eighth, c.step, number, 1u), r.k0, r.k1));
            *reinterpret_cast<u32x2 *>((uint8_t *)t.m + at) = wm;
            *reinterpret_cast<u32x2 *>((uint8_t *)t.v + at) = wv;
            if ((i & 127) == 0) {
                ((uint8_t *)t.m_exps)[at / 128] = (uint8_t)em;
                ((uint8_t *)t.v_exps)[at / 128] = (uint8_t)ev;
            }
        } else if (i < n) {
            store8((float *)t.m + base + i, n - i, m);
            store8((float *)t.v + base + i, n - i, v);
        }
    }
}

// ---------------------------------------------------------------------------
// the values of a moment: 33.6M to bf16 16 us, 6.2 TB/s

template <typename T, bool SECOND>
__global__ __launch_bounds__(kThreads) void k_moment8_restore(const uint8_t *__restrict__ codes,
                                                              const uint8_t *__restrict__ exps,
                                                              int64_t n, T *__restrict__ out)
{
    const int64_t i = 8 * ((int64_t)blockIdx.x * kThreads + threadIdx.x);
    if (i >= n)
        return;
    const u32x2 w = *reinterpret_cast<const u32x2 *>(codes + i);
    const float step = step_of(exps[i / 128]);
    float v[8];
    if constexpr (SECOND)
        e5m3_values(w, step, v);
    else
        e4m3_values(w, step, v);
    store8(out + i, (int)min(n - i, (int64_t)8), v);
}

// ---------------------------------------------------------------------------
// the norm

// Each block adds the squares of a chunk whose loads are all out at once, and
// a last one their sums, in a fixed order.  fp64 throughout: 8 fused
// operations for 16 or 32 bytes stay behind the memory, and no scaling is
// needed against overflow.  33.6M fp32 in a graph with k_norm 27 us, 4.9
// TB/s; bf16 13.
constexpr int64_t kNormChunk = kStep * 8;

// The sum of v over the block, in thread 0.
__device__ __forceinline__ double block_sum(double v)
{
    __shared__ double lds[kThreads / 64];
#pragma unroll
    for (int o = 1; o < 64; o <<= 1)
        v += __shfl_xor(v, o);
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w)
        v += lds[w];
    return v;
}

template <typename G>
__global__ __launch_bounds__(kThreads) void k_square_sums(const Tensors a,
                                                          double *__restrict__ parts)
{
    const int j = tensor_of(a, blockIdx.x);
    const int64_t base = (int64_t)(blockIdx.x - a.first[j]) * kNormChunk;
    const int32_t n = (int32_t)min(a.t[j].n - base, kNormChunk);
    const G *const g = (const G *)a.t[j].g + base;
    double sum = 0.0;
    const auto add = [&](const Raw8<G> &r) {
        float v[8];
        unpack(r, v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            sum = fma((double)v[k], (double)v[k], sum);
    };
    if (n == kNormChunk) { // all loads at once
        Raw8<G> r[kNormChunk / kStep];
#pragma unroll
        for (int k = 0; k < kNormChunk / kStep; ++k)
            load_words(g + 8 * threadIdx.x + k * kStep, r[k]);
#pragma unroll
        for (int k = 0; k < kNormChunk / kStep; ++k)
            add(r[k]);
    } else {
        for (int32_t i = 8 * threadIdx.x; i < n; i += kStep) {
            Raw8<G> r;
            load_ahead(g, i, n, r);
            settle(g, i, n, r);
            add(r);
        }
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0)
        parts[blockIdx.x] = sum;
}

__global__ __launch_bounds__(kThreads) void k_norm(const double *__restrict__ parts, int64_t count,
                                                   double max_norm, float *__restrict__ norm,
                                                   float *__restrict__ scale)
{
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < count; i += kThreads)
        sum += parts[i];
    sum = sqrt(block_sum(sum));
    if (threadIdx.x == 0) {
        *norm = (float)sum;
        if (scale) {
            const double s = max_norm / (sum + 1e-6);
            *scale = s > 1.0 ? 1.0f : (float)s; // a NaN stays
        }
    }
}

// ---------------------------------------------------------------------------
// host

// Begins a launch at tensor `from`: as many as fit, skipping empty ones.
// Returns the tensor behind them.
int64_t gather(const gqs_tensor *tensors, int64_t count, int64_t from, int64_t chunk, Tensors &a,
               bool number_each)
{
    a.chunk = (int32_t)chunk;
    a.count = 0;
    a.first[0] = 0;
    a.number = (uint32_t)from;
    for (; from < count && a.count < kTensors; ++from) {
        const int64_t n = tensors[from].n;
        if (n == 0) {
            // numbers run with the list: an empty tensor ends a launch that
            // goes by them, unless nothing came before it
            if (!number_each)
                continue;
            if (a.count)
                break;
            ++a.number;
            continue;
        }
        const int64_t blocks = (n + chunk - 1) / chunk;
        if (a.count && a.first[a.count] + blocks >= ((int64_t)1 << 23))
            break;
        a.t[a.count] = tensors[from];
        a.first[a.count + 1] = a.first[a.count] + (uint32_t)blocks;
        ++a.count;
    }
    return from;
}

int32_t check_list(const gqs_tensor *tensors, int64_t count)
{
    if (count < 0 || count >= ((int64_t)1 << 31))
        return fail(GQ_ERR_ARG, "%lld tensors", (long long)count);
    if (count > 0 && !tensors)
        return fail(GQ_ERR_NULL, "the list of tensors is NULL");
    for (int64_t i = 0; i < count; ++i)
        if (tensors[i].n < 0 || tensors[i].n >= kMaxElements)
            return fail(GQ_ERR_ARG, "tensor %lld has %lld elements", (long long)i,
                        (long long)tensors[i].n);
    return GQ_OK;
}

struct Range {
    uintptr_t begin, end;
};

// Whether what the step writes overlaps: two lanes would update one element.
// The ranges mostly come in order, as they were allocated, and sort at once.
int32_t check_overlap(const gqs_tensor *tensors, int64_t count, int64_t p_bytes, int bits)
{
    const int arrays = bits == 8 ? 5 : 3;
    Range few[5 * kTensors], *all = few;
    if (count > kTensors && !(all = new (std::nothrow) Range[arrays * count]))
        return fail(GQ_ERR_UNSUPPORTED, "%lld tensors", (long long)count);
    int64_t used = 0;
    const auto add = [&](const void *p, int64_t bytes) {
        all[used++] = {(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes};
    };
    for (int which = 0; which < arrays; ++which)
        for (int64_t i = 0; i < count; ++i) {
            const gqs_tensor &t = tensors[i];
            const void *const at[5] = {t.p, t.m, t.v, t.m_exps, t.v_exps};
            const int64_t state = bits == 8 ? fp8_pitch(t.n) : 4 * t.n;
            if (t.n > 0)
                add(at[which], which == 0 ? p_bytes * t.n : which < 3 ? state : blocks_of(t.n));
        }
    const auto before = [](const Range &a, const Range &b) { return a.begin < b.begin; };
    if (!std::is_sorted(all, all + used, before))
        std::sort(all, all + used, before);
    bool overlap = false;
    for (int64_t i = 1; i < used; ++i)
        overlap |= all[i].begin < all[i - 1].end;
    if (all != few)
        delete[] all;
    return overlap ? fail(GQ_ERR_ARG, "two of the tensors overlap") : GQ_OK;
}

template <typename P, typename G, int BITS>
int32_t launch_adamw(const gqs_tensor *tensors, int64_t count, const Coefs &c, const Coefs *device,
                     const Rates &r, const float *scale, hipStream_t st)
{
    // Long chunks share the search for the tensor, short ones fill the card.
    int64_t all = 0;
    for (int64_t i = 0; i < count; ++i)
        all += tensors[i].n;
    const int64_t chunk = all < kFew ? kStep : 4 * kStep;
    Tensors a;
    for (int64_t at = 0; at < count;) {
        at = gather(tensors, count, at, chunk, a, true);
        if (a.count) {
            k_adamw<P, G, BITS><<<a.first[a.count], kThreads, 0, st>>>(a, c, device, r, scale);
            GQT_TRY(check_launch("k_adamw"));
        }
    }
    return ok();
}

template <int BITS>
int32_t launch_types(const gqs_tensor *tensors, int64_t count, int32_t p, int32_t g,
                     const Coefs &c, const Coefs *device, const Rates &r, const float *scale,
                     hipStream_t st)
{
    if (p == GQ_IN_F32)
        return g == GQ_IN_F32
                   ? launch_adamw<float, float, BITS>(tensors, count, c, device, r, scale, st)
                   : launch_adamw<float, bf16, BITS>(tensors, count, c, device, r, scale, st);
    return g == GQ_IN_F32
               ? launch_adamw<bf16, float, BITS>(tensors, count, c, device, r, scale, st)
               : launch_adamw<bf16, bf16, BITS>(tensors, count, c, device, r, scale, st);
}

} // namespace
} // namespace gqt

using namespace gqt;

extern "C" {

const char *gqs_last_error(void) { return g_err; }

int32_t gqs_adamw(const gqs_tensor *tensors, int64_t count, int32_t p_dtype, int32_t g_dtype,
                  const gqs_adamw_args *args, void *workspace, int64_t workspace_bytes,
                  void *stream)
{
    if (!args)
        return fail(GQ_ERR_NULL, "args is NULL");
    if (!dtype_ok(p_dtype) || !dtype_ok(g_dtype))
        return fail(GQ_ERR_ARG, "p_dtype %d or g_dtype %d is neither GQ_IN_F32 nor GQ_IN_BF16",
                    p_dtype, g_dtype);
    if (args->bits != 32 && args->bits != 8)
        return fail(GQ_ERR_ARG, "bits = %d: 32 or 8", args->bits);
    if (!(args->beta1 >= 0.0 && args->beta1 < 1.0 && args->beta2 >= 0.0 && args->beta2 < 1.0))
        return fail(GQ_ERR_ARG, "beta1 = %g, beta2 = %g: from 0 to below 1", args->beta1,
                    args->beta2);
    if (!(args->lr >= 0.0 && args->lr < INFINITY && args->eps >= 0.0 && args->eps < INFINITY &&
          args->weight_decay >= 0.0 && args->weight_decay < INFINITY))
        return fail(GQ_ERR_ARG, "lr = %g, eps = %g, weight_decay = %g: finite and not negative",
                    args->lr, args->eps, args->weight_decay);
    if (args->step < 1 && !args->step_device)
        return fail(GQ_ERR_ARG, "step = %lld: steps count from 1", (long long)args->step);
    GQT_TRY(check_list(tensors, count));
    for (int64_t i = 0; i < count; ++i) {
        const gqs_tensor &t = tensors[i];
        if (t.n == 0)
            continue;
        if (!t.p || !t.g || !t.m || !t.v || (args->bits == 8 && (!t.m_exps || !t.v_exps)))
            return fail(GQ_ERR_NULL, "tensor %lld lacks an array", (long long)i);
        const int64_t state = args->bits == 8 ? 16 : 4;
        if (!aligned_to(t.p, elem_bytes(p_dtype)) || !aligned_to(t.g, elem_bytes(g_dtype)) ||
            !aligned_to(t.m, state) || !aligned_to(t.v, state))
            return fail(GQ_ERR_ALIGN, "tensor %lld: p and g are aligned to their elements, 32-bit "
                        "moments to 4 bytes, codes to 16", (long long)i);
    }
    GQT_TRY(check_overlap(tensors, count, elem_bytes(p_dtype), args->bits));
    if (!aligned_to(args->scale, 4) || !aligned_to(args->lr_device, 4) ||
        !aligned_to(args->step_device, 8))
        return fail(GQ_ERR_ALIGN, "scale, lr_device or step_device is not aligned");
    const bool device = args->lr_device || args->step_device;
    if (device && !workspace)
        return fail(GQ_ERR_NULL, "workspace is NULL");
    if (device && workspace_bytes < (int64_t)sizeof(Coefs))
        return fail(GQ_ERR_WORKSPACE, "workspace of %lld bytes, %lld are needed",
                    (long long)workspace_bytes, (long long)sizeof(Coefs));
    if (device && !aligned_to(workspace, 16))
        return fail(GQ_ERR_ALIGN, "workspace is not 16-byte aligned");
    if (count == 0)
        return ok();
    const hipStream_t st = (hipStream_t)stream;
    Coefs c{}, *ws = nullptr;
    if (device) {
        ws = (Coefs *)workspace;
        k_coefs<<<1, 1, 0, st>>>(args->lr, args->lr_device, args->beta1, args->beta2,
                                 args->weight_decay, args->step, args->step_device, ws);
        GQT_TRY(check_launch("k_coefs"));
    } else {
        c = coefs_of(args->lr, args->beta1, args->beta2, args->weight_decay, args->step);
    }
    const Rates r{(float)args->beta1,
                  (float)(1.0 - args->beta1),
                  (float)args->beta2,
                  (float)(1.0 - args->beta2),
                  (float)args->eps,
                  (uint32_t)args->seed,
                  (uint32_t)(args->seed >> 32),
                  args->random};
    return args->bits == 8
               ? launch_types<8>(tensors, count, p_dtype, g_dtype, c, ws, r, args->scale, st)
               : launch_types<32>(tensors, count, p_dtype, g_dtype, c, ws, r, args->scale, st);
}

int32_t gqs_moment8_restore(const void *codes, const void *exps, int64_t n, int32_t second,
                            int32_t dtype, void *out, void *stream)
{
    if (!dtype_ok(dtype))
        return fail(GQ_ERR_ARG, "dtype %d is neither GQ_IN_F32 nor GQ_IN_BF16", dtype);
    if (n < 0 || n >= kMaxElements)
        return fail(GQ_ERR_ARG, "n = %lld", (long long)n);
    if (n == 0)
        return ok();
    if (!codes || !exps || !out)
        return fail(GQ_ERR_NULL, "codes, exps or out is NULL");
    if (!aligned_to(codes, 16) || !aligned_to(out, elem_bytes(dtype)))
        return fail(GQ_ERR_ALIGN, "codes are aligned to 16 bytes, out to its elements");
    const uint32_t grid = (uint32_t)((n + 8 * kThreads - 1) / (8 * kThreads));
    const uint8_t *c = (const uint8_t *)codes, *e = (const uint8_t *)exps;
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == GQ_IN_F32) {
        if (second)
            k_moment8_restore<float, true><<<grid, kThreads, 0, st>>>(c, e, n, (float *)out);
        else
            k_moment8_restore<float, false><<<grid, kThreads, 0, st>>>(c, e, n, (float *)out);
    } else {
        if (second)
            k_moment8_restore<bf16, true><<<grid, kThreads, 0, st>>>(c, e, n, (bf16 *)out);
        else
            k_moment8_restore<bf16, false><<<grid, kThreads, 0, st>>>(c, e, n, (bf16 *)out);
    }
    return check_launch("k_moment8_restore");
}

int64_t gqs_grad_norm_workspace_bytes(const gqs_tensor *tensors, int64_t count)
{
    if (check_list(tensors, count) != GQ_OK)
        return -1;
    int64_t blocks = 0;
    for (int64_t i = 0; i < count; ++i)
        blocks += (tensors[i].n + kNormChunk - 1) / kNormChunk;
    return 8 * blocks;
}

int32_t gqs_grad_norm(const gqs_tensor *tensors, int64_t count, int32_t dtype, double max_norm,
                      float *norm, float *scale, void *workspace, int64_t workspace_bytes,
                      void *stream)
{
    if (!dtype_ok(dtype))
        return fail(GQ_ERR_ARG, "dtype %d is neither GQ_IN_F32 nor GQ_IN_BF16", dtype);
    GQT_TRY(check_list(tensors, count));
    for (int64_t i = 0; i < count; ++i) {
        if (tensors[i].n > 0 && !tensors[i].g)
            return fail(GQ_ERR_NULL, "tensor %lld has no gradient", (long long)i);
        if (!aligned_to(tensors[i].g, elem_bytes(dtype)))
            return fail(GQ_ERR_ALIGN, "gradient %lld is not aligned to its elements",
                        (long long)i);
    }
    if (!norm)
        return fail(GQ_ERR_NULL, "norm is NULL");
    if (!aligned_to(norm, 4) || !aligned_to(scale, 4))
        return fail(GQ_ERR_ALIGN, "norm or scale is not aligned");
    if (scale && !(max_norm >= 0.0 && max_norm < INFINITY))
        return fail(GQ_ERR_ARG, "max_norm = %g: finite and not negative", max_norm);
    const int64_t need = gqs_grad_norm_workspace_bytes(tensors, count);
    if (need > 0 && !workspace)
        return fail(GQ_ERR_NULL, "workspace is NULL");
    if (workspace_bytes < need)
        return fail(GQ_ERR_WORKSPACE, "workspace of %lld bytes, %lld are needed",
                    (long long)workspace_bytes, (long long)need);
    if (!aligned_to(workspace, 16))
        return fail(GQ_ERR_ALIGN, "workspace is not 16-byte aligned");
    double *const parts = (double *)workspace;
    const hipStream_t st = (hipStream_t)stream;
    Tensors a;
    int64_t done = 0;
    for (int64_t at = 0; at < count;) {
        at = gather(tensors, count, at, kNormChunk, a, false);
        if (!a.count)
            continue;
        const uint32_t grid = a.first[a.count];
        if (dtype == GQ_IN_F32)
            k_square_sums<float><<<grid, kThreads, 0, st>>>(a, parts + done);
        else
            k_square_sums<bf16><<<grid, kThreads, 0, st>>>(a, parts + done);
        GQT_TRY(check_launch("k_square_sums"));
        done += grid;
    }
    k_norm<<<1, kThreads, 0, st>>>(parts, done, max_norm, norm, scale);
    return check_launch("k_norm");
}

} // extern "C"
