// adamw.cu -- one AdamW step over many tensors in one launch:
//   m = b1 m + (1-b1) g,  v = b2 v + (1-b2) g^2,
//   p = p (1 - lr wd) - lr (m / (1-b1^t)) / (sqrt(v / (1-b2^t)) + eps)
// with the states m, v in float32 or in 8 bits.
//
// 8 bits: 256 consecutive values share a float32 scale, their largest magnitude / 1.875.
// A code is a small float with 3 mantissa bits, nearest even; m: sign and 4 exponent
// bits (bias 15), v: 5 exponent bits (bias 31), so that v keeps the square of m's range;
// a v that is not zero never gets code 0, which would make the next step's quotient huge.
// The moments are formed in float64: a value next to the border of two codes then falls
// on the side the formula says.
//
// Measured on 26 million parameters.  float32 states: 90 us, which is 591 MB at the
// measured copy rate, so what is left is the memory's.  8 bits: 111 us for 420 MB (64 us):
// bound by issue (69 % of the cycles) and by the loads' latency, about 95 instructions a
// value, of which 14 are float64.  Square root and quotient to two units of the last place
// instead of correctly rounded and powers of beta on the host saved a fifth; codes read and
// written as the high words of doubles 2^1008 (2^992) times too small, a multiplication for
// a change of the bias and a case for small codes, an eighth.
#include <float.h>
#include <math.h>

#include <algorithm>
#include <memory>
#include <new>

#include "device_util.cuh"
#include "encoder_internal.h"

namespace semicrf {
namespace {

constexpr int kThreads = 256, kPer = 8;            // values of one thread at a time
constexpr int kBlock = 256;                        // values that share a scale
constexpr int kSpan = 2 * kThreads * kPer;         // values of one thread block
constexpr int kFew = 48, kMany = 440;              // tensors of one launch (3.4 and 32 KB of arguments)

struct Entry {
    semicrf_adamw_tensor t;
    long long first;   // first thread block
};

struct Factors {
    float b1, b2, n1, n2, decay, lr, root2, eps;
};

template <int N>
struct AdamArgs {
    Entry e[N];
    int count;
    semicrf_adamw_config c;
    Factors f;   // of c, where step and lr are host values
};

__host__ __device__ inline Factors factors_of(const semicrf_adamw_config &c, double step, double lr)
{
    Factors f;
    f.b1 = (float)c.beta1;
    f.b2 = (float)c.beta2;
    f.n1 = (float)(1.0 - c.beta1);
    f.n2 = (float)(1.0 - c.beta2);
    f.decay = (float)(1.0 - lr * c.weight_decay);
    f.lr = (float)(lr / (1.0 - pow(c.beta1, step)));
    f.root2 = (float)(1.0 / sqrt(1.0 - pow(c.beta2, step)));
    f.eps = (float)c.eps;
    return f;
}

template <typename R, typename T>
__device__ __forceinline__ R cvt(T v)
{
    if constexpr (sizeof(T) == 2)
        return (R)to_f<T>(v);
    else
        return (R)v;
}

// 8 values from index i on (cnt of them exist); vec: whole and 16-byte aligned; float64 ones
// to float times `by`.
template <typename R, typename T>
__device__ __forceinline__ void load8(const void *p, long long i, int cnt, bool vec, R (&o)[kPer], double by = 1.0)
{
    auto cast = [&](T v) {
        if constexpr (sizeof(T) == 8 && sizeof(R) == 4)
            return (R)(v * by);
        else
            return cvt<R, T>(v);
    };
    const T *s = static_cast<const T *>(p) + i;
    constexpr int n = 16 / sizeof(T);
    if (vec) {
        Pack<T, n> h[kPer / n];
#pragma unroll
        for (int j = 0; j < kPer / n; ++j) h[j] = reinterpret_cast<const Pack<T, n> *>(s)[j];
        if constexpr (sizeof(T) == 2) {
            float f[kPer];
            unpack(h[0], f);
#pragma unroll
            for (int j = 0; j < kPer; ++j) o[j] = (R)f[j];
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j) o[j] = cast(h[j / n].v[j % n]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) o[j] = j < cnt ? cast(s[j]) : (R)0;
    }
}

template <typename R>
__device__ __forceinline__ void load_as(const void *p, int type, long long i, int cnt, bool vec, R (&o)[kPer])
{
    if (type == SEMICRF_F32)
        load8<R, float>(p, i, cnt, vec, o);
    else if (type == SEMICRF_BF16)
        load8<R, __nv_bfloat16>(p, i, cnt, vec, o);
    else if (type == SEMICRF_F16)
        load8<R, __half>(p, i, cnt, vec, o);
    else
        load8<R, double>(p, i, cnt, vec, o);
}

template <typename T>
__device__ __forceinline__ void store8(void *p, long long i, int cnt, bool vec, const float (&o)[kPer])
{
    T *s = static_cast<T *>(p) + i;
    constexpr int n = 16 / sizeof(T);
    if (vec) {
#pragma unroll
        for (int j = 0; j < kPer / n; ++j) {
            float f[n];
#pragma unroll
            for (int e = 0; e < n; ++e) f[e] = o[j * n + e];
            reinterpret_cast<Pack<T, n> *>(s)[j] = pack<T, n>(f);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j < cnt) s[j] = from_f<T>(o[j]);
    }
}

__device__ __forceinline__ bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Code of y >= 0: y 2^(BIAS - 1023), whose bits are the code's with 49 more behind it, small
// codes included (those are a double's own small values, which the product rounds 49 bits
// below a code's last); nearest even, the low word only decides ties.
template <int BIAS>
__device__ __forceinline__ uint32_t code_of(double y)
{
    const double x = y * pow2(BIAS - 1023);
    const uint32_t h = (uint32_t)__double2hiint(x) | (__double2loint(x) != 0);
    return (h + 0xffffu + ((h >> 17) & 1u)) >> 17;
}

// The value of a code without its block's scale, the other way round: the code's bits (of a
// sign at bit 31 and exponent and mantissa from bit 17 on) are those of a double's high word.
template <int BIAS>
__device__ __forceinline__ double value_of(uint32_t high)
{
    return __hiloint2double((int)high, 0) * pow2(1023 - BIAS);
}

template <int BIAS>
__device__ __forceinline__ float float_value_of(uint32_t c)
{
    return __uint_as_float(c << 20) * __uint_as_float((127u + 127u - BIAS) << 23);   // (a float's own small values)
}

// NaN where the largest is not finite: an infinite scale would give codes of 0 that read as
// NaN and others that read as infinity, which a second moment's root turns into no update.
__device__ __forceinline__ float block_scale(float most)
{
    const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
    if (bits >= 0x7f800000u) return __uint_as_float(0x7fffffffu);
    return (float)((double)__uint_as_float(bits) / 1.875);
}

__device__ __forceinline__ float next_param(float p, float m, float v, const Factors &f)
{
    // square root and quotient to two units of the last place: far inside the parameter's rounding
    float root;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(root) : "f"(v));
    return fmaf(p, f.decay, __fdividef(-f.lr * m, fmaf(root, f.root2, f.eps)));
}

__device__ __forceinline__ void store_param(const semicrf_adamw_tensor &t, long long i, int cnt, bool vec,
                                            const float (&p)[kPer])
{
    if (t.param_dtype == SEMICRF_F32)
        store8<float>(t.param, i, cnt, vec, p);
    else if (t.param_dtype == SEMICRF_BF16)
        store8<__nv_bfloat16>(t.param, i, cnt, vec, p);
    else
        store8<__half>(t.param, i, cnt, vec, p);
}

// One call of a warp: 256 consecutive values, which is one block of scales.
__device__ __forceinline__ void step8(const semicrf_adamw_tensor &t, const semicrf_adamw_config &c, const Factors &f,
                                      long long i, int cnt, bool vec)
{
    float p[kPer];
    load_as<float>(t.param, t.param_dtype, i, cnt, vec, p);
    double g[kPer];
    load_as<double>(t.grad, t.grad_dtype, i, cnt, vec, g);
    const int lane = threadIdx.x & 31;
    const long long blk = (i - lane * kPer) / kBlock;
    const bool any = cnt > 0;
    uint8_t *mc = static_cast<uint8_t *>(t.exp_avg) + i, *vc = static_cast<uint8_t *>(t.exp_avg_sq) + i;
    uint32_t cm[2] = {0, 0}, cv[2] = {0, 0};   // the codes, four to a word
    const bool wide = vec && reinterpret_cast<uintptr_t>(mc) % 8 == 0 && reinterpret_cast<uintptr_t>(vc) % 8 == 0;
    if (wide) {
        const uint2 wm = *reinterpret_cast<const uint2 *>(mc), wv = *reinterpret_cast<const uint2 *>(vc);
        cm[0] = wm.x, cm[1] = wm.y;
        cv[0] = wv.x, cv[1] = wv.y;
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            cm[j / 4] |= (uint32_t)(j < cnt ? mc[j] : 0) << (j % 4 * 8);
            cv[j / 4] |= (uint32_t)(j < cnt ? vc[j] : 0) << (j % 4 * 8);
        }
    }
    // a warp enters with its first lane inside the tensor, so the block's scale exists
    const double sm = t.exp_avg_scale[blk], sv = t.exp_avg_sq_scale[blk];
    const double n1 = 1.0 - c.beta1, n2 = 1.0 - c.beta2;
    double m[kPer], v[kPer];
    float mm = 0.f, mv = 0.f;
    const bool scaled = c.grad_scale != 1.0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const double gj = scaled ? g[j] * c.grad_scale : g[j];
        const double old = value_of<15>((uint32_t)((int32_t)(cm[j / 4] << (24 - j % 4 * 8)) >> 7) & 0x80fe0000u);
        // (rounded operation by operation: what the formula gives on any machine, ties included)
        m[j] = __dadd_rn(__dmul_rn(c.beta1, __dmul_rn(old, sm)), __dmul_rn(n1, gj));
        v[j] = __dadd_rn(__dmul_rn(c.beta2, __dmul_rn(value_of<31>((cv[j / 4] << (24 - j % 4 * 8)) >> 7 & 0x1fe0000u), sv)), __dmul_rn(__dmul_rn(n2, gj), gj));
        const float fm = (float)m[j], fv = (float)v[j];
        p[j] = next_param(p[j], fm, fv, f);
        mm = __uint_as_float(max(__float_as_uint(mm), __float_as_uint(fabsf(fm))));   // NaN above infinity
        mv = __uint_as_float(max(__float_as_uint(mv), __float_as_uint(fv)));
    }
    store_param(t, i, cnt, vec, p);   // (now: its registers are wanted)
    const float scm = block_scale(mm), scv = block_scale(mv);
    const double im = scm > 0.f ? 1.0 / (double)scm : scm == 0.f ? 0.0 : (double)scm;
    const double iv = scv > 0.f ? 1.0 / (double)scv : scv == 0.f ? 0.0 : (double)scv;
    cm[0] = cm[1] = cv[0] = cv[1] = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const uint32_t a = min(code_of<15>(fabs(m[j]) * im), 127u);
        uint32_t b = min(code_of<31>(v[j] * iv), 255u);
        if (v[j] > 0.0 && scv > 0.f) b = max(b, 1u);
        cm[j / 4] |= (a | (m[j] < 0.0 ? 128u : 0u)) << (j % 4 * 8);
        cv[j / 4] |= b << (j % 4 * 8);
    }
    if (wide) {
        *reinterpret_cast<uint2 *>(mc) = make_uint2(cm[0], cm[1]);
        *reinterpret_cast<uint2 *>(vc) = make_uint2(cv[0], cv[1]);
    } else if (any) {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j < cnt) {
                mc[j] = (uint8_t)(cm[j / 4] >> (j % 4 * 8));
                vc[j] = (uint8_t)(cv[j / 4] >> (j % 4 * 8));
            }
    }
    __syncwarp();
    if (lane == 0) {
        t.exp_avg_scale[blk] = scm;
        t.exp_avg_sq_scale[blk] = scv;
    }
}

__device__ __forceinline__ void step32(const semicrf_adamw_tensor &t, const semicrf_adamw_config &c, const Factors &f,
                                       long long i, int cnt, bool vec)
{
    float p[kPer], g[kPer], m[kPer], v[kPer];
    load_as<float>(t.param, t.param_dtype, i, cnt, vec, p);
    if (t.grad_dtype == SEMICRF_F64)   // scaled before it is rounded: the product may fit where the gradient does not
        load8<float, double>(t.grad, i, cnt, vec, g, c.grad_scale);
    else
        load_as<float>(t.grad, t.grad_dtype, i, cnt, vec, g);
    load8<float, float>(t.exp_avg, i, cnt, vec, m);
    load8<float, float>(t.exp_avg_sq, i, cnt, vec, v);
    const float gs = t.grad_dtype == SEMICRF_F64 ? 1.f : (float)c.grad_scale;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const float gj = g[j] * gs;
        m[j] = fmaf(f.b1, m[j], f.n1 * gj);
        v[j] = fmaf(f.b2, v[j], f.n2 * gj * gj);
        p[j] = next_param(p[j], m[j], v[j], f);
    }
    store8<float>(t.exp_avg, i, cnt, vec, m);
    store8<float>(t.exp_avg_sq, i, cnt, vec, v);
    store_param(t, i, cnt, vec, p);
}

template <int N>
__device__ __forceinline__ int entry_of(const AdamArgs<N> &a, long long block)
{
    int lo = 0, hi = a.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (a.e[mid].first <= block)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Blocks of a multiprocessor: 8 bits with 4 (64 registers, 20 bytes of them in memory) a tenth
// faster than with 3 (74 registers); 32 bits with 5 (47 registers) 90 us, with 3 (74) 107.
template <int N, bool EIGHT>
__global__ __launch_bounds__(kThreads, EIGHT ? 4 : 5) void adamw_kernel(const __grid_constant__ AdamArgs<N> a)
{
    const Entry &en = a.e[entry_of<N>(a, blockIdx.x)];
    const semicrf_adamw_tensor &t = en.t;
    const semicrf_adamw_config &c = a.c;
    Factors f = a.f;
    if (c.step_ptr || c.lr_ptr) {   // two float64 powers: not each block's work where the host knows them
        __shared__ Factors sf;
        if (threadIdx.x == 0)
            sf = factors_of(c, (double)(c.step_ptr ? *c.step_ptr : c.step), c.lr_ptr ? (double)*c.lr_ptr : c.lr);
        __syncthreads();
        f = sf;
    }
    const bool all = aligned16(t.param) && aligned16(t.grad) &&
                     (EIGHT || (aligned16(t.exp_avg) && aligned16(t.exp_avg_sq)));
    const long long from = (blockIdx.x - en.first) * (long long)kSpan;
#pragma unroll 1
    for (int k = 0; k < kSpan / (kThreads * kPer); ++k) {
        const long long i = from + (long long)k * kThreads * kPer + threadIdx.x * kPer;
        // whole warps leave together: 256 values, one block of scales
        if (i - (threadIdx.x & 31) * kPer >= t.n) break;
        const int cnt = (int)max(0LL, min((long long)kPer, t.n - i));
        const bool vec = all && cnt == kPer;
        if (EIGHT)
            step8(t, c, f, i, cnt, vec);
        else
            step32(t, c, f, i, cnt, vec);
    }
}

// Codes to the values they stand for: t.param receives exp_avg (or exp_avg_sq) in float32.
template <int N, bool SECOND>
__global__ __launch_bounds__(kThreads) void adamw_values_kernel(const __grid_constant__ AdamArgs<N> a)
{
    const Entry &en = a.e[entry_of<N>(a, blockIdx.x)];
    const semicrf_adamw_tensor &t = en.t;
    const uint8_t *codes = static_cast<const uint8_t *>(SECOND ? t.exp_avg_sq : t.exp_avg);
    const float *scale = SECOND ? t.exp_avg_sq_scale : t.exp_avg_scale;
    const long long from = (blockIdx.x - en.first) * (long long)kSpan;
#pragma unroll
    for (int k = 0; k < kSpan / (kThreads * kPer); ++k) {
        const long long i = from + (long long)k * kThreads * kPer + threadIdx.x * kPer;
        if (i >= t.n) break;
        const int cnt = (int)min((long long)kPer, t.n - i);
        const float s = scale[i / kBlock];
        const bool vec = cnt == kPer && aligned16(t.param);
        Pack<uint8_t, 8> c;
        if (vec && reinterpret_cast<uintptr_t>(codes + i) % 8 == 0) {
            c = *reinterpret_cast<const Pack<uint8_t, 8> *>(codes + i);
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j) c.v[j] = j < cnt ? codes[i + j] : 0;
        }
        float o[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const float mag = (SECOND ? float_value_of<31>(c.v[j]) : float_value_of<15>(c.v[j] & 127u)) * s;
            o[j] = SECOND ? mag : __uint_as_float(__float_as_uint(mag) | (uint32_t)(c.v[j] & 128u) << 24);
        }
        store8<float>(t.param, i, cnt, vec, o);
    }
}

template <int N, typename F>
cudaError_t launch_some(const semicrf_adamw_tensor *t, int count, const semicrf_adamw_config &c, cudaStream_t st, int *n,
                        F &&kernel)
{
    static thread_local AdamArgs<N> a;   // 32 KB at most: kept off the stack
    a.c = c;
    a.f = factors_of(c, (double)c.step, c.lr);
    a.count = 0;
    long long blocks = 0;
    for (int i = 0; i < count; ++i) {
        if (t[i].n == 0) continue;
        a.e[a.count].t = t[i];
        a.e[a.count++].first = blocks;
        blocks += (t[i].n + kSpan - 1) / kSpan;
    }
    if (!blocks) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    return timed_launch(st, n, [&] { kernel(a, (unsigned)blocks); });
}

template <typename F>
cudaError_t launch_all(const semicrf_adamw_tensor *t, int count, const semicrf_adamw_config &c, cudaStream_t st, int *n,
                       F &&kernel)
{
    *n = 0;
    for (int i = 0; i < count;) {
        const int left = count - i;
        cudaError_t e;
        if (left <= kFew) {
            e = launch_some<kFew>(t + i, left, c, st, n, kernel);
            i = count;
        } else {
            const int some = left < kMany ? left : kMany;
            e = launch_some<kMany>(t + i, some, c, st, n, kernel);
            i += some;
        }
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Whether what a step writes overlaps anything else that it touches (the thread blocks of one
// tensor would race with another's); gradients are only read and may be shared.
struct Range {
    uintptr_t from, to;
    bool written;
};

semicrf_status apart(const semicrf_adamw_tensor *t, int count)
{
    const std::unique_ptr<Range[]> all(new (std::nothrow) Range[(size_t)count * 6]);
    if (!all) return SEMICRF_ERR_INVALID_ARG;
    size_t n = 0;
    auto add = [&](const void *p, long long bytes, bool written) {
        const uintptr_t from = reinterpret_cast<uintptr_t>(p);
        if (p) all[n++] = {from, from + bytes, written};
    };
    for (int i = 0; i < count; ++i) {
        if (t[i].n == 0) continue;
        const bool eight = t[i].exp_avg_scale;
        const long long state = t[i].n * (eight ? 1 : 4), scales = (t[i].n + kBlock - 1) / kBlock * 4;
        add(t[i].param, t[i].n * (t[i].param_dtype == SEMICRF_F32 ? 4 : 2), true);
        add(t[i].grad, t[i].n * (t[i].grad_dtype == SEMICRF_F64 ? 8 : t[i].grad_dtype == SEMICRF_F32 ? 4 : 2), false);
        add(t[i].exp_avg, state, true);
        add(t[i].exp_avg_sq, state, true);
        add(t[i].exp_avg_scale, scales, true);
        add(t[i].exp_avg_sq_scale, scales, true);
    }
    std::sort(all.get(), all.get() + n, [](const Range &a, const Range &b) { return a.from < b.from; });
    uintptr_t end = 0, written = 0;   // of all ranges so far, of those that are written
    for (size_t i = 0; i < n; ++i) {
        if (all[i].from < (all[i].written ? end : written)) return SEMICRF_ERR_INVALID_ARG;
        end = std::max(end, all[i].to);
        if (all[i].written) written = std::max(written, all[i].to);
    }
    return SEMICRF_OK;
}

bool tensors_ok(const semicrf_adamw_tensor *t, int count)
{
    if (count < 0 || (count > 0 && !t)) return false;
    for (int i = 0; i < count; ++i)
        if (t[i].n < 0) return false;
    return true;
}

}  // namespace
}  // namespace semicrf

using namespace semicrf;

extern "C" semicrf_status semicrf_adamw(const semicrf_adamw_tensor *tensors, int32_t count,
                                        const semicrf_adamw_config *config, void *stream)
{
    prof_reset();
    if (!config || !tensors_ok(tensors, count)) return SEMICRF_ERR_INVALID_ARG;
    const semicrf_adamw_config &c = *config;
    // (negated comparisons: NaN is refused too)
    if (!(c.beta1 >= 0.0 && c.beta1 < 1.0) || !(c.beta2 >= 0.0 && c.beta2 < 1.0) || !(c.eps >= 0.0) ||
        !(c.weight_decay >= 0.0) || !isfinite(c.grad_scale) || (!c.lr_ptr && !(c.lr >= 0.0)) ||
        (!c.step_ptr && c.step < 1))
        return SEMICRF_ERR_INVALID_ARG;
    // eps enters the quotient as float32, grad_scale a gradient that is not float64
    if (c.eps > 0.0 && c.eps < FLT_MIN) return SEMICRF_ERR_INVALID_ARG;
    const double scale = fabs(c.grad_scale);
    const bool scale_fits = scale == 0.0 || (scale >= FLT_MIN && scale <= FLT_MAX);
    int eight = 0, filled = 0;
    for (int i = 0; i < count; ++i) {
        const semicrf_adamw_tensor &t = tensors[i];
        if (t.param_dtype < SEMICRF_F32 || t.param_dtype > SEMICRF_F16 || t.grad_dtype < SEMICRF_F32 ||
            t.grad_dtype > SEMICRF_F64)
            return SEMICRF_ERR_INVALID_ARG;
        if (t.n == 0) continue;
        if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq || !t.exp_avg_scale != !t.exp_avg_sq_scale)
            return SEMICRF_ERR_INVALID_ARG;
        ++filled;
        eight += t.exp_avg_scale != nullptr;
        if (!scale_fits && !t.exp_avg_scale && t.grad_dtype != SEMICRF_F64) return SEMICRF_ERR_INVALID_ARG;
    }
    if (eight && eight != filled) return SEMICRF_ERR_INVALID_ARG;   // one kind of state a call
    if (const semicrf_status s = apart(tensors, count)) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int n = 0;
    cudaError_t e = launch_all(tensors, count, c, st, &n, [&](const auto &a, unsigned blocks) {
        constexpr int N = sizeof(a.e) / sizeof(Entry);
        if (eight)
            adamw_kernel<N, true><<<blocks, kThreads, 0, st>>>(a);
        else
            adamw_kernel<N, false><<<blocks, kThreads, 0, st>>>(a);
    });
    return ended(e, n);
}

extern "C" semicrf_status semicrf_adamw_state_values(const semicrf_adamw_tensor *tensors, int32_t count, int32_t second,
                                                     void *stream)
{
    prof_reset();
    if (!tensors_ok(tensors, count) || (second != 0 && second != 1)) return SEMICRF_ERR_INVALID_ARG;
    for (int i = 0; i < count; ++i) {
        const semicrf_adamw_tensor &t = tensors[i];
        if (t.n && (!t.param || !(second ? t.exp_avg_sq : t.exp_avg) || !(second ? t.exp_avg_sq_scale : t.exp_avg_scale)))
            return SEMICRF_ERR_INVALID_ARG;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int n = 0;
    const semicrf_adamw_config none = {};
    cudaError_t e = launch_all(tensors, count, none, st, &n, [&](const auto &a, unsigned blocks) {
        constexpr int N = sizeof(a.e) / sizeof(Entry);
        if (second)
            adamw_values_kernel<N, true><<<blocks, kThreads, 0, st>>>(a);
        else
            adamw_values_kernel<N, false><<<blocks, kThreads, 0, st>>>(a);
    });
    return ended(e, n);
}
