// la_common.cuh -- what the walks of linear attention share: which part of the work a
// block does, powers of the decay, states.
#pragma once

#include <math.h>

#include "device_util.cuh"
#include "encoder_internal.h"

namespace semicrf {
namespace {

constexpr int kChunk = 128;     // positions of one step of the chunked walk

// lam^n from the float32 log_decay, exact to float32's rounding at any n (exponents in float64).
__device__ __forceinline__ double decay_pow(float log_decay, long long n)
{
    return n == 0 ? 1.0 : exp((double)log_decay * (double)n);
}

// One block of the walk: (sequence b, head h, segment seg).
struct LaSpan {
    int b, h, seg, L, p0, pe, p1;
    bool last;
};

__device__ __forceinline__ LaSpan la_span(const LaArgs &a, int idx)
{
    LaSpan s;
    s.seg = idx % a.nseg;
    const int bh = idx / a.nseg;
    s.h = bh % a.H;
    s.b = bh / a.H;
    int L = a.T;
    if (a.lengths) {
        L = a.lengths[s.b];
        if (L < 0 || L > a.T) {
            if (threadIdx.x == 0) set_status(a.status, SEMICRF_ERR_INVALID_LENGTH);
            L = max(0, min(L, a.T));
        }
    }
    s.L = L;
    const long long q0 = (long long)s.seg * a.seg_len;
    s.p0 = (int)min(q0, (long long)a.T);
    s.p1 = (int)min(q0 + a.seg_len, (long long)a.T);
    s.pe = max(s.p0, min(s.p1, L));
    s.last = L == 0 ? s.seg == 0 : (L - 1) / a.seg_len == s.seg;
    return s;
}

// Positions behind the sequence's end: zeros.
template <typename T>
__device__ __forceinline__ void zero_rows(const LaWalk &w, const LaSpan &s, int d_begin, int d_end)
{
    T *o = static_cast<T *>(w.o) + s.b * w.os[0] + s.h * w.os[2];
    const int n = d_end - d_begin;
    const int from = max(s.p0, s.L);
    for (long long i = threadIdx.x; i < (long long)(s.p1 - from) * n; i += blockDim.x)
        o[(from + i / n) * w.os[1] + d_begin + i % n] = from_f<T>(0.f);
}

// A sequence without positions hands its state on.
__device__ __forceinline__ void copy_state(const LaWalk &w, const LaArgs &a, const LaSpan &s, int j0, int j1)
{
    if (!w.s_out) return;
    const long long base = ((long long)s.b * a.H + s.h) * w.dk * w.dv;
    const int n = j1 - j0;
    for (int i = threadIdx.x; i < w.dk * n; i += blockDim.x) {
        const long long at = base + (long long)(i / n) * w.s_rs + (long long)(j0 + i % n) * w.s_cs;
        w.s_out[at] = w.s_in ? w.s_in[at] : 0.f;
    }
}

// Where the walk of this segment takes its state from, element (i, j) at i * rs + j * cs.
struct StateAt {
    const float *p;
    int rs, cs;
};

__device__ __forceinline__ StateAt state_from(const LaWalk &w, const LaArgs &a, const LaSpan &s)
{
    const long long bh = (long long)s.b * a.H + s.h, sz = (long long)w.dk * w.dv;
    if (w.seg) return {w.seg + (bh * a.nseg + s.seg) * sz, w.dv, 1};
    return {w.s_in ? w.s_in + bh * sz : nullptr, w.s_rs, w.s_cs};
}

// Products of operands in NA and NB terms: go(x, y, accumulate) for the pairs of terms
// with x + y < N, the smallest first.
template <int NA, int NB, int N, typename F>
__device__ __forceinline__ void mma_terms(F &&go)
{
    bool acc = false;
#pragma unroll
    for (int sum = N - 1; sum >= 0; --sum)
#pragma unroll
        for (int x = 0; x <= sum; ++x)
            if (x < NA && sum - x < NB) {
                go(x, sum - x, acc);
                acc = true;
            }
}

template <typename F>
cudaError_t timed_launch(cudaStream_t st, int *n, F &&go)
{
    prof_before(st);
    go();
    prof_after(st);
    ++*n;
    return cudaGetLastError();
}

}  // namespace
}  // namespace semicrf
