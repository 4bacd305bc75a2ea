// la_common.cuh -- what the walks of linear attention share: which part of the work a
// block does, powers of the decay, states.
#pragma once

#include <cuda.h>
#include <math.h>

#include "encoder_internal.h"
#include "findings.cuh"

namespace semicrf {

// What the copy engine knows of each walk's operands.
struct LaMaps {
    struct {
        CUtensorMap q, k, v, o;
    } w[3];
};

namespace {

constexpr int kChunk = 128;     // positions of one step of the chunked walk

// lam^n from the float32 log_decay, exact to float32's rounding at any n (exponents in float64).
__device__ __forceinline__ double decay_pow(float log_decay, long long n)
{
    return n == 0 ? 1.0 : exp((double)log_decay * (double)n);
}

// One block of the walk: sequence b, head h, columns j0 .. j0 + dv of the values (slice z),
// rows d0 .. d0 + dk of the state, segment seg.
struct LaSpan {
    int b, h, z, seg, L, p0, pe, p1;
    int d0, dk, j0, dv;   // dk or dv <= 0: nothing here
    bool last;
};

__device__ __forceinline__ LaSpan la_span(const LaArgs &a, const LaWalk &w, int idx)
{
    LaSpan s;
    s.seg = idx % a.nseg;
    const int bhz = idx / a.nseg, bh = bhz / a.slices;
    s.z = bhz % a.slices;
    s.h = bh % a.H;
    s.b = bh / a.H;
    s.d0 = a.kblock * a.width;
    s.dk = min(a.width, w.dk - s.d0);
    s.j0 = s.z * a.width;
    s.dv = min(a.width, w.dv - s.j0);
    int L = a.T;
    if (a.lengths) {
        L = a.lengths[s.b];
        if (L < 0 || L > a.T) {
            if (threadIdx.x == 0) report(a.status, SEMICRF_ERR_INVALID_LENGTH);
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
__device__ __forceinline__ void zero_rows(const LaWalk &w, const LaSpan &s)
{
    T *o = static_cast<T *>(w.o) + s.b * w.os[0] + s.h * w.os[2] + s.j0;
    const int from = max(s.p0, s.L);
    for (long long i = threadIdx.x; i < (long long)(s.p1 - from) * s.dv; i += blockDim.x)
        o[(from + i / s.dv) * w.os[1] + i % s.dv] = from_f<T>(0.f);
}

// Where this block's rows and columns of a given or returned state begin.
__device__ __forceinline__ long long state_at(const LaWalk &w, const LaArgs &a, const LaSpan &s)
{
    return ((long long)s.b * a.H + s.h) * w.dk * w.dv + (long long)s.d0 * w.s_rs + (long long)s.j0 * w.s_cs;
}

// A sequence without positions hands its state on.
__device__ __forceinline__ void copy_state(const LaWalk &w, const LaArgs &a, const LaSpan &s)
{
    if (!w.s_out) return;
    const long long base = state_at(w, a, s);
    for (int i = threadIdx.x; i < s.dk * s.dv; i += blockDim.x) {
        const long long at = base + (long long)(i / s.dv) * w.s_rs + (long long)(i % s.dv) * w.s_cs;
        w.s_out[at] = w.s_in ? w.s_in[at] : 0.f;
    }
}

// This segment's state in the workspace: width x width.
__device__ __forceinline__ float *segment_at(const LaWalk &w, const LaArgs &a, const LaSpan &s)
{
    const long long bhz = ((long long)s.b * a.H + s.h) * a.slices + s.z;
    return w.seg + (bhz * a.nseg + s.seg) * a.width * a.width;
}

// Where the walk of this segment takes its state from, element (i, j) at i * rs + j * cs.
struct StateAt {
    const float *p;
    int rs, cs;
};

__device__ __forceinline__ StateAt state_from(const LaWalk &w, const LaArgs &a, const LaSpan &s)
{
    if (w.seg) return {segment_at(w, a, s), a.width, 1};
    return {w.s_in ? w.s_in + state_at(w, a, s) : nullptr, w.s_rs, w.s_cs};
}

// Products of operands in NA and NB terms: go(x, y, accumulate) for the pairs of terms
// with x + y < N, the smallest first.  What is left out: 2^-23 of each product of three
// terms, 2^-16 (both second terms) of two; for float16 that fourth product costs 8 % of a
// call and takes the outputs' distance from 64 bits from 4.2e-5 to 3.5e-5, most of which is
// their own rounding.
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

}  // namespace
}  // namespace semicrf
