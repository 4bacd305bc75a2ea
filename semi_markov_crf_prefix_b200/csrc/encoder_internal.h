// encoder_internal.h -- what the translation units of the operators around the loss
// (linear attention, group norm, AdamW) share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "semicrf.h"

namespace semicrf {

void prof_reset();
void prof_before(cudaStream_t st);
void prof_after(cudaStream_t st);
void record_launches(int n);
int device_sm_count();

// One launch, counted in *n and between the profile's events.
template <typename F>
cudaError_t timed_launch(cudaStream_t st, int *n, F &&go)
{
    prof_before(st);
    go();
    prof_after(st);
    ++*n;
    return cudaGetLastError();
}

// How an entry point ends after its launches.
inline semicrf_status ended(cudaError_t e, int launches)
{
    if (e != cudaSuccess) return SEMICRF_ERR_CUDA;
    record_launches(launches);
    return SEMICRF_OK;
}

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f<double>(double v) { return (float)v; }

template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// N values as one load or store of N * sizeof(T) bytes (16 at most), which the address must be aligned to.
template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
    T v[N];
};

// The values of a pack as floats, and back: two 16-bit values of a word at a time.
template <typename T, int N>
__device__ __forceinline__ void unpack(const Pack<T, N> &p, float (&o)[N])
{
    if constexpr (sizeof(T) == 2 && N % 2 == 0) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&p);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            if constexpr (__is_same(T, __half)) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                o[2 * i] = f.x;
                o[2 * i + 1] = f.y;
            } else {
                o[2 * i] = __uint_as_float(w[i] << 16);
                o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = to_f<T>(p.v[i]);
    }
}

template <typename T, int N>
__device__ __forceinline__ Pack<T, N> pack(const float (&f)[N])
{
    Pack<T, N> p;
    if constexpr (sizeof(T) == 2 && N % 2 == 0) {
        uint32_t *w = reinterpret_cast<uint32_t *>(&p);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            if constexpr (__is_same(T, __half)) {
                const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) p.v[i] = from_f<T>(f[i]);
    }
    return p;
}

// Findings of each source's kernels on the current device, read and cleared (findings.cuh).
cudaError_t la_found(int32_t *to);
cudaError_t la_tma_found(int32_t *to);
cudaError_t norm_found(int32_t *to);
cudaError_t la_clear_found(cudaStream_t st);
cudaError_t la_tma_clear_found(cudaStream_t st);
cudaError_t norm_clear_found(cudaStream_t st);

// ---- linear attention ----

// One walk over all sequences and heads: S_p = lam S_{p-1} + c k_p v_p^T, o_p = b q_p S_p.  The forward is
// one walk; the backward is three (exchanged operands, two of them against the direction of time).
struct LaWalk {
    const void *q, *k, *v;
    void *o;
    long long qs[3], ks[3], vs[3], os[3];   // strides of sequence, position, head (elements); the last axis is dense
    int dk, dv;
    const float *s_in;                      // [B,H] states, element (i,j) at i * s_rs + j * s_cs, or null
    float *s_out;                           // same addressing, or null
    int s_rs, s_cs;
    float *seg;                             // [B,H,slices,nseg] states at the segments' starts (width x width), or null
    float *part;                            // [B,T,H,dv] float32 sums over the first blocks of the contraction, or null
    float b, c;
    int reverse;                            // walk from the last valid position to the first
    int lead;                               // power of lam the given state has at the first position
    int out_decay;                          // s_out takes one more factor lam
    int q_vec, k_vec, v_vec, o_vec;         // whole 8-value pieces can be moved in one (two) 16-byte accesses
};

struct LaArgs {
    LaWalk w[3];
    int nwalk;
    int B, T, H;
    int nseg, seg_len;                      // segments of seg_len positions (whole sequences when nseg == 1)
    int width, slices, kblock;              // tiles of `width`: a launch takes block kblock of dk, and every slice of dv
    const float *log_decay;
    const int32_t *lengths;                 // or null
    int32_t *status;
};

struct LaStepArgs {
    const void *q, *k, *v;
    void *o;
    long long qs[2], ks[2], vs[2], os[2];   // strides of sequence and head
    float *state;
    const float *log_decay;
    int B, H, dk, dv;
    float scale;
};

struct LaMaps;

// Workspace of these operands, and the most that any operands of these sizes need.
size_t la_need(const LaArgs &a, int dtype);
size_t la_workspace(int B, int T, int H, int dk, int dv, int dtype, int nwalk);
// *small: the workspace does not hold the plan that the operands turned out to need.
cudaError_t launch_la(LaArgs a, int dtype, unsigned char *ws, size_t ws_bytes, cudaStream_t st, int *launches, bool *small);
bool la_tma_ok(const LaArgs &a, int dtype);
bool la_tma_maps(const LaArgs &a, LaMaps *maps);
cudaError_t launch_la_tma(const LaArgs &a, const LaMaps &maps, bool state_only, cudaStream_t st, int *launches);
cudaError_t launch_la_step(const LaStepArgs &a, int dtype, cudaStream_t st, int *launches);

// ---- group norm ----

struct NormArgs {
    int N, S, C, G;
    int act, wdtype;
    float eps;
    const void *x, *dy;
    const void *weight, *bias;              // [C] or null
    const int32_t *lengths;                 // [N] or null
    void *y;                                // y, or dx in the backward
    float *stats;                           // [N,G,2] mean and 1/std
    float *dw, *db;                         // [C]
    double *part;                           // scratch
    int32_t *status;
};

size_t norm_scratch(int N, int S, int C, int G, int dtype, bool backward);
cudaError_t launch_norm(const NormArgs &a, int dtype, bool backward, cudaStream_t st, int *launches);

}  // namespace semicrf
