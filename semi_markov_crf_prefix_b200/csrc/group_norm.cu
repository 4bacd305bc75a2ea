// group_norm.cu -- group norm with an activation on channels-last rows x [N][S][C]:
//   y = act(xh w_c + b_c),  xh = (x - mu_{n,g}) rstd_{n,g},
// statistics over the valid positions s < L_n and the C/G channels of group g, and its
// gradient  dz = dy act'(z),  dx = rstd (w dz - mean(w dz) - xh mean(w dz xh)),
// dw_c = sum dz xh,  db_c = sum dz.
//
// Bound by memory: x once where a row block fits a thread block's registers
// (norm_reg_kernel, norm_row_kernel), twice where it does not.  Measured, with the bytes
// that each form moves against the copy rate: 64 000 positions of 512 channels in bf16
// 43 us forward (131 MB, 47 %) and 60 us backward (197 MB, 50 %), with silu's two
// transcendentals a value; 4 x 200 000 x 256 bf16 with gelu 251 us in three kernels (410 MB
// read, then 820 MB read and written: 188 us at the copy rate).  The second pass is as near
// to the issue rate (22 operations a value) as to the memory's.
#include <float.h>
#include <math.h>

#include "encoder_internal.h"
#include "findings.cuh"

namespace semicrf {
namespace {

// ---- the elementwise part ----

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The upper tail 1 - Phi(|z|) of the normal distribution, and exp(-z^2 / 2): Abramowitz
// and Stegun 7.1.26, erfc(x) = (a1 t + .. + a5 t^5) exp(-x^2) with t = 1 / (1 + p x) and an
// error below 1.5e-7, at x = |z| / sqrt 2 with the half and the root in the constants.
// Eleven operations of which two are transcendental; with the library's erfcf the
// two-pass kernel ran at a fifth of the memory's rate.  The bound is absolute: of GELU's
// value itself 5e-5 at z = -3, where that is -4e-3, and more further out.
__device__ __forceinline__ float normal_tail(float z, float &e)
{
    e = exp2_approx(z * z * -0.72134752044448170f);
    const float t = rcp_approx(fmaf(0.23164189f, fabsf(z), 1.f));
    return t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 0.5307027145f, -0.7265760135f), 0.7107068705f), -0.142248368f),
                    0.127414796f) * e;
}

__device__ __forceinline__ float sigmoid(float z) { return rcp_approx(1.f + exp2_approx(z * -1.4426950408889634f)); }

template <int ACT>
__device__ __forceinline__ float activate(float z)
{
    float e;
    if constexpr (ACT == SEMICRF_ACT_SILU) return z * sigmoid(z);
    if constexpr (ACT == SEMICRF_ACT_GELU) return fmaf(-fabsf(z), normal_tail(z, e), fmaxf(z, 0.f));
    return z;
}

template <int ACT>
__device__ __forceinline__ float slope(float z)
{
    if constexpr (ACT == SEMICRF_ACT_SILU) {
        const float s = sigmoid(z);
        return s * fmaf(z, 1.f - s, 1.f);
    }
    if constexpr (ACT == SEMICRF_ACT_GELU) {
        float e;
        const float tail = normal_tail(z, e);
        return fmaf(z * 0.39894228040143268f, e, z < 0.f ? tail : 1.f - tail);
    }
    return 1.f;
}

template <int N>
struct Int {
    static constexpr int value = N;
};

// The loop body for the call's activation: chosen once for many values.
template <typename F>
__device__ __forceinline__ void by_activation(int act, F &&body)
{
    if (act == SEMICRF_ACT_SILU)
        body(Int<SEMICRF_ACT_SILU>());
    else if (act == SEMICRF_ACT_GELU)
        body(Int<SEMICRF_ACT_GELU>());
    else
        body(Int<SEMICRF_ACT_NONE>());
}

template <typename T>
__device__ __forceinline__ float weight_at(const void *p, int wdtype, int c, float none)
{
    if (!p) return none;
    return wdtype == SEMICRF_F32 ? static_cast<const float *>(p)[c] : to_f<T>(static_cast<const T *>(p)[c]);
}

__device__ __forceinline__ int norm_length(const NormArgs &a, int n)
{
    if (!a.lengths) return a.S;
    const int L = a.lengths[n];
    if (L < 0 || L > a.S) {
        report(a.status, SEMICRF_ERR_INVALID_LENGTH);
        return max(0, min(L, a.S));
    }
    return L;
}

// ---- rows that fit a block's registers ----
//
// Thread (r, col) holds U vectors of VEC channels: rows rl, rl + RL, ... of row block n.
// NB row blocks lie side by side in a thread block, RL lanes of rows in each.  One read of
// x (and dy), the statistics from registers in two exact passes (mean, then squares about
// it), one write.  Rows of more vectors than threads are cut into slices of whole groups
// (blockIdx.y), which have nothing to do with one another.
struct RegShape {
    int CV, G, slices;   // vectors and groups of a slice's row (the last slice may have fewer); slices
    int RL, NB, W;       // row lanes a block; row blocks a thread block; lanes that sum one group
};

constexpr int kRegThreads = 512;

template <typename V>
__device__ __forceinline__ V warp_sum(V v, int width)
{
    for (int o = width >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums red[r][col] over a group's columns and its row block's lanes, for every (row block, group), into out.
__device__ __forceinline__ void group_sums(const float *red, float *out, const RegShape &sh, int G, int CgV)
{
    const int per = kRegThreads / sh.W, w = threadIdx.x % sh.W, items = sh.RL * CgV;
    for (int base = 0; base < sh.NB * G; base += per) {
        const int o = base + threadIdx.x / sh.W;
        float s = 0.f;
        if (o < sh.NB * G) {
            const int nb = o / G, g = o % G;
            for (int i = w; i < items; i += sh.W) s += red[(nb * sh.RL + i / CgV) * sh.CV + g * CgV + i % CgV];
        }
        s = warp_sum(s, sh.W);
        if (w == 0 && o < sh.NB * G) out[o] = s;
    }
}

// Two and three blocks an SM for one vector a thread spill 252 and 124 bytes at 16 bits and 8
// values a vector, and are faster all the same: 16 000 row blocks of 8 x 512 forward 192 us
// (205 with two blocks and no spill), forward and backward 467 (545 with one).
template <typename T, int VEC, int U, bool BWD>
__global__ __launch_bounds__(kRegThreads, U == 1 ? (BWD ? 2 : 3) : 1) void norm_reg_kernel(const __grid_constant__ NormArgs a, const RegShape sh)
{
    extern __shared__ float shm[];
    float *red = shm, *red2 = red + kRegThreads, *mean = red2 + kRegThreads, *aux = mean + sh.NB * sh.G;
    const int tid = threadIdx.x, col = tid % sh.CV, r = tid / sh.CV, nb = r / sh.RL, rl = r % sh.RL;
    const int Cg = a.C / a.G, CgV = Cg / VEC, c0 = (blockIdx.y * sh.CV + col) * VEC, g = col / CgV;
    const bool mine = nb < sh.NB && c0 < a.C;
    float wt[VEC], bs[VEC], dw[VEC], db[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        wt[e] = mine ? weight_at<T>(a.weight, a.wdtype, c0 + e, 1.f) : 0.f;
        bs[e] = mine ? weight_at<T>(a.bias, a.wdtype, c0 + e, 0.f) : 0.f;
        dw[e] = db[e] = 0.f;
    }
    // a thread's share to its group's sum over the row block
    auto total = [&](float share, float *red, float *out) {
        red[tid] = share;
        __syncthreads();
        group_sums(red, out, sh, sh.G, CgV);
        __syncthreads();
        return mine ? out[nb * sh.G + g] : 0.f;
    };
    auto fetch = [&](int n0, Pack<T, VEC>(&x)[U], Pack<T, VEC>(&dy)[BWD ? U : 1]) {
        const int n = n0 + nb;
        const int L = mine && n < a.N ? norm_length(a, n) : 0;
        const long long base = ((long long)n * a.S) * a.C + c0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = rl + u * sh.RL;
            if (s < L) {
                x[u] = *reinterpret_cast<const Pack<T, VEC> *>(static_cast<const T *>(a.x) + base + (long long)s * a.C);
                if (BWD)
                    dy[BWD ? u : 0] =
                        *reinterpret_cast<const Pack<T, VEC> *>(static_cast<const T *>(a.dy) + base + (long long)s * a.C);
            }
        }
        return L;
    };
    for (int n0 = blockIdx.x * sh.NB; n0 < a.N; n0 += gridDim.x * sh.NB) {
        const int n = n0 + nb;
        const bool on = mine && n < a.N;
        const long long base = ((long long)n * a.S) * a.C + c0;
        Pack<T, VEC> x[U], dy[BWD ? U : 1];
        const int L = fetch(n0, x, dy);
        const float inv = 1.f / fmaxf((float)L * Cg, 1.f);
        float mu, rs;
        if (!BWD) {
            float sum = 0.f, f[VEC];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (rl + u * sh.RL < L) {
                    unpack(x[u], f);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) sum += f[e];
                }
            mu = total(sum, red, mean) / fmaxf((float)L * Cg, 1.f);   // (a constant's mean is that constant)
            sum = 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (rl + u * sh.RL < L) {
                    unpack(x[u], f);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) sum = fmaf(f[e] - mu, f[e] - mu, sum);
                }
            rs = rsqrtf(fmaf(total(sum, red2, aux), inv, a.eps));
            if (on && a.stats && rl == 0 && c0 % Cg == 0) {
                float *st = a.stats + 2 * ((long long)n * a.G + blockIdx.y * sh.G + g);
                st[0] = mu;
                st[1] = rs;
            }
            by_activation(a.act, [&](auto act) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int s = rl + u * sh.RL;
                    if (!on || s >= a.S) continue;
                    float y[VEC];
                    unpack(x[u], f);
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        y[e] = s < L ? activate<act.value>(fmaf((f[e] - mu) * rs, wt[e], bs[e])) : 0.f;
                    *reinterpret_cast<Pack<T, VEC> *>(static_cast<T *>(a.y) + base + (long long)s * a.C) = pack<T, VEC>(y);
                }
            });
        } else {
            const float *st = a.stats + 2 * ((long long)(on ? n : 0) * a.G + (mine ? blockIdx.y * sh.G + g : 0));
            mu = st[0];
            rs = st[1];
            float s1 = 0.f, s2 = 0.f;
            float gz[U][VEC];
            by_activation(a.act, [&](auto act) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (rl + u * sh.RL >= L) continue;
                    float f[VEC], g[VEC];
                    unpack(x[u], f);
                    unpack(dy[BWD ? u : 0], g);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float xh = (f[e] - mu) * rs;
                        const float dz = g[e] * slope<act.value>(fmaf(xh, wt[e], bs[e]));
                        gz[u][e] = dz * wt[e];
                        s1 += gz[u][e];
                        s2 = fmaf(gz[u][e], xh, s2);
                        dw[e] = fmaf(dz, xh, dw[e]);
                        db[e] += dz;
                    }
                }
            });
            s1 = inv * total(s1, red, mean);
            s2 = inv * total(s2, red2, aux);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int s = rl + u * sh.RL;
                if (!on || s >= a.S) continue;
                float y[VEC], f[VEC];
                unpack(x[u], f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) y[e] = s < L ? rs * (gz[u][e] - s1 - (f[e] - mu) * rs * s2) : 0.f;
                *reinterpret_cast<Pack<T, VEC> *>(static_cast<T *>(a.y) + base + (long long)s * a.C) = pack<T, VEC>(y);
            }
        }
        __syncthreads();   // the sums' buffers serve the next row blocks
    }
    if (BWD) {
        // this block's share of dw and db: part[block][2][C]
        float *acc = shm;   // [rows][2] of one channel vector element at a time
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            __syncthreads();
            acc[tid] = mine ? dw[e] : 0.f;
            acc[kRegThreads + tid] = mine ? db[e] : 0.f;
            __syncthreads();
            if (r == 0 && mine) {
                double sw = 0.0, sb = 0.0;
                for (int j = col; j < sh.NB * sh.RL * sh.CV; j += sh.CV) {
                    sw += (double)acc[j];
                    sb += (double)acc[kRegThreads + j];
                }
                double *p = a.part + (long long)blockIdx.x * 2 * a.C + c0 + e;
                p[0] = sw;
                p[a.C] = sb;
            }
        }
    }
}

// Row blocks of one row whose groups lie in `lanes` neighbouring threads (a power of two):
// normalising each position by itself.  A thread keeps its channels, so their weights
// stay in registers, and steps from row to row with the next one already on its way;
// sums are shuffles.
template <typename T, int VEC, bool BWD>
__global__ __launch_bounds__(256) void norm_row_kernel(const __grid_constant__ NormArgs a, int CV, int rows, int lanes)
{
    __shared__ float acc[BWD ? 2 : 1][BWD ? 256 : 1];
    const int tid = threadIdx.x, col = tid % CV, r = tid / CV, c0 = col * VEC;
    const bool mine = r < rows;
    const float inv = 1.f / (float)(a.C / a.G);
    float wt[VEC], bs[VEC], dw[VEC], db[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        wt[e] = weight_at<T>(a.weight, a.wdtype, c0 + e, 1.f);
        bs[e] = weight_at<T>(a.bias, a.wdtype, c0 + e, 0.f);
        dw[e] = db[e] = 0.f;
    }
    const int step = gridDim.x * rows;
    const long long stride = (long long)step * CV;
    int n = blockIdx.x * rows + r;
    const long long at = (long long)n * CV + col;
    const Pack<T, VEC> *px = static_cast<const Pack<T, VEC> *>(a.x) + at, *pd = static_cast<const Pack<T, VEC> *>(a.dy) + at;
    Pack<T, VEC> *py = static_cast<Pack<T, VEC> *>(a.y) + at;
    float *st = a.stats + 2 * ((long long)n * a.G + c0 / (a.C / a.G));
    const long long ststep = 2LL * step * a.G;
    Pack<T, VEC> nx, nd;
    auto fetch = [&](int m) {   // false: nothing there
        const bool on = mine && m < a.N && (!a.lengths || norm_length(a, m) == 1);
        if (on) {
            nx = *px;
            if (BWD) nd = *pd;
        }
        px += stride;
        if (BWD) pd += stride;
        return on;
    };
    by_activation(a.act, [&](auto act) {
        bool next = fetch(n);
        // (every lane takes part in the shuffles: the block's last rows decide)
        for (int first = n - r; first < a.N; first += step) {
            const bool on = next, write = mine && n < a.N;
            float f[VEC], g[VEC], y[VEC], sum = 0.f, sq = 0.f;
            if (on) {
                unpack(nx, f);
                if (BWD) unpack(nd, g);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) f[e] = g[e] = 0.f;
            }
            next = fetch(n + step);
            if constexpr (!BWD) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) sum += f[e];
                const float mu = warp_sum(sum, lanes) / (float)(a.C / a.G);   // (a constant's mean is that constant)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    f[e] -= mu;
                    sq = fmaf(f[e], f[e], sq);
                }
                const float rs = rsqrtf(fmaf(warp_sum(sq, lanes), inv, a.eps));
                if (write && col % lanes == 0) *reinterpret_cast<float2 *>(st) = make_float2(mu, rs);
#pragma unroll
                for (int e = 0; e < VEC; ++e) y[e] = activate<act.value>(fmaf(f[e] * rs, wt[e], bs[e]));
            } else {
                float2 s = make_float2(0.f, 0.f);
                if (on) s = *reinterpret_cast<const float2 *>(st);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    f[e] = (f[e] - s.x) * s.y;
                    const float dz = g[e] * slope<act.value>(fmaf(f[e], wt[e], bs[e]));
                    dw[e] = fmaf(dz, f[e], dw[e]);
                    db[e] += dz;
                    g[e] = dz * wt[e];
                    sum += g[e];
                    sq = fmaf(g[e], f[e], sq);
                }
                sum = warp_sum(sum, lanes) * inv;
                sq = warp_sum(sq, lanes) * inv;
#pragma unroll
                for (int e = 0; e < VEC; ++e) y[e] = s.y * (g[e] - fmaf(f[e], sq, sum));
            }
            if (!on) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) y[e] = 0.f;
            }
            if (write) *py = pack<T, VEC>(y);
            py += stride;
            st += ststep;
            n += step;
        }
    });
    if constexpr (BWD) {
        // this block's share of dw and db: part[block][2][C]
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            __syncthreads();
            acc[0][tid] = mine ? dw[e] : 0.f;
            acc[1][tid] = mine ? db[e] : 0.f;
            __syncthreads();
            if (r == 0) {
                double sw = 0.0, sb = 0.0;
                for (int j = col; j < rows * CV; j += CV) {
                    sw += (double)acc[0][j];
                    sb += (double)acc[1][j];
                }
                double *p = a.part + (long long)blockIdx.x * 2 * a.C + c0 + e;
                p[0] = sw;
                p[a.C] = sb;
            }
        }
    }
}

// dw[c], db[c] from P rows of partial sums [P][2][C]: 8 channels and 64 strands of rows a block.
// Row blocks that come in pieces: sums so far in acc [2][C], dw and db with the last piece.
__global__ __launch_bounds__(512) void norm_params_kernel(const double *part, int P, int C, float *dw, float *db,
                                                          double *acc, bool first, bool last)
{
    __shared__ double sh[2][64][8];
    const int c = blockIdx.x * 8 + threadIdx.x, j = threadIdx.y;
    double w = 0.0, b = 0.0;
    if (c < C) {
#pragma unroll 4
        for (int i = j; i < P; i += 64) {
            w += part[(long long)i * 2 * C + c];
            b += part[(long long)i * 2 * C + C + c];
        }
    }
    sh[0][j][threadIdx.x] = w;
    sh[1][j][threadIdx.x] = b;
    for (int half = 32; half > 0; half >>= 1) {
        __syncthreads();
        if (j < half) {
            sh[0][j][threadIdx.x] += sh[0][j + half][threadIdx.x];
            sh[1][j][threadIdx.x] += sh[1][j + half][threadIdx.x];
        }
    }
    if (j == 0 && c < C) {
        w = sh[0][0][threadIdx.x] + (first ? 0.0 : acc[c]);
        b = sh[1][0][threadIdx.x] + (first ? 0.0 : acc[C + c]);
        if (!last) {
            acc[c] = w;
            acc[C + c] = b;
        } else {
            if (dw) dw[c] = (float)w;
            if (db) db[c] = (float)b;
        }
    }
}

// ---- long rows: two passes over the data ----
//
// Pass 1: two numbers for each channel of a strip of positions, part[n][strip][2][C] in
// float64: forward the mean and the sum of squares about it, backward the sums of dz xh and
// dz.  A thread takes a strip's values of a channel, kRun at most, in float32 less the mean
// of its first eight (so that a mean far from zero costs no bits), eight at a time: the sums
// s of their distances d from the mean m of the n before them and t of the squares,
//   m += s / (n + 8),   M2 += t - s^2 / (n + 8),
// where at least half of t stays, whatever the values are.  (Sums about the first value
// alone lost 2^-13 of the variance where that one was an outlier.)  Means and squares of row
// lanes, strips and channels are joined about a common value in float64.  Then
// the groups' statistics, then pass 2 writes y or dx, strips in the opposite order: the
// ones that pass 1 read last are still in the L2 cache.
constexpr int kLongThreads = 256, kRun = 128;

struct LongShape {
    int CV, tiles, R, strips, rows;   // vectors a row, column tiles of <= 256 of them, row lanes, strips, rows a strip
};

template <typename T, int VEC, bool BWD>
__global__ __launch_bounds__(kLongThreads, 3) void norm_sums_kernel(const __grid_constant__ NormArgs a, const LongShape sh)
{
    extern __shared__ double dsm[];
    const int cols = min(sh.CV, kLongThreads), tid = threadIdx.x, r = tid / cols;
    const int cv = blockIdx.y * kLongThreads + tid % cols, n = blockIdx.x / sh.strips, strip = blockIdx.x % sh.strips;
    const bool mine = r < sh.R && cv < sh.CV;
    const int L = norm_length(a, n), s0 = strip * sh.rows, s1 = min(L, s0 + sh.rows), c0 = cv * VEC;
    const long long base = (long long)n * a.S * a.C + c0;
    float p[VEC], q[VEC], about[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) p[e] = q[e] = about[e] = 0.f;
    int cnt = 0;
    if (mine && s0 + r < s1) {
        const T *px = static_cast<const T *>(a.x) + base, *pd = static_cast<const T *>(a.dy) + base;
        if constexpr (!BWD) {
            constexpr int U = 8;   // loads in flight
            // the first m of x to the mean p (less about) and the squares q of the cnt before them
            auto add = [&](const Pack<T, VEC> (&x)[U], auto whole, int m) {
                const float n = (float)(cnt + m), inv = 1.f / n;
                float f[VEC];
                if (cnt == 0) {
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (whole.value || u < m) {
                            unpack(x[u], f);
#pragma unroll
                            for (int e = 0; e < VEC; ++e) about[e] = fmaf(f[e], inv, about[e]);
                        }
                }
                float sum[VEC], sq[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) sum[e] = sq[e] = 0.f;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (whole.value || u < m) {
                        unpack(x[u], f);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            const float d = f[e] - about[e] - p[e];
                            sum[e] = fmaf(d, inv, sum[e]);   // (divided, so that no finite values overflow)
                            sq[e] = fmaf(d, d, sq[e]);
                        }
                    }
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    p[e] += sum[e];
                    q[e] += sq[e] <= FLT_MAX ? fmaf(-sum[e], sum[e] * n, sq[e]) : sq[e];
                }
                cnt += m;
            };
            int s = s0 + r;
            for (; s + (U - 1) * sh.R < s1; s += U * sh.R) {
                Pack<T, VEC> x[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    x[u] = *reinterpret_cast<const Pack<T, VEC> *>(px + (long long)(s + u * sh.R) * a.C);
                add(x, Int<1>(), U);
            }
            if (s < s1) {   // the strip's last rows, together as well
                Pack<T, VEC> x[U];
#pragma unroll
                for (int u = 0; u < U - 1; ++u)
                    if (s + u * sh.R < s1)
                        x[u] = *reinterpret_cast<const Pack<T, VEC> *>(px + (long long)(s + u * sh.R) * a.C);
                add(x, Int<0>(), (s1 - s + sh.R - 1) / sh.R);
            }
        } else {
            float wt[VEC], bs[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                wt[e] = weight_at<T>(a.weight, a.wdtype, c0 + e, 1.f);
                bs[e] = weight_at<T>(a.bias, a.wdtype, c0 + e, 0.f);
            }
            const float *st = a.stats + 2 * ((long long)n * a.G + c0 / (a.C / a.G));   // a vector lies inside one group
            const float mu = st[0], rs = st[1];
            by_activation(a.act, [&](auto act) {
                auto add = [&](const Pack<T, VEC> &x, const Pack<T, VEC> &dy) {
                    float f[VEC], g[VEC];
                    unpack(x, f);
                    unpack(dy, g);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float xh = (f[e] - mu) * rs;
                        const float dz = g[e] * slope<act.value>(fmaf(xh, wt[e], bs[e]));
                        p[e] = fmaf(dz, xh, p[e]);
                        q[e] += dz;
                    }
                };
                constexpr int U = 4;
                for (int s = s0 + r; s < s1; s += U * sh.R) {
                    Pack<T, VEC> x[U], dy[U];
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (s + u * sh.R < s1) {
                            x[u] = *reinterpret_cast<const Pack<T, VEC> *>(px + (long long)(s + u * sh.R) * a.C);
                            dy[u] = *reinterpret_cast<const Pack<T, VEC> *>(pd + (long long)(s + u * sh.R) * a.C);
                        }
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (s + u * sh.R < s1) add(x[u], dy[u]);
                }
            });
        }
    }
    double *out = a.part + ((long long)n * sh.strips + strip) * 2 * a.C;
    if (sh.R == 1) {   // nothing to join
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (mine) {
                out[c0 + e] = (double)about[e] + (double)p[e];
                out[a.C + c0 + e] = (double)q[e];
            }
        return;
    }
    // dsm[e][2][thread]; then a thread joins the row lanes of one channel
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        dsm[2 * e * kLongThreads + tid] = (double)about[e] + (double)p[e];
        dsm[(2 * e + 1) * kLongThreads + tid] = (double)q[e];
    }
    __syncthreads();
    for (int i = tid; i < cols * VEC; i += kLongThreads) {
        const int col = i % cols, e = i / cols, c = (blockIdx.y * kLongThreads + col) * VEC + e;
        if (c >= a.C) continue;
        const double *u = dsm + 2 * e * kLongThreads + col, *v = u + kLongThreads;
        double x = 0.0, y = 0.0;
        if constexpr (BWD) {
            for (int j = 0; j < sh.R; ++j) {
                x += u[j * cols];
                y += v[j * cols];
            }
        } else if (s0 < s1) {
            // row lane j took the strip's rows j, j + R, ..: about the first lane's mean
            const double first = u[0];
            const int each = (s1 - s0) / sh.R, more = (s1 - s0) % sh.R;
            for (int j = 0; j < sh.R && s0 + j < s1; ++j) {
                const double d = u[j * cols] - first, all = (double)(each + (j < more)) * d;
                x += all;
                y += fma(all, d, v[j * cols]);
            }
            const double m = x / (double)(s1 - s0);
            y -= x * m;
            x = first + m;
        }
        out[c] = x;
        out[a.C + c] = y;
    }
}

// (n, g): mean and 1/std (forward), or the means of w dz and w dz xh (backward, to gsum
// [N,G,2]) and row block n's share of dw and db (to total [N][2][C]).  Thread (x, y): channel
// x of the group (and x + X, ..), strand y of the strips.
template <typename T, bool BWD>
__global__ __launch_bounds__(256) void norm_group_kernel(const __grid_constant__ NormArgs a, int strips, int rows,
                                                         float *gsum, double *total, int X)
{
    const int n = blockIdx.x / a.G, g = blockIdx.x % a.G, Cg = a.C / a.G, Y = 256 / X;
    const int x = threadIdx.x % X, y = threadIdx.x / X;
    const double *part = a.part + (long long)n * strips * 2 * a.C + g * Cg;
    __shared__ double sa[256], sb[256];
    double A = 0.0, B = 0.0;   // the group's
    // forward: sums about the first strip's mean of the first channel
    const int L = norm_length(a, n);
    const double about = BWD ? 0.0 : part[0];
    for (int c0 = 0; c0 < Cg; c0 += X) {
        const int c = c0 + x;
        double p = 0.0, q = 0.0;
        if (c < Cg) {
#pragma unroll 4
            for (int i = y; i < strips; i += Y) {
                const double u = part[(long long)i * 2 * a.C + c], v = part[(long long)i * 2 * a.C + a.C + c];
                if constexpr (BWD) {
                    p += u;
                    q += v;
                } else {
                    const long long have = min((long long)rows, (long long)L - (long long)i * rows);
                    if (have <= 0) break;
                    const double d = u - about, all = (double)have * d;
                    p += all;
                    q += fma(all, d, v);
                }
            }
        }
        if (!BWD) {
            A += p;
            B += q;
            continue;
        }
        __syncthreads();
        sa[threadIdx.x] = p;
        sb[threadIdx.x] = q;
        for (int half = Y / 2; half > 0; half >>= 1) {
            __syncthreads();
            if (y < half) {
                sa[threadIdx.x] += sa[threadIdx.x + half * X];
                sb[threadIdx.x] += sb[threadIdx.x + half * X];
            }
        }
        if (y == 0 && c < Cg) {
            const double w = (double)weight_at<T>(a.weight, a.wdtype, g * Cg + c, 1.f);
            A += w * sa[x];
            B += w * sb[x];
            double *t = total + (long long)n * 2 * a.C + g * Cg + c;
            t[0] = sa[x];
            t[a.C] = sb[x];
        }
    }
    __syncthreads();
    A = warp_sum(A, 32);
    B = warp_sum(B, 32);
    if ((threadIdx.x & 31) == 0) {
        sa[threadIdx.x >> 5] = A;
        sb[threadIdx.x >> 5] = B;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        A = B = 0.0;
        for (int j = 0; j < 8; ++j) {
            A += sa[j];
            B += sb[j];
        }
        const double cnt = fmax((double)L * Cg, 1.0);
        float *o = (BWD ? gsum : a.stats) + 2 * (long long)blockIdx.x;
        if (BWD) {
            o[0] = (float)(B / cnt);   // mean of w dz
            o[1] = (float)(A / cnt);   // mean of w dz xh
        } else {
            const double m = A / cnt, variance = B / cnt - m * m;
            o[0] = (float)(about + m);
            o[1] = (float)(1.0 / sqrt((variance < 0.0 ? 0.0 : variance) + (double)a.eps));   // (NaN stays NaN)
        }
    }
}

template <typename T, int VEC, bool BWD>
__global__ __launch_bounds__(kLongThreads, BWD ? 3 : 4) void norm_apply_kernel(const __grid_constant__ NormArgs a,
                                                                               const LongShape sh, const float *gsum)
{
    const int cols = min(sh.CV, kLongThreads), tid = threadIdx.x, r = tid / cols;
    const int cv = blockIdx.y * kLongThreads + tid % cols;
    const int back = gridDim.x - 1 - blockIdx.x, n = back / sh.strips, strip = back % sh.strips;
    if (r >= sh.R || cv >= sh.CV) return;
    const int L = norm_length(a, n), s0 = strip * sh.rows, s1 = min(a.S, s0 + sh.rows), c0 = cv * VEC;
    const long long base = (long long)n * a.S * a.C + c0;
    float wt[VEC], bs[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        wt[e] = weight_at<T>(a.weight, a.wdtype, c0 + e, 1.f);
        bs[e] = weight_at<T>(a.bias, a.wdtype, c0 + e, 0.f);
    }
    const long long at = 2 * ((long long)n * a.G + c0 / (a.C / a.G));   // a vector lies inside one group
    const float mu = a.stats[at], rs = a.stats[at + 1], g1 = BWD ? gsum[at] : 0.f, g2 = BWD ? gsum[at + 1] : 0.f;
    if (!BWD)
#pragma unroll
        for (int e = 0; e < VEC; ++e) wt[e] *= rs;
    const T *px = static_cast<const T *>(a.x) + base, *pd = static_cast<const T *>(a.dy) + base;
    T *py = static_cast<T *>(a.y) + base;
    const int in = min(s1, L);
    by_activation(a.act, [&](auto act) {
        auto value = [&](const Pack<T, VEC> &x, const Pack<T, VEC> &dy) {
            float y[VEC], f[VEC], g[VEC];
            unpack(x, f);
            if (BWD) unpack(dy, g);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float d = f[e] - mu;
                if constexpr (BWD) {
                    const float xh = d * rs, z = fmaf(xh, wt[e], bs[e]);
                    y[e] = rs * (g[e] * slope<act.value>(z) * wt[e] - g1 - xh * g2);
                } else {
                    y[e] = activate<act.value>(fmaf(d, wt[e], bs[e]));
                }
            }
            return pack<T, VEC>(y);
        };
        constexpr int U = 4;
        int s = s0 + r;
        for (; s + (U - 1) * sh.R < in; s += sh.R * U) {
            Pack<T, VEC> x[U], dy[BWD ? U : 1];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                x[u] = *reinterpret_cast<const Pack<T, VEC> *>(px + (long long)(s + u * sh.R) * a.C);
                if (BWD) dy[BWD ? u : 0] = *reinterpret_cast<const Pack<T, VEC> *>(pd + (long long)(s + u * sh.R) * a.C);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                *reinterpret_cast<Pack<T, VEC> *>(py + (long long)(s + u * sh.R) * a.C) = value(x[u], dy[BWD ? u : 0]);
        }
        for (; s < in; s += sh.R) {
            const Pack<T, VEC> x = *reinterpret_cast<const Pack<T, VEC> *>(px + (long long)s * a.C);
            *reinterpret_cast<Pack<T, VEC> *>(py + (long long)s * a.C) =
                value(x, BWD ? *reinterpret_cast<const Pack<T, VEC> *>(pd + (long long)s * a.C) : x);
        }
        // behind the row block's end: zeros
        for (; s < s1; s += sh.R) {
            Pack<T, VEC> y;
#pragma unroll
            for (int e = 0; e < VEC; ++e) y.v[e] = from_f<T>(0.f);
            *reinterpret_cast<Pack<T, VEC> *>(py + (long long)s * a.C) = y;
        }
    });
}

// ---- launches ----

int pow2_at_least(int v, int most)
{
    int p = 1;
    while (p < v && p < most) p <<= 1;
    return p;
}

// The widest vector that stays inside one group: 16 bytes, 4 bytes or one value.
int norm_vec(int C, int G, int dtype)
{
    const int most = dtype == SEMICRF_F32 ? 4 : 8, Cg = C / G;
    if (Cg % most == 0) return most;
    return dtype != SEMICRF_F32 && Cg % 2 == 0 ? 2 : 1;
}

// The next narrower vector (0 behind the narrowest).
int narrower(int vec, int dtype) { return vec == 1 ? 0 : vec > 2 && dtype != SEMICRF_F32 ? 2 : 1; }

// Registers hold a row block where its rows take at most 32 values a thread.
bool reg_shape(int S, int C, int G, int vec, RegShape *sh)
{
    const int CgV = C / G / vec;
    if (CgV > kRegThreads) return false;
    sh->slices = (G + kRegThreads / CgV - 1) / (kRegThreads / CgV);
    sh->G = (G + sh->slices - 1) / sh->slices;
    sh->slices = (G + sh->G - 1) / sh->G;
    sh->CV = sh->G * CgV;
    const int R = kRegThreads / sh->CV;
    sh->RL = R < S ? R : S;
    sh->NB = R / sh->RL;
    if ((S + sh->RL - 1) / sh->RL > 32 / vec) return false;
    sh->W = pow2_at_least(sh->RL * (C / G / vec), 32);
    return true;
}

LongShape long_shape(int N, int S, int C, int vec)
{
    LongShape sh;
    sh.CV = C / vec;
    sh.tiles = (sh.CV + kLongThreads - 1) / kLongThreads;
    const int cols = sh.CV < kLongThreads ? sh.CV : kLongThreads;
    sh.R = kLongThreads / cols;
    // strips: eight blocks an SM over everything, each at least one batch of rows deep
    long long strips = (8LL * device_sm_count() + (long long)N * sh.tiles - 1) / ((long long)N * sh.tiles);
    const long long most = (S + sh.R * 8 - 1) / (sh.R * 8);
    if (strips > most) strips = most;
    const long long least = (S + (long long)sh.R * kRun - 1) / ((long long)sh.R * kRun);
    if (strips < least) strips = least;
    sh.rows = (int)((S + strips - 1) / strips);
    sh.strips = (S + sh.rows - 1) / sh.rows;
    return sh;
}

// The long form's scratch is 16 bytes for each channel, strip and row block (and as much again
// for a row block's dw and db), which for many short row blocks of wide rows is several
// times x.  Row blocks are taken in pieces whose scratch stays within 64 MB, half of the L2
// cache: a piece has 2048 thread blocks at least, so the GPU stays full.
struct LongPlan {
    LongShape sh;
    int rows;                        // row blocks of a piece
    size_t total, acc, gsum, bytes;  // offsets behind the strips' sums, and the whole
};

constexpr size_t kLongScratch = (size_t)64 << 20;

LongPlan long_plan(int N, int S, int C, int G, int vec, bool backward)
{
    LongPlan p;
    p.sh = long_shape(N, S, C, vec);
    const size_t strips = (size_t)p.sh.strips * 2 * C * sizeof(double), row = 2 * (size_t)C * sizeof(double),
                 group = 2 * (size_t)G * sizeof(float), each = strips + (backward ? row + group : 0);
    const size_t most = kLongScratch / each;
    p.rows = most < 1 ? 1 : most < (size_t)N ? (int)most : N;
    p.total = p.rows * strips;
    p.acc = p.total + (backward ? p.rows * row : 0);
    p.gsum = p.acc + (backward ? row : 0);
    p.bytes = p.gsum + (backward ? p.rows * group : 0);
    return p;
}

int reg_blocks(int N, const RegShape &sh)
{
    const int blocks = (N + sh.NB - 1) / sh.NB, most = 6 * device_sm_count() / sh.slices;
    return blocks < most ? blocks : most > 1 ? most : 1;
}

// Lanes of a group in norm_row_kernel, 0 where it does not apply.
int row_lanes(int S, int C, int G, int vec)
{
    const int CgV = C / G / vec;
    return S == 1 && C / vec <= 256 && CgV <= 32 && (CgV & (CgV - 1)) == 0 ? CgV : 0;
}

// As many as an SM holds of them (48 and 80 registers a thread).
int row_blocks(int N, int rows, bool backward)
{
    const int blocks = (N + rows - 1) / rows, most = (backward ? 3 : 5) * device_sm_count();
    return blocks < most ? blocks : most;
}

template <typename T, int VEC, bool BWD>
cudaError_t norm_go(NormArgs a, cudaStream_t st, int *n)
{
    RegShape rsh;
    cudaError_t e;
    int prows;
    if (const int lanes = row_lanes(a.S, a.C, a.G, VEC)) {
        const int CV = a.C / VEC, rows = 256 / CV, blocks = row_blocks(a.N, rows, BWD);
        e = timed_launch(st, n, [&] { norm_row_kernel<T, VEC, BWD><<<blocks, 256, 0, st>>>(a, CV, rows, lanes); });
        if (e != cudaSuccess) return e;
        prows = blocks;
    } else if (reg_shape(a.S, a.C, a.G, VEC, &rsh)) {
        const int blocks = reg_blocks(a.N, rsh);
        const dim3 grid(blocks, rsh.slices);
        const size_t smem = (2 * kRegThreads + 2 * (size_t)rsh.NB * rsh.G) * sizeof(float);
        e = timed_launch(st, n, [&] {
            if ((a.S + rsh.RL - 1) / rsh.RL == 1)
                norm_reg_kernel<T, VEC, 1, BWD><<<grid, kRegThreads, smem, st>>>(a, rsh);
            else
                norm_reg_kernel<T, VEC, 32 / VEC, BWD><<<grid, kRegThreads, smem, st>>>(a, rsh);
        });
        if (e != cudaSuccess) return e;
        prows = blocks;
    } else {
        const LongPlan p = long_plan(a.N, a.S, a.C, a.G, VEC, BWD);
        const LongShape &sh = p.sh;
        unsigned char *scratch = reinterpret_cast<unsigned char *>(a.part);
        double *total = reinterpret_cast<double *>(scratch + p.total), *acc = reinterpret_cast<double *>(scratch + p.acc);
        float *gsum = reinterpret_cast<float *>(scratch + p.gsum);
        const int X = pow2_at_least(a.C / a.G, 256);
        for (int n0 = 0; n0 < a.N; n0 += p.rows) {
            NormArgs b = a;
            b.N = a.N - n0 < p.rows ? a.N - n0 : p.rows;
            const size_t at = (size_t)n0 * a.S * a.C;
            b.x = static_cast<const T *>(a.x) + at;
            if (BWD) b.dy = static_cast<const T *>(a.dy) + at;
            b.y = static_cast<T *>(a.y) + at;
            b.stats = a.stats + (size_t)n0 * a.G * 2;
            if (a.lengths) b.lengths = a.lengths + n0;
            const dim3 grid((unsigned)(b.N * sh.strips), sh.tiles);
            e = timed_launch(st, n, [&] {
                norm_sums_kernel<T, VEC, BWD><<<grid, kLongThreads, 2 * VEC * kLongThreads * sizeof(double), st>>>(b, sh);
            });
            if (e != cudaSuccess) return e;
            e = timed_launch(st, n, [&] {
                norm_group_kernel<T, BWD><<<b.N * a.G, 256, 0, st>>>(b, sh.strips, sh.rows, gsum, total, X);
            });
            if (e != cudaSuccess) return e;
            e = timed_launch(st, n, [&] { norm_apply_kernel<T, VEC, BWD><<<grid, kLongThreads, 0, st>>>(b, sh, gsum); });
            if (e != cudaSuccess) return e;
            if (!BWD || (!a.dw && !a.db)) continue;
            e = timed_launch(st, n, [&] {
                norm_params_kernel<<<(a.C + 7) / 8, dim3(8, 64), 0, st>>>(total, b.N, a.C, a.dw, a.db, acc, n0 == 0,
                                                                        n0 + b.N == a.N);
            });
            if (e != cudaSuccess) return e;
        }
        return cudaSuccess;
    }
    if (!BWD || (!a.dw && !a.db)) return cudaSuccess;
    return timed_launch(st, n, [&] {
        norm_params_kernel<<<(a.C + 7) / 8, dim3(8, 64), 0, st>>>(a.part, prows, a.C, a.dw, a.db, nullptr, true, true);
    });
}

template <typename T, bool BWD>
cudaError_t norm_type(const NormArgs &a, int vec, cudaStream_t st, int *n)
{
    if constexpr (sizeof(T) == 2)
        if (vec == 8) return norm_go<T, 8, BWD>(a, st, n);
    if constexpr (sizeof(T) == 4)
        if (vec == 4) return norm_go<T, 4, BWD>(a, st, n);
    if constexpr (sizeof(T) == 2)
        if (vec == 2) return norm_go<T, 2, BWD>(a, st, n);
    return norm_go<T, 1, BWD>(a, st, n);
}

}  // namespace

size_t norm_scratch(int N, int S, int C, int G, int dtype, bool backward)
{
    // a vector width below norm_vec (misaligned tensors) may take the other path: room for either
    size_t most = 0;
    for (int vec = norm_vec(C, G, dtype); vec >= 1; vec = narrower(vec, dtype)) {
        RegShape rsh;
        size_t n;
        if (row_lanes(S, C, G, vec)) {
            n = backward ? (size_t)row_blocks(N, 256 / (C / vec), true) * 2 * C * sizeof(double) : 0;
        } else if (reg_shape(S, C, G, vec, &rsh)) {
            n = backward ? (size_t)reg_blocks(N, rsh) * 2 * C * sizeof(double) : 0;
        } else {
            n = long_plan(N, S, C, G, vec, backward).bytes;
        }
        if (n > most) most = n;
    }
    return most;
}

cudaError_t launch_norm(const NormArgs &a, int dtype, bool backward, cudaStream_t st, int *launches)
{
    *launches = 0;
    int vec = norm_vec(a.C, a.G, dtype);
    // the vector accesses need their own alignment: rows are C values apart
    const size_t size = dtype == SEMICRF_F32 ? 4 : 2;
    const uintptr_t all = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y) |
                          reinterpret_cast<uintptr_t>(backward ? a.dy : a.x);
    while (vec > 1 && all % (vec * size)) vec = narrower(vec, dtype);
    if (dtype == SEMICRF_F32)
        return backward ? norm_type<float, true>(a, vec, st, launches) : norm_type<float, false>(a, vec, st, launches);
    if (dtype == SEMICRF_BF16)
        return backward ? norm_type<__nv_bfloat16, true>(a, vec, st, launches)
                        : norm_type<__nv_bfloat16, false>(a, vec, st, launches);
    return backward ? norm_type<__half, true>(a, vec, st, launches) : norm_type<__half, false>(a, vec, st, launches);
}

cudaError_t norm_found(int32_t *to) { return read_found(to); }
cudaError_t norm_clear_found(cudaStream_t st) { return clear_found(st); }

}  // namespace semicrf
