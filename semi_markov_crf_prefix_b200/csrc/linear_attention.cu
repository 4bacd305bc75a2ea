// linear_attention.cu -- linear attention with a decay for each head:
//   S_p = lam S_{p-1} + c k_p v_p^T,   o_p = b q_p S_p = b c sum_{j<=p} lam^{p-j} (q_p . k_j) v_j + b lam^{p+1} q_p S_in
// over whole sequences (la_chunk_kernel, la_token_kernel) and for single tokens
// (la_step_kernel).  The backward runs the same walks with exchanged operands:
//   dq = walk(dO, V, K)   dv = walk back in time(K, Q, dO)   dk = walk back in time(V, dO, Q).
#include <math.h>

#include "device_util.cuh"
#include "encoder_internal.h"
#include "tensor_core.cuh"

namespace semicrf {
namespace {

constexpr int kChunk = 128;     // positions of one step of the chunked walk

template <typename T>
constexpr int kTerms = sizeof(T) == 4 ? 3 : 1;
template <>
constexpr int kTerms<__half> = 2;   // 11 bits: two bf16 terms hold them exactly

// Shapes of the chunked walk for padded width D.  Operands enter the matrix unit as
// sums of bf16 terms: NI for the inputs (exact), NM for the products P and for the
// state as an operand of q S (2: 2^-17 relative, far inside the rounding of a 16-bit
// output; 3 for float32), NK = 3 for the decayed keys, whose products make the
// float32 state.
template <typename T, int D>
struct LaCfg {
    static constexpr int NI = kTerms<T>, NM = NI == 3 ? 3 : 2, NK = 3;
    static constexpr bool kStateTmem = D == 128;   // the state itself: float32 in tensor memory, or
    static constexpr int NS = kStateTmem ? NM : 3; // three bf16 terms (24 bits) in shared memory
    static constexpr int kTile = tile_bytes(kChunk, D), kSTile = tile_bytes(D, D);
    static constexpr int kQ = 0, kK = kQ + NI * kTile, kV = kK + NK * kTile, kS = kV + NI * kTile;
    static constexpr int kDec = kS + NS * kSTile, kMisc = kDec + (kChunk + 4) * 4;
    static constexpr int kSmem = kMisc + 32;
    // tensor memory columns: scores (P replaces them where two terms fit the same columns), o, k v^T, state
    static constexpr int kP = NM == 3 ? 128 : 0, kO = NM == 3 ? 320 : 128, kKV = kO + D, kState = kKV + D;
    static constexpr int kCols = kState + (kStateTmem ? D : 0) <= 256 ? 256 : 512;
    static constexpr int kBlocks = kCols == 256 && kSmem <= 114 * 1024 ? 2 : 1;
    static constexpr int NP = kChunk * (D / 8) / 256;   // 8-value pieces of a tile for each of 256 threads
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

template <typename T>
struct Piece {
    Pack<T, 16 / sizeof(T)> h[sizeof(T) / 2];   // 8 values
    __device__ __forceinline__ float get(int i) const
    {
        constexpr int n = 16 / sizeof(T);
        return to_f<T>(h[i / n].v[i % n]);
    }
};

// 8 values of row p (of the walk) from column d8 * 8 on; zeros outside the sequence and the width.
template <typename T>
__device__ __forceinline__ Piece<T> load_piece(const T *base, long long st, long long t, int d0, int d, bool in, int vec)
{
    constexpr int n = 16 / sizeof(T);
    Piece<T> r;
    if (vec) {
        if (in && d0 < d) {
            const Pack<T, n> *src = reinterpret_cast<const Pack<T, n> *>(base + t * st + d0);
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.h[i] = src[i];
            return r;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        r.h[i / n].v[i % n] = !vec && in && d0 + i < d ? base[t * st + d0 + i] : from_f<T>(0.f);
    return r;
}

union U16 {
    __nv_bfloat16 b[8];
    uint4 u;
};

// The piece in NT bf16 terms to its places of NT tiles.
template <typename T, int NT>
__device__ __forceinline__ void store_terms(unsigned char *tile, int tile_stride, int at, const Piece<T> &p, float w)
{
    U16 o[NT];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        __nv_bfloat16 t[NT];
        bf16_terms<NT>(w == 1.f ? p.get(i) : p.get(i) * w, t);
#pragma unroll
        for (int j = 0; j < NT; ++j) o[j].b[i] = t[j];
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) *reinterpret_cast<uint4 *>(tile + j * tile_stride + at) = o[j].u;
}

template <int N>
__device__ __forceinline__ float term_sum(const uint4 (&u)[N], int i)
{
    float s = 0.f;
#pragma unroll
    for (int j = N - 1; j >= 0; --j) {
        const uint32_t w = reinterpret_cast<const uint32_t *>(&u[j])[i >> 1];
        s += __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
    }
    return s;
}

__device__ __forceinline__ uint32_t pack2(__nv_bfloat16 lo, __nv_bfloat16 hi)
{
    return (uint32_t)__bfloat16_as_ushort(lo) | (uint32_t)__bfloat16_as_ushort(hi) << 16;
}

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

// The chunked walk: 128 positions at a time,
//   scores = Q K^T and Q S                           (tensor memory)
//   P = b c lam^{i-j} scores (j <= i), K~ = c lam^{end-j} K   (threads; P to tensor memory, K~ to shared)
//   o = P V + b lam^{i+1} (Q S),  KV = K~^T V        (tensor memory, read back by rows)
//   S = lam^n S + KV                                 (threads, float32)
// The matrix unit's accumulators round towards zero (measured: -1.4e-7 relative for
// each 8 steps of 16), which a state carried in them over thousands of chunks would
// show; so they hold one chunk's sums only, small terms first, and the state is
// advanced by float32 multiply-adds to nearest.
template <typename T, int D, bool STATE_ONLY>
__global__ __launch_bounds__(256, (LaCfg<T, D>::kBlocks)) void la_chunk_kernel(const __grid_constant__ LaArgs args)
{
    using G = LaCfg<T, D>;
    constexpr int NI = G::NI, NM = G::NM, NK = G::NK, NS = G::NS, NP = G::NP;
    extern __shared__ __align__(128) unsigned char sm[];
    const LaWalk &w = args.w[blockIdx.y];
    const LaSpan s = la_span(args, blockIdx.x);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, quad = warp & 3, half = warp >> 2;
    if (STATE_ONLY && s.seg == args.nseg - 1) return;
    if (!STATE_ONLY) {
        zero_rows<T>(w, s, 0, w.dv);
        if (s.L == 0 && s.last) copy_state(w, args, s, 0, w.dv);
    }
    if (s.pe == s.p0) return;

    float *dec = reinterpret_cast<float *>(sm + G::kDec);
    uint32_t *slot = reinterpret_cast<uint32_t *>(sm + G::kMisc + 16);
    const uint32_t smem = static_cast<uint32_t>(__cvta_generic_to_shared(sm));
    const uint32_t bar1 = smem + G::kMisc, bar2 = bar1 + 8;
    const float ld = args.log_decay[s.h], pa = w.b * w.c;
    if (warp == 0) tmem_alloc(static_cast<uint32_t>(__cvta_generic_to_shared(slot)), G::kCols);
    if (tid == 0) {
        mbar_init(bar1, 1);
        mbar_init(bar2, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid <= kChunk) dec[tid] = (float)decay_pow(ld, tid);

    const T *qb = static_cast<const T *>(w.q) + s.b * w.qs[0] + s.h * w.qs[2];
    const T *kb = static_cast<const T *>(w.k) + s.b * w.ks[0] + s.h * w.ks[2];
    const T *vb = static_cast<const T *>(w.v) + s.b * w.vs[0] + s.h * w.vs[2];
    Piece<T> rq[NP], rk[NP], rv[NP];
    auto fetch = [&](int pc) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int idx = tid + i * 256, d0 = idx % (D / 8) * 8, p = pc + idx / (D / 8);
            const bool in = p < s.pe;
            const long long t = w.reverse ? s.L - 1 - p : p;
            if (!STATE_ONLY) rq[i] = load_piece<T>(qb, w.qs[1], t, d0, w.dk, in, w.q_vec);
            rk[i] = load_piece<T>(kb, w.ks[1], t, d0, w.dk, in, w.k_vec);
            rv[i] = load_piece<T>(vb, w.vs[1], t, d0, w.dv, in, w.v_vec);
        }
    };
    fetch(s.p0);

    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tm = *slot, tlane = tm + ((uint32_t)(quad * 32) << 16);

    // this thread's row of the state (64 rows lie in the first 16 lanes of each quadrant)
    // and its half of the columns
    const int srow = D == 64 ? quad * 16 + (lane & 15) : quad * 32 + lane;
    const bool has_row = D == 128 || lane < 16;
    const int nv = (w.dv + 15) / 16 * 16, kd = (w.dk + 15) / 16;
    {
        const StateAt from = STATE_ONLY ? StateAt{nullptr, 0, 0} : state_from(w, args, s);
#pragma unroll 1
        for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 16) {
            uint32_t r[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const bool in = from.p && has_row && srow < w.dk && c + e < w.dv;
                r[e] = __float_as_uint(in ? from.p[(long long)srow * from.rs + (long long)(c + e) * from.cs] : 0.f);
            }
            if (G::kStateTmem) tmem_st16(tlane + G::kState + c, r);
            if (has_row) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    U16 o[NS];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        __nv_bfloat16 t[NS];
                        bf16_terms<NS>(__uint_as_float(r[g * 8 + e]), t);
#pragma unroll
                        for (int j = 0; j < NS; ++j) o[j].b[e] = t[j];
                    }
#pragma unroll
                    for (int j = 0; j < NS; ++j)
                        *reinterpret_cast<uint4 *>(sm + G::kS + j * G::kSTile + tile_at(D, srow, c / 8 + g)) = o[j].u;
                }
            }
        }
        if (G::kStateTmem) tmem_wait_st();
    }

    bool alive = true;
    uint32_t parity = 0;
    for (int pc = s.p0; pc < s.pe; pc += kChunk, parity ^= 1) {
        const int cnt = min(kChunk, s.pe - pc);
        const int lead = pc == 0 ? w.lead : 1;
        // operands to shared memory; the state-only walk needs K~ alone
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int idx = tid + i * 256, r = idx / (D / 8), at = tile_at(kChunk, r, idx % (D / 8));
            if (STATE_ONLY) {
                store_terms<T, NK>(sm + G::kK, G::kTile, at, rk[i], r < cnt ? w.c * dec[cnt - 1 - r] : 0.f);
            } else {
                store_terms<T, NI>(sm + G::kQ, G::kTile, at, rq[i], 1.f);
                store_terms<T, NI>(sm + G::kK, G::kTile, at, rk[i], 1.f);
            }
            store_terms<T, NI>(sm + G::kV, G::kTile, at, rv[i], 1.f);
        }
        smem_to_mma();
        tc_before_sync();
        if (__syncthreads_or(!alive)) break;

        if (!STATE_ONLY && tid == 0) {
            tc_after_sync();
            const uint32_t i1 = mma_idesc(128, 128, false, false), i2 = mma_idesc(128, nv, false, true);
            bool acc = false;
            for (int sum = NI - 1; sum >= 0; --sum)
                for (int x = 0; x <= sum; ++x)
                    for (int k = 0; k < kd; ++k) {
                        mma_ss(tm, desc_k(smem + G::kQ + x * G::kTile, kChunk, k),
                               desc_k(smem + G::kK + (sum - x) * G::kTile, kChunk, k), i1, acc);
                        acc = true;
                    }
            acc = false;
            for (int sum = NM - 1; sum >= 0; --sum)
                for (int x = 0; x <= sum && x < NI; ++x)
                    for (int k = 0; k < kd; ++k) {
                        mma_ss(tm + G::kO, desc_k(smem + G::kQ + x * G::kTile, kChunk, k),
                               desc_mn(smem + G::kS + (sum - x) * G::kSTile, D, k), i2, acc);
                        acc = true;
                    }
            mma_commit(bar1);
        }

        float qs[D / 2];
        if (!STATE_ONLY) {
            alive = mbar_wait_bounded(bar1, parity) && alive;
            __syncwarp();
            tc_after_sync();
            // K -> K~ in place
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int idx = tid + i * 256, r = idx / (D / 8), at = tile_at(kChunk, r, idx % (D / 8));
                uint4 u[NI];
#pragma unroll
                for (int j = 0; j < NI; ++j) u[j] = *reinterpret_cast<const uint4 *>(sm + G::kK + j * G::kTile + at);
                const float wk = r < cnt ? w.c * dec[cnt - 1 - r] : 0.f;
                U16 o[NK];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    __nv_bfloat16 t[NK];
                    bf16_terms<NK>(term_sum(u, e) * wk, t);
#pragma unroll
                    for (int j = 0; j < NK; ++j) o[j].b[e] = t[j];
                }
#pragma unroll
                for (int j = 0; j < NK; ++j) *reinterpret_cast<uint4 *>(sm + G::kK + j * G::kTile + at) = o[j].u;
            }
            // scores -> P: sixteen scores at a time become 8 columns of each term
            const int row = quad * 32 + lane;
#pragma unroll 1
            for (int c = half * 64; c < half * 64 + 64; c += 16) {
                uint32_t r[16], o[NM][8];
                tmem_ld16(tlane + c, r);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    __nv_bfloat16 t0[NM], t1[NM];
                    const int far = row - c - e;
                    bf16_terms<NM>(far >= 0 ? __uint_as_float(r[e]) * (pa * dec[far]) : 0.f, t0);
                    bf16_terms<NM>(far >= 1 ? __uint_as_float(r[e + 1]) * (pa * dec[far - 1]) : 0.f, t1);
#pragma unroll
                    for (int j = 0; j < NM; ++j) o[j][e / 2] = pack2(t0[j], t1[j]);
                }
#pragma unroll
                for (int j = 0; j < NM; ++j) tmem_st8(tlane + G::kP + c / 16 * (8 * NM) + j * 8, o[j]);
            }
            // q S, kept until the scores' part of o is there
#pragma unroll
            for (int c = 0; c < D / 2; c += 16) {
                uint32_t r[16];
                tmem_ld16(tlane + G::kO + half * (D / 2) + c, r);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) qs[c + e] = __uint_as_float(r[e]);
            }
            tmem_wait_st();
            smem_to_mma();
            tc_before_sync();
            __syncthreads();
        }
        if (tid == 0) {
            tc_after_sync();
            const uint32_t i3 = mma_idesc(128, nv, false, true), i4 = mma_idesc(D, nv, true, true);
            bool acc = false;
            if (!STATE_ONLY) {
                for (int sum = NM - 1; sum >= 0; --sum)
                    for (int x = 0; x <= sum; ++x) {
                        if (sum - x >= NI) continue;
                        for (int k = 0; k < kChunk / 16; ++k) {
                            mma_ts(tm + G::kO, tm + G::kP + k * (8 * NM) + x * 8,
                                   desc_mn(smem + G::kV + (sum - x) * G::kTile, kChunk, k), i3, acc);
                            acc = true;
                        }
                    }
                acc = false;
            }
            for (int sum = NK - 1; sum >= 0; --sum)
                for (int x = 0; x <= sum; ++x) {
                    if (sum - x >= NI) continue;
                    for (int k = 0; k < kChunk / 16; ++k) {
                        mma_ss(tm + G::kKV, desc_mn(smem + G::kK + x * G::kTile, kChunk, k),
                               desc_mn(smem + G::kV + (sum - x) * G::kTile, kChunk, k), i4, acc);
                        acc = true;
                    }
                }
            mma_commit(bar2);
        }
        if (pc + kChunk < s.pe) fetch(pc + kChunk);
        alive = mbar_wait_bounded(bar2, parity) && alive;
        __syncwarp();
        tc_after_sync();

        if (!STATE_ONLY) {
            const int row = quad * 32 + lane, p = pc + row;
            const float f = w.b * dec[min(row + lead, kChunk)];
            T *ob = static_cast<T *>(w.o) + s.b * w.os[0] + s.h * w.os[2] +
                    (w.reverse ? s.L - 1 - p : p) * w.os[1];
#pragma unroll
            for (int c = 0; c < D / 2; c += 16) {
                uint32_t r[16];
                tmem_ld16(tlane + G::kO + half * (D / 2) + c, r);
                tmem_wait_ld();
                const int col = half * (D / 2) + c;
                if (p < s.pe) {
                    constexpr int n = 16 / sizeof(T);
#pragma unroll
                    for (int g = 0; g < 16 / n; ++g) {
                        Pack<T, n> o;
#pragma unroll
                        for (int e = 0; e < n; ++e)
                            o.v[e] = from_f<T>(fmaf(f, qs[c + g * n + e], __uint_as_float(r[g * n + e])));
                        const int c0 = col + g * n;
                        if (w.o_vec) {
                            if (c0 < w.dv) *reinterpret_cast<Pack<T, n> *>(ob + c0) = o;
                        } else {
#pragma unroll
                            for (int e = 0; e < n; ++e)
                                if (c0 + e < w.dv) ob[c0 + e] = o.v[e];
                        }
                    }
                }
            }
        }
        // S = lam^n S + KV, and its terms for the next chunk.  The float32 rounding of
        // lam^n alone would bias a state that lives for many chunks: two parts.
        const double step = decay_pow(ld, cnt - 1 + lead);
        const float hi = (float)step, lo = (float)(step - (double)hi);
#pragma unroll 1
        for (int c = half * (D / 2); c < min((half + 1) * (D / 2), nv); c += 16) {
            uint32_t r[16], old[16];
            tmem_ld16(tlane + G::kKV + c, r);
            if (G::kStateTmem) tmem_ld16(tlane + G::kState + c, old);
            tmem_wait_ld();
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                uint4 u[NS];
                U16 o[NS];
                const int at = tile_at(D, srow, c / 8 + g);
                if (!G::kStateTmem) {
#pragma unroll
                    for (int j = 0; j < NS; ++j) u[j] = *reinterpret_cast<const uint4 *>(sm + G::kS + j * G::kSTile + at);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float prev = G::kStateTmem ? __uint_as_float(old[g * 8 + e]) : term_sum(u, e);
                    const float next = fmaf(prev, hi, fmaf(prev, lo, __uint_as_float(r[g * 8 + e])));
                    old[g * 8 + e] = __float_as_uint(next);
                    __nv_bfloat16 t[NS];
                    bf16_terms<NS>(next, t);
#pragma unroll
                    for (int j = 0; j < NS; ++j) o[j].b[e] = t[j];
                }
                if (has_row) {
#pragma unroll
                    for (int j = 0; j < NS; ++j) *reinterpret_cast<uint4 *>(sm + G::kS + j * G::kSTile + at) = o[j].u;
                }
            }
            if (G::kStateTmem) tmem_st16(tlane + G::kState + c, old);
        }
        if (G::kStateTmem) tmem_wait_st();
    }
    if (!alive && tid == 0) set_status(args.status, SEMICRF_ERR_DEVICE_TIMEOUT);

    // the state behind the last position (or behind this segment)
    const long long bh = (long long)s.b * args.H + s.h, sz = (long long)w.dk * w.dv;
    float *to = STATE_ONLY ? w.seg + (bh * args.nseg + s.seg) * sz : s.last && w.s_out ? w.s_out + bh * sz : nullptr;
    if (to) {
        const int rs = STATE_ONLY ? w.dv : w.s_rs, cs = STATE_ONLY ? 1 : w.s_cs;
        const float f = !STATE_ONLY && w.out_decay ? dec[1] : 1.f;
#pragma unroll 1
        for (int c = half * (D / 2); c < min((half + 1) * (D / 2), nv); c += 16) {
            uint32_t r[16];
            if (G::kStateTmem) {
                tmem_ld16(tlane + G::kState + c, r);
                tmem_wait_ld();
            }
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                uint4 u[NS];
                if (!G::kStateTmem) {
#pragma unroll
                    for (int j = 0; j < NS; ++j)
                        u[j] = *reinterpret_cast<const uint4 *>(sm + G::kS + j * G::kSTile + tile_at(D, srow, c / 8 + g));
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int col = c + g * 8 + e;
                    const float v = G::kStateTmem ? __uint_as_float(r[g * 8 + e]) : term_sum(u, e);
                    if (has_row && srow < w.dk && col < w.dv) to[(long long)srow * rs + (long long)col * cs] = f * v;
                }
            }
        }
    }
    tc_before_sync();
    __syncthreads();
    if (warp == 0) tmem_free(tm, G::kCols);
}

// States at the segments' starts from what each segment adds: in place, one thread an element.
__global__ void la_join_kernel(const __grid_constant__ LaArgs args)
{
    const LaWalk &w = args.w[blockIdx.z];
    const int sz = w.dk * w.dv, i = blockIdx.y * blockDim.x + threadIdx.x;
    const LaSpan s = la_span(args, blockIdx.x * args.nseg);
    if (i >= sz) return;
    const long long bh = blockIdx.x;
    float *seg = w.seg + bh * args.nseg * sz + i;
    const float ld = args.log_decay[s.h];
    float carry = w.s_in ? w.s_in[bh * sz + (long long)(i / w.dv) * w.s_rs + (long long)(i % w.dv) * w.s_cs] : 0.f;
    for (int j = 0; j < args.nseg; ++j) {
        const long long left = (long long)s.L - (long long)j * args.seg_len;
        const int len = (int)max(0LL, min(left, (long long)args.seg_len));
        const bool more = j + 1 < args.nseg && len == args.seg_len;
        const float add = more ? seg[(long long)j * sz] : 0.f;
        seg[(long long)j * sz] = carry;
        if (more) carry = (float)(decay_pow(ld, len - 1 + (j == 0 ? w.lead : 1)) * (double)carry + (double)add);
    }
}

// The walk token by token, for widths and types whose chunk tiles do not fit one SM.
// A block holds 32 of the state's columns: lane = column, warp = an eighth of the
// rows (RP registers a thread).  Inside 16 positions the state is kept relative to
// its block's start, A = sum lam^{-p} c k v^T, so that a position costs two
// multiply-adds a state element and rounding enters once in 16 positions; where
// lam^{-16} would be large (few positions remembered) the decay is applied at each position.

template <typename T, int RP, bool STATE_ONLY>
__global__ __launch_bounds__(256) void la_token_kernel(const __grid_constant__ LaArgs args, int slices)
{
    const LaWalk &w = args.w[blockIdx.y];
    const LaSpan s = la_span(args, blockIdx.x / slices);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int j0 = blockIdx.x % slices * 32, j1 = min(w.dv, j0 + 32), col = j0 + lane;
    if (j0 >= w.dv) return;
    if (STATE_ONLY && s.seg == args.nseg - 1) return;
    if (!STATE_ONLY) {
        zero_rows<T>(w, s, j0, j1);
        if (s.L == 0 && s.last) copy_state(w, args, s, j0, j1);
    }
    if (s.pe == s.p0) return;
    constexpr int DK = RP * 8, kTok = RP > 16 ? 8 : 16;   // (the tiles stay below 48 KB)
    __shared__ __align__(16) float sq[STATE_ONLY ? 1 : kTok][DK], sk[kTok][DK], sv[kTok][32];
    __shared__ float red[kTok][8][33], sg[kTok], sd[kTok];
    const float ld = args.log_decay[s.h];
    const bool far = ld * kTok < -20.f;   // lam^-16 > e^20
    const double lam1 = decay_pow(ld, 1);
    if (tid < kTok) {
        sg[tid] = far ? w.c : (float)(w.c * decay_pow(ld, -(tid + 1)));
        sd[tid] = far ? 1.f : (float)decay_pow(ld, tid + 1);
    }
    const T *qb = static_cast<const T *>(w.q) + s.b * w.qs[0] + s.h * w.qs[2];
    const T *kb = static_cast<const T *>(w.k) + s.b * w.ks[0] + s.h * w.ks[2];
    const T *vb = static_cast<const T *>(w.v) + s.b * w.vs[0] + s.h * w.vs[2];
    T *ob = static_cast<T *>(w.o) + s.b * w.os[0] + s.h * w.os[2];
    float S[RP];
    const StateAt from = STATE_ONLY ? StateAt{nullptr, 0, 0} : state_from(w, args, s);
#pragma unroll
    for (int i = 0; i < RP; ++i) {
        const int row = warp * RP + i;
        S[i] = from.p && row < w.dk && col < w.dv ? from.p[(long long)row * from.rs + (long long)col * from.cs] : 0.f;
    }
    int skip = s.seg == 0 && w.lead == 0;   // the given state's first decay is left out
    for (int pc = s.p0; pc < s.pe; pc += kTok) {
        const int cnt = min(kTok, s.pe - pc);
        __syncthreads();
        for (int i = tid; i < kTok * DK; i += 256) {
            const int r = i / DK, d = i % DK, p = pc + r;
            const long long t = w.reverse ? s.L - 1 - p : p;
            const bool in = r < cnt && d < w.dk;
            if (!STATE_ONLY) sq[r][d] = in ? to_f<T>(qb[t * w.qs[1] + d]) : 0.f;
            sk[r][d] = in ? to_f<T>(kb[t * w.ks[1] + d]) : 0.f;
        }
        for (int i = tid; i < kTok * 32; i += 256) {
            const int r = i / 32, d = j0 + i % 32, p = pc + r;
            const long long t = w.reverse ? s.L - 1 - p : p;
            sv[r][i % 32] = r < cnt && d < w.dv ? to_f<T>(vb[t * w.vs[1] + d]) : 0.f;
        }
        __syncthreads();
        if (skip && !far) {   // lam^{p} instead of lam^{p+1} for the state that was given
            const double up = decay_pow(ld, -1);
#pragma unroll
            for (int i = 0; i < RP; ++i) S[i] = (float)((double)S[i] * up);
            skip = 0;
        }
#pragma unroll 1
        for (int r = 0; r < cnt; ++r) {
            if (far) {
                if (!skip) {
#pragma unroll
                    for (int i = 0; i < RP; ++i) S[i] *= (float)lam1;
                }
                skip = 0;
            }
            const float vc = sv[r][lane] * sg[r];
            float o = 0.f;
#pragma unroll
            for (int i = 0; i < RP; i += 4) {
                const float4 k4 = *reinterpret_cast<const float4 *>(&sk[r][warp * RP + i]);
                S[i] = fmaf(k4.x, vc, S[i]);
                S[i + 1] = fmaf(k4.y, vc, S[i + 1]);
                S[i + 2] = fmaf(k4.z, vc, S[i + 2]);
                S[i + 3] = fmaf(k4.w, vc, S[i + 3]);
                if (!STATE_ONLY) {
                    const float4 q4 = *reinterpret_cast<const float4 *>(&sq[r][warp * RP + i]);
                    o = fmaf(q4.x, S[i], o);
                    o = fmaf(q4.y, S[i + 1], o);
                    o = fmaf(q4.z, S[i + 2], o);
                    o = fmaf(q4.w, S[i + 3], o);
                }
            }
            if (!STATE_ONLY) red[r][warp][lane] = o * sd[r];
        }
        if (!far) {
            const double step = decay_pow(ld, cnt);
            const float hi = (float)step, lo = (float)(step - (double)hi);
#pragma unroll
            for (int i = 0; i < RP; ++i) S[i] = fmaf(S[i], hi, S[i] * lo);
        }
        if (!STATE_ONLY) {
            __syncthreads();
            for (int i = tid; i < cnt * 32; i += 256) {
                const int r = i / 32, d = i % 32, p = pc + r;
                const long long t = w.reverse ? s.L - 1 - p : p;
                float o = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) o += red[r][j][d];
                if (j0 + d < w.dv) ob[t * w.os[1] + j0 + d] = from_f<T>(w.b * o);
            }
        }
    }
    const long long bh = (long long)s.b * args.H + s.h, sz = (long long)w.dk * w.dv;
    float *to = STATE_ONLY ? w.seg + (bh * args.nseg + s.seg) * sz : s.last && w.s_out ? w.s_out + bh * sz : nullptr;
    if (to && col < w.dv) {
        const int rs = STATE_ONLY ? w.dv : w.s_rs, cs = STATE_ONLY ? 1 : w.s_cs;
        const float f = !STATE_ONLY && w.out_decay ? (float)lam1 : 1.f;
#pragma unroll
        for (int i = 0; i < RP; ++i) {
            const int row = warp * RP + i;
            if (row < w.dk) to[(long long)row * rs + (long long)col * cs] = f * S[i];
        }
    }
}

// One token: S = lam S + k v^T in place, o = scale q S.  A block holds 32 columns of
// one head's state (lane = column, so that rows are read whole), its 8 warps share the rows.
template <typename T>
__global__ __launch_bounds__(256) void la_step_kernel(const __grid_constant__ LaStepArgs a, int slices)
{
    const int bh = blockIdx.x / slices, h = bh % a.H, b = bh / a.H;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x % slices * 32 + lane;
    const T *q = static_cast<const T *>(a.q) + b * a.qs[0] + h * a.qs[1];
    const T *k = static_cast<const T *>(a.k) + b * a.ks[0] + h * a.ks[1];
    const T *v = static_cast<const T *>(a.v) + b * a.vs[0] + h * a.vs[1];
    float *S = a.state + (long long)bh * a.dk * a.dv;
    const double lam = decay_pow(a.log_decay[h], 1);
    const float hi = (float)lam, lo = (float)(lam - (double)hi);
    const bool in = col < a.dv;
    const float vv = in ? to_f<T>(v[col]) : 0.f;
    float o = 0.f;
#pragma unroll 4
    for (int i = warp; i < a.dk; i += 8) {
        const float kk = to_f<T>(k[i]), qq = to_f<T>(q[i]);
        if (in) {
            const float s = S[(long long)i * a.dv + col];
            const float n = fmaf(s, hi, fmaf(s, lo, kk * vv));
            S[(long long)i * a.dv + col] = n;
            o = fmaf(qq, n, o);
        }
    }
    __shared__ float red[8][32];
    red[warp][lane] = o;
    __syncthreads();
    if (warp == 0 && in) {
        o = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) o += red[j][lane];
        (static_cast<T *>(a.o) + b * a.os[0] + h * a.os[1])[col] = from_f<T>(a.scale * o);
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

// Which walk serves these widths: the padded width of the chunked walk (64 or 128), or 0
// for the token walk.  Chunk tiles hold kTerms terms of q, k, v: 128 columns fit an SM's
// shared memory in one term (bf16) only.
int la_width(int dk, int dv, int dtype)
{
    const int d = dk > dv ? dk : dv;
    if (d <= 64) return 64;
    return d <= 128 && dtype == SEMICRF_BF16 ? 128 : 0;
}

template <typename T, int D, bool STATE_ONLY>
cudaError_t go_chunk(const LaArgs &a, cudaStream_t st, int *n)
{
    using G = LaCfg<T, D>;
    cudaError_t e = cudaFuncSetAttribute(la_chunk_kernel<T, D, STATE_ONLY>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         G::kSmem);
    if (e != cudaSuccess) return e;
    return timed_launch(st, n, [&] {
        la_chunk_kernel<T, D, STATE_ONLY><<<dim3(a.B * a.H * a.nseg, a.nwalk), 256, G::kSmem, st>>>(a);
    });
}

template <typename T, int RP, bool STATE_ONLY>
cudaError_t go_token(const LaArgs &a, cudaStream_t st, int *n)
{
    int dv = 0;
    for (int i = 0; i < a.nwalk; ++i) dv = a.w[i].dv > dv ? a.w[i].dv : dv;
    const int slices = (dv + 31) / 32;
    return timed_launch(st, n, [&] {
        la_token_kernel<T, RP, STATE_ONLY><<<dim3(a.B * a.H * a.nseg * slices, a.nwalk), 256, 0, st>>>(a, slices);
    });
}

template <typename T, bool STATE_ONLY>
cudaError_t go_walk(const LaArgs &a, int width, cudaStream_t st, int *n)
{
    if (width == 64) return go_chunk<T, 64, STATE_ONLY>(a, st, n);
    if constexpr (sizeof(T) == 2 && kTerms<T> == 1)
        if (width == 128) return go_chunk<T, 128, STATE_ONLY>(a, st, n);
    int dk = 0;
    for (int i = 0; i < a.nwalk; ++i) dk = a.w[i].dk > dk ? a.w[i].dk : dk;
    if (dk <= 64) return go_token<T, 8, STATE_ONLY>(a, st, n);
    if (dk <= 128) return go_token<T, 16, STATE_ONLY>(a, st, n);
    return go_token<T, 32, STATE_ONLY>(a, st, n);
}

template <typename T>
cudaError_t go(const LaArgs &a, int width, cudaStream_t st, int *n)
{
    cudaError_t e = cudaSuccess;
    if (a.nseg > 1) {
        e = go_walk<T, true>(a, width, st, n);
        if (e != cudaSuccess) return e;
        const int sz = a.w[0].dk * a.w[0].dv;
        e = timed_launch(st, n, [&] { la_join_kernel<<<dim3(a.B * a.H, (sz + 255) / 256, a.nwalk), 256, 0, st>>>(a); });
        if (e != cudaSuccess) return e;
    }
    return go_walk<T, false>(a, width, st, n);
}

template <typename T>
cudaError_t go_step(const LaStepArgs &a, cudaStream_t st, int *n)
{
    const int slices = (a.dv + 31) / 32;
    return timed_launch(st, n, [&] { la_step_kernel<T><<<a.B * a.H * slices, 256, 0, st>>>(a, slices); });
}

}  // namespace

// Segments of each sequence: one where the sequences and heads alone fill the GPU,
// else enough for two blocks an SM, of 512 positions or more.  A split walk reads K and
// V twice (once for each segment's own state).
int la_segments(int B, int T, int H, int dk, int dv, int dtype, int nwalk, int *seg_len)
{
    const int width = la_width(dk, dv, dtype);
    const long long per = width ? 1 : (dv + 31) / 32;
    const long long rows = (long long)B * H * nwalk * per, slots = 2LL * device_sm_count();
    long long n = slots / rows;
    if (n > T / 512) n = T / 512;
    if (n < 2) {
        *seg_len = (T + kChunk - 1) / kChunk * kChunk;
        return 1;
    }
    long long len = (T + n - 1) / n;
    len = (len + kChunk - 1) / kChunk * kChunk;
    *seg_len = (int)len;
    return (int)((T + len - 1) / len);
}

cudaError_t launch_la(const LaArgs &a, int dtype, cudaStream_t st, int *launches)
{
    int d = 0;
    for (int i = 0; i < a.nwalk; ++i) {
        d = a.w[i].dk > d ? a.w[i].dk : d;
        d = a.w[i].dv > d ? a.w[i].dv : d;
    }
    const int width = la_width(d, d, dtype);
    *launches = 0;
    if (dtype == SEMICRF_F32) return go<float>(a, width, st, launches);
    if (dtype == SEMICRF_BF16) return go<__nv_bfloat16>(a, width, st, launches);
    return go<__half>(a, width, st, launches);
}

cudaError_t launch_la_step(const LaStepArgs &a, int dtype, cudaStream_t st, int *launches)
{
    *launches = 0;
    if (dtype == SEMICRF_F32) return go_step<float>(a, st, launches);
    if (dtype == SEMICRF_BF16) return go_step<__nv_bfloat16>(a, st, launches);
    return go_step<__half>(a, st, launches);
}

}  // namespace semicrf
