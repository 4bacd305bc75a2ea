// linear_attention.cu -- linear attention with a decay for each head:
//   S_p = lam S_{p-1} + c k_p v_p^T,   o_p = b q_p S_p = b c sum_{j<=p} lam^{p-j} (q_p . k_j) v_j + b lam^{p+1} q_p S_in
// over whole sequences (la_chunk_kernel, la_token_kernel) and for single tokens
// (la_step_kernel).  The backward runs the same walks with exchanged operands:
//   dq = walk(dO, V, K)   dv = walk back in time(K, Q, dO)   dk = walk back in time(V, dO, Q).
#include "la_common.cuh"
#include "tensor_core.cuh"

namespace semicrf {
namespace {

template <typename T>
constexpr int kTerms = sizeof(T) == 4 ? 3 : 1;
template <>
constexpr int kTerms<__half> = 2;   // 11 bits: two bf16 terms hold them exactly

// One operand as a block walks it: element d of position p lies at at + p * step + d.
struct Track {
    unsigned char *at;
    long long step;
    int d, vec;
};

// What a block's loop needs of the arguments, in shared memory: the loop has no
// registers to spare for it, and a spilled register comes back from L2 (400 cycles:
// the tiles leave next to nothing of the L1 cache).
struct LaHot {
    Track q, k, v, o;
    float b, c;
    int lead, pe;
};

// Shapes of the chunked walk for padded width D.  Operands enter the matrix unit as
// sums of bf16 terms: NI for the inputs (exact), NM for the products P and for the
// state as an operand of q S (2: 2^-17 relative, far inside the rounding of a 16-bit
// output; 3 for float32), NK = 3 for the decayed keys, whose products make the
// float32 state.
template <typename T, int D>
struct LaCfg {
    static constexpr int NI = kTerms<T>, NM = NI == 3 ? 3 : 2, NK = 3;
    static constexpr bool kStateTmem = D == 128;   // the float32 state: tensor memory, or 16 registers a thread
    static constexpr int kCol = tile_col(kChunk), kSCol = D * 16;   // (threads write S along columns)
    static constexpr int kTile = D / 8 * kCol, kSTile = D / 8 * kSCol;
    static constexpr int kQ = 0, kK = kQ + NI * kTile, kV = kK + NK * kTile, kS = kV + NI * kTile;
    // decays lam^0 .. lam^128, and P's factors by (row - column) + 127, zero above the diagonal
    static constexpr int kDec = kS + NM * kSTile, kPf = kDec + (kChunk + 4) * 4, kMisc = kPf + 2 * kChunk * 4;
    static constexpr int kSmem = kMisc + 32 + (int)sizeof(LaHot);
    // tensor memory columns: scores (P replaces them where two terms fit the same columns), o, k v^T, state
    static constexpr int kP = NM == 3 ? 128 : 0, kO = NM == 3 ? 320 : 128, kKV = kO + D, kState = kKV + D;
    static constexpr int kCols = kState + (kStateTmem ? D : 0) <= 256 ? 256 : 512;
    static constexpr int kBlocks = kCols == 256 && kSmem <= 113 * 1024 ? 2 : 1;
    // where q S waits for the scores' part of o: scaled in its accumulator, or (float32,
    // where that costs 1e-6 to the accumulator's rounding) in registers
    static constexpr bool kKeep = NI == 3;
    static constexpr int NP = kChunk * (D / 8) / 256;   // 8-value pieces of a tile for each of 256 threads
    static constexpr int kRows = 256 / (D / 8);         // tile rows between a thread's pieces
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static_assert((NK - (NI == 3 ? 0 : NI)) * kTile >= kChunk * D * (int)sizeof(T), "room for a chunk's outputs");
};

template <typename T>
struct Piece {
    static constexpr int n = 16 / sizeof(T);
    Pack<T, n> h[8 / n];   // 8 values
    __device__ __forceinline__ float get(int i) const { return to_f<T>(h[i / n].v[i % n]); }
};

// The piece in NT bf16 terms to its place of NT tiles, times w if WEIGHTED.
template <typename T, int NT, bool WEIGHTED>
__device__ __forceinline__ void store_terms(unsigned char *at, int tile_stride, const Piece<T> &p, float w)
{
    if constexpr (kTerms<T> == 1 && NT == 1 && !WEIGHTED) {
        *reinterpret_cast<uint4 *>(at) = *reinterpret_cast<const uint4 *>(&p);
        return;
    }
    uint32_t o[NT][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t t[NT];
        split2<NT>(WEIGHTED ? p.get(2 * i) * w : p.get(2 * i), WEIGHTED ? p.get(2 * i + 1) * w : p.get(2 * i + 1), t);
#pragma unroll
        for (int j = 0; j < NT; ++j) o[j][i] = t[j];
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
        *reinterpret_cast<uint4 *>(at + j * tile_stride) = make_uint4(o[j][0], o[j][1], o[j][2], o[j][3]);
}

template <typename T>
__device__ __forceinline__ Track track_of(const void *base, const long long (&st)[3], int d, int vec, const LaSpan &s,
                                          int reverse)
{
    const T *p = static_cast<const T *>(base) + s.b * st[0] + s.h * st[2] + (reverse ? (s.L - 1) * st[1] : 0);
    return {reinterpret_cast<unsigned char *>(const_cast<T *>(p)), reverse ? -st[1] : st[1], d, vec};
}

// This thread's pieces of an operand: 8 values at column d0 of positions p, p + ROWS, ...
// of which those below `end` lie inside the sequence.  Whole pieces: loads under a
// predicate, none waits for another.
template <typename T, int NP, int ROWS>
__device__ __forceinline__ void load_pieces(const Track &g, Piece<T> (&o)[NP], int p, int end, int d0)
{
    constexpr int n = Piece<T>::n;
    const long long step = g.step;
    const int d = g.d;
    const T *src = reinterpret_cast<const T *>(g.at) + p * step + d0;
    if (g.vec) {
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
            for (int i = 0; i < 8 / n; ++i) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (p + j * ROWS < end && d0 < d) v = reinterpret_cast<const uint4 *>(src + j * ROWS * step)[i];
                *reinterpret_cast<uint4 *>(&o[j].h[i]) = v;
            }
    } else {
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                T v = from_f<T>(0.f);
                if (p + j * ROWS < end && d0 + i < d) v = src[j * ROWS * step + i];
                o[j].h[i / n].v[i % n] = v;
            }
    }
}

// bf16 operands need no conversion: whole pieces go from global to shared memory on
// their own (to be waited for with cp_async_wait), others by way of registers.
template <typename T, int NP, int ROWS>
__device__ __forceinline__ void bring_pieces(const Track &g, unsigned char *to, int p, int end, int d0)
{
    if (g.vec) {
        const long long step = g.step;
        const T *src = reinterpret_cast<const T *>(g.at) + p * step + d0;
        const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(to));
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            const bool in = p + j * ROWS < end && d0 < g.d;
            const void *from = in ? static_cast<const void *>(src + j * ROWS * step) : g.at;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + j * ROWS * 16), "l"(from),
                         "r"(in ? 16 : 0)
                         : "memory");
        }
    } else {
#pragma unroll 1
        for (int j = 0; j < NP; ++j) {
            Piece<T> o[1];
            load_pieces<T, 1, ROWS>(g, o, p + j * ROWS, end, d0);
            *reinterpret_cast<uint4 *>(to + j * ROWS * 16) = *reinterpret_cast<const uint4 *>(&o[0]);
        }
    }
}

// The chunked walk: 128 positions at a time,
//   scores = Q K^T and Q S                              (tensor memory)
//   K~ = c lam^{end-j} K,  P = b c lam^{i-j} scores     (threads; P to tensor memory, K~ over K)
//   KV = K~^T V (while P is formed),  o = b lam^{i+1} (Q S) + P V
//   S = lam^n S + KV                                    (threads, float32)
// The matrix unit's accumulators round towards zero (measured: -1.4e-7 relative for
// each 8 steps of 16), which a state carried in them over thousands of chunks would
// show; so they hold one chunk's sums only, small terms first, and the state is
// advanced by float32 multiply-adds to nearest.
template <typename T, int D, bool STATE_ONLY>
__global__ __launch_bounds__(256, (LaCfg<T, D>::kBlocks)) void la_chunk_kernel(const __grid_constant__ LaArgs args)
{
    using G = LaCfg<T, D>;
    constexpr int NI = G::NI, NM = G::NM, NK = G::NK, NP = G::NP;
    // steps of 16 values of a contraction, and of one tile, in a descriptor's units
    constexpr uint64_t kCol2 = 2 * G::kCol >> 4, kRow2 = 2 * 128 >> 4, 
                       kTileD = G::kTile >> 4, kSTileD = G::kSTile >> 4;
    extern __shared__ __align__(128) unsigned char sm[];
    const LaWalk &w = args.w[blockIdx.y];
    const LaSpan s = la_span(args, blockIdx.x);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int quad = warp & 3, half = warp >> 2;
    if (STATE_ONLY && s.seg == args.nseg - 1) return;
    if (!STATE_ONLY) {
        zero_rows<T>(w, s, 0, w.dv);
        if (s.L == 0 && s.last) copy_state(w, args, s, 0, w.dv);
    }
    if (s.pe == s.p0) return;

    float *dec = reinterpret_cast<float *>(sm + G::kDec), *pf = reinterpret_cast<float *>(sm + G::kPf);
    float *full = reinterpret_cast<float *>(sm + G::kMisc + 24);   // lam^128 in two floats
    LaHot &hot = *reinterpret_cast<LaHot *>(sm + G::kMisc + 32);
    uint32_t *slot = reinterpret_cast<uint32_t *>(sm + G::kMisc + 16);
    const uint32_t smem = static_cast<uint32_t>(__cvta_generic_to_shared(sm));
    const uint32_t bar1 = smem + G::kMisc, bar2 = bar1 + 8;
    const float ld = args.log_decay[s.h];
    if (warp == 0) tmem_alloc(static_cast<uint32_t>(__cvta_generic_to_shared(slot)), G::kCols);
    if (tid == 0) {
        mbar_init(bar1, 1);
        mbar_init(bar2, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid <= kChunk) {
        const double v = decay_pow(ld, tid);
        dec[tid] = (float)v;
        if (tid < kChunk) {
            pf[kChunk - 1 + tid] = (float)(v * (double)(w.b * w.c));
        } else {
            full[0] = (float)v;
            full[1] = (float)(v - (double)full[0]);
        }
    } else {
        pf[tid - kChunk - 1] = 0.f;   // 127 entries
    }

    const int r0 = tid / (D / 8), d8 = tid % (D / 8), at0 = d8 * G::kCol + r0 * 16;
    if (tid == 0) {
        hot.q = track_of<T>(w.q, w.qs, w.dk, w.q_vec, s, w.reverse);
        hot.k = track_of<T>(w.k, w.ks, w.dk, w.k_vec, s, w.reverse);
        hot.v = track_of<T>(w.v, w.vs, w.dv, w.v_vec, s, w.reverse);
        hot.o = track_of<T>(w.o, w.os, w.dv, w.o_vec, s, w.reverse);
        hot.b = w.b;
        hot.c = w.c;
        hot.lead = w.lead;
        hot.pe = s.pe;
    }
    __syncthreads();
    const int pe = s.pe;
    // float32 and float16 are prefetched in registers and split on their way to shared
    // memory; the state-only walk weights its keys there
    constexpr bool kDirect = NI == 1 && !STATE_ONLY;
    Piece<T> rk[kDirect ? 1 : NP], rv[kDirect ? 1 : NP];
    auto fetch = [&](const Track &g, Piece<T> (&to)[NP], int pc) {
        load_pieces<T, NP, G::kRows>(g, to, pc + r0, hot.pe, d8 * 8);
    };
    auto bring = [&](const Track &g, int tile, int pc) {
        bring_pieces<T, NP, G::kRows>(g, sm + tile + at0, pc + r0, hot.pe, d8 * 8);
    };

    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tm = __shfl_sync(0xffffffffu, *slot, 0), tlane = tm + ((uint32_t)(quad * 32) << 16);
    const int nv = (w.dv + 15) / 16 * 16, kd = (w.dk + 15) / 16, c0 = half * (D / 2);

    // The state.  D = 64: rows quad * 16 + lane / 4 (+ 8), column pairs c0 + 8 j + 2 (lane % 4)
    // in registers; D = 128: row quad * 32 + lane, columns c0 .. c0 + 63 in tensor memory.
    float S[G::kStateTmem ? 1 : 16];
    const StateAt from = STATE_ONLY ? StateAt{nullptr, 0, 0} : state_from(w, args, s);
    auto given = [&](int row, int col) {
        return from.p && row < w.dk && col < w.dv ? from.p[(long long)row * from.rs + (long long)col * from.cs] : 0.f;
    };
    auto put_pairs = [&] {   // D = 64: the terms of S to shared memory
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                uint32_t t[NM];
                split2<NM>(S[4 * j + 2 * a], S[4 * j + 2 * a + 1], t);
                unsigned char *to = sm + G::kS + (half * 4 + j) * G::kSCol + (quad * 16 + (lane >> 2) + 8 * a) * 16 + 4 * (lane & 3);
#pragma unroll
                for (int x = 0; x < NM; ++x) *reinterpret_cast<uint32_t *>(to + x * G::kSTile) = t[x];
            }
    };
    auto put_row = [&](int c, const uint32_t (&r)[16]) {   // D = 128: 16 columns of this thread's row
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            uint32_t o[NM][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t t[NM];
                split2<NM>(__uint_as_float(r[8 * g + 2 * e]), __uint_as_float(r[8 * g + 2 * e + 1]), t);
#pragma unroll
                for (int x = 0; x < NM; ++x) o[x][e] = t[x];
            }
#pragma unroll
            for (int x = 0; x < NM; ++x)
                *reinterpret_cast<uint4 *>(sm + G::kS + x * G::kSTile + (c / 8 + g) * G::kSCol + (quad * 32 + lane) * 16) =
                    make_uint4(o[x][0], o[x][1], o[x][2], o[x][3]);
        }
    };
    if constexpr (G::kStateTmem) {
#pragma unroll 1
        for (int c = c0; c < c0 + D / 2; c += 16) {
            uint32_t r[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(given(quad * 32 + lane, c + e));
            tmem_st16(tlane + G::kState + c, r);
            put_row(c, r);
        }
        tmem_wait_st();
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            S[i] = given(quad * 16 + (lane >> 2) + (i & 2) * 4, c0 + (i >> 2) * 8 + (lane & 3) * 2 + (i & 1));
        put_pairs();
    }

    if constexpr (kDirect) {
        bring(hot.q, G::kQ, s.p0);
        bring(hot.k, G::kK, s.p0);
        bring(hot.v, G::kV, s.p0);
    } else {
        if (!STATE_ONLY) {
            Piece<T> rq[NP];
            fetch(hot.q, rq, s.p0);
#pragma unroll
            for (int i = 0; i < NP; ++i)
                store_terms<T, NI, false>(sm + G::kQ + at0 + i * G::kRows * 16, G::kTile, rq[i], 1.f);
        }
        fetch(hot.k, rk, s.p0);
        fetch(hot.v, rv, s.p0);
    }

    bool alive = true;
    uint32_t parity = 0;
    for (int pc = s.p0; pc < pe; pc += kChunk, parity ^= 1) {
        const int cnt = min(kChunk, pe - pc);
        const int lead = pc == 0 ? hot.lead : 1;
        const bool more = pc + kChunk < pe;
        if constexpr (kDirect) {
            cp_async_commit();
            cp_async_wait<0>();
        } else {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int r = r0 + i * G::kRows, at = at0 + i * G::kRows * 16;
                if (STATE_ONLY)
                    store_terms<T, NK, true>(sm + G::kK + at, G::kTile, rk[i], r < cnt ? hot.c * dec[cnt - 1 - r] : 0.f);
                else
                    store_terms<T, NI, false>(sm + G::kK + at, G::kTile, rk[i], 1.f);
                store_terms<T, NI, false>(sm + G::kV + at, G::kTile, rv[i], 1.f);
            }
        }
        smem_to_mma();
        tc_before_sync();
        if (__syncthreads_or(!alive)) break;

        if (!STATE_ONLY) {
            if (warp == 0 && elect_lane()) {
                tc_after_sync();
                const uint32_t i1 = mma_idesc(128, 128, false, false), i2 = mma_idesc(128, nv, false, true);
                const uint64_t dq = desc_k(smem + G::kQ, G::kCol), dk = desc_k(smem + G::kK, G::kCol);
                const uint64_t ds = desc_mn(smem + G::kS, G::kSCol);
                mma_terms<NI, NI, NI>([&](int x, int y, bool acc) {
#pragma unroll 1
                    for (int k = 0; k < kd; ++k, acc = true)
                        mma_ss(tm, dq + x * kTileD + k * kCol2, dk + y * kTileD + k * kCol2, i1, acc);
                });
                mma_terms<NI, NM, NM>([&](int x, int y, bool acc) {
#pragma unroll 1
                    for (int k = 0; k < kd; ++k, acc = true)
                        mma_ss(tm + G::kO, dq + x * kTileD + k * kCol2, ds + y * kSTileD + k * kRow2, i2, acc);
                });
                mma_commit(bar1);
            }
            // the next queries travel while the scores are formed; then their tile is free
            Piece<T> rq[kDirect ? 1 : NP];
            if constexpr (!kDirect)
                if (more) fetch(hot.q, rq, pc + kChunk);
            alive = mbar_wait_bounded(bar1, parity) && alive;
            __syncwarp();
            tc_after_sync();
            if (more) {
                if constexpr (kDirect) {
                    bring(hot.q, G::kQ, pc + kChunk);
                } else {
#pragma unroll
                    for (int i = 0; i < NP; ++i)
                        store_terms<T, NI, false>(sm + G::kQ + at0 + i * G::kRows * 16, G::kTile, rq[i], 1.f);
                }
            }
            // K -> K~ in place
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int r = r0 + i * G::kRows;
                unsigned char *at = sm + G::kK + at0 + i * G::kRows * 16;
                const float wk = r < cnt ? hot.c * dec[cnt - 1 - r] : 0.f;
                uint4 u[NI];
#pragma unroll
                for (int j = 0; j < NI; ++j) u[j] = *reinterpret_cast<const uint4 *>(at + j * G::kTile);
                uint32_t o[NK][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t t[NI], n[NK];
#pragma unroll
                    for (int j = 0; j < NI; ++j) t[j] = reinterpret_cast<const uint32_t *>(&u[j])[e];
                    float x, y;
                    join2<NI>(t, x, y);
                    split2<NK>(x * wk, y * wk, n);
#pragma unroll
                    for (int j = 0; j < NK; ++j) o[j][e] = n[j];
                }
#pragma unroll
                for (int j = 0; j < NK; ++j)
                    *reinterpret_cast<uint4 *>(at + j * G::kTile) = make_uint4(o[j][0], o[j][1], o[j][2], o[j][3]);
            }
            smem_to_mma();
            __syncthreads();
        }
        if (warp == 0 && elect_lane()) {
            tc_after_sync();
            const uint32_t i4 = mma_idesc(D, nv, true, true);
            const uint64_t dk = desc_mn(smem + G::kK, G::kCol), dv = desc_mn(smem + G::kV, G::kCol);
            mma_terms<NK, NI, NK>([&](int x, int y, bool acc) {
#pragma unroll 1
                for (int k = 0; k < kChunk / 16; ++k, acc = true)
                    mma_ss(tm + G::kKV, dk + x * kTileD + k * kRow2, dv + y * kTileD + k * kRow2, i4, acc);
            });
            if (STATE_ONLY) mma_commit(bar2);
        }
        float qs[!STATE_ONLY && G::kKeep ? D / 2 : 1];
        if (!STATE_ONLY) {
            // scores -> P: 32 scores at a time become 16 columns of each term
            const int row = quad * 32 + lane;
#pragma unroll 1
            for (int c = half * 64; c < half * 64 + 64; c += 32) {
                uint32_t r[32];
                if (c <= quad * 32 + 31) {   // some row of this warp reaches these keys
                    tmem_ld32(tlane + c, r);
                    tmem_wait_ld();
                    const float *f = pf + (kChunk - 1) + row - c;
#pragma unroll
                    for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f[-e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) r[e] = 0;
                }
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    uint32_t o[NM][8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        uint32_t t[NM];
                        split2<NM>(__uint_as_float(r[16 * g + 2 * e]), __uint_as_float(r[16 * g + 2 * e + 1]), t);
#pragma unroll
                        for (int j = 0; j < NM; ++j) o[j][e] = t[j];
                    }
#pragma unroll
                    for (int j = 0; j < NM; ++j) tmem_st8(tlane + G::kP + (c / 16 + g) * (8 * NM) + j * 8, o[j]);
                }
            }
            // o starts as b lam^{i+1} q S
            const float f = hot.b * dec[row + lead];
#pragma unroll
            for (int c = 0; c < D / 2; c += 16) {
                uint32_t r[16];
                tmem_ld16(tlane + G::kO + c0 + c, r);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
                if constexpr (G::kKeep) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) qs[c + e] = __uint_as_float(r[e]);
                } else {
                    tmem_st16(tlane + G::kO + c0 + c, r);
                }
            }
            tmem_wait_st();
            tc_before_sync();
            __syncthreads();
            if (warp == 0 && elect_lane()) {
                tc_after_sync();
                const uint32_t i3 = mma_idesc(128, nv, false, true);
                const uint64_t dv = desc_mn(smem + G::kV, G::kCol);
                mma_terms<NM, NI, NM>([&](int x, int y, bool acc) {
                    acc |= !G::kKeep;
#pragma unroll 1
                    for (int k = 0; k < kChunk / 16; ++k, acc = true)
                        mma_ts(tm + G::kO, tm + G::kP + k * (8 * NM) + x * 8, dv + y * kTileD + k * kRow2, i3, acc);
                });
                mma_commit(bar2);
            }
        }
        if constexpr (!kDirect)
            if (more) {
                fetch(hot.k, rk, pc + kChunk);
                fetch(hot.v, rv, pc + kChunk);
            }
        alive = mbar_wait_bounded(bar2, parity) && alive;
        __syncwarp();
        tc_after_sync();
        if constexpr (kDirect)
            if (more) {   // (the outputs below use the parts of K~ behind the keys' own tile)
                bring(hot.k, G::kK, pc + kChunk);
                bring(hot.v, G::kV, pc + kChunk);
            }

        if (!STATE_ONLY) {
            // rows to shared memory (the part of K~'s tiles that the next keys leave
            // alone), then whole rows to global memory; 16-byte pieces of a row are
            // exchanged by the row's number so that neither side meets bank conflicts
            constexpr int n = 16 / sizeof(T), W = D / n;   // values of a piece, pieces of a row
            unsigned char *ob = sm + G::kK + (NI == 3 ? 0 : NI * G::kTile);
            const int row = quad * 32 + lane;
#pragma unroll
            for (int c = 0; c < D / 2; c += 16) {
                uint32_t r[16];
                tmem_ld16(tlane + G::kO + c0 + c, r);
                tmem_wait_ld();
#pragma unroll
                for (int g = 0; g < 16 / n; ++g) {
                    Pack<T, n> o;
#pragma unroll
                    for (int e = 0; e < n; ++e)
                        o.v[e] = from_f<T>(__uint_as_float(r[g * n + e]) + (G::kKeep ? qs[G::kKeep ? c + g * n + e : 0] : 0.f));
                    *reinterpret_cast<Pack<T, n> *>(ob + (row * W + (((c0 + c) / n + g) ^ (row & 7))) * 16) = o;
                }
            }
            asm volatile("bar.sync %0, 64;" ::"r"(1 + quad) : "memory");   // the two halves of these 32 rows
            const Track to = hot.o;
            T *og = reinterpret_cast<T *>(to.at) + pc * to.step;
#pragma unroll
            for (int j = 0; j < W / 2; ++j) {
                const int i = j * 64 + half * 32 + lane, rr = quad * 32 + i / W, piece = i % W, col = piece * n;
                if (pc + rr >= hot.pe || col >= to.d) continue;
                const Pack<T, n> o = *reinterpret_cast<const Pack<T, n> *>(ob + (rr * W + (piece ^ (rr & 7))) * 16);
                T *at = og + rr * to.step + col;
                if (to.vec) {
                    *reinterpret_cast<Pack<T, n> *>(at) = o;
                } else {
#pragma unroll
                    for (int e = 0; e < n; ++e)
                        if (col + e < to.d) at[e] = o.v[e];
                }
            }
            if (NI == 3) __syncthreads();   // the next keys go where these rows were
        }
        // S = lam^n S + KV, and its terms for the next chunk.  The float32 rounding of
        // lam^n alone would bias a state that lives for many chunks: two parts.
        float hi = full[0], lo = full[1];
        if (cnt - 1 + lead != kChunk) {
            const double step = decay_pow(ld, cnt - 1 + lead);
            hi = (float)step;
            lo = (float)(step - (double)hi);
        }
        if constexpr (G::kStateTmem) {
#pragma unroll 1
            for (int c = c0; c < min(c0 + D / 2, nv); c += 16) {
                uint32_t r[16], old[16];
                tmem_ld16(tlane + G::kKV + c, r);
                tmem_ld16(tlane + G::kState + c, old);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float prev = __uint_as_float(old[e]);
                    old[e] = __float_as_uint(fmaf(prev, hi, fmaf(prev, lo, __uint_as_float(r[e]))));
                }
                tmem_st16(tlane + G::kState + c, old);
                if (!STATE_ONLY) put_row(c, old);
            }
            tmem_wait_st();
        } else {
            uint32_t r[16];
            tmem_ld16x256(tlane + G::kKV + c0, r);
            tmem_wait_ld();
            // (columns from nv on are not computed: their values stay out of every result)
#pragma unroll
            for (int i = 0; i < 16; ++i) S[i] = fmaf(S[i], hi, fmaf(S[i], lo, __uint_as_float(r[i])));
            if (!STATE_ONLY) put_pairs();
        }
    }
    if (!alive && tid == 0) set_status(args.status, SEMICRF_ERR_DEVICE_TIMEOUT);

    // the state behind the last position (or behind this segment)
    const long long bh = (long long)s.b * args.H + s.h, sz = (long long)w.dk * w.dv;
    float *to = STATE_ONLY ? w.seg + (bh * args.nseg + s.seg) * sz : s.last && w.s_out ? w.s_out + bh * sz : nullptr;
    if (to) {
        const int rs = STATE_ONLY ? w.dv : w.s_rs, cs = STATE_ONLY ? 1 : w.s_cs;
        const float f = !STATE_ONLY && w.out_decay ? dec[1] : 1.f;
        auto keep = [&](int row, int col, float v) {
            if (row < w.dk && col < w.dv) to[(long long)row * rs + (long long)col * cs] = f * v;
        };
        if constexpr (G::kStateTmem) {
#pragma unroll 1
            for (int c = c0; c < min(c0 + D / 2, nv); c += 16) {
                uint32_t r[16];
                tmem_ld16(tlane + G::kState + c, r);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) keep(quad * 32 + lane, c + e, __uint_as_float(r[e]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                keep(quad * 16 + (lane >> 2) + (i & 2) * 4, c0 + (i >> 2) * 8 + (lane & 3) * 2 + (i & 1), S[i]);
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
    const int sz = w.dk * w.dv, i = blockIdx.y * blockDim.x + threadIdx.x, nseg = args.nseg;
    const LaSpan s = la_span(args, blockIdx.x * nseg);
    __shared__ double power[2];   // of a whole segment: the first one, the others
    if (threadIdx.x < 2)
        power[threadIdx.x] = decay_pow(args.log_decay[s.h], args.seg_len - 1 + (threadIdx.x ? 1 : w.lead));
    __syncthreads();
    if (i >= sz) return;
    const long long bh = blockIdx.x;
    float *seg = w.seg + bh * nseg * sz + i;
    // segments before the last one that are whole: their sums exist
    const int whole = min(nseg - 1, s.L / args.seg_len);
    float carry = w.s_in ? w.s_in[bh * sz + (long long)(i / w.dv) * w.s_rs + (long long)(i % w.dv) * w.s_cs] : 0.f;
    constexpr int U = 8;   // loads in flight
    for (int j0 = 0; j0 <= whole; j0 += U) {
        float add[U];
#pragma unroll
        for (int u = 0; u < U; ++u) add[u] = j0 + u < whole ? seg[(long long)(j0 + u) * sz] : 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j0 + u > whole) break;
            seg[(long long)(j0 + u) * sz] = carry;
            carry = (float)(power[j0 + u > 0] * (double)carry + (double)add[u]);
        }
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

// One token: S = lam S + k v^T in place, o = scale q S.  Bound by the state, read and
// written once: VEC columns a lane, `lanes` lanes a row, the rows shared by 8 warps with
// four loads of each thread in flight.
template <typename T, int VEC>
__global__ __launch_bounds__(256) void la_step_kernel(const __grid_constant__ LaStepArgs a, int slices, int lanes)
{
    const int bh = blockIdx.x / slices, h = bh % a.H, b = bh / a.H, tid = threadIdx.x;
    const int lane = tid & 31, warp = tid >> 5, sub = lane / lanes, rows = 8 * (32 / lanes);
    const int first = blockIdx.x % slices * lanes * VEC, col = first + lane % lanes * VEC;
    __shared__ float sq[SEMICRF_MAX_HEAD], sk[SEMICRF_MAX_HEAD], red[8][32 * VEC];
    for (int i = tid; i < a.dk; i += 256) {
        sq[i] = to_f<T>((static_cast<const T *>(a.q) + b * a.qs[0] + h * a.qs[1])[i]);
        sk[i] = to_f<T>((static_cast<const T *>(a.k) + b * a.ks[0] + h * a.ks[1])[i]);
    }
    const T *v = static_cast<const T *>(a.v) + b * a.vs[0] + h * a.vs[1];
    float *S = a.state + (long long)bh * a.dk * a.dv + col;
    const double lam = decay_pow(a.log_decay[h], 1);
    const float hi = (float)lam, lo = (float)(lam - (double)hi);
    const bool in = col < a.dv;   // (VEC divides dv)
    float vv[VEC], o[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        vv[e] = in ? to_f<T>(v[col + e]) : 0.f;
        o[e] = 0.f;
    }
    __syncthreads();
    if (in) {
        constexpr int U = 4;
        for (int i0 = warp * (32 / lanes) + sub; i0 < a.dk; i0 += U * rows) {
            Pack<float, VEC> s[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u * rows < a.dk)
                    s[u] = *reinterpret_cast<const Pack<float, VEC> *>(S + (long long)(i0 + u * rows) * a.dv);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * rows;
                if (i >= a.dk) break;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    s[u].v[e] = fmaf(s[u].v[e], hi, fmaf(s[u].v[e], lo, sk[i] * vv[e]));
                    o[e] = fmaf(sq[i], s[u].v[e], o[e]);
                }
                *reinterpret_cast<Pack<float, VEC> *>(S + (long long)i * a.dv) = s[u];
            }
        }
    }
    // the row lanes' shares: red[warp][lane][e]
#pragma unroll
    for (int e = 0; e < VEC; ++e) red[warp][lane * VEC + e] = o[e];
    __syncthreads();
    if (tid < lanes * VEC && first + tid < a.dv) {
        float sum = 0.f;
        for (int w = 0; w < 8; ++w)
            for (int j = 0; j < 32 / lanes; ++j) sum += red[w][j * lanes * VEC + tid];
        (static_cast<T *>(a.o) + b * a.os[0] + h * a.os[1])[first + tid] = from_f<T>(a.scale * sum);
    }
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
    if constexpr (sizeof(T) == 2 && kTerms<T> == 1) {
        cudaError_t e;
        if (width && la_tma_walk(a, width, STATE_ONLY, st, n, &e)) return e;
    }
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

template <typename T, int VEC>
cudaError_t go_step(const LaStepArgs &a, cudaStream_t st, int *n)
{
    int lanes = 1;   // of one row: a power of two, 32 at most
    while (lanes < 32 && lanes * VEC < a.dv) lanes *= 2;
    const int slices = (a.dv + lanes * VEC - 1) / (lanes * VEC);
    return timed_launch(st, n, [&] { la_step_kernel<T, VEC><<<a.B * a.H * slices, 256, 0, st>>>(a, slices, lanes); });
}

template <typename T>
cudaError_t step_type(const LaStepArgs &a, cudaStream_t st, int *n)
{
    const bool wide = a.dv % 4 == 0 && reinterpret_cast<uintptr_t>(a.state) % 16 == 0;
    return wide ? go_step<T, 4>(a, st, n) : go_step<T, 1>(a, st, n);
}

}  // namespace

// Segments of each sequence, which walk side by side: a split walk first forms what each
// segment adds to the state (K and V read twice), so it pays where the sequences and
// heads leave most of the GPU idle.  Blocks that share an SM (two at width 64 in bf16)
// take 4.6 us a chunk and 1.8 us for the state alone, one by itself 3.2 us: three
// segments are the fewest that gain (100 000 positions of 8 heads: 151 us in 36 segments,
// 209 us in 18; 4000 positions of 128 heads: 115 us in two, 102 us in one).  One block an
// SM elsewhere (4.6 and 3.0 us a chunk at width 128): two gain.
int la_segments(int B, int T, int H, int dk, int dv, int dtype, int nwalk, int *seg_len)
{
    const int width = la_width(dk, dv, dtype);
    const bool shared = width == 0 || (width == 64 && dtype == SEMICRF_BF16);
    const long long rows = (long long)B * H * nwalk * (width ? 1 : (dv + 31) / 32);
    long long n = (shared ? 2LL : 1LL) * device_sm_count() / rows;
    if (n > T / 512) n = T / 512;
    if (n < (shared ? 3 : 2)) {
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
    if (dtype == SEMICRF_F32) return step_type<float>(a, st, launches);
    if (dtype == SEMICRF_BF16) return step_type<__nv_bfloat16>(a, st, launches);
    return step_type<__half>(a, st, launches);
}

}  // namespace semicrf
