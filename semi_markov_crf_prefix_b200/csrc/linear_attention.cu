// linear_attention.cu -- linear attention with a decay for each head:
//   S_p = lam S_{p-1} + c k_p v_p^T,   o_p = b q_p S_p = b c sum_{j<=p} lam^{p-j} (q_p . k_j) v_j + b lam^{p+1} q_p S_in
// over whole sequences (la_chunk_kernel; la_tma_kernel for bf16 that the copy engine can
// address) and for single tokens (la_step_kernel).  The backward runs the same walks with exchanged operands:
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
    Track q, k, v, o, part;
    float b, c;
    int lead, pe, adds, final;
};

// Shapes of the chunked walk.  Tiles are 64 wide: wider heads are sums over blocks of
// the contraction (o is linear in the scores, and the state's rows are independent), a
// launch each, and slices of the values' columns, which are independent.  Operands
// enter the matrix unit as sums of bf16 terms: NI for the inputs (exact), NM for the
// products P and for the state as an operand of q S (2: 2^-17 relative, far inside the
// rounding of a 16-bit output, 2^-11 at best; 3 for float32), NK = 3 for the decayed keys,
// whose products make the float32 state.
constexpr int D = 64;

template <typename T>
struct LaCfg {
    static constexpr int NI = kTerms<T>, NM = NI == 3 ? 3 : 2, NK = 3;
    static constexpr int kCol = tile_col(kChunk), kSCol = D * 16;   // (threads write S along columns)
    static constexpr int kTile = D / 8 * kCol, kSTile = D / 8 * kSCol;
    static constexpr int kQ = 0, kK = kQ + NI * kTile, kV = kK + NK * kTile, kS = kV + NI * kTile;
    // decays lam^0 .. lam^128, and P's factors by (row - column) + 127, zero above the diagonal
    static constexpr int kDec = kS + NM * kSTile, kPf = kDec + (kChunk + 4) * 4, kMisc = kPf + 2 * kChunk * 4;
    static constexpr int kSmem = kMisc + 32 + (int)sizeof(LaHot);
    // tensor memory columns: scores (P replaces them where two terms fit the same columns), o, k v^T
    static constexpr int kP = NM == 3 ? 128 : 0, kO = NM == 3 ? 320 : 128, kKV = kO + D;
    static constexpr int kCols = kKV + D <= 256 ? 256 : 512;
    static constexpr int kBlocks = kCols == 256 && kSmem <= 113 * 1024 ? 2 : 1;
    // where q S waits for the scores' part of o: scaled in its accumulator, or (float32,
    // where that costs 1e-6 to the accumulator's rounding) in registers
    static constexpr bool kKeep = NI == 3;
    static constexpr int NP = kChunk * (D / 8) / 256;   // 8-value pieces of a tile for each of 256 threads
    static constexpr int kRows = 256 / (D / 8);         // tile rows between a thread's pieces
    // a chunk's outputs on their way, in float32: in K~'s tiles, behind the one that the next keys of
    // bf16 go to at once
    static constexpr int kOut = kK + (NI == 1 ? kTile : 0);
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static_assert(kK + NK * kTile - kOut >= kChunk * D * 4, "room for a chunk's outputs");
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
__device__ __forceinline__ Track track_of(const void *base, const long long (&st)[3], int from, int d, int vec,
                                          const LaSpan &s, int reverse)
{
    const T *p = static_cast<const T *>(base) + s.b * st[0] + s.h * st[2] + (reverse ? (s.L - 1) * st[1] : 0) + from;
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
// Measured (16 x 4000 positions, 8 heads of 64): float32 264 us of 80 at the copy rate,
// float16 204 of 40; backward 768 and 591.  One block an SM; bound by the six products a term pair asks for in
// float32 (144 matrix instructions a chunk, 5500 cycles at shared memory's rate of 128
// bytes a cycle, issued from one of the computing warps) and by splitting and staging
// between them.  32 sentences of 512 positions and 4 heads: 39 us, four chunks in a row.
template <typename T, bool STATE_ONLY>
__global__ __launch_bounds__(256, (LaCfg<T>::kBlocks)) void la_chunk_kernel(const __grid_constant__ LaArgs args)
{
    using G = LaCfg<T>;
    constexpr int NI = G::NI, NM = G::NM, NK = G::NK, NP = G::NP;
    // steps of 16 values of a contraction, and of one tile, in a descriptor's units
    constexpr uint64_t kCol2 = 2 * G::kCol >> 4, kRow2 = 2 * 128 >> 4, 
                       kTileD = G::kTile >> 4, kSTileD = G::kSTile >> 4;
    extern __shared__ __align__(128) unsigned char sm[];
    const LaWalk &w = args.w[blockIdx.y];
    const LaSpan s = la_span(args, w, blockIdx.x);
    if (s.dk <= 0 || s.dv <= 0) return;
    const bool final = s.d0 + s.dk == w.dk;   // this launch completes the sums of o
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int quad = warp & 3, half = warp >> 2;
    if (STATE_ONLY && s.seg == args.nseg - 1) return;
    if (!STATE_ONLY) {
        if (final) zero_rows<T>(w, s);
        if (s.L == 0 && s.last) copy_state(w, args, s);
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
        hot.q = track_of<T>(w.q, w.qs, s.d0, s.dk, w.q_vec, s, w.reverse);
        hot.k = track_of<T>(w.k, w.ks, s.d0, s.dk, w.k_vec, s, w.reverse);
        hot.v = track_of<T>(w.v, w.vs, s.j0, s.dv, w.v_vec, s, w.reverse);
        hot.o = track_of<T>(w.o, w.os, s.j0, s.dv, w.o_vec, s, w.reverse);
        // sums over the contraction's first blocks: in o itself where that is float32
        const long long ps[3] = {(long long)args.T * args.H * w.dv, (long long)args.H * w.dv, w.dv};
        hot.part = sizeof(T) == 4 ? hot.o : track_of<float>(w.part, ps, s.j0, s.dv, w.dv % 4 == 0, s, w.reverse);
        hot.adds = s.d0 > 0;
        hot.final = final;
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
    const int nv = (s.dv + 15) / 16 * 16, kd = (s.dk + 15) / 16, c0 = half * (D / 2);

    // the state: rows quad * 16 + lane / 4 (+ 8), column pairs c0 + 8 j + 2 (lane % 4)
    float S[16];
    const StateAt from = STATE_ONLY ? StateAt{nullptr, 0, 0} : state_from(w, args, s);
    auto given = [&](int row, int col) {
        return from.p && row < s.dk && col < s.dv ? from.p[(long long)row * from.rs + (long long)col * from.cs] : 0.f;
    };
    auto put_pairs = [&] {   // its terms to shared memory
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
#pragma unroll
    for (int i = 0; i < 16; ++i)
        S[i] = given(quad * 16 + (lane >> 2) + (i & 2) * 4, c0 + (i >> 2) * 8 + (lane & 3) * 2 + (i & 1));
    put_pairs();

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
            // rows to shared memory, then whole rows to global memory; 16-byte pieces of a
            // row are exchanged by the row's number so that neither side meets bank conflicts
            constexpr int W = D / 4;   // pieces of a row
            unsigned char *ob = sm + G::kOut;
            const int row = quad * 32 + lane;
#pragma unroll
            for (int c = 0; c < D / 2; c += 16) {
                uint32_t r[16];
                tmem_ld16(tlane + G::kO + c0 + c, r);
                tmem_wait_ld();
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[e] = __uint_as_float(r[g * 4 + e]) + (G::kKeep ? qs[G::kKeep ? c + g * 4 + e : 0] : 0.f);
                    *reinterpret_cast<float4 *>(ob + (row * W + (((c0 + c) / 4 + g) ^ (row & 7))) * 16) =
                        make_float4(o[0], o[1], o[2], o[3]);
                }
            }
            asm volatile("bar.sync %0, 64;" ::"r"(1 + quad) : "memory");   // the two halves of these 32 rows
            const Track to = hot.o, part = hot.part;
            const bool adds = hot.adds, ends = hot.final;
            T *og = reinterpret_cast<T *>(to.at) + pc * to.step;
            float *pg = reinterpret_cast<float *>(part.at) + pc * part.step;
#pragma unroll 2
            for (int j = 0; j < W / 2; ++j) {
                const int i = j * 64 + half * 32 + lane, rr = quad * 32 + i / W, piece = i % W, col = piece * 4;
                if (pc + rr >= hot.pe || col >= to.d) continue;
                const float4 v = *reinterpret_cast<const float4 *>(ob + (rr * W + (piece ^ (rr & 7))) * 16);
                float o[4] = {v.x, v.y, v.z, v.w};
                float *p = pg + rr * part.step + col;
                T *at = og + rr * to.step + col;
                if (adds) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (col + e < to.d) o[e] += p[e];
                }
                if (!ends) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (col + e < to.d) p[e] = o[e];
                } else if (to.vec) {
                    *reinterpret_cast<Pack<T, 4> *>(at) = pack<T, 4>(o);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (col + e < to.d) at[e] = from_f<T>(o[e]);
                }
            }
            if (NI != 1) __syncthreads();   // the next keys go where these rows were
        }
        // S = lam^n S + KV, and its terms for the next chunk.  The float32 rounding of
        // lam^n alone would bias a state that lives for many chunks: two parts.
        float hi = full[0], lo = full[1];
        if (cnt - 1 + lead != kChunk) {
            const double step = decay_pow(ld, cnt - 1 + lead);
            hi = (float)step;
            lo = (float)(step - (double)hi);
        }
        uint32_t r[16];
        tmem_ld16x256(tlane + G::kKV + c0, r);
        tmem_wait_ld();
        // (columns from nv on are not computed: their values stay out of every result)
#pragma unroll
        for (int i = 0; i < 16; ++i) S[i] = fmaf(S[i], hi, fmaf(S[i], lo, __uint_as_float(r[i])));
        if (!STATE_ONLY) put_pairs();
    }
    if (!alive && tid == 0) report(args.status, SEMICRF_ERR_DEVICE_TIMEOUT);

    // the state behind the last position (or behind this segment)
    float *to = STATE_ONLY ? segment_at(w, args, s) : s.last && w.s_out ? w.s_out + state_at(w, args, s) : nullptr;
    if (to) {
        const int rs = STATE_ONLY ? args.width : w.s_rs, cs = STATE_ONLY ? 1 : w.s_cs;
        const float f = !STATE_ONLY && w.out_decay ? dec[1] : 1.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int row = quad * 16 + (lane >> 2) + (i & 2) * 4, col = c0 + (i >> 2) * 8 + (lane & 3) * 2 + (i & 1);
            if (row < s.dk && col < s.dv) to[(long long)row * rs + (long long)col * cs] = f * S[i];
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
    const int W = args.width, i = blockIdx.y * blockDim.x + threadIdx.x, row = i / W, col = i % W, nseg = args.nseg;
    const LaSpan s = la_span(args, w, blockIdx.x * nseg);
    __shared__ double power[2];   // of a whole segment: the first one, the others
    if (threadIdx.x < 2)
        power[threadIdx.x] = decay_pow(args.log_decay[s.h], args.seg_len - 1 + (threadIdx.x ? 1 : w.lead));
    __syncthreads();
    if (row >= s.dk || col >= s.dv) return;
    float *seg = segment_at(w, args, s) + i;
    const long long sz = (long long)W * W;
    // segments before the last one that are whole: their sums exist
    const int whole = min(nseg - 1, s.L / args.seg_len);
    float carry = w.s_in ? w.s_in[state_at(w, args, s) + (long long)row * w.s_rs + (long long)col * w.s_cs] : 0.f;
    constexpr int U = 8;   // loads in flight
    for (int j0 = 0; j0 <= whole; j0 += U) {
        float add[U];
#pragma unroll
        for (int u = 0; u < U; ++u) add[u] = j0 + u < whole ? seg[(j0 + u) * sz] : 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j0 + u > whole) break;
            seg[(j0 + u) * sz] = carry;
            carry = (float)(power[j0 + u > 0] * (double)carry + (double)add[u]);
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

template <typename T, bool STATE_ONLY>
cudaError_t go_chunk(const LaArgs &a, cudaStream_t st, int *n)
{
    using G = LaCfg<T>;
    cudaError_t e = cudaFuncSetAttribute(la_chunk_kernel<T, STATE_ONLY>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::kSmem);
    if (e != cudaSuccess) return e;
    return timed_launch(st, n, [&] {
        la_chunk_kernel<T, STATE_ONLY><<<dim3(a.B * a.H * a.slices * a.nseg, a.nwalk), 256, G::kSmem, st>>>(a);
    });
}

template <bool STATE_ONLY>
cudaError_t go_walk(const LaArgs &a, int dtype, cudaStream_t st, int *n)
{
    if (dtype == SEMICRF_F32) return go_chunk<float, STATE_ONLY>(a, st, n);
    if (dtype == SEMICRF_BF16) return go_chunk<__nv_bfloat16, STATE_ONLY>(a, st, n);
    return go_chunk<__half, STATE_ONLY>(a, st, n);
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

namespace {

// How a call is walked: by the copy engine's kernel in one tile of 64 or 128, or in tiles of
// 64; and its segments, which walk side by side.  A split walk first forms what each
// segment adds to the state (K and V read twice) and joins the states, so it pays where the
// sequences and heads leave most of the GPU idle.  Measured on forward calls, the rule's
// choice against one walk (rows: sequences times heads):
//   bf16, width 64   48 rows of 4096 positions 62 us in 6 segments, 105 in one; 98 rows 97 in
//                    three, 107 in one, but of 2048 positions 66 and 60; two never gain (128
//                    rows of 4096: 129 and 109), as two blocks share an SM and its rate
//   bf16, width 128  48 rows of 4096 positions 130 us in three, 154 in one; 74 rows in two 171
//                    and 156, of 20 000 positions 620 and 713, of 2048 115 and 86
//   float32          74 rows of 2048 positions 109 us in two, 138 in one; 98 rows have one
//   float16          74 rows of 2048 positions 86 us in two, 104 in one
struct LaPlan {
    int width, slices, kblocks, nseg, seg_len;
    size_t seg_bytes, part_bytes;   // of one walk
};

LaPlan la_plan(int B, int T, int H, int dk, int dv, int dtype, int nwalk, bool tma)
{
    const int most = dk > dv ? dk : dv;   // (the backward's walks exchange the two)
    LaPlan p;
    p.width = tma && most > 64 ? 128 : 64;
    p.slices = ((nwalk > 1 ? most : dv) + p.width - 1) / p.width;
    p.kblocks = ((nwalk > 1 ? most : dk) + p.width - 1) / p.width;
    const bool shared = p.width == 64 && dtype == SEMICRF_BF16;
    const long long rows = (long long)B * H * nwalk * p.slices;
    long long n = (shared ? 2LL : 1LL) * device_sm_count() / rows;
    if (n > T / 512) n = T / 512;
    if (n < (shared ? 3 : 2)) n = 1;
    if (dtype == SEMICRF_BF16 && ((n == 2 && T < 8192) || (n == 3 && T < 3072))) n = 1;
    const long long len = ((T + n - 1) / n + kChunk - 1) / kChunk * kChunk;
    p.seg_len = (int)len;
    p.nseg = (int)((T + len - 1) / len);
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    p.seg_bytes = p.nseg > 1 ? up((size_t)B * H * p.slices * p.nseg * p.width * p.width * sizeof(float)) : 0;
    p.part_bytes = p.kblocks > 1 && dtype != SEMICRF_F32 ? up((size_t)B * T * H * (nwalk > 1 ? most : dv) * sizeof(float)) : 0;
    return p;
}

}  // namespace

size_t la_need(const LaArgs &a, int dtype)
{
    const LaPlan p = la_plan(a.B, a.T, a.H, a.w[0].dk, a.w[0].dv, dtype, a.nwalk, la_tma_ok(a, dtype));
    return a.nwalk * (p.seg_bytes + p.part_bytes);
}

size_t la_workspace(int B, int T, int H, int dk, int dv, int dtype, int nwalk)
{
    size_t most = 0;   // operands that the copy engine cannot address take the other plan: room for either
    for (int tma = 0; tma < 2; ++tma) {
        if (tma && (dtype != SEMICRF_BF16 || dk > 128 || dv > 128)) continue;
        const LaPlan p = la_plan(B, T, H, dk, dv, dtype, nwalk, tma);
        const size_t n = nwalk * (p.seg_bytes + p.part_bytes);
        if (n > most) most = n;
    }
    return most;
}

cudaError_t launch_la(LaArgs a, int dtype, unsigned char *ws, size_t ws_bytes, cudaStream_t st, int *launches, bool *small)
{
    *launches = 0;
    *small = false;
    LaPlan p;
    LaMaps maps;
    bool tma = la_tma_ok(a, dtype);
    for (;;) {
        p = la_plan(a.B, a.T, a.H, a.w[0].dk, a.w[0].dv, dtype, a.nwalk, tma);
        a.width = p.width;
        a.slices = p.slices;
        a.nseg = p.nseg;
        a.seg_len = p.seg_len;
        if (!tma || la_tma_maps(a, &maps)) break;
        cudaGetLastError();
        tma = false;   // the kernel for any operands
    }
    *small = ws_bytes < a.nwalk * (p.seg_bytes + p.part_bytes);
    if (*small) return cudaSuccess;
    for (int i = 0; i < a.nwalk; ++i) {
        a.w[i].seg = p.seg_bytes ? reinterpret_cast<float *>(ws) : nullptr;
        ws += p.seg_bytes;
        a.w[i].part = p.part_bytes ? reinterpret_cast<float *>(ws) : nullptr;
        ws += p.part_bytes;
    }
    for (a.kblock = 0; a.kblock < p.kblocks; ++a.kblock) {
        cudaError_t e;
        if (a.nseg > 1) {
            e = tma ? launch_la_tma(a, maps, true, st, launches) : go_walk<true>(a, dtype, st, launches);
            if (e != cudaSuccess) return e;
            e = timed_launch(st, launches, [&] {
                la_join_kernel<<<dim3(a.B * a.H * a.slices, a.width * a.width / 256, a.nwalk), 256, 0, st>>>(a);
            });
            if (e != cudaSuccess) return e;
        }
        e = tma ? launch_la_tma(a, maps, false, st, launches) : go_walk<false>(a, dtype, st, launches);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_la_step(const LaStepArgs &a, int dtype, cudaStream_t st, int *launches)
{
    *launches = 0;
    if (dtype == SEMICRF_F32) return step_type<float>(a, st, launches);
    if (dtype == SEMICRF_BF16) return step_type<__nv_bfloat16>(a, st, launches);
    return step_type<__half>(a, st, launches);
}

cudaError_t la_found(int32_t *to) { return read_found(to); }
cudaError_t la_clear_found(cudaStream_t st) { return clear_found(st); }

}  // namespace semicrf
