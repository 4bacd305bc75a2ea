// linear_attention_tma.cu -- the chunked walk of linear attention for bf16 operands that
// the copy engine can address (16-byte aligned rows and strides).
//
// Eight warps compute, a ninth issues: it alone starts copies and matrix instructions,
// so that neither a full queue of the matrix unit nor a full queue of loads holds up a
// warp that has arithmetic to do.  A chunk of 128 positions:
//
//   copies   Q, K, V tiles, each fetched again as soon as its last reader is done
//   matrix   o = Q S  |  KV = K~^T V                 |  o += P V            next scores = Q K^T
//   warps    K~       |  P from the scores, o scaled |  S = lam^128 S + KV, o out  |
//
// with K~ = c lam^{end-i} K and P = b c lam^{i-j} scores; between the bars all warps meet.
// Two blocks share an SM at width 64 (112 KB of tiles, 256 columns of tensor memory
// each), one computing while the other waits.  Accumulators hold one chunk's sums only:
// they round towards zero, which the state, float32 in registers (tensor memory at
// width 128), must not.
//
// Measured: 512 sequences and heads of 1024 positions at width 64 (268 MB, 41 us at the copy
// rate) 79 us; of 128 x 4000, which fill the SMs once, 109 us, the time of one block's 32
// chunks in a row (3.4 us each).  A chunk moves 368 KB through shared memory, 2900 cycles at
// 128 bytes a cycle (matrix operands 208 KB, K~ 64, tiles in and out 80, the state 16); the
// matrix unit is busy 42 % of the time.  The chain of a chunk's steps, each behind a meeting
// of all warps, is what bounds it.
//
// A walk against time takes a chunk's rows in memory order too: row r is position
// 127 - r of the chunk, and the tables of decays are mirrored.
#include "la_common.cuh"
#include "tensor_core.cuh"

namespace semicrf {
namespace {

constexpr int kWorkers = 256, kThreads = kWorkers + 32;

struct LaTables {
    float diag[64];   // b c lam^d by 31 + (row - column) inside a 32 x 32 block, 0 where the column lies ahead
    float side[32];   // by column: the rest of lam^d in the blocks beside the diagonal
    float block[4];   // lam^{32 m}
    float full[2];    // lam^128 in two floats
};

template <int D>
struct TmaCfg {
    static constexpr int NM = 2, NK = 3;            // terms of P and S, and of K~
    static constexpr int kTile = D / 64 * 16384;    // 128 rows
    static constexpr int kSTile = D * D * 2;
    static constexpr bool kApart = D == 64;         // K has a tile of its own beside K~, or becomes K~'s first term
    static constexpr bool kStateTmem = D == 128;
    static constexpr int kQ = 0, kK = kQ + kTile, kKt = kApart ? kK + kTile : kK, kV = kKt + 3 * kTile,
                         kS = kV + kTile, kTab = kS + NM * kSTile, kBars = kTab + (int)sizeof(LaTables),
                         kSmem = kBars + 64;
    static constexpr int kO = 128, kKV = kO + D, kCols = D == 64 ? 256 : 512;
    static constexpr int kState = kKV + (kStateTmem ? D : 0);
    static constexpr int kOut = kKt + 2 * kTile;    // outputs on their way, where K~'s third term is
    static constexpr int NP = kChunk * (D / 8) / kWorkers, kRows = kWorkers / (D / 8);
    static constexpr int kBlocks = D == 64 ? 2 : 1;
    static_assert(kSmem <= (kBlocks == 2 ? 113 : 227) * 1024, "shared memory");
};

// K~ has three terms (24 bits), as the float32 state wants.  Where no state leaves the call
// two would do for 16-bit outputs and take 6 % (width 64) to 14 % (width 128) less time, but
// then outputs would differ in their last bits with whether the state is asked for.
template <int D>
__global__ __launch_bounds__(kThreads, (TmaCfg<D>::kBlocks)) void la_tma_kernel(const __grid_constant__ LaArgs args,
                                                                                const __grid_constant__ LaMaps maps)
{
    using G = TmaCfg<D>;
    using T = __nv_bfloat16;
    constexpr int NM = G::NM, NK = G::NK, NP = G::NP;
    constexpr int kUnroll = D == 128 ? 8 : 1;   // of the matrix instructions: no registers for it at width 64
    constexpr uint64_t kTileD = G::kTile >> 4, kSTileD = G::kSTile >> 4, kRow16 = 2048 >> 4;
    extern __shared__ __align__(1024) unsigned char sm[];
    const LaWalk &w = args.w[blockIdx.y];
    const LaSpan s = la_span(args, w, blockIdx.x);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    zero_rows<T>(w, s);
    if (s.L == 0 && s.last) copy_state(w, args, s);
    if (s.pe == s.p0) return;

    LaTables &tab = *reinterpret_cast<LaTables *>(sm + G::kTab);
    uint32_t *slot = reinterpret_cast<uint32_t *>(sm + G::kBars + 56);
    const uint32_t smem = static_cast<uint32_t>(__cvta_generic_to_shared(sm)), bars = smem + G::kBars;
    const uint32_t full_q = bars, full_k = bars + 8, full_v = bars + 16;
    const uint32_t done_qk = bars + 24, done_qs = bars + 32, done_kv = bars + 40, done_pv = bars + 48;
    const float ld = args.log_decay[s.h], pa = w.b * w.c;
    const int rev = w.reverse;
    if (warp == 8) {
        tmem_alloc(static_cast<uint32_t>(__cvta_generic_to_shared(slot)), G::kCols);
        if (lane == 0) {
            for (int i = 0; i < 7; ++i) mbar_init(bars + 8 * i, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    } else if (tid < 64) {
        const int d = rev ? 31 - tid : tid - 31;
        tab.diag[tid] = d >= 0 && tid < 63 ? (float)(decay_pow(ld, d) * (double)pa) : 0.f;
    } else if (tid < 96) {
        tab.side[tid - 64] = (float)decay_pow(ld, rev ? tid - 64 : 95 - tid);
    } else if (tid < 100) {
        tab.block[tid - 96] = (float)decay_pow(ld, 32 * (tid - 96));
    } else if (tid == 100) {
        const double v = decay_pow(ld, kChunk);
        tab.full[0] = (float)v;
        tab.full[1] = (float)(v - (double)tab.full[0]);
    }
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tm = __shfl_sync(0xffffffffu, *slot, 0);
    const int nv = (w.dv + 15) / 16 * 16, kd = (w.dk + 15) / 16;
    const int chunks = (s.pe - s.p0 + kChunk - 1) / kChunk, whole = (s.pe - s.p0) / kChunk;
    // first row in memory of chunk n
    auto row_of = [&](int n) { return rev ? s.L - s.p0 - (n + 1) * kChunk : s.p0 + n * kChunk; };
    bool alive = true;

    if (warp == 8) {
        const auto &map = maps.w[blockIdx.y];
        // all of these in a branch of one lane, which is elected anew each time: a flag of the
        // election kept in a variable made each instruction 60 to 180 cycles long
        auto await = [&](uint32_t bar, uint32_t parity) { alive = mbar_wait_bounded(bar, parity) && alive; };
        int fetched[3] = {0, 0, 0};   // tiles of Q, K, V asked for
        auto fetch = [&](const CUtensorMap &m, int tile, uint32_t bar, int n) {
            ++fetched[(bar - bars) / 8];
            mbar_expect(bar, G::kTile);
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
                tma_load(smem + tile + c * 16384, &m, c * 64, s.h, row_of(n), s.b, bar);
        };
        auto scores = [&](int n) {   // Q K^T of chunk n
            if (n < whole) {
                await(full_q, n & 1);
                await(full_k, n & 1);
            }
            tc_after_sync();
            const uint64_t dq = desc_swz(smem + G::kQ, 16), dk = desc_swz(smem + G::kK, 16);
#pragma unroll(kUnroll)
            for (int k = 0; k < kd; ++k) {
                const uint64_t at = (uint64_t)((k >> 2) * 16384 + (k & 3) * 32) >> 4;
                mma_ss(tm, dq + at, dk + at, mma_idesc(128, 128, false, false), k > 0);
            }
            mma_commit(done_qk);
        };
        // the warp whole again, then all warps: false once a wait has run out
        bool broken = false;
        auto meet = [&] {
            __syncwarp();
            broken = __syncthreads_or(!alive);
            return !broken;
        };
        if (whole > 0 && elect_lane()) {
            fetch(map.q, G::kQ, full_q, 0);
            fetch(map.k, G::kK, full_k, 0);
            fetch(map.v, G::kV, full_v, 0);
            if (G::kApart) scores(0);
        }
        meet();   // the state's terms are there
        for (int n = 0; n < chunks; ++n) {
            const uint32_t parity = n & 1;
            const bool next = n + 1 < whole;
            if (n >= whole && !meet()) break;   // the shorter chunk's tiles are there
            if (elect_lane()) {
                if (n >= whole || !G::kApart) scores(n);
                tc_after_sync();
                const uint32_t i2 = mma_idesc(128, nv, false, true);
                const uint64_t dq = desc_swz(smem + G::kQ, 16), ds = desc_swz(smem + G::kS, 16384);
#pragma unroll(kUnroll)
                for (int i = 0; i < 2 * kd; ++i) {   // the state's second term first
                    const int k = i < kd ? i : i - kd;
                    const uint64_t at = (uint64_t)((k >> 2) * 16384 + (k & 3) * 32) >> 4;
                    mma_ss(tm + G::kO, dq + at, ds + (i < kd ? kSTileD : 0) + k * kRow16, i2, i > 0);
                }
                mma_commit(done_qs);
                tma_store_read();   // the last outputs have left
            }
            if (!meet()) break;   // K~'s third term may be written
            if (next && elect_lane()) {
                await(done_qs, parity);
                fetch(map.q, G::kQ, full_q, n + 1);
            }
            if (!meet()) break;   // K~ is there
            if (elect_lane()) {
                if (G::kApart && next) fetch(map.k, G::kK, full_k, n + 1);
                if (n < whole) await(full_v, parity);
                tc_after_sync();
                const uint32_t i4 = mma_idesc(D, nv, true, true);
                const uint64_t dk = desc_swz(smem + G::kKt, 16384), dv = desc_swz(smem + G::kV, 16384);
#pragma unroll
                for (int x = NK - 1; x >= 0; --x)
#pragma unroll(kUnroll)
                    for (int k = 0; k < kChunk / 16; ++k)
                        mma_ss(tm + G::kKV, dk + x * kTileD + k * kRow16, dv + k * kRow16, i4, x < NK - 1 || k > 0);
                mma_commit(done_kv);
            }
            if (!meet()) break;   // P is there, o scaled
            if (elect_lane()) {
                tc_after_sync();
                const uint32_t i3 = mma_idesc(128, nv, false, true);
                const uint64_t dv = desc_swz(smem + G::kV, 16384);
#pragma unroll
                for (int x = NM - 1; x >= 0; --x)
#pragma unroll(kUnroll)
                    for (int k = 0; k < kChunk / 16; ++k)
                        mma_ts(tm + G::kO, tm + k * (8 * NM) + x * 8, dv + k * kRow16, i3, true);
                mma_commit(done_pv);
                if (next) {
                    if (!G::kApart) {
                        await(done_kv, parity);
                        fetch(map.k, G::kK, full_k, n + 1);
                    }
                    await(done_pv, parity);   // P is read: its columns take the next scores
                    fetch(map.v, G::kV, full_v, n + 1);
                    if (G::kApart) scores(n + 1);
                }
            }
            if (!meet()) break;   // this chunk's outputs lie in shared memory, the next state's terms too
            if (n < whole && elect_lane()) {
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    tma_store(smem + G::kOut + c * 16384, &map.o, c * 64, s.h, row_of(n), s.b);
                tma_store_commit();
            }
        }
        if (elect_lane()) {
            tma_store_done();
            if (!alive) report(args.status, SEMICRF_ERR_DEVICE_TIMEOUT);
            if (broken) {   // somebody's wait has run out: the copies under way end before the block does
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    if (fetched[i]) mbar_wait_bounded(bars + 8 * i, (fetched[i] - 1) & 1);
            }
        }
        __syncwarp();
    } else {
        auto await = [&](uint32_t bar, uint32_t parity) {
            alive = mbar_wait_bounded(bar, parity) && alive;
            __syncwarp();
        };
        const int quad = warp & 3, half = warp >> 2, row = quad * 32 + lane, c0 = half * (D / 2);
        const uint32_t tlane = tm + ((uint32_t)(quad * 32) << 16);
        // pieces of K this thread turns into K~: column piece j8 of rows r0, r0 + kRows, ...
        const int r0 = tid / (D / 8), j8 = tid % (D / 8);
        const int at0 = (j8 >> 3) * 16384 + swz(r0, j8 & 7);   // (kRows is a multiple of 8)
        float wk[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int far = rev ? r0 + i * G::kRows : kChunk - 1 - r0 - i * G::kRows;   // positions to the chunk's end
            const int low = far & 31;
            wk[i] = w.c * tab.side[rev ? low : 31 - low] * tab.block[far >> 5];
        }
        const float beside = pa * (float)decay_pow(ld, rev ? 32 - lane : lane + 1);
        const float ofull = w.b * (float)decay_pow(ld, (rev ? kChunk - 1 - row : row) + 1);

        float S[G::kStateTmem ? 1 : 16];
        auto put_pairs = [&] {   // D = 64: rows quad * 16 + lane / 4 (+ 8), column pairs c0 + 8 j + 2 (lane % 4)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    uint32_t t[NM];
                    split2<NM>(S[4 * j + 2 * a], S[4 * j + 2 * a + 1], t);
                    unsigned char *to = sm + G::kS + swz(quad * 16 + (lane >> 2) + 8 * a, half * 4 + j) + 4 * (lane & 3);
#pragma unroll
                    for (int x = 0; x < NM; ++x) *reinterpret_cast<uint32_t *>(to + x * G::kSTile) = t[x];
                }
        };
        auto put_row = [&](int c, const uint32_t (&r)[16]) {   // D = 128: columns c .. c + 15 of row `row`
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
                const int p = c / 8 + g;
#pragma unroll
                for (int x = 0; x < NM; ++x)
                    *reinterpret_cast<uint4 *>(sm + G::kS + x * G::kSTile + (p >> 3) * 16384 + swz(row, p & 7)) =
                        make_uint4(o[x][0], o[x][1], o[x][2], o[x][3]);
            }
        };
        {
            const StateAt from = state_from(w, args, s);
            auto given = [&](int i, int j) {
                return from.p && i < w.dk && j < w.dv ? from.p[(long long)i * from.rs + (long long)j * from.cs] : 0.f;
            };
            if constexpr (G::kStateTmem) {
#pragma unroll 1
                for (int c = c0; c < c0 + D / 2; c += 16) {
                    uint32_t r[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(given(row, c + e));
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
        }

        smem_to_mma();
        __syncthreads_or(!alive);
        for (int n = 0; n < chunks; ++n) {
            const uint32_t parity = n & 1;
            const int cnt = min(kChunk, s.pe - s.p0 - n * kChunk);
            const bool is_whole = n < whole;
            if (!is_whole) {
                // the last, shorter chunk: rows outside the sequence have to be zeros
                auto bring = [&](const void *base, const long long (&st)[3], int d, int tile) {
                    const T *p = static_cast<const T *>(base) + s.b * st[0] + s.h * st[2] + (long long)j8 * 8;
#pragma unroll 1
                    for (int i = 0; i < NP; ++i) {
                        const int r = r0 + i * G::kRows, pos = rev ? kChunk - 1 - r : r;
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (pos < cnt && j8 * 8 < d) v = *reinterpret_cast<const uint4 *>(p + (row_of(n) + r) * st[1]);
                        *reinterpret_cast<uint4 *>(sm + tile + at0 + i * G::kRows * 128) = v;
                    }
                };
                bring(w.q, w.qs, w.dk, G::kQ);
                bring(w.k, w.ks, w.dk, G::kK);
                bring(w.v, w.vs, w.dv, G::kV);
            }
            if (!is_whole) {
                smem_to_mma();
                if (__syncthreads_or(!alive)) break;
            }
            const int lead = s.p0 + n == 0 ? w.lead : 1;
            if (is_whole) await(full_k, parity);
            if (!G::kApart) await(done_qk, parity);   // K~ replaces K
            uint4 third[NP];   // K~'s third term, whose tile the last outputs may still be leaving
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const unsigned char *at = sm + G::kK + at0 + i * G::kRows * 128;
                const uint4 u = *reinterpret_cast<const uint4 *>(at);
                float f = wk[i];
                if (!is_whole) {
                    const int r = r0 + i * G::kRows, pos = rev ? kChunk - 1 - r : r;
                    f = pos < cnt ? w.c * (float)decay_pow(ld, cnt - 1 - pos) : 0.f;
                }
                uint32_t o[NK][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t v = reinterpret_cast<const uint32_t *>(&u)[e];
                    uint32_t t[NK];
                    split2<NK>(__uint_as_float(v << 16) * f, __uint_as_float(v & 0xffff0000u) * f, t);
#pragma unroll
                    for (int x = 0; x < NK; ++x) o[x][e] = t[x];
                }
#pragma unroll
                for (int x = 0; x < NK; ++x) {
                    const uint4 v = make_uint4(o[x][0], o[x][1], o[x][2], o[x][3]);
                    if (x == 2)
                        third[i] = v;
                    else
                        *reinterpret_cast<uint4 *>(sm + G::kKt + x * G::kTile + at0 + i * G::kRows * 128) = v;
                }
            }
            if (__syncthreads_or(!alive)) break;
#pragma unroll
            for (int i = 0; i < NP; ++i)
                *reinterpret_cast<uint4 *>(sm + G::kKt + 2 * G::kTile + at0 + i * G::kRows * 128) = third[i];
            smem_to_mma();
            if (__syncthreads_or(!alive)) break;

            if (G::kApart) await(done_qk, parity);
            tc_after_sync();
            // scores -> P: 32 columns at a time, 16 scores becoming 8 columns of each term
#pragma unroll 1
            for (int c = half * 64; c < half * 64 + 64; c += 32) {
                const int away = rev ? c / 32 - quad : quad - c / 32;
                uint32_t r[32];
                if (away >= 0) {
                    tmem_ld32(tlane + c, r);
                    tmem_wait_ld();
                }
                if (away > 0) {
                    const float g = beside * tab.block[away - 1];
#pragma unroll
                    for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * (g * tab.side[e]));
                } else if (away == 0) {
                    const float *f = tab.diag + 31 + lane;
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
                        for (int x = 0; x < NM; ++x) o[x][e] = t[x];
                    }
#pragma unroll
                    for (int x = 0; x < NM; ++x) tmem_st8(tlane + (c / 16 + g) * (8 * NM) + x * 8, o[x]);
                }
            }
            // o starts as b lam^{i+1} q S
            await(done_qs, parity);
            tc_after_sync();
            const float f = lead ? ofull : w.b * (float)decay_pow(ld, rev ? kChunk - 1 - row : row);
#pragma unroll 1
            for (int c = 0; c < D / 2; c += 32) {
                uint32_t r[2][16];
#pragma unroll
                for (int g = 0; g < 2; ++g) tmem_ld16(tlane + G::kO + c0 + c + 16 * g, r[g]);
                tmem_wait_ld();
#pragma unroll
                for (int g = 0; g < 2; ++g) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) r[g][e] = __float_as_uint(__uint_as_float(r[g][e]) * f);
                    tmem_st16(tlane + G::kO + c0 + c + 16 * g, r[g]);
                }
            }
            tmem_wait_st();
            tc_before_sync();
            if (__syncthreads_or(!alive)) break;
            await(done_kv, parity);
            tc_after_sync();
            // S = lam^n S + KV; the float32 rounding of lam^n alone would bias a state that
            // lives for many chunks: two parts
            float hi = tab.full[0], lo = tab.full[1];
            if (cnt - 1 + lead != kChunk) {
                const double step = decay_pow(ld, cnt - 1 + lead);
                hi = (float)step;
                lo = (float)(step - (double)hi);
            }
            if constexpr (G::kStateTmem) {
#pragma unroll 1
                for (int c = c0; c < min(c0 + D / 2, nv); c += 32) {
                    uint32_t r[2][16], old[2][16];
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        tmem_ld16(tlane + G::kKV + c + 16 * g, r[g]);
                        tmem_ld16(tlane + G::kState + c + 16 * g, old[g]);
                    }
                    tmem_wait_ld();
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float prev = __uint_as_float(old[g][e]);
                            old[g][e] = __float_as_uint(fmaf(prev, hi, fmaf(prev, lo, __uint_as_float(r[g][e]))));
                        }
                        tmem_st16(tlane + G::kState + c + 16 * g, old[g]);
                        put_row(c + 16 * g, old[g]);
                    }
                }
                tmem_wait_st();
                tc_before_sync();
            } else {
                uint32_t r[16];
                tmem_ld16x256(tlane + G::kKV + c0, r);
                tmem_wait_ld();
                tc_before_sync();
                // (columns from nv on are not computed: their values stay out of every result)
#pragma unroll
                for (int i = 0; i < 16; ++i) S[i] = fmaf(S[i], hi, fmaf(S[i], lo, __uint_as_float(r[i])));
                put_pairs();
            }
            await(done_pv, parity);
            tc_after_sync();
#pragma unroll 1
            for (int c = 0; c < D / 2; c += 32) {
                uint32_t r[32];
                tmem_ld32(tlane + G::kO + c0 + c, r);
                tmem_wait_ld();
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(r[8 * g + 2 * e]),
                                                                      __uint_as_float(r[8 * g + 2 * e + 1]));
                        o[e] = *reinterpret_cast<const uint32_t *>(&v);
                    }
                    const int p = (c0 + c) / 8 + g;
                    *reinterpret_cast<uint4 *>(sm + G::kOut + (p >> 3) * 16384 + swz(row, p & 7)) =
                        make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            smem_to_mma();
            tc_before_sync();
            if (__syncthreads_or(!alive)) break;
            if (!is_whole && j8 * 8 < w.dv) {
                T *o = static_cast<T *>(w.o) + s.b * w.os[0] + s.h * w.os[2] + (long long)j8 * 8;
#pragma unroll 1
                for (int i = 0; i < NP; ++i) {
                    const int r = r0 + i * G::kRows, pos = rev ? kChunk - 1 - r : r;
                    if (pos < cnt)
                        *reinterpret_cast<uint4 *>(o + (row_of(n) + r) * w.os[1]) =
                            *reinterpret_cast<const uint4 *>(sm + G::kOut + at0 + i * G::kRows * 128);
                }
            }
        }

        // the state behind the last position (or behind this segment)
        float *to = s.last && w.s_out ? w.s_out + state_at(w, args, s) : nullptr;
        if (to) {
            const int rs = w.s_rs, cs = w.s_cs;
            const float f = w.out_decay ? (float)decay_pow(ld, 1) : 1.f;
            auto keep = [&](int i, int j, float v) {
                if (i < w.dk && j < w.dv) to[(long long)i * rs + (long long)j * cs] = f * v;
            };
            if constexpr (G::kStateTmem) {
#pragma unroll 1
                for (int c = c0; c < min(c0 + D / 2, nv); c += 16) {
                    uint32_t r[16];
                    tmem_ld16(tlane + G::kState + c, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) keep(row, c + e, __uint_as_float(r[e]));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    keep(quad * 16 + (lane >> 2) + (i & 2) * 4, c0 + (i >> 2) * 8 + (lane & 3) * 2 + (i & 1), S[i]);
            }
        }
        if (!alive && tid == 0) report(args.status, SEMICRF_ERR_DEVICE_TIMEOUT);
    }
    tc_before_sync();
    __syncthreads();
    if (warp == 8) tmem_free(tm, G::kCols);
}

// What a whole segment adds to the state: KV of each chunk as above, S = lam^128 S + KV.
// V's tile is double, so that the next one travels while a chunk's products run; the sums of
// a chunk are taken up before the next keys are weighted into K~'s only tiles (three of
// 32 KB at width 128).
// Segments that end inside the sequence's last chunk are not asked for.
//
// Measured: 96 walks of 40 chunks at width 128 in 111 us, 2.8 us a chunk (of which the matrix
// unit is busy a third); at width 64, where two blocks share an SM, 51 us for 280 walks of 22
// chunks.
template <int D>
struct StateCfg {
    static constexpr int kTile = D / 64 * 16384, NK = 3;   // (terms of K~)
    static constexpr int kK = 0, kV = kK + kTile, kKt = kV + 2 * kTile, kBars = kKt + NK * kTile, kSmem = kBars + 64;
    static constexpr int kKV = 0, kState = 2 * D, kCols = D == 64 ? 128 : 512;
    static constexpr int NP = kChunk * (D / 8) / kWorkers, kRows = kWorkers / (D / 8);
    static constexpr int kBlocks = D == 64 ? 2 : 1;
    static_assert(kSmem <= (kBlocks == 2 ? 113 : 227) * 1024, "shared memory");
};

template <int D>
__global__ __launch_bounds__(kThreads, (StateCfg<D>::kBlocks)) void la_state_kernel(const __grid_constant__ LaArgs args,
                                                                                  const __grid_constant__ LaMaps maps)
{
    using G = StateCfg<D>;
    constexpr int NK = G::NK, NP = G::NP;
    constexpr uint64_t kTileD = G::kTile >> 4, kRow16 = 2048 >> 4;
    extern __shared__ __align__(1024) unsigned char sm[];
    const LaWalk &w = args.w[blockIdx.y];
    const LaSpan s = la_span(args, w, blockIdx.x);
    if (s.seg == args.nseg - 1 || s.pe - s.p0 < args.seg_len) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    uint32_t *slot = reinterpret_cast<uint32_t *>(sm + G::kBars + 56);
    const uint32_t smem = static_cast<uint32_t>(__cvta_generic_to_shared(sm)), bars = smem + G::kBars;
    const uint32_t full_k = bars, full_v = bars + 8, done = bars + 24;   // K; V, even and odd; KV, even and odd
    if (warp == 8) {
        tmem_alloc(static_cast<uint32_t>(__cvta_generic_to_shared(slot)), G::kCols);
        if (lane == 0) {
            for (int i = 0; i < 5; ++i) mbar_init(bars + 8 * i, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    }
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tm = __shfl_sync(0xffffffffu, *slot, 0);
    const int nv = (w.dv + 15) / 16 * 16, chunks = args.seg_len / kChunk, rev = w.reverse;
    const float ld = args.log_decay[s.h];
    bool alive = true;

    if (warp == 8) {
        const auto &map = maps.w[blockIdx.y];
        int fetched[3] = {0, 0, 0};
        auto await = [&](uint32_t bar, uint32_t parity) { alive = mbar_wait_bounded(bar, parity) && alive; };
        auto fetch = [&](const CUtensorMap &m, int tile, int which, int n) {
            ++fetched[which];
            mbar_expect(bars + 8 * which, G::kTile);
            const int row = rev ? s.L - s.p0 - (n + 1) * kChunk : s.p0 + n * kChunk;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
                tma_load(smem + tile + c * 16384, &m, c * 64, s.h, row, s.b, bars + 8 * which);
        };
        if (elect_lane()) {
            fetch(map.k, G::kK, 0, 0);
            fetch(map.v, G::kV, 1, 0);
            if (chunks > 1) fetch(map.v, G::kV + G::kTile, 2, 1);
        }
        bool broken = false;
        for (int n = 0; n < chunks && !broken; ++n) {
            __syncwarp();
            broken = __syncthreads_or(!alive);   // K~ is there
            if (!broken && elect_lane()) {
                const int odd = n & 1;
                if (n + 1 < chunks) fetch(map.k, G::kK, 0, n + 1);
                await(full_v + 8 * odd, n >> 1 & 1);
                tc_after_sync();
                const uint32_t id = mma_idesc(D, nv, true, true);
                const uint64_t dk = desc_swz(smem + G::kKt, 16384);
                const uint64_t dv = desc_swz(smem + G::kV + odd * G::kTile, 16384);
#pragma unroll
                for (int x = NK - 1; x >= 0; --x)
#pragma unroll(D == 128 ? 8 : 1)
                    for (int k = 0; k < kChunk / 16; ++k)
                        mma_ss(tm + G::kKV + odd * D, dk + x * kTileD + k * kRow16, dv + k * kRow16, id, x < NK - 1 || k > 0);
                mma_commit(done + 8 * odd);
                if (n > 0 && n + 1 < chunks) {   // the other tile of V is free once its products are there
                    await(done + 8 * (odd ^ 1), (n - 1) >> 1 & 1);
                    if (odd)
                        fetch(map.v, G::kV, 1, n + 1);
                    else
                        fetch(map.v, G::kV + G::kTile, 2, n + 1);
                }
            }
        }
        if (elect_lane()) {
            if (!alive) report(args.status, SEMICRF_ERR_DEVICE_TIMEOUT);
            if (broken) {   // somebody's wait has run out: the copies under way end before the block does
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    if (fetched[i]) mbar_wait_bounded(bars + 8 * i, (fetched[i] - 1) & 1);
            }
        }
        __syncwarp();
    } else {
        auto await = [&](uint32_t bar, uint32_t parity) {
            alive = mbar_wait_bounded(bar, parity) && alive;
            __syncwarp();
        };
        const int quad = warp & 3, half = warp >> 2, row = quad * 32 + lane, c0 = half * (D / 2);
        const uint32_t tlane = tm + ((uint32_t)(quad * 32) << 16);
        const int r0 = tid / (D / 8), j8 = tid % (D / 8);
        const int at0 = (j8 >> 3) * 16384 + swz(r0, j8 & 7);
        float wk[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int r = r0 + i * G::kRows;
            wk[i] = (float)(w.c * decay_pow(ld, rev ? r : kChunk - 1 - r));
        }
        const double full = decay_pow(ld, kChunk);
        const float whole_hi = (float)full, whole_lo = (float)(full - (double)whole_hi);
        float S[D == 64 ? 16 : 1];
        if constexpr (D == 64) {
#pragma unroll
            for (int i = 0; i < 16; ++i) S[i] = 0.f;
        }
        auto take_up = [&](int n) {   // S = lam^128 S + KV of chunk n
            await(done + 8 * (n & 1), n >> 1 & 1);
            tc_after_sync();
            float hi = whole_hi, lo = whole_lo;
            if (n == 0) hi = lo = 0.f;
            if constexpr (D == 64) {
                uint32_t r[16];
                tmem_ld16x256(tlane + G::kKV + (n & 1) * D + c0, r);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) S[i] = fmaf(S[i], hi, fmaf(S[i], lo, __uint_as_float(r[i])));
            } else {
#pragma unroll 1
                for (int c = c0; c < min(c0 + D / 2, nv); c += 32) {
                    uint32_t r[32], old[2][16];
                    tmem_ld32(tlane + G::kKV + (n & 1) * D + c, r);
                    if (n > 0) {
#pragma unroll
                        for (int g = 0; g < 2; ++g) tmem_ld16(tlane + G::kState + c + 16 * g, old[g]);
                    }
                    tmem_wait_ld();
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float prev = n > 0 ? __uint_as_float(old[g][e]) : 0.f;
                            old[g][e] = __float_as_uint(fmaf(prev, hi, fmaf(prev, lo, __uint_as_float(r[16 * g + e]))));
                        }
                        tmem_st16(tlane + G::kState + c + 16 * g, old[g]);
                    }
                }
                tmem_wait_st();
            }
            tc_before_sync();
        };
        bool broken = false;
        for (int n = 0; n < chunks && !broken; ++n) {
            if (n > 0) take_up(n - 1);   // K~'s tiles are read
            await(full_k, n & 1);
            unsigned char *to = sm + G::kKt + at0;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const uint4 u = *reinterpret_cast<const uint4 *>(sm + G::kK + at0 + i * G::kRows * 128);
                uint32_t o[NK][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t v = reinterpret_cast<const uint32_t *>(&u)[e];
                    uint32_t t[NK];
                    split2<NK>(__uint_as_float(v << 16) * wk[i], __uint_as_float(v & 0xffff0000u) * wk[i], t);
#pragma unroll
                    for (int x = 0; x < NK; ++x) o[x][e] = t[x];
                }
#pragma unroll
                for (int x = 0; x < NK; ++x)
                    *reinterpret_cast<uint4 *>(to + x * G::kTile + i * G::kRows * 128) =
                        make_uint4(o[x][0], o[x][1], o[x][2], o[x][3]);
            }
            smem_to_mma();
            broken = __syncthreads_or(!alive);
        }
        if (!broken) take_up(chunks - 1);
        float *to = segment_at(w, args, s);
        auto keep = [&](int i, int j, float v) {
            if (i < w.dk && j < w.dv) to[i * D + j] = v;
        };
        if constexpr (D == 64) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                keep(quad * 16 + (lane >> 2) + (i & 2) * 4, c0 + (i >> 2) * 8 + (lane & 3) * 2 + (i & 1), S[i]);
        } else {
#pragma unroll 1
            for (int c = c0; c < min(c0 + D / 2, nv); c += 16) {
                uint32_t r[16];
                tmem_ld16(tlane + G::kState + c, r);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) keep(row, c + e, __uint_as_float(r[e]));
            }
        }
        if (!alive && tid == 0) report(args.status, SEMICRF_ERR_DEVICE_TIMEOUT);
    }
    tc_before_sync();
    __syncthreads();
    if (warp == 8) tmem_free(tm, G::kCols);
}

using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                            const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Encode encoder()
{
    static const Encode fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<Encode>(p);
    }();
    return fn;
}

// The map of a [B][T][H][d] operand: boxes of 64 columns and 128 positions of one head.
bool make_map(CUtensorMap *m, const void *p, const long long (&st)[3], int d, const LaArgs &a)
{
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)a.H, (cuuint64_t)a.T, (cuuint64_t)a.B};
    // (an axis of length one may have any stride; the map wants one it could use)
    auto bytes = [](long long stride, int length) { return length > 1 ? (cuuint64_t)stride * 2 : (cuuint64_t)256; };
    const cuuint64_t strides[3] = {bytes(st[2], a.H), bytes(st[1], a.T), bytes(st[0], a.B)};
    const cuuint32_t box[4] = {64, 1, kChunk, 1}, step[4] = {1, 1, 1, 1};
    return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims, strides, box, step,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

using Kernel = void (*)(LaArgs, LaMaps);

// The kernel for a width and a pass, and its shared memory.
Kernel kernel_of(int width, bool state_only, int *smem)
{
    if (state_only) {
        *smem = width == 64 ? StateCfg<64>::kSmem : StateCfg<128>::kSmem;
        return width == 64 ? la_state_kernel<64> : la_state_kernel<128>;
    }
    *smem = width == 64 ? TmaCfg<64>::kSmem : TmaCfg<128>::kSmem;
    return width == 64 ? la_tma_kernel<64> : la_tma_kernel<128>;
}

}  // namespace

// Whether the copy engine should be able to address every operand of these widths: aligned,
// and no axis repeated by a stride of 0 (an expanded tensor's).  la_tma_maps has the last word.
bool la_tma_ok(const LaArgs &a, int dtype)
{
    if (dtype != SEMICRF_BF16 || !encoder()) return false;
    for (int i = 0; i < a.nwalk; ++i) {
        const LaWalk &w = a.w[i];
        if (w.dk > 128 || w.dv > 128 || !w.q_vec || !w.k_vec || !w.v_vec || !w.o_vec) return false;
        const int length[3] = {a.B, a.T, a.H};
        for (int j = 0; j < 3; ++j)
            if (length[j] > 1 && (w.qs[j] == 0 || w.ks[j] == 0 || w.vs[j] == 0)) return false;
    }
    return true;
}

// The maps of all operands; false where the driver's encoder refuses one.
bool la_tma_maps(const LaArgs &a, LaMaps *maps)
{
    for (int state = 0; state < (a.nseg > 1 ? 2 : 1); ++state) {
        int smem;
        const Kernel k = kernel_of(a.width, state, &smem);
        // (also binds the device's context to a thread that makes its first call, which the
        // encoder wants: the backward pass runs in a thread of its own)
        if (cudaFuncSetAttribute(reinterpret_cast<const void *>(k), cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return false;
    }
    for (int i = 0; i < a.nwalk; ++i) {
        const LaWalk &w = a.w[i];
        auto &m = maps->w[i];
        if (!make_map(&m.q, w.q, w.qs, w.dk, a) || !make_map(&m.k, w.k, w.ks, w.dk, a) ||
            !make_map(&m.v, w.v, w.vs, w.dv, a) || !make_map(&m.o, w.o, w.os, w.dv, a))
            return false;
    }
    return true;
}

cudaError_t launch_la_tma(const LaArgs &a, const LaMaps &maps, bool state_only, cudaStream_t st, int *n)
{
    int smem;
    const Kernel k = kernel_of(a.width, state_only, &smem);
    return timed_launch(st, n, [&] { k<<<dim3(a.B * a.H * a.nseg, a.nwalk), kThreads, smem, st>>>(a, maps); });
}

cudaError_t la_tma_found(int32_t *to) { return read_found(to); }
cudaError_t la_tma_clear_found(cudaStream_t st) { return clear_found(st); }

}  // namespace semicrf
