// tensor_core.cuh -- sm_100a matrix instructions (tcgen05) on tiles that threads
// write to shared memory: descriptors, tensor-memory loads and stores, bounded waits.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace semicrf {

// A tile X[R][D] of 16-bit values lies in shared memory as 8 x 8 blocks: 8 rows of
// 16 bytes, 128 bytes in all, the blocks of one column of 8 values one after the
// other: row r, column d at (d/8) * col + r * 16 + (d%8) * 2.  col is 16 R, or
// tile_col(R) = 16 R + 16 where threads write along rows: eight lanes with one row's
// pieces then fall into eight different bank groups.  The same image serves both
// ways a product can read it:
//   contraction over d (K-major):   row groups 128 apart, k groups col apart
//   contraction over r (MN-major):  d groups col apart, k groups 128 apart
// so no tile is ever transposed or kept twice.
__host__ __device__ constexpr int tile_col(int R) { return R * 16 + 16; }

// Descriptor of an unswizzled operand: start address, leading and stride byte
// offsets in 16-byte units, and the constant 1 in bits 46..48.
__device__ __forceinline__ uint64_t mma_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo)
{
    return (uint64_t)((saddr & 0x3ffff) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 |
           (uint64_t)1 << 46;
}

__device__ __forceinline__ uint64_t desc_k(uint32_t tile, int col) { return mma_desc(tile, col, 128); }    // K-major
__device__ __forceinline__ uint64_t desc_mn(uint32_t tile, int col) { return mma_desc(tile, 128, col); }   // MN-major

// Tiles that the copy engine writes: 64 columns (128 bytes) a row, the 16-byte pieces
// of row r exchanged by r % 8 (128-byte swizzle), 8 rows to 1024 bytes; wider tiles are
// several of them.  Both readings again, steps along k within a tile: K-major 32 bytes
// for 16 columns, MN-major 2048 bytes for 16 rows (the next 64 columns `wide` apart).
__device__ __forceinline__ int swz(int r, int piece) { return r * 128 + ((piece ^ (r & 7)) << 4); }
__device__ __forceinline__ uint64_t desc_swz(uint32_t tile, int wide)
{
    return mma_desc(tile, wide, 1024) | (uint64_t)2 << 61;
}

// Instruction descriptor: bf16 x bf16 -> fp32, M x N, operands K-major unless flagged.
__host__ __device__ constexpr uint32_t mma_idesc(int M, int N, bool a_mn, bool b_mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
           (uint32_t)(N >> 3) << 17 | (uint32_t)(M >> 4) << 24;
}

// The instructions below belong to one thread: they stand in a branch of the lane that
// elect_lane names, with the warp whole before and behind it.  (Under a predicate of
// the whole warp instead, a commit after a loop that one lane had left late signalled
// its barrier twice.)
__device__ __forceinline__ bool elect_lane()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
                 : "memory");
}

// A in tensor memory: row i in lane i, two 16-bit values of the contraction in each column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
                 : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t mbar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(mbar) : "memory");
}

__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}

__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
}

__device__ __forceinline__ void tc_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// shared-memory writes of this thread become visible to the matrix unit
__device__ __forceinline__ void smem_to_mma() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 16 columns of this warp's 32 lanes; `addr` carries the lane quadrant in bits 16..31.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr));
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
                   "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
                   "=r"(r[30]), "=r"(r[31])
                 : "r"(addr));
}

// 16 lanes and 32 columns spread over all 32 threads: r[4j + 2a + b] is lane
// (thread / 4) + 8 a, column 8 j + 2 (thread % 4) + b.
__device__ __forceinline__ void tmem_ld16x256(uint32_t addr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr));
}

__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

__device__ __forceinline__ void mbar_init(uint32_t mbar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(mbar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_expect(uint32_t mbar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(mbar), "r"(bytes) : "memory");
}

// One box of a tensor [b][t][h][column] to shared memory, and back.
__device__ __forceinline__ void tma_load(uint32_t dst, const void *map, int col, int h, int t, int b, uint32_t mbar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
                 "l"(map), "r"(col), "r"(h), "r"(t), "r"(b), "r"(mbar)
                 : "memory");
}

__device__ __forceinline__ void tma_store(uint32_t src, const void *map, int col, int h, int t, int b)
{
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(map),
                 "r"(src), "r"(col), "r"(h), "r"(t), "r"(b)
                 : "memory");
}

__device__ __forceinline__ void tma_store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// the shared memory of every committed store may be written again / the stores are done
__device__ __forceinline__ void tma_store_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_store_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Waits for the phase of `parity`; false once 2^31 cycles (about a second) have passed.
__device__ __forceinline__ bool mbar_wait_bounded(uint32_t mbar, uint32_t parity)
{
    const long long t0 = clock64();
    for (;;) {
        uint32_t done;
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(done)
                     : "r"(mbar), "r"(parity)
                     : "memory");
        if (done) return true;
        if (clock64() - t0 > (1LL << 31)) return false;
    }
}

// Two floats to bf16, nearest, a low and b high; what rounds past the largest finite value
// becomes that value.
__device__ __forceinline__ uint32_t bf16_pair_finite(float a, float b)
{
    uint32_t r;
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Two floats as sums of NT bf16 terms, packed (a low, b high), each the nearest to what is
// left.  Three terms hold a float exactly; two leave 2^-17 of the value at most, one 2^-9.
// (First terms that are cut off instead, which needs no conversion, leave twice as much of
// one sign, and the calls take the same time.)  All but the last term are finite: float32's
// largest values, which bf16 rounds to infinity, are sums of finite terms too.
template <int NT>
__device__ __forceinline__ void split2(float a, float b, uint32_t (&t)[NT])
{
#pragma unroll
    for (int i = 0; i + 1 < NT; ++i) {
        t[i] = bf16_pair_finite(a, b);
        a -= __uint_as_float(t[i] << 16);
        b -= __uint_as_float(t[i] & 0xffff0000u);
    }
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    t[NT - 1] = *reinterpret_cast<const uint32_t *>(&r);
}

// The floats that NT packed terms stand for.
template <int NT>
__device__ __forceinline__ void join2(const uint32_t (&t)[NT], float &a, float &b)
{
    a = __uint_as_float(t[NT - 1] << 16);
    b = __uint_as_float(t[NT - 1] & 0xffff0000u);
#pragma unroll
    for (int i = NT - 2; i >= 0; --i) {
        a += __uint_as_float(t[i] << 16);
        b += __uint_as_float(t[i] & 0xffff0000u);
    }
}

}  // namespace semicrf
