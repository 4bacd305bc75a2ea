// tensor_core.cuh -- sm_100a matrix instructions (tcgen05) on tiles that threads
// write to shared memory: descriptors, tensor-memory loads and stores, bounded waits.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace semicrf {

// A tile X[R][D] of 16-bit values lies in shared memory as 8 x 8 blocks: 8 rows of
// 16 bytes, 128 bytes in all.  Block (r/8, d/8) starts at (d/8) * col + (r/8) * 128,
// where col = tile_col(R) pads each column of blocks by 16 bytes: eight lanes that
// write one row's pieces then fall into eight different bank groups.  The same image
// serves both ways a product can read it:
//   contraction over d (K-major):   row groups 128 apart, k groups col apart
//   contraction over r (MN-major):  d groups col apart, k groups 128 apart
// so no tile is ever transposed or kept twice.
__host__ __device__ constexpr int tile_col(int R) { return R * 16 + 16; }
__host__ __device__ constexpr int tile_bytes(int R, int D) { return D / 8 * tile_col(R); }
__device__ __forceinline__ int tile_at(int R, int r, int d8) { return d8 * tile_col(R) + (r >> 3) * 128 + (r & 7) * 16; }

// Descriptor of an unswizzled operand: start address, leading and stride byte
// offsets in 16-byte units, and the constant 1 in bits 46..48.
__device__ __forceinline__ uint64_t mma_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo)
{
    return (uint64_t)((saddr & 0x3ffff) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 |
           (uint64_t)1 << 46;
}

// K-major operand: step k (16 values of the contraction) of a tile with R rows.
__device__ __forceinline__ uint64_t desc_k(uint32_t tile, int R, int k)
{
    return mma_desc(tile + 2 * k * tile_col(R), tile_col(R), 128);
}

// MN-major operand (contraction over the tile's rows): step k (16 rows).
__device__ __forceinline__ uint64_t desc_mn(uint32_t tile, int R, int k)
{
    return mma_desc(tile + 2 * k * 128, 128, tile_col(R));
}

// Instruction descriptor: bf16 x bf16 -> fp32, M x N, operands K-major unless flagged.
__host__ __device__ constexpr uint32_t mma_idesc(int M, int N, bool a_mn, bool b_mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
           (uint32_t)(N >> 3) << 17 | (uint32_t)(M >> 4) << 24;
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

// v = t[0] + t[1] + ... in bf16 terms: each takes the nearest value of what is left,
// so n terms carry 8 n bits of the float.
template <int NT>
__device__ __forceinline__ void bf16_terms(float v, __nv_bfloat16 (&t)[NT])
{
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        t[i] = __float2bfloat16_rn(v);
        if (i + 1 < NT) v -= __bfloat162float(t[i]);
    }
}

}  // namespace semicrf
