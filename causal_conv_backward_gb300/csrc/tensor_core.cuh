// tensor_core.cuh - tcgen05 instructions on one CTA's tensor memory, the
// descriptors of their operands, and 32-bit values as two fp16 terms.
#pragma once

#include "device_common.cuh"

namespace mcc1d {

// ------------------------------------------------------------------ tensor memory
// An address is a lane (bits 16..31) and a 32-bit column (bits 0..15). A warp
// reaches the 32 lanes that its number modulo 4 stands for.
__device__ __forceinline__ void tmem_alloc(uint32_t smem_slot, int columns)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_slot), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t at, int columns)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Columns of this thread's lane. The loaded registers are valid after tmem_wait,
// which names them so that nothing uses them earlier.
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                   "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};"
                 :
                 : "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(at)
                 : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
                 :
                 : "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
                   "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(at)
                 : "memory");
}

// ------------------------------------------------------------------ operands
// A matrix of 16-bit values in shared memory as panels of 64 adjacent values:
// rows of 128 bytes, each eight of them with their 16-byte pieces exchanged (piece
// p of row r at p ^ (r % 8)), panels aligned to 1024 bytes.
__device__ __forceinline__ uint32_t panel_at(int row, int piece) { return (uint32_t)(row * 128 + ((piece ^ (row & 7)) * 16)); }

constexpr uint64_t kDescSwizzled = (uint64_t)1 << 46 | (uint64_t)2 << 61;
// Rows are the operand's rows (its M or N), the panel's 64 values run along the sum.
__device__ __forceinline__ uint64_t desc_rows(uint32_t smem)
{
    return kDescSwizzled | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 16 | (smem >> 4);
}
// Rows run along the sum, the panel's 64 values (and those of the panel `next`
// bytes on) are the operand's N.
__device__ __forceinline__ uint64_t desc_columns(uint32_t smem, uint32_t next)
{
    return kDescSwizzled | (uint64_t)(1024 >> 4) << 32 | (uint64_t)(next >> 4) << 16 | (smem >> 4);
}

// fp16 operands, fp32 sums, M = 128; A or B by columns where its rows run along the sum.
__device__ constexpr uint32_t mma_kind(int N, bool b_columns, bool a_columns = false)
{
    return 1u << 4 | (a_columns ? 1u << 15 : 0u) | (b_columns ? 1u << 16 : 0u) | (uint32_t)(N / 8) << 17 | (128u / 16) << 24;
}

// D (+)= A B^T over 16 values of the sum, A in tensor memory (8 columns of
// packed pairs), by one thread.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t kind, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(kind), "r"((uint32_t)add)
        : "memory");
}
// The same with A in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(kind), "r"((uint32_t)add)
        : "memory");
}
// The barrier gets one arrival when all of this thread's products so far are done.
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// This thread's writes to shared memory are seen by copies and products that
// are ordered after it.
__device__ __forceinline__ void shared_to_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Whether a barrier's phase is over, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// ------------------------------------------------------------------ two terms
// The power of two that takes a largest magnitude to 2^14..2^15 (1 for zero; for
// infinity, which a bound may be where no value is, what takes the largest number
// there), and its reciprocal. A value times it is hi + lo, two fp16
// numbers, with 22 bits from the largest down to 2^-24 of it, and an absolute
// error of 2^-40 of the largest below.
__device__ __forceinline__ float scale_for(float largest)
{
    const int e = (int)(__float_as_uint(largest) >> 23);         // sign 0
    return e == 0 ? 1.f : __uint_as_float((uint32_t)min(268 - min(e, 254), 253) << 23);
}
__device__ __forceinline__ float inverse_scale(float scale)
{
    return __uint_as_float((254u << 23) - __float_as_uint(scale));
}

__device__ __forceinline__ uint32_t pack_half2(float2 v)
{
    union {
        __half2 h;
        uint32_t u;
    } c;
    c.h = __floats2half2_rn(v.x, v.y);
    return c.u;
}
// Two scaled values as packed first and second terms.
__device__ __forceinline__ void two_terms(float2 v, uint32_t &hi, uint32_t &lo)
{
    union {
        __half2 h;
        uint32_t u;
    } c;
    c.h = __floats2half2_rn(v.x, v.y);
    hi = c.u;
    lo = pack_half2(sub2(v, __half22float2(c.h)));
}

// A tile of a described tensor [batch,head,token,value] to shared memory (128-byte
// aligned), completing on an mbarrier; `x` is a multiple of eight.
__device__ __forceinline__ void tile_g2s(uint32_t dst, const void *map, int x, int token, int head, int batch, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst), "l"(map),
                 "r"(x), "r"(token), "r"(head), "r"(batch), "r"(bar)
                 : "memory");
}

}  // namespace mcc1d
