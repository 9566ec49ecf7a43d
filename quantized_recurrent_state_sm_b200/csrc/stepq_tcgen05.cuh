// Fifth-generation tensor cores: tensor memory, matrix products with the left
// operand in tensor memory and the right one in shared memory, as inline PTX.
#pragma once

#include <cstdint>

#include "stepq_device.cuh"

namespace stepq {
namespace tc {

// Tensor memory of a CTA: 128 lanes x columns of 32 bits.  An address holds the
// lane in its upper and the column in its lower half.  Warp w reaches lanes
// 32 (w % 4) .. + 31.  Allocation and release: one whole warp, the same one.
__device__ __forceinline__ void alloc(uint32_t *slot, uint32_t columns)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dev::smem_addr(slot)), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc(uint32_t addr, uint32_t columns)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 (or 8) columns of the warp's lanes: register i of a lane holds column
// i.  The wait for a load is part of its statement, so that no use of the
// registers can be moved before it.
__device__ __forceinline__ void ld16(uint32_t *r, uint32_t addr)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void st8(uint32_t addr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Right operand in shared memory in rows of 128 bytes whose 16-byte chunks are
// permuted by the row (the 128-byte swizzle; bases at multiples of 1024 bytes).
// stride: bytes from one group of eight rows to the next; lead: for an operand
// whose rows run along the product's inner dimension, bytes from one 64-column
// half to the next (unused otherwise).
__device__ __forceinline__ uint64_t desc(uint32_t smem, uint32_t lead, uint32_t stride)
{
    return (uint64_t)((smem & 0x3ffff) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}

// 128 rows, n columns, binary16 operands, fp32 sums.  inner_rows: the right
// operand's rows in memory run along the inner dimension (it is read
// transposed).
__host__ __device__ constexpr uint32_t idesc(int n, bool inner_rows)
{
    return (1u << 4) | ((inner_rows ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// One lane of a converged warp.  Products issued under this predicate go out at
// the tensor cores' rate (32 cycles for 64 columns); under a comparison of the
// lane number, whose branch the compiler takes for divergent, each takes about
// 55 cycles to issue.
__device__ __forceinline__ bool elect()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// D (tensor memory) = A (tensor memory, two binary16 numbers a column) B, plus D
// if `add`; 16 inner elements.  One thread.
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"((uint32_t)add)
        : "memory");
}

// The barrier gets an arrival when the products issued so far are done.
__device__ __forceinline__ void commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(dev::smem_addr(bar)) : "memory");
}

}  // namespace tc
}  // namespace stepq
