// Warp-level tensor-core helpers of the prompt kernels, and the split of fp32
// numbers into two binary16 halves they multiply.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

namespace stepq {
namespace dev {

// D = A B + D: A 16 x 16 (rows), B 16 x 8 (columns), binary16, sums in fp32.
// With g = lane / 4, c = lane % 4: a0 holds A[g][2c..], a1 A[g+8][2c..], a2
// A[g][2c+8..], a3 A[g+8][2c+8..]; b0 B[2c..][g], b1 B[2c+8..][g]; d0, d1
// D[g][2c..], d2, d3 D[g+8][2c..].
__device__ __forceinline__ void mma16816(float *d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four 8 x 8 matrices of 16-bit elements; lane l gives the address of row l % 8
// of matrix l / 8.
__device__ __forceinline__ void ldsm4(uint32_t *r, uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t *r, uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// The same into two right operands of two registers each.
__device__ __forceinline__ void ldsm4(uint32_t *p, uint32_t *q, uint32_t addr)
{
    uint32_t r[4];
    ldsm4(r, addr);
    p[0] = r[0]; p[1] = r[1]; q[0] = r[2]; q[1] = r[3];
}
__device__ __forceinline__ void ldsm4_t(uint32_t *p, uint32_t *q, uint32_t addr)
{
    uint32_t r[4];
    ldsm4_t(r, addr);
    p[0] = r[0]; p[1] = r[1]; q[0] = r[2]; q[1] = r[3];
}

// Powers of two that bring a row whose largest magnitude is m near 2^13, and
// back.  A value is then held as two binary16 halves, hi + lo, to 22 bits of
// itself or 2^-38 of the row's largest, whichever is coarser: the products
// hi hi + hi lo + lo hi keep fp32's precision relative to the row.
__device__ __forceinline__ void row_scale(float m, float *scale, float *back)
{
    int e = (int)((__float_as_uint(m) >> 23) & 255);
    e = e < 14 ? 14 : (e > 254 ? 254 : e);
    *scale = __uint_as_float((uint32_t)(267 - e) << 23);
    *back = __uint_as_float((uint32_t)(e - 13) << 23);
}

__device__ __forceinline__ uint32_t pack_half(float x, float y)
{
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// hi and lo halves of two scaled numbers.
__device__ __forceinline__ void split_half(float2 x, uint32_t *hi, uint32_t *lo)
{
    const __half2 h = __float22half2_rn(x);
    *hi = *reinterpret_cast<const uint32_t *>(&h);
    float a, b;  // x - h, exact (0xbc00 is -1)
    asm("{\n\t.reg .b16 l, u, m;\n\tmov.b32 {l, u}, %2;\n\tmov.b16 m, 0xbc00;\n\t"
        "fma.rn.f32.f16 %0, l, m, %3;\n\tfma.rn.f32.f16 %1, u, m, %4;\n\t}"
        : "=f"(a), "=f"(b)
        : "r"(*hi), "f"(x.x), "f"(x.y));
    *lo = pack_half(a, b);
}
__device__ __forceinline__ void split_half(float x, float y, uint32_t *hi, uint32_t *lo) { split_half(make_float2(x, y), hi, lo); }

}  // namespace dev
}  // namespace stepq
