// The operands of a prompt's blocks: everything of a block of 64 tokens that
// does not depend on the state, for all blocks at once.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "stepq_device.cuh"
#include "stepq_mma.cuh"
#include "stepq_prompt_blocks.cuh"

namespace stepq {
namespace {

using dev::ldsm4;
using dev::ldsm4_t;
using dev::mma16816;

constexpr unsigned kFull = 0xffffffffu;

// Four consecutive elements.
__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __half *p)
{
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&v.x)), b = __half22float2(*reinterpret_cast<const __half2 *>(&v.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p)
{
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xffff0000u));
}

// Largest magnitude of a warp's numbers (as integers: the order is the same).
__device__ __forceinline__ float warp_max(float4 x)
{
    const float m = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
    return __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(m)));
}

// One row of an operand (4 elements a lane) as scaled halves into a tile, in
// shared or global memory; returns the row's unscale.  NP: halves kept.  EXACT:
// binary16 inputs are their own halves.
template <int NP, bool EXACT>
__device__ __forceinline__ float put_row(float4 x, int row, int l, char *tile)
{
    float scale = 1.f, back = 1.f;
    if (!EXACT) dev::row_scale(warp_max(x), &scale, &back);
    uint32_t hi[2], lo[2];
    dev::split_half(x.x * scale, x.y * scale, &hi[0], &lo[0]);
    dev::split_half(x.z * scale, x.w * scale, &hi[1], &lo[1]);
    const int at = tile_at(row, 4 * l);
    *reinterpret_cast<uint2 *>(tile + at) = make_uint2(hi[0], hi[1]);
    if (NP == 2) *reinterpret_cast<uint2 *>(tile + kTileBytes + at) = make_uint2(lo[0], lo[1]);
    return back;
}

// Bulk copies from shared memory to the scratch, by one thread; the shared
// memory may be written again after the wait.
__device__ __forceinline__ void bulk_s2g(void *dst, const void *src, int bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(dev::smem_addr(src)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// acc[j] = rows 16 m .. 16 m + 15 of A times rows 8 j .. of B transposed, for
// the column tiles j < tiles (a multiple of 2): A and B operand tiles in
// shared memory.  Each pass goes over all sums before it returns to the first.
// Where products are three, the loop's turns stay apart, for its instructions to
// stay near (prompts of 16 requests in fp32 265 us instead of 271); of one, not
// (one long prompt in bf16 592 us instead of 598).
template <int NP>
__device__ __forceinline__ void rows_product(float (*acc)[4], const char *A, const char *B, int m, int tiles)
{
    const int l = threadIdx.x & 31;
    const uint32_t a0 = dev::smem_addr(A), b0 = dev::smem_addr(B);
    const int arow = 16 * m + (l & 7) + ((l >> 3) & 1) * 8, acol = (l >> 4) * 8;  // of the A matrices
    const int brow = (l & 7) + (l >> 4) * 8, bcol = ((l >> 3) & 1) * 8;           // of two column tiles
#pragma unroll(NP == 2 ? 1 : kDK / 16)
    for (int i = 0; i < kDK / 16; i++) {
        uint32_t ah[4], al[4];
        ldsm4(ah, a0 + tile_at(arow, 16 * i + acol));
        if (NP == 2) ldsm4(al, a0 + kTileBytes + tile_at(arow, 16 * i + acol));
        uint32_t b[kC / 8][2];
#pragma unroll
        for (int j = 0; j < kC / 8; j += 2)
            if (j < tiles) ldsm4(b[j], b[j + 1], b0 + tile_at(8 * j + brow, 16 * i + bcol));
        if (NP == 2) {
#pragma unroll
            for (int j = 0; j < kC / 8; j++)
                if (j < tiles) mma16816(acc[j], al[0], al[1], al[2], al[3], b[j][0], b[j][1]);
        }
#pragma unroll
        for (int j = 0; j < kC / 8; j++)
            if (j < tiles) mma16816(acc[j], ah[0], ah[1], ah[2], ah[3], b[j][0], b[j][1]);
        if (NP == 2) {
#pragma unroll
            for (int j = 0; j < kC / 8; j += 2)
                if (j < tiles) ldsm4(b[j], b[j + 1], b0 + kTileBytes + tile_at(8 * j + brow, 16 * i + bcol));
#pragma unroll
            for (int j = 0; j < kC / 8; j++)
                if (j < tiles) mma16816(acc[j], ah[0], ah[1], ah[2], ah[3], b[j][0], b[j][1]);
        }
    }
}

// ---- the inverse and the squares ---------------------------------------------
//
// A (strictly lower triangular, [64][64]) and P are held as accumulators: warp m
// of 0-3 has rows 16 m .. of A, all columns, and warp m or 7 - m those of P.  With
// T = (I + A)^-1 in blocks of 16: T_mm by substitution, then row by row
//   T_m = T_mm - (T_mm A_m) T_(<m),
// products on the tensor cores; P T likewise.  A left operand comes from the
// accumulators of its own warp, a right one from halves in shared memory, whose
// row scales (inner indices of the product) are multiplied into the left one.

// Rows 16 m .. that a warp has: a warp of the second four shares its scheduler with
// one of the first, and m + 1 blocks of columns count, so the orders are opposite.
__device__ __forceinline__ int rows_of(int w) { return w < 4 ? w : 7 - w; }

constexpr int kDiagLd = 20;
struct Squares {
    __align__(128) char a[kSquareBytes], t[kSquareBytes];  // halves of A, and later of P T; of T
    float diag[4][16][kDiagLd], tdiag[4][16][kDiagLd];  // the diagonal blocks of A and T
    float a_back[kC], t_back[kC], p_back[kC];           // unscales of the rows
};

__device__ __forceinline__ float quad_max(float m)
{
    m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
    return fmaxf(m, __shfl_xor_sync(kFull, m, 2));
}

// Scales of rows g and g + 8 of an accumulator of which `tiles` column tiles count.
template <int N>
__device__ __forceinline__ void row_scales(const float (*x)[4], int tiles, float *scale, float *back)
{
    float m0 = 0.f, m1 = 0.f;
#pragma unroll
    for (int j = 0; j < N; j++)
        if (j < tiles) {
            m0 = fmaxf(m0, fmaxf(fabsf(x[j][0]), fabsf(x[j][1])));
            m1 = fmaxf(m1, fmaxf(fabsf(x[j][2]), fabsf(x[j][3])));
        }
    dev::row_scale(quad_max(m0), &scale[0], &back[0]);
    dev::row_scale(quad_max(m1), &scale[1], &back[1]);
}

// `tiles` column tiles of an accumulator as halves into a square's rows 16 m ..
template <int N>
__device__ __forceinline__ void put_tiles(const float (*x)[4], int tiles, const float *scale, char *square, int m)
{
    const int l = threadIdx.x & 31, g = l >> 2, c = l & 3;
#pragma unroll
    for (int j = 0; j < N; j++)
        if (j < tiles)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                uint32_t hi, lo;
                dev::split_half(x[j][2 * e] * scale[e], x[j][2 * e + 1] * scale[e], &hi, &lo);
                char *at = square + square_at(16 * m + g + 8 * e, 8 * j + 2 * c);
                *reinterpret_cast<uint32_t *>(at) = hi;
                *reinterpret_cast<uint32_t *>(at + kSquareBytes / 2) = lo;
            }
}

// One block of a product with T, in place: the 16 columns J of x (tiles 2 J and 2 J
// + 1) times T's 16 rows J, which reach columns 16 J + 15.  The columns before hold
// what earlier blocks gave and are added to; those of J itself are done with and
// hold their sum's first share.
template <int J>
__device__ __forceinline__ void add_block(float (*x)[4], const Squares &sq)
{
    const int l = threadIdx.x & 31, c = l & 3;
    float y[2][4], scale[2], back[2];
#pragma unroll
    for (int e = 0; e < 2; e++) {
        const float2 f = *reinterpret_cast<const float2 *>(&sq.t_back[16 * J + 8 * e + 2 * c]);
        y[e][0] = x[2 * J + e][0] * f.x; y[e][1] = x[2 * J + e][1] * f.y; y[e][2] = x[2 * J + e][2] * f.x; y[e][3] = x[2 * J + e][3] * f.y;
    }
    row_scales<2>(y, 2, scale, back);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 2; e++) {
        dev::split_half(y[e][0] * scale[0], y[e][1] * scale[0], &hi[2 * e], &lo[2 * e]);
        dev::split_half(y[e][2] * scale[1], y[e][3] * scale[1], &hi[2 * e + 1], &lo[2 * e + 1]);
    }
    const uint32_t y0 = dev::smem_addr(sq.t);
#pragma unroll
    for (int j = 0; j < 2 * J + 2; j += 2) {
        uint32_t b[2][2], d[2][2];
        float p[2][4] = {};
        const uint32_t at = y0 + square_at(16 * J + (l & 15), 8 * j + (l >> 4) * 8);
        ldsm4_t(b[0], b[1], at);
        ldsm4_t(d[0], d[1], at + kSquareBytes / 2);
#pragma unroll
        for (int e = 0; e < 2; e++) mma16816(p[e], lo[0], lo[1], lo[2], lo[3], b[e][0], b[e][1]);
#pragma unroll
        for (int e = 0; e < 2; e++) mma16816(p[e], hi[0], hi[1], hi[2], hi[3], d[e][0], d[e][1]);
#pragma unroll
        for (int e = 0; e < 2; e++) mma16816(p[e], hi[0], hi[1], hi[2], hi[3], b[e][0], b[e][1]);
#pragma unroll
        for (int e = 0; e < 2; e++)
#pragma unroll
            for (int i = 0; i < 4; i++) x[j + e][i] = j == 2 * J ? p[e][i] * back[i >> 1] : fmaf(p[e][i], back[i >> 1], x[j + e][i]);
    }
}

// From A and P (the accumulators of warps 0-3 and PW .. PW + 3, zero above the
// diagonal) to the halves of T and P T in sq.  Ends with a barrier.
template <bool DELTA, int PW>
__device__ __forceinline__ void finish(float (*acc)[4], float (*accp)[4], Squares &sq)
{
    const int tid = threadIdx.x, w = tid >> 5, l = tid & 31, g = l >> 2, c = l & 3, m = rows_of(w);
    float scale[2], back[2];
    if constexpr (DELTA) {
        if (w < 4) {
            row_scales<6>(acc, 2 * m, scale, back);
            put_tiles<6>(acc, 2 * m, scale, sq.a, m);
            if (c == 0) {
                sq.a_back[16 * m + g] = back[0];
                sq.a_back[16 * m + g + 8] = back[1];
            }
#pragma unroll
            for (int j = 0; j < 8; j += 2)
                if (j == 2 * m)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        *reinterpret_cast<float2 *>(&sq.diag[m][g][8 * e + 2 * c]) = make_float2(acc[j + e][0], acc[j + e][1]);
                        *reinterpret_cast<float2 *>(&sq.diag[m][g + 8][8 * e + 2 * c]) = make_float2(acc[j + e][2], acc[j + e][3]);
                    }
        }
        __syncthreads();
        if (tid < kC) {  // T_mm, a column a thread
            const int b = tid >> 4, j = tid & 15;
            float x[16];
#pragma unroll
            for (int r = 0; r < 16; r++) {
                float s0 = 0.f, s1 = 0.f;
#pragma unroll
                for (int i = 0; i < r; i += 4) {
                    const float4 y = *reinterpret_cast<const float4 *>(&sq.diag[b][r][i]);
                    s0 = fmaf(y.x, x[i], s0);
                    if (i + 1 < r) s1 = fmaf(y.y, x[i + 1], s1);
                    if (i + 2 < r) s0 = fmaf(y.z, x[i + 2], s0);
                    if (i + 3 < r) s1 = fmaf(y.w, x[i + 3], s1);
                }
                x[r] = r < j ? 0.f : (r == j ? 1.f : -(s0 + s1));
                sq.tdiag[b][r][j] = x[r];
            }
        }
        __syncthreads();
        float td[2][4];  // T_mm as an accumulator of two column tiles
        if (w < 4) {
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const float2 x = *reinterpret_cast<const float2 *>(&sq.tdiag[m][g][8 * e + 2 * c]), y = *reinterpret_cast<const float2 *>(&sq.tdiag[m][g + 8][8 * e + 2 * c]);
                td[e][0] = x.x; td[e][1] = x.y; td[e][2] = y.x; td[e][3] = y.y;
            }
            if (m == 0) {
                row_scales<2>(td, 2, scale, back);
                put_tiles<2>(td, 2, scale, sq.t, 0);
                if (c == 0) {
                    sq.t_back[g] = back[0];
                    sq.t_back[g + 8] = back[1];
                }
            } else {
                float x[2][4];
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const float2 f = *reinterpret_cast<const float2 *>(&sq.a_back[16 * m + 8 * e + 2 * c]);
                    x[e][0] = td[e][0] * f.x; x[e][1] = td[e][1] * f.y; x[e][2] = td[e][2] * f.x; x[e][3] = td[e][3] * f.y;
                }
                row_scales<2>(x, 2, scale, back);
                // T_mm A_m takes A_m's place (the products of one block of 16 rows of A)
                float y[6][4] = {};
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    dev::split_half(x[e][0] * scale[0], x[e][1] * scale[0], &hi[2 * e], &lo[2 * e]);
                    dev::split_half(x[e][2] * scale[1], x[e][3] * scale[1], &hi[2 * e + 1], &lo[2 * e + 1]);
                }
                const uint32_t y0 = dev::smem_addr(sq.a);
#pragma unroll
                for (int j = 0; j < 6; j += 2) {
                    if (j >= 2 * m) continue;
                    uint32_t b[2][2], d[2][2];
                    const uint32_t at = y0 + square_at(16 * m + (l & 15), 8 * j + (l >> 4) * 8);
                    ldsm4_t(b[0], b[1], at);
                    ldsm4_t(d[0], d[1], at + kSquareBytes / 2);
#pragma unroll
                    for (int e = 0; e < 2; e++) mma16816(y[j + e], lo[0], lo[1], lo[2], lo[3], b[e][0], b[e][1]);
#pragma unroll
                    for (int e = 0; e < 2; e++) mma16816(y[j + e], hi[0], hi[1], hi[2], hi[3], d[e][0], d[e][1]);
#pragma unroll
                    for (int e = 0; e < 2; e++) mma16816(y[j + e], hi[0], hi[1], hi[2], hi[3], b[e][0], b[e][1]);
                }
#pragma unroll
                for (int j = 0; j < 6; j++) {
                    acc[j][0] = y[j][0] * back[0]; acc[j][1] = y[j][1] * back[0];
                    acc[j][2] = y[j][2] * back[1]; acc[j][3] = y[j][3] * back[1];
                }
            }
        }
        // T_0 is there.  Where T_j is, every later row takes its share of it at once,
        // and the next row is complete; P T grows beside, the warp that makes the next
        // row one turn behind.
        const bool has_p = w >= PW;
        auto turn = [&](auto J) {
            constexpr int j = decltype(J)::value;
            __syncthreads();
            if constexpr (j < 3) {
                if (w < 4 && m > j) add_block<j>(acc, sq);
                if (w < 4 && m == j + 1) {
#pragma unroll
                    for (int i = 0; i < 2 * j + 2; i++)
#pragma unroll
                        for (int e = 0; e < 4; e++) acc[i][e] = -acc[i][e];
#pragma unroll
                    for (int e = 0; e < 2; e++)
#pragma unroll
                        for (int i = 0; i < 4; i++) acc[2 * j + 2 + e][i] = td[e][i];
                    row_scales<2 * j + 4>(acc, 2 * j + 4, scale, back);
                    put_tiles<2 * j + 4>(acc, 2 * j + 4, scale, sq.t, j + 1);
                    if (c == 0) {
                        sq.t_back[16 * (j + 1) + g] = back[0];
                        sq.t_back[16 * (j + 1) + g + 8] = back[1];
                    }
                }
            }
            if constexpr (PW == 0 && j > 0) {
                if (m == j) add_block<j - 1>(accp, sq);
            }
            if (has_p && m >= j && !(PW == 0 && m == j + 1)) add_block<j>(accp, sq);
        };
        turn(std::integral_constant<int, 0>{});
        turn(std::integral_constant<int, 1>{});
        turn(std::integral_constant<int, 2>{});
        turn(std::integral_constant<int, 3>{});
    }
    if (w >= PW && w < PW + 4) {
        row_scales<8>(accp, 2 * m + 2, scale, back);
        put_tiles<8>(accp, 2 * m + 2, scale, sq.a, m);
        if (c == 0) {
            sq.p_back[16 * m + g] = back[0];
            sq.p_back[16 * m + g + 8] = back[1];
        }
    }
    fence_async();
    __syncthreads();
}

// The halves into the scratch (one thread; they may be written again after bulk_wait_read).
template <bool DELTA>
__device__ __forceinline__ void put_squares(const Squares &sq, uint8_t *inv_image, uint8_t *p_image)
{
    if (DELTA) bulk_s2g(inv_image, sq.t, kSquareBytes);
    bulk_s2g(p_image, sq.a, kSquareBytes);
    bulk_commit();
}

// What a CTA works on: a block of a live request.
struct Block {
    int b, t0, n;  // block of this launch, first token row, tokens
};

__device__ __forceinline__ bool find_block(const PromptArgs &a, int first_block, int b, Block *k)
{
    const int g = first_block + b, r = a.p.block_request[g];
    k->b = b;
    if (r < 0 || a.p.live[r] < 0) return false;
    k->t0 = a.p.starts[r] + a.p.block_first[g];
    k->n = min(kC, a.p.starts[r + 1] - k->t0);
    return true;
}

// ---------------------------------------------------------------------------
// One gate a head.  A CTA of four warps takes a block and a value head: K K^T and
// Q K^T on the tensor cores (16 rows a warp), the decays, the inverse and the
// squares.  Most of it is a chain of short steps, so what counts is how many
// CTAs lie side by side on an SM; value heads that share a query / key head make
// its products anew, and the first of them writes its operands.  The decay from
// token s to token t is the product of what is left of s at the end of its 16
// tokens, of the 16s between, and of t's 16 up to t; inside 16 tokens it is
// multiplied out.
// Measured: bf16, 128 blocks of 32 heads 121 us, 214 MB moved (47 % issue, 14 %
// of the tensor pipe); fp32, 101 blocks of 32 heads 150 us, where all products
// are three; plain, binary16, 64 blocks of 32 heads 31 us, without the inverse.
// ---------------------------------------------------------------------------
constexpr int kTileThreads = 128;

__device__ __forceinline__ void cp_async16(void *dst, const void *src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dev::smem_addr(dst)), "l"(src), "r"(in ? 16 : 0) : "memory");
}

// Where the 16-byte piece `part` of a row lies before the row is split: in the
// bytes of the row's halves.
template <class T>
__device__ __forceinline__ int raw_at(int row, int part)
{
    if constexpr (sizeof(T) == 2) return tile_at(row, 8 * part);
    return (part >> 4) * kTileBytes + ((part >> 3) & 1) * (kTileBytes / 2) + row * 128 + (part & 7) * 16;
}

template <class T, int V, int NP>
__global__ void __launch_bounds__(kTileThreads, NP == 1 ? 4 : 3) k_block_tiles(PromptArgs a, int first_block, Scratch sc)
{
    extern __shared__ __align__(128) char smem[];
    __shared__ float ek[kC], eq[kC], s_beta[kC], s_pre[kC], s_suf[kC], s_blk[4], s_diag[4][16][17];
    __shared__ double s_keep[2];
    const int tid = threadIdx.x, w = tid >> 5, l = tid & 31, g = l >> 2, c = l & 3;
    Block k;
    const int h = blockIdx.x % a.heads, hq = h / a.share;
    if (!find_block(a, first_block, blockIdx.x / a.heads, &k)) return;
    const int tok = tid & (kC - 1);
    float alpha = 1.f, beta = 0.f;
    if (tok < k.n) {
        alpha = a.alpha[(long long)(k.t0 + tok) * a.heads + h];
        beta = a.beta[(long long)(k.t0 + tok) * a.heads + h];
    }
    // the rows as they are, into the places of their halves
    char *tk = smem, *tq = smem + NP * kTileBytes;
    const T *kg = static_cast<const T *>(a.k) + (long long)k.t0 * a.stride_k + hq * kDK, *qg = static_cast<const T *>(a.q) + (long long)k.t0 * a.stride_q + hq * kDK;
    constexpr int pieces = kDK * sizeof(T) / 16;  // of a row
#pragma unroll
    for (int i = 0; i < kC * pieces / kTileThreads; i++) {
        const int x = i * kTileThreads + tid, row = x / pieces, part = x % pieces, from = min(row, k.n - 1);
        const int at = raw_at<T>(row, part);
        cp_async16(tk + at, kg + from * a.stride_k + part * (16 / (int)sizeof(T)), row < k.n);
        cp_async16(tq + at, qg + from * a.stride_q + part * (16 / (int)sizeof(T)), row < k.n);
    }
    if (tid < kC) {
        float p = alpha, q = __shfl_down_sync(kFull, alpha, 1, 16);
        if ((l & 15) == 15) q = 1.f;
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) {
            const float x = __shfl_up_sync(kFull, p, d, 16), y = __shfl_down_sync(kFull, q, d, 16);
            if ((l & 15) >= d) p *= x;
            if ((l & 15) + d < 16) q *= y;
        }
        // what a block keeps of the state is multiplied up block after block: its
        // product is rounded once
        double all = (double)alpha;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) all *= __shfl_xor_sync(kFull, all, d);
        if (l == 0) s_keep[w] = all;
        s_pre[tid] = p;
        s_suf[tid] = q;
        s_beta[tid] = beta;
        if ((l & 15) == 15) s_blk[tid >> 4] = p;
    } else {
        float p = 1.f;
#pragma unroll
        for (int t = 0; t < 16; t++) {
            const float x = __shfl_sync(kFull, alpha, t, 16);
            if (t > (l & 15)) p *= x;
            s_diag[tok >> 4][t][l & 15] = p;
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    if constexpr (std::is_same<T, __half>::value) {  // binary16 rows are their own halves
        if (tid < kC) ek[tid] = eq[tid] = 1.f;
    } else {
#pragma unroll 4
        for (int i = 0; i < 16; i++) {
            const int row = 16 * w + i;
            const float4 x = load4(reinterpret_cast<const T *>(tk + raw_at<T>(row, 4 * l * (int)sizeof(T) / 16)) + 4 * l % (16 / (int)sizeof(T))),
                         y = load4(reinterpret_cast<const T *>(tq + raw_at<T>(row, 4 * l * (int)sizeof(T) / 16)) + 4 * l % (16 / (int)sizeof(T)));
            __syncwarp();
            const float bk = put_row<NP, false>(x, row, l, tk), bq = put_row<NP, false>(y, row, l, tq);
            if (l == 0) {
                ek[row] = bk;
                eq[row] = bq;
            }
        }
    }
    const bool writes = h % a.share == 0;
    if (writes) fence_async();
    __syncthreads();
    if (tid == 0 && writes) {
        const size_t at = ((size_t)k.b * (a.heads / a.share) + hq) * NP * kTileBytes;
        bulk_s2g(a.scratch + sc.k + at, tk, NP * kTileBytes);
        bulk_s2g(a.scratch + sc.q + at, tq, NP * kTileBytes);
        bulk_commit();
    }
    const int m = w;  // rows 16 m + g, + 8
    const float b0 = s_beta[16 * m + g], b1 = s_beta[16 * m + g + 8];
    // the products times the rows' unscales and the decays (and, for A, beta)
    auto decayed = [&](float (*x)[4], bool is_q) {
        const float *er = is_q ? eq : ek;
        const float r0 = er[16 * m + g] * (is_q ? 1.f : b0), r1 = er[16 * m + g + 8] * (is_q ? 1.f : b1);
        float f0 = s_pre[16 * m + g] * r0, f1 = s_pre[16 * m + g + 8] * r1;
#pragma unroll
        for (int jb = kC / 16 - 1; jb >= 0; jb--) {
            if (jb > m) continue;
            if (jb + 1 < m) {  // another 16 tokens between
                f0 *= s_blk[jb + 1];
                f1 *= s_blk[jb + 1];
            }
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int s = 16 * jb + 8 * e + 2 * c, si = 8 * e + 2 * c;
                float *y = x[2 * jb + e];
                const float2 u = *reinterpret_cast<const float2 *>(&ek[s]);
                if (jb == m) {
                    const int d = is_q ? 0 : 1;  // P has its diagonal, A does not
                    y[0] = si + d <= g ? y[0] * (s_diag[m][g][si] * r0 * u.x) : 0.f;
                    y[1] = si + 1 + d <= g ? y[1] * (s_diag[m][g][si + 1] * r0 * u.y) : 0.f;
                    y[2] = si + d <= g + 8 ? y[2] * (s_diag[m][g + 8][si] * r1 * u.x) : 0.f;
                    y[3] = si + 1 + d <= g + 8 ? y[3] * (s_diag[m][g + 8][si + 1] * r1 * u.y) : 0.f;
                } else {
                    const float2 q = *reinterpret_cast<const float2 *>(&s_suf[s]);
                    y[0] *= f0 * q.x * u.x; y[1] *= f0 * q.y * u.y;
                    y[2] *= f1 * q.x * u.x; y[3] *= f1 * q.y * u.y;
                }
            }
        }
    };
    float acc[kC / 8][4] = {}, accp[kC / 8][4] = {};
    rows_product<NP>(accp, tq, tk, m, 2 * m + 2);
    if (V != kLinear) rows_product<NP>(acc, tk, tk, m, 2 * m + 2);
    if (tid == 0 && writes) bulk_wait_read();
    __syncthreads();
    // the tiles are done with: their room holds the squares
    Squares &sq = *reinterpret_cast<Squares *>(smem);
    decayed(accp, true);
    if (V != kLinear) decayed(acc, false);
    finish<V != kLinear, 0>(acc, accp, sq);
    const size_t bh = (size_t)k.b * a.heads + h;
    if (tid == 0) put_squares<V != kLinear>(sq, a.scratch + sc.inv + bh * kSquareBytes, a.scratch + sc.p + bh * kSquareBytes);
    if (tid < kC) {
        float *sv = reinterpret_cast<float *>(a.scratch + sc.sv) + bh * kStateFloats;
        float *ov = reinterpret_cast<float *>(a.scratch + sc.ov) + bh * kOutFloats;
        const int b = tid >> 4;
        float ct = s_pre[tid], left = s_suf[tid];
        for (int i = 0; i < b; i++) ct *= s_blk[i];
        for (int i = b + 1; i < 4; i++) left *= s_blk[i];
        left *= ek[tid];
        sv[tid] = -s_beta[tid] * ct * ek[tid];
        sv[kC + tid] = s_beta[tid];
        sv[2 * kC + tid] = V == kLinear ? left : sq.t_back[tid] * left;
        if (tid == 0) sv[3 * kC] = (float)(s_keep[0] * s_keep[1]);
        ov[tid] = ct * eq[tid];
        ov[kC + tid] = sq.p_back[tid];
    }
    if (tid == 0) bulk_wait();
}

// ---------------------------------------------------------------------------
// A gate per key row.  A CTA takes a block and a value head.  The decays differ
// from row to row, so no product of K and Q alone serves: between blocks of 16
// tokens the rows are multiplied by what is left of them at the blocks' border
// (all factors at most 1 for gates at most 1) and then go to the tensor cores.
// Inside 16 tokens they do so, too, with the border at their end and the left
// rows divided by the gates behind them, as long as no product of the 16 gates is
// below kNear; a block of 16 that forgets faster takes the sums over the
// multiplied-out decays.  All these products share one right operand, K times
// what is left at the end of its 16, whose halves are made once.  Gates, K and Q
// are held in fp32, and give their places to the multiplied rows: what is needed
// of shared memory decides how many CTAs lie side by side (two).
// Measured: bf16, 105 blocks of 32 heads 256 us, 540 MB moved; a CTA takes 44
// thousand cycles, of which loads 10, products 10, the inverse and squares 13.
// With the right operand's halves made by each warp that reads it the kernel took
// 343 us, and with every 16 tokens multiplied out 371 us.
// ---------------------------------------------------------------------------
constexpr int kGateThreads = 256;
constexpr int kRowLd = kDK + 4;  // row of a [64][128] fp32 matrix
// Left rows, below 2^14 after scaling, grow by at most 1 / kNear; times kRoom they
// stay below 2^15.  Values that do not grow then have 2^-2 at most, in halves that
// resolve 2^-25, and right ones that shrink by 2^-16 the same: 22 bits are kept.
// Gates of at least a half (half-lives of a token or more) always qualify.
constexpr float kNear = 1.f / 65536, kRoom = 1.f / 32768;
struct GateRows {
    // gates, K, Q; then K times what is left (at last its halves, 256 bytes of each), K and Q times what was kept
    __align__(128) float a[kC][kRowLd], k[kC][kRowLd], q[kC][kRowLd];
    float diag_a[4][16][16], diag_p[4][16][16];  // A and P inside 16 tokens that forget fast
    float blk[4][kDK], inv[4][kDK];              // products of 16 tokens' gates, and kRoom by them
    float ek[kC], eq[kC], ek2[kC], beta[kC];
    float ks[kC], qs[kC];                        // scales of the rows of K and Q
    int fast[4];                                 // 16 tokens without a product of gates below kNear
};
static_assert(sizeof(GateRows) <= 115712 && sizeof(Squares) <= sizeof(GateRows::a) + sizeof(GateRows::k), "two CTAs of an SM; room for the squares");

__device__ __forceinline__ float4 mul4(float4 x, float4 y) { return make_float4(x.x * y.x, x.y * y.y, x.z * y.z, x.w * y.w); }
__device__ __forceinline__ float4 at4(const float *p) { return *reinterpret_cast<const float4 *>(p); }

template <class T>
__global__ void __launch_bounds__(kGateThreads, 2) k_gate_tiles(PromptArgs a, int first_block, Scratch sc)
{
    extern __shared__ __align__(128) char smem[];
    GateRows &r = *reinterpret_cast<GateRows *>(smem);
    const int tid = threadIdx.x, w = tid >> 5, l = tid & 31, g = l >> 2, c = l & 3;
    Block k;
    const int h = blockIdx.x % a.heads, hq = h / a.share;
    if (!find_block(a, first_block, blockIdx.x / a.heads, &k)) return;
    {
        const float *ag = a.alpha + ((long long)k.t0 * a.heads + h) * kDK;
        for (int x = tid; x < kC * (kDK / 4); x += kGateThreads) {
            const int row = x / (kDK / 4), d = x % (kDK / 4) * 4;
            if (row < k.n)
                cp_async16(&r.a[row][d], ag + (long long)row * a.heads * kDK + d, true);
            else
                *reinterpret_cast<float4 *>(&r.a[row][d]) = make_float4(1.f, 1.f, 1.f, 1.f);
        }
        const T *kg = static_cast<const T *>(a.k) + (long long)k.t0 * a.stride_k + hq * kDK + 4 * l, *qg = static_cast<const T *>(a.q) + (long long)k.t0 * a.stride_q + hq * kDK + 4 * l;
        float4 x[8], y[8];
        // without branches, so that all loads are under way at once
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int row = min(8 * w + i, k.n - 1);
            x[i] = load4(kg + row * a.stride_k);
            y[i] = load4(qg + row * a.stride_q);
        }
        if (tid < 4) r.fast[tid] = 1;
        if (tid < kC) r.beta[tid] = tid < k.n ? a.beta[(long long)(k.t0 + tid) * a.heads + h] : 0.f;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int row = 8 * w + i;
            if (row >= k.n) x[i] = y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4 *>(&r.k[row][4 * l]) = x[i];
            *reinterpret_cast<float4 *>(&r.q[row][4 * l]) = y[i];
            float sk, sq, back;
            dev::row_scale(warp_max(x[i]), &sk, &back);
            dev::row_scale(warp_max(y[i]), &sq, &back);
            if (l == 0) {
                r.ks[row] = sk;
                r.qs[row] = sq;
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    __syncthreads();
    for (int x = tid; x < 4 * kDK; x += kGateThreads) {  // 16 tokens of a key row
        float p = 1.f;
#pragma unroll
        for (int i = 0; i < 16; i++) p *= r.a[x / kDK * 16 + i][x % kDK];
        if (!(p >= kNear)) r.fast[x / kDK] = 0;
    }
    __syncthreads();
    // inside 16 tokens that forget fast: a warp takes four columns s at a time,
    // four key rows a lane, and walks down the rows t; two turns of four columns,
    // a long and a short one
#pragma unroll 1
    for (int turn = 0; turn < 2; turn++) {
        if (r.fast[w >> 1]) break;
        const int b = w >> 1, i0 = (w & 1) ? 4 + 4 * turn : 12 * turn, first = 16 * b;
        float2 x[4][2];
#pragma unroll
        for (int u = 0; u < 4; u++) {
            const float4 y = at4(&r.k[first + i0 + u][4 * l]);
            x[u][0] = make_float2(y.x, y.y);
            x[u][1] = make_float2(y.z, y.w);
        }
#pragma unroll 1
        for (int t = i0; t < 16; t++) {
            const float4 al = at4(&r.a[first + t][4 * l]), y = at4(&r.k[first + t][4 * l]), z = at4(&r.q[first + t][4 * l]);
            const float2 a0 = make_float2(al.x, al.y), a1 = make_float2(al.z, al.w), y0 = make_float2(y.x, y.y), y1 = make_float2(y.z, y.w),
                         z0 = make_float2(z.x, z.y), z1 = make_float2(z.z, z.w);
            float v[8];  // sums of the four columns with K, then with Q
#pragma unroll
            for (int u = 0; u < 4; u++) {
                if (t > i0 + u) {
                    x[u][0] = __fmul2_rn(x[u][0], a0);
                    x[u][1] = __fmul2_rn(x[u][1], a1);
                }
                const float2 p = __ffma2_rn(x[u][1], y1, __fmul2_rn(x[u][0], y0)), q = __ffma2_rn(x[u][1], z1, __fmul2_rn(x[u][0], z0));
                v[u] = p.x + p.y;
                v[4 + u] = q.x + q.y;
            }
            // eight sums over 32 lanes: each exchange halves the values a lane keeps
#pragma unroll
            for (int n = 4; n >= 1; n >>= 1) {
                const bool up = l & (4 * n);
#pragma unroll
                for (int i = 0; i < n; i++) {
                    const float keep = up ? v[i + n] : v[i], give = up ? v[i] : v[i + n];
                    v[i] = keep + __shfl_xor_sync(kFull, give, 4 * n);
                }
            }
            v[0] += __shfl_xor_sync(kFull, v[0], 2);
            v[0] += __shfl_xor_sync(kFull, v[0], 1);
            if (c == 0) {  // lane bits 4, 3, 2: K or Q, and the column
                const int s = i0 + (g & 3);
                if (g < 4)
                    r.diag_a[b][t][s] = t > s ? v[0] * r.beta[first + t] : 0.f;
                else
                    r.diag_p[b][t][s] = t >= s ? v[0] : 0.f;
            }
        }
        // the rows above
        if (l < i0) {
#pragma unroll
            for (int u = 0; u < 4; u++) r.diag_a[b][l][i0 + u] = r.diag_p[b][l][i0 + u] = 0.f;
        }
    }
    __syncthreads();
    // what a block keeps of a key row is multiplied up block after block: its
    // product is rounded once
    double keep = 1.0;
    if (tid >= kDK) {
        double part[4] = {1.0, 1.0, 1.0, 1.0};  // side by side
#pragma unroll 4
        for (int i = 0; i < 16; i++)
#pragma unroll
            for (int b = 0; b < 4; b++) part[b] *= (double)r.a[16 * b + i][tid - kDK];
        keep = (part[0] * part[1]) * (part[2] * part[3]);
    }
    __syncthreads();
    // gates of 16 tokens of a key row: what is kept from the 16's start, and what
    // is left at its end
#pragma unroll 1
    for (int x = tid; x < 4 * kDK; x += kGateThreads) {
        const int b = x / kDK, d = x % kDK;
        float al[16], kk[16];
        float p = 1.f;
#pragma unroll
        for (int i = 0; i < 16; i++) {
            al[i] = r.a[16 * b + i][d];
            kk[i] = r.k[16 * b + i][d];
            p *= al[i];
            r.k[16 * b + i][d] = kk[i] * p;
            r.q[16 * b + i][d] *= p;
        }
        r.blk[b][d] = p;
        r.inv[b][d] = kRoom / p;  // counts where p is at least kNear
        p = 1.f;
#pragma unroll
        for (int i = 15; i >= 0; i--) {
            r.a[16 * b + i][d] = kk[i] * p;
            p *= al[i];
        }
    }
    __syncthreads();
    // the operands that meet the state: K and Q times the running products, K
    // times what is left at the block's end
    const size_t bh = (size_t)k.b * a.heads + h;
    {
        char *img = reinterpret_cast<char *>(a.scratch) + bh * 2 * kTileBytes;
        const int b = w >> 1;  // the 16 tokens of this warp's rows
        float4 before = make_float4(1.f, 1.f, 1.f, 1.f), behind = before;
        for (int i = 0; i < b; i++) before = mul4(before, at4(&r.blk[i][4 * l]));
        for (int i = b + 1; i < 4; i++) behind = mul4(behind, at4(&r.blk[i][4 * l]));
#pragma unroll 4
        for (int i = 0; i < 8; i++) {
            const int row = 8 * w + i;
            const float4 left = at4(&r.a[row][4 * l]);
            const float b0 = put_row<2, false>(mul4(at4(&r.k[row][4 * l]), before), row, l, img + sc.k),
                        b1 = put_row<2, false>(mul4(at4(&r.q[row][4 * l]), before), row, l, img + sc.q),
                        b2 = put_row<2, false>(mul4(left, behind), row, l, img + sc.k2);
            // the right operand's halves, in the row's own place
            const float scale = r.ks[row];
            uint32_t hi[2], lo[2];
            dev::split_half(left.x * scale, left.y * scale, &hi[0], &lo[0]);
            dev::split_half(left.z * scale, left.w * scale, &hi[1], &lo[1]);
            __syncwarp();
            char *at = reinterpret_cast<char *>(r.a[row]) + 8 * l;
            *reinterpret_cast<uint2 *>(at) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2 *>(at + 2 * kDK) = make_uint2(lo[0], lo[1]);
            if (l == 0) {
                r.ek[row] = b0;
                r.eq[row] = b1;
                r.ek2[row] = b2;
            }
        }
    }
    __syncthreads();
    // rows of 16 tokens m against those of the earlier 16s and their own, K by
    // warps 0-3, Q by 4-7 in the opposite order
    const int m = rows_of(w);
    const bool is_q = w >= 4, fast = r.fast[m] != 0;
    float acc[kC / 8][4] = {};
    {
        const float(*src)[kRowLd] = is_q ? r.q : r.k;
        const int r0 = 16 * m + g, r1 = r0 + 8;
        const float s0 = (is_q ? r.qs : r.ks)[r0], s1 = (is_q ? r.qs : r.ks)[r1];
        const uint32_t right = dev::smem_addr(r.a[(l & 7) + (l >> 4) * 8]) + ((l >> 3) & 1) * 16;
        auto pair = [&](const float *row, int col) { return *reinterpret_cast<const float2 *>(row + col); };
        float own[2][4] = {};
        // left rows (times rows of factors f) by those of 16 tokens j: a loop of its own for each j,
        // so that the loads and halves of two steps overlap (eight take 391 us instead
        // of 376 for prompts of 16 requests: more instructions than lie near)
        auto product = [&](float (*out)[4], int j, const float (*f)[kDK], auto factors) {
            const uint32_t at = right + 16 * j * (kRowLd * 4);
#pragma unroll 2
            for (int ks = 0; ks < kDK / 16; ks++) {
                uint32_t ah[4], al[4], bh_[2][2], bl[2][2];
                ldsm4(bh_[0], bh_[1], at + 32 * ks);
                ldsm4(bl[0], bl[1], at + 32 * ks + 2 * kDK);
#pragma unroll
                for (int e = 0; e < 2; e++) {  // columns 2 c.., 2 c + 8..
                    const int col = 16 * ks + 8 * e + 2 * c;
                    float2 x0 = __fmul2_rn(pair(src[r0], col), make_float2(s0, s0)), x1 = __fmul2_rn(pair(src[r1], col), make_float2(s1, s1));
#pragma unroll
                    for (int i = 0; i < decltype(factors)::value; i++) {
                        const float2 u = pair(f[i], col);
                        x0 = __fmul2_rn(x0, u);
                        x1 = __fmul2_rn(x1, u);
                    }
                    dev::split_half(x0, &ah[2 * e], &al[2 * e]);
                    dev::split_half(x1, &ah[2 * e + 1], &al[2 * e + 1]);
                }
#pragma unroll
                for (int e = 0; e < 2; e++) mma16816(out[e], al[0], al[1], al[2], al[3], bh_[e][0], bh_[e][1]);
#pragma unroll
                for (int e = 0; e < 2; e++) mma16816(out[e], ah[0], ah[1], ah[2], ah[3], bl[e][0], bl[e][1]);
#pragma unroll
                for (int e = 0; e < 2; e++) mma16816(out[e], ah[0], ah[1], ah[2], ah[3], bh_[e][0], bh_[e][1]);
            }
        };
        if (fast) product(own, m, &r.inv[m], std::integral_constant<int, 1>{});
#pragma unroll
        for (int j = 0; j < 3; j++) {  // the 16s between
            if (j + 1 == m)
                product(&acc[2 * j], j, nullptr, std::integral_constant<int, 0>{});
            else if (j + 2 == m)
                product(&acc[2 * j], j, &r.blk[j + 1], std::integral_constant<int, 1>{});
            else if (j + 3 == m)
                product(&acc[2 * j], j, &r.blk[j + 1], std::integral_constant<int, 2>{});
        }
        // unscales: exact quotients of powers of two
        const float f0 = (is_q ? 1.f : r.beta[r0]) / s0, f1 = (is_q ? 1.f : r.beta[r1]) / s1;
        const float(*diag)[16] = is_q ? r.diag_p[m] : r.diag_a[m];
#pragma unroll
        for (int j = 0; j < kC / 8; j++) {
            const int i = 8 * (j & 1) + 2 * c, d = is_q ? 0 : 1;  // P has its diagonal, A does not
            const float2 sb = *reinterpret_cast<const float2 *>(&r.ks[8 * j + 2 * c]);
            const float2 kb = make_float2(1.f / sb.x, 1.f / sb.y);
            if (j < 2 * m) {
                acc[j][0] *= f0 * kb.x; acc[j][1] *= f0 * kb.y; acc[j][2] *= f1 * kb.x; acc[j][3] *= f1 * kb.y;
            } else if (j < 2 * m + 2 && fast) {
                const float *x = own[j & 1];
                const float big = 1.f / kRoom;
                acc[j][0] = i + d <= g ? x[0] * (f0 * kb.x) * big : 0.f;
                acc[j][1] = i + 1 + d <= g ? x[1] * (f0 * kb.y) * big : 0.f;
                acc[j][2] = i + d <= g + 8 ? x[2] * (f1 * kb.x) * big : 0.f;
                acc[j][3] = i + 1 + d <= g + 8 ? x[3] * (f1 * kb.y) * big : 0.f;
            } else if (j < 2 * m + 2) {
                acc[j][0] = diag[g][i]; acc[j][1] = diag[g][i + 1]; acc[j][2] = diag[g + 8][i]; acc[j][3] = diag[g + 8][i + 1];
            }
        }
    }
    __syncthreads();
    // the rows are done with: their room holds the squares
    Squares &sq = *reinterpret_cast<Squares *>(smem);
    finish<true, 4>(acc, acc, sq);
    if (tid == 0) put_squares<true>(sq, a.scratch + sc.inv + bh * kSquareBytes, a.scratch + sc.p + bh * kSquareBytes);
    float *sv = reinterpret_cast<float *>(a.scratch + sc.sv) + bh * kStateFloats;
    if (tid < kC) {
        float *ov = reinterpret_cast<float *>(a.scratch + sc.ov) + bh * kOutFloats;
        sv[tid] = -r.beta[tid] * r.ek[tid];
        sv[kC + tid] = r.beta[tid];
        sv[2 * kC + tid] = sq.t_back[tid] * r.ek2[tid];
        ov[tid] = r.eq[tid];
        ov[kC + tid] = sq.p_back[tid];
    } else if (tid >= kDK) {
        sv[3 * kC + tid - kDK] = (float)keep;
    }
    if (tid == 0) bulk_wait();
}

template <class T, int V, int NP>
cudaError_t launch_tiles(const PromptArgs &a, int first, int n, const Scratch &sc, cudaStream_t s)
{
    const int dyn = std::max(2 * NP * kTileBytes, (int)sizeof(Squares));
    cudaError_t e = cudaFuncSetAttribute(k_block_tiles<T, V, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, dyn);
    if (e != cudaSuccess) return e;
    k_block_tiles<T, V, NP><<<(unsigned)n * (unsigned)a.heads, kTileThreads, dyn, s>>>(a, first, sc);
    return cudaGetLastError();
}

template <class T>
cudaError_t launch_tiles_v(const PromptArgs &a, int first, int n, const Scratch &sc, cudaStream_t s)
{
    constexpr int NP = sizeof(T) == 4 ? 2 : 1;
    if (a.variant == kGdn) return launch_tiles<T, kGdn, NP>(a, first, n, sc, s);
    if (a.variant == kLinear) return launch_tiles<T, kLinear, NP>(a, first, n, sc, s);
    cudaError_t e = cudaFuncSetAttribute(k_gate_tiles<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(GateRows));
    if (e != cudaSuccess) return e;
    k_gate_tiles<T><<<(unsigned)n * (unsigned)a.heads, kGateThreads, sizeof(GateRows), s>>>(a, first, sc);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_tiles(const PromptArgs &a, int first_block, int n, const Scratch &sc, cudaStream_t s)
{
    switch (a.dtype) {
        case kF32: return launch_tiles_v<float>(a, first_block, n, sc, s);
        case kF16: return launch_tiles_v<__half>(a, first_block, n, sc, s);
        default: return launch_tiles_v<__nv_bfloat16>(a, first_block, n, sc, s);
    }
}

}  // namespace stepq
