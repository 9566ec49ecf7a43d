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
using dev::mma16816;

constexpr unsigned kFull = 0xffffffffu;
constexpr int kLd = kC + 4;  // row of a [64][64] fp32 matrix in shared memory

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

// One row of an operand (4 elements a lane) as scaled halves into the tile's
// image in the scratch, and into the tile in shared memory if there is one;
// returns the row's unscale.  NP: halves kept.  EXACT: binary16 inputs are
// their own halves.
template <int NP, bool EXACT>
__device__ __forceinline__ float put_row(float4 x, int row, int l, char *tile, char *image)
{
    float scale = 1.f, back = 1.f;
    if (!EXACT) dev::row_scale(warp_max(x), &scale, &back);
    uint32_t hi[2], lo[2];
    dev::split_half(x.x * scale, x.y * scale, &hi[0], &lo[0]);
    dev::split_half(x.z * scale, x.w * scale, &hi[1], &lo[1]);
    const int at = tile_at(row, 4 * l);
    const uint2 h = make_uint2(hi[0], hi[1]), o = make_uint2(lo[0], lo[1]);
    *reinterpret_cast<uint2 *>(image + at) = h;
    if (tile) *reinterpret_cast<uint2 *>(tile + at) = h;
    if (NP == 2) {
        *reinterpret_cast<uint2 *>(image + kTileBytes + at) = o;
        if (tile) *reinterpret_cast<uint2 *>(tile + kTileBytes + at) = o;
    }
    return back;
}

// acc[j] = rows 16 m .. 16 m + 15 of A times rows 8 j .. of B transposed, for
// the column tiles j < tiles (a multiple of 2): A and B operand tiles in
// shared memory.  Each pass goes over all sums before it returns to the first.
template <int NP>
__device__ __forceinline__ void rows_product(float (*acc)[4], const char *A, const char *B, int m, int tiles)
{
    const int l = threadIdx.x & 31;
    const uint32_t a0 = dev::smem_addr(A), b0 = dev::smem_addr(B);
    const int arow = 16 * m + (l & 7) + ((l >> 3) & 1) * 8, acol = (l >> 4) * 8;  // of the A matrices
    const int brow = (l & 7) + (l >> 4) * 8, bcol = ((l >> 3) & 1) * 8;           // of two column tiles
#pragma unroll
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

// ---- [64][64] lower-triangular fp32 matrices in shared memory --------------

// acc += x . the rows m .. m + 3 of Y at four columns.
__device__ __forceinline__ void fma4(float4 &acc, float4 x, const float *Y)
{
    const float4 y0 = *reinterpret_cast<const float4 *>(Y), y1 = *reinterpret_cast<const float4 *>(Y + kLd),
                 y2 = *reinterpret_cast<const float4 *>(Y + 2 * kLd), y3 = *reinterpret_cast<const float4 *>(Y + 3 * kLd);
    acc.x = fmaf(x.x, y0.x, fmaf(x.y, y1.x, fmaf(x.z, y2.x, fmaf(x.w, y3.x, acc.x))));
    acc.y = fmaf(x.x, y0.y, fmaf(x.y, y1.y, fmaf(x.z, y2.y, fmaf(x.w, y3.y, acc.y))));
    acc.z = fmaf(x.x, y0.z, fmaf(x.y, y1.z, fmaf(x.z, y2.z, fmaf(x.w, y3.z, acc.z))));
    acc.w = fmaf(x.x, y0.w, fmaf(x.y, y1.w, fmaf(x.z, y2.w, fmaf(x.w, y3.w, acc.w))));
}

// inv_21 = -inv_22 A_21 inv_11 for the pairs of H x H diagonal blocks; tmp: room
// for another matrix.
template <int H>
__device__ __forceinline__ void invert_step(const float *A, float *inv, float *tmp)
{
    const int tid = threadIdx.x;
    constexpr int tasks = kC / (2 * H) * H * H / 4;  // four columns of a row each: at most 256
    const int pair = tid / (H * H / 4), i = tid / (H / 4) % H, j = tid % (H / 4) * 4;
    const int lo = 2 * H * pair, hi = lo + H;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (tid < tasks) {
#pragma unroll
        for (int m = 0; m < H; m += 4) fma4(x, *reinterpret_cast<const float4 *>(A + (hi + i) * kLd + lo + m), inv + (lo + m) * kLd + lo + j);
        *reinterpret_cast<float4 *>(tmp + (hi + i) * kLd + lo + j) = x;
    }
    __syncthreads();
    if (tid < tasks) {
        x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int m = 0; m < H; m += 4) fma4(x, *reinterpret_cast<const float4 *>(inv + (hi + i) * kLd + hi + m), tmp + (hi + m) * kLd + lo + j);
        *reinterpret_cast<float4 *>(inv + (hi + i) * kLd + lo + j) = make_float4(-x.x, -x.y, -x.z, -x.w);
    }
    __syncthreads();
}

// inv = (I + A)^-1 for the strictly lower triangular A: the four diagonal blocks
// of 16 by substitution, a column a thread, then the blocks below in two steps.
// Blocks above the diagonal stay as they are, except 16 x 32 ones inside a
// diagonal block of 32, which are set to zero (they are read as such).
__device__ __forceinline__ void invert_lower(const float *A, float *inv, float *tmp)
{
    const int tid = threadIdx.x;
    if (tid < kC) {
        const int b = tid & ~15, j = tid & 15;
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; r++) {
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int m = 0; m < r; m += 4) {
                const float4 y = *reinterpret_cast<const float4 *>(A + (b + r) * kLd + b + m);
                s0 = fmaf(y.x, x[m], s0);
                if (m + 1 < r) s1 = fmaf(y.y, x[m + 1], s1);
                if (m + 2 < r) s0 = fmaf(y.z, x[m + 2], s0);
                if (m + 3 < r) s1 = fmaf(y.w, x[m + 3], s1);
            }
            x[r] = r < j ? 0.f : (r == j ? 1.f : -(s0 + s1));
            inv[(b + r) * kLd + b + j] = x[r];
        }
    } else if (tid < 2 * kC) {
        // the upper 16 x 16 blocks of the two diagonal blocks of 32
        const int b = (tid - kC) >> 5, i = (tid - kC) & 15, e = (tid - kC) >> 4 & 1;
#pragma unroll
        for (int j = 0; j < 8; j += 4) *reinterpret_cast<float4 *>(inv + (32 * b + i) * kLd + 32 * b + 16 + 8 * e + j) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
    invert_step<16>(A, inv, tmp);
    invert_step<32>(A, inv, tmp);
}

// out = X Y for lower-triangular X and Y, two rows and four columns a thread and
// turn; the blocks of 16 x 16 on and below the diagonal are written (those of X
// and Y hold zeros above the diagonal).
__device__ __forceinline__ void lower_product(const float *X, const float *Y, float *out)
{
    for (int x = threadIdx.x; x < kC / 2 * (kC / 4); x += blockDim.x) {
        const int i = x / (kC / 4) * 2, j = x % (kC / 4) * 4;
        if ((j & ~15) > i) continue;
        float4 a0 = make_float4(0.f, 0.f, 0.f, 0.f), a1 = a0;
        const int last = i | 3;
        for (int m = j; m <= last; m += 4) {
            const float4 x0 = *reinterpret_cast<const float4 *>(X + i * kLd + m), x1 = *reinterpret_cast<const float4 *>(X + (i + 1) * kLd + m);
            fma4(a0, x0, Y + m * kLd + j);
            fma4(a1, x1, Y + m * kLd + j);
        }
        *reinterpret_cast<float4 *>(out + i * kLd + j) = a0;
        *reinterpret_cast<float4 *>(out + (i + 1) * kLd + j) = a1;
    }
}

// The lower triangle of a matrix, rows as scaled halves, into the scratch (256
// threads, numbered x); the rows' unscales into back[].  Columns past the row's
// block of 16 are not written (and not read).
__device__ __forceinline__ void put_square(int x, const float *sq, char *image, float *back)
{
    const int row = x >> 2, part = x & 3;  // 16 columns each
    const bool inside = part <= row >> 4;
    float v[16], m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (inside) y = *reinterpret_cast<const float4 *>(sq + row * kLd + 16 * part + i);
        v[i] = y.x; v[i + 1] = y.y; v[i + 2] = y.z; v[i + 3] = y.w;
        m = fmaxf(fmaxf(fmaxf(m, fabsf(y.x)), fabsf(y.y)), fmaxf(fabsf(y.z), fabsf(y.w)));
    }
    m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
    m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
    float scale, b;
    dev::row_scale(m, &scale, &b);
    if (part == 0) back[row] = b;
    if (!inside) return;
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int i = 0; i < 8; i++) dev::split_half(v[2 * i] * scale, v[2 * i + 1] * scale, &hi[i], &lo[i]);
#pragma unroll
    for (int e = 0; e < 2; e++) {
        const int at = square_at(row, 16 * part + 8 * e);
        *reinterpret_cast<uint4 *>(image + at) = make_uint4(hi[4 * e], hi[4 * e + 1], hi[4 * e + 2], hi[4 * e + 3]);
        *reinterpret_cast<uint4 *>(image + kSquareBytes / 2 + at) = make_uint4(lo[4 * e], lo[4 * e + 1], lo[4 * e + 2], lo[4 * e + 3]);
    }
}

// From A (strictly lower triangular) and P to the squares of the scratch:
// (I + A)^-1 and P (I + A)^-1 (without an A, P itself).  I, tmp: room for two
// matrices.  Begins and ends with a barrier.
template <bool DELTA>
__device__ __forceinline__ void finish(float *A, float *P, float *I, float *tmp, char *inv_image, char *p_image, float *s_inv, float *s_p)
{
    const int x = threadIdx.x;
    __syncthreads();
    const float *out = P;
    if (DELTA) {
        invert_lower(A, I, tmp);
        lower_product(P, I, tmp);
        out = tmp;
        __syncthreads();
    }
    if (x < 256) put_square(x, out, p_image, s_p);
    if (DELTA) {  // by the other half of the threads, where there are that many
        if (blockDim.x == 256)
            put_square(x, I, inv_image, s_inv);
        else if (x >= 256)
            put_square(x - 256, I, inv_image, s_inv);
    }
    __syncthreads();
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
// One gate a head.  A CTA takes a block and a query / key head: K K^T and Q K^T
// on the tensor cores (warps 0-3 and 4-7, 16 rows each), then for each value
// head of the group the decays, the inverse and the squares.  The decay from
// token s to token t is the product of what is left of s at the end of its 16
// tokens, of the 16s between, and of t's 16 up to t; inside 16 tokens it is
// multiplied out.
// ---------------------------------------------------------------------------
template <class T, int V, int NP>
__global__ void __launch_bounds__(256) k_block_tiles(PromptArgs a, int first_block, Scratch sc)
{
    extern __shared__ __align__(128) char smem[];
    __shared__ float ek[kC], eq[kC], s_beta[kC], s_pre[kC], s_suf[kC], s_inv[kC], s_p[kC], s_blk[4], s_diag[4][16][17];
    const int tid = threadIdx.x, w = tid >> 5, l = tid & 31, g = l >> 2, c = l & 3;
    const int heads_k = a.heads / a.share;
    Block k;
    const int hq = blockIdx.x % heads_k;
    if (!find_block(a, first_block, blockIdx.x / heads_k, &k)) return;
    // the gates of the first value head, while the tiles are made
    const int tok = tid & (kC - 1);
    const bool in = tok < k.n;
    const long long gate0 = (long long)(k.t0 + (in ? tok : 0)) * a.heads + hq * a.share;
    float alpha = 1.f, beta = 0.f;
    if (in) {
        alpha = a.alpha[gate0];
        beta = a.beta[gate0];
    }
    char *tk = smem, *tq = smem + NP * kTileBytes;
    {
        const size_t at = ((size_t)k.b * heads_k + hq) * NP * kTileBytes;
        char *ik = reinterpret_cast<char *>(a.scratch) + sc.k + at, *iq = reinterpret_cast<char *>(a.scratch) + sc.q + at;
        const T *kg = static_cast<const T *>(a.k) + hq * kDK, *qg = static_cast<const T *>(a.q) + hq * kDK;
        constexpr bool exact = std::is_same<T, __half>::value;
        float4 xk[kC / 8], xq[kC / 8];
#pragma unroll
        for (int i = 0; i < kC / 8; i++) {
            const int row = 8 * w + i;
            xk[i] = xq[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row < k.n) {
                xk[i] = load4(kg + (long long)(k.t0 + row) * a.stride_k + 4 * l);
                xq[i] = load4(qg + (long long)(k.t0 + row) * a.stride_q + 4 * l);
            }
        }
#pragma unroll
        for (int i = 0; i < kC / 8; i++) {
            const int row = 8 * w + i;
            const float bk = put_row<NP, exact>(xk[i], row, l, tk, ik), bq = put_row<NP, exact>(xq[i], row, l, tq, iq);
            if (l == 0) {
                ek[row] = bk;
                eq[row] = bq;
            }
        }
    }
    __syncthreads();
    const int m = w & 3;  // rows 16 m + g, + 8
    const bool is_q = w >= 4;
    float acc[kC / 8][4] = {};
    if (is_q || V != kLinear) rows_product<NP>(acc, is_q ? tq : tk, tk, m, 2 * m + 2);
    {
        const float r0 = (is_q ? eq : ek)[16 * m + g], r1 = (is_q ? eq : ek)[16 * m + g + 8];
#pragma unroll
        for (int j = 0; j < kC / 8; j++) {
            const float c0 = ek[8 * j + 2 * c], c1 = ek[8 * j + 2 * c + 1];
            acc[j][0] *= r0 * c0; acc[j][1] *= r0 * c1; acc[j][2] *= r1 * c0; acc[j][3] *= r1 * c1;
        }
    }
    // the tiles are done with: their room holds the fp32 matrices
    float *sA = reinterpret_cast<float *>(smem), *sP = sA + kC * kLd, *sI = sP + kC * kLd, *sX = sI + kC * kLd;
    for (int v = 0; v < a.share; v++) {
        const int h = hq * a.share + v;
        if (tid < kC) {
            float p = alpha, q = __shfl_down_sync(kFull, alpha, 1, 16);
            if ((l & 15) == 15) q = 1.f;
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) {
                const float x = __shfl_up_sync(kFull, p, d, 16), y = __shfl_down_sync(kFull, q, d, 16);
                if ((l & 15) >= d) p *= x;
                if ((l & 15) + d < 16) q *= y;
            }
            s_pre[tid] = p;
            s_suf[tid] = q;
            s_beta[tid] = beta;
            if ((l & 15) == 15) s_blk[tid >> 4] = p;
        } else if (tid < 2 * kC) {
            float p = 1.f;
#pragma unroll
            for (int t = 0; t < 16; t++) {
                const float x = __shfl_sync(kFull, alpha, t, 16);
                if (t > (l & 15)) p *= x;
                s_diag[tok >> 4][t][l & 15] = p;
            }
        }
        if (v + 1 < a.share && in) {
            alpha = a.alpha[gate0 + v + 1];
            beta = a.beta[gate0 + v + 1];
        }
        __syncthreads();
        if (is_q || V != kLinear) {
            float *dst = is_q ? sP : sA;
            const int i0 = g, i1 = g + 8;  // rows within the block of 16
            const float b0 = is_q ? 1.f : s_beta[16 * m + i0], b1 = is_q ? 1.f : s_beta[16 * m + i1];
            float f0 = s_pre[16 * m + i0] * b0, f1 = s_pre[16 * m + i1] * b1;
#pragma unroll
            for (int jb = kC / 16 - 1; jb >= 0; jb--) {
                if (jb > m) continue;
                if (jb + 1 < m) {  // another 16 tokens between
                    f0 *= s_blk[jb + 1];
                    f1 *= s_blk[jb + 1];
                }
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int j = 2 * jb + e, s = 8 * j + 2 * c, si = s & 15;
                    float2 x, y;
                    if (jb == m) {
                        x.x = (is_q ? si <= i0 : si < i0) ? acc[j][0] * s_diag[m][i0][si] * b0 : 0.f;
                        x.y = (is_q ? si + 1 <= i0 : si + 1 < i0) ? acc[j][1] * s_diag[m][i0][si + 1] * b0 : 0.f;
                        y.x = (is_q ? si <= i1 : si < i1) ? acc[j][2] * s_diag[m][i1][si] * b1 : 0.f;
                        y.y = (is_q ? si + 1 <= i1 : si + 1 < i1) ? acc[j][3] * s_diag[m][i1][si + 1] * b1 : 0.f;
                    } else {
                        const float2 q = *reinterpret_cast<const float2 *>(&s_suf[s]);
                        x = make_float2(acc[j][0] * (f0 * q.x), acc[j][1] * (f0 * q.y));
                        y = make_float2(acc[j][2] * (f1 * q.x), acc[j][3] * (f1 * q.y));
                    }
                    *reinterpret_cast<float2 *>(dst + (16 * m + i0) * kLd + s) = x;
                    *reinterpret_cast<float2 *>(dst + (16 * m + i1) * kLd + s) = y;
                }
            }
        }
        const size_t bh = (size_t)k.b * a.heads + h;
        finish<V != kLinear>(sA, sP, sI, sX, reinterpret_cast<char *>(a.scratch) + sc.inv + bh * kSquareBytes,
                             reinterpret_cast<char *>(a.scratch) + sc.p + bh * kSquareBytes, s_inv, s_p);
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
            sv[2 * kC + tid] = V == kLinear ? left : s_inv[tid] * left;
            if (tid == kC - 1) sv[3 * kC] = ct;
            ov[tid] = ct * eq[tid];
            ov[kC + tid] = s_p[tid];
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// A gate per key row.  A CTA takes a block and a value head.  The decays differ
// from row to row, so no product of K and Q alone serves: between blocks of 16
// tokens the rows are multiplied by what is left of them at the blocks' border
// (all factors at most 1 for gates at most 1) and then go to the tensor cores,
// inside 16 tokens the sums run over the multiplied-out decays.
// ---------------------------------------------------------------------------
constexpr int kGateThreads = 512;
constexpr int kRowLd = kDK + 8;  // row of a [64][128] fp32 matrix: fragments of 8 rows x 8 columns fall into different banks
constexpr int kGateBytes = (5 * kC * kRowLd + 2 * kC * kLd) * 4;

__device__ __forceinline__ float4 mul4(float4 x, float4 y) { return make_float4(x.x * y.x, x.y * y.y, x.z * y.z, x.w * y.w); }

template <class T>
__global__ void __launch_bounds__(kGateThreads) k_gate_tiles(PromptArgs a, int first_block, Scratch sc)
{
    extern __shared__ __align__(128) char smem[];
    __shared__ float ek[kC], eq[kC], ek2[kC], s_beta[kC], s_inv[kC], s_p[kC];
    __shared__ float s_ks[kC], s_kb[kC], s_qs[kC], s_qb[kC];  // scale and unscale of the rows of K and Q
    __shared__ __align__(16) float s_blk[4][kDK];
    float *sa = reinterpret_cast<float *>(smem), *sk = sa + kC * kRowLd, *sq = sk + kC * kRowLd, *pre = sq + kC * kRowLd, *suf = pre + kC * kRowLd;
    float *sA = suf + kC * kRowLd, *sP = sA + kC * kLd, *sI = sk, *sX = sq;  // the last two when K and Q are done with
    const int tid = threadIdx.x, w = tid >> 5, l = tid & 31, g = l >> 2, c = l & 3;
    Block k;
    const int h = blockIdx.x % a.heads;
    if (!find_block(a, first_block, blockIdx.x / a.heads, &k)) return;
    const int hq = h / a.share;
    // gates of 16 tokens of a key row a thread: running products from the 16's
    // start, and what is left at its end
    {
        const int b = tid >> 7, d = tid & (kDK - 1);
        const float *ag = a.alpha + ((long long)(k.t0 + 16 * b) * a.heads + h) * kDK + d;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; i++) x[i] = 16 * b + i < k.n ? ag[(long long)i * a.heads * kDK] : 1.f;
        float p = 1.f;
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const int at = (16 * b + i) * kRowLd + d;
            p *= x[i];
            sa[at] = x[i];
            pre[at] = p;
        }
        s_blk[b][d] = p;
        p = 1.f;
#pragma unroll
        for (int i = 15; i >= 0; i--) {
            suf[(16 * b + i) * kRowLd + d] = p;
            p *= x[i];
        }
    }
    {
        const T *kg = static_cast<const T *>(a.k) + hq * kDK, *qg = static_cast<const T *>(a.q) + hq * kDK;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int row = 4 * w + i;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
            if (row < k.n) {
                x = load4(kg + (long long)(k.t0 + row) * a.stride_k + 4 * l);
                y = load4(qg + (long long)(k.t0 + row) * a.stride_q + 4 * l);
            }
            *reinterpret_cast<float4 *>(sk + row * kRowLd + 4 * l) = x;
            *reinterpret_cast<float4 *>(sq + row * kRowLd + 4 * l) = y;
            float s, b, s2, b2;
            dev::row_scale(warp_max(x), &s, &b);
            dev::row_scale(warp_max(y), &s2, &b2);
            if (l == 0) {
                s_ks[row] = s; s_kb[row] = b;
                s_qs[row] = s2; s_qb[row] = b2;
            }
        }
        if (tid < kC) s_beta[tid] = tid < k.n ? a.beta[(long long)(k.t0 + tid) * a.heads + h] : 0.f;
        // zeros above the diagonal
        for (int i = tid; i < kC * kLd; i += kGateThreads) sA[i] = sP[i] = 0.f;
    }
    __syncthreads();
    // the operands that meet the state: K and Q times the running products, K
    // times what is left at the block's end
    const size_t bh = (size_t)k.b * a.heads + h;
    {
        char *img = reinterpret_cast<char *>(a.scratch) + bh * 2 * kTileBytes;
        const int b = w >> 2;  // the 16 tokens of this warp's rows
        float4 before = make_float4(1.f, 1.f, 1.f, 1.f), behind = before;
        for (int i = 0; i < b; i++) before = mul4(before, *reinterpret_cast<const float4 *>(&s_blk[i][4 * l]));
        for (int i = b + 1; i < 4; i++) behind = mul4(behind, *reinterpret_cast<const float4 *>(&s_blk[i][4 * l]));
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int row = 4 * w + i, at = row * kRowLd + 4 * l;
            const float4 ct = mul4(before, *reinterpret_cast<const float4 *>(pre + at)), left = mul4(behind, *reinterpret_cast<const float4 *>(suf + at));
            const float4 x = *reinterpret_cast<const float4 *>(sk + at), y = *reinterpret_cast<const float4 *>(sq + at);
            const float b0 = put_row<2, false>(mul4(x, ct), row, l, nullptr, img + sc.k), b1 = put_row<2, false>(mul4(y, ct), row, l, nullptr, img + sc.q),
                        b2 = put_row<2, false>(mul4(x, left), row, l, nullptr, img + sc.k2);
            if (l == 0) {
                ek[row] = b0;
                eq[row] = b1;
                ek2[row] = b2;
            }
        }
    }
    // rows of 16 tokens i against those of an earlier 16 j, K by warps 0-5, Q by 6-11
    if (w < 12) {
        const int task = w % 6, i = task < 1 ? 1 : (task < 3 ? 2 : 3), j = task - (i == 1 ? 0 : (i == 2 ? 1 : 3));
        const bool is_q = w >= 6;
        const float *src = is_q ? sq : sk;
        const int r0 = 16 * i + g, r1 = r0 + 8;
        const float s0 = (is_q ? s_qs : s_ks)[r0], s1 = (is_q ? s_qs : s_ks)[r1];
        const int c0 = 16 * j + g, c1 = c0 + 8;  // right rows of the two column tiles
        const float k0 = s_ks[c0], k1 = s_ks[c1];
        float acc[2][4] = {};
        auto pair = [&](const float *x, const float *y, int row, int col, float scale) {
            const float2 u = *reinterpret_cast<const float2 *>(x + row * kRowLd + col), v = *reinterpret_cast<const float2 *>(y + row * kRowLd + col);
            return make_float2(u.x * v.x * scale, u.y * v.y * scale);
        };
#pragma unroll
        for (int ks = 0; ks < kDK / 16; ks++) {
            uint32_t ah[4], al[4];
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int col = 16 * ks + 8 * e + 2 * c;
                dev::split_half(pair(src, pre, r0, col, s0), &ah[2 * e], &al[2 * e]);
                dev::split_half(pair(src, pre, r1, col, s1), &ah[2 * e + 1], &al[2 * e + 1]);
            }
            uint32_t bh_[2][2], bl[2][2];
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int col = 16 * ks + 8 * e + 2 * c;
                float2 x = pair(sk, suf, c0, col, k0), y = pair(sk, suf, c1, col, k1);
                for (int b = j + 1; b < i; b++) {  // the 16s between
                    const float2 f = *reinterpret_cast<const float2 *>(&s_blk[b][col]);
                    x.x *= f.x; x.y *= f.y; y.x *= f.x; y.y *= f.y;
                }
                dev::split_half(x, &bh_[0][e], &bl[0][e]);
                dev::split_half(y, &bh_[1][e], &bl[1][e]);
            }
#pragma unroll
            for (int e = 0; e < 2; e++) mma16816(acc[e], al[0], al[1], al[2], al[3], bh_[e][0], bh_[e][1]);
#pragma unroll
            for (int e = 0; e < 2; e++) mma16816(acc[e], ah[0], ah[1], ah[2], ah[3], bl[e][0], bl[e][1]);
#pragma unroll
            for (int e = 0; e < 2; e++) mma16816(acc[e], ah[0], ah[1], ah[2], ah[3], bh_[e][0], bh_[e][1]);
        }
        float *dst = is_q ? sP : sA;
        const float f0 = is_q ? s_qb[r0] : s_kb[r0] * s_beta[r0], f1 = is_q ? s_qb[r1] : s_kb[r1] * s_beta[r1];
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const int s = 16 * j + 8 * e + 2 * c;
            const float2 kb = *reinterpret_cast<const float2 *>(&s_kb[s]);
            *reinterpret_cast<float2 *>(dst + r0 * kLd + s) = make_float2(acc[e][0] * (f0 * kb.x), acc[e][1] * (f0 * kb.y));
            *reinterpret_cast<float2 *>(dst + r1 * kLd + s) = make_float2(acc[e][2] * (f1 * kb.x), acc[e][3] * (f1 * kb.y));
        }
    }
    // inside 16 tokens: a warp takes four columns s of a block, eight lanes each
    // over the key rows, and walks down the rows t
    {
        const int b = 16 * (w >> 2), i0 = 4 * (w & 3), s = b + i0 + (l >> 3), d0 = 4 * (l & 7);
        float4 x[4];
#pragma unroll
        for (int i = 0; i < 4; i++) x[i] = *reinterpret_cast<const float4 *>(sk + s * kRowLd + d0 + 32 * i);
        for (int t = b + i0; t < b + 16; t++) {
            float ka = 0.f, qa = 0.f;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int at = t * kRowLd + d0 + 32 * i;
                if (t > s) x[i] = mul4(x[i], *reinterpret_cast<const float4 *>(sa + at));
                const float4 y = *reinterpret_cast<const float4 *>(sk + at), z = *reinterpret_cast<const float4 *>(sq + at);
                ka = fmaf(x[i].x, y.x, fmaf(x[i].y, y.y, fmaf(x[i].z, y.z, fmaf(x[i].w, y.w, ka))));
                qa = fmaf(x[i].x, z.x, fmaf(x[i].y, z.y, fmaf(x[i].z, z.z, fmaf(x[i].w, z.w, qa))));
            }
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) {
                ka += __shfl_xor_sync(kFull, ka, d);
                qa += __shfl_xor_sync(kFull, qa, d);
            }
            if ((l & 7) == 0) {
                if (t > s) sA[t * kLd + s] = ka * s_beta[t];
                if (t >= s) sP[t * kLd + s] = qa;
            }
        }
    }
    finish<true>(sA, sP, sI, sX, reinterpret_cast<char *>(a.scratch) + sc.inv + bh * kSquareBytes,
                 reinterpret_cast<char *>(a.scratch) + sc.p + bh * kSquareBytes, s_inv, s_p);
    float *sv = reinterpret_cast<float *>(a.scratch + sc.sv) + bh * kStateFloats;
    if (tid < kC) {
        float *ov = reinterpret_cast<float *>(a.scratch + sc.ov) + bh * kOutFloats;
        sv[tid] = -s_beta[tid] * ek[tid];
        sv[kC + tid] = s_beta[tid];
        sv[2 * kC + tid] = s_inv[tid] * ek2[tid];
        ov[tid] = eq[tid];
        ov[kC + tid] = s_p[tid];
    } else if (tid >= 128 && tid < 128 + kDK) {
        const int d = tid - 128;
        sv[3 * kC + d] = s_blk[0][d] * s_blk[1][d] * s_blk[2][d] * s_blk[3][d];
    }
}

template <class T, int V, int NP>
cudaError_t launch_tiles(const PromptArgs &a, int first, int n, const Scratch &sc, cudaStream_t s)
{
    const int dyn = std::max(2 * NP * kTileBytes, 4 * kC * kLd * 4);
    cudaError_t e = cudaFuncSetAttribute(k_block_tiles<T, V, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, dyn);
    if (e != cudaSuccess) return e;
    k_block_tiles<T, V, NP><<<(unsigned)n * (unsigned)(a.heads / a.share), 256, dyn, s>>>(a, first, sc);
    return cudaGetLastError();
}

template <class T>
cudaError_t launch_tiles_v(const PromptArgs &a, int first, int n, const Scratch &sc, cudaStream_t s)
{
    constexpr int NP = sizeof(T) == 4 ? 2 : 1;
    if (a.variant == kGdn) return launch_tiles<T, kGdn, NP>(a, first, n, sc, s);
    if (a.variant == kLinear) return launch_tiles<T, kLinear, NP>(a, first, n, sc, s);
    cudaError_t e = cudaFuncSetAttribute(k_gate_tiles<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGateBytes);
    if (e != cudaSuccess) return e;
    k_gate_tiles<T><<<(unsigned)n * (unsigned)a.heads, kGateThreads, kGateBytes, s>>>(a, first, sc);
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
