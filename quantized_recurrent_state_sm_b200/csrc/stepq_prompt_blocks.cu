// The prompt pass in blocks of 64 tokens.
//
// With S the state before a block, c_t the running product of the gates inside
// it, and decay_ts = prod_(s<r<=t) alpha_r, the recurrence of a block is
//   A_ts = beta_t sum_d k_td decay_ts,d k_sd (s < t),     P_ts = sum_d q_td decay_ts,d k_sd (s <= t),
//   U = (I + A)^-1 (beta (V - (c K) S)),
//   out = (c Q) S + P U,        S <- c_64 S + (decay_64 K)^T U
// (plain linear attention: U = beta V).  What does not depend on the state --
// (I + A)^-1, P and the operands in the form the tensor cores take -- is made
// for all blocks at once by a first kernel; a second walks each request's
// blocks in order and carries the state in registers.
//
// Every product runs on the tensor cores with its fp32 operands split into two
// binary16 halves (three products, two where an operand is exact in binary16),
// rows scaled by powers of two so that the halves keep 22 bits: the state and
// the sums stay at fp32's precision.  Decays are products of gates, never
// quotients or differences of logarithms, so gates of 0 and products that
// underflow need no care.
#include <cuda_bf16.h>

#include <algorithm>

#include "stepq_device.cuh"
#include "stepq_mma.cuh"
#include "stepq_serve.cuh"

namespace stepq {
namespace {

using dev::ldsm4;
using dev::ldsm4_t;
using dev::mma16816;

constexpr unsigned kFull = 0xffffffffu;
constexpr int kC = kBlockTokens;
constexpr int kTileBytes = kC * kDK * 2;    // one binary16 half of a [64][128] operand
constexpr int kSquareBytes = kC * kC * 2 * 2;  // hi and lo of a [64][64] operand
// per block and head, for the state: unscale of the K rows times c_t, beta,
// unscale of the inverse's rows, scale of U for the state update, kept share of S
constexpr int kStateFloats = 4 * kC + kDK;
constexpr int kOutFloats = 2 * kC;          // for the output: unscale of the Q rows times c_t, of the P rows
constexpr long long kWaitLimit = 1LL << 32;  // cycles, about two seconds

// Byte of element (row, col) of an operand tile: 16-byte chunks of a row are
// permuted by the row, so that eight rows of one column block lie in different
// banks.
__device__ __forceinline__ int tile_at(int row, int col) { return row * 256 + ((((col >> 3) ^ row) & 7) | (col >> 3 & 8)) * 16 + (col & 7) * 2; }
__device__ __forceinline__ int square_at(int row, int col) { return row * 128 + (((col >> 3) ^ row) & 7) * 16 + (col & 7) * 2; }

// The scratch of a launch over `blocks` blocks.
struct Scratch {
    int heads_k;  // heads the K and Q tiles are made for
    int halves;   // binary16 halves of K and Q
    size_t k, q, k2, inv, p, sv, ov, total;
};

__host__ __device__ Scratch scratch_of(int variant, int dtype, int heads, int share, long long blocks)
{
    Scratch s;
    s.heads_k = variant == kKda ? heads : heads / share;
    s.halves = variant == kKda || dtype == kF32 ? 2 : 1;
    const size_t tiles = (size_t)blocks * s.heads_k * s.halves * kTileBytes, bh = (size_t)blocks * heads;
    size_t o = 0;
    s.k = o;   o += tiles;
    s.q = o;   o += tiles;
    s.k2 = o;  o += variant == kKda ? tiles : 0;
    s.inv = o; o += variant == kLinear ? 0 : bh * kSquareBytes;
    s.p = o;   o += bh * kSquareBytes;
    s.sv = o;  o += bh * kStateFloats * 4;
    s.ov = o;  o += bh * kOutFloats * 4;
    s.total = o;
    return s;
}

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

__device__ __forceinline__ float warp_max(float m)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
    return m;
}

// One row of an operand (4 elements a lane) as scaled halves, into the tile in
// shared memory and its image in the scratch; returns the row's unscale.
template <int NP, bool EXACT>
__device__ __forceinline__ float put_row(float4 x, int row, int l, char *tile, char *image)
{
    float scale = 1.f, back = 1.f;
    if (!EXACT) {  // binary16 inputs are their own halves
        const float m = warp_max(fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w))));
        dev::row_scale(m, &scale, &back);
    }
    uint32_t hi[2], lo[2];
    dev::split_half(x.x * scale, x.y * scale, &hi[0], &lo[0]);
    dev::split_half(x.z * scale, x.w * scale, &hi[1], &lo[1]);
    const int at = tile_at(row, 4 * l);
    const uint2 h = make_uint2(hi[0], hi[1]), o = make_uint2(lo[0], lo[1]);
    *reinterpret_cast<uint2 *>(tile + at) = h;
    *reinterpret_cast<uint2 *>(image + at) = h;
    if (NP == 2) {
        *reinterpret_cast<uint2 *>(tile + kTileBytes + at) = o;
        *reinterpret_cast<uint2 *>(image + kTileBytes + at) = o;
    }
    return back;
}

// acc[j] = rows 16 m .. 16 m + 15 of A times rows 8 j .. of B transposed, for
// the column tiles j < tiles (a multiple of 2): A and B operand tiles in
// shared memory.
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
#pragma unroll
        for (int j = 0; j < kC / 8; j += 2) {
            if (j >= tiles) continue;
            uint32_t bh[4], bl[4];
            ldsm4(bh, b0 + tile_at(8 * j + brow, 16 * i + bcol));
            if (NP == 2) {
                ldsm4(bl, b0 + kTileBytes + tile_at(8 * j + brow, 16 * i + bcol));
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    mma16816(acc[j + e], al[0], al[1], al[2], al[3], bh[2 * e], bh[2 * e + 1]);
                    mma16816(acc[j + e], ah[0], ah[1], ah[2], ah[3], bl[2 * e], bl[2 * e + 1]);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; e++) mma16816(acc[j + e], ah[0], ah[1], ah[2], ah[3], bh[2 * e], bh[2 * e + 1]);
        }
    }
}

constexpr int kLd = kC + 4;  // row of a [64][64] fp32 matrix in shared memory

// The lower triangle of a [64][64] fp32 matrix, rows as scaled halves, into the
// scratch; the rows' unscales into back[].  Columns past the row's block of 16
// are not written (and not read).
__device__ __forceinline__ void put_square(const float *x, char *image, float *back)
{
    const int row = threadIdx.x >> 2, part = threadIdx.x & 3;  // 256 threads: 16 columns each
    const bool inside = part <= row >> 4;
    float v[16], m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (inside) y = *reinterpret_cast<const float4 *>(x + row * kLd + 16 * part + i);
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

// inv = (I + A)^-1 for the strictly lower triangular A [64][64] (both in shared
// memory, 256 threads): the four diagonal blocks of 16 by substitution, then
// twice the rule inv_21 = -inv_22 A_21 inv_11 for the blocks below.  tmp: room
// for a [32][33] matrix.  Only the lower triangle of inv (and the rest of its
// diagonal blocks of 16) is written.
__device__ void invert_lower(const float *A, float *inv, float *tmp)
{
    const int tid = threadIdx.x;
    if (tid < kC) {
        const int b = tid & ~15, j = tid & 15;
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; r++) {
            float s = 0.f;
#pragma unroll
            for (int m = 0; m < r; m++) s = fmaf(A[(b + r) * kLd + b + m], x[m], s);
            x[r] = r < j ? 0.f : (r == j ? 1.f : -s);
            inv[(b + r) * kLd + b + j] = x[r];
        }
    }
    __syncthreads();
#pragma unroll
    for (int h = 16; h <= 32; h *= 2) {
        // 64 / 2h pairs of h x h outputs, h h / 2 ... : 4 (h = 32) or 2 rows of one column a thread
        const int rows = h / 8;
        const int j = tid & (h - 1), i0 = (tid / h) % (h / rows) * rows, pair = tid / (h * (h / rows));
        const int lo = 2 * h * pair, hi = lo + h;
        float x[4] = {};
        for (int m = 0; m < h; m++) {
            const float t = inv[(lo + m) * kLd + lo + j];
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (e < rows) x[e] = fmaf(A[(hi + i0 + e) * kLd + lo + m], m >= j ? t : 0.f, x[e]);
        }
        float *X = tmp + pair * h * (h + 1);
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (e < rows) X[(i0 + e) * (h + 1) + j] = x[e];
        __syncthreads();
        float y[4] = {};
        for (int m = 0; m < h; m++) {
            const float t = X[m * (h + 1) + j];
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (e < rows) y[e] = fmaf(m <= i0 + e ? inv[(hi + i0 + e) * kLd + hi + m] : 0.f, t, y[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (e < rows) inv[(hi + i0 + e) * kLd + lo + j] = -y[e];
        __syncthreads();
    }
}

// What a tile kernel's CTA works on: a block of a live request.
struct Block {
    int b, r, t0, n;  // block of this launch, request, first token row, tokens
};

__device__ __forceinline__ bool find_block(const PromptArgs &a, int first_block, int b, Block *k)
{
    const int g = first_block + b;
    k->b = b;
    k->r = a.p.block_request[g];
    if (k->r < 0 || a.p.live[k->r] < 0) return false;
    const int end = a.p.starts[k->r + 1];
    k->t0 = a.p.starts[k->r] + a.p.block_first[g];
    k->n = min(kC, end - k->t0);
    return true;
}

// ---------------------------------------------------------------------------
// The blocks' own products, one gate a head.  A CTA takes a block and a query /
// key head: K K^T and Q K^T on the tensor cores (warps 0-3 and 4-7, 16 rows
// each), then for each value head of the group the decays, the inverse and P.
// ---------------------------------------------------------------------------
template <class T, int V, int NP>
__global__ void __launch_bounds__(256) k_block_tiles(PromptArgs a, int first_block, Scratch sc)
{
    extern __shared__ __align__(128) char smem[];
    __shared__ float ek[kC], eq[kC], s_alpha[kC], s_beta[kC], s_inv[kC], s_p[kC];
    const int tid = threadIdx.x, w = tid >> 5, l = tid & 31, g = l >> 2, c = l & 3;
    const int heads_k = a.heads / a.share;
    Block k;
    const int hq = blockIdx.x % heads_k;
    if (!find_block(a, first_block, blockIdx.x / heads_k, &k)) return;
    char *tk = smem, *tq = smem + NP * kTileBytes;
    {
        const size_t at = ((size_t)k.b * heads_k + hq) * NP * kTileBytes;
        char *ik = reinterpret_cast<char *>(a.scratch) + sc.k + at, *iq = reinterpret_cast<char *>(a.scratch) + sc.q + at;
        const T *kg = static_cast<const T *>(a.k) + hq * kDK, *qg = static_cast<const T *>(a.q) + hq * kDK;
        constexpr bool exact = sizeof(T) == 2 && !std::is_same<T, __nv_bfloat16>::value;
#pragma unroll
        for (int i = 0; i < kC / 8; i++) {
            const int row = 8 * w + i;
            float4 xk = make_float4(0.f, 0.f, 0.f, 0.f), xq = xk;
            if (row < k.n) {
                xk = load4(kg + (long long)(k.t0 + row) * a.stride_k + 4 * l);
                xq = load4(qg + (long long)(k.t0 + row) * a.stride_q + 4 * l);
            }
            const float bk = put_row<NP, exact>(xk, row, l, tk, ik), bq = put_row<NP, exact>(xq, row, l, tq, iq);
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
    float *sD = reinterpret_cast<float *>(smem), *sA = sD + kC * kLd, *sP = sA + kC * kLd, *sI = sP + kC * kLd;
    for (int v = 0; v < a.share; v++) {
        const int h = hq * a.share + v;
        __syncthreads();
        if (tid < kC) {
            const bool in = tid < k.n;
            s_alpha[tid] = in ? a.alpha[(long long)(k.t0 + tid) * a.heads + h] : 1.f;
            s_beta[tid] = in ? a.beta[(long long)(k.t0 + tid) * a.heads + h] : 0.f;
        }
        __syncthreads();
        {
            // decay_ts: column s, 16 rows a thread
            const int s = tid & (kC - 1), seg = 16 * (tid / kC);
            float p = 1.f;
            for (int r = s + 1; r < seg; r++) p *= s_alpha[r];
#pragma unroll
            for (int i = 0; i < 16; i++) {
                const int t = seg + i;
                if (t > s) p *= s_alpha[t];
                sD[t * kLd + s] = t >= s ? p : 0.f;
            }
        }
        __syncthreads();
        {
            float *dst = is_q ? sP : sA;
            const int t0 = 16 * m + g, t1 = t0 + 8;
            const float b0 = is_q ? 1.f : s_beta[t0], b1 = is_q ? 1.f : s_beta[t1];
            if (is_q || V != kLinear) {
#pragma unroll
                for (int j = 0; j < kC / 8; j++) {
                    if (j >= 2 * m + 2) continue;
                    const int s = 8 * j + 2 * c;
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const bool in0 = is_q ? s + e <= t0 : s + e < t0, in1 = is_q ? s + e <= t1 : s + e < t1;
                        dst[t0 * kLd + s + e] = in0 ? acc[j][e] * sD[t0 * kLd + s + e] * b0 : 0.f;
                        dst[t1 * kLd + s + e] = in1 ? acc[j][2 + e] * sD[t1 * kLd + s + e] * b1 : 0.f;
                    }
                }
            }
        }
        const size_t bh = (size_t)k.b * a.heads + h;
        float *sv = reinterpret_cast<float *>(a.scratch + sc.sv) + bh * kStateFloats;
        float *ov = reinterpret_cast<float *>(a.scratch + sc.ov) + bh * kOutFloats;
        const float a0 = s_alpha[0];
        if (tid < kC) {
            const float ct = sD[tid * kLd] * a0;
            sv[tid] = ct * ek[tid];
            sv[kC + tid] = s_beta[tid];
            sv[3 * kC + tid] = sD[(kC - 1) * kLd + tid] * ek[tid];
            ov[tid] = ct * eq[tid];
            if (tid == 0) sv[4 * kC] = sD[(kC - 1) * kLd] * a0;
        }
        __syncthreads();
        if (V != kLinear) invert_lower(sA, sI, sD);
        put_square(sP, reinterpret_cast<char *>(a.scratch) + sc.p + bh * kSquareBytes, s_p);
        if (V != kLinear) put_square(sI, reinterpret_cast<char *>(a.scratch) + sc.inv + bh * kSquareBytes, s_inv);
        __syncthreads();
        if (tid < kC) {
            sv[2 * kC + tid] = V == kLinear ? 1.f : s_inv[tid];
            ov[kC + tid] = s_p[tid];
        }
    }
}

// ---------------------------------------------------------------------------
// The walk over a request's blocks.  The state is held transposed: a state warp
// owns 16 value columns x 128 key rows as fp32 accumulators, whose register
// layout is also the layout of a product's left operand, so state, U and the
// state's update pass from product to product without leaving the registers.
// A second warp beside each state warp makes the output from the same halves,
// off the chain from block to block.  Operand tiles come by bulk copies.
// ---------------------------------------------------------------------------
enum { kPartK, kPartInv, kPartQ, kPartP, kPartK2, kParts };

template <class T, int V, int NP, int NR>
struct Walk {
    static constexpr int kKStages = V == kKda ? 1 : 2;  // K is read again at the block's end
    static constexpr int kThreads = 32 * 2 * NR;  // no copying warp: a ninth warp would cost the others a third of their registers
    static constexpr int kKBytes = NP * kTileBytes;
    static constexpr int kInvBytes = (V == kLinear ? 0 : kSquareBytes) + kStateFloats * 4;
    static constexpr int kPBytes = kSquareBytes + kOutFloats * 4;
    static constexpr int kVRow = sizeof(T) == 4 ? 80 : 48;  // bytes of a V row in shared memory (16 columns and a pad)
    // exchange of a state warp with its output warp: halves of S (8 k-steps x 2 x 512), of U (4 x 2 x 512), unscales
    static constexpr int kXBytes = 8192 + 4096 + 128;
    static constexpr int oK = 0;
    static constexpr int oInv = oK + kKStages * kKBytes;
    static constexpr int oQ = oInv + kInvBytes;
    static constexpr int oP = oQ + kKBytes;
    static constexpr int oK2 = oP + kPBytes;
    static constexpr int oX = oK2 + (V == kKda ? kKBytes : 0);
    static constexpr int oV = oX + NR * kXBytes;
    static constexpr int oBar = oV + NR * 2 * kC * kVRow;
    static constexpr int kBars = kParts + 1 + 4 * NR;
    static constexpr int oCount = oBar + 8 * kBars;
    static constexpr int kBytes = oCount + 4 * (kParts + 1);
    static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
};

__device__ __forceinline__ void cp_async16(void *dst, const void *src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dev::smem_addr(dst)), "l"(src), "r"(in ? 16 : 0) : "memory");
}

// Maximum over the four lanes that share a row of an accumulator.
__device__ __forceinline__ float quad_max(float m)
{
    m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
    return fmaxf(m, __shfl_xor_sync(kFull, m, 2));
}

// An accumulator of N column tiles as the halves of a left operand; the rows'
// unscales in back0 (row g) and back1 (row g + 8).
template <int N>
__device__ __forceinline__ void split_rows(const float (*x)[4], uint32_t (*hi)[4], uint32_t (*lo)[4], float *back0, float *back1)
{
    float m0 = 0.f, m1 = 0.f;
#pragma unroll
    for (int j = 0; j < N; j++) {
        m0 = fmaxf(m0, fmaxf(fabsf(x[j][0]), fabsf(x[j][1])));
        m1 = fmaxf(m1, fmaxf(fabsf(x[j][2]), fabsf(x[j][3])));
    }
    float s0, s1;
    dev::row_scale(quad_max(m0), &s0, back0);
    dev::row_scale(quad_max(m1), &s1, back1);
#pragma unroll
    for (int i = 0; i < N / 2; i++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
            dev::split_half(x[2 * i + e][0] * s0, x[2 * i + e][1] * s0, &hi[i][2 * e], &lo[i][2 * e]);
            dev::split_half(x[2 * i + e][2] * s1, x[2 * i + e][3] * s1, &hi[i][2 * e + 1], &lo[i][2 * e + 1]);
        }
}

__device__ __forceinline__ void v_pair(const char *tile, int row, int col, float *x, float)
{
    x[0] = *reinterpret_cast<const float *>(tile + row * 80 + col * 4);
    x[1] = *reinterpret_cast<const float *>(tile + (row + 1) * 80 + col * 4);
}

template <class T, int V, int NP, int NR>
__global__ void __launch_bounds__(Walk<T, V, NP, NR>::kThreads, 1) k_block_walk(PromptArgs a, int first_block, int n_blocks, Scratch sc)
{
    using W = Walk<T, V, NP, NR>;
    extern __shared__ __align__(128) char smem[];
    // a barrier and a counter for each part (K has two stages, the second last), four barriers a pair of warps
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + W::oBar), *xbar = full + kParts + 1;
    unsigned *used = reinterpret_cast<unsigned *>(smem + W::oCount);
    const int tid = threadIdx.x, w = tid >> 5, l = tid & 31, g = l >> 2, c = l & 3;
    constexpr int slices = kDV / (16 * NR);
    const int slice = blockIdx.x % slices, item = blockIdx.x / slices;
    const int r = item / a.heads, h = item - r * a.heads;
    const int live = a.p.live[r];
    if (live < 0) return;
    // the request's blocks of this launch
    const int all0 = a.p.block_starts[r], b0 = max(all0, first_block), b1 = min(a.p.block_starts[r + 1], first_block + n_blocks);
    if (b0 >= b1) return;
    const int row0 = a.p.starts[r], row_end = a.p.starts[r + 1];
    if (tid == 0) {
        for (int i = 0; i <= kParts; i++) {
            dev::mbar_init(&full[i], 1);
            used[i] = 0;
        }
        for (int i = 0; i < 4 * NR; i++) dev::mbar_init(&xbar[i], 1);
        dev::fence_barrier_init();
    }
    __syncthreads();
    const int count = b1 - b0;
    int *status = a.p.head;
    auto wait = [&](uint64_t *bar, int parity) -> bool {
        if (dev::mbar_wait_bounded(bar, (uint32_t)parity, kWaitLimit)) return true;
        atomicOr(status, kPlanTimeout);
        return false;
    };
    // the copies of a part of the request's it-th block (one thread)
    auto copy = [&](int part, int it) {
        const int heads_k = V == kKda ? a.heads : a.heads / a.share, hk = V == kKda ? h : h / a.share;
        const size_t b = (size_t)(b0 - first_block + it);
        const size_t tile = (b * heads_k + hk) * W::kKBytes, bh = b * a.heads + h;
        const int stage = part == kPartK ? it % W::kKStages : 0;
        uint64_t *f = &full[stage ? kParts : part];
        const uint8_t *src = a.scratch;
        if (part == kPartInv) {
            dev::mbar_arrive_expect_tx(f, W::kInvBytes);
            if (V != kLinear) dev::bulk_g2s(smem + W::oInv, src + sc.inv + bh * kSquareBytes, kSquareBytes, f);
            dev::bulk_g2s(smem + W::oInv + W::kInvBytes - kStateFloats * 4, src + sc.sv + bh * kStateFloats * 4, kStateFloats * 4, f);
        } else if (part == kPartP) {
            dev::mbar_arrive_expect_tx(f, W::kPBytes);
            dev::bulk_g2s(smem + W::oP, src + sc.p + bh * kSquareBytes, kSquareBytes, f);
            dev::bulk_g2s(smem + W::oP + kSquareBytes, src + sc.ov + bh * kOutFloats * 4, kOutFloats * 4, f);
        } else {
            const int dst = part == kPartK ? W::oK + stage * W::kKBytes : (part == kPartQ ? W::oQ : W::oK2);
            dev::mbar_arrive_expect_tx(f, W::kKBytes);
            dev::bulk_g2s(smem + dst, src + (part == kPartK ? sc.k : (part == kPartQ ? sc.q : sc.k2)) + tile, W::kKBytes, f);
        }
    };
    // A warp is done with a part of block it: the last of the NR warps that read
    // it has the next block's copied into its place.
    auto release = [&](int part, int it) {
        __syncwarp();
        if (l == 0) {
            const int stages = part == kPartK ? W::kKStages : 1;
            unsigned *n = &used[part == kPartK && it % W::kKStages ? kParts : part], old;
            asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], 1;" : "=r"(old) : "r"(dev::smem_addr(n)) : "memory");
            if (old % NR == NR - 1 && it + stages < count) copy(part, it + stages);
        }
    };
    if (tid == 0) {
        copy(kPartK, 0);
        copy(kPartInv, 0);
        copy(kPartQ, 0);
        copy(kPartP, 0);
        if (V == kKda) copy(kPartK2, 0);
        if (W::kKStages == 2 && count > 1) copy(kPartK, 1);
    }

    const bool out_warp = w >= NR;
    const int wr = out_warp ? w - NR : w;  // row group of the CTA
    const int col0 = slice * 16 * NR + 16 * wr;  // its 16 value columns
    uint64_t *sfull = &xbar[4 * wr], *sempty = sfull + 1, *ufull = sfull + 2, *uempty = sfull + 3;
    char *xs = smem + W::oX + wr * W::kXBytes, *xu = xs + 8192;
    float *xback = reinterpret_cast<float *>(xs + 8192 + 4096);  // unscales of S [16] and of U [16]
    const int arow = (l & 7) + ((l >> 3) & 1) * 8, acol = (l >> 4) * 8;  // ldmatrix: rows of a left operand
    const int brow = (l & 7) + (l >> 4) * 8, bcol = ((l >> 3) & 1) * 8;  // two column tiles of a right operand

    if (out_warp) {
        // ---- output: rows are tokens ----
        const uint32_t q0 = dev::smem_addr(smem + W::oQ), p0 = dev::smem_addr(smem + W::oP);
        const float *ov = reinterpret_cast<const float *>(smem + W::oP + kSquareBytes);
        T *out = static_cast<T *>(a.out);
        for (int it = 0; it < count; it++) {
            const int par = it & 1, t0 = row0 + (b0 - all0 + it) * kC, n = min(kC, row_end - t0), nm = (n + 15) / 16;
            uint32_t hi[8][4], lo[8][4];
            if (!wait(sfull, par)) return;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const uint4 x = *reinterpret_cast<const uint4 *>(xs + (2 * i) * 512 + l * 16), y = *reinterpret_cast<const uint4 *>(xs + (2 * i + 1) * 512 + l * 16);
                hi[i][0] = x.x; hi[i][1] = x.y; hi[i][2] = x.z; hi[i][3] = x.w;
                lo[i][0] = y.x; lo[i][1] = y.y; lo[i][2] = y.z; lo[i][3] = y.w;
            }
            float sb[2][2];
#pragma unroll
            for (int e = 0; e < 2; e++) { sb[e][0] = xback[8 * e + 2 * c]; sb[e][1] = xback[8 * e + 2 * c + 1]; }
            __syncwarp();
            if (l == 0) dev::mbar_arrive(sempty);
            if (!wait(&full[kPartQ], par)) return;
            float o[4][2][4] = {};
#pragma unroll
            for (int i = 0; i < 8; i++)
#pragma unroll
                for (int m = 0; m < 4; m++) {
                    if (m >= nm) continue;
                    uint32_t x[4];
                    ldsm4(x, q0 + tile_at(16 * m + arow, 16 * i + acol));
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        mma16816(o[m][e], x[0], x[1], x[2], x[3], lo[i][e], lo[i][2 + e]);
                        mma16816(o[m][e], x[0], x[1], x[2], x[3], hi[i][e], hi[i][2 + e]);
                    }
                    if (NP == 2) {
                        ldsm4(x, q0 + kTileBytes + tile_at(16 * m + arow, 16 * i + acol));
#pragma unroll
                        for (int e = 0; e < 2; e++) mma16816(o[m][e], x[0], x[1], x[2], x[3], hi[i][e], hi[i][2 + e]);
                    }
                }
            release(kPartQ, it);
            if (!wait(ufull, par)) return;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint4 x = *reinterpret_cast<const uint4 *>(xu + (2 * i) * 512 + l * 16), y = *reinterpret_cast<const uint4 *>(xu + (2 * i + 1) * 512 + l * 16);
                hi[i][0] = x.x; hi[i][1] = x.y; hi[i][2] = x.z; hi[i][3] = x.w;
                lo[i][0] = y.x; lo[i][1] = y.y; lo[i][2] = y.z; lo[i][3] = y.w;
            }
            float ub[2][2];
#pragma unroll
            for (int e = 0; e < 2; e++) { ub[e][0] = xback[16 + 8 * e + 2 * c]; ub[e][1] = xback[16 + 8 * e + 2 * c + 1]; }
            __syncwarp();
            if (l == 0) dev::mbar_arrive(uempty);
            if (!wait(&full[kPartP], par)) return;
#pragma unroll
            for (int m = 0; m < 4; m++) {
                if (m >= nm) continue;
                float p[2][4] = {};
#pragma unroll
                for (int i = 0; i <= m; i++) {
                    uint32_t x[4], y[4];
                    ldsm4(x, p0 + square_at(16 * m + arow, 16 * i + acol));
                    ldsm4(y, p0 + kSquareBytes / 2 + square_at(16 * m + arow, 16 * i + acol));
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        mma16816(p[e], x[0], x[1], x[2], x[3], lo[i][e], lo[i][2 + e]);
                        mma16816(p[e], y[0], y[1], y[2], y[3], hi[i][e], hi[i][2 + e]);
                        mma16816(p[e], x[0], x[1], x[2], x[3], hi[i][e], hi[i][2 + e]);
                    }
                }
#pragma unroll
                for (int d = 0; d < 2; d++) {
                    const int t = 16 * m + g + 8 * d;
                    if (t >= n) continue;
                    const float fq = ov[t], fp = ov[kC + t];
                    T *dst = out + ((long long)(t0 + t) * a.heads + h) * kDV + col0 + 2 * c;
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const float x = fmaf(o[m][e][2 * d], fq * sb[e][0], p[e][2 * d] * (fp * ub[e][0]));
                        const float y = fmaf(o[m][e][2 * d + 1], fq * sb[e][1], p[e][2 * d + 1] * (fp * ub[e][1]));
                        if constexpr (sizeof(T) == 4) {
                            *reinterpret_cast<float2 *>(dst + 8 * e) = make_float2(x, y);
                        } else if constexpr (std::is_same<T, __half>::value) {
                            *reinterpret_cast<__half2 *>(dst + 8 * e) = __floats2half2_rn(x, y);
                        } else {
                            *reinterpret_cast<__nv_bfloat162 *>(dst + 8 * e) = __floats2bfloat162_rn(x, y);
                        }
                    }
                }
            }
            release(kPartP, it);
        }
        return;
    }

    // ---- state: rows are value columns ----
    float *Sp = a.S + ((long long)(a.by_slot ? live : r) * a.heads + h) * (kDK * kDV) + col0 + g;
    float s[16][4];
    const bool zero = a.p.fresh[r] != 0 && b0 == all0;
#pragma unroll
    for (int j = 0; j < 16; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) s[j][e] = zero ? 0.f : Sp[(8 * j + 2 * c + (e & 1)) * kDV + 8 * (e >> 1)];
    char *vt = smem + W::oV + wr * 2 * kC * W::kVRow;
    const T *vg = static_cast<const T *>(a.v) + h * kDV + col0;
    auto fetch_v = [&](int it) {
        const int t0 = row0 + (b0 - all0 + it) * kC;
        char *dst = vt + (it & 1) * kC * W::kVRow;
        constexpr int chunks = 16 * sizeof(T) / 16;  // 16-byte pieces of a row
#pragma unroll
        for (int i = 0; i < chunks * kC / 32; i++) {
            const int x = i * 32 + l, row = x / chunks, part = x % chunks, t = t0 + row;
            cp_async16(dst + row * W::kVRow + part * 16, vg + (long long)min(t, row_end - 1) * a.stride_v + part * (16 / (int)sizeof(T)), t < row_end);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch_v(0);
    const float *sv = reinterpret_cast<const float *>(smem + W::oInv + W::kInvBytes - kStateFloats * 4);
    const uint32_t inv0 = dev::smem_addr(smem + W::oInv);
    for (int it = 0; it < count; it++) {
        const int par = it & 1, t0 = row0 + (b0 - all0 + it) * kC, nk = (min(kC, row_end - t0) + 15) / 16;
        const int stage = it % W::kKStages, kpar = (it / W::kKStages) & 1;
        uint64_t *kfull = &full[stage ? kParts : kPartK];
        const uint32_t k0 = dev::smem_addr(smem + W::oK + stage * W::kKBytes);
        if (it + 1 < count) {
            fetch_v(it + 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncwarp();
        float y[8][4] = {};
        float sb0, sb1;
        {
            uint32_t hi[8][4], lo[8][4];
            split_rows<16>(s, hi, lo, &sb0, &sb1);
            // the output warp has taken the halves of the block before
            if (!wait(sempty, par ^ 1)) return;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                *reinterpret_cast<uint4 *>(xs + (2 * i) * 512 + l * 16) = make_uint4(hi[i][0], hi[i][1], hi[i][2], hi[i][3]);
                *reinterpret_cast<uint4 *>(xs + (2 * i + 1) * 512 + l * 16) = make_uint4(lo[i][0], lo[i][1], lo[i][2], lo[i][3]);
            }
            if (c == 0) { xback[g] = sb0; xback[g + 8] = sb1; }
            __syncwarp();
            if (l == 0) dev::mbar_arrive(sfull);
            if (V != kLinear || it == 0)
                if (!wait(kfull, kpar)) return;
            if (V != kLinear) {
#pragma unroll
                for (int i = 0; i < 8; i++)
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        if (j >= 2 * nk) continue;
                        uint32_t x[4];
                        ldsm4(x, k0 + tile_at(8 * j + brow, 16 * i + bcol));
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            mma16816(y[j + e], lo[i][0], lo[i][1], lo[i][2], lo[i][3], x[2 * e], x[2 * e + 1]);
                            mma16816(y[j + e], hi[i][0], hi[i][1], hi[i][2], hi[i][3], x[2 * e], x[2 * e + 1]);
                        }
                        if (NP == 2) {
                            ldsm4(x, k0 + kTileBytes + tile_at(8 * j + brow, 16 * i + bcol));
#pragma unroll
                            for (int e = 0; e < 2; e++) mma16816(y[j + e], hi[i][0], hi[i][1], hi[i][2], hi[i][3], x[2 * e], x[2 * e + 1]);
                        }
                    }
            }
        }
        if (V == kKda) release(kPartK, it);
        if (!wait(&full[kPartInv], par)) return;
        // r = beta (v - y)
        {
            const char *tile = vt + (it & 1) * kC * W::kVRow;
            const uint32_t v0 = dev::smem_addr(tile);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                float v[2][4];  // of column tiles j, j + 1: rows g and g + 8, tokens 2 c, 2 c + 1
                if constexpr (sizeof(T) == 4) {
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        v_pair(tile, 8 * (j + e) + 2 * c, g, &v[e][0], 0.f);
                        v_pair(tile, 8 * (j + e) + 2 * c, g + 8, &v[e][2], 0.f);
                    }
                } else {
                    // matrices: tokens 8 j.. x columns 0.., tokens 8 j.. x columns 8.., then tokens 8 (j + 1)..
                    uint32_t x[4];
                    ldsm4_t(x, v0 + (8 * j + (l & 7) + (l >> 4) * 8) * W::kVRow + ((l >> 3) & 1) * 16);
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        float2 f;
                        if constexpr (std::is_same<T, __half>::value)
                            f = __half22float2(*reinterpret_cast<const __half2 *>(&x[e]));
                        else
                            f = make_float2(__uint_as_float(x[e] << 16), __uint_as_float(x[e] & 0xffff0000u));
                        v[e >> 1][2 * (e & 1)] = f.x;
                        v[e >> 1][2 * (e & 1) + 1] = f.y;
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int t = 8 * (j + e) + 2 * c;
                    const float2 fy = *reinterpret_cast<const float2 *>(&sv[t]), be = *reinterpret_cast<const float2 *>(&sv[kC + t]);
                    float *yy = y[j + e];
                    yy[0] = be.x * fmaf(-yy[0], fy.x * sb0, v[e][0]);
                    yy[1] = be.y * fmaf(-yy[1], fy.y * sb0, v[e][1]);
                    yy[2] = be.x * fmaf(-yy[2], fy.x * sb1, v[e][2]);
                    yy[3] = be.y * fmaf(-yy[3], fy.y * sb1, v[e][3]);
                }
            }
        }
        uint32_t hi[4][4], lo[4][4];
        float b0s, b1s;
        if (V != kLinear) {
            split_rows<8>(y, hi, lo, &b0s, &b1s);
            // u = inv r: column tile j needs tokens s < 8 j + 8
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
#pragma unroll
                for (int e = 0; e < 2; e++)
#pragma unroll
                    for (int d = 0; d < 4; d++) y[j + e][d] = 0.f;
                if (j >= 2 * nk) continue;
#pragma unroll
                for (int i = 0; i <= j / 2; i++) {
                    uint32_t x[4], z[4];
                    ldsm4(x, inv0 + square_at(8 * j + brow, 16 * i + bcol));
                    ldsm4(z, inv0 + kSquareBytes / 2 + square_at(8 * j + brow, 16 * i + bcol));
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        mma16816(y[j + e], lo[i][0], lo[i][1], lo[i][2], lo[i][3], x[2 * e], x[2 * e + 1]);
                        mma16816(y[j + e], hi[i][0], hi[i][1], hi[i][2], hi[i][3], z[2 * e], z[2 * e + 1]);
                        mma16816(y[j + e], hi[i][0], hi[i][1], hi[i][2], hi[i][3], x[2 * e], x[2 * e + 1]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const float2 ft = *reinterpret_cast<const float2 *>(&sv[2 * kC + 8 * (j + e) + 2 * c]);
                    y[j + e][0] *= ft.x * b0s; y[j + e][1] *= ft.y * b0s;
                    y[j + e][2] *= ft.x * b1s; y[j + e][3] *= ft.y * b1s;
                }
            }
        }
        split_rows<8>(y, hi, lo, &b0s, &b1s);
        if (!wait(uempty, par ^ 1)) return;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            *reinterpret_cast<uint4 *>(xu + (2 * i) * 512 + l * 16) = make_uint4(hi[i][0], hi[i][1], hi[i][2], hi[i][3]);
            *reinterpret_cast<uint4 *>(xu + (2 * i + 1) * 512 + l * 16) = make_uint4(lo[i][0], lo[i][1], lo[i][2], lo[i][3]);
        }
        if (c == 0) { xback[16 + g] = b0s; xback[24 + g] = b1s; }
        __syncwarp();
        if (l == 0) dev::mbar_arrive(ufull);
        // u for the state: what of each token is left at the block's end
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const float2 fu = *reinterpret_cast<const float2 *>(&sv[3 * kC + 8 * j + 2 * c]);
            y[j][0] *= fu.x; y[j][1] *= fu.y; y[j][2] *= fu.x; y[j][3] *= fu.y;
        }
        split_rows<8>(y, hi, lo, &b0s, &b1s);
        const float keep = V == kKda ? 0.f : sv[4 * kC];
        if (V == kKda)
            if (!wait(&full[kPartK2], par)) return;
        if (V == kLinear && it > 0)
            if (!wait(kfull, kpar)) return;
        const uint32_t kk = V == kKda ? dev::smem_addr(smem + W::oK2) : k0;
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            // sums start from zero and are added to the state once, rounded to nearest
            float d[2][4] = {};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                if (i >= nk) continue;
                uint32_t x[4];
                // matrices: tokens 16 i.., 16 i + 8.. of key rows 8 j.., then of key rows 8 (j + 1)..
                ldsm4_t(x, kk + tile_at(16 * i + (l & 15), 8 * j + (l >> 4) * 8));
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    mma16816(d[e], lo[i][0], lo[i][1], lo[i][2], lo[i][3], x[2 * e], x[2 * e + 1]);
                    mma16816(d[e], hi[i][0], hi[i][1], hi[i][2], hi[i][3], x[2 * e], x[2 * e + 1]);
                }
                if (NP == 2) {
                    ldsm4_t(x, kk + kTileBytes + tile_at(16 * i + (l & 15), 8 * j + (l >> 4) * 8));
#pragma unroll
                    for (int e = 0; e < 2; e++) mma16816(d[e], hi[i][0], hi[i][1], hi[i][2], hi[i][3], x[2 * e], x[2 * e + 1]);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; e++) {
                float2 kp = make_float2(keep, keep);
                if (V == kKda) kp = *reinterpret_cast<const float2 *>(&sv[4 * kC + 8 * (j + e) + 2 * c]);
                s[j + e][0] = fmaf(kp.x, s[j + e][0], d[e][0] * b0s);
                s[j + e][1] = fmaf(kp.y, s[j + e][1], d[e][1] * b0s);
                s[j + e][2] = fmaf(kp.x, s[j + e][2], d[e][2] * b1s);
                s[j + e][3] = fmaf(kp.y, s[j + e][3], d[e][3] * b1s);
            }
        }
        release(kPartInv, it);
        release(V == kKda ? kPartK2 : kPartK, it);
    }
#pragma unroll
    for (int j = 0; j < 16; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) Sp[(8 * j + 2 * c + (e & 1)) * kDV + 8 * (e >> 1)] = s[j][e];
}

// Blocks of a launch: the scratch stays near this size however long the batch is.
constexpr size_t kScratchTarget = (size_t)256 << 20;

int launch_blocks(const PromptArgs &a)
{
    const size_t one = scratch_of(a.variant, a.dtype, a.heads, a.share, 1).total;
    const long long fit = (long long)(kScratchTarget / one);
    return (int)std::max(1LL, std::min((long long)a.p.blocks, fit));
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

template <class T, int V, int NP, int NR>
cudaError_t launch_walk(const PromptArgs &a, int first, int n, const Scratch &sc, cudaStream_t s)
{
    using W = Walk<T, V, NP, NR>;
    cudaError_t e = cudaFuncSetAttribute(k_block_walk<T, V, NP, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, W::kBytes);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)a.p.requests * (unsigned)a.heads * (kDV / (16 * NR));
    k_block_walk<T, V, NP, NR><<<grid, W::kThreads, W::kBytes, s>>>(a, first, n, sc);
    return cudaGetLastError();
}

template <class T, int V, int NP>
cudaError_t launch_t(const PromptArgs &a, cudaStream_t s)
{
    const int step = launch_blocks(a);
    const Scratch sc = scratch_of(a.variant, a.dtype, a.heads, a.share, step);
    const long long items = (long long)a.p.requests * a.heads;
    for (int first = 0; first < a.p.blocks; first += step) {
        const int n = std::min(step, a.p.blocks - first);
        cudaError_t e = launch_tiles<T, V, NP>(a, first, n, sc, s);
        if (e != cudaSuccess) return e;
        e = items >= 74 ? launch_walk<T, V, NP, 4>(a, first, n, sc, s) : launch_walk<T, V, NP, 2>(a, first, n, sc, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <class T>
cudaError_t launch_v(const PromptArgs &a, cudaStream_t s)
{
    constexpr int NP = sizeof(T) == 4 ? 2 : 1;
    switch (a.variant) {
        case kGdn: return launch_t<T, kGdn, NP>(a, s);
        case kKda: return launch_prompt_steps(a, s);
        default: return launch_t<T, kLinear, NP>(a, s);
    }
}

}  // namespace

size_t prompt_scratch_bytes(const PromptArgs &a)
{
    if (a.p.blocks == 0 || a.variant == kKda) return 0;
    return scratch_of(a.variant, a.dtype, a.heads, a.share, launch_blocks(a)).total;
}

cudaError_t launch_prompt_blocks(const PromptArgs &a, cudaStream_t s)
{
    if (a.p.requests == 0 || a.p.tokens == 0) return cudaSuccess;
    switch (a.dtype) {
        case kF32: return launch_v<float>(a, s);
        case kF16: return launch_v<__half>(a, s);
        default: return launch_v<__nv_bfloat16>(a, s);
    }
}

}  // namespace stepq
