// The prompt pass in blocks of 64 tokens.
//
// With S the state before a block, c_t the running product of the gates inside
// it, and decay_ts = prod_(s<r<=t) alpha_r, the recurrence of a block is
//   A_ts = beta_t sum_d k_td decay_ts,d k_sd (s < t),     P_ts = sum_d q_td decay_ts,d k_sd (s <= t),
//   U = (I + A)^-1 (beta (V - (c K) S)),
//   out = (c Q) S + P U,        S <- c_64 S + (decay_64 K)^T U
// (plain linear attention: U = beta V).  What does not depend on the state is
// made for all blocks at once by a first kernel: decay_64 (I + A)^-1, which
// takes the residual R = beta (V - (c K) S) to the U the state's update needs,
// P (I + A)^-1, which takes it to the output, and the operands in the form the
// tensor cores take.  A second kernel walks each request's blocks in order and
// carries the state in registers.
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
#include "stepq_prompt_blocks.cuh"
#include "stepq_tcgen05.cuh"

namespace stepq {
namespace {

constexpr long long kWaitLimit = 1LL << 32;  // cycles, about two seconds

// ---------------------------------------------------------------------------
// The walk over a request's blocks: one CTA a state, all products on the
// fifth-generation tensor cores.  Everything is held transposed, value columns
// as the 128 lanes of tensor memory, so that each product's result, read from
// tensor memory by the threads of its lanes, scaled and split, goes back there
// as the next product's left operand:
//   Y = S^T K^T  ->  R = beta (V^T - Y)  ->  U = R (decay inv)^T  ->  S^T <- keep S^T + U K,
//   out^T = S^T Q^T + R (P inv)^T.
// Warps 0-15 keep the state (32 key rows of one value column a thread) and walk
// this chain; warps 16-19 finish the output, off the chain; warp 20 issues the
// products and the copies of the operands, warp 21 copies V.  Sums in tensor
// memory never pass from block to block: the state is updated in registers,
// rounded to nearest.
// A block is a chain of four products and three meetings of the 512 threads: 3.8
// us, 7.2 thousand cycles, with a gate a head in bf16 (one state's 128 blocks 484
// us: bound by that chain, not by bytes), 3.1 us plain.  512 states of 101 blocks
// in all, fp32: 120 us, 504 MB at 4.2 TB/s.
// ---------------------------------------------------------------------------
constexpr int kStateWarps = 16, kOutWarps = 4;
constexpr int kIssueWarp = kStateWarps + kOutWarps, kValueWarp = kIssueWarp + 1;
constexpr int kWalkThreads = 32 * (kValueWarp + 1);
// columns of tensor memory: Y, then the halves of R; S^T Q^T; U, then its
// halves; the output's second part; the state's update; the halves of S
constexpr int kColY = 0, kColSQ = 64, kColU = 128, kColUP = 192, kColD = 256, kColS = 384, kColumns = 512;

template <class T, int V, int NP>
struct Walk {
    // K is read again at the block's end, so that two lie side by side, except
    // with a gate per key row, which has other rows there; two Q (and the
    // output's scales), for the output may lag behind
    static constexpr int kKStages = V == kKda ? 1 : 2;
    static constexpr int kKBytes = NP * kTileBytes;
    static constexpr int kVRow = kDV * sizeof(T);
    static constexpr int oK = 0;
    static constexpr int oQ = oK + kKStages * kKBytes;
    static constexpr int oK2 = oQ + 2 * kKBytes;
    static constexpr int oInv = oK2 + (V == kKda ? kKBytes : 0);
    static constexpr int oP = oInv + (V == kLinear ? 0 : kSquareBytes);
    static constexpr int oV = oP + kSquareBytes;
    static constexpr int oSv = oV + kC * kVRow;
    static constexpr int oOv = oSv + 2 * kStateFloats * 4;
    static constexpr int oMax = oOv + 2 * kOutFloats * 4;   // [3][4][128] row maxima of the four quarters of the state warps
    static constexpr int oBack = oMax + 3 * 4 * kDV * 4;    // [2][2][128] unscales of S and R
    static constexpr int oBar = oBack + 2 * 2 * kDV * 4;
    static constexpr int oFlags = oBar + 8 * 32;            // tensor memory address; whether a wait gave up
    static constexpr int kBytes = oFlags + 8;
    static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
};

// Barriers.  Copies: K (2), Q with the output's scales (2), K2, the inverse, P,
// V, the state's scales (2).  Products done: Y, S^T Q^T, U, U P^T, update.
// Halves written: the even 16 key rows of S, and the odd ones; R, U.  Output
// read: S^T Q^T, U P^T.  The update's product comes in two, 64 key rows each.
enum {
    kFullK = 0, kFullQ = 2, kFullK2 = 4, kFullInv, kFullP, kFullV, kFullSv, kDoneY = 10, kDoneSQ, kDoneU, kDoneUP, kDoneD,
    kGotS0 = kDoneD + 2, kGotS, kGotR, kGotU, kReadSQ, kReadUP, kBarriers
};

__device__ __forceinline__ void cp_async16(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dev::smem_addr(dst)), "l"(src) : "memory");
}

// Row maxima of the four quarters of the state warps, exchanged: scale and
// unscale of N rows (one a thread), in one meeting of the 512 threads.
template <int N>
__device__ __forceinline__ void meet(float *sm, int quarter, int lane, const float *m, float *scale, float *back)
{
#pragma unroll
    for (int i = 0; i < N; i++) sm[(4 * i + quarter) * kDV + lane] = m[i];
    asm volatile("bar.sync 1, 512;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; i++) {
        const float *x = sm + 4 * i * kDV + lane;
        dev::row_scale(fmaxf(fmaxf(x[0], x[kDV]), fmaxf(x[2 * kDV], x[3 * kDV])), &scale[i], &back[i]);
    }
}

// N pairs x(i) of a row's numbers, times its scale, as halves into tensor memory.
template <int N, class F>
__device__ __forceinline__ void store_halves(uint32_t hi_at, uint32_t lo_at, float scale, const F &x)
{
    const float2 sc = make_float2(scale, scale);
#pragma unroll
    for (int i = 0; i < N; i += 8) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int j = 0; j < 8; j++) dev::split_half(__fmul2_rn(x(i + j), sc), &hi[j], &lo[j]);
        tc::st8(hi_at + i, hi);
        tc::st8(lo_at + i, lo);
    }
}

// The larger of m and the magnitudes of a pair.
__device__ __forceinline__ float max_abs(float m, float2 x)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(x.x)), "f"(fabsf(x.y)));
    return r;
}

__device__ __forceinline__ float2 pair_at(const float *p) { return *reinterpret_cast<const float2 *>(p); }

template <class T>
__device__ __forceinline__ float v_at(const char *row, int i);
template <>
__device__ __forceinline__ float v_at<float>(const char *row, int i) { return reinterpret_cast<const float *>(row)[i]; }
template <>
__device__ __forceinline__ float v_at<__half>(const char *row, int i) { return __half2float(reinterpret_cast<const __half *>(row)[i]); }
template <>
__device__ __forceinline__ float v_at<__nv_bfloat16>(const char *row, int i) { return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(row)[i]); }

template <class T>
__device__ __forceinline__ T to_t(float x);
template <>
__device__ __forceinline__ float to_t<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half to_t<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 to_t<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Requests of a batch up to which they are ordered: the ranking is a thread a
// request; with more, no request is long against the whole.
constexpr int kOrdered = 256;
static_assert(kOrdered <= kWalkThreads, "a request a thread");

template <class T, int V, int NP>
__global__ void __launch_bounds__(kWalkThreads, 1) k_block_walk(PromptArgs a, int first_block, int n_blocks, Scratch sc)
{
    using W = Walk<T, V, NP>;
    // no other shared memory, so that it starts at an aligned address the compiler knows
    extern __shared__ __align__(1024) char smem[];
    volatile int *s_dead = reinterpret_cast<volatile int *>(smem + W::oFlags + 4);
    const int tid = threadIdx.x, w = tid >> 5, l = tid & 31;
    int r = blockIdx.x / a.heads;
    const int h = blockIdx.x - r * a.heads;
    if (a.p.requests <= kOrdered) {
        // the requests with the most blocks go first: of a batch that fills the
        // GPU a few times over, a long one at the end would be waited for alone (16
        // requests of 1 to 1023 tokens, 32 heads: 120 us instead of 157, with a gate
        // per key row 126 instead of 172)
        int *n = reinterpret_cast<int *>(smem), *at = n + kOrdered;
        if (tid < a.p.requests) n[tid] = a.p.block_starts[tid + 1] - a.p.block_starts[tid];
        __syncthreads();
        if (tid < a.p.requests) {
            const int mine = n[tid];
            int rank = 0;
            for (int i = 0; i < a.p.requests; i++) rank += n[i] > mine || (n[i] == mine && i < tid);
            if (rank == r) *at = tid;
        }
        __syncthreads();
        r = *at;
        __syncthreads();
    }
    const int live = a.p.live[r];
    if (live < 0) return;
    // the request's blocks of this launch
    const int all0 = a.p.block_starts[r], b0 = max(all0, first_block), b1 = min(a.p.block_starts[r + 1], first_block + n_blocks);
    if (b0 >= b1) return;
    const int row0 = a.p.starts[r] + (b0 - all0) * kC, row_end = a.p.starts[r + 1], count = b1 - b0;
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + W::oBar);
    if (w == kIssueWarp) tc::alloc(reinterpret_cast<uint32_t *>(smem + W::oFlags), kColumns);
    if (tid == 0) {
        // operands have to lie at multiples of 1024 bytes
        *s_dead = (dev::smem_addr(smem) & 1023) != 0;
        if (*s_dead) atomicOr(a.p.head, kPlanTimeout);
        for (int i = 0; i < kBarriers; i++)
            dev::mbar_init(&bar[i], i == kGotS0 || i == kGotS || i == kGotR || i == kGotU ? kStateWarps : (i == kReadSQ || i == kReadUP ? kOutWarps : (i == kFullV ? 32 : 1)));
        dev::fence_barrier_init();
    }
    // rows of V behind the request's last are multiplied by zero: they must be finite
    for (int i = tid; i < kC * W::kVRow / 16; i += kWalkThreads) *reinterpret_cast<uint4 *>(smem + W::oV + 16 * i) = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    constexpr uint32_t tm = 0;  // all columns are this CTA's: they start at 0
    // Bounded: a wait that gives up marks the CTA dead, and nothing waits any
    // more; every thread runs to the end.
    auto wait = [&](int i, int parity) {
        if (dev::mbar_try_wait(&bar[i], (uint32_t)parity)) return;
        const long long t0 = clock64();
        while (!*s_dead && !dev::mbar_try_wait(&bar[i], (uint32_t)parity))
            if (clock64() - t0 > kWaitLimit) {
                *s_dead = 1;
                atomicOr(a.p.head, kPlanTimeout);
            }
    };
    auto arrive = [&](int i) {
        __syncwarp();
        if (l == 0) dev::mbar_arrive(&bar[i]);
    };
    const float *sv_all = reinterpret_cast<const float *>(smem + W::oSv), *ov_all = reinterpret_cast<const float *>(smem + W::oOv);
    float *s_max = reinterpret_cast<float *>(smem + W::oMax), *s_back = reinterpret_cast<float *>(smem + W::oBack);

    if (w == kValueWarp) {
        // ---- V: rows of the request's tokens, as 16-byte copies of all lanes (a bulk copy a row would cost its issue, 64 times) ----
        const T *vg = static_cast<const T *>(a.v) + h * kDV;
        constexpr int pieces = W::kVRow / 16, rows = 32 / pieces;  // rows at a time: two of 16-bit, one of 32-bit elements
        const T *src = vg + (long long)(row0 + l / pieces) * a.stride_v + l % pieces * (16 / (int)sizeof(T));
        char *dst = smem + W::oV + l / pieces * W::kVRow + l % pieces * 16;
        for (int it = 0; it < count; it++, src += kC * a.stride_v) {
            const int n = min(kC, row_end - row0 - it * kC);
            if (it > 0) wait(V == kLinear ? kGotU : kGotR, (it - 1) & 1);  // the rows before are read
            const T *p = src;
#pragma unroll 8
            for (int i = 0; i < kC / rows; i++, p += rows * a.stride_v)
                if (i * rows + l / pieces < n) cp_async16(dst + i * rows * W::kVRow, p);
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(dev::smem_addr(&bar[kFullV])) : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (w == kIssueWarp) {
        // ---- products and copies ----
        const int heads_k = V == kKda ? a.heads : a.heads / a.share, hk = V == kKda ? h : h / a.share;
        const size_t first = (size_t)(b0 - first_block);
        const uint8_t *src = a.scratch;
        auto tile = [&](int it) { return ((first + it) * heads_k + hk) * (size_t)W::kKBytes; };
        auto bh = [&](int it) { return (first + it) * a.heads + h; };
        auto copy = [&](int b, int dst, size_t from, int bytes) {
            if (tc::elect()) {
                dev::mbar_arrive_expect_tx(&bar[b], bytes);
                dev::bulk_g2s(smem + dst, src + from, bytes, &bar[b]);
            }
        };
        auto copy_k = [&](int it) { copy(kFullK + it % W::kKStages, W::oK + it % W::kKStages * W::kKBytes, sc.k + tile(it), W::kKBytes); };
        auto copy_q = [&](int it) {
            if (tc::elect()) {
                uint64_t *f = &bar[kFullQ + (it & 1)];
                dev::mbar_arrive_expect_tx(f, W::kKBytes + kOutFloats * 4);
                dev::bulk_g2s(smem + W::oQ + (it & 1) * W::kKBytes, src + sc.q + tile(it), W::kKBytes, f);
                dev::bulk_g2s(smem + W::oOv + (it & 1) * kOutFloats * 4, src + sc.ov + bh(it) * kOutFloats * 4, kOutFloats * 4, f);
            }
        };
        auto copy_sv = [&](int it) { copy(kFullSv + (it & 1), W::oSv + (it & 1) * kStateFloats * 4, sc.sv + bh(it) * kStateFloats * 4, kStateFloats * 4); };
        copy_k(0);
        copy_sv(0);
        copy_q(0);
        if (V == kKda) copy(kFullK2, W::oK2, sc.k2 + tile(0), W::kKBytes);
        if (V != kLinear) copy(kFullInv, W::oInv, sc.inv + bh(0) * kSquareBytes, kSquareBytes);
        copy(kFullP, W::oP, sc.p + bh(0) * kSquareBytes, kSquareBytes);
        const uint32_t base = dev::smem_addr(smem);
        // Products that share a right operand follow one another: in an order by
        // halves instead (low ones first, while the sums, which are cut off at
        // every product, are small) the operand is fetched anew each time, and a
        // block took 7.9 thousand cycles instead of 7.2, for an error of fp32
        // prompts of 5.2e-7 instead of 7e-7.
        // products of S^T with the rows of an operand tile, the even or odd 16s of key rows
        auto with_rows = [&](uint32_t d, uint32_t rows, int odd) {
            bool add = odd != 0;
#pragma unroll
            for (int i = odd; i < kDK / 16; i += 2) {
                const uint32_t at = rows + (i >> 2) * (kTileBytes / 2) + (i & 3) * 32;
                tc::mma(tm + d, tm + kColS + 64 + 8 * i, tc::desc(at, 16, 1024), tc::idesc(kC, false), add);
                add = true;
                if (NP == 2) tc::mma(tm + d, tm + kColS + 8 * i, tc::desc(at + kTileBytes, 16, 1024), tc::idesc(kC, false), add);
                tc::mma(tm + d, tm + kColS + 8 * i, tc::desc(at, 16, 1024), tc::idesc(kC, false), add);
            }
        };
        // products of a [128][64] left operand with a lower-triangular square, transposed
        auto with_square = [&](uint32_t d, uint32_t left, uint32_t square, int nk) {
#pragma unroll
            for (int i = 0; i < kC / 16; i++) {
                if (i >= nk) break;
                const uint32_t at = square + i * 2048 + i * 32, id = tc::idesc(kC - 16 * i, false);
                tc::mma(tm + d + 16 * i, tm + left + 32 + 8 * i, tc::desc(at, 16, 1024), id, i > 0);
                tc::mma(tm + d + 16 * i, tm + left + 8 * i, tc::desc(at + kSquareBytes / 2, 16, 1024), id, true);
                tc::mma(tm + d + 16 * i, tm + left + 8 * i, tc::desc(at, 16, 1024), id, true);
            }
        };
        // U times 64 columns of the rows of K: the inner dimension runs over tokens
        auto update = [&](uint32_t rows, int nk) {
#pragma unroll
            for (int e = 0; e < 2; e++) {
#pragma unroll
                for (int i = 0; i < kC / 16; i++) {
                    if (i >= nk) break;
                    const uint32_t at = rows + e * (kTileBytes / 2) + i * 2048, id = tc::idesc(kDK / 2, true), d = tm + kColD + 64 * e;
                    tc::mma(d, tm + kColU + 32 + 8 * i, tc::desc(at, kTileBytes / 2, 1024), id, i > 0);
                    if (NP == 2) tc::mma(d, tm + kColU + 8 * i, tc::desc(at + kTileBytes, kTileBytes / 2, 1024), id, true);
                    tc::mma(d, tm + kColU + 8 * i, tc::desc(at, kTileBytes / 2, 1024), id, true);
                }
                tc::commit(&bar[kDoneD + e]);
            }
        };
        for (int it = 0; it < count; it++) {
            const int par = it & 1, nk = (min(kC, row_end - row0 - it * kC) + 15) / 16;
            const uint32_t kt = base + W::oK + it % W::kKStages * W::kKBytes;
            const int kpar = (it / W::kKStages) & 1, qpar = (it >> 1) & 1;
            // S is there: the block before has updated the state, and read its
            // K, its P and its scales for the last time
            wait(kGotS0, par);
            tc::fence_after();
            if (V != kLinear) {
                wait(kFullK + it % W::kKStages, kpar);
                if (tc::elect()) with_rows(kColY, kt, 0);
            }
            wait(kGotS, par);
            tc::fence_after();
            if (V != kLinear && tc::elect()) {
                with_rows(kColY, kt, 1);
                tc::commit(&bar[kDoneY]);
            }
            if (it + 1 < count) {
                if (V != kKda) copy_k(it + 1);
                copy_sv(it + 1);
            }
            if (it > 0) {
                copy(kFullP, W::oP, sc.p + bh(it) * kSquareBytes, kSquareBytes);
                if (V == kKda) copy(kFullK2, W::oK2, sc.k2 + tile(it), W::kKBytes);
            }
            if (V == kLinear) {
                wait(kGotU, par);
                tc::fence_after();
                wait(kFullK + it % W::kKStages, kpar);
                if (tc::elect()) update(kt, nk);
            }
            wait(kFullQ + (it & 1), qpar);
            if (it > 0) wait(kReadSQ, par ^ 1);
            tc::fence_after();
            if (tc::elect()) {
                with_rows(kColSQ, base + W::oQ + (it & 1) * W::kKBytes, 0);
                with_rows(kColSQ, base + W::oQ + (it & 1) * W::kKBytes, 1);
                tc::commit(&bar[kDoneSQ]);
            }
            if (V != kLinear) {
                wait(kGotR, par);
                tc::fence_after();
                wait(kFullInv, par);
                if (tc::elect()) {
                    with_square(kColU, kColY, base + W::oInv, nk);
                    tc::commit(&bar[kDoneU]);
                }
                if (V == kKda && it + 1 < count) copy_k(it + 1);
            }
            wait(kFullP, par);
            if (it > 0) wait(kReadUP, par ^ 1);
            tc::fence_after();
            if (tc::elect()) {
                with_square(kColUP, kColY, base + W::oP, nk);
                tc::commit(&bar[kDoneUP]);
            }
            if (it + 1 < count) copy_q(it + 1);  // the output of the block before is out
            if (V != kLinear) {
                wait(kGotU, par);
                tc::fence_after();
                if (V == kKda) wait(kFullK2, par);
                if (tc::elect()) update(V == kKda ? base + W::oK2 : kt, nk);
                if (it + 1 < count) copy(kFullInv, W::oInv, sc.inv + bh(it + 1) * kSquareBytes, kSquareBytes);
            }
        }
        wait(kDoneUP, (count - 1) & 1);
    } else if (w >= kStateWarps) {
        // ---- output: a value column a thread ----
        const int lane = 32 * (w & 3) + l;
        const uint32_t tl = tm + ((uint32_t)(32 * (w & 3)) << 16);
        T *out = static_cast<T *>(a.out) + (long long)h * kDV + lane;
        const long long row = (long long)a.heads * kDV;
        for (int it = 0; it < count; it++) {
            const int par = it & 1, t0 = row0 + it * kC, n = min(kC, row_end - t0);
            const float *ov = ov_all + (it & 1) * kOutFloats;
            wait(kFullQ + (it & 1), (it >> 1) & 1);
            wait(kDoneSQ, par);
            wait(kDoneUP, par);
            tc::fence_after();
            const float sb = s_back[(2 * (it & 1)) * kDV + lane], rb = s_back[(2 * (it & 1) + 1) * kDV + lane];
            T *dst = out + (long long)t0 * row;
#pragma unroll
            for (int t1 = 0; t1 < kC; t1 += 16) {
                float2 o[8], p[8];
                tc::ld16(reinterpret_cast<uint32_t *>(o), tl + kColSQ + t1);
                tc::ld16(reinterpret_cast<uint32_t *>(p), tl + kColUP + t1);
#pragma unroll
                for (int t = 0; t < 8; t++) {
                    const float2 fq = __fmul2_rn(pair_at(ov + t1 + 2 * t), make_float2(sb, sb)), fp = __fmul2_rn(pair_at(ov + kC + t1 + 2 * t), make_float2(rb, rb));
                    o[t] = __ffma2_rn(p[t], fp, __fmul2_rn(o[t], fq));
                }
                if (n == kC) {
#pragma unroll
                    for (int t = 0; t < 8; t++, dst += 2 * row) {
                        dst[0] = to_t<T>(o[t].x);
                        dst[row] = to_t<T>(o[t].y);
                    }
                } else {
#pragma unroll
                    for (int t = 0; t < 8; t++, dst += 2 * row) {
                        if (t1 + 2 * t < n) dst[0] = to_t<T>(o[t].x);
                        if (t1 + 2 * t + 1 < n) dst[row] = to_t<T>(o[t].y);
                    }
                }
            }
            tc::fence_before();
            arrive(kReadSQ);
            arrive(kReadUP);
        }
    } else {
        // ---- state: 32 key rows of a value column a thread ----
        const int part = w >> 2, lane = 32 * (w & 3) + l;  // quarter of the key rows, and of the tokens; value column
        const uint32_t tl = tm + ((uint32_t)(32 * (w & 3)) << 16);
        float *Sp = a.S + ((long long)(a.by_slot ? live : r) * a.heads + h) * (kDK * kDV) + (32 * part) * kDV + lane;
        float2 s[16];
        const bool zero = a.p.fresh[r] != 0 && b0 == all0;
#pragma unroll
        for (int j = 0; j < 16; j++) s[j] = zero ? make_float2(0.f, 0.f) : make_float2(Sp[2 * j * kDV], Sp[(2 * j + 1) * kDV]);
        const char *vt = smem + W::oV + 16 * part * W::kVRow;
        auto v_pair = [&](int t) { return make_float2(v_at<T>(vt + 2 * t * W::kVRow, lane), v_at<T>(vt + (2 * t + 1) * W::kVRow, lane)); };
        // 16 key rows of the 32, and word of them
        auto store_s = [&](int e, float scale) {
            const uint32_t at = tl + kColS + 16 * part + 8 * e;
            store_halves<8>(at, at + 64, scale, [&](int j) { return s[8 * e + j]; });
            tc::wait_st();
            tc::fence_before();
            arrive(e == 0 ? kGotS0 : kGotS);
        };
        for (int it = 0; it < count; it++) {
            const int par = it & 1;
            // the block's scales: of this quarter's tokens
            const float *sv = sv_all + (it & 1) * kStateFloats, *fy = sv + 16 * part, *be = fy + kC, *fu = be + kC;
            float *s_out = s_back + (2 * (it & 1)) * kDV + lane;  // unscales of S and R for the output
            float m[3], scale[3], back[3];
            float2 y[8];
            m[0] = 0.f;
#pragma unroll
            for (int j = 0; j < 16; j++) m[0] = max_abs(m[0], s[j]);
            if (V == kLinear) {
                wait(kFullSv + (it & 1), (it >> 1) & 1);
                wait(kFullV, par);
                m[1] = m[2] = 0.f;
#pragma unroll
                for (int t = 0; t < 8; t++) {
                    y[t] = __fmul2_rn(pair_at(be + 2 * t), v_pair(t));
                    m[1] = max_abs(m[1], y[t]);
                    m[2] = max_abs(m[2], __fmul2_rn(y[t], pair_at(fu + 2 * t)));
                }
                meet<3>(s_max, part, lane, m, scale, back);
                // the output of the block before has read the halves of R
                if (it > 0) wait(kDoneUP, par ^ 1);
                tc::fence_after();
                store_halves<8>(tl + kColU + 8 * part, tl + kColU + 32 + 8 * part, scale[2], [&](int t) { return __fmul2_rn(y[t], pair_at(fu + 2 * t)); });
                store_halves<8>(tl + kColY + 8 * part, tl + kColY + 32 + 8 * part, scale[1], [&](int t) { return y[t]; });
                if (part == 0) {
                    s_out[0] = back[0];
                    s_out[kDV] = back[1];
                }
                tc::wait_st();
                tc::fence_before();
                arrive(kGotU);
                store_s(0, scale[0]);
                store_s(1, scale[0]);
            } else {
                meet<1>(s_max, part, lane, m, scale, back);
                const float2 sb = make_float2(back[0], back[0]);
                if (part == 0) s_out[0] = back[0];
                store_s(0, scale[0]);
                store_s(1, scale[0]);
                // r = beta (v - y), beta v before y is there
                wait(kFullSv + (it & 1), (it >> 1) & 1);
                wait(kFullV, par);
                float2 bv[8];
#pragma unroll
                for (int t = 0; t < 8; t++) bv[t] = __fmul2_rn(pair_at(be + 2 * t), v_pair(t));
                wait(kDoneY, par);
                tc::fence_after();
                tc::ld16(reinterpret_cast<uint32_t *>(y), tl + kColY + 16 * part);
                m[0] = 0.f;
#pragma unroll
                for (int t = 0; t < 8; t++) {
                    y[t] = __ffma2_rn(y[t], __fmul2_rn(pair_at(fy + 2 * t), sb), bv[t]);
                    m[0] = max_abs(m[0], y[t]);
                }
                meet<1>(s_max + 4 * kDV, part, lane, m, scale, back);
                store_halves<8>(tl + kColY + 8 * part, tl + kColY + 32 + 8 * part, scale[0], [&](int t) { return y[t]; });
                if (part == 0) s_out[kDV] = back[0];
                tc::wait_st();
                tc::fence_before();
                arrive(kGotR);
                // what of u = inv r is left at the block's end
                wait(kDoneU, par);
                tc::fence_after();
                const float2 rb = make_float2(back[0], back[0]);
                tc::ld16(reinterpret_cast<uint32_t *>(y), tl + kColU + 16 * part);
                m[0] = 0.f;
#pragma unroll
                for (int t = 0; t < 8; t++) {
                    y[t] = __fmul2_rn(y[t], __fmul2_rn(pair_at(fu + 2 * t), rb));
                    m[0] = max_abs(m[0], y[t]);
                }
                meet<1>(s_max + 8 * kDV, part, lane, m, scale, back);
                store_halves<8>(tl + kColU + 8 * part, tl + kColU + 32 + 8 * part, scale[0], [&](int t) { return y[t]; });
                tc::wait_st();
                tc::fence_before();
                arrive(kGotU);
                back[2] = back[0];
            }
            wait(kDoneD + (part >> 1), par);
            tc::fence_after();
            const float2 ub = make_float2(back[2], back[2]);
            const float keep = V == kKda ? 0.f : sv[3 * kC];
#pragma unroll
            for (int j1 = 0; j1 < 16; j1 += 8) {
                float2 d[8];
                tc::ld16(reinterpret_cast<uint32_t *>(d), tl + kColD + 32 * part + 2 * j1);
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const float2 kp = V == kKda ? pair_at(sv + 3 * kC + 32 * part + 2 * (j1 + j)) : make_float2(keep, keep);
                    s[j1 + j] = __ffma2_rn(kp, s[j1 + j], __fmul2_rn(d[j], ub));
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 16; j++) {
            Sp[2 * j * kDV] = s[j].x;
            Sp[(2 * j + 1) * kDV] = s[j].y;
        }
    }
    tc::fence_before();
    __syncthreads();
    if (w == kIssueWarp) tc::dealloc(tm, kColumns);
}

// Blocks of a launch: the scratch stays near this size however long the batch is.
// Longer batches go in turns of it, the state passing through memory between them
// (1 GB holds 658 blocks of 32 value and 16 query and key heads in bf16, with a
// gate a head).
constexpr size_t kScratchTarget = (size_t)1 << 30;

int launch_blocks(const PromptArgs &a)
{
    const size_t one = scratch_of(a.variant, a.dtype, a.heads, a.share, 1).total;
    const long long fit = (long long)(kScratchTarget / one);
    return (int)std::max(1LL, std::min((long long)a.p.blocks, fit));
}

template <class T, int V, int NP>
cudaError_t launch_walk(const PromptArgs &a, int first, int n, const Scratch &sc, cudaStream_t s)
{
    using W = Walk<T, V, NP>;
    cudaError_t e = cudaFuncSetAttribute(k_block_walk<T, V, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, W::kBytes);
    if (e != cudaSuccess) return e;
    k_block_walk<T, V, NP><<<(unsigned)a.p.requests * (unsigned)a.heads, kWalkThreads, W::kBytes, s>>>(a, first, n, sc);
    return cudaGetLastError();
}

template <class T, int V, int NP>
cudaError_t launch_t(const PromptArgs &a, cudaStream_t s)
{
    const int step = launch_blocks(a);
    const Scratch sc = scratch_of(a.variant, a.dtype, a.heads, a.share, step);
    for (int first = 0; first < a.p.blocks; first += step) {
        const int n = std::min(step, a.p.blocks - first);
        cudaError_t e = launch_block_tiles(a, first, n, sc, s);
        if (e != cudaSuccess) return e;
        e = launch_walk<T, V, NP>(a, first, n, sc, s);
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
        case kKda: return launch_t<T, kKda, 2>(a, s);
        default: return launch_t<T, kLinear, NP>(a, s);
    }
}

}  // namespace

size_t prompt_scratch_bytes(const PromptArgs &a)
{
    if (a.p.blocks == 0) return 0;
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
