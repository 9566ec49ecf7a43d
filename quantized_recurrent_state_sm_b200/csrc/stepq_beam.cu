// Beam search: selection over beams and vocabulary, and the reordering of the
// beams' rows (packed states, or any other per-request rows).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "stepq_serve.cuh"

namespace stepq {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kScanThreads = 256;
constexpr int kMergeThreads = 256;
constexpr int kMaxBeams = 64;        // STEPQ_MAX_BEAMS: beams of a group, and candidates
constexpr int kMaxMerge = 16384;     // candidates a group's merge looks at
constexpr int kMergeList = kMaxMerge / kMergeThreads * kMaxBeams;  // of which this many may pass its threshold

// A candidate of a row as one number: larger is better, equal values go to the
// lower token.  0: none (-inf, NaN).
__device__ __forceinline__ unsigned long long key_of(float x, int token)
{
    if (!(x > -INFINITY)) return 0;
    const unsigned u = __float_as_uint(x + 0.f);  // -0 and 0 are one value
    const unsigned o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return ((unsigned long long)o << 32) | (0xffffffffu - (unsigned)token);
}

__device__ __forceinline__ float value_of(unsigned long long key)
{
    const unsigned o = (unsigned)(key >> 32);
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

__device__ __forceinline__ int token_of(unsigned long long key) { return (int)(0xffffffffu - (unsigned)key); }

__device__ __forceinline__ void unpack4(const float4 &v, float *x, float)
{
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void unpack4(const float4 &v, float *x, __half)
{
    const __half2 *h = reinterpret_cast<const __half2 *>(&v);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 f = __half22float2(h[i]);
        x[2 * i] = f.x; x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void unpack4(const float4 &v, float *x, __nv_bfloat16)
{
    const unsigned *h = reinterpret_cast<const unsigned *>(&v);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        x[2 * i] = __uint_as_float(h[i] << 16); x[2 * i + 1] = __uint_as_float(h[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ float load_f(const float *p) { return *p; }
__device__ __forceinline__ float load_f(const __half *p) { return __half2float(*p); }
__device__ __forceinline__ float load_f(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

// Words first .. first + 4 of the 16-byte vectors a, b, moved down by `bits`.
template <int FIRST>
__device__ __forceinline__ float4 join_words(const uint4 &a, const uint4 &b, int bits)
{
    const unsigned w[9] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, 0};
    return make_float4(__uint_as_float(__funnelshift_r(w[FIRST], w[FIRST + 1], bits)),
                       __uint_as_float(__funnelshift_r(w[FIRST + 1], w[FIRST + 2], bits)),
                       __uint_as_float(__funnelshift_r(w[FIRST + 2], w[FIRST + 3], bits)),
                       __uint_as_float(__funnelshift_r(w[FIRST + 3], w[FIRST + 4], bits)));
}

// The 16 bytes at p, which lies `shift` bytes past a 16-byte boundary: both
// vectors they lie in must be readable.
__device__ __forceinline__ float4 load_16(const void *p, int shift)
{
    if (shift == 0) return *static_cast<const float4 *>(p);
    const uint4 *v = reinterpret_cast<const uint4 *>(static_cast<const char *>(p) - shift);
    const uint4 a = v[0], b = v[1];
    const int bits = (shift & 3) * 8;
    switch (shift >> 2) {
        case 0: return join_words<0>(a, b, bits);
        case 1: return join_words<1>(a, b, bits);
        case 2: return join_words<2>(a, b, bits);
        default: return join_words<3>(a, b, bits);
    }
}

__device__ __forceinline__ float max3(float x, float y, float z)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// What a CTA leaves of its part of a row: the n best, and the softmax
// statistics (largest logit, sum of exponentials below it).
struct RowStats {
    double sum;
    float top;
    int pad;
};

// ---------------------------------------------------------------------------
// One pass over the logits.  A CTA takes every `splits`-th tile of a row into
// registers (PER values a thread), sums the exponentials under a running
// maximum, and keeps the n best keys.  The worst of those kept so far bounds the
// n-th best from below, so a later tile mostly adds few values or none.  Where
// more than n threads are above that, the n-th largest of the maxima of 64 groups
// of four threads is a first bound, and the n-th largest of the few threads'
// maxima that reach it the second: at most n threads hold values above, which
// bounds the list that is ranked.
// Measured: 512 rows of 100003 bf16 logits (102 MB; odd rows, so every 16 bytes
// come from two loads) 75 us, bound by the tiles' chains of load, maximum and
// barriers (41 % issue); 4 rows of 32001 fp32 logits 6 us.
// ---------------------------------------------------------------------------
constexpr int kGroups = kScanThreads / 4;
static_assert(kGroups >= kMaxBeams, "as many groups as values can be kept");

template <class T, int PER>
__global__ void __launch_bounds__(kScanThreads) k_beam_scan(BeamArgs a, int splits, RowStats *stats,
                                                            unsigned long long *best)
{
    constexpr int E = 16 / sizeof(T), NV = PER / E;
    __shared__ unsigned long long s_group[kGroups], s_near[kScanThreads], s_list[kMaxBeams * PER + kMaxBeams], s_keep[kMaxBeams];
    __shared__ float s_top[kScanThreads / 32];
    __shared__ double s_sum[kScanThreads / 32];
    __shared__ unsigned long long s_low, s_tau;
    __shared__ int s_count, s_reach;
    const int tid = threadIdx.x, w = tid >> 5, l = tid & 31;
    const int row = blockIdx.x / splits, part = blockIdx.x - row * splits;
    const T *x0 = static_cast<const T *>(a.logits) + (long long)row * a.stride;
    // runs of 16 bytes from the row's first token, wherever it lies: equal rows
    // are then summed in the same order, and their ties stay ties
    const int shift = (int)(reinterpret_cast<uintptr_t>(x0) & 15);
    const int n_vec = (a.vocab + E - 1) / E;
    float top = -INFINITY;
    double sum = 0.0;
    int kept = 0;
    for (int v0 = part * kScanThreads * NV; v0 < n_vec; v0 += splits * kScanThreads * NV) {
        float x[PER];
        // token of value i: runs of E tokens, kScanThreads runs apart
        auto token = [&](int i) { return (v0 + i / E * kScanThreads + tid) * E + i % E; };
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int j = v0 + i * kScanThreads + tid, at = j * E;
            // the row's first and last run one by one where their vectors reach past the row
            if (j < n_vec && at + (shift ? 2 * E : E) <= a.vocab && (j > 0 || shift == 0)) {
                unpack4(load_16(x0 + at, shift), &x[i * E], T{});
            } else {
#pragma unroll
                for (int e = 0; e < E; e++)
                    x[i * E + e] = (j < n_vec && at + e < a.vocab) ? load_f(x0 + at + e) : -INFINITY;
            }
        }
        float m = -INFINITY;  // passes over NaN
#pragma unroll
        for (int i = 0; i < PER; i += 2) m = max3(m, x[i], x[i + 1]);
        // the thread's best, where it may count: of equal values the first
        const unsigned long long floor_key = kept == a.n ? s_keep[a.n - 1] : 0;
        unsigned long long mine = 0;
        if (m > -INFINITY && (floor_key == 0 || m >= value_of(floor_key))) {
            int first = 0;
#pragma unroll
            for (int i = PER - 1; i >= 0; i--) first = x[i] == m ? i : first;
            mine = key_of(m, token(first));
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
        if (l == 0) s_top[w] = m;
        if (tid == 0) {
            s_low = s_tau = 1;
            s_count = kept;
            s_reach = 0;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kScanThreads / 32; i++) m = fmaxf(m, s_top[i]);
        m = fmaxf(m, top);
        if (m > -INFINITY) {
            // a term e^-d is off by 2^-23 (2 + d) of itself: 1e-6 of the sum if all
            // lie 5 below the maximum, and so 1e-6 of a unit of the score
            float2 terms = make_float2(0.f, 0.f);
            const float2 off = make_float2(-m, -m), base = make_float2(1.44269504f, 1.44269504f);
#pragma unroll
            for (int i = 0; i < PER; i += 2) {
                const float2 d = __fmul2_rn(__fadd2_rn(make_float2(x[i], x[i + 1]), off), base);
                terms = __fadd2_rn(terms, make_float2(exp2_fast(d.x), exp2_fast(d.y)));
            }
            float part_sum = terms.x + terms.y;
            if (part_sum != part_sum) {  // NaN counts as barred; a value of +inf is the maximum
                part_sum = 0.f;
#pragma unroll
                for (int i = 0; i < PER; i++) part_sum += x[i] == m ? 1.f : (x[i] < m ? expf(x[i] - m) : 0.f);
            }
            sum = sum * (top == m ? 1.0 : (double)expf(top - m)) + (double)part_sum;
            top = m;
        }
        const int above = __syncthreads_count(mine > floor_key);
        if (above == 0) continue;  // the tile adds nothing
        if (above > a.n) {
            unsigned long long group = mine;
#pragma unroll
            for (int d = 1; d < 4; d <<= 1) {
                const unsigned long long other = __shfl_xor_sync(kFull, group, d);
                group = other > group ? other : group;
            }
            if ((l & 3) == 0) s_group[tid >> 2] = group;
            __syncthreads();
            int rank = 0;
#pragma unroll
            for (int i = 0; i < kGroups / 4; i++) rank += s_group[4 * i + (l & 3)] > group;
            rank += __shfl_xor_sync(kFull, rank, 1);
            rank += __shfl_xor_sync(kFull, rank, 2);
            if ((l & 3) == 0 && group != 0 && rank == a.n - 1) s_low = group;
            __syncthreads();
            const bool near = mine > floor_key && mine >= s_low;
            if (near) s_near[atomicAdd(&s_reach, 1)] = mine;
            __syncthreads();
            if (near) {
                const int reach = s_reach;
                int before = 0;
                for (int i = 0; i < reach; i++) before += s_near[i] > mine;
                if (before == a.n - 1) s_tau = mine;
            }
        }
        if (tid < kept) s_list[tid] = s_keep[tid];
        __syncthreads();
        const unsigned long long tau = s_tau > floor_key ? s_tau : floor_key + 1;
        if (mine >= tau) {
#pragma unroll
            for (int i = 0; i < PER; i++) {
                const unsigned long long k = key_of(x[i], token(i));
                if (k >= tau) s_list[atomicAdd(&s_count, 1)] = k;
            }
        }
        __syncthreads();
        const int count = s_count;
        for (int i = tid; i < count; i += kScanThreads) {
            const unsigned long long k = s_list[i];
            int better = 0;
            for (int j = 0; j < count; j++) better += s_list[j] > k;
            if (better < a.n) s_keep[better] = k;
        }
        kept = min(count, a.n);
        __syncthreads();
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
    if (l == 0) s_sum[w] = sum;
    __syncthreads();
    if (tid == 0) {
        double all = 0.0;
        for (int i = 0; i < kScanThreads / 32; i++) all += s_sum[i];
        stats[blockIdx.x] = RowStats{all, top, 0};
    }
    if (tid < a.n) best[(long long)blockIdx.x * a.n + tid] = tid < kept ? s_keep[tid] : 0;
}

struct Cand {
    double score;
    int beam, token;
};

__device__ __forceinline__ bool better(const Cand &x, const Cand &y)
{
    // without branches; beams and tokens are not negative
    const unsigned long long at_x = (unsigned long long)(unsigned)x.beam << 32 | (unsigned)x.token, at_y = (unsigned long long)(unsigned)y.beam << 32 | (unsigned)y.token;
    return (x.score > y.score) | ((x.score == y.score) & (at_x < at_y));
}

// One CTA a group: the rows' log-sums in fp64, then the n best of all parts'
// candidates, by the same threshold.  One group of 4 beams 9 us, 64 of 8 beams 8.6
// us: the chain of three rounds to memory and the 64-bit exponentials.
__global__ void __launch_bounds__(kMergeThreads) k_beam_merge(BeamArgs a, int splits, const RowStats *stats,
                                                              const unsigned long long *best)
{
    extern __shared__ Cand s_list[];
    __shared__ Cand s_best[kMergeThreads];
    __shared__ double s_top[kMaxBeams], s_add[kMaxBeams];  // per beam: largest logit; score - log of the sum
    __shared__ Cand s_tau;
    __shared__ int s_count;
    const int tid = threadIdx.x, g = blockIdx.x, B = a.beams, n = a.n;
    const Cand none = {-INFINITY, 0x7fffffff, 0x7fffffff};
    // a warp a beam and turn, a lane a part: one wait for all of a beam's statistics
    for (int b = tid >> 5; b < B; b += kMergeThreads / 32) {
        const RowStats *st = stats + (long long)(g * B + b) * splits;
        float top = -INFINITY;
        for (int i = tid & 31; i < splits; i += 32) top = fmaxf(top, st[i].top);
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
        double sum = 0.0;
        for (int i = tid & 31; i < splits; i += 32)
            if (st[i].top > -INFINITY) sum += st[i].sum * (st[i].top == top ? 1.0 : exp((double)st[i].top - (double)top));
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
        if ((tid & 31) == 0) {
            const float s = a.scores[(long long)g * B + b];
            s_top[b] = top;
            s_add[b] = sum > 0.0 && s > -INFINITY ? (double)s - log(sum) : -INFINITY;
        }
    }
    if (tid == 0) { s_tau = none; s_count = 0; }
    __syncthreads();
    const int per_beam = splits * n, total = B * per_beam;
    const unsigned long long *keys = best + (long long)g * total;
    auto cand = [&](int i) -> Cand {
        const unsigned long long k = keys[i];
        if (k == 0) return none;
        const int b = i / per_beam;
        const double x = value_of(k);
        const double s = s_add[b] + (x == s_top[b] ? 0.0 : x - s_top[b]);
        return s > -INFINITY ? Cand{s, b, token_of(k)} : none;
    };
    Cand mine = none;
    for (int i = tid; i < total; i += kMergeThreads) {
        const Cand c = cand(i);
        if (better(c, mine)) mine = c;
    }
    s_best[tid] = mine;
    __syncthreads();
    int rank = 0;
    const int holders = min(kMergeThreads, total);  // threads that saw a candidate
#pragma unroll 8
    for (int i = 0; i < holders; i++) rank += better(s_best[i], mine);
    if (mine.score > -INFINITY && rank == n - 1) s_tau = mine;
    __syncthreads();
    const Cand tau = s_tau;
    if (mine.score > -INFINITY && !better(tau, mine)) {
        for (int i = tid; i < total; i += kMergeThreads) {
            const Cand c = cand(i);
            if (c.score > -INFINITY && !better(tau, c)) s_list[atomicAdd(&s_count, 1)] = c;
        }
    }
    __syncthreads();
    const int count = s_count;
    const long long o = (long long)g * n;
    for (int i = tid; i < count; i += kMergeThreads) {
        const Cand c = s_list[i];
        int above = 0;
        for (int j = 0; j < count; j++) above += better(s_list[j], c);
        if (above < n) {
            a.scores_out[o + above] = (float)c.score;
            a.parents[o + above] = c.beam;
            a.tokens[o + above] = c.token;
        }
    }
    for (int i = count + tid; i < n; i += kMergeThreads) {
        a.scores_out[o + i] = -INFINITY;
        a.parents[o + i] = -1;
        a.tokens[o + i] = -1;
    }
}

// Parts of a row: as many CTAs as lie on the GPU at once (four an SM), no more
// than the row has tiles, and no more candidates than the merge takes.  A CTA
// ranks most in its first tile, so few long ones beat many short ones: 512 rows
// of 100003 bf16 logits take 87 us in one part each, 96 in three.
struct BeamPlan {
    int per, splits;
};

BeamPlan beam_plan(int groups, int beams, int vocab, int n)
{
    BeamPlan p;
    const long long rows = std::max(1LL, (long long)groups * beams);
    // tiles of 8192 values, or of 2048 where those leave SMs without work: 4 rows of
    // 32001 fp32 logits take 18 us instead of 21, but 64 rows would take 25 instead of
    // 21 and 512 rows of 100003 bf16 logits 106 instead of 87
    p.per = rows * ((vocab + 8191) / 8192) < 148 ? 8 : 32;
    const long long tiles = ((long long)vocab + p.per * kScanThreads - 1) / (p.per * kScanThreads);
    const long long fill = 148 * 4 / rows;
    p.splits = (int)std::max(1LL, std::min({tiles, fill, (long long)kMaxMerge / ((long long)beams * n)}));
    return p;
}

template <class T>
cudaError_t launch_scan(const BeamArgs &a, const BeamPlan &p, RowStats *stats, unsigned long long *best, cudaStream_t s)
{
    const unsigned grid = (unsigned)((long long)a.groups * a.beams * p.splits);
    if (p.per == 8)
        k_beam_scan<T, 8><<<grid, kScanThreads, 0, s>>>(a, p.splits, stats, best);
    else
        k_beam_scan<T, 32><<<grid, kScanThreads, 0, s>>>(a, p.splits, stats, best);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Reordering in place.  A CTA takes the same few hundred bytes of every row of
// a group, holds those that some other row asks for in shared memory, and
// writes them back under their new owners: no second buffer, each moved byte
// read and written once.  512 packed states of 442 KB, seven of eight moved: 42
// us; rows that several take are read once, so that 44 MB are read and 132 written.
// ---------------------------------------------------------------------------
constexpr int kReorderBytes = 32768;
constexpr int kRun = 256;  // vectors of 16 bytes that a warp has under way

__global__ void __launch_bounds__(256) k_reorder(uint8_t *base, long long row_bytes, int beams, int tiles, int tile_vecs,
                                                 const int *parents)
{
    __shared__ __align__(16) uint4 buf[kReorderBytes / 16];
    __shared__ int s_parent[kMaxBeams], s_used[kMaxBeams], s_moves;
    const int tid = threadIdx.x;
    const int g = blockIdx.x / tiles, tile = blockIdx.x - g * tiles;
    if (tid < beams) {
        const int p = parents[(long long)g * beams + tid];
        s_parent[tid] = (p >= 0 && p < beams) ? p : tid;
        s_used[tid] = 0;
    }
    if (tid == 0) s_moves = 0;
    __syncthreads();
    if (tid < beams && s_parent[tid] != tid) {
        s_used[s_parent[tid]] = 1;
        s_moves = 1;
    }
    __syncthreads();
    if (!s_moves) return;
    const long long v0 = (long long)tile * tile_vecs, vecs = row_bytes / 16;
    const int nv = (int)min((long long)tile_vecs, vecs - v0);
    uint4 *rows = reinterpret_cast<uint4 *>(base) + (long long)g * beams * vecs + v0;
    // a warp a row and kRun of its vectors
    const int w = tid >> 5, l = tid & 31, runs = (nv + kRun - 1) / kRun;
    for (int x = w; x < beams * runs; x += 8) {
        const int b = x / runs, at = (x - b * runs) * kRun + l;
        if (!s_used[b]) continue;
#pragma unroll
        for (int v = at; v < at + kRun; v += 32)
            if (v < nv) buf[b * tile_vecs + v] = rows[(long long)b * vecs + v];
    }
    __syncthreads();
    for (int x = w; x < beams * runs; x += 8) {
        const int b = x / runs, at = (x - b * runs) * kRun + l;
        if (s_parent[b] == b) continue;
#pragma unroll
        for (int v = at; v < at + kRun; v += 32)
            if (v < nv) rows[(long long)b * vecs + v] = buf[s_parent[b] * tile_vecs + v];
    }
}

}  // namespace

size_t beam_scratch_bytes(int groups, int beams, int vocab, int n)
{
    const BeamPlan p = beam_plan(groups, beams, vocab, n);
    const size_t parts = (size_t)groups * beams * p.splits;
    return parts * (sizeof(RowStats) + 8 * (size_t)n);
}

cudaError_t launch_beam_select(const BeamArgs &a, cudaStream_t s)
{
    const BeamPlan p = beam_plan(a.groups, a.beams, a.vocab, a.n);
    RowStats *stats = reinterpret_cast<RowStats *>(a.scratch);
    unsigned long long *best = reinterpret_cast<unsigned long long *>(stats + (size_t)a.groups * a.beams * p.splits);
    cudaError_t e;
    switch (a.dtype) {
        case kF32: e = launch_scan<float>(a, p, stats, best, s); break;
        case kF16: e = launch_scan<__half>(a, p, stats, best, s); break;
        default: e = launch_scan<__nv_bfloat16>(a, p, stats, best, s); break;
    }
    if (e != cudaSuccess) return e;
    // at most n threads hold candidates above the threshold
    const size_t per_thread = ((size_t)a.beams * p.splits * a.n + kMergeThreads - 1) / kMergeThreads;
    const size_t dyn = per_thread * (size_t)a.n * sizeof(Cand);
    static_assert(kMergeList * sizeof(Cand) <= 96 * 1024, "the merge's list has to fit in shared memory");
    if (dyn > 32 * 1024) {
        e = cudaFuncSetAttribute(k_beam_merge, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kMergeList * sizeof(Cand)));
        if (e != cudaSuccess) return e;
    }
    k_beam_merge<<<a.groups, kMergeThreads, dyn, s>>>(a, p.splits, stats, best);
    return cudaGetLastError();
}

cudaError_t launch_reorder(uint8_t *base, size_t row_bytes, int groups, int beams, const int *parents, cudaStream_t s)
{
    const long long vecs = (long long)(row_bytes / 16);
    const int tile_vecs = (int)std::min(vecs, (long long)(kReorderBytes / 16 / beams));
    const long long tiles = (vecs + tile_vecs - 1) / tile_vecs;
    k_reorder<<<(unsigned)(tiles * groups), 256, 0, s>>>(base, (long long)row_bytes, beams, (int)tiles, tile_vecs, parents);
    return cudaGetLastError();
}

}  // namespace stepq
