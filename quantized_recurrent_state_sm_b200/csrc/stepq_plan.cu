// The plan of a ragged batch: block table and slot map from request lengths.
//
// One launch.  Every CTA scans all lengths for itself (at most 65536 of them,
// from L2) instead of waiting for a scan kernel: the plan is latency-bound, and
// a second launch would cost more than the repeated scan.  The first CTA
// resolves the slots; the others each write 2048 entries of the token map or of
// the block table, which is a search for the request that covers an entry: the
// requests that begin in the CTA's range mark their first entry, and a running
// maximum over the marks finds the last request at or before each entry.
#include "stepq_serve.cuh"

namespace stepq {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanRange = 2048;  // entries of a CTA
constexpr int kPer = kPlanRange / kPlanThreads;
constexpr unsigned kFull = 0xffffffffu;
constexpr unsigned kSat = 1u << 30;  // sums stop here (the largest token count is 2^28)

// Sums of non-negative lengths that stay below 2^31: associative, so a scan may
// group them in any way.
__device__ __forceinline__ unsigned sat_add(unsigned a, unsigned b) { return min(a + b, kSat); }

// Length of request r as the token rows see it: at least 0, and small enough to add.
__device__ __forceinline__ unsigned length_of(const PlanArgs &a, int r)
{
    const int n = a.lengths[r];
    return n <= 0 ? 0u : min((unsigned)n, kSat);
}

__device__ __forceinline__ unsigned blocks_of(unsigned len) { return (len + kBlockTokens - 1) / kBlockTokens; }

struct Pair {
    unsigned tokens, blocks;
};

__device__ __forceinline__ Pair add(Pair x, Pair y) { return {sat_add(x.tokens, y.tokens), x.blocks + y.blocks}; }

// Exclusive sum over the CTA's threads; *total gets the sum of all.
__device__ Pair block_scan(Pair v, Pair *sm, Pair *total)
{
    const int tid = threadIdx.x, w = tid >> 5, l = tid & 31;
    Pair inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        Pair o = {__shfl_up_sync(kFull, inc.tokens, d), __shfl_up_sync(kFull, inc.blocks, d)};
        if (l >= d) inc = add(o, inc);
    }
    if (l == 31) sm[w] = inc;
    Pair ex = {__shfl_up_sync(kFull, inc.tokens, 1), __shfl_up_sync(kFull, inc.blocks, 1)};
    if (l == 0) ex = {0, 0};
    __syncthreads();
    Pair base = {0, 0}, all = {0, 0};
    for (int i = 0; i < kPlanThreads / 32; i++) {
        if (i == w) base = all;
        all = add(all, sm[i]);
    }
    __syncthreads();
    *total = all;
    return add(base, ex);
}

// Running maximum over the CTA's entries (kPer consecutive ones a thread).
__device__ void scan_max(int *v, int *sm)
{
    const int tid = threadIdx.x, w = tid >> 5, l = tid & 31;
#pragma unroll
    for (int i = 1; i < kPer; i++) v[i] = max(v[i], v[i - 1]);
    int inc = v[kPer - 1];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kFull, inc, d);
        if (l >= d) inc = max(inc, o);
    }
    if (l == 31) sm[w] = inc;
    int before = __shfl_up_sync(kFull, inc, 1);
    if (l == 0) before = -1;
    __syncthreads();
    for (int i = 0; i < w; i++) before = max(before, sm[i]);
#pragma unroll
    for (int i = 0; i < kPer; i++) v[i] = max(v[i], before);
}

// Slots, live flags and starts of all requests, and the plan's head.
__device__ void resolve(const PlanArgs &a, int r0, int r1, Pair at, Pair *sm, int *flags)
{
    const PlanView &p = a.p;
    const int tid = threadIdx.x;
    __shared__ unsigned rows_used, blocks_used;
    if (tid == 0) { *flags = 0; rows_used = 0; blocks_used = 0; }
    __syncthreads();
    // A request whose tokens pass the capacity ends the batch: it and all after
    // it have no tokens.
    unsigned need = 0, rows = 0, blocks = 0;
    int bad = 0;
    for (int r = r0; r < r1; r++) {
        const unsigned len = length_of(a, r);
        if (a.lengths[r] < 0) bad |= kPlanBadLength;
        const Pair end = add(at, {len, blocks_of(len)});
        const bool fits = end.tokens <= (unsigned)p.tokens;
        if (fits) {
            if (r == 0) p.starts[0] = p.block_starts[0] = 0;
            p.starts[r + 1] = (int)end.tokens;
            p.block_starts[r + 1] = (int)end.blocks;
            rows = end.tokens;
            blocks = end.blocks;
        } else {
            if (r == 0) p.starts[0] = p.block_starts[0] = 0;
            p.starts[r + 1] = -1;  // set to the last end below
            bad |= kPlanTooMany;
        }
        const bool tokens = fits && len > 0;
        const int ctx = a.contexts ? a.contexts[r] : 0;
        int s = a.slots ? a.slots[r] : r;
        bool take = tokens;
        if (tokens && a.lengths[r] > a.max_length) { bad |= kPlanBadLength; take = false; }
        if (s < 0 || s >= p.slots) {
            if (take && s == -1 && ctx == 0 && a.busy) {
                need++;
                s = -2;  // gets a free slot below
            } else {
                if (take) bad |= kPlanBadSlot;
                take = false;
                s = -1;
            }
        }
        p.slot[r] = s;
        p.live[r] = take ? s : -1;
        p.fresh[r] = ctx == 0;
        if (take && s >= 0 && a.slots) p.owner[s] = 0x7fffffff;
        at = end;
    }
    for (int r = a.n + tid; r < p.requests; r += kPlanThreads) {
        p.slot[r] = -1;
        p.live[r] = -1;
        p.fresh[r] = 0;
        p.starts[r + 1] = -1;
    }
    if (a.n == 0 && tid == 0) p.starts[0] = p.block_starts[0] = 0;
    if (rows) atomicMax(&rows_used, rows);
    if (blocks) atomicMax(&blocks_used, blocks);
    if (bad) atomicOr(flags, bad);
    Pair all;
    Pair rank = block_scan({need, 0}, sm, &all);  // orders the writes above, too
    for (int r = tid; r < p.requests; r += kPlanThreads)
        if (p.starts[r + 1] < 0) {
            p.starts[r + 1] = (int)rows_used;
            p.block_starts[r + 1] = (int)blocks_used;
        }
    if (a.slots) {
        // a slot named twice belongs to the first request with tokens
        for (int r = r0; r < r1; r++)
            if (p.live[r] >= 0) atomicMin(&p.owner[p.live[r]], r);
        __syncthreads();
        for (int r = r0; r < r1; r++) {
            const int s = p.live[r];
            if (s < 0) continue;
            if (atomicAdd(&p.owner[s], 0) != r) {
                p.live[r] = -1;
                atomicOr(flags, kPlanSlotTwice);
            } else if (a.busy) {
                a.busy[s] = 1;
            }
        }
        __syncthreads();
        if (all.tokens > 0) {
            // the lowest free slots, in order, as far as they are needed
            unsigned found = 0;
            for (int s0 = 0; s0 < p.slots && found < all.tokens; s0 += 16 * kPlanThreads) {
                const int b0 = s0 + 16 * tid;
                unsigned free = 0;
                for (int i = 0; i < 16; i++)
                    if (b0 + i < p.slots && a.busy[b0 + i] == 0) free |= 1u << i;
                Pair sum;
                unsigned k = found + block_scan({(unsigned)__popc(free), 0}, sm, &sum).tokens;
                for (; free && k < all.tokens; free &= free - 1) p.list[k++] = b0 + __ffs(free) - 1;
                found += sum.tokens;
            }
            __syncthreads();
            unsigned k = rank.tokens;
            for (int r = r0; r < r1; r++) {
                if (p.slot[r] != -2) continue;
                if (k < found) {
                    const int s = p.list[k];
                    p.slot[r] = s;
                    p.live[r] = s;
                    a.busy[s] = 1;
                } else {
                    p.slot[r] = -1;
                    p.live[r] = -1;
                    atomicOr(flags, kPlanNoSlot);
                }
                k++;
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        p.head[0] = *flags;
        p.head[1] = a.n;
        p.head[2] = (int)rows_used;
        p.head[3] = (int)blocks_used;
    }
}

__global__ void __launch_bounds__(kPlanThreads) k_plan(PlanArgs a, int token_ctas)
{
    __shared__ Pair sm[kPlanThreads / 32];
    __shared__ int smi[kPlanThreads / 32];
    __shared__ int mark[kPlanRange], from[kPlanRange];
    __shared__ int flags;
    const PlanView &p = a.p;
    const int tid = threadIdx.x;
    const int per = (a.n + kPlanThreads - 1) / kPlanThreads;
    const int r0 = min(a.n, tid * per), r1 = min(a.n, r0 + per);
    Pair mine = {0, 0}, all;
    for (int r = r0; r < r1; r++) {
        const unsigned len = length_of(a, r);
        mine = add(mine, {len, blocks_of(len)});
    }
    Pair at = block_scan(mine, sm, &all);
    if (blockIdx.x == 0) {
        resolve(a, r0, r1, at, sm, &flags);
        return;
    }
    const int c = blockIdx.x - 1;
    const bool tokens = c < token_ctas;
    const unsigned x0 = (unsigned)(tokens ? c : c - token_ctas) * kPlanRange;
    const unsigned x1 = min(x0 + kPlanRange, (unsigned)(tokens ? p.tokens : p.blocks));
    for (int i = tid; i < kPlanRange; i += kPlanThreads) mark[i] = -1;
    __syncthreads();
    // mark[x] = request whose entries begin at x0 + x (or before, for x = 0);
    // from[x] = where they begin
    for (int r = r0; r < r1; r++) {
        const unsigned len = length_of(a, r);
        const Pair end = add(at, {len, blocks_of(len)});
        if (end.tokens > (unsigned)p.tokens) break;  // this request and all after it have no tokens
        const unsigned lo = tokens ? at.tokens : at.blocks, hi = tokens ? end.tokens : end.blocks;
        if (lo < hi && lo < x1 && hi > x0) {
            const int x = lo > x0 ? (int)(lo - x0) : 0;
            mark[x] = r;
            from[x] = (int)lo;
        }
        at = end;
    }
    __syncthreads();
    int last[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i++) last[i] = mark[kPer * tid + i] >= 0 ? kPer * tid + i : -1;
    scan_max(last, smi);
    // the rows used: beyond them the last request's mark does not count
    __shared__ unsigned end_of_batch;
    if (tid == 0) end_of_batch = 0;
    __syncthreads();
    // at: the end of this thread's last request, or of the last that fits
    if (at.tokens <= (unsigned)p.tokens) atomicMax(&end_of_batch, tokens ? at.tokens : at.blocks);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        const unsigned x = x0 + kPer * tid + i;
        if (x >= x1) continue;
        int r = -1, v = -1;
        if (last[i] >= 0 && x < end_of_batch) {
            r = mark[last[i]];
            v = (int)x - from[last[i]];
            v = tokens ? v + (a.contexts ? a.contexts[r] : 0) : v * kBlockTokens;
        }
        (tokens ? p.token_request : p.block_request)[x] = r;
        (tokens ? p.token_position : p.block_first)[x] = v;
    }
}

}  // namespace

cudaError_t launch_plan(const PlanArgs &a, cudaStream_t s)
{
    const int tc = (a.p.tokens + kPlanRange - 1) / kPlanRange, bc = (a.p.blocks + kPlanRange - 1) / kPlanRange;
    k_plan<<<1 + tc + bc, kPlanThreads, 0, s>>>(a, tc);
    return cudaGetLastError();
}

}  // namespace stepq
