// The plan of a ragged batch: block table and slot map from request lengths.
//
// One launch.  Every CTA scans all lengths for itself (at most 65536 of them,
// from L2) instead of waiting for a scan kernel: the plan is latency-bound, and
// a second launch would cost more than the repeated scan.  The first CTA
// resolves the slots; the others each write 4096 entries of the token map or of
// the block table, which is a search for the request that covers an entry: the
// requests that begin in the CTA's range mark their first entry, and a running
// maximum over the marks finds the last request at or before each entry.
// Measured: 8 requests 7.5 us (a launch and three rounds to L2), 8192 requests of
// 454 thousand tokens, half of them taking free slots, 28 us (4 MB written).
#include "stepq_serve.cuh"

namespace stepq {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanRange = 4096;  // entries of a CTA, and requests of a turn
constexpr int kPer = kPlanRange / kPlanThreads;
constexpr unsigned kFull = 0xffffffffu;
constexpr unsigned kSat = 1u << 30;  // sums stop here (the largest token count is 2^28)

// Sums of non-negative lengths that stay below 2^31: associative, so a scan may
// group them in any way.
__device__ __forceinline__ unsigned sat_add(unsigned a, unsigned b) { return min(a + b, kSat); }

// A length as the token rows see it: at least 0, and small enough to add.
__device__ __forceinline__ unsigned length_of(int n) { return n <= 0 ? 0u : min((unsigned)n, kSat); }

__device__ __forceinline__ unsigned blocks_of(unsigned len) { return (len + kBlockTokens - 1) / kBlockTokens; }

struct Sums {
    unsigned tokens, blocks, fresh;  // fresh: requests that ask for a slot
};

__device__ __forceinline__ Sums add(Sums x, Sums y) { return {sat_add(x.tokens, y.tokens), x.blocks + y.blocks, x.fresh + y.fresh}; }

struct Shared {
    Sums sums[kPlanThreads / 32];
    int maxima[kPlanThreads / 32];
    int mark[kPlanRange], from[kPlanRange];
    int flags;
    unsigned rows, blocks;
};

// Exclusive sum over the CTA's threads; *total gets the sum of all.
__device__ Sums block_scan(Sums v, Shared &sm, Sums *total)
{
    const int tid = threadIdx.x, w = tid >> 5, l = tid & 31;
    Sums inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Sums o = {__shfl_up_sync(kFull, inc.tokens, d), __shfl_up_sync(kFull, inc.blocks, d), __shfl_up_sync(kFull, inc.fresh, d)};
        if (l >= d) inc = add(o, inc);
    }
    if (l == 31) sm.sums[w] = inc;
    Sums ex = {__shfl_up_sync(kFull, inc.tokens, 1), __shfl_up_sync(kFull, inc.blocks, 1), __shfl_up_sync(kFull, inc.fresh, 1)};
    if (l == 0) ex = {0, 0, 0};
    __syncthreads();
    Sums base = {0, 0, 0}, all = base;
#pragma unroll
    for (int i = 0; i < kPlanThreads / 32; i++) {
        if (i == w) base = all;
        all = add(all, sm.sums[i]);
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

// Four consecutive entries from r on (a multiple of 4) of n: as one vector where
// that is aligned.  0 past the end; nothing is written there.
__device__ __forceinline__ void four(const int *p, int r, int n, int *x)
{
    if (r + kPer <= n && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        const int4 v = *reinterpret_cast<const int4 *>(p + r);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
#pragma unroll
        for (int i = 0; i < kPer; i++) x[i] = r + i < n ? p[r + i] : 0;
    }
}
__device__ __forceinline__ void put_four(int *p, int r, int n, const int *x)  // p aligned: an array of the plan
{
    if (r + kPer <= n) {
        *reinterpret_cast<int4 *>(p + r) = make_int4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; i++)
            if (r + i < n) p[r + i] = x[i];
    }
}

// Which of 16 bytes from `at` on are zero, as bits.
__device__ __forceinline__ unsigned zero_bytes(const uint8_t *p, int at, int n)
{
    unsigned z = 0;
    if (at + 16 <= n && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p + at);
        const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 16; i++) z |= (unsigned)(((w[i >> 2] >> (8 * (i & 3))) & 255) == 0) << i;
    } else {
        for (int i = 0; i < 16; i++)
            if (at + i < n && p[at + i] == 0) z |= 1u << i;
    }
    return z;
}

// Slots, live flags and starts of all requests, and the plan's head.
__device__ void resolve(const PlanArgs &a, Shared &sm)
{
    const PlanView &p = a.p;
    const int tid = threadIdx.x;
    if (tid == 0) {
        sm.flags = 0;
        sm.rows = sm.blocks = 0;
    }
    __syncthreads();
    Sums carry = {0, 0, 0};
    for (int r0 = 0; r0 < a.n; r0 += kPlanRange) {
        const int r = r0 + kPer * tid;
        int n[kPer], ctx[kPer] = {}, slot[kPer], ask[kPer];
        unsigned len[kPer];
        four(a.lengths, r, a.n, n);
        if (a.contexts) four(a.contexts, r, a.n, ctx);
        if (a.slots) four(a.slots, r, a.n, slot);
        Sums mine = {0, 0, 0};
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            if (!a.slots) slot[i] = r + i;
            len[i] = length_of(n[i]);
            // a new request that asks for a free slot (whether its tokens fit is not known yet:
            // the requests that do not fit are the last, so they take nobody's rank)
            ask[i] = len[i] > 0 && n[i] <= a.max_length && slot[i] == -1 && ctx[i] == 0 && a.busy != nullptr;
            mine = add(mine, {len[i], blocks_of(len[i]), (unsigned)ask[i]});
        }
        Sums all, at = add(carry, block_scan(mine, sm, &all));
        carry = add(carry, all);
        unsigned rows = 0, blocks = 0;
        int bad = 0, start[kPer], bstart[kPer], live[kPer], fresh[kPer];
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            // a request whose tokens pass the capacity ends the batch: it and all after it have none
            start[i] = at.tokens <= (unsigned)p.tokens ? (int)at.tokens : -1;  // -1: set to the last end below
            bstart[i] = (int)at.blocks;
            const unsigned rank = at.fresh;
            at = add(at, {len[i], blocks_of(len[i]), (unsigned)ask[i]});
            live[i] = fresh[i] = 0;
            if (r + i >= a.n) continue;
            const bool fits = at.tokens <= (unsigned)p.tokens;
            if (fits) {
                rows = at.tokens;
                blocks = at.blocks;
            } else {
                bad |= kPlanTooMany;
            }
            if (n[i] < 0) bad |= kPlanBadLength;
            bool take = fits && len[i] > 0;
            if (take && n[i] > a.max_length) {
                bad |= kPlanBadLength;
                take = false;
            }
            int s = slot[i];
            if (s < 0 || s >= p.slots) {
                if (take && ask[i]) {
                    s = -2 - (int)rank;  // gets the free slot of this rank below
                } else {
                    if (take) bad |= kPlanBadSlot;
                    take = false;
                    s = -1;
                }
            }
            slot[i] = s;
            live[i] = take && s >= 0 ? s : -1;
            fresh[i] = ctx[i] == 0;
            if (take && s >= 0 && a.slots) p.owner[s] = 0x7fffffff;
        }
        put_four(p.starts, r, a.n, start);
        put_four(p.block_starts, r, a.n, bstart);
        put_four(p.slot, r, a.n, slot);
        put_four(p.live, r, a.n, live);
        put_four(p.fresh, r, a.n, fresh);
        if (rows) atomicMax(&sm.rows, rows);
        if (blocks) atomicMax(&sm.blocks, blocks);
        if (bad) atomicOr(&sm.flags, bad);
    }
    __syncthreads();
    const int rows = (int)sm.rows, blocks = (int)sm.blocks;
    if (sm.flags & kPlanTooMany)
        for (int r = tid; r < a.n; r += kPlanThreads)
            if (p.starts[r] < 0) {
                p.starts[r] = rows;
                p.block_starts[r] = blocks;
            }
    for (int r = a.n + tid; r <= p.requests; r += kPlanThreads) {
        p.starts[r] = rows;
        p.block_starts[r] = blocks;
        if (r == p.requests) break;
        p.slot[r] = -1;
        p.live[r] = -1;
        p.fresh[r] = 0;
    }
    if (a.slots) {
        // a slot named twice belongs to the first request with tokens
        for (int r0 = tid; r0 < a.n; r0 += 4 * kPlanThreads) {
            int s[4];
#pragma unroll
            for (int i = 0; i < 4; i++) s[i] = r0 + i * kPlanThreads < a.n ? p.live[r0 + i * kPlanThreads] : -1;
#pragma unroll
            for (int i = 0; i < 4; i++)
                if (s[i] >= 0) atomicMin(&p.owner[s[i]], r0 + i * kPlanThreads);
        }
        __syncthreads();
        for (int r0 = tid; r0 < a.n; r0 += 4 * kPlanThreads) {
            int s[4], o[4];
#pragma unroll
            for (int i = 0; i < 4; i++) s[i] = r0 + i * kPlanThreads < a.n ? p.live[r0 + i * kPlanThreads] : -1;
#pragma unroll
            for (int i = 0; i < 4; i++) o[i] = s[i] >= 0 ? __ldcg(&p.owner[s[i]]) : 0;  // atomics work in L2
#pragma unroll
            for (int i = 0; i < 4; i++) {
                if (s[i] < 0) continue;
                if (o[i] != r0 + i * kPlanThreads) {
                    p.live[r0 + i * kPlanThreads] = -1;
                    atomicOr(&sm.flags, kPlanSlotTwice);
                } else if (a.busy) {
                    a.busy[s[i]] = 1;
                }
            }
        }
        __syncthreads();
        if (carry.fresh > 0) {
            // the lowest free slots, in order, as far as they are needed
            unsigned found = 0;
            for (int s0 = 0; s0 < p.slots && found < carry.fresh; s0 += 16 * kPlanThreads) {
                const int b0 = s0 + 16 * tid;
                unsigned free = b0 < p.slots ? zero_bytes(a.busy, b0, p.slots) : 0;
                Sums sum;
                unsigned k = found + block_scan({0, 0, (unsigned)__popc(free)}, sm, &sum).fresh;
                for (; free && k < carry.fresh; free &= free - 1) p.list[k++] = b0 + __ffs(free) - 1;
                found += sum.fresh;
            }
            __syncthreads();
            for (int r0 = tid; r0 < a.n; r0 += 4 * kPlanThreads) {
                int s[4], got[4];
#pragma unroll
                for (int i = 0; i < 4; i++) s[i] = r0 + i * kPlanThreads < a.n ? p.slot[r0 + i * kPlanThreads] : -1;
#pragma unroll
                for (int i = 0; i < 4; i++) got[i] = s[i] <= -2 && (unsigned)(-2 - s[i]) < found ? p.list[-2 - s[i]] : -1;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    if (s[i] > -2) continue;
                    if (got[i] >= 0)
                        a.busy[got[i]] = 1;
                    else
                        atomicOr(&sm.flags, kPlanNoSlot);
                    p.slot[r0 + i * kPlanThreads] = got[i];
                    p.live[r0 + i * kPlanThreads] = got[i];
                }
            }
        }
        __syncthreads();
    }
    if (tid == 0) {
        p.head[0] = sm.flags;
        p.head[1] = a.n;
        p.head[2] = rows;
        p.head[3] = blocks;
    }
}

__global__ void __launch_bounds__(kPlanThreads) k_plan(PlanArgs a, int token_ctas)
{
    __shared__ Shared sm;
    const PlanView &p = a.p;
    const int tid = threadIdx.x;
    if (blockIdx.x == 0) {
        resolve(a, sm);
        return;
    }
    const int c = blockIdx.x - 1;
    const bool tokens = c < token_ctas;
    const unsigned x0 = (unsigned)(tokens ? c : c - token_ctas) * kPlanRange;
    const unsigned x1 = min(x0 + kPlanRange, (unsigned)(tokens ? p.tokens : p.blocks));
    for (int i = tid; i < kPlanRange; i += kPlanThreads) sm.mark[i] = -1;
    if (tid == 0) sm.rows = 0;
    __syncthreads();
    // mark[x]: the request whose entries begin at x0 + x (or before, for x = 0);
    // from[x]: where they begin
    Sums carry = {0, 0, 0};
    for (int r0 = 0; r0 < a.n; r0 += kPlanRange) {
        const int r = r0 + kPer * tid;
        int n[kPer];
        four(a.lengths, r, a.n, n);
        Sums mine = {0, 0, 0};
#pragma unroll
        for (int i = 0; i < kPer; i++) mine = add(mine, {length_of(n[i]), blocks_of(length_of(n[i])), 0});
        Sums all, at = add(carry, block_scan(mine, sm, &all));
        carry = add(carry, all);
        unsigned end = 0;
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            const unsigned len = length_of(n[i]), lo = tokens ? at.tokens : at.blocks;
            at = add(at, {len, blocks_of(len), 0});
            if (at.tokens > (unsigned)p.tokens) break;  // this request and all after it have no tokens
            const unsigned hi = tokens ? at.tokens : at.blocks;
            end = hi;
            if (lo < hi && lo < x1 && hi > x0) {
                const int x = lo > x0 ? (int)(lo - x0) : 0;
                sm.mark[x] = r + i;
                sm.from[x] = (int)lo;
            }
        }
        if (end > x0) atomicMax(&sm.rows, end);  // how far the batch reaches
        if ((tokens ? carry.tokens : carry.blocks) >= x1 || carry.tokens > (unsigned)p.tokens) break;
    }
    __syncthreads();
    int last[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i++) last[i] = sm.mark[kPer * tid + i] >= 0 ? kPer * tid + i : -1;
    scan_max(last, sm.maxima);
    const unsigned reach = sm.rows;
    int r_of[kPer], v_of[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        const unsigned x = x0 + kPer * tid + i;
        r_of[i] = v_of[i] = -1;
        if (last[i] >= 0 && x < reach) {
            const int r = sm.mark[last[i]], v = (int)x - sm.from[last[i]];
            r_of[i] = r;
            v_of[i] = tokens ? v + (a.contexts ? a.contexts[r] : 0) : v * kBlockTokens;
        }
    }
    int *of = tokens ? p.token_request : p.block_request, *first = tokens ? p.token_position : p.block_first;
    const unsigned x = x0 + kPer * tid;
    static_assert(kPer == 4, "an entry group is one 16-byte vector");
    if (x + kPer <= x1) {
        *reinterpret_cast<int4 *>(of + x) = make_int4(r_of[0], r_of[1], r_of[2], r_of[3]);
        *reinterpret_cast<int4 *>(first + x) = make_int4(v_of[0], v_of[1], v_of[2], v_of[3]);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; i++)
            if (x + i < x1) {
                of[x + i] = r_of[i];
                first[x + i] = v_of[i];
            }
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
