// Host side of the serving entry points of include/stepq.h: plans, prompts,
// packing by request, beam selection and reordering.  Argument validation and
// launches; no device allocation.
#include <climits>

#include "stepq_host.cuh"
#include "stepq_serve.cuh"

using namespace stepq::host;
using stepq::kDK;
using stepq::kDV;

static_assert(STEPQ_BLOCK == stepq::kBlockTokens, "block size");
static_assert(STEPQ_F32 == stepq::kF32 && STEPQ_F16 == stepq::kF16 && STEPQ_BF16 == stepq::kBF16, "element types");
static_assert(STEPQ_GDN == stepq::kGdn && STEPQ_KDA == stepq::kKda && STEPQ_LINEAR == stepq::kLinear, "variants");
static_assert(STEPQ_PLAN_BAD_LENGTH == stepq::kPlanBadLength && STEPQ_PLAN_TOO_MANY == stepq::kPlanTooMany &&
                  STEPQ_PLAN_BAD_SLOT == stepq::kPlanBadSlot && STEPQ_PLAN_SLOT_TWICE == stepq::kPlanSlotTwice &&
                  STEPQ_PLAN_NO_SLOT == stepq::kPlanNoSlot && STEPQ_PLAN_TIMEOUT == stepq::kPlanTimeout,
              "status bits");

namespace {

size_t up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// A device tensor of this call: non-null, aligned, and memory of the current
// device (one query a tensor; these calls are short).
stepq_status check_here(const void *ptr, const char *name, size_t align)
{
    if (!ptr) return fail(STEPQ_ERR_INVALID_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(ptr) % align) return fail(STEPQ_ERR_INVALID_ARG, "%s is not %zu-byte aligned", name, align);
    cudaPointerAttributes at{};
    int dev = 0;
    cudaError_t e = cudaPointerGetAttributes(&at, ptr);
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(STEPQ_ERR_INVALID_ARG, "%s: cannot query pointer (%s)", name, cudaGetErrorString(e));
    }
    if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged)
        return fail(STEPQ_ERR_INVALID_ARG, "%s is not device memory", name);
    if (at.type == cudaMemoryTypeDevice && at.device != dev)
        return fail(STEPQ_ERR_INVALID_ARG, "%s is on device %d, the current device is %d", name, at.device, dev);
    return STEPQ_OK;
}

stepq_status plan_regions(const stepq_plan_desc *d, stepq_plan_regions *r)
{
    if (!d) return fail(STEPQ_ERR_INVALID_ARG, "plan descriptor is NULL");
    if (d->requests < 0 || d->requests > STEPQ_MAX_REQUESTS)
        return fail(STEPQ_ERR_INVALID_ARG, "requests %d outside 0..%d", d->requests, STEPQ_MAX_REQUESTS);
    if (d->tokens < 0 || d->tokens > STEPQ_MAX_TOKENS)
        return fail(STEPQ_ERR_INVALID_ARG, "tokens %d outside 0..%d", d->tokens, STEPQ_MAX_TOKENS);
    if (d->slots < 0 || d->slots > STEPQ_MAX_SLOTS)
        return fail(STEPQ_ERR_INVALID_ARG, "slots %d outside 0..%d", d->slots, STEPQ_MAX_SLOTS);
    const size_t R = d->requests, T = d->tokens;
    r->blocks = d->tokens / STEPQ_BLOCK + d->requests;
    size_t o = 0;
    r->head = o;           o = up(o + 16, 16);
    r->starts = o;         o = up(o + 4 * (R + 1), 16);
    r->slot = o;           o = up(o + 4 * R, 16);
    r->live = o;           o = up(o + 4 * R, 16);
    r->fresh = o;          o = up(o + 4 * R, 16);
    r->token_request = o;  o = up(o + 4 * T, 16);
    r->token_position = o; o = up(o + 4 * T, 16);
    r->block_starts = o;   o = up(o + 4 * (R + 1), 16);
    r->block_request = o;  o = up(o + 4 * (size_t)r->blocks, 16);
    r->block_first = o;    o = up(o + 4 * (size_t)r->blocks, 16);
    r->scratch = o;        o = up(o + 4 * ((size_t)d->slots + R), 16);
    r->total = o;
    return STEPQ_OK;
}

// The plan buffer of a call: regions, size, pointer.
stepq_status plan_view(const stepq_plan_desc *d, const void *plan, size_t bytes, stepq::PlanView *v)
{
    stepq_plan_regions r;
    stepq_status st = plan_regions(d, &r);
    if (st != STEPQ_OK) return st;
    if (bytes < r.total) return fail(STEPQ_ERR_INVALID_ARG, "plan of %zu bytes < %zu required", bytes, r.total);
    if ((st = check_here(plan, "plan", 16)) != STEPQ_OK) return st;
    char *p = const_cast<char *>(static_cast<const char *>(plan));
    auto at = [&](size_t o) { return reinterpret_cast<int *>(p + o); };
    v->requests = d->requests;
    v->tokens = d->tokens;
    v->slots = d->slots;
    v->blocks = r.blocks;
    v->head = at(r.head);
    v->starts = at(r.starts);
    v->slot = at(r.slot);
    v->live = at(r.live);
    v->fresh = at(r.fresh);
    v->token_request = at(r.token_request);
    v->token_position = at(r.token_position);
    v->block_starts = at(r.block_starts);
    v->block_request = at(r.block_request);
    v->block_first = at(r.block_first);
    v->owner = at(r.scratch);
    v->list = at(r.scratch) + d->slots;
    return STEPQ_OK;
}

size_t item_size(int dtype) { return dtype == STEPQ_F32 ? 4 : 2; }

stepq_status check_prompt_desc(const stepq_plan_desc *pd, const stepq_prompt_desc *d)
{
    stepq_plan_regions r;
    stepq_status st = plan_regions(pd, &r);
    if (st != STEPQ_OK) return st;
    if (!d) return fail(STEPQ_ERR_INVALID_ARG, "prompt descriptor is NULL");
    if (d->variant != STEPQ_GDN && d->variant != STEPQ_KDA && d->variant != STEPQ_LINEAR)
        return fail(STEPQ_ERR_INVALID_ARG, "variant %d is none of STEPQ_GDN, STEPQ_KDA, STEPQ_LINEAR", d->variant);
    if (d->dtype != STEPQ_F32 && d->dtype != STEPQ_F16 && d->dtype != STEPQ_BF16)
        return fail(STEPQ_ERR_INVALID_ARG, "dtype %d is none of STEPQ_F32, STEPQ_F16, STEPQ_BF16", d->dtype);
    if (d->heads < 1) return fail(STEPQ_ERR_INVALID_ARG, "heads %d < 1", d->heads);
    if (d->heads > 65535) return fail(STEPQ_ERR_UNSUPPORTED, "heads %d > 65535", d->heads);
    if (d->heads_qk < 1 || d->heads % d->heads_qk != 0)
        return fail(STEPQ_ERR_INVALID_ARG, "heads_qk %d does not divide heads %d", d->heads_qk, d->heads);
    if (d->dk < 1 || d->dv < 1) return fail(STEPQ_ERR_INVALID_ARG, "dk, dv must be positive");
    if (d->dk != kDK || d->dv != kDV)
        return fail(STEPQ_ERR_UNSUPPORTED, "only dk = dv = 128 is implemented (got %d x %d)", d->dk, d->dv);
    if ((long long)pd->requests * d->heads > STEPQ_MAX_ITEMS)
        return fail(STEPQ_ERR_INVALID_ARG, "requests * heads exceeds %d", STEPQ_MAX_ITEMS);
    if (d->max_length < 0) return fail(STEPQ_ERR_INVALID_ARG, "max_length %d < 0", d->max_length);
    const long long e = (long long)item_size(d->dtype);
    const long long qk = (long long)d->heads_qk * kDK, vv = (long long)d->heads * kDV, most = 1LL << 40;
    if (d->stride_q < qk || d->stride_k < qk || d->stride_v < vv || d->stride_q > most || d->stride_k > most ||
        d->stride_v > most)
        return fail(STEPQ_ERR_INVALID_ARG, "token stride smaller than a token's row, or above 2^40");
    if (d->stride_q * e % 16 || d->stride_k * e % 16 || d->stride_v * e % 16)
        return fail(STEPQ_ERR_INVALID_ARG, "token strides must be multiples of 16 bytes");
    return STEPQ_OK;
}

// Bytes a [tokens] tensor with a row stride spans.
size_t span(size_t tokens, long long stride, size_t row, size_t e)
{
    return tokens == 0 ? 0 : ((tokens - 1) * (size_t)stride + row) * e;
}

}  // namespace

extern "C" {

stepq_status stepq_plan_layout(const stepq_plan_desc *desc, stepq_plan_regions *out)
{
    if (!out) return fail(STEPQ_ERR_INVALID_ARG, "out is NULL");
    return plan_regions(desc, out);
}

size_t stepq_plan_bytes(const stepq_plan_desc *desc)
{
    stepq_plan_regions r;
    return plan_regions(desc, &r) == STEPQ_OK ? r.total : 0;
}

stepq_status stepq_plan_build(const stepq_plan_desc *desc, void *plan, size_t plan_bytes, int n, const int *lengths,
                              const int *contexts, const int *slots, uint8_t *busy, int max_length, void *cuda_stream)
{
    stepq_plan_regions r;
    stepq_status st = plan_regions(desc, &r);
    if (st != STEPQ_OK) return st;
    if (n < 0 || n > desc->requests)
        return fail(STEPQ_ERR_INVALID_ARG, "%d requests, the plan holds %d", n, desc->requests);
    if (max_length < 0) return fail(STEPQ_ERR_INVALID_ARG, "max_length %d < 0", max_length);
    stepq::PlanArgs a{};
    if ((st = plan_view(desc, plan, plan_bytes, &a.p)) != STEPQ_OK) return st;
    if (n > 0 && (st = check_here(lengths, "lengths", 4)) != STEPQ_OK) return st;
    if (n > 0 && contexts && (st = check_here(contexts, "contexts", 4)) != STEPQ_OK) return st;
    if (n > 0 && slots && (st = check_here(slots, "slots", 4)) != STEPQ_OK) return st;
    if (busy && !slots) return fail(STEPQ_ERR_INVALID_ARG, "busy without slots");
    if (busy && desc->slots > 0 && (st = check_here(busy, "busy", 1)) != STEPQ_OK) return st;
    const size_t nb = 4 * (size_t)n;
    if (overlaps(plan, r.total, lengths, nb) || (contexts && overlaps(plan, r.total, contexts, nb)) ||
        (slots && overlaps(plan, r.total, slots, nb)) || (busy && overlaps(plan, r.total, busy, desc->slots)))
        return fail(STEPQ_ERR_INVALID_ARG, "an input overlaps the plan");
    a.n = n;
    a.lengths = lengths;
    a.contexts = contexts;
    a.slots = slots;
    a.busy = desc->slots > 0 ? busy : nullptr;
    a.max_length = max_length;
    cudaError_t e = stepq::launch_plan(a, static_cast<cudaStream_t>(cuda_stream));
    return e == cudaSuccess ? STEPQ_OK : cuda_fail(e, "stepq_plan_build launch");
}

stepq_status stepq_plan_check(const stepq_plan_desc *desc, const void *plan, size_t plan_bytes, void *cuda_stream)
{
    stepq::PlanView v;
    stepq_status st = plan_view(desc, plan, plan_bytes, &v);
    if (st != STEPQ_OK) return st;
    int bits = 0;
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    cudaError_t e = cudaMemcpyAsync(&bits, v.head, sizeof bits, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "stepq_plan_check read");
    if (bits == 0) return STEPQ_OK;
    if (bits & STEPQ_PLAN_TIMEOUT)
        return fail(STEPQ_ERR_CUDA, "a prompt kernel gave up waiting for a copy; its requests' states and rows are not valid");
    return fail(STEPQ_ERR_INVALID_ARG, "the plan refused requests%s%s%s%s%s",
                bits & STEPQ_PLAN_BAD_LENGTH ? "; a length below 0 or above max_length" : "",
                bits & STEPQ_PLAN_TOO_MANY ? "; more tokens than the plan's capacity" : "",
                bits & STEPQ_PLAN_BAD_SLOT ? "; a slot out of range, or none given" : "",
                bits & STEPQ_PLAN_SLOT_TWICE ? "; two requests in one slot" : "",
                bits & STEPQ_PLAN_NO_SLOT ? "; no free slot left" : "");
}

size_t stepq_prompt_scratch_bytes(const stepq_plan_desc *plan_desc, const stepq_prompt_desc *desc)
{
    if (check_prompt_desc(plan_desc, desc) != STEPQ_OK) return (size_t)-1;
    if (plan_desc->requests == 0 || plan_desc->tokens == 0 || desc->max_length <= STEPQ_STEP_TOKENS) return 0;
    stepq::PromptArgs a{};
    a.p.requests = plan_desc->requests;
    a.p.blocks = plan_desc->tokens / STEPQ_BLOCK + plan_desc->requests;
    a.variant = desc->variant;
    a.dtype = desc->dtype;
    a.heads = desc->heads;
    a.share = desc->heads / desc->heads_qk;
    return stepq::prompt_scratch_bytes(a);
}

stepq_status stepq_prompt(const stepq_plan_desc *plan_desc, const void *plan, size_t plan_bytes,
                          const stepq_prompt_desc *desc, const void *q, const void *k, const void *v,
                          const float *alpha, const float *beta, float *S, void *out, void *scratch,
                          size_t scratch_bytes, void *cuda_stream)
{
    stepq_status st = check_prompt_desc(plan_desc, desc);
    if (st != STEPQ_OK) return st;
    const size_t need = stepq_prompt_scratch_bytes(plan_desc, desc);
    const size_t T = plan_desc->tokens, R = plan_desc->requests, H = desc->heads;
    stepq::PromptArgs a{};
    if ((st = plan_view(plan_desc, plan, plan_bytes, &a.p)) != STEPQ_OK) return st;
    if (T == 0 || R == 0) return STEPQ_OK;
    if ((st = check_here(q, "q", 16)) != STEPQ_OK) return st;
    if ((st = check_here(k, "k", 16)) != STEPQ_OK) return st;
    if ((st = check_here(v, "v", 16)) != STEPQ_OK) return st;
    if ((st = check_here(alpha, "alpha", desc->variant == STEPQ_KDA ? 16 : 4)) != STEPQ_OK) return st;
    if ((st = check_here(beta, "beta", 4)) != STEPQ_OK) return st;
    if ((st = check_here(S, "S", 16)) != STEPQ_OK) return st;
    if ((st = check_here(out, "out", 16)) != STEPQ_OK) return st;
    if (scratch_bytes < need)
        return fail(STEPQ_ERR_INVALID_ARG, "scratch of %zu bytes < %zu required", scratch_bytes, need);
    if (need > 0 && (st = check_here(scratch, "scratch", 256)) != STEPQ_OK) return st;
    const size_t e = item_size(desc->dtype);
    struct { const void *p; size_t n; const char *name; } in[] = {
        {q, span(T, desc->stride_q, (size_t)desc->heads_qk * kDK, e), "q"},
        {k, span(T, desc->stride_k, (size_t)desc->heads_qk * kDK, e), "k"},
        {v, span(T, desc->stride_v, H * kDV, e), "v"},
        {alpha, T * H * (desc->variant == STEPQ_KDA ? kDK : 1) * 4, "alpha"},
        {beta, T * H * 4, "beta"},
        {plan, plan_bytes, "plan"},
    };
    struct { const void *p; size_t n; const char *name; } wr[] = {
        {out, T * H * kDV * e, "out"},
        {S, (desc->by_slot ? (size_t)plan_desc->slots : R) * H * kDK * kDV * 4, "S"},
        {scratch, need, "scratch"},
    };
    for (int i = 0; i < 3; i++) {
        for (const auto &x : in)
            if (overlaps(wr[i].p, wr[i].n, x.p, x.n)) return fail(STEPQ_ERR_INVALID_ARG, "%s overlaps %s", wr[i].name, x.name);
        for (int j = 0; j < i; j++)
            if (overlaps(wr[i].p, wr[i].n, wr[j].p, wr[j].n))
                return fail(STEPQ_ERR_INVALID_ARG, "%s overlaps %s", wr[i].name, wr[j].name);
    }
    a.variant = desc->variant;
    a.dtype = desc->dtype;
    a.heads = desc->heads;
    a.share = desc->heads / desc->heads_qk;
    a.by_slot = desc->by_slot != 0;
    a.stride_q = desc->stride_q;
    a.stride_k = desc->stride_k;
    a.stride_v = desc->stride_v;
    a.q = q;
    a.k = k;
    a.v = v;
    a.alpha = alpha;
    a.beta = beta;
    a.S = S;
    a.out = out;
    a.scratch = static_cast<uint8_t *>(scratch);
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    // Token by token or in blocks, 8 tokens a request, us: gated Delta rule 4 requests
    // of 16 heads 19 / 28, 128 of 32 397 / 345 (6 tokens: 304 / 345); a gate per key
    // row 19 / 44 and 399 / 685; plain 17 / 22 and 288 / 292.  Blocks cost the same for
    // 1 to 64 tokens, so the forms meet near 8 whatever the batch.
    cudaError_t err = desc->max_length <= STEPQ_STEP_TOKENS ? stepq::launch_prompt_steps(a, s) : stepq::launch_prompt_blocks(a, s);
    return err == cudaSuccess ? STEPQ_OK : cuda_fail(err, "stepq_prompt launch");
}

stepq_status stepq_pack_requests(stepq_pool *pool, const stepq_plan_desc *plan_desc, const void *plan,
                                 size_t plan_bytes, const float *S, int by_slot)
{
    stepq_status st = check_pool(pool);
    if (st != STEPQ_OK) return st;
    stepq::PlanView v;
    if ((st = plan_view(plan_desc, plan, plan_bytes, &v)) != STEPQ_OK) return st;
    if (v.slots != pool->desc.batch)
        return fail(STEPQ_ERR_INVALID_ARG, "the plan has %d slots, the pool %d requests", v.slots, pool->desc.batch);
    const size_t H = pool->desc.heads;
    if ((size_t)v.requests * H > STEPQ_MAX_ITEMS)
        return fail(STEPQ_ERR_INVALID_ARG, "requests * heads exceeds %d", STEPQ_MAX_ITEMS);
    if (v.requests == 0 || v.slots == 0) return STEPQ_OK;
    if ((st = check_here(S, "S", 16)) != STEPQ_OK) return st;
    const size_t rows = by_slot ? v.slots : v.requests;
    if (overlaps(S, rows * H * kDK * kDV * 4, pool->dev, pool->bytes) || overlaps(plan, plan_bytes, pool->dev, pool->bytes))
        return fail(STEPQ_ERR_INVALID_ARG, "S or the plan overlaps the pool buffer");
    stepq::StepArgs a = base_args(pool);
    a.n_items = v.requests * (int)H;
    a.S_in = S;
    a.live = v.live;
    a.by_slot = by_slot != 0;
    cudaError_t e = stepq::launch_pack(a, pool->stream);
    return e == cudaSuccess ? STEPQ_OK : cuda_fail(e, "stepq_pack_requests launch");
}

static stepq_status check_beam(int groups, int beams, int vocab, int n)
{
    if (groups < 0) return fail(STEPQ_ERR_INVALID_ARG, "groups %d < 0", groups);
    if (beams < 1 || beams > STEPQ_MAX_BEAMS)
        return fail(STEPQ_ERR_INVALID_ARG, "beams %d outside 1..%d", beams, STEPQ_MAX_BEAMS);
    if (n < 1 || n > STEPQ_MAX_BEAMS) return fail(STEPQ_ERR_INVALID_ARG, "n %d outside 1..%d", n, STEPQ_MAX_BEAMS);
    if (vocab < 1 || vocab > (1 << 30)) return fail(STEPQ_ERR_INVALID_ARG, "vocab %d outside 1..2^30", vocab);
    if ((long long)groups * beams > STEPQ_MAX_ITEMS)
        return fail(STEPQ_ERR_INVALID_ARG, "groups * beams exceeds %d", STEPQ_MAX_ITEMS);
    return STEPQ_OK;
}

size_t stepq_beam_scratch_bytes(int groups, int beams, int vocab, int n)
{
    if (check_beam(groups, beams, vocab, n) != STEPQ_OK) return 0;
    return up(stepq::beam_scratch_bytes(groups, beams, vocab, n), 16) + 16;
}

stepq_status stepq_beam_select(int groups, int beams, int vocab, int n, int dtype, const void *logits, long long stride,
                               const float *scores, float *scores_out, int *parents, int *tokens, void *scratch,
                               size_t scratch_bytes, void *cuda_stream)
{
    stepq_status st = check_beam(groups, beams, vocab, n);
    if (st != STEPQ_OK) return st;
    if (dtype != STEPQ_F32 && dtype != STEPQ_F16 && dtype != STEPQ_BF16)
        return fail(STEPQ_ERR_INVALID_ARG, "dtype %d is none of STEPQ_F32, STEPQ_F16, STEPQ_BF16", dtype);
    if (stride < vocab || stride > (1LL << 40)) return fail(STEPQ_ERR_INVALID_ARG, "stride %lld of rows of %d", stride, vocab);
    if (groups == 0) return STEPQ_OK;
    const size_t e = item_size(dtype), G = groups, B = beams, N = n;
    if ((st = check_here(logits, "logits", e)) != STEPQ_OK) return st;
    if ((st = check_here(scores, "scores", 4)) != STEPQ_OK) return st;
    if ((st = check_here(scores_out, "scores_out", 4)) != STEPQ_OK) return st;
    if ((st = check_here(parents, "parents", 4)) != STEPQ_OK) return st;
    if ((st = check_here(tokens, "tokens", 4)) != STEPQ_OK) return st;
    const size_t need = stepq::beam_scratch_bytes(groups, beams, vocab, n);
    if (scratch_bytes < need)
        return fail(STEPQ_ERR_INVALID_ARG, "scratch of %zu bytes < %zu required", scratch_bytes, need);
    if ((st = check_here(scratch, "scratch", 16)) != STEPQ_OK) return st;
    struct { const void *p; size_t n; } x[] = {{scores_out, 4 * G * N}, {parents, 4 * G * N}, {tokens, 4 * G * N}, {scratch, need},
                                               {logits, ((G * B - 1) * (size_t)stride + vocab) * e}, {scores, 4 * G * B}};
    for (int i = 0; i < 4; i++)
        for (int j = 0; j < 6; j++)
            if (i != j && overlaps(x[i].p, x[i].n, x[j].p, x[j].n))
                return fail(STEPQ_ERR_INVALID_ARG, "an output or the scratch overlaps another tensor");
    const stepq::BeamArgs a = {groups, beams, vocab, n, dtype, logits, stride, scores, scores_out, parents, tokens,
                               static_cast<uint8_t *>(scratch)};
    cudaError_t err = stepq::launch_beam_select(a, static_cast<cudaStream_t>(cuda_stream));
    return err == cudaSuccess ? STEPQ_OK : cuda_fail(err, "stepq_beam_select launch");
}

static stepq_status reorder(uint8_t *base, size_t row_bytes, int groups, int beams, const int *parents, cudaStream_t s)
{
    stepq_status st;
    if (groups == 0 || row_bytes == 0) return STEPQ_OK;
    if ((st = check_here(base, "base", 16)) != STEPQ_OK) return st;
    if ((st = check_here(parents, "parents", 4)) != STEPQ_OK) return st;
    if (overlaps(base, row_bytes * groups * beams, parents, 4 * (size_t)groups * beams))
        return fail(STEPQ_ERR_INVALID_ARG, "parents overlaps the rows");
    // a CTA takes at least 512 bytes of every row of its group
    if (row_bytes / 512 + 1 > (size_t)INT_MAX / groups)
        return fail(STEPQ_ERR_UNSUPPORTED, "%d groups of rows of %zu bytes", groups, row_bytes);
    cudaError_t e = stepq::launch_reorder(base, row_bytes, groups, beams, parents, s);
    return e == cudaSuccess ? STEPQ_OK : cuda_fail(e, "reorder launch");
}

stepq_status stepq_reorder_rows(void *base, size_t row_bytes, int groups, int beams, const int *parents, void *cuda_stream)
{
    stepq_status st = check_beam(groups, beams, 1, 1);
    if (st != STEPQ_OK) return st;
    if (row_bytes % 16) return fail(STEPQ_ERR_INVALID_ARG, "row_bytes %zu is not a multiple of 16", row_bytes);
    return reorder(static_cast<uint8_t *>(base), row_bytes, groups, beams, parents, static_cast<cudaStream_t>(cuda_stream));
}

stepq_status stepq_pool_reorder(stepq_pool *pool, int first, int groups, int beams, const int *parents)
{
    stepq_status st = check_pool(pool);
    if (st != STEPQ_OK) return st;
    if ((st = check_beam(groups, beams, 1, 1)) != STEPQ_OK) return st;
    if (first < 0 || (long long)first + (long long)groups * beams > pool->desc.batch)
        return fail(STEPQ_ERR_INVALID_ARG, "%d groups of %d beams from request %d pass the pool's %d requests", groups,
                    beams, first, pool->desc.batch);
    return reorder(pool->dev + (size_t)first * (size_t)pool->req_bytes, (size_t)pool->req_bytes, groups, beams, parents,
                   pool->stream);
}

}  // extern "C"
