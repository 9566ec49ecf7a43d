// Internal declarations of the serving kernels: the plan of a ragged batch, the
// prompt pass, beam selection and reordering.  Not part of the C ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "stepq_internal.cuh"

namespace stepq {

constexpr int kBlockTokens = 64;  // STEPQ_BLOCK
constexpr int kF32 = 0, kF16 = 1, kBF16 = 2;         // STEPQ_F32 ...
constexpr int kGdn = 0, kKda = 1, kLinear = 2;       // STEPQ_GDN ...
// bits of a plan's status word (STEPQ_PLAN_*)
constexpr int kPlanBadLength = 1, kPlanTooMany = 2, kPlanBadSlot = 4, kPlanSlotTwice = 8, kPlanNoSlot = 16, kPlanTimeout = 32;

// The arrays of a plan's buffer (stepq_plan_regions).
struct PlanView {
    int requests, tokens, slots, blocks;  // capacity
    int *starts, *slot, *live, *fresh;
    int *token_request, *token_position;
    int *block_starts, *block_request, *block_first;
    int *head;
    int *owner, *list;  // scratch: [slots] the request that names a slot, [requests] free slots
};

struct PlanArgs {
    PlanView p;
    int n;  // requests of this batch
    const int *lengths, *contexts, *slots;
    uint8_t *busy;
    int max_length;
};
cudaError_t launch_plan(const PlanArgs &a, cudaStream_t s);

struct PromptArgs {
    PlanView p;
    int variant, dtype, heads, share;  // share: value heads of a query / key head
    int by_slot;
    long long stride_q, stride_k, stride_v;  // elements
    const void *q, *k, *v;
    const float *alpha, *beta;
    float *S;
    void *out;
    uint8_t *scratch;
};
// The recurrence token by token (any length; meant for a few tokens a request).
cudaError_t launch_prompt_steps(const PromptArgs &a, cudaStream_t s);
// The recurrence in blocks of tokens, and the scratch that takes.
size_t prompt_scratch_bytes(const PromptArgs &a);
cudaError_t launch_prompt_blocks(const PromptArgs &a, cudaStream_t s);

struct BeamArgs {
    int groups, beams, vocab, n, dtype;
    const void *logits;
    long long stride;  // elements
    const float *scores;
    float *scores_out;
    int *parents, *tokens;
    uint8_t *scratch;
};
size_t beam_scratch_bytes(int groups, int beams, int vocab, int n);
cudaError_t launch_beam_select(const BeamArgs &a, cudaStream_t s);
cudaError_t launch_reorder(uint8_t *base, size_t row_bytes, int groups, int beams, const int *parents, cudaStream_t s);

}  // namespace stepq
