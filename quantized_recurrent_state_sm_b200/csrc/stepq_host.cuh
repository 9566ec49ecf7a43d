// What the host files of the C ABI share: the pool handle and the argument
// checks.  Not part of the C ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <vector>

#include "stepq.h"
#include "stepq_internal.cuh"

struct stepq_pool {
    stepq_desc desc;  // table pointers cleared; the tables are copied below
    std::vector<uint8_t> bits;
    std::vector<float> rho;
    uint8_t *dev = nullptr;
    size_t bytes = 0, state_bytes = 0;
    long long req_bytes = 0;
    cudaStream_t stream = nullptr;
    stepq::Tables t{};
    int n_pivot_items = 0;
    int max_n16 = 0;  // the most leading 16-bit field positions of a staged head
    int scale_mode = STEPQ_SCALE_DUAL;
    int nslots = 0, slot_bytes = 0;
    int off_q = 0, off_k = 0, off_v = 0, off_alpha = 0, off_ab = 0, off_rec = 0;
    // the active request set: decode steps update requests active[0..n_active)
    int n_active = 0;
    std::vector<int> kind;               // per head: kHeadQuant / kHeadAllPivot / kHeadMixed
    std::vector<long long> item_bytes;   // per head
    std::vector<long long> head_off;     // per head
    std::vector<int> active_tables;      // host copy of the uploaded order and staging records
    size_t guard[7] = {};                // offsets of the guard regions (kGuardRegions)
    size_t total = 0;                    // bytes of the pool's regions, guards included
};

namespace stepq {
namespace host {

// Sets the calling thread's error text (stepq_last_error) and returns s.
stepq_status fail(stepq_status s, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// A live pool handle.
stepq_status check_pool(const stepq_pool *p);
// A device tensor argument: non-null, aligned, and memory the GPU can address.
stepq_status check_dev(const void *ptr, const char *name, size_t align);
bool overlaps(const void *a, size_t na, const void *b, size_t nb);
stepq_status cuda_fail(cudaError_t e, const char *what);
StepArgs base_args(const stepq_pool *p);

}  // namespace host
}  // namespace stepq
