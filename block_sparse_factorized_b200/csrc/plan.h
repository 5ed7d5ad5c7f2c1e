// plan.h -- parameters and launch of the serving step's plan (internal).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace st {

constexpr int PLAN_MAX_REQUESTS = 8192;  // four arrays in one CTA's shared memory

struct PlanParams {
    const int32_t *lens, *new_tokens, *free_pages, *free_count;
    int32_t *block_table, *lens_out, *free_left, *offsets, *slots, *positions, *status;
    int64_t tokens, max_pages, table_stride, page_size, free_capacity;
    int32_t requests;
};

cudaError_t launch_plan(const PlanParams &p, cudaStream_t s);

}  // namespace st
