// paged_decode.h -- parameters and launch of attention over a paged cache (internal).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace st {

constexpr int PD_TILE = 16;             // keys a warp takes at a time
constexpr int PD_CTAS_PER_SM = 3;
constexpr int PD_MAX_GRID = 1024;       // CTAs at most: a row's parts have their weights in shared memory
constexpr int PD_MAX_REQUESTS = 8192;   // the tile prefix sums live in shared memory

struct PagedParams {
    const void *q;              // [requests, heads, d]
    const char *k, *v;          // pages
    int64_t k_page, k_head, k_row, v_page, v_head, v_row;  // strides in bytes
    const int32_t *table, *lens;
    void *o;                    // [requests, heads, d]
    float *lse;                 // [requests, heads]
    float *parts;               // [grid, 2] partial results of split rows (workspace)
    int32_t *prefix;            // [requests + 1] tiles before each request (workspace)
    int32_t *err;
    int64_t table_stride, num_pages;
    int32_t capacity, window, sinks;  // <= 2^30
    int32_t requests, heads, kv, group, blocks, page_size, grid;  // blocks: head blocks per group
    float scale_log2;
};

// Floats of one partial result: per head M, L and O[d].
inline __host__ __device__ int pd_heads(int group) { return group <= 8 ? 8 : 16; }
inline __host__ __device__ int pd_part(int group, int d) { return pd_heads(group) * (d + 2); }

cudaError_t launch_paged_decode(const PagedParams &p, int dtype, int d, cudaStream_t s);

}  // namespace st
