// rope.h -- parameters and launch of the norm-and-rotation kernels (internal).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace st {

enum { ROPE_FWD = 0, ROPE_APPEND = 1, ROPE_BWD = 2 };

struct RopeTensor {
    char *p;
    int64_t batch, head, row;  // strides in bytes
};

struct RopeParams {
    RopeTensor q, k, v;        // inputs (v: append)
    RopeTensor gq, gk;         // backward: gradients of the outputs
    RopeTensor qo, ko, vo;     // outputs (append: ko, vo are the pages, batch = page)
    const void *wq, *wk;       // [d] weights or NULL
    const uint64_t *turns;     // [rot / 2], 2^-64 turns per position
    const int32_t *positions;  // or NULL: start + t
    const int32_t *slots;      // append
    int64_t n, start, pos_batch, page_size, nslots;
    int64_t batch, items;      // items: (token, run of its rows)
    int32_t heads, kv, d, rot, interleaved, w_f32;
    int64_t tokens0;           // forward: tokens that one group takes whole, before those cut into runs
    int32_t run, parts;        // rows of a run, runs of a token
    int64_t items_k;           // backward: of the keys (the others: of the queries)
    int32_t run_k, parts_k, q_ctas;
    float eps, mscale, inv_d;
    float *partial;            // backward: [CTAs, d] partial weight gradients
};

// CTAs of a backward for the queries and for the keys.
struct RopeCtas {
    int64_t q, k;
};
RopeCtas rope_bwd_ctas(int64_t tokens, int heads, int kv, int d);
cudaError_t launch_rope(RopeParams &p, int dtype, int mode, float *dwq, float *dwk, cudaStream_t s);

}  // namespace st
