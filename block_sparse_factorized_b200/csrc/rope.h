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
    const double *turns;       // [rot / 2]
    const int32_t *positions;  // or NULL: start + t
    const int32_t *slots;      // append
    int64_t n, start, pos_batch, tiles, page_size, nslots;
    int64_t batch;
    int32_t heads, kv, d, rot, interleaved, tile, w_f32;
    float eps, mscale, inv_d;
    float *partial;            // backward: [CTAs, 2, d] partial weight gradients
};

// Tokens a CTA takes at a time, and the CTAs of a backward over `tiles` tiles.
int rope_tile(int64_t tokens);
int64_t rope_bwd_ctas(int64_t tiles);
cudaError_t launch_rope(RopeParams &p, int dtype, int mode, float *dwq, float *dwk, cudaStream_t s);

}  // namespace st
