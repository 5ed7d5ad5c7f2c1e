// window.h -- parameters, work units and launches of sliding-window attention (internal).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "frames.cuh"

namespace st {

// Geometry of a call, and the raw tensors for the tiles that cannot come by TMA (those with rows at
// or past the sequence's length, which are read as zeros).
struct WindowGeom {
    const int32_t *lens;         // [batch] or NULL
    int32_t batch, heads, kv, group, nq, nk, q_start, window, sinks;
    int32_t nqt, nkt;            // query and key tiles of 128 rows
    float scale_log2, scale;     // log2(e) / sqrt(d), 1 / sqrt(d)
    int32_t *err;
};

struct RawTensor {
    const char *p;
    int64_t batch, head, row;    // strides in bytes
};

// Sequence length of batch element b.
ST_HD int32_t window_len(const WindowGeom &g, int32_t b)
{
    if (!g.lens) return g.nk;
    const int32_t x = g.lens[b];
    return x < 0 ? 0 : (x > g.nk ? g.nk : x);
}

// Key tiles that the live rows of a query tile read: 0 .. ns - 1 and kb0 .. kb1.
struct KeyRange {
    int32_t kb0, kb1, ns;
    bool any;                    // some row of the tile is live
};

// Rows row0 .. row0 + 127 of a sequence of length len.
ST_HD KeyRange key_range(const WindowGeom &g, int32_t row0, int32_t len)
{
    KeyRange r{0, -1, 0, false};
    const int32_t p0 = g.q_start + row0;
    const int32_t rows = g.nq - row0 < 128 ? g.nq - row0 : 128;
    const int32_t z = p0 + rows - 1 < len - 1 ? p0 + rows - 1 : len - 1;  // last live position
    if (rows <= 0 || z < p0) return r;
    r.any = true;
    const int32_t lo = g.window && p0 - g.window + 1 > 0 ? p0 - g.window + 1 : 0;
    r.kb0 = lo / 128;
    r.kb1 = z / 128;
    const int32_t s = g.sinks < z + 1 ? g.sinks : z + 1, ns = (s + 127) / 128;
    r.ns = ns < r.kb0 ? ns : r.kb0;
    return r;
}

// Query tiles whose rows read key tile t: i0 .. i1 (i1 < i0: none), for a sequence of nk positions (a
// shorter one has no others).
ST_HD void query_range(const WindowGeom &g, int32_t t, int32_t &i0, int32_t &i1)
{
    const int32_t k0 = t * 128, k1 = k0 + 127 < g.nk - 1 ? k0 + 127 : g.nk - 1;
    const int32_t first = k0 - g.q_start;  // first query row at or past the tile's first key
    i0 = first > 0 ? first / 128 : 0;
    int64_t last = static_cast<int64_t>(g.nq) - 1;
    if (g.window && k0 >= g.sinks) {       // no sinks in the tile: the window ends the run
        const int64_t w = static_cast<int64_t>(k1) + g.window - 1 - g.q_start;
        if (w < last) last = w;
    }
    i1 = last < 0 || first > last ? i0 - 1 : static_cast<int32_t>(last / 128);
}

struct WindowFwdParams {
    CUtensorMap q, k, v;
    WindowGeom g;
    RawTensor vraw;
    char *o;
    int64_t o_batch, o_head, o_row;  // strides in bytes
    float *lse;
    int32_t units, pair_rows;        // pair_rows: a unit is two row tiles of a head, not two heads
};

struct OutTensor {
    char *p;
    int64_t batch, head, row;        // strides in bytes
};

// Chunks of at most `chunk` steps that a key tile's steps are cut into (one for a tile without any,
// whose gradients are zero).
ST_HD int32_t chunks_of(int32_t steps, int32_t chunk) { return steps <= chunk ? 1 : (steps + chunk - 1) / chunk; }

struct WindowBwdParams {
    CUtensorMap q, k, v, dout;
    WindowGeom g;
    RawTensor qraw, kraw, vraw, oraw, doraw;
    OutTensor dq, dk, dv;
    const float *lse;
    float *delta;                    // [batch, heads, nq] D_i (workspace)
    float *parts;                    // fp32 dV, dK partials of chunked key tiles (workspace)
    int2 *entries;                   // (key tile, chunk) units, chunked tiles first (workspace)
    int32_t *counters;               // next unit of dk_dv, of dq; whether dq may read (workspace)
    uint32_t *maxima;                // fp16: [batch, kv, 2] largest squared norms of dO and V (workspace)
    int32_t nentries, nsplit, chunk; // units a key head, those of chunked tiles, steps a chunk at most
};

cudaError_t launch_window_bwd(const WindowBwdParams &p, int dtype, int d, cudaStream_t s);
cudaError_t launch_window_fwd(const WindowFwdParams &p, int dtype, int d, cudaStream_t s);

}  // namespace st
