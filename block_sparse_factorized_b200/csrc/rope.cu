// rope.cu -- per-head RMS norm of queries and keys with the position rotation in the same pass, its
// gradient, and the same pass storing new keys and values into the pages of a cache.
//
// One head row x of d elements, at position p:
//   y = r x w,  r = (mean(x^2) + eps)^(-1/2);   pair (y0, y1) with angle a = 2 pi p turns[i]:
//   z0 = m (y0 cos a - y1 sin a),  z1 = m (y1 cos a + y0 sin a)
// Gradient of g = dL/dz: the transposed rotation gives g' = (m (g0 cos a + g1 sin a),
// m (g1 cos a - g0 sin a)); with u = r x,  dw = sum g' u  and  dx = r (g' w - u mean(g' w u)).
//
// Bound by memory: two passes over the rows (three for the gradient) and about 3 operations per
// byte, so each row is read once, kept in registers (8 elements a lane, 4 to 32 lanes a row) and
// written once.  cos and sin are shared by all heads of a token: a CTA takes a few tokens, puts
// their (cos, sin) pairs into shared memory once and then works through the heads.  The angle is
// p turns[i] in 64 bits less its nearest whole number, exact to 2^-25 turns wherever p stands; a
// table of cosines would have to be read for every position instead.
#include "elem.cuh"
#include "kernels.h"
#include "lm.h"
#include "rope.h"

namespace st {
namespace {

constexpr int THREADS = 256;
constexpr int MAX_TOKENS = 8;  // tokens a CTA takes at a time
constexpr int MAX_PAIRS = 128;

struct Work {
    const RopeParams &p;
    int l, grp;       // lane in the row's group, group in the CTA
    bool active;      // the lane holds elements of the row (d / 8 need not be a power of two)
    bool turns;       // the lane's elements are rotated
    int pair0, src;   // first pair of the lane's elements; the lane with the partners (half layout)
    bool second;      // half layout: the lane holds the second elements of its pairs

    template <int L>
    __device__ static Work make(const RopeParams &p)
    {
        const int l = threadIdx.x % L, e0 = 8 * l, half = p.rot / 2;
        Work w{p, l, static_cast<int>(threadIdx.x) / L, e0 < p.d, e0 < p.rot, 0, l, false};
        if (p.interleaved) {
            w.pair0 = e0 / 2;
        } else {
            w.second = e0 >= half;
            w.pair0 = w.second ? e0 - half : e0;
            if (w.turns) w.src = w.second ? l - half / 8 : l + half / 8;
        }
        return w;
    }
};

template <int L>
__device__ __forceinline__ float group_sum(float x)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The rotation (dir = 1) or its transpose (dir = -1) of the lane's 8 elements.  Every lane of the
// warp takes part in the exchange.
template <int L>
__device__ __forceinline__ void rotate(const Work &w, const float2 *cs, float dir, float (&x)[8])
{
    if (w.p.interleaved) {
        if (!w.turns) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 t = cs[w.pair0 + e];
            const float s = dir * t.y, a = x[2 * e], b = x[2 * e + 1];
            x[2 * e] = a * t.x - b * s;
            x[2 * e + 1] = b * t.x + a * s;
        }
        return;
    }
    const float sign = w.second ? dir : -dir;
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], w.src, L);
    if (!w.turns) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float2 t = cs[w.pair0 + e];
        x[e] = x[e] * t.x + sign * t.y * y[e];
    }
}

// (cos, sin) times mscale of the tile's tokens t0 .. t0 + nt - 1 of batch element b.
__device__ __forceinline__ void fill_angles(const RopeParams &p, int64_t b, int64_t t0, int nt, float2 *cs)
{
    const int half = p.rot / 2;
    for (int i = threadIdx.x; i < nt * half; i += THREADS) {
        const int tk = i / half, k = i - tk * half;
        const int64_t t = t0 + tk;
        const double pos = p.positions ? static_cast<double>(p.positions[b * p.pos_batch + t])
                                       : static_cast<double>(p.start + t);
        double a = pos * p.turns[k];
        a -= rint(a);
        float s, c;
        sincospif(2.f * static_cast<float>(a), &s, &c);
        cs[i] = make_float2(c * p.mscale, s * p.mscale);
    }
}

template <int DT>
__device__ __forceinline__ void load_weights(const RopeParams &p, const void *w, const Work &k, float (&x)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
    if (!w || !k.active) return;
    if (p.w_f32)
        widen8<ST_FP32>(load8<ST_FP32>(static_cast<const float *>(w) + 8 * k.l), x);
    else
        widen8<DT>(load8<DT>(static_cast<const char *>(w) + 8 * k.l * (DT == ST_FP32 ? 4 : 2)), x);
}

__device__ __forceinline__ char *row_at(const RopeTensor &t, int64_t b, int64_t h, int64_t r)
{
    return t.p + b * t.batch + h * t.head + r * t.row;
}

constexpr int UNROLL = 4;  // rows a group has in flight

// Head row j of a token: 0 .. heads - 1 queries, then the keys, then (append) the values.
template <int DT, int L, bool APPEND>
__global__ void __launch_bounds__(THREADS) rope_fwd_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int ES = DT == ST_FP32 ? 4 : 2, NG = THREADS / L;
    __shared__ float2 cs[MAX_TOKENS * MAX_PAIRS];
    const int64_t b = blockIdx.x / p.tiles, t0 = (blockIdx.x - b * p.tiles) * static_cast<int64_t>(p.tile);
    const int nt = static_cast<int>(min(static_cast<int64_t>(p.tile), p.n - t0));
    const Work w = Work::make<L>(p);
    float wq[8], wk[8];
    load_weights<DT>(p, p.wq, w, wq);
    load_weights<DT>(p, p.wk, w, wk);
    fill_angles(p, b, t0, nt, cs);
    __syncthreads();
    const int nh = p.heads + p.kv + (APPEND ? p.kv : 0), rows = nt * nh;
    for (int r0 = 0; r0 < rows; r0 += UNROLL * NG) {
        Vec8<DT> v[UNROLL];
        char *dst[UNROLL];
        int tk[UNROLL], j[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int r = r0 + u * NG + w.grp;
            dst[u] = nullptr;
            tk[u] = r / nh;
            j[u] = r - tk[u] * nh;
#pragma unroll
            for (auto &q : v[u].r) q = make_uint4(0u, 0u, 0u, 0u);
            if (r >= rows) {
                tk[u] = 0;
                continue;
            }
            const int64_t t = t0 + tk[u];
            const bool isq = j[u] < p.heads, isk = !isq && j[u] < p.heads + p.kv;
            const int h = isq ? j[u] : (isk ? j[u] - p.heads : j[u] - p.heads - p.kv);
            if constexpr (APPEND) {
                const int64_t slot = p.slots[t];
                if (slot < 0 || slot >= p.nslots) continue;
                const int64_t page = slot / p.page_size, at = slot - page * p.page_size;
                dst[u] = isq ? row_at(p.qo, 0, h, t) : row_at(isk ? p.ko : p.vo, page, h, at);
            } else {
                dst[u] = row_at(isq ? p.qo : p.ko, b, h, t);
            }
            if (w.active) v[u] = load8<DT>(row_at(isq ? p.q : (isk ? p.k : p.v), b, h, t) + 8 * w.l * ES);
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const bool copy = APPEND && j[u] >= p.heads + p.kv;  // a value row
            float x[8];
            widen8<DT>(v[u], x);
            if (p.wq) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
                const float r = rsqrtf(group_sum<L>(ss) * p.inv_d + p.eps);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = x[e] * r * (j[u] < p.heads ? wq[e] : wk[e]);
            }
            rotate<L>(w, cs + tk[u] * (p.rot / 2), 1.f, x);
            if (dst[u] && w.active) store8<DT>(dst[u] + 8 * w.l * ES, copy ? v[u] : round8<DT>(x));
        }
    }
}

// One CTA walks tiles blockIdx.x, blockIdx.x + gridDim.x, ...: the weights' gradients stay in its
// registers and leave as one partial row a CTA, added in a fixed order by rope_dw_kernel.
template <int DT, int L>
__global__ void __launch_bounds__(THREADS) rope_bwd_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int ES = DT == ST_FP32 ? 4 : 2, NG = THREADS / L, U = 2;
    __shared__ float2 cs[MAX_TOKENS * MAX_PAIRS];
    __shared__ float red[NG][8 * L];
    const Work w = Work::make<L>(p);
    float wq[8], wk[8], aq[8], ak[8];
    load_weights<DT>(p, p.wq, w, wq);
    load_weights<DT>(p, p.wk, w, wk);
#pragma unroll
    for (int e = 0; e < 8; ++e) aq[e] = ak[e] = 0.f;
    const int nh = p.heads + p.kv;
    for (int64_t tile = blockIdx.x; tile < static_cast<int64_t>(p.batch) * p.tiles; tile += gridDim.x) {
        const int64_t b = tile / p.tiles, t0 = (tile - b * p.tiles) * p.tile;
        const int nt = static_cast<int>(min(static_cast<int64_t>(p.tile), p.n - t0)), rows = nt * nh;
        __syncthreads();  // the previous tile's angles are no longer read
        fill_angles(p, b, t0, nt, cs);
        __syncthreads();
        for (int r0 = 0; r0 < rows; r0 += U * NG) {
            Vec8<DT> vx[U], vg[U];
            char *dst[U];
            int tk[U], j[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + u * NG + w.grp;
                tk[u] = r / nh;
                j[u] = r - tk[u] * nh;
                dst[u] = nullptr;
#pragma unroll
                for (auto &q : vx[u].r) q = make_uint4(0u, 0u, 0u, 0u);
                vg[u] = vx[u];
                if (r >= rows) {
                    tk[u] = 0;
                    continue;
                }
                const bool isq = j[u] < p.heads;
                const int h = isq ? j[u] : j[u] - p.heads;
                const int64_t t = t0 + tk[u];
                dst[u] = row_at(isq ? p.qo : p.ko, b, h, t);
                if (w.active) {
                    if (p.wq) vx[u] = load8<DT>(row_at(isq ? p.q : p.k, b, h, t) + 8 * w.l * ES);
                    vg[u] = load8<DT>(row_at(isq ? p.gq : p.gk, b, h, t) + 8 * w.l * ES);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float g[8];
                widen8<DT>(vg[u], g);
                rotate<L>(w, cs + tk[u] * (p.rot / 2), -1.f, g);
                if (p.wq) {
                    const bool isq = j[u] < p.heads;
                    float x[8], ss = 0.f, dot = 0.f;
                    widen8<DT>(vx[u], x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
                    const float r = rsqrtf(group_sum<L>(ss) * p.inv_d + p.eps);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x[e] *= r;
                        const float t = g[e] * x[e];
                        aq[e] += isq ? t : 0.f;  // rows past the tile were loaded as zeros
                        ak[e] += isq ? 0.f : t;
                        g[e] *= isq ? wq[e] : wk[e];
                        dot = fmaf(g[e], x[e], dot);
                    }
                    dot = group_sum<L>(dot) * p.inv_d;
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[e] = r * (g[e] - x[e] * dot);
                }
                if (dst[u] && w.active) store8<DT>(dst[u] + 8 * w.l * ES, round8<DT>(g));
            }
        }
    }
    if (!p.wq) return;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) red[w.grp][8 * w.l + e] = which ? ak[e] : aq[e];
        __syncthreads();
        for (int c = threadIdx.x; c < p.d; c += THREADS) {
            float s = 0.f;
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) s += red[gi][c];
            p.partial[(static_cast<size_t>(blockIdx.x) * 2 + which) * p.d + c] = s;
        }
    }
}

// dw = sum of the CTAs' partial rows: 32 columns by 32 row lanes a CTA, the lanes added in order.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float *partial, int32_t rows, int32_t d, float *dwq, float *dwk)
{
    __shared__ float red[32][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), lane = threadIdx.x >> 5;
    float s = 0.f;
    if (c < 2 * d)
#pragma unroll 8
        for (int r = lane; r < rows; r += 32) s += partial[static_cast<size_t>(r) * 2 * d + c];
    red[lane][threadIdx.x & 31] = s;
    __syncthreads();
    if (lane == 0 && c < 2 * d) {
        s = 0.f;
        for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
        (c < d ? dwq[c] : dwk[c - d]) = s;
    }
}

template <int DT, int L>
cudaError_t launch_l(const RopeParams &p, int mode, int64_t grid, cudaStream_t s)
{
    const unsigned g = static_cast<unsigned>(grid);
    if (mode == ROPE_FWD) rope_fwd_kernel<DT, L, false><<<g, THREADS, 0, s>>>(p);
    else if (mode == ROPE_APPEND) rope_fwd_kernel<DT, L, true><<<g, THREADS, 0, s>>>(p);
    else rope_bwd_kernel<DT, L><<<g, THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

template <int DT>
cudaError_t launch_t(const RopeParams &p, int mode, int64_t grid, cudaStream_t s)
{
    if (p.d <= 32) return launch_l<DT, 4>(p, mode, grid, s);
    if (p.d <= 64) return launch_l<DT, 8>(p, mode, grid, s);
    if (p.d <= 128) return launch_l<DT, 16>(p, mode, grid, s);
    return launch_l<DT, 32>(p, mode, grid, s);
}

}  // namespace

int rope_tile(int64_t tokens)
{
    // tokens a CTA takes: 8, fewer while that leaves under eight CTAs an SM
    int tile = MAX_TOKENS;
    while (tile > 1 && tokens / tile < 8ll * sm_count()) tile /= 2;
    return tile;
}

int64_t rope_bwd_ctas(int64_t tiles)
{
    const int64_t cap = 4ll * sm_count();
    return tiles < cap ? tiles : cap;
}

cudaError_t launch_rope(RopeParams &p, int dtype, int mode, float *dwq, float *dwk, cudaStream_t s)
{
    p.tile = rope_tile(p.batch * p.n);
    p.tiles = (p.n + p.tile - 1) / p.tile;
    const int64_t all = p.batch * p.tiles, grid = mode == ROPE_BWD ? rope_bwd_ctas(all) : all;
    cudaError_t e = dtype == ST_BF16   ? launch_t<ST_BF16>(p, mode, grid, s)
                    : dtype == ST_FP16 ? launch_t<ST_FP16>(p, mode, grid, s)
                                       : launch_t<ST_FP32>(p, mode, grid, s);
    if (e != cudaSuccess || mode != ROPE_BWD || !p.wq) return e;
    rope_dw_kernel<<<static_cast<unsigned>((2 * p.d + 31) / 32), 1024, 0, s>>>(p.partial, static_cast<int32_t>(grid), p.d, dwq, dwk);
    return cudaGetLastError();
}

}  // namespace st
