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
// byte, so each row is read once, kept in registers and written once, and the instructions a row costs
// decide: at 130 a row and warp the kernel was bound by issue at a third of the memory's rate.  So a
// lane holds 16 elements, both of each of its eight pairs (in the half layout two pieces of 8, rot / 2
// apart), and the rotation needs no exchange; a group of 2 to 16 lanes takes one token and a run of
// its heads, whose cosines and sines stay in registers; and a run's last rows are repeated rather than
// predicated.  The angle is p turns[i] modulo a turn, with turns[i] in units of 2^-64 turns and the
// product in 64-bit integers: exact to 2^-25 turns wherever p stands, and a few integer instructions (in
// fp64 the conversions alone took a fifth of the kernel's time); a table of cosines would have to be
// read for every position instead.
//
// Measured, bf16, d = 128 (of 6549 GB/s for a copy): forward of 24576 tokens of 16 + 4 heads 51 us,
// 4.9 TB/s; append of 8192 tokens of 32 + 8 + 8 heads 41 us, 4.8 TB/s; backward of 16390 tokens of 16 + 4
// heads 70 us, 3.6 TB/s, where neither the memory (49% busy) nor issue (57%) is full: a group has one row
// on its way besides the one it works on, at 128 registers a thread and two CTAs an SM.  In fp32: forward 88 us,
// 5.7 TB/s; append 94 us, 4.3 TB/s; backward 124 us, 4.1 TB/s.
#include "elem.cuh"
#include "kernels.h"
#include "lm.h"
#include "rope.h"

namespace st {
namespace {

// Threads a CTA.  The forward's CTAs end with their items, so small ones, at the same number of warps an
// SM, leave less of the memory idle at the end (24576 tokens of 20 rows: 53 us with 256, 51 with 128 or 64);
// the backward's walk, and each leaves a partial row.
constexpr int FWD_THREADS = 128, THREADS = 256;
constexpr int U = 4;  // rows a group has in flight

// The lane's part in its group's rows: elements a .. a + 7 and b .. b + 7.
template <int L>
struct Lane {
    int l, grp, a, b;
    uint32_t mask;    // the group's lanes of the warp
    bool active;      // d / 16 need not be a power of two
    bool turns;       // the elements are rotated: eight pairs, the first being pair 8 l
    bool inter;       // pairs (a, a + 1), (a + 2, a + 3), ..; else (a + i, b + i)

    __device__ explicit Lane(const RopeParams &p)
    {
        l = threadIdx.x % L;
        grp = threadIdx.x / L;
        mask = ((1u << L) - 1u) << ((threadIdx.x & 31) / L * L);
        active = 16 * l < p.d;
        turns = 16 * l < p.rot;
        inter = p.interleaved != 0;
        a = turns && !inter ? 8 * l : (active ? 16 * l : 0);  // (an idle lane reads lane 0's place)
        b = turns && !inter ? p.rot / 2 + 8 * l : a + 8;
    }
    __device__ float sum(float x) const
    {
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(mask, x, o);
        return x;
    }
};

// cos and sin (times mscale) of the lane's pairs.  For 16-bit rows the fast forms do: their error of some
// 2^-21 is far below the rounding of the result (2^-12 and 2^-9).
template <int DT, int L>
__device__ __forceinline__ void angles(const RopeParams &p, const Lane<L> &w, int64_t pos, float (&c)[8], float (&s)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint64_t a = w.turns ? static_cast<uint64_t>(pos) * p.turns[8 * w.l + e] : 0ull;
        const float half_turns = static_cast<float>(static_cast<int32_t>(a >> 32)) * 0x1p-31f;  // -1 .. 1
        if constexpr (DT == ST_FP32)
            sincospif(half_turns, &s[e], &c[e]);
        else
            __sincosf(half_turns * 3.14159265f, &s[e], &c[e]);
        c[e] *= p.mscale;
        s[e] *= p.mscale;
    }
}

// The rotation (of the transpose: s negated) of the lane's elements x[0 .. 7] = a .., x[8 .. 15] = b ..
template <int L>
__device__ __forceinline__ void rotate(const Lane<L> &w, const float (&c)[8], const float (&s)[8], float (&x)[16])
{
    if (!w.turns) return;
    if (w.inter) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float u = x[2 * e], v = x[2 * e + 1];
            x[2 * e] = u * c[e] - v * s[e];
            x[2 * e + 1] = v * c[e] + u * s[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float u = x[e], v = x[e + 8];
            x[e] = u * c[e] - v * s[e];
            x[e + 8] = v * c[e] + u * s[e];
        }
    }
}

// The lane's two pieces of a row, as loaded.
template <int DT>
struct Row {
    Vec8<DT> a, b;
};

template <int DT>
__device__ __forceinline__ Row<DT> load_row(const char *row, int a, int b)
{
    constexpr int ES = DT == ST_FP32 ? 4 : 2;
    return {load8<DT>(row + ES * a), load8<DT>(row + ES * b)};
}

template <int DT>
__device__ __forceinline__ void store_row(char *row, int a, int b, const Row<DT> &v)
{
    constexpr int ES = DT == ST_FP32 ? 4 : 2;
    store8<DT>(row + ES * a, v.a);
    store8<DT>(row + ES * b, v.b);
}

template <int DT>
__device__ __forceinline__ void widen(const Row<DT> &v, float (&x)[16])
{
    widen8<DT>(v.a, *reinterpret_cast<float(*)[8]>(&x[0]));
    widen8<DT>(v.b, *reinterpret_cast<float(*)[8]>(&x[8]));
}

template <int DT>
__device__ __forceinline__ Row<DT> narrow(const float (&x)[16])
{
    return {round8<DT>(*reinterpret_cast<const float(*)[8]>(&x[0])), round8<DT>(*reinterpret_cast<const float(*)[8]>(&x[8]))};
}

template <int DT, int L>
__device__ __forceinline__ void load_weights(const RopeParams &p, const void *w, const Lane<L> &k, float (&x)[16])
{
    if (!w) {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = 1.f;
    } else if (p.w_f32) {
        widen<ST_FP32>(load_row<ST_FP32>(static_cast<const char *>(w), k.a, k.b), x);
    } else {
        widen<DT>(load_row<DT>(static_cast<const char *>(w), k.a, k.b), x);
    }
}

// A group's item: a token (b, t) and the rows j0 .. j1 - 1 of its heads (queries, then keys, then for
// an append values).
struct Item {
    int64_t b, t;
    int j0, j1;
};

__device__ __forceinline__ Item item_of(const RopeParams &p, uint32_t i, int64_t first, int nh, int run, int parts)
{
    Item r;
    uint32_t token = i / static_cast<uint32_t>(parts);
    const uint32_t part = i - token * parts;
    token += static_cast<uint32_t>(first);
    r.b = token / static_cast<uint32_t>(p.n);
    r.t = token - static_cast<uint32_t>(r.b) * static_cast<uint32_t>(p.n);
    r.j0 = static_cast<int>(part) * run;
    r.j1 = min(nh, r.j0 + run);
    return r;
}

__device__ __forceinline__ int64_t position(const RopeParams &p, const Item &it)
{
    return p.positions ? p.positions[it.b * p.pos_batch + it.t] : p.start + it.t;
}

template <int DT, int L, bool APPEND>
__global__ void __launch_bounds__(FWD_THREADS, DT == ST_FP32 ? 2 : 4) rope_fwd_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int NG = FWD_THREADS / L;
    const Lane<L> w(p);
    const uint32_t i = blockIdx.x * NG + w.grp;
    if (i >= p.items) return;
    const int nh = p.heads + p.kv + (APPEND ? p.kv : 0);
    const Item it = i < p.tokens0 ? item_of(p, i, 0, nh, nh, 1)
                                  : item_of(p, i - static_cast<uint32_t>(p.tokens0), p.tokens0, nh, p.run, p.parts);
    int64_t page = 0, at = 0;
    if constexpr (APPEND) {
        const int32_t slot = p.slots[it.t];
        if (slot < 0 || slot >= p.nslots) return;
        page = static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.page_size);
        at = slot - page * p.page_size;
    }
    float c[8], s[8];
    angles<DT>(p, w, position(p, it), c, s);
    const bool norm = p.wq != nullptr;
    // rows lo .. hi - 1 of a token's heads from src (head 0) to dst, U at a time; the last are repeated
    auto part = [&](int lo, int hi, const char *src, int64_t src_head, char *dst, int64_t dst_head, const void *weights, bool copy) {
        const int first = max(it.j0, lo), n = min(it.j1, hi) - first;
        if (n <= 0) return;
        float wt[16];
        load_weights<DT>(p, weights, w, wt);
        src += (first - lo) * src_head;
        dst += (first - lo) * dst_head;
        for (int j = 0; j < n; j += U) {
            Row<DT> v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = load_row<DT>(src + min(j + u, n - 1) * src_head, w.a, w.b);
            if (!copy) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float x[16];
                    widen<DT>(v[u], x);
                    if (norm) {
                        float ss = 0.f;
#pragma unroll
                        for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
                        const float r = rsqrtf(w.sum(w.active ? ss : 0.f) * p.inv_d + p.eps);
#pragma unroll
                        for (int e = 0; e < 16; ++e) x[e] *= r * wt[e];
                    }
                    rotate(w, c, s, x);
                    v[u] = narrow<DT>(x);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (w.active) store_row<DT>(dst + min(j + u, n - 1) * dst_head, w.a, w.b, v[u]);
        }
    };
    auto row = [&](const RopeTensor &t) { return t.p + it.b * t.batch + it.t * t.row; };
    part(0, p.heads, row(p.q), p.q.head, row(p.qo), p.qo.head, p.wq, false);
    if constexpr (APPEND) {
        part(p.heads, p.heads + p.kv, row(p.k), p.k.head, p.ko.p + page * p.ko.batch + at * p.ko.row, p.ko.head, p.wk, false);
        part(p.heads + p.kv, p.heads + 2 * p.kv, row(p.v), p.v.head, p.vo.p + page * p.vo.batch + at * p.vo.row, p.vo.head, nullptr, true);
    } else {
        part(p.heads, p.heads + p.kv, row(p.k), p.k.head, row(p.ko), p.ko.head, p.wk, false);
    }
}

// The first q_ctas CTAs take the queries, the others the keys; a group walks its tokens and keeps the
// weights and their gradient in its registers, which leave as one partial row a CTA, added in a fixed
// order by rope_dw_kernel.
template <int DT, int L>
__global__ void __launch_bounds__(THREADS, DT == ST_FP32 ? 1 : 2) rope_bwd_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int NG = THREADS / L;
    __shared__ float red[NG][16 * L];
    const Lane<L> w(p);
    const bool norm = p.wq != nullptr, isq = blockIdx.x < static_cast<unsigned>(p.q_ctas);
    const RopeTensor &xs = isq ? p.q : p.k, &gs = isq ? p.gq : p.gk, &ds = isq ? p.qo : p.ko;
    const uint32_t cta = isq ? blockIdx.x : blockIdx.x - p.q_ctas, ctas = isq ? p.q_ctas : gridDim.x - p.q_ctas;
    const int rows = isq ? p.heads : p.kv, run = isq ? p.run : p.run_k, parts = isq ? p.parts : p.parts_k;
    const uint32_t items = isq ? p.items : p.items_k;
    float wt[16], acc[16];
    load_weights<DT>(p, isq ? p.wq : p.wk, w, wt);
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.f;
    for (uint32_t i = cta * NG + w.grp; i < items; i += ctas * NG) {
        const Item it = item_of(p, i, 0, rows, run, parts);
        const int n = it.j1 - it.j0;
        const char *xp = xs.p + it.b * xs.batch + it.t * xs.row + it.j0 * xs.head;
        const char *gp = gs.p + it.b * gs.batch + it.t * gs.row + it.j0 * gs.head;
        char *dp = ds.p + it.b * ds.batch + it.t * ds.row + it.j0 * ds.head;
        Row<DT> ng = load_row<DT>(gp, w.a, w.b), nx = ng;  // the next row, on its way
        if (norm) nx = load_row<DT>(xp, w.a, w.b);
        float c[8], s[8];
        angles<DT>(p, w, position(p, it), c, s);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = -s[e];  // the transpose
        for (int j = 0; j < n; ++j) {
            const Row<DT> vg = ng, vx = nx;
            if (j + 1 < n) {
                ng = load_row<DT>(gp + (j + 1) * gs.head, w.a, w.b);
                if (norm) nx = load_row<DT>(xp + (j + 1) * xs.head, w.a, w.b);
            }
            float g[16];
            widen<DT>(vg, g);
            rotate(w, c, s, g);
            if (norm) {  // with t = r g' x: dw += t, dx = r w g' - x r^2 mean(w t)
                float x[16], ss = 0.f, dot = 0.f;
                widen<DT>(vx, x);
#pragma unroll
                for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
                const float r = rsqrtf(w.sum(w.active ? ss : 0.f) * p.inv_d + p.eps);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float t = g[e] * (x[e] * r);
                    acc[e] += t;
                    dot = fmaf(t, wt[e], dot);
                }
                const float k = -(w.sum(w.active ? dot : 0.f) * p.inv_d) * r * r;
#pragma unroll
                for (int e = 0; e < 16; ++e) g[e] = fmaf(x[e], k, g[e] * (wt[e] * r));
            }
            if (w.active) store_row<DT>(dp + j * ds.head, w.a, w.b, narrow<DT>(g));
        }
    }
    if (!norm) return;
    if (w.active) {
#pragma unroll
        for (int e = 0; e < 16; ++e) red[w.grp][e < 8 ? w.a + e : w.b + e - 8] = acc[e];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.d; c += THREADS) {
        float t = 0.f;
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) t += red[gi][c];
        p.partial[static_cast<size_t>(blockIdx.x) * p.d + c] = t;
    }
}

// dw = sum of the CTAs' partial rows (rows 0 .. q_rows - 1: the queries', the others the keys'): 32
// columns by 32 row lanes a CTA, the lanes added in order.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float *partial, int32_t q_rows, int32_t rows, int32_t d, float *dwq, float *dwk)
{
    __shared__ float red[32][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), lane = threadIdx.x >> 5, lo = blockIdx.y ? q_rows : 0, hi = blockIdx.y ? rows : q_rows;
    float s = 0.f;
    if (c < d)
#pragma unroll 8
        for (int r = lo + lane; r < hi; r += 32) s += partial[static_cast<size_t>(r) * d + c];
    red[lane][threadIdx.x & 31] = s;
    __syncthreads();
    if (lane == 0 && c < d) {
        s = 0.f;
        for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
        (blockIdx.y ? dwk : dwq)[c] = s;
    }
}

template <int DT, int L>
cudaError_t launch_l(const RopeParams &p, int mode, int64_t grid, cudaStream_t s)
{
    const unsigned g = static_cast<unsigned>(grid);
    if (mode == ROPE_FWD) rope_fwd_kernel<DT, L, false><<<g, FWD_THREADS, 0, s>>>(p);
    else if (mode == ROPE_APPEND) rope_fwd_kernel<DT, L, true><<<g, FWD_THREADS, 0, s>>>(p);
    else rope_bwd_kernel<DT, L><<<g, THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

template <int DT>
cudaError_t launch_t(const RopeParams &p, int mode, int64_t grid, cudaStream_t s)
{
    if (p.d <= 32) return launch_l<DT, 2>(p, mode, grid, s);
    if (p.d <= 64) return launch_l<DT, 4>(p, mode, grid, s);
    if (p.d <= 128) return launch_l<DT, 8>(p, mode, grid, s);
    return launch_l<DT, 16>(p, mode, grid, s);
}

// Lanes a row.
int lanes_of(int d) { return d <= 32 ? 2 : (d <= 64 ? 4 : (d <= 128 ? 8 : 16)); }

// How tokens of `rows` head rows are dealt out: the first `whole` to a group each, of the others `run`
// rows a group.
struct RopeSplit {
    int64_t whole;
    int32_t run, parts;
    int64_t items;
};

// Runs of the `tokens` tokens, `parts` of them each or fewer; never fewer than U rows.
RopeSplit split_runs(int64_t whole, int64_t tokens, int64_t parts, int rows)
{
    RopeSplit s;
    const int64_t most = (rows + U - 1) / U;
    if (parts > most) parts = most;
    s.whole = whole;
    s.run = static_cast<int>((rows + parts - 1) / parts + U - 1) / U * U;
    s.parts = (rows + s.run - 1) / s.run;
    s.items = whole + tokens * s.parts;
    return s;
}

// A group has its angles to compute and its weights to load first, so tokens stay whole as long as
// they fill the SMs (4 CTAs each), and what is left over is cut into as many runs as still fit on them
// at once.  (Append of 8192 tokens, 9472 groups fit: whole 41 us, in two runs 55; 10000 tokens whole 62.)
RopeSplit fwd_split(int64_t tokens, int rows, int d)
{
    const int64_t fit = 4ll * sm_count() * FWD_THREADS / lanes_of(d), rest = tokens % fit;
    return split_runs(tokens - rest, rest, rest ? fit / rest : 1, rows);
}

// The backward's groups walk; its runs are as many as the SMs hold groups at a time or some more (768
// threads).
RopeSplit bwd_split(int64_t tokens, int rows, int d)
{
    const int64_t groups = 768ll * sm_count() / lanes_of(d);
    return split_runs(0, tokens, (groups + tokens - 1) / tokens, rows);
}

int64_t ctas_of(const RopeSplit &s, int threads, int d)
{
    const int per = threads / lanes_of(d);
    return (s.items + per - 1) / per;
}

}  // namespace

RopeCtas rope_bwd_ctas(int64_t tokens, int heads, int kv, int d)
{
    // Two CTAs an SM that walk, or fewer where the rows run out, dealt out by the rows of each kind.
    const int64_t q = ctas_of(bwd_split(tokens, heads, d), THREADS, d), k = ctas_of(bwd_split(tokens, kv, d), THREADS, d);
    const int64_t cap = 2ll * sm_count(), share = (cap * kv + (heads + kv) / 2) / (heads + kv);
    const int64_t kc = share < 1 ? 1 : (share > cap - 1 ? cap - 1 : share);
    return {q < cap - kc ? q : cap - kc, k < kc ? k : kc};
}

cudaError_t launch_rope(RopeParams &p, int dtype, int mode, float *dwq, float *dwk, cudaStream_t s)
{
    const int64_t tokens = p.batch * p.n;
    const bool bwd = mode == ROPE_BWD;
    const RopeSplit r = bwd ? bwd_split(tokens, p.heads, p.d)
                            : fwd_split(tokens, p.heads + p.kv + (mode == ROPE_APPEND ? p.kv : 0), p.d);
    p.tokens0 = r.whole;
    p.run = r.run;
    p.parts = r.parts;
    p.items = r.items;
    int64_t ctas = ctas_of(r, FWD_THREADS, p.d);
    if (bwd) {
        const RopeSplit k = bwd_split(tokens, p.kv, p.d);
        p.run_k = k.run;
        p.parts_k = k.parts;
        p.items_k = k.items;
        const RopeCtas c = rope_bwd_ctas(tokens, p.heads, p.kv, p.d);
        p.q_ctas = static_cast<int32_t>(c.q);
        ctas = c.q + c.k;
    }
    cudaError_t e = dtype == ST_BF16   ? launch_t<ST_BF16>(p, mode, ctas, s)
                    : dtype == ST_FP16 ? launch_t<ST_FP16>(p, mode, ctas, s)
                                       : launch_t<ST_FP32>(p, mode, ctas, s);
    if (e != cudaSuccess || !bwd || !p.wq) return e;
    rope_dw_kernel<<<dim3((p.d + 31) / 32, 2), 1024, 0, s>>>(p.partial, p.q_ctas, static_cast<int32_t>(ctas), p.d, dwq, dwk);
    return cudaGetLastError();
}

}  // namespace st
