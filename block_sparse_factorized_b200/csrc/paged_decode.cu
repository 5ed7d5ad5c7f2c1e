// paged_decode.cu -- attention of one new token per request over a paged key/value cache, with a
// sliding window and sinks.
//
//   O = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j - m),  s_j = q . k_j log2(e) / sqrt(d)
// over the keys j < len with j >= len - window or j < sinks; parts of a row join by
//   m = max m_c,  L = sum 2^(m_c - m) L_c,  O = sum 2^(m_c - m) O_c / L.
//
// Bound by memory: each key and value row is read once for up to 16 query heads that share it (a larger
// group G in blocks of 16 heads, each with its own read), about 2 G multiply-adds per byte, more than the FMA
// pipes do at the memory's rate from G = 4 on, so both products run on the tensor cores (mma.sync m16n8k16:
// the operands are a row block of at most 16 heads, held in registers, and a 16-key tile straight from
// memory; the tcgen05 forms want 64 or 128 rows, most of them empty here).
//   - No shared memory on the way: the order of a contraction is free, so a lane's 16-byte load of a
//     key row (elements 8c .. 8c + 7 of each 32, c = lane % 4) is the B operand of two K = 16 steps,
//     with the query's fragments laid out alike; a lane's 16-byte loads of value rows 2c, 2c + 1,
//     2c + 8, 2c + 9 become B operands by interleaving halves, column n of step j being element
//     8n + j.  16 loads of 16 bytes a lane are in flight before the first product.
//   - One launch splits everything evenly: with tiles of 16 keys numbered request by request, key
//     head by key head, each CTA takes an equal run of them, whatever the lengths are; rows that
//     cross CTAs leave (m, L, O) parts, which a second, overlapped launch joins in order.
//   - With bf16 and at most 8 heads P goes in as two 16-bit parts (hi + lo, 16 bits of mantissa
//     together), the second in the rows 8 .. 15 that would be empty; rounding it to 8 bits would cost
//     as much accuracy as the output's own rounding.  With more heads it is rounded to 8 bits (a second
//     product would cost 13% of the kernel's time), and fp16's 11 bits are kept as they are.  Measured
//     over 2000 keys, relative to exact results: 8 heads 0.00160, the output's own rounding; 16 heads
//     0.00174, of which 0.00169 is that rounding.
// Measured, bf16, d = 128, 32 heads on 8 (of 6549 GB/s for a copy): one request of 131072 keys (537 MB)
// 99 us, 5.4 TB/s; 200 requests of 1 .. 12288 keys behind a window of 4096 (2.8 GB) 470 to 490 us, 5.9 TB/s.
// One request of 131072 keys on one key head (67 MB): 8 heads 63 us, 16 heads 67, 64 heads 73.
#include "elem.cuh"
#include "kernels.h"
#include "lm.h"
#include "paged_decode.h"
#include "sm100.cuh"
#include "tiles.cuh"

namespace st {
namespace {

constexpr int WARPS = 4, THREADS = 32 * WARPS;
constexpr int MIN_TILES = 2 * WARPS;  // tiles a CTA takes at least

// The keys of one request: tiles 0 .. ns - 1 (sinks), then tiles b0 .. of 16 keys.
struct Span {
    int32_t len, lo;  // keys lo .. len - 1 are in the window
    int32_t ns, b0, nt;
};

__device__ __forceinline__ Span span_of(const PagedParams &p, int r)
{
    Span s;
    const int32_t len = min(max(p.lens[r], 0), p.capacity);
    s.len = len;
    s.lo = p.window && len > p.window ? len - p.window : 0;
    s.b0 = s.lo / PD_TILE;
    s.ns = min((min(p.sinks, s.lo) + PD_TILE - 1) / PD_TILE, s.b0);
    s.nt = len > 0 ? s.ns + (len + PD_TILE - 1) / PD_TILE - s.b0 : 0;
    return s;
}

// The request whose run of tiles holds x: the last r with first[r] <= x (runs may be empty).
__device__ __forceinline__ int find(const int32_t *first, int n, int64_t x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Tiles a CTA takes, of `all` in the grid.
__device__ __forceinline__ int64_t share_of(int64_t all, int32_t grid)
{
    const int64_t per = (all + grid - 1) / grid;
    return per < MIN_TILES ? MIN_TILES : per;
}

template <int DT>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    if constexpr (DT == ST_BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// HB heads of a row block: 8 (rows 8 .. 15 of the product stay zero) or 16.
template <int DT, int D, int HB>
__global__ void __launch_bounds__(THREADS, PD_CTAS_PER_SM) paged_kernel(const __grid_constant__ PagedParams p)
{
    constexpr int RW = HB / 8;        // rows of the product a lane holds
    constexpr int KC = D / 32;        // 16-byte chunks of a key row a lane loads
    constexpr int VB = D / 64;        // 64-element blocks of a value row
    constexpr int PART = HB * (D + 2);
    extern __shared__ int32_t prefix[];  // [requests + 1]
    __shared__ float red_o[WARPS][HB][D + 4];
    __shared__ float red_m[WARPS][HB], red_l[WARPS][HB];
    __shared__ int32_t sums[WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int R = p.requests;
    // tiles before each request: every thread sums a run of requests, then the runs are scanned
    const int per_thread = (R + THREADS - 1) / THREADS, r0 = threadIdx.x * per_thread, r1 = min(R, r0 + per_thread);
    int32_t mine = 0;
    for (int r = r0; r < r1; ++r) mine += span_of(p, r).nt;
    int32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int32_t at = incl - mine;
    for (int w = 0; w < warp; ++w) at += sums[w];
    for (int r = r0; r < r1; ++r) {
        prefix[r] = at;
        if (blockIdx.x == 0) p.prefix[r] = at;
        at += span_of(p, r).nt;
    }
    if (r0 < R && r1 == R) {
        prefix[R] = at;
        if (blockIdx.x == 0) p.prefix[R] = at;
    }
    __syncthreads();
    // the joining launch may start setting up; it waits for this one's memory before it reads
    asm volatile("griddepcontrol.launch_dependents;");
    const int rows_per = p.kv * p.blocks;  // rows (key head, head block) of one request
    const int64_t all = static_cast<int64_t>(prefix[R]) * rows_per;
    const int64_t per = share_of(all, p.grid), t0 = per * blockIdx.x, t1 = min(all, t0 + per);

    // requests without keys: O = 0, lse = -inf
    for (int r = blockIdx.x; r < R; r += gridDim.x) {
        if (prefix[r + 1] != prefix[r]) continue;
        uint32_t *o = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.o) + static_cast<int64_t>(r) * p.heads * D);
        for (int i = threadIdx.x; i < p.heads * (D / 2); i += THREADS) o[i] = 0u;
        for (int i = threadIdx.x; i < p.heads; i += THREADS) p.lse[static_cast<int64_t>(r) * p.heads + i] = -INFINITY;
    }

    for (int64_t t = t0; t < t1;) {
        const int r = find(prefix, R, t / rows_per);
        const Span sp = span_of(p, r);
        const int64_t before = static_cast<int64_t>(prefix[r]) * rows_per;
        const int row = static_cast<int>((t - before) / sp.nt);  // (key head, head block) of the request
        const int64_t row0 = before + static_cast<int64_t>(row) * sp.nt;
        const int ta = static_cast<int>(t - row0), tb = static_cast<int>(min(static_cast<int64_t>(sp.nt), t1 - row0));
        const int hk = row / p.blocks, hb = row - hk * p.blocks;
        const int nh = min(HB, p.group - hb * HB);  // heads of this block
        const int64_t qrow = static_cast<int64_t>(r) * p.heads + hk * p.group + hb * HB;

        uint4 qf[RW][KC];
#pragma unroll
        for (int i = 0; i < RW; ++i)
#pragma unroll
            for (int k = 0; k < KC; ++k) {
                qf[i][k] = make_uint4(0u, 0u, 0u, 0u);
                if (g + 8 * i < nh)
                    qf[i][k] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + (qrow + g + 8 * i) * D + 32 * k + 8 * c);
            }
        float o[VB * 8][RW == 1 ? 2 : 4], m[RW], l[RW];
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < VB * 8; ++j)
#pragma unroll
            for (int e = 0; e < (RW == 1 ? 2 : 4); ++e) o[j][e] = 0.f;

        const char *kh = p.k + hk * p.k_head, *vh = p.v + hk * p.v_head;
        const int32_t *table = p.table + r * p.table_stride;
        // first key of a tile, and its page
        auto key_of = [&](int tile) { return (tile < sp.ns ? tile : sp.b0 + tile - sp.ns) * PD_TILE; };
        auto page_of = [&](int tile) { return static_cast<uint32_t>(key_of(tile)) / static_cast<uint32_t>(p.page_size); };
        int tile = ta + warp;
        int32_t next_page = tile < tb ? table[page_of(tile)] : 0;
        for (; tile < tb; tile += WARPS) {
            const int32_t key0 = key_of(tile);
            const int32_t page = next_page;
            if (tile + WARPS < tb) next_page = table[page_of(tile + WARPS)];
            if (page < 0 || page >= p.num_pages) {  // not seen
                if (lane == 0) atomicOr(p.err, ERR_PAGE);
                continue;
            }
            const int64_t at0 = static_cast<uint32_t>(key0) % static_cast<uint32_t>(p.page_size);
            uint4 kf[2][KC], vf[VB][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const char *src = kh + page * p.k_page + (at0 + 8 * n + g) * p.k_row + 16 * c;
#pragma unroll
                for (int k = 0; k < KC; ++k) kf[n][k] = __ldg(reinterpret_cast<const uint4 *>(src + 64 * k));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const char *src = vh + page * p.v_page + (at0 + 2 * c + (e & 1) + 8 * (e >> 1)) * p.v_row + 16 * g;
#pragma unroll
                for (int b = 0; b < VB; ++b) vf[b][e] = __ldg(reinterpret_cast<const uint4 *>(src + 128 * b));
            }
            // S: rows are heads, columns keys 2c, 2c + 1 of each of the tile's halves
            float s[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
                for (int k = 0; k < KC; ++k) {
                    const uint4 a = qf[0][k], x = RW > 1 ? qf[RW - 1][k] : make_uint4(0u, 0u, 0u, 0u);
                    mma<DT>(s[n], a.x, x.x, a.y, x.y, kf[n][k].x, kf[n][k].y);
                    mma<DT>(s[n], a.z, x.z, a.w, x.w, kf[n][k].z, kf[n][k].w);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] *= p.scale_log2;
            }
            // a tile that the window, the sinks or the length cut: keys not seen get -inf, and their
            // value rows are dropped (a zero weight would not silence a NaN)
            const bool whole = key0 + PD_TILE <= sp.len && (key0 >= sp.lo || key0 + PD_TILE <= p.sinks);
            if (!whole) {
                auto seen = [&](int e) {
                    const int32_t key = key0 + 2 * c + (e & 1) + 8 * (e >> 1);
                    return key < sp.len && (key >= sp.lo || key < p.sinks);
                };
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (seen(e)) continue;
                    s[e >> 1][e & 1] = -INFINITY;
                    s[e >> 1][2 + (e & 1)] = -INFINITY;
#pragma unroll
                    for (int b = 0; b < VB; ++b) vf[b][e] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
            uint32_t hi[RW][2], lo[RW][2];
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                float mt = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
                mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
                mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
                const float mn = fmaxf(m[i], mt);
                const float base = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: all weights 0
                const float alpha = ex2(m[i] - base);
                m[i] = mn;
                l[i] *= alpha;
#pragma unroll
                for (int j = 0; j < VB * 8; ++j) {
                    o[j][2 * i] *= alpha;
                    o[j][2 * i + 1] *= alpha;
                }
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float p0 = ex2(s[n][2 * i] - base), p1 = ex2(s[n][2 * i + 1] - base);
                    l[i] += p0 + p1;
                    hi[i][n] = pack16<DT>(p0, p1);
                    if constexpr (DT == ST_BF16 && RW == 1) lo[i][n] = pack16<DT>(p0 - bf16_lo(hi[i][n]), p1 - bf16_hi(hi[i][n]));
                }
            }
            // O += P V: value column 8n + j of each 64 in step j
#pragma unroll
            for (int b = 0; b < VB; ++b)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    auto word = [&](const uint4 &x) { return j < 2 ? x.x : (j < 4 ? x.y : (j < 6 ? x.z : x.w)); };
                    const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
                    const uint32_t b0 = __byte_perm(word(vf[b][0]), word(vf[b][1]), sel), b1 = __byte_perm(word(vf[b][2]), word(vf[b][3]), sel);
                    if constexpr (RW == 1) {
                        float acc[4] = {o[b * 8 + j][0], o[b * 8 + j][1], 0.f, 0.f};
                        if constexpr (DT == ST_BF16) {  // rows 8 .. 15: the low parts of the same heads
                            mma<DT>(acc, hi[0][0], lo[0][0], hi[0][1], lo[0][1], b0, b1);
                            o[b * 8 + j][0] = acc[0] + acc[2];
                            o[b * 8 + j][1] = acc[1] + acc[3];
                        } else {
                            mma<DT>(acc, hi[0][0], 0u, hi[0][1], 0u, b0, b1);
                            o[b * 8 + j][0] = acc[0];
                            o[b * 8 + j][1] = acc[1];
                        }
                    } else {
                        mma<DT>(o[b * 8 + j], hi[0][0], hi[RW - 1][0], hi[0][1], hi[RW - 1][1], b0, b1);
                    }
                }
        }
        // the warps' parts of this run, joined in warp order
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            if (c == 0) {
                red_m[warp][g + 8 * i] = m[i];
                red_l[warp][g + 8 * i] = l[i];
            }
#pragma unroll
            for (int b = 0; b < VB; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float4 *dst = reinterpret_cast<float4 *>(&red_o[warp][g + 8 * i][64 * b + 16 * c + 8 * e]);
                    dst[0] = make_float4(o[b * 8][2 * i + e], o[b * 8 + 1][2 * i + e], o[b * 8 + 2][2 * i + e], o[b * 8 + 3][2 * i + e]);
                    dst[1] = make_float4(o[b * 8 + 4][2 * i + e], o[b * 8 + 5][2 * i + e], o[b * 8 + 6][2 * i + e], o[b * 8 + 7][2 * i + e]);
                }
        }
        __syncthreads();
        const bool full = ta == 0 && tb == sp.nt;
        float *part = p.parts + (2 * static_cast<int64_t>(blockIdx.x) + (t == t0 ? 0 : 1)) * PART;
        for (int i = threadIdx.x; i < nh * (D / 2); i += THREADS) {
            const int h = i / (D / 2), x = 2 * (i - h * (D / 2));
            float mx = red_m[0][h];
#pragma unroll
            for (int w = 1; w < WARPS; ++w) mx = fmaxf(mx, red_m[w][h]);
            const float base = mx == -INFINITY ? 0.f : mx;
            float sum = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float f = ex2(red_m[w][h] - base);
                sum = fmaf(f, red_l[w][h], sum);
                o0 = fmaf(f, red_o[w][h][x], o0);
                o1 = fmaf(f, red_o[w][h][x + 1], o1);
            }
            if (full) {
                const bool none = sum == 0.f;  // nothing seen; a NaN, from a score that is one or +inf, goes through
                const float inv = none ? 0.f : 1.f / sum;
                reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.o) + (qrow + h) * D)[x / 2] = pack16<DT>(o0 * inv, o1 * inv);
                if (x == 0) p.lse[qrow + h] = none ? -INFINITY : (mx + lg2(sum)) * LN2;
            } else {
                *reinterpret_cast<float2 *>(part + 2 * HB + h * D + x) = make_float2(o0, o1);
                if (x == 0) {
                    part[h] = mx;
                    part[HB + h] = sum;
                }
            }
        }
        __syncthreads();  // red_* is reused by the next run
        t = row0 + tb;
    }
}

// Join the parts of the row that CTA blockIdx.x + 1's first tile lies inside, if no earlier CTA's
// first tile does.  blockIdx.y: head of the block.  The parts' weights first, one a thread, then their
// O in groups of D / 2 threads (two elements each), the groups' sums added in order.
constexpr int JOIN_THREADS = 256;

template <int DT, int D, int HB>
__global__ void __launch_bounds__(JOIN_THREADS) paged_join_kernel(const __grid_constant__ PagedParams p)
{
    constexpr int PART = HB * (D + 2), NG = JOIN_THREADS / (D / 2);
    __shared__ float weight[PD_MAX_GRID];
    __shared__ float red[JOIN_THREADS / 32], sum_o[NG][D + 2];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int R = p.requests, rows_per = p.kv * p.blocks;
    const int64_t all = static_cast<int64_t>(p.prefix[R]) * rows_per, per = share_of(all, p.grid);
    const int64_t cut = per * (blockIdx.x + 1);
    if (cut >= all) return;
    const int r = find(p.prefix, R, cut / rows_per);
    const int64_t before = static_cast<int64_t>(p.prefix[r]) * rows_per;
    const int64_t nt = p.prefix[r + 1] - p.prefix[r];
    const int row = static_cast<int>((cut - before) / nt);
    const int64_t row0 = before + row * nt, end = row0 + nt;
    if (cut == row0 || cut - per > row0) return;  // a row's first tile, or an earlier CTA's row
    const int hk = row / p.blocks, hb = row - hk * p.blocks, h = blockIdx.y;
    if (h >= min(HB, p.group - hb * HB)) return;
    // CTAs c0 .. c0 + n - 1 hold the row's parts; a CTA's is its first (slot 0) where the row covers the
    // CTA's first tile
    const int64_t c0 = row0 / per;
    const int n = static_cast<int>((end - 1) / per - c0) + 1;
    auto part_of = [&](int i) { return p.parts + (2 * (c0 + i) + ((c0 + i) * per >= row0 ? 0 : 1)) * PART; };
    auto block_reduce = [&](float x, bool max) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float y = __shfl_xor_sync(0xffffffffu, x, o);
            x = max ? fmaxf(x, y) : x + y;
        }
        __syncthreads();
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
        __syncthreads();
        x = red[0];
        for (int w = 1; w < JOIN_THREADS / 32; ++w) x = max ? fmaxf(x, red[w]) : x + red[w];
        return x;
    };
    float m = -INFINITY;
    for (int i = threadIdx.x; i < n; i += JOIN_THREADS) {
        weight[i] = part_of(i)[h];
        m = fmaxf(m, weight[i]);
    }
    m = block_reduce(m, true);
    const float base = m == -INFINITY ? 0.f : m;
    float sum = 0.f;
    for (int i = threadIdx.x; i < n; i += JOIN_THREADS) {
        weight[i] = ex2(weight[i] - base);
        sum = fmaf(weight[i], part_of(i)[HB + h], sum);
    }
    sum = block_reduce(sum, false);  // (also: every weight is written)
    const int grp = threadIdx.x / (D / 2), x = 2 * (threadIdx.x % (D / 2));
    float o0 = 0.f, o1 = 0.f;
#pragma unroll 4
    for (int i = grp; i < n; i += NG) {
        const float2 o = *reinterpret_cast<const float2 *>(part_of(i) + 2 * HB + h * D + x);
        o0 = fmaf(weight[i], o.x, o0);
        o1 = fmaf(weight[i], o.y, o1);
    }
    sum_o[grp][x] = o0;
    sum_o[grp][x + 1] = o1;
    __syncthreads();
    if (grp != 0) return;
    for (int i = 1; i < NG; ++i) {
        o0 += sum_o[i][x];
        o1 += sum_o[i][x + 1];
    }
    const int64_t q = static_cast<int64_t>(r) * p.heads + hk * p.group + hb * HB + h;
    const bool none = sum == 0.f;
    const float inv = none ? 0.f : 1.f / sum;
    reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.o) + q * D)[x / 2] = pack16<DT>(o0 * inv, o1 * inv);
    if (x == 0) p.lse[q] = none ? -INFINITY : (m + lg2(sum)) * LN2;
}

template <int DT, int D, int HB>
cudaError_t launch_h(const PagedParams &p, cudaStream_t s)
{
    const int smem = 4 * (p.requests + 1);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(paged_kernel<DT, D, HB>, 4 * (PD_MAX_REQUESTS + 1), done);
    if (e != cudaSuccess) return e;
    paged_kernel<DT, D, HB><<<static_cast<unsigned>(p.grid), THREADS, smem, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (p.grid == 1) return cudaSuccess;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.grid - 1), static_cast<unsigned>(p.group < HB ? p.group : HB));
    cfg.blockDim = dim3(JOIN_THREADS);
    cfg.stream = s;
    cudaLaunchAttribute a{};
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &a;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_join_kernel<DT, D, HB>, p);
}

template <int DT, int D>
cudaError_t launch_d(const PagedParams &p, cudaStream_t s)
{
    return p.group <= 8 ? launch_h<DT, D, 8>(p, s) : launch_h<DT, D, 16>(p, s);
}

}  // namespace

cudaError_t launch_paged_decode(const PagedParams &p, int dtype, int d, cudaStream_t s)
{
    if (dtype == ST_BF16) return d == 64 ? launch_d<ST_BF16, 64>(p, s) : launch_d<ST_BF16, 128>(p, s);
    return d == 64 ? launch_d<ST_FP16, 64>(p, s) : launch_d<ST_FP16, 128>(p, s);
}

}  // namespace st
