// window_bwd.cu -- backward pass of attention with a sliding window and sinks on sm_100a.
//
// With P_ij = exp(q_i . k_j / sqrt d - lse_i) over the allowed pairs and D_i = dO_i . O_i:
//   dV_j = sum_i P_ij dO_i,  dS_ij = P_ij (dO_i . v_j - D_i) / sqrt d,
//   dK_j = sum_i dS_ij q_i,  dQ_i = sum_j dS_ij k_j.
// Two kernels, each owning what it sums (no atomics: the order of every sum is fixed, and no fp32
// accumulator in memory), at the price of recomputing S and dP once more (7 products in place of 5):
//   dk_dv  a unit is a tile of 128 keys (of a key head) and a run of (query tile, head of the group)
//          steps.  All four products are transposed, keys as rows: S^T = K Q^T and dP^T = V dO^T,
//          then dV += P^T dO and dK += dS^T Q with P^T and dS^T read from TMEM, where they overwrite
//          S^T and dP^T -- nothing but the tiles themselves goes through shared memory.
//   dq     a unit is a query tile of one head: S = Q K^T, dP = dO V^T, dQ += dS K, dS in TMEM.
// A key tile that very many query tiles read (a sink; early keys without a window) is cut into
// chunks whose fp32 partial sums a third launch adds in order.
//
// One CTA an SM, persistent: a producer warp (TMA), a warp that issues the products, two softmax
// warpgroups with 64 columns each.  The issuing warp walks its steps as a whole and an elected lane issues
// (dk_dv 447 us; a loop of one lane, whose branches depend on loaded values, 489).
//
// Measured, bf16, n = 12288, 2 x 16 heads on 4, window 1024, 16 sinks (10 d operations a pair, of 1616
// TFLOP/s for a library product):
//   d 128   841 us, 596 TFLOP/s: preparation 43, dk_dv 460, dq 392 (partly beside dk_dv), join 6
//   d 64    644 us, 389 TFLOP/s: preparation 23, dk_dv 360, dq 308, join 5
// and 1 x 16 heads over the whole past at d 128: 1832 us, 844 TFLOP/s.  Bound by the chains of a step: at
// d = 128 a step of dk_dv takes 3400 cycles for 2048 of products (the tensor pipe is 56% busy, shared
// memory's 57%): S, dP, dV and dK fill TMEM, so S^T of the next step waits for dV, which reads P from its
// columns.  One of dq takes 2850 for 1536; at d = 64 the softmax warps take longer than the products.
// A tile of sinks is a whole step for its few live keys: in turns on a warm card 861 us with 16 sinks and
// 778 without (d 64: 654, 589); 4 x 8 heads on 2 of 4096 rows, d 64, window 256: 130 with 4 sinks, 103 without.
//
// fp16 has a narrow range: P is kept 2^14 larger, and dS scaled by a power of two per (batch, key
// head) from the bound |dS| <= 2 max|dO_i| max|v_j| / sqrt d, so that neither overflows nor fades; the
// results are scaled back in fp32.
#include "kernels.h"
#include "lm.h"
#include "window_tiles.cuh"

namespace st {
namespace {

constexpr int THREADS = 384;   // producer, MMA issuer, 2 warps for zeros, then two softmax warpgroups
constexpr int NSM = 256;       // softmax threads: warpgroup w owns columns 64 w .. of a score tile

template <int DT>
constexpr float PBIAS = DT == ST_FP16 ? 14.f : 0.f;  // log2 of the factor on P

// The factor on dS (a power of two) of batch element b, key head hk.
template <int DT>
__device__ __forceinline__ float ds_factor(const WindowBwdParams &p, int32_t b, int32_t hk)
{
    if constexpr (DT == ST_BF16) return 1.f;
    const uint32_t *most = p.maxima + 2 * (b * p.g.kv + hk);
    const float a = __uint_as_float(__ldcg(most)), v = __uint_as_float(__ldcg(most + 1));
    const float bound = 2.f * p.g.scale * sqrtf(a) * sqrtf(v);
    if (!(bound > 0.f) || !isfinite(bound)) return 1.f;
    const int e = ilogbf(32768.f / bound);
    return ldexpf(1.f, e < -100 ? -100 : (e > 100 ? 100 : e));
}

// dq runs beside dk_dv and so cannot wait for the grids before it by griddepcontrol.wait, which would
// wait for dk_dv's end.  What the preparation wrote reaches it through a word instead: dk_dv has waited
// for the preparation, and releases the word; a thread of each of dq's CTAs acquires it, so that all
// that dk_dv saw by then, that CTA sees.  The preparation clears the word; dq's CTAs start after dk_dv's
// first have let them, so the wait is short.
__device__ __forceinline__ void publish(int32_t *word)
{
    asm volatile("st.release.gpu.global.s32 [%0], 1;" ::"l"(word) : "memory");
}

__device__ __forceinline__ bool await_published(const int32_t *word, int32_t *err)
{
    const uint64_t t0 = globaltimer();
    for (;;) {
        int32_t x;
        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(x) : "l"(word) : "memory");
        if (x != 0) return true;
        if (globaltimer() - t0 > WAIT_NS) {
            atomicOr(err, ERR_TIMEOUT);
            return false;
        }
    }
}

// Chunks of key tile t, and the steps (query tile, head) of it.
__device__ __forceinline__ int32_t tile_steps(const WindowGeom &g, int32_t t, int32_t &i0)
{
    int32_t i1;
    query_range(g, t, i0, i1);
    return i1 < i0 ? 0 : (i1 - i0 + 1) * g.group;
}

// Units with steps are taken from a counter as CTAs come to need them, so that a padded batch, whose
// units differ by what its lengths leave, spreads evenly; which CTA takes a unit changes no sum.  The
// producer takes them and hands them on through a small ring.  Units
// without steps never enter the ring (the issuer looks one unit ahead and must not wait for one that
// is behind several that it does nothing for): two warps that have nothing else to do write their zeros.
constexpr int NU = 4;

template <typename Unit>
struct UnitRing {
    uint64_t full[NU], empty[NU];
    Unit unit[NU];
    int32_t steps[NU];  // 0: the end

    __device__ void init()
    {
        for (int i = 0; i < NU; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1 + NSM / 32);  // the issuer and each softmax warp
        }
    }

    // The producer warp's k-th unit (false: the last was the end, or a wait ran out).  taken: whether
    // the CTA has had its first number, which is its own.
    __device__ bool put(const WindowBwdParams &p, int32_t *counter, int32_t k, bool &taken, Unit &U, volatile int32_t *abort, int32_t *err)
    {
        bool more;
        do {
            int64_t at = blockIdx.x;
            if (taken) {
                int32_t n = (threadIdx.x & 31) == 0 ? atomicAdd(counter, 1) : 0;
                at = static_cast<int64_t>(gridDim.x) + __shfl_sync(0xffffffffu, n, 0);
            }
            taken = true;
            more = get_unit(p, at, U);
        } while (more && U.steps() == 0);
        if (k >= NU && !__all_sync(0xffffffffu, mbar_wait(&empty[k % NU], (k / NU - 1) & 1, abort, err))) return false;
        if ((threadIdx.x & 31) == 0) {
            unit[k % NU] = U;
            steps[k % NU] = more ? U.steps() : 0;
            mbar_arrive(&full[k % NU]);
        }
        __syncwarp();
        return more;
    }

    // The k-th unit for a softmax warp.
    __device__ bool take(int32_t k, Unit &U, volatile int32_t *abort, int32_t *err)
    {
        if (!__all_sync(0xffffffffu, mbar_wait(&full[k % NU], (k / NU) & 1, abort, err))) return false;
        U = unit[k % NU];
        const bool more = steps[k % NU] != 0;
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[k % NU]);
        return more;
    }

    // The k-th unit's steps for the issuer warp, 0 at the end.  The reduction puts the number where the
    // compiler knows it to be the same for the warp.
    __device__ int32_t take_steps(int32_t k, volatile int32_t *abort, int32_t *err)
    {
        if (!__all_sync(0xffffffffu, mbar_wait(&full[k % NU], (k / NU) & 1, abort, err))) return 0;
        const int32_t n = static_cast<int32_t>(__reduce_max_sync(0xffffffffu, static_cast<uint32_t>(steps[k % NU])));
        if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[k % NU]);
        return n;
    }
};

// ---- preparation ------------------------------------------------------------------------------
// D_i (0 for padding rows), the unit list of dk_dv (block 0: the chunked key tiles first), and for fp16 the largest squared norms
// of live dO and V rows.  D / 8 lanes a row; memory-bound.
constexpr int PRE_ROWS = 256;

template <int DT, int D>
__global__ void __launch_bounds__(256) window_pre_kernel(const __grid_constant__ WindowBwdParams p)
{
    constexpr int L = D / 8, NG = 256 / L;
    const WindowGeom &g = p.g;
    asm volatile("griddepcontrol.launch_dependents;");
    if (blockIdx.x == 0) {  // 256 tiles at a time
        if (threadIdx.x < 3) p.counters[threadIdx.x] = 0;
        __shared__ int2 sums[8];
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        int32_t split = 0, plain = p.nsplit;  // next entry of a chunked tile, of another
        for (int32_t base = 0; base < g.nkt; base += 256) {
            const int32_t t = base + threadIdx.x;
            int32_t i0, c = 0;
            if (t < g.nkt) c = chunks_of(tile_steps(g, t, i0), p.chunk);
            int32_t x = c > 1 ? c : 0, y = c == 1 ? 1 : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
                if (lane >= o) {
                    x += u;
                    y += v;
                }
            }
            if (lane == 31) sums[warp] = make_int2(x, y);
            __syncthreads();
            int32_t at = c > 1 ? split + x - c : plain + y - 1;
            for (int w = 0; w < 8; ++w) {
                if (w < warp) at += c > 1 ? sums[w].x : sums[w].y;
                split += sums[w].x;
                plain += sums[w].y;
            }
            for (int32_t i = 0; i < c; ++i) p.entries[at + i] = make_int2(t, i);
            __syncthreads();
        }
        return;
    }
    // 256 rows of one (batch, head) of dO and O, or of one (batch, key head) of V, a CTA
    const int l = threadIdx.x % L, grp = threadIdx.x / L;
    const int32_t qc = (g.nq + PRE_ROWS - 1) / PRE_ROWS, vc = (g.nk + PRE_ROWS - 1) / PRE_ROWS;
    int64_t i = blockIdx.x - 1;
    const bool is_v = i >= static_cast<int64_t>(g.batch) * g.heads * qc;
    if (is_v) i -= static_cast<int64_t>(g.batch) * g.heads * qc;
    const int32_t per = is_v ? vc : qc, heads = is_v ? g.kv : g.heads, n = is_v ? g.nk : g.nq;
    const int32_t bh = static_cast<int32_t>(i / per), row0 = static_cast<int32_t>(i - static_cast<int64_t>(bh) * per) * PRE_ROWS;
    const int32_t b = bh / heads, h = bh - b * heads;
    const int32_t live = min(n, window_len(g, b) - (is_v ? 0 : g.q_start));  // rows before the sequence's end
    const RawTensor &y = is_v ? p.vraw : p.doraw;
    const char *yp = y.p + b * y.batch + h * y.head + 16 * l, *op = p.oraw.p + b * p.oraw.batch + h * p.oraw.head + 16 * l;
    float *delta = p.delta + static_cast<int64_t>(bh) * g.nq;
    float most = 0.f;
    for (int r0 = 0; r0 < PRE_ROWS; r0 += 4 * NG) {
        Vec8<DT> vy[4], vo[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int32_t r = row0 + r0 + u * NG + grp;
            vy[u].r[0] = vo[u].r[0] = make_uint4(0u, 0u, 0u, 0u);
            if (r < live) {
                vy[u] = load8<DT>(yp + r * y.row);
                if (!is_v) vo[u] = load8<DT>(op + r * p.oraw.row);
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int32_t r = row0 + r0 + u * NG + grp;
            float a[8], c[8], dot = 0.f, sq = 0.f;
            widen8<DT>(vy[u], a);
            widen8<DT>(vo[u], c);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dot = fmaf(a[e], c[e], dot);
                sq = fmaf(a[e], a[e], sq);
            }
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) {
                dot += __shfl_xor_sync(0xffffffffu, dot, o);
                if (DT == ST_FP16) sq += __shfl_xor_sync(0xffffffffu, sq, o);
            }
            if (!is_v && l == 0 && r < g.nq) delta[r] = dot;  // (0 for padding rows: nothing was loaded)
            if (DT == ST_FP16) most = sq > most || sq != sq ? sq : most;  // a NaN stays
        }
    }
    if constexpr (DT == ST_FP16) {  // non-negative floats, NaN above all, order as integers
        uint32_t u = __float_as_uint(most) & 0x7FFFFFFFu;
        u = __reduce_max_sync(0xffffffffu, u);
        if ((threadIdx.x & 31) == 0) atomicMax(p.maxima + 2 * (b * g.kv + (is_v ? h : h / g.group)) + (is_v ? 1 : 0), u);
    }
}

// ---- dK, dV -----------------------------------------------------------------------------------
template <int D>
struct KCfg {
    static constexpr uint32_t TB = 128 * D * 2;
    static constexpr int NST = D == 64 ? 4 : 2;               // Q/dO ring
    static constexpr uint32_t OFF_V = TB, OFF_Q = 2 * TB, OFF_DO = OFF_Q + NST * TB, OFF_ROW = OFF_DO + NST * TB;
    static constexpr uint32_t ROW_BYTES = 2 * 128 * 4;        // per stage: -lse (log2 units), -D scaled
    static constexpr uint32_t OFF_BAR = OFF_ROW + NST * ROW_BYTES;
    static constexpr uint32_t SMEM = OFF_BAR + 512;
    // d = 64 has columns for S of even and odd steps
    static constexpr int NSB = D == 64 ? 2 : 1;
    static constexpr uint32_t COL_S = 0, COL_DP = 128 * NSB, COL_DV = COL_DP + 128, COL_DK = COL_DV + D;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct KUnit {
    int32_t b, hk, len, tile, i0, begin, end, entry;
    __device__ int32_t steps() const { return end - begin; }
};

__device__ __forceinline__ bool get_unit(const WindowBwdParams &p, int64_t at, KUnit &U)
{
    const WindowGeom &g = p.g;
    const int32_t n = g.batch * g.kv;
    if (at >= static_cast<int64_t>(p.nentries) * n) return false;
    const int32_t e = static_cast<int32_t>(at / n), bh = static_cast<int32_t>(at - static_cast<int64_t>(e) * n);
    const int2 en = p.entries[e];
    U.tile = en.x;
    U.entry = e;
    U.b = bh / g.kv;
    U.hk = bh - U.b * g.kv;
    U.len = window_len(g, U.b);
    const int32_t steps = tile_steps(g, U.tile, U.i0);
    const int32_t n_chunks = chunks_of(steps, p.chunk);
    U.begin = static_cast<int32_t>(static_cast<int64_t>(steps) * en.y / n_chunks);
    U.end = static_cast<int32_t>(static_cast<int64_t>(steps) * (en.y + 1) / n_chunks);
    // query tiles whose rows are all padding, and key tiles past the end, have nothing to add
    const int32_t live = U.len - g.q_start;  // query rows before the sequence's end
    const int32_t last = live > 0 && U.tile * 128 < U.len ? ((live + 127) / 128 - U.i0) * g.group : 0;
    U.end = max(U.begin, min(U.end, last));
    return true;
}

struct KBars {
    uint64_t k_full, k_empty, v_full, v_empty, qdo_full[4], qdo_empty[4];
    uint64_t s_full[2], dp_full, p_ready, ds_ready, acc_full, acc_free, mma_idle;
    UnitRing<KUnit> units;
    uint32_t tmem_base;
    int32_t abort;
};
static_assert(sizeof(KBars) <= 512, "barrier block");

template <int DT, int D>
__global__ void __launch_bounds__(THREADS, 1) window_dkdv_kernel(const __grid_constant__ WindowBwdParams p)
{
    using C = KCfg<D>;
    constexpr int NST = C::NST;
    constexpr uint32_t TB = C::TB;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    KBars *bars = reinterpret_cast<KBars *>(smem + C::OFF_BAR);
    volatile int32_t *abort = &bars->abort;
    const WindowGeom &g = p.g;
    int32_t *err = g.err;

    if (threadIdx.x == 0) {
        mbar_init(&bars->k_full, 1);
        mbar_init(&bars->k_empty, 1);
        mbar_init(&bars->v_full, 1);
        mbar_init(&bars->v_empty, 1);
        for (int i = 0; i < NST; ++i) {
            mbar_init(&bars->qdo_full[i], 1);
            mbar_init(&bars->qdo_empty[i], 1 + NSM / 32);  // the products, and each softmax warp's row data
        }
        mbar_init(&bars->s_full[0], 1);
        mbar_init(&bars->s_full[1], 1);
        mbar_init(&bars->dp_full, 1);
        mbar_init(&bars->p_ready, NSM);
        bars->units.init();
        mbar_init(&bars->ds_ready, NSM);
        mbar_init(&bars->acc_full, 1);
        mbar_init(&bars->acc_free, NSM);
        mbar_init(&bars->mma_idle, 1);
        bars->abort = (smem_u32(smem) & 1023u) ? 1 : 0;
        if (bars->abort) atomicOr(err, 2);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&bars->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = bars->tmem_base;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the preparation's results
    // ... and handed on to dq, which starts beside this kernel and needs nothing else of it
    if (blockIdx.x == 0 && threadIdx.x == 0) publish(p.counters + 2);
    asm volatile("griddepcontrol.launch_dependents;");
    const bool run = (*abort == 0);

    // I counts units with steps, J steps over all of them.
    if (warp == 0) {
        if (run) {
            if (lane == 0) {
                tma_prefetch(&p.q);
                tma_prefetch(&p.dout);
                tma_prefetch(&p.k);
                tma_prefetch(&p.v);
            }
            int32_t IK = 0, IV = 0, J = 0;
            bool ok = true;
            auto wait = [&](uint64_t *bar, int32_t n) { return __all_sync(0xffffffffu, mbar_wait(bar, n & 1, abort, err)); };
            KUnit U;
            bool taken = false;
            for (int32_t k = 0; ok && bars->units.put(p, p.counters, k, taken, U, abort, err); ++k) {
                const float dsc = g.scale * ds_factor<DT>(p, U.b, U.hk) * exp2f(-PBIAS<DT>);
                for (int32_t s = U.begin; ok && s < U.end; ++s) {
                    const int st = J % NST;
                    const int32_t qt = U.i0 + s / g.group, h = U.hk * g.group + s % g.group, row0 = qt * 128;
                    // row data of the step, on its way while the stage is awaited
                    float ls[4], de[4];
                    const int64_t base = (static_cast<int64_t>(U.b) * g.heads + h) * g.nq;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int32_t i = row0 + 32 * e + lane;
                        const bool live = i < g.nq && g.q_start + i < U.len;
                        ls[e] = live ? p.lse[base + i] : 0.f;
                        de[e] = live ? p.delta[base + i] : 0.f;
                    }
                    if (J >= NST && !(ok = wait(&bars->qdo_empty[st], J / NST - 1))) break;
                    uint64_t *bar = &bars->qdo_full[st];
                    uint8_t *sQ = smem + C::OFF_Q + st * TB, *sDO = smem + C::OFF_DO + st * TB;
                    const int32_t valid = U.len - g.q_start - row0;
                    const bool plain = valid < 128 && valid < g.nq - row0;  // rows past the end in the tile
                    if (!plain && lane == 0) {
                        mbar_expect_tx(bar, 2 * TB);
                        tma_tile<D>(&p.q, sQ, bar, row0, h, U.b);
                        tma_tile<D>(&p.dout, sDO, bar, row0, h, U.b);
                    }
                    __syncwarp();
                    if (plain) {
                        load_tile_rows<D>(p.qraw.p + U.b * p.qraw.batch + h * p.qraw.head + row0 * p.qraw.row, p.qraw.row, valid, sQ);
                        load_tile_rows<D>(p.doraw.p + U.b * p.doraw.batch + h * p.doraw.head + row0 * p.doraw.row, p.doraw.row, valid, sDO);
                    }
                    float *rows = reinterpret_cast<float *>(smem + C::OFF_ROW + st * C::ROW_BYTES);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        rows[32 * e + lane] = PBIAS<DT> - ls[e] * LOG2E;
                        rows[128 + 32 * e + lane] = -de[e] * dsc;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar);
                    ++J;
                    if (s == U.begin) {  // K and V of the unit, behind its first Q and dO
                        if (IK > 0 && !(ok = wait(&bars->k_empty, IK - 1))) break;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&bars->k_full, TB);
                            tma_tile<D>(&p.k, smem, &bars->k_full, U.tile * 128, U.hk, U.b);
                        }
                        __syncwarp();
                        ++IK;
                        if (IV > 0 && !(ok = wait(&bars->v_empty, IV - 1))) break;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&bars->v_full, TB);
                            tma_tile<D>(&p.v, smem + C::OFF_V, &bars->v_full, U.tile * 128, U.hk, U.b);
                        }
                        __syncwarp();
                        ++IV;
                    }
                }
            }
            if (*abort) {  // drain the copies in flight before the CTA leaves
                volatile int32_t never = 0;
                if (IK > 0) mbar_wait(&bars->k_full, (IK - 1) & 1, &never, err);
                if (IV > 0) mbar_wait(&bars->v_full, (IV - 1) & 1, &never, err);
                for (int32_t i = (J > NST ? J - NST : 0); i < J; ++i) mbar_wait(&bars->qdo_full[i % NST], (i / NST) & 1, &never, err);
            }
        }
    } else if (warp == 1) {
        if (run) {
            constexpr uint32_t id_s = idesc16<DT>(128, 128, false, false);  // S^T, dP^T
            constexpr uint32_t id_a = idesc16<DT>(128, D, false, true);     // dV, dK
            const uint32_t sK = smem_u32(smem), sV = smem_u32(smem + C::OFF_V);
            auto sQ = [&](int32_t t) { return smem_u32(smem + C::OFF_Q + (t % NST) * TB); };
            auto sDO = [&](int32_t t) { return smem_u32(smem + C::OFF_DO + (t % NST) * TB); };
            auto commit = [&](uint64_t *bar) {
                if (elect_one()) mma_commit(bar);
                __syncwarp();
            };
            auto wait = [&](uint64_t *bar, int32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err)); };
            auto issue_nn = [&](uint32_t col, uint32_t a, uint32_t b, uint64_t *bar) {
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_bf16_ss(tbase + col, Tile<D>::kmajor(a, k), Tile<D>::kmajor(b, k), id_s, k > 0 ? 1u : 0u);
                    mma_commit(bar);
                }
                __syncwarp();
            };
            // (P^T or dS^T in TMEM: 8 columns a step of 16 queries, the second 64 queries at + 64) B
            auto issue_acc = [&](uint32_t acc, uint32_t a, uint32_t b, bool first) {
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_bf16_ts(tbase + acc, tbase + a + (k >> 2) * 64 + (k & 3) * 8, Tile<D>::mnmajor(b, k), id_a,
                                    (!first || k > 0) ? 1u : 0u);
                }
                __syncwarp();
            };
            int32_t I = 0, J = 0;
            // S^T of step t, the unit's first or last
            auto s_of = [&](int32_t t, bool first, bool last) {
                if ((first && !wait(&bars->k_full, I & 1)) ||
                    !wait(&bars->qdo_full[t % NST], (t / NST) & 1))
                    return false;
                tc_fence_after();
                issue_nn(C::COL_S + 128 * (t % C::NSB), sK, sQ(t), &bars->s_full[t % C::NSB]);
                if (last) commit(&bars->k_empty);
                return true;
            };
            // dP^T of step t, whose dO is there if its S^T has been issued
            auto dp_of = [&](int32_t t, bool first, bool last) {
                if (first && !wait(&bars->v_full, I & 1)) return false;
                tc_fence_after();
                issue_nn(C::COL_DP, sV, sDO(t), &bars->dp_full);
                if (last) commit(&bars->v_empty);
                return true;
            };
            int32_t n = bars->units.take_steps(0, abort, err), s = 0;  // steps of unit I, the step in it
            const bool ok = n > 0 && s_of(0, true, n == 1) && dp_of(0, true, n == 1);
            // per step: dV += P^T dO and S^T of the next step, in this order where they share columns |
            // dK += dS^T Q | dP^T of the next step
            while (n > 0 && ok) {
                const int32_t t = J, i = I;
                const bool first = s == 0, last = s + 1 == n;
                ++s;
                if (last) {
                    n = bars->units.take_steps(++I, abort, err);
                    s = 0;
                }
                const bool more = n > 0, fin = s + 1 == n;  // fin: the next step is its unit's last
                if (C::NSB == 2 && more && !s_of(t + 1, last, fin)) break;
                if (!wait(&bars->p_ready, t & 1)) break;
                if (first && i > 0 && !wait(&bars->acc_free, (i - 1) & 1)) break;
                tc_fence_after();
                issue_acc(C::COL_DV, C::COL_S + 128 * (t % C::NSB), sDO(t), first);
                if (C::NSB == 1 && more && !s_of(t + 1, last, fin)) break;
                if (!wait(&bars->ds_ready, t & 1)) break;
                tc_fence_after();
                issue_acc(C::COL_DK, C::COL_DP, sQ(t), first);
                commit(&bars->qdo_empty[t % NST]);
                if (last) commit(&bars->acc_full);
                if (more && !dp_of(t + 1, last, fin)) break;
                ++J;
            }
            commit(&bars->mma_idle);
            volatile int32_t never = 0;
            mbar_wait(&bars->mma_idle, 0, &never, err);
        }
    } else if (warp < 4) {  // zeros of the units without steps
        const int t = threadIdx.x - 64;
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        KUnit U;
        for (int64_t at = blockIdx.x; get_unit(p, at, U); at += gridDim.x) {
            if (U.steps() != 0) continue;
            if (U.entry < p.nsplit) {  // the chunk's partial
                const int64_t slot = static_cast<int64_t>(U.b * g.kv + U.hk) * p.nsplit + U.entry;
                uint4 *dst = reinterpret_cast<uint4 *>(p.parts) + slot * (2 * (D / 4) * 128);
                for (int i = t; i < 2 * (D / 4) * 128; i += 64) dst[i] = zero;
                continue;
            }
            for (int i = t; i < 2 * 128 * (D / 8); i += 64) {
                const OutTensor &o = i < 128 * (D / 8) ? p.dv : p.dk;
                const int32_t kpos = U.tile * 128 + i / (D / 8) % 128;
                if (kpos < g.nk) *reinterpret_cast<uint4 *>(o.p + U.b * o.batch + U.hk * o.head + kpos * o.row + 16 * (i % (D / 8))) = zero;
            }
        }
    } else {
        const int w = (warp - 4) >> 2, q4 = warp & 3, row = q4 * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
        const uint32_t tS = tbase + lane_off + C::COL_S + 64 * w, tDP = tbase + lane_off + C::COL_DP + 64 * w;
        const uint64_t sc2 = f32x2(g.scale_log2, g.scale_log2);
        bool ok = run;
        int32_t I = 0, J = 0;
        auto wait_all = [&](uint64_t *bar, int32_t n) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, n & 1, abort, err));
            if (ok) tc_fence_after();
            return ok;
        };
        KUnit U;
        for (int32_t k = 0; ok; ++k) {
            if (!bars->units.take(k, U, abort, err)) break;
            const float fac = ds_factor<DT>(p, U.b, U.hk), dsc = g.scale * fac * exp2f(-PBIAS<DT>);
            const uint64_t dsc2 = f32x2(dsc, dsc);
            const int32_t kpos = U.tile * 128 + row;
            for (int32_t s = U.begin; ok && s < U.end; ++s, ++J) {
                const int st = J % NST;
                const int32_t base = g.q_start + (U.i0 + s / g.group) * 128 + 64 * w;  // position of this slice's first query
                // the queries that see this key: kpos .. up to the window's end (a sink: all later ones)
                const int32_t end = min(U.len, g.q_start + g.nq) - 1;
                const int32_t hi = (g.window == 0 || kpos < g.sinks) ? end : min(end, kpos + g.window - 1);
                const int32_t lo = kpos < U.len ? kpos - base : 64, up = hi - base;
                const bool whole = lo <= 0 && up >= 63;
                uint32_t sv[64];
                if (!wait_all(&bars->qdo_full[st], J / NST) || !wait_all(&bars->s_full[J % C::NSB], J / C::NSB)) break;
                const uint32_t rows = smem_u32(smem + C::OFF_ROW + st * C::ROW_BYTES) + 256 * w;
                const uint32_t tSj = tS + 128 * (J % C::NSB);
                tmem_ld32(tSj, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
                tmem_wait_ld();
                tmem_ld32(tSj + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
                const uint64_t keep = whole ? ~0ull : interval_bits64(lo, up);
                float pr[64];
#pragma unroll
                for (int c = 0; c < 64; c += 4) {
                    if (c == 32) tmem_wait_ld();
                    const uint4 r = ld_shared_v4(rows + 4 * c);
                    float x0, x1, x2, x3;
                    f32x2_split(fma2(f32x2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), sc2, f32x2(__uint_as_float(r.x), __uint_as_float(r.y))), x0, x1);
                    f32x2_split(fma2(f32x2(__uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3])), sc2, f32x2(__uint_as_float(r.z), __uint_as_float(r.w))), x2, x3);
                    pr[c] = ex2(x0);
                    pr[c + 1] = ex2(x1);
                    pr[c + 2] = ex2(x2);
                    pr[c + 3] = ex2(x3);
                }
                if (!whole) {
                    const uint32_t kw[2] = {static_cast<uint32_t>(keep), static_cast<uint32_t>(keep >> 32)};
#pragma unroll
                    for (int c = 0; c < 64; ++c) pr[c] = (kw[c >> 5] & (1u << (c & 31))) ? pr[c] : 0.f;
                }
                uint32_t pk[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) pk[c] = pack16<DT>(pr[2 * c], pr[2 * c + 1]);
                tmem_st32(tSj, pk);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&bars->p_ready);
                if (!wait_all(&bars->dp_full, J)) break;
                tmem_ld32(tDP, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
                tmem_wait_ld();
                tmem_ld32(tDP + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
#pragma unroll
                for (int c = 0; c < 64; c += 4) {
                    if (c == 32) tmem_wait_ld();
                    const uint4 r = ld_shared_v4(rows + 512 + 4 * c);
                    float x0, x1, x2, x3;
                    f32x2_split(mul2(f32x2(pr[c], pr[c + 1]), fma2(f32x2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), dsc2, f32x2(__uint_as_float(r.x), __uint_as_float(r.y)))), x0, x1);
                    f32x2_split(mul2(f32x2(pr[c + 2], pr[c + 3]), fma2(f32x2(__uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3])), dsc2, f32x2(__uint_as_float(r.z), __uint_as_float(r.w)))), x2, x3);
                    sv[c] = __float_as_uint(x0);
                    sv[c + 1] = __float_as_uint(x1);
                    sv[c + 2] = __float_as_uint(x2);
                    sv[c + 3] = __float_as_uint(x3);
                }
                if (!whole) {  // a masked entry may have been 0 times a NaN
                    const uint32_t kw[2] = {static_cast<uint32_t>(keep), static_cast<uint32_t>(keep >> 32)};
#pragma unroll
                    for (int c = 0; c < 64; ++c) sv[c] = (kw[c >> 5] & (1u << (c & 31))) ? sv[c] : 0u;
                }
#pragma unroll
                for (int c = 0; c < 32; ++c) pk[c] = pack16<DT>(__uint_as_float(sv[2 * c]), __uint_as_float(sv[2 * c + 1]));
                tmem_st32(tDP, pk);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&bars->ds_ready);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->qdo_empty[st]);
            }
            if (!ok) break;
            if (!wait_all(&bars->acc_full, I)) break;
            // dV, then dK: this warpgroup's half of the columns, 32 at a time
#pragma unroll
            for (int out = 0; out < 2; ++out) {
                const float f = out == 0 ? exp2f(-PBIAS<DT>) : 1.f / fac;
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    const int col = (D / 2) * w + 32 * c;
                    uint32_t a[32];
                    tmem_ld32(tbase + lane_off + (out == 0 ? C::COL_DV : C::COL_DK) + col, a);
                    tmem_wait_ld();
                    if (*abort) continue;
                    if (U.entry < p.nsplit) {  // fp32 partial of this chunk, quads of columns by 128 rows
                        const int64_t slot = static_cast<int64_t>(U.b * g.kv + U.hk) * p.nsplit + U.entry;
                        float4 *dst = reinterpret_cast<float4 *>(p.parts) + ((slot * 2 + out) * (D / 4) + col / 4) * 128 + row;
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            dst[q * 128] = make_float4(__uint_as_float(a[4 * q]) * f, __uint_as_float(a[4 * q + 1]) * f,
                                                       __uint_as_float(a[4 * q + 2]) * f, __uint_as_float(a[4 * q + 3]) * f);
                    } else if (kpos < g.nk) {
                        const OutTensor &t = out == 0 ? p.dv : p.dk;
                        uint4 *dst = reinterpret_cast<uint4 *>(t.p + U.b * t.batch + U.hk * t.head + kpos * t.row + 2 * col);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            float x[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(a[8 * q + e]) * f;
                            dst[q] = make_uint4(pack16<DT>(x[0], x[1]), pack16<DT>(x[2], x[3]), pack16<DT>(x[4], x[5]), pack16<DT>(x[6], x[7]));
                        }
                    }
                }
            }
            ++I;
            tc_fence_before();
            mbar_arrive(&bars->acc_free);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

// dK, dV of the key tiles cut into chunks: their partials added in chunk order.  A thread takes 8
// columns of one key row.
template <int DT, int D>
__global__ void __launch_bounds__(128) window_join_kernel(const __grid_constant__ WindowBwdParams p)
{
    const WindowGeom &g = p.g;
    const uint32_t e = blockIdx.x % static_cast<uint32_t>(p.nsplit), bo = blockIdx.x / static_cast<uint32_t>(p.nsplit);
    const int32_t ch = static_cast<int32_t>(bo % (D / 8)), out = static_cast<int32_t>(bo / (D / 8) & 1), bh = static_cast<int32_t>(bo / (D / 4));
    const int2 en = p.entries[e];
    if (en.y != 0) return;  // once a key tile: at its first chunk
    int32_t i0;
    const int32_t n = chunks_of(tile_steps(g, en.x, i0), p.chunk), row = threadIdx.x, kpos = en.x * 128 + row;
    if (kpos >= g.nk) return;
    const int64_t slot = static_cast<int64_t>(bh) * p.nsplit + e;
    const int32_t b = bh / g.kv, hk = bh - b * g.kv;
    const OutTensor &t = out == 0 ? p.dv : p.dk;
    float x[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = 0.f;
#pragma unroll 4
    for (int32_t c = 0; c < n; ++c) {
        const float4 *src = reinterpret_cast<const float4 *>(p.parts) + (((slot + c) * 2 + out) * (D / 4) + 2 * ch) * 128 + row;
        const float4 a = src[0], d = src[128];
        x[0] += a.x; x[1] += a.y; x[2] += a.z; x[3] += a.w;
        x[4] += d.x; x[5] += d.y; x[6] += d.z; x[7] += d.w;
    }
    *reinterpret_cast<uint4 *>(t.p + b * t.batch + hk * t.head + kpos * t.row + 16 * ch) =
        make_uint4(pack16<DT>(x[0], x[1]), pack16<DT>(x[2], x[3]), pack16<DT>(x[4], x[5]), pack16<DT>(x[6], x[7]));
}

// ---- dQ ---------------------------------------------------------------------------------------
template <int D>
struct QCfg {
    static constexpr uint32_t TB = 128 * D * 2;
    static constexpr int NS = D == 64 ? 8 : 5;                // K/V ring
    static constexpr uint32_t OFF_DO = TB, OFF_KV = 2 * TB;
    static constexpr uint32_t OFF_BAR = OFF_KV + NS * TB;
    static constexpr uint32_t SMEM = OFF_BAR + 512;
    // S of even and odd steps (dS overwrites it), dP, dQ
    static constexpr uint32_t COL_S = 0, COL_DP = 256, COL_DQ = 384;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct QUnit {
    int32_t b, h, len, row0;
    KeyRange r;
    __device__ int32_t steps() const { return r.any ? r.ns + r.kb1 - r.kb0 + 1 : 0; }
    __device__ int32_t tile(int32_t s) const { return s < r.ns ? s : r.kb0 + s - r.ns; }
};

// Longest (last rows) first.
__device__ __forceinline__ bool get_unit(const WindowBwdParams &p, int64_t at, QUnit &U)
{
    const WindowGeom &g = p.g;
    const int32_t n = g.batch * g.heads;
    if (at >= static_cast<int64_t>(n) * g.nqt) return false;
    const int32_t u = static_cast<int32_t>(at), qi = u / n, bh = u - qi * n;
    U.b = bh / g.heads;
    U.h = bh - U.b * g.heads;
    U.len = window_len(g, U.b);
    U.row0 = (g.nqt - 1 - qi) * 128;
    U.r = key_range(g, U.row0, U.len);
    return true;
}

struct QBars {
    uint64_t q_full, q_empty, do_full, do_empty, kv_full[8], kv_empty[8];
    uint64_t s_full[2], dp_full, dp_free, ds_ready, acc_full, acc_free, mma_idle;
    UnitRing<QUnit> units;
    uint32_t tmem_base;
    int32_t abort;
};
static_assert(sizeof(QBars) <= 512, "barrier block");

template <int DT, int D>
__global__ void __launch_bounds__(THREADS, 1) window_dq_kernel(const __grid_constant__ WindowBwdParams p)
{
    using C = QCfg<D>;
    constexpr int NS = C::NS;
    constexpr uint32_t TB = C::TB;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    QBars *bars = reinterpret_cast<QBars *>(smem + C::OFF_BAR);
    volatile int32_t *abort = &bars->abort;
    const WindowGeom &g = p.g;
    int32_t *err = g.err;

    if (threadIdx.x == 0) {
        mbar_init(&bars->q_full, 1);
        mbar_init(&bars->q_empty, 1);
        mbar_init(&bars->do_full, 1);
        mbar_init(&bars->do_empty, 1);
        for (int i = 0; i < NS; ++i) {
            mbar_init(&bars->kv_full[i], 1);
            mbar_init(&bars->kv_empty[i], 1);
        }
        mbar_init(&bars->s_full[0], 1);
        mbar_init(&bars->s_full[1], 1);
        mbar_init(&bars->dp_full, 1);
        bars->units.init();
        mbar_init(&bars->dp_free, NSM);
        mbar_init(&bars->ds_ready, NSM);
        mbar_init(&bars->acc_full, 1);
        mbar_init(&bars->acc_free, NSM);
        mbar_init(&bars->mma_idle, 1);
        bars->abort = (smem_u32(smem) & 1023u) ? 1 : 0;
        if (bars->abort) atomicOr(err, 2);
        fence_barrier_init();
        // D, the maxima and the counters: the barrier below passes them on to the CTA
        if (!await_published(p.counters + 2, err)) bars->abort = 1;
    }
    if (warp == 1) {
        tmem_alloc(&bars->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = bars->tmem_base;
    const bool run = (*abort == 0);

    // Ring entry 2 s is K of step s, 2 s + 1 its V, steps counted over all units; I counts units with
    // steps.
    if (warp == 0) {
        if (run) {
            if (lane == 0) {
                tma_prefetch(&p.q);
                tma_prefetch(&p.dout);
                tma_prefetch(&p.k);
                tma_prefetch(&p.v);
            }
            int32_t c = 0, IQ = 0, ID = 0;
            bool ok = true;
            auto wait = [&](uint64_t *bar, int32_t n) { return __all_sync(0xffffffffu, mbar_wait(bar, n & 1, abort, err)); };
            QUnit U;
            bool taken = false;
            for (int32_t k = 0; ok && bars->units.put(p, p.counters + 1, k, taken, U, abort, err); ++k) {
                const int32_t hk = U.h / g.group;
                for (int32_t s = 0; ok && s < U.steps(); ++s) {
                    const int32_t row = U.tile(s) * 128;
                    for (int v = 0; ok && v < 2; ++v, ++c) {
                        if (s == 0) {  // Q with the first K, dO with the first V
                            uint64_t *full = v ? &bars->do_full : &bars->q_full;
                            int32_t &n = v ? ID : IQ;
                            if (n > 0 && !(ok = wait(v ? &bars->do_empty : &bars->q_empty, n - 1))) break;
                            if (lane == 0) {
                                mbar_arrive_expect_tx(full, TB);
                                tma_tile<D>(v ? &p.dout : &p.q, smem + v * C::OFF_DO, full, U.row0, U.h, U.b);
                            }
                            __syncwarp();
                            ++n;
                        }
                        if (c >= NS && !(ok = wait(&bars->kv_empty[c % NS], c / NS - 1))) break;
                        uint8_t *dst = smem + C::OFF_KV + (c % NS) * TB;
                        uint64_t *bar = &bars->kv_full[c % NS];
                        if (!v && row + 128 > U.len && U.len < g.nk) {
                            load_tile_rows<D>(p.kraw.p + U.b * p.kraw.batch + hk * p.kraw.head + row * p.kraw.row, p.kraw.row, U.len - row, dst);
                            if (lane == 0) mbar_arrive(bar);
                        } else if (lane == 0) {
                            mbar_arrive_expect_tx(bar, TB);
                            tma_tile<D>(v ? &p.v : &p.k, dst, bar, row, hk, U.b);
                        }
                        __syncwarp();
                    }
                }
            }
            if (*abort) {  // drain the copies in flight before the CTA leaves
                volatile int32_t never = 0;
                if (IQ > 0) mbar_wait(&bars->q_full, (IQ - 1) & 1, &never, err);
                if (ID > 0) mbar_wait(&bars->do_full, (ID - 1) & 1, &never, err);
                for (int32_t i = (c > NS ? c - NS : 0); i < c; ++i) mbar_wait(&bars->kv_full[i % NS], (i / NS) & 1, &never, err);
            }
        }
    } else if (warp == 1) {
        if (run) {
            constexpr uint32_t id_s = idesc16<DT>(128, 128, false, false), id_q = idesc16<DT>(128, D, false, true);
            const uint32_t sQ = smem_u32(smem), sDO = smem_u32(smem + C::OFF_DO);
            auto slot = [&](int32_t c) { return smem_u32(smem + C::OFF_KV + (c % NS) * TB); };
            auto commit = [&](uint64_t *bar) {
                if (elect_one()) mma_commit(bar);
                __syncwarp();
            };
            // (a wait that runs out for some lanes only ends it for all: the warp walks as a whole)
            auto wait = [&](uint64_t *bar, int32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err)); };
            auto kv_wait = [&](int32_t c) { return wait(&bars->kv_full[c % NS], (c / NS) & 1); };
            auto issue_nn = [&](uint32_t col, uint32_t a, uint32_t b, uint64_t *bar) {
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_bf16_ss(tbase + col, Tile<D>::kmajor(a, k), Tile<D>::kmajor(b, k), id_s, k > 0 ? 1u : 0u);
                    mma_commit(bar);
                }
                __syncwarp();
            };
            int32_t n = 0, st = 0, I = -1;  // step st of unit I, which has n, is issued next
            auto next = [&]() {
                if (++st < n) return true;
                n = bars->units.take_steps(++I, abort, err);
                st = 0;
                return n > 0;
            };
            // S and dP of step t (step st of unit I), dP once that of t - 1 is in registers
            auto s_dp_of = [&](int32_t t) {
                if ((st == 0 && !wait(&bars->q_full, I & 1)) || !kv_wait(2 * t)) return false;
                tc_fence_after();
                issue_nn(C::COL_S + 128 * (t & 1), sQ, slot(2 * t), &bars->s_full[t & 1]);
                if (st + 1 == n) commit(&bars->q_empty);
                if ((st == 0 && !wait(&bars->do_full, I & 1)) || !kv_wait(2 * t + 1) ||
                    (t > 0 && !wait(&bars->dp_free, (t - 1) & 1)))
                    return false;
                tc_fence_after();
                issue_nn(C::COL_DP, sDO, slot(2 * t + 1), &bars->dp_full);
                commit(&bars->kv_empty[(2 * t + 1) % NS]);
                if (st + 1 == n) commit(&bars->do_empty);
                return true;
            };
            bool more = next();
            const bool ok = more && s_dp_of(0);
            for (int32_t t = 0; ok && more; ++t) {
                const bool first = st == 0, last = st + 1 == n;
                const int32_t i = I;
                auto dq_of = [&]() {
                    if (!wait(&bars->ds_ready, t & 1) ||
                        (first && i > 0 && !wait(&bars->acc_free, (i - 1) & 1)))
                        return false;
                    tc_fence_after();
                    const uint32_t a = tbase + C::COL_S + 128 * (t & 1), b = slot(2 * t);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            mma_bf16_ts(tbase + C::COL_DQ, a + (k >> 2) * 64 + (k & 3) * 8, Tile<D>::mnmajor(b, k), id_q,
                                        (!first || k > 0) ? 1u : 0u);
                    }
                    __syncwarp();
                    commit(&bars->kv_empty[(2 * t) % NS]);
                    if (last) commit(&bars->acc_full);
                    return true;
                };
                // the next step's S and dP ahead of dQ, but behind it where they wait for another
                // unit's Q and dO
                if (last && !dq_of()) break;
                more = next();
                if (more && !s_dp_of(t + 1)) break;
                if (!last && !dq_of()) break;
            }
            commit(&bars->mma_idle);
            volatile int32_t never = 0;
            mbar_wait(&bars->mma_idle, 0, &never, err);
        }
    } else if (warp < 4) {  // zeros of the units without steps
        QUnit U;
        for (int64_t at = blockIdx.x; get_unit(p, at, U); at += gridDim.x) {
            if (U.steps() != 0) continue;
            for (int i = threadIdx.x - 64; i < 128 * (D / 8); i += 64) {
                const int32_t row = U.row0 + i / (D / 8);
                if (row < g.nq)
                    *reinterpret_cast<uint4 *>(p.dq.p + U.b * p.dq.batch + U.h * p.dq.head + row * p.dq.row + 16 * (i % (D / 8))) =
                        make_uint4(0u, 0u, 0u, 0u);
            }
        }
    } else {
        const int w = (warp - 4) >> 2, q4 = warp & 3, row = q4 * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
        const uint32_t tS = tbase + lane_off + C::COL_S + 64 * w, tDP = tbase + lane_off + C::COL_DP + 64 * w;
        const uint64_t sc2 = f32x2(g.scale_log2, g.scale_log2);
        bool ok = run;
        int32_t I = 0, J = 0;
        auto wait_all = [&](uint64_t *bar, int32_t n) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, n & 1, abort, err));
            if (ok) tc_fence_after();
            return ok;
        };
        QUnit U;
        for (int32_t k = 0; ok; ++k) {
            if (!bars->units.take(k, U, abort, err)) break;
            const int32_t i = U.row0 + row, pos = g.q_start + i;
            const bool live = i < g.nq && pos < U.len;
            const float fac = ds_factor<DT>(p, U.b, U.h / g.group), dsc = g.scale * fac;
            float nlse = 0.f, nd = 0.f;
            if (live) {
                const int64_t r = (static_cast<int64_t>(U.b) * g.heads + U.h) * g.nq + i;
                nlse = -p.lse[r] * LOG2E;
                nd = -__ldcg(p.delta + r) * dsc;
            }
            const uint64_t nl2 = f32x2(nlse, nlse), nd2 = f32x2(nd, nd), dsc2 = f32x2(dsc, dsc);
            for (int32_t s = 0; ok && s < U.steps(); ++s, ++J) {
                const int32_t base = U.tile(s) * 128 + 64 * w;
                const bool whole = live && base + 63 <= pos && (g.window == 0 || base > pos - g.window || base + 64 <= g.sinks);
                const uint64_t keep = whole ? ~0ull : (live ? window_bits64(pos, g.window, g.sinks, base) : 0ull);
                const uint32_t kw[2] = {static_cast<uint32_t>(keep), static_cast<uint32_t>(keep >> 32)};
                uint32_t sv[64];
                float pr[64];
                if (!wait_all(&bars->s_full[J & 1], J >> 1)) break;
                tmem_ld32(tS + 128 * (J & 1), *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
                tmem_ld32(tS + 128 * (J & 1) + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                    float x0, x1;
                    f32x2_split(fma2(f32x2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), sc2, nl2), x0, x1);
                    pr[c] = ex2(x0);
                    pr[c + 1] = ex2(x1);
                }
                if (!wait_all(&bars->dp_full, J)) break;
                tmem_ld32(tDP, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
                tmem_ld32(tDP + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
                tmem_wait_ld();
                tc_fence_before();
                mbar_arrive(&bars->dp_free);
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                    float x0, x1;
                    f32x2_split(mul2(f32x2(pr[c], pr[c + 1]), fma2(f32x2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), dsc2, nd2)), x0, x1);
                    sv[c] = __float_as_uint(x0);
                    sv[c + 1] = __float_as_uint(x1);
                }
                if (!whole) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) sv[c] = (kw[c >> 5] & (1u << (c & 31))) ? sv[c] : 0u;
                }
                uint32_t pk[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) pk[c] = pack16<DT>(__uint_as_float(sv[2 * c]), __uint_as_float(sv[2 * c + 1]));
                tmem_st32(tS + 128 * (J & 1), pk);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&bars->ds_ready);
            }
            if (!ok) break;
            if (!wait_all(&bars->acc_full, I)) break;
            const float f = 1.f / fac;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const int col = (D / 2) * w + 32 * c;
                uint32_t a[32];
                tmem_ld32(tbase + lane_off + C::COL_DQ + col, a);
                tmem_wait_ld();
                if (i >= g.nq || *abort) continue;
                uint4 *dst = reinterpret_cast<uint4 *>(p.dq.p + U.b * p.dq.batch + U.h * p.dq.head + i * p.dq.row + 2 * col);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = live ? __uint_as_float(a[8 * q + e]) * f : 0.f;
                    dst[q] = make_uint4(pack16<DT>(x[0], x[1]), pack16<DT>(x[2], x[3]), pack16<DT>(x[4], x[5]), pack16<DT>(x[6], x[7]));
                }
            }
            ++I;
            tc_fence_before();
            mbar_arrive(&bars->acc_free);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what follows in the stream follows dk_dv too
}

template <int DT, int D>
cudaError_t launch(const WindowBwdParams &p, cudaStream_t s)
{
    static std::atomic<uint64_t> done_k{0}, done_q{0};
    cudaError_t e = allow_smem(window_dkdv_kernel<DT, D>, KCfg<D>::SMEM, done_k);
    if (e == cudaSuccess) e = allow_smem(window_dq_kernel<DT, D>, QCfg<D>::SMEM, done_q);
    if (e != cudaSuccess) return e;
    const WindowGeom &g = p.g;
    const int64_t cap = sm_count();
    if (DT == ST_FP16 && (e = cudaMemsetAsync(p.maxima, 0, sizeof(uint32_t) * 2 * g.batch * g.kv, s)) != cudaSuccess) return e;
    int64_t pre = 1 + static_cast<int64_t>(g.batch) * g.heads * ((g.nq + PRE_ROWS - 1) / PRE_ROWS);
    if (DT == ST_FP16) pre += static_cast<int64_t>(g.batch) * g.kv * ((g.nk + PRE_ROWS - 1) / PRE_ROWS);
    window_pre_kernel<DT, D><<<static_cast<unsigned>(pre), 256, 0, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int64_t ku = static_cast<int64_t>(p.nentries) * g.batch * g.kv, qu = static_cast<int64_t>(g.batch) * g.heads * g.nqt;
    // dk_dv is set up while the preparation ends; dq runs on the SMs that dk_dv leaves or does not need: it
    // starts once every CTA of dk_dv has (and the preparation has ended; await_published), and ends after it.
    // (All of dk_dv's CTAs fit at once, one an SM, so none waits for an SM that dq holds.)
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ku < cap ? ku : cap));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = KCfg<D>::SMEM;
    cfg.stream = s;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, window_dkdv_kernel<DT, D>, p)) != cudaSuccess) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(qu < cap ? qu : cap));
    cfg.dynamicSmemBytes = QCfg<D>::SMEM;
    if ((e = cudaLaunchKernelEx(&cfg, window_dq_kernel<DT, D>, p)) != cudaSuccess || p.nsplit == 0) return e;
    window_join_kernel<DT, D><<<static_cast<unsigned>(p.nsplit) * g.batch * g.kv * (D / 4), 128, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_bwd(const WindowBwdParams &p, int dtype, int d, cudaStream_t s)
{
    if (dtype == ST_BF16) return d == 64 ? launch<ST_BF16, 64>(p, s) : launch<ST_BF16, 128>(p, s);
    return d == 64 ? launch<ST_FP16, 64>(p, s) : launch<ST_FP16, 128>(p, s);
}

}  // namespace st
