// window_fwd.cu -- forward pass of attention with a sliding window and sinks on sm_100a.
//
// Row i at position p = q_start + i:  O_i = sum_j P_ij v_j, P = softmax over the keys j <= p with
// j > p - window or j < sinks; lse_i = ln sum_j exp(q_i . k_j / sqrt d).  Online over tiles of 128
// keys: with the running maximum m, p = 2^(s log2(e) / sqrt d - m), l = sum p, O = sum p v, both
// rescaled by 2^(m - m') when the maximum grows by more than 2^8 (a stale maximum is as good: O and l
// share it).  Only the tiles that some row of a query tile sees are visited.
//
// One CTA an SM, persistent.  A work unit is two query tiles ("subs") that read the same keys: two
// heads of a group where the group is even (one key tile feeds both), else two row tiles of a head.
//   warp 0      producer: Q of both subs (double buffered), K and V tiles through one ring
//   warp 1      MMA issuer: S_x = Q_x K^T into 128 columns of TMEM, O_x += P_x V with P_x read from TMEM
//   warps 4..7, 8..11  softmax of sub 0 and of sub 1, one query row a thread; P_x overwrites S_x
// While one sub's softmax runs the tensor core works on the other's: S_x(t + 1) is issued right after
// O_x += P_x(t) V(t), which orders it behind the last read of P_x(t).  Units are dealt out in turns
// (there and back), longest first; no counter, so no memory to clear and the same order every time.
// Per 128 x 128 tile the tensor core needs 1024 cycles at d = 128 and the exponentials 1024 cycles of
// the special-function units.
#include "kernels.h"
#include "lm.h"
#include "window_tiles.cuh"

namespace st {
namespace {

constexpr int THREADS = 384;
// registers a thread: 168 at launch; the first warpgroup hands some to the two softmax warpgroups
// (80 + 2 x 208 <= 3 x 168)
#define ST_REGS_DEC "setmaxnreg.dec.sync.aligned.u32 80;"
#define ST_REGS_INC "setmaxnreg.inc.sync.aligned.u32 208;"
constexpr float RESCALE_LOG2 = 8.0f;

template <int DT, int D>
struct Cfg {
    static constexpr uint32_t TB = 128 * D * 2;        // bytes of a tile
    static constexpr int NS = D == 64 ? 8 : 3;         // K/V ring slots
    static constexpr int NQB = 2;                      // Q buffers (of two subs)
    static constexpr uint32_t OFF_KV = NQB * 2 * TB;
    static constexpr uint32_t OFF_BAR = OFF_KV + NS * TB;
    static constexpr uint32_t SMEM = OFF_BAR + 512;
    static constexpr uint32_t COL_O = 256;             // S_x at 128 x, O_x at 256 + D x
    // fp16 weights are kept 2^6 larger: small ones stay normal numbers, and 2^(8 + 6) is in range
    static constexpr float BIAS = DT == ST_FP16 ? 6.f : 0.f;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct Bars {
    uint64_t q_full[2], q_empty[2], kv_full[8], kv_empty[8];
    uint64_t s_full[2], p_full[2], o_done[2], o_free[2], mma_idle;
    uint32_t tmem_base;
    int32_t abort;
};
static_assert(sizeof(Bars) <= 512, "barrier block");

struct Unit {
    int32_t b, len, head[2], row0[2];
    KeyRange r[2];
    int32_t kb0, ns, steps;  // tiles 0 .. ns - 1, then kb0 ..

    __device__ int32_t tile(int32_t s) const { return s < ns ? s : kb0 + s - ns; }
};

// Unit k of this CTA (false: no more).  Longest (last rows) first; odd turns run backwards.
__device__ __forceinline__ bool get_unit(const WindowFwdParams &p, int32_t k, Unit &U)
{
    const int64_t at = static_cast<int64_t>(k) * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    if (at >= p.units) return false;
    const WindowGeom &g = p.g;
    const int32_t u = static_cast<int32_t>(at), cols = p.pair_rows ? g.heads : g.heads / 2;  // units of a batch element and row tile
    const int32_t n = cols * g.batch, qi = u / n, hb = u - qi * n;
    U.b = hb / cols;
    const int32_t h = hb - U.b * cols;
    U.len = window_len(g, U.b);
    const int32_t nrow = p.pair_rows ? (g.nqt + 1) / 2 : g.nqt, rt = nrow - 1 - qi;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        U.head[x] = p.pair_rows ? h : 2 * h + x;
        U.row0[x] = (p.pair_rows ? 2 * rt + x : rt) * 128;
        U.r[x] = key_range(g, U.row0[x], U.len);
    }
    const KeyRange &a = U.r[0], &c = U.r[1];
    U.steps = U.ns = U.kb0 = 0;
    if (a.any || c.any) {
        U.kb0 = !c.any ? a.kb0 : (!a.any ? c.kb0 : min(a.kb0, c.kb0));
        const int32_t kb1 = max(a.kb1, c.kb1);
        U.ns = min(max(a.ns, c.ns), U.kb0);
        U.steps = U.ns + kb1 - U.kb0 + 1;
    }
    return true;
}

__device__ __forceinline__ float max128(const uint32_t (&v)[128])
{
    float a[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = fmaxf(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
#pragma unroll
    for (int c = 16; c < 128; c += 2)
        a[(c >> 1) & 7] = max3f(a[(c >> 1) & 7], __uint_as_float(v[c]), __uint_as_float(v[c + 1]));
    return max3f(max3f(a[0], a[1], a[2]), max3f(a[3], a[4], a[5]), fmaxf(a[6], a[7]));
}

__device__ __forceinline__ uint32_t (&part32(uint32_t (&v)[128], int e))[32]
{
    return *reinterpret_cast<uint32_t(*)[32]>(&v[e]);
}

template <int DT, int D>
__global__ void __launch_bounds__(THREADS, 1) window_fwd_kernel(const __grid_constant__ WindowFwdParams p)
{
    using C = Cfg<DT, D>;
    constexpr int NS = C::NS;
    constexpr uint32_t TB = C::TB;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Bars *bars = reinterpret_cast<Bars *>(smem + C::OFF_BAR);
    volatile int32_t *abort = &bars->abort;
    int32_t *err = p.g.err;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->q_full[i], 1);
            mbar_init(&bars->q_empty[i], 1);
            mbar_init(&bars->s_full[i], 1);
            mbar_init(&bars->p_full[i], 128);
            mbar_init(&bars->o_done[i], 1);
            mbar_init(&bars->o_free[i], 128);
        }
        for (int i = 0; i < NS; ++i) {
            mbar_init(&bars->kv_full[i], 1);
            mbar_init(&bars->kv_empty[i], 1);
        }
        mbar_init(&bars->mma_idle, 1);
        bars->abort = (smem_u32(smem) & 1023u) ? 1 : 0;  // the 128-byte swizzle needs aligned tiles
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
    const bool run = (*abort == 0);

    // Ring entry 2 s is K of step s, 2 s + 1 its V, steps counted over all units of the CTA; entry c
    // uses slot c % NS for the (c / NS)-th time.
    if (warp < 4) asm volatile(ST_REGS_DEC);
    if (warp == 0) {
        if (run) {
            if (lane == 0) {
                tma_prefetch(&p.q);
                tma_prefetch(&p.k);
                tma_prefetch(&p.v);
            }
            int32_t c = 0, uq = 0;  // ring entries and units with steps so far
            bool ok = true;
            auto claim = [&](int32_t n) {  // the slot of entry n is free
                return n < NS || __all_sync(0xffffffffu, mbar_wait(&bars->kv_empty[n % NS], ((n / NS) - 1) & 1, abort, err));
            };
            Unit U;
            for (int32_t k = 0; ok && get_unit(p, k, U); ++k) {
                if (U.steps == 0) continue;
                const int qb = uq & 1;
                if (uq >= 2 && !__all_sync(0xffffffffu, mbar_wait(&bars->q_empty[qb], ((uq >> 1) - 1) & 1, abort, err))) break;
                ++uq;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bars->q_full[qb], (U.r[0].any + U.r[1].any) * TB);
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        if (U.r[x].any)
                            tma_tile<D>(&p.q, smem + (2 * qb + x) * TB, &bars->q_full[qb], U.row0[x], U.head[x], U.b);
                }
                __syncwarp();
                const int32_t hk = U.head[0] / p.g.group;
                for (int32_t s = 0; ok && s < U.steps; ++s) {
                    const int32_t row = U.tile(s) * 128;
                    for (int v = 0; ok && v < 2; ++v, ++c) {
                        ok = claim(c);
                        if (!ok) break;
                        uint8_t *dst = smem + C::OFF_KV + (c % NS) * TB;
                        uint64_t *bar = &bars->kv_full[c % NS];
                        if (v && row + 128 > U.len && U.len < p.g.nk) {
                            load_tile_rows<D>(p.vraw.p + U.b * p.vraw.batch + hk * p.vraw.head + row * p.vraw.row, p.vraw.row,
                                              U.len - row, dst);
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
                for (int32_t i = (uq > 2 ? uq - 2 : 0); i < uq; ++i) mbar_wait(&bars->q_full[i & 1], (i >> 1) & 1, &never, err);
                for (int32_t i = (c > NS ? c - NS : 0); i < c; ++i) mbar_wait(&bars->kv_full[i % NS], (i / NS) & 1, &never, err);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && run) {
            constexpr uint32_t idS = idesc16<DT>(128, 128, false, false), idO = idesc16<DT>(128, D, false, true);
            Unit U, N;                   // the current unit and the one the next step belongs to
            int32_t kn = 0, uq = 0;      // next unit to fetch; units with steps begun (N's, once fetched)
            int32_t su = 0, sn = 0;      // step within U and N
            int32_t st = 0;              // steps done over all units
            int32_t nP[2] = {0, 0}, nO[2] = {0, 0};  // P tiles consumed, units with an O begun
            auto fetch = [&]() {         // the next unit that has steps
                while (get_unit(p, kn, N)) {
                    ++kn;
                    if (N.steps > 0) {
                        ++uq;
                        return true;
                    }
                }
                return false;
            };
            auto kv_wait = [&](int32_t c) { return mbar_wait(&bars->kv_full[c % NS], (c / NS) & 1, abort, err); };
            auto issue_s = [&](int x, int32_t step) {
                const uint32_t sQ = smem_u32(smem + (2 * ((uq - 1) & 1) + x) * TB), sK = smem_u32(smem + C::OFF_KV + ((2 * step) % NS) * TB);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_bf16_ss(tbase + 128 * x, Tile<D>::kmajor(sQ, k), Tile<D>::kmajor(sK, k), idS, k > 0 ? 1u : 0u);
                mma_commit(&bars->s_full[x]);
            };
            // Q and K of the next step, once for both subs
            auto next_ready = [&](int32_t step) {
                return (sn > 0 || mbar_wait(&bars->q_full[(uq - 1) & 1], ((uq - 1) >> 1) & 1, abort, err)) && kv_wait(2 * step);
            };
            auto next_issued = [&](int32_t step) {
                mma_commit(&bars->kv_empty[(2 * step) % NS]);
                if (sn + 1 == N.steps) mma_commit(&bars->q_empty[(uq - 1) & 1]);  // the unit's last S
            };
            bool more = fetch(), ok = true;
            if (more && (ok = next_ready(0))) {
                tc_fence_after();
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    if (N.r[x].has(N.tile(0))) issue_s(x, 0);
                next_issued(0);
            }
            while (ok && more) {
                U = N;
                su = sn;
                if (sn + 1 < N.steps) {
                    ++sn;
                } else {
                    more = fetch();
                    sn = 0;
                }
                const int32_t tc = U.tile(su);
                bool have_v = false, have_n = false;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (ok && U.r[x].has(tc)) {
                        if (!have_v) ok = kv_wait(2 * st + 1);
                        have_v = true;
                        ok = ok && mbar_wait(&bars->p_full[x], nP[x] & 1, abort, err);
                        ++nP[x];
                        // first and last tile of this sub in the unit
                        const int32_t first = U.r[x].ns > 0 ? 0 : U.r[x].kb0;
                        if (ok && tc == first) {
                            if (nO[x] > 0) ok = mbar_wait(&bars->o_free[x], (nO[x] - 1) & 1, abort, err);
                            ++nO[x];
                        }
                        if (ok) {
                            tc_fence_after();
                            const uint32_t sV = smem_u32(smem + C::OFF_KV + ((2 * st + 1) % NS) * TB);
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                mma_bf16_ts(tbase + C::COL_O + D * x, tbase + 128 * x + 8 * k, Tile<D>::mnmajor(sV, k), idO,
                                            (tc != first || k > 0) ? 1u : 0u);
                            if (tc == U.r[x].kb1) mma_commit(&bars->o_done[x]);
                        }
                    }
                    if (ok && more && N.r[x].has(N.tile(sn))) {
                        if (!have_n) ok = next_ready(st + 1);
                        have_n = true;
                        if (ok) {
                            tc_fence_after();
                            issue_s(x, st + 1);
                        }
                    }
                }
                if (!ok) break;
                mma_commit(&bars->kv_empty[(2 * st + 1) % NS]);
                if (more) next_issued(st + 1);
                ++st;
            }
            mma_commit(&bars->mma_idle);  // no product may run when TMEM is released
            volatile int32_t never = 0;
            mbar_wait(&bars->mma_idle, 0, &never, err);
        }
    } else if (warp >= 4) {
        asm volatile(ST_REGS_INC);
        const int x = (warp - 4) >> 2, q4 = warp & 3;  // sub; TMEM lane quarter
        const int row = q4 * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
        const uint32_t tS = tbase + lane_off + 128 * x, tO = tbase + lane_off + C::COL_O + D * x;
        const float sc = p.g.scale_log2;
        uint32_t v[128];
        bool ok = run;
        int32_t nS = 0, nO = 0;
        auto wait_all = [&](uint64_t *bar, int32_t n) {
            if (!__all_sync(0xffffffffu, mbar_wait(bar, n & 1, abort, err))) return false;
            tc_fence_after();
            return true;
        };
        Unit U;
        for (int32_t k = 0; ok && get_unit(p, k, U); ++k) {
            const KeyRange r = x ? U.r[1] : U.r[0];
            const int32_t head = x ? U.head[1] : U.head[0];
            const int32_t i = (x ? U.row0[1] : U.row0[0]) + row, pos = p.g.q_start + i;
            const bool live = i < p.g.nq && pos < U.len;
            float m = -INFINITY, l = 0.f;
            for (int32_t s = 0; ok && s < U.steps; ++s) {
                const int32_t tile = U.tile(s);
                if (!r.has(tile)) continue;
                if (!(ok = wait_all(&bars->s_full[x], nS))) break;
                ++nS;
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, part32(v, 32 * c));
                tmem_wait_ld();
                const int32_t base = tile * 128;
                const bool whole = live && base + 127 <= pos && (p.g.window == 0 || base > pos - p.g.window || base + 128 <= p.g.sinks);
                if (!whole) {
                    const uint64_t b0 = live ? window_bits64(pos, p.g.window, p.g.sinks, base) : 0ull;
                    const uint64_t b1 = live ? window_bits64(pos, p.g.window, p.g.sinks, base + 64) : 0ull;
                    const uint32_t kw[4] = {static_cast<uint32_t>(b0), static_cast<uint32_t>(b0 >> 32), static_cast<uint32_t>(b1), static_cast<uint32_t>(b1 >> 32)};
#pragma unroll
                    for (int c = 0; c < 128; ++c) v[c] = (kw[c >> 5] & (1u << (c & 31))) ? v[c] : 0xFF800000u;
                }
                const float m_new = fmaxf(m, max128(v) * sc);
                const bool grow = m_new > m + RESCALE_LOG2;  // also true for the first finite maximum
                const float m_use = grow ? m_new : m;
                const float alpha = grow ? ex2(m - m_use) : 1.f;
                const float nb = (m_use == -INFINITY) ? 0.f : C::BIAS - m_use;
                const uint64_t sc2 = f32x2(sc, sc), nb2 = f32x2(nb, nb);
                uint64_t ps2[2] = {0ull, 0ull};
#pragma unroll
                for (int c = 0; c < 128; c += 2) {
                    float x0, x1;
                    f32x2_split(fma2(f32x2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), sc2, nb2), x0, x1);
                    const float p0 = ex2(x0), p1 = ex2(x1);
                    ps2[(c >> 1) & 1] = add2(ps2[(c >> 1) & 1], f32x2(p0, p1));
                    v[c >> 1] = pack16<DT>(p0, p1);
                }
                // S_x(t) complete means every product issued before it is: O holds all earlier tiles
                if (__any_sync(0xffffffffu, grow && m != -INFINITY)) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(tO + 32 * c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st32(tO + 32 * c, o);
                    }
                }
                tmem_st32(tS, part32(v, 0));
                tmem_st32(tS + 32, part32(v, 32));
                tmem_wait_st();
                float s0, s1, s2, s3;
                f32x2_split(ps2[0], s0, s1);
                f32x2_split(ps2[1], s2, s3);
                l = l * alpha + ((s0 + s1) + (s2 + s3));
                m = m_use;
                tc_fence_before();
                mbar_arrive(&bars->p_full[x]);
            }
            if (!ok) break;
            if (r.any && !(ok = wait_all(&bars->o_done[x], nO))) break;
            const bool write = i < p.g.nq && *abort == 0;
            const float inv = live ? 1.f / l : 0.f;
            uint4 *dst = reinterpret_cast<uint4 *>(p.o + U.b * p.o_batch + head * p.o_head + i * p.o_row);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (r.any) {
                    tmem_ld32(tO + 32 * c, o);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float a[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) a[e] = live ? __uint_as_float(o[8 * q + e]) * inv : 0.f;
                    if (write)
                        dst[4 * c + q] = make_uint4(pack16<DT>(a[0], a[1]), pack16<DT>(a[2], a[3]), pack16<DT>(a[4], a[5]),
                                                    pack16<DT>(a[6], a[7]));
                }
            }
            if (r.any) {
                ++nO;
                tc_fence_before();
                mbar_arrive(&bars->o_free[x]);
            }
            if (!write) continue;
            p.lse[(static_cast<int64_t>(U.b) * p.g.heads + head) * p.g.nq + i] =
                live ? (m - C::BIAS + lg2(l)) * LN2 : -INFINITY;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

template <int DT, int D>
cudaError_t launch(const WindowFwdParams &p, cudaStream_t s)
{
    using C = Cfg<DT, D>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(window_fwd_kernel<DT, D>, C::SMEM, done);
    if (e != cudaSuccess) return e;
    const int32_t cap = sm_count();
    window_fwd_kernel<DT, D><<<static_cast<unsigned>(p.units < cap ? p.units : cap), THREADS, C::SMEM, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_fwd(const WindowFwdParams &p, int dtype, int d, cudaStream_t s)
{
    if (dtype == ST_BF16) return d == 64 ? launch<ST_BF16, 64>(p, s) : launch<ST_BF16, 128>(p, s);
    return d == 64 ? launch<ST_FP16, 64>(p, s) : launch<ST_FP16, 128>(p, s);
}

}  // namespace st
