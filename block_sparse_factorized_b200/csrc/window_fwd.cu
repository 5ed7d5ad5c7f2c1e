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
//   warp 0      producer: the units (into a ring that the others read), Q of both subs, K and V tiles
//               through one ring
//   warps 1, 2  MMA issuers of sub 0 and of sub 1: S_x = Q_x K^T into 128 columns of TMEM, O_x += P_x V
//               with P_x read from TMEM; all that they have to know of a step is a word of flags that the
//               producer leaves.  Two, because the tensor core's queue holds only some four products: one
//               issuer's waits and commits (some 500 cycles a tile) would leave it dry
//   warp 3      writes the zeros of units without live rows
//   warps 4..7, 8..11  softmax of sub 0 and of sub 1, one query row a thread; a unit's O is written out
//               (staged, whole rows) after the next unit's first exponentials, while its last product runs
// d = 64 has TMEM columns for P of its own, so S of the next tile runs during the softmax; at d = 128
// (S 2 x 128, O 2 x 128) P overwrites S, and the other sub's softmax covers the products.  Units are
// dealt out in turns (there and back), longest first; no counter, which would need memory of the call's own.  Per 128 x 128 tile the tensor core needs 1024 cycles at d = 128 (512 at d = 64) and
// the exponentials 1024 cycles of the special-function units.
//
// Measured, bf16, n = 12288 (of 1616 TFLOP/s for a library product):
//   d 128, 2 x 16 heads on 4, window 1024, 16 sinks   289 us    694 TFLOP/s
//   d 128, 1 x 16 heads on 4, the whole past          598 us   1034 TFLOP/s
//   d 64,  2 x 16 heads on 4, window 1024, 16 sinks   254 us    395 TFLOP/s
//   d 64,  1 x 16 heads on 4, the whole past          551 us    561 TFLOP/s
// and a padded batch (lengths 4099, 2300, 1200, 1; 16 heads on 4, d 128, window 1024) 105 us.  The tile of
// the sinks is a whole step for its few live keys: in turns, on a card warm from the backward, 307 us with
// 16 sinks and 281 without at d 128, 261 and 238 at d 64.
// Bound at d = 64 by the softmax warps: 4400 cycles a pair of tiles, 2050 of them exponentials, the rest
// latencies of two warps a scheduler (TMEM loads and stores, barriers); starting one sub later changes
// nothing.  At d = 128 by the chain softmax -> P V -> S of a sub, 4900 cycles a step, 1800 of them waiting
// for the products, which the other sub's share the tensor core with.  S of a step's first 64 keys ahead of
// P V, into the columns that P leaves, does not shorten it (307 us): the subs' turns mix again.
#include <type_traits>

#include "kernels.h"
#include "lm.h"
#include "window_tiles.cuh"

namespace st {
namespace {

constexpr int THREADS = 384;
// registers a thread: 168 at launch; the first warpgroup hands some to the two softmax warpgroups
// (104 + 2 x 200 <= 3 x 168)
#define ST_REGS_DEC "setmaxnreg.dec.sync.aligned.u32 104;"
#define ST_REGS_INC "setmaxnreg.inc.sync.aligned.u32 200;"
constexpr float RESCALE_LOG2 = 8.0f;
constexpr int NU = 4;  // unit ring

template <int DT, int D>
struct Cfg {
    static constexpr uint32_t TB = 128 * D * 2;        // bytes of a tile
    static constexpr int NS = D == 64 ? 4 : 2;         // slots of the K ring and of the V ring
    static constexpr int NQB = D == 64 ? 2 : 1;        // Q buffers (of two subs)
    static constexpr uint32_t OFF_K = NQB * 2 * TB, OFF_V = OFF_K + NS * TB;
    static constexpr uint32_t OFF_STG = OFF_V + NS * TB;  // per softmax warp: 32 rows of 64 columns of O
    static constexpr uint32_t OFF_BAR = OFF_STG + 8 * 4096;
    static constexpr uint32_t SMEM = OFF_BAR + 1024;
    static constexpr bool OWN_P = D == 64;             // P has columns of its own
    static constexpr uint32_t COL_O = 256, COL_P = 384;  // S_x at 128 x, O_x at 256 + D x, own P_x at 384 + 64 x
    // fp16 weights are kept 2^6 larger: small ones stay normal numbers, and 2^(8 + 6) is in range
    static constexpr float BIAS = DT == ST_FP16 ? 6.f : 0.f;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

// Tiles of one sub: 0 .. ns - 1, then kb0 .. kb1 (none if !any).
struct Sub {
    int32_t head, row0, kb0, kb1, ns, any;
};

struct Unit {
    int32_t b, len;
    int32_t kb0, ns, steps;  // tiles of either sub, in the order they are loaded: 0 .. ns - 1, then kb0 ..
    int32_t valid;           // 0: no more units
    Sub s[2];
};
static_assert(sizeof(Unit) <= 80, "unit slot");

struct Bars {
    uint64_t q_full[2], q_empty[2], k_full[4], k_empty[4], v_full[4], v_empty[4], u_full[NU], u_empty[NU];
    uint64_t s_full[2], s_free[2], p_full[2], pv_done[2], o_done[2], o_free[2], mma_idle[2];
    uint32_t tmem_base;
    int32_t abort;
    int32_t turn;            // 1 while an issuer holds the tensor core's queue
    uint32_t steps[8];       // flags of step s at s % 8, there with its K tile
    Unit units[NU];
};
static_assert(sizeof(Bars) <= 1024, "barrier block");

// Units of a batch element and row tile (pair of row tiles).
__device__ __forceinline__ int32_t unit_cols(const WindowFwdParams &p) { return p.pair_rows ? p.g.heads : p.g.heads / 2; }

// The unit of row tile (or pair) rt and heads c of batch element b.
__device__ __forceinline__ void make_unit(const WindowFwdParams &p, int32_t b, int32_t rt, int32_t h, Unit &U)
{
    const WindowGeom &g = p.g;
    U.valid = 1;
    U.b = b;
    U.len = window_len(g, b);
    KeyRange r[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int32_t row0 = (p.pair_rows ? 2 * rt + x : rt) * 128;
        r[x] = key_range(g, row0, U.len);
        U.s[x] = {p.pair_rows ? h : 2 * h + x, row0, r[x].kb0, r[x].kb1, r[x].ns, r[x].any ? 1 : 0};
    }
    U.steps = U.ns = U.kb0 = 0;
    if (r[0].any || r[1].any) {
        U.kb0 = !r[1].any ? r[0].kb0 : (!r[0].any ? r[1].kb0 : min(r[0].kb0, r[1].kb0));
        const int32_t kb1 = max(r[0].kb1, r[1].kb1);
        U.ns = min(max(r[0].ns, r[1].ns), U.kb0);
        U.steps = U.ns + kb1 - U.kb0 + 1;
    }
}

// The units with live rows, as one CTA takes them: 32 batch elements at a time, last row tiles (the longest
// units) first, dealt out there and back over the CTAs.  Padding is left out before they are dealt, so
// that a batch of different lengths spreads evenly.  A warp walks them together.
struct LiveUnits {
    int32_t b0 = -32, tiles = 0;         // batch elements b0 ..; lane: live row tiles (or pairs) of b0 + lane
    int32_t rt = 0, base = 0, count = 0; // the row tile walked, units before it, its units
    int32_t k = 0;

    __device__ bool next(const WindowFwdParams &p, Unit &U)
    {
        const WindowGeom &g = p.g;
        const int lane = threadIdx.x & 31;
        const int32_t cols = unit_cols(p);
        const int64_t at = static_cast<int64_t>(k) * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        ++k;
        U.valid = 0;
        while (at >= static_cast<int64_t>(base) + count) {
            base += count;
            if (--rt < 0) {
                b0 += 32;
                if (b0 >= g.batch) return false;
                const int32_t b = b0 + lane, rows = b < g.batch ? min(g.nq, window_len(g, b) - g.q_start) : 0;
                tiles = rows > 0 ? (rows + 127) / 128 : 0;
                if (p.pair_rows) tiles = (tiles + 1) / 2;
                rt = __reduce_max_sync(0xffffffffu, tiles) - 1;
            }
            count = __popc(__ballot_sync(0xffffffffu, tiles > rt && rt >= 0)) * cols;
        }
        const int32_t x = static_cast<int32_t>(at - base), nth = x / cols;
        const uint32_t set = __ballot_sync(0xffffffffu, tiles > rt);
        const uint32_t it = __ballot_sync(0xffffffffu, tiles > rt && __popc(set & ((1u << lane) - 1u)) == nth);
        make_unit(p, b0 + __ffs(it) - 1, rt, x - nth * cols, U);
        return true;
    }
};

// Flags of a step: sub x reads the tile, it is the sub's first or last tile of the unit; the unit's
// first or last step; no more steps.
enum : uint32_t { F_ACT = 1, F_FIRST = 4, F_LAST = 16, F_UNIT = 64, F_DONE = 128, F_END = 256 };

__device__ __forceinline__ uint32_t step_flags(const Unit &U, int32_t step, int32_t tile)
{
    uint32_t f = (step == 0 ? F_UNIT : 0u) | (step + 1 == U.steps ? F_DONE : 0u);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const Sub &r = U.s[x];
        if (!r.any || !(tile < r.ns || (tile >= r.kb0 && tile <= r.kb1))) continue;
        f |= F_ACT << x;
        if (tile == (r.ns > 0 ? 0 : r.kb0)) f |= F_FIRST << x;
        if (tile == r.kb1) f |= F_LAST << x;
    }
    return f;
}

__device__ __forceinline__ float max32(const uint32_t (&v)[32])
{
    float a[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] = fmaxf(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
#pragma unroll
    for (int c = 8; c < 32; c += 2) a[(c >> 1) & 3] = max3f(a[(c >> 1) & 3], __uint_as_float(v[c]), __uint_as_float(v[c + 1]));
    return max3f(a[0], a[1], fmaxf(a[2], a[3]));
}

// p = 2^(s sc + nb) of 32 scores: their sums into ps, packed pairs into pk[at ..].
template <int DT>
__device__ __forceinline__ void weights(const uint32_t (&v)[32], float sc, float nb, float (&ps)[4], uint32_t (&pk)[32], int at)
{
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        float x0, x1;
        f32x2_split(fma2(f32x2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), f32x2(sc, sc), f32x2(nb, nb)), x0, x1);
        const float p0 = ex2(x0), p1 = ex2(x1);
        f32x2_split(add2(f32x2(ps[e & 2], ps[(e & 2) + 1]), f32x2(p0, p1)), ps[e & 2], ps[(e & 2) + 1]);
        pk[at + (e >> 1)] = pack16<DT>(p0, p1);
    }
}

template <int DT, int D>
__global__ void __launch_bounds__(THREADS, 1) window_fwd_kernel(const __grid_constant__ WindowFwdParams p)
{
    using C = Cfg<DT, D>;
    constexpr int NS = C::NS, NQB = C::NQB;
    constexpr uint32_t TB = C::TB;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Bars *bars = reinterpret_cast<Bars *>(smem + C::OFF_BAR);
    volatile int32_t *abort = &bars->abort;
    int32_t *err = p.g.err;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->q_full[i], 1);
            mbar_init(&bars->q_empty[i], 2);  // the two issuers, as for K and V
            mbar_init(&bars->s_full[i], 1);
            mbar_init(&bars->s_free[i], 4);
            mbar_init(&bars->p_full[i], 128);
            mbar_init(&bars->pv_done[i], 1);
            mbar_init(&bars->o_done[i], 1);
            mbar_init(&bars->o_free[i], 128);
            mbar_init(&bars->mma_idle[i], 1);
        }
        for (int i = 0; i < NS; ++i) {
            mbar_init(&bars->k_full[i], 1);
            mbar_init(&bars->k_empty[i], 2);
            mbar_init(&bars->v_full[i], 1);
            mbar_init(&bars->v_empty[i], 2);
        }
        for (int i = 0; i < NU; ++i) {
            mbar_init(&bars->u_full[i], 1);
            mbar_init(&bars->u_empty[i], 8);  // the softmax warps
        }
        bars->turn = 0;
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

    // Steps are counted over all units of the CTA: K and V of step t use slot t % NS for the (t / NS)-th
    // time.
    if (warp < 4) asm volatile(ST_REGS_DEC);
    if (warp == 0) {
        if (run) {
            if (lane == 0) {
                tma_prefetch(&p.q);
                tma_prefetch(&p.k);
                tma_prefetch(&p.v);
            }
            int32_t tk = 0, tv = 0, uq = 0;  // K tiles, V tiles, units with steps so far
            bool ok = true;
            auto wait = [&](uint64_t *bar, int32_t n) { return __all_sync(0xffffffffu, mbar_wait(bar, n & 1, abort, err)); };
            Unit U;
            LiveUnits units;
            for (int32_t k = 0; ok; ++k) {
                const bool more = units.next(p, U);
                if (k >= NU && !(ok = wait(&bars->u_empty[k % NU], k / NU - 1))) break;
                if (lane == 0) {
                    bars->units[k % NU] = U;
                    mbar_arrive(&bars->u_full[k % NU]);
                }
                if (!more) break;
                const int qb = uq % NQB;
                if (uq >= NQB && !(ok = wait(&bars->q_empty[qb], uq / NQB - 1))) break;
                ++uq;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bars->q_full[qb], (U.s[0].any + U.s[1].any) * TB);
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        if (U.s[x].any)
                            tma_tile<D>(&p.q, smem + (2 * qb + x) * TB, &bars->q_full[qb], U.s[x].row0, U.s[x].head, U.b);
                }
                __syncwarp();
                const int32_t hk = U.s[0].head / p.g.group;
                for (int32_t s = 0; s < U.steps; ++s) {
                    const int32_t tile = s < U.ns ? s : U.kb0 + s - U.ns, row = tile * 128;
                    const int sk = tk % NS, sv = tv % NS;
                    if (tk >= NS && !(ok = wait(&bars->k_empty[sk], tk / NS - 1))) break;
                    if (lane == 0) {
                        bars->steps[tk & 7] = step_flags(U, s, tile);
                        mbar_arrive_expect_tx(&bars->k_full[sk], TB);
                        tma_tile<D>(&p.k, smem + C::OFF_K + sk * TB, &bars->k_full[sk], row, hk, U.b);
                    }
                    __syncwarp();
                    ++tk;
                    if (tv >= NS && !(ok = wait(&bars->v_empty[sv], tv / NS - 1))) break;
                    uint8_t *dst = smem + C::OFF_V + sv * TB;
                    if (row + 128 > U.len && U.len < p.g.nk) {
                        load_tile_rows<D>(p.vraw.p + U.b * p.vraw.batch + hk * p.vraw.head + row * p.vraw.row, p.vraw.row,
                                          U.len - row, dst);
                        if (lane == 0) mbar_arrive(&bars->v_full[sv]);
                    } else if (lane == 0) {
                        mbar_arrive_expect_tx(&bars->v_full[sv], TB);
                        tma_tile<D>(&p.v, dst, &bars->v_full[sv], row, hk, U.b);
                    }
                    __syncwarp();
                    ++tv;
                }
            }
            if (ok && (tk < NS || wait(&bars->k_empty[tk % NS], tk / NS - 1))) {  // the step after the last
                if (lane == 0) {
                    bars->steps[tk & 7] = F_END;
                    mbar_arrive(&bars->k_full[tk % NS]);
                }
            }
            if (*abort) {  // drain the copies in flight before the CTA leaves
                volatile int32_t never = 0;
                for (int32_t i = (uq > NQB ? uq - NQB : 0); i < uq; ++i) mbar_wait(&bars->q_full[i % NQB], (i / NQB) & 1, &never, err);
                for (int32_t i = (tk > NS ? tk - NS : 0); i < tk; ++i) mbar_wait(&bars->k_full[i % NS], (i / NS) & 1, &never, err);
                for (int32_t i = (tv > NS ? tv - NS : 0); i < tv; ++i) mbar_wait(&bars->v_full[i % NS], (i / NS) & 1, &never, err);
            }
        }
    } else if (warp < 3) {
        if (lane == 0 && run) {  // (the warp walking and one lane elected to issue: 3% slower here)
            const int x = warp - 1;
            constexpr uint32_t idS = idesc16<DT>(128, 128, false, false), idO = idesc16<DT>(128, D, false, true);
            const uint32_t tS = tbase + 128 * x, tO = tbase + C::COL_O + D * x, tP = C::OWN_P ? tbase + C::COL_P + 64 * x : tS;
            const uint32_t act = F_ACT << x;
            int32_t nS = 0, nP = 0, nO = 0;  // S issued, P V issued, O begun
            int32_t uq = -1;                 // unit of the step last taken
            bool ok = true;
            // flags of step t, once its K (and a new unit's Q) has landed
            auto take = [&](int32_t t) {
                if (!mbar_wait(&bars->k_full[t % NS], (t / NS) & 1, abort, err)) {
                    ok = false;
                    return static_cast<uint32_t>(F_END);
                }
                const uint32_t f = *reinterpret_cast<volatile uint32_t *>(&bars->steps[t & 7]);
                if (f & F_UNIT) {
                    ++uq;
                    ok = mbar_wait(&bars->q_full[uq % NQB], (uq / NQB) & 1, abort, err);
                }
                return f;
            };
            // One issuer's products of a step go into the queue together.  Interleaved with the other's they
            // would end at the same time, and both subs' softmax would then run, and wait, together.
            auto lock = [&]() {
                uint64_t t0 = 0;
                for (uint32_t it = 0; atomicCAS_block(&bars->turn, 0, 1) != 0; ++it) {
                    if (*abort) return false;
                    if ((it & 255u) == 255u) {
                        if (t0 == 0) t0 = globaltimer();
                        else if (globaltimer() - t0 > WAIT_NS) {
                            *abort = 1;
                            atomicOr(err, ERR_TIMEOUT);
                            return false;
                        }
                    }
                }
                return true;
            };
            // S of step t; its columns are free: the softmax holds the last S (own P), or P V went ahead
            auto issue_s = [&](int32_t t) {
                const uint32_t sQ = smem_u32(smem + (2 * (uq % NQB) + x) * TB), sK = smem_u32(smem + C::OFF_K + (t % NS) * TB);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_bf16_ss(tS, Tile<D>::kmajor(sQ, k), Tile<D>::kmajor(sK, k), idS, k > 0 ? 1u : 0u);
            };
            // S of step t (flags f) is issued, or not this sub's: give back its share of K and Q
            auto end_s = [&](int32_t t, uint32_t f) {
                if (f & act) {
                    mma_commit(&bars->s_full[x]);
                    mma_commit(&bars->k_empty[t % NS]);
                    ++nS;
                } else {
                    mbar_arrive(&bars->k_empty[t % NS]);
                }
                if (f & F_DONE) mma_commit(&bars->q_empty[uq % NQB]);
            };
            // V of step t, the unit before read out of O, and P
            auto p_ready = [&](int32_t t, uint32_t f) {
                return mbar_wait(&bars->v_full[t % NS], (t / NS) & 1, abort, err) &&
                       (!(f & act) || ((!(f & (F_FIRST << x)) || nO == 0 || mbar_wait(&bars->o_free[x], (nO - 1) & 1, abort, err)) &&
                                       mbar_wait(&bars->p_full[x], nP & 1, abort, err)));
            };
            auto issue_pv = [&](int32_t t, bool first) {
                const uint32_t sV = smem_u32(smem + C::OFF_V + (t % NS) * TB);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma_bf16_ts(tO, tP + 8 * k, Tile<D>::mnmajor(sV, k), idO, (!first || k > 0) ? 1u : 0u);
            };
            auto end_pv = [&](int32_t t, uint32_t f) {
                if (!(f & act)) {
                    mbar_arrive(&bars->v_empty[t % NS]);
                    return;
                }
                if (C::OWN_P) mma_commit(&bars->pv_done[x]);
                if (f & (F_LAST << x)) mma_commit(&bars->o_done[x]);
                mma_commit(&bars->v_empty[t % NS]);
                ++nP;
                if (f & (F_FIRST << x)) ++nO;
            };
            uint32_t cur = take(0);
            if (ok && !(cur & F_END)) {
                tc_fence_after();
                if (cur & act) issue_s(0);
                end_s(0, cur);
            }
            for (int32_t t = 0; ok && !(cur & F_END); ++t) {
                const uint32_t next = take(t + 1);
                if (!ok) break;
                if (C::OWN_P) {
                    if (next & act) {
                        if (nS > 0 && !mbar_wait(&bars->s_free[x], (nS - 1) & 1, abort, err)) break;
                        tc_fence_after();
                        issue_s(t + 1);
                    }
                    if (!(next & F_END)) end_s(t + 1, next);
                    if (!p_ready(t, cur)) break;
                    tc_fence_after();
                    if (cur & act) issue_pv(t, cur & (F_FIRST << x));
                    end_pv(t, cur);
                } else {
                    if (!p_ready(t, cur)) break;
                    const bool hold = cur & act;
                    if (hold && !lock()) break;
                    tc_fence_after();
                    if (hold) issue_pv(t, cur & (F_FIRST << x));
                    if (next & act) issue_s(t + 1);
                    if (hold) atomicExch_block(&bars->turn, 0);
                    if (!(next & F_END)) end_s(t + 1, next);
                    end_pv(t, cur);
                }
                cur = next;
            }
            mma_commit(&bars->mma_idle[x]);  // no product may run when TMEM is released
            volatile int32_t never = 0;
            mbar_wait(&bars->mma_idle[x], 0, &never, err);
        }
    } else if (warp == 3) {
        // O = 0, lse = -inf of the units without steps.  They never enter the ring: the issuers look one step
        // ahead and must not wait for a step that is behind several units that only the softmax warps,
        // which wait for the issuers, could take.
        Unit U;
        const int32_t cols = unit_cols(p), n = cols * p.g.batch;
        for (int64_t at = blockIdx.x; at < p.units; at += gridDim.x) {
            const int32_t u = static_cast<int32_t>(at), rt = u / n, b = (u - rt * n) / cols;
            make_unit(p, b, rt, u - rt * n - b * cols, U);
            if (U.steps != 0) continue;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const Sub &r = U.s[x];
                const int32_t rows = min(128, p.g.nq - r.row0);
                char *o = p.o + U.b * p.o_batch + r.head * p.o_head + r.row0 * p.o_row;
                float *lse = p.lse + (static_cast<int64_t>(U.b) * p.g.heads + r.head) * p.g.nq + r.row0;
                for (int32_t j = lane; j < rows * (D / 8); j += 32)
                    *reinterpret_cast<uint4 *>(o + j / (D / 8) * p.o_row + 16 * (j % (D / 8))) = make_uint4(0u, 0u, 0u, 0u);
                for (int32_t j = lane; j < rows; j += 32) lse[j] = -INFINITY;
            }
        }
    } else if (warp >= 4) {
        asm volatile(ST_REGS_INC);
        const int x = (warp - 4) >> 2, q4 = warp & 3;  // sub; TMEM lane quarter
        const int row = q4 * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
        const uint32_t tS = tbase + lane_off + 128 * x, tO = tbase + lane_off + C::COL_O + D * x;
        const uint32_t tP = C::OWN_P ? tbase + lane_off + C::COL_P + 64 * x : tS;
        const uint32_t stg = smem_u32(smem + C::OFF_STG + (warp - 4) * 4096);
        const float sc = p.g.scale_log2;
        bool ok = run;
        int32_t nS = 0, nO = 0;
        auto wait_all = [&](uint64_t *bar, int32_t n) {
            if (!__all_sync(0xffffffffu, mbar_wait(bar, n & 1, abort, err))) return false;
            tc_fence_after();
            return true;
        };
        // The unit whose O is still to be written: batch, head, first row; this row's l and m (l = 0: a
        // padding row).
        struct Pending {
            int32_t b, head, row0;
            float l, m;
        } e{};
        bool pending = false;
        // O / l and lse of the pending unit (or zeros: a sub without live rows has no O), 64 columns at a
        // time through the warp's staging
        auto epilogue = [&](bool has_o) {
            if (has_o && !wait_all(&bars->o_done[x], nO)) return false;
            const bool none = e.l == 0.f;  // (a NaN, from a score that is one or +inf, goes through)
            const float inv = none ? 0.f : 1.f / e.l;
            const int32_t r0 = e.row0 + 32 * q4, rows = *abort == 0 ? p.g.nq - r0 : 0;  // rows to write
            char *dst0 = p.o + e.b * p.o_batch + e.head * p.o_head + (r0 + (lane >> 3)) * p.o_row + 16 * (lane & 7);
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                __syncwarp();  // the staging has been read
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t o[32];
                    if (has_o) {
                        tmem_ld32(tO + 64 * h + 32 * c, o);
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float a[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) a[i] = has_o ? __uint_as_float(o[8 * q + i]) * inv : 0.f;
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[i] = none ? 0u : pack16<DT>(a[2 * i], a[2 * i + 1]);
                        st_shared_v4(stg + sw128_off(lane, 4 * c + q), w[0], w[1], w[2], w[3]);
                    }
                }
                __syncwarp();
                // whole row pieces of 128 bytes, four rows a warp store
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int i = 4 * j + (lane >> 3);
                    const uint4 y = ld_shared_v4(stg + sw128_off(i, lane & 7));
                    if (i < rows) *reinterpret_cast<uint4 *>(dst0 + 128 * h + 4 * j * p.o_row) = y;
                }
            }
            if (has_o) {
                ++nO;
                tc_fence_before();
                mbar_arrive(&bars->o_free[x]);
            }
            if (lane < rows)
                p.lse[(static_cast<int64_t>(e.b) * p.g.heads + e.head) * p.g.nq + e.row0 + row] =
                    none ? -INFINITY : (e.m - C::BIAS + lg2(e.l)) * LN2;
            pending = false;
            return true;
        };
        for (int32_t k = 0; ok; ++k) {
            if (!(ok = wait_all(&bars->u_full[k % NU], k / NU))) break;
            const Unit &U = bars->units[k % NU];
            const bool valid = U.valid != 0;
            const int32_t batch = U.b, len = U.len;
            const Sub r = U.s[x];
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->u_empty[k % NU]);
            if (!valid) break;
            if (!r.any) {  // no live row (also: no row at all)
                if (pending && !(ok = epilogue(true))) break;
                e = Pending{batch, r.head, r.row0, 0.f, 0.f};
                epilogue(false);
                continue;
            }
            const int32_t i = r.row0 + row, pos = p.g.q_start + i;
            const bool live = i < p.g.nq && pos < len;
            float m = -INFINITY, l = 0.f;
            for (int32_t tile = r.ns > 0 ? 0 : r.kb0;; tile = tile + 1 == r.ns ? r.kb0 : tile + 1) {
                if (!(ok = wait_all(&bars->s_full[x], nS))) break;
                const int32_t base = tile * 128;
                const bool whole = live && base + 127 <= pos && (p.g.window == 0 || base > pos - p.g.window || base + 128 <= p.g.sinks);
                // The exponentials of a 32-column piece are taken with the maximum so far while the next
                // pieces load and their maxima are found: once the last piece is in registers the tile's
                // maximum is known, and if it is more than 2^8 larger (or the first), the tile is read
                // again with the new one.  Until then nothing has overwritten it.
                float alpha = 1.f, ps[4];
                uint32_t v0[32], v1[32], v2[32], pk[32];
                auto first_half = [&](auto masked) {
                    uint32_t kw[4];  // columns this row sees
                    if constexpr (decltype(masked)::value) {
                        const uint64_t b0 = live ? window_bits64(pos, p.g.window, p.g.sinks, base) : 0ull;
                        const uint64_t b1 = live ? window_bits64(pos, p.g.window, p.g.sinks, base + 64) : 0ull;
                        kw[0] = static_cast<uint32_t>(b0);
                        kw[1] = static_cast<uint32_t>(b0 >> 32);
                        kw[2] = static_cast<uint32_t>(b1);
                        kw[3] = static_cast<uint32_t>(b1 >> 32);
                    }
                    auto mask = [&](uint32_t (&v)[32], int c) {
                        if constexpr (decltype(masked)::value) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = (kw[c] & (1u << e)) ? v[e] : 0xFF800000u;
                        }
                    };
                    bool seek = __any_sync(0xffffffffu, m == -INFINITY);
                    for (;;) {
                        float mt = -INFINITY;
                        if (seek) {
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                tmem_ld32(tS + 32 * c, v0);
                                tmem_wait_ld();
                                mask(v0, c);
                                mt = fmaxf(mt, max32(v0));
                            }
                            const float m_new = fmaxf(m, mt * sc);
                            if (m_new > m + RESCALE_LOG2) {  // also the first finite maximum
                                alpha *= ex2(m - m_new);
                                m = m_new;
                            }
                        }
                        const float nb = (m == -INFINITY) ? 0.f : C::BIAS - m;
                        ps[0] = ps[1] = ps[2] = ps[3] = 0.f;
                        tmem_ld32(tS, v0);
                        tmem_wait_ld();
                        tmem_ld32(tS + 32, v1);
                        mask(v0, 0);
                        mt = max32(v0);
                        tmem_wait_ld();
                        tmem_ld32(tS + 64, v2);
                        mask(v1, 1);
                        mt = fmaxf(mt, max32(v1));
                        weights<DT>(v0, sc, nb, ps, pk, 0);
                        tmem_wait_ld();
                        tmem_ld32(tS + 96, v0);
                        mask(v2, 2);
                        mt = fmaxf(mt, max32(v2));
                        weights<DT>(v1, sc, nb, ps, pk, 16);
                        tmem_wait_ld();
                        mask(v0, 3);
                        mt = fmaxf(mt, max32(v0));
                        if (!__any_sync(0xffffffffu, mt * sc > m + RESCALE_LOG2)) break;
                        seek = true;
                    }
                };
                // (one straight piece of code for the tiles that need no mask, three in four and more)
                if (__all_sync(0xffffffffu, whole)) first_half(std::false_type());
                else first_half(std::true_type());
                if (C::OWN_P) {  // S is no longer needed
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->s_free[x]);
                }
                if (pending && !(ok = epilogue(true))) break;  // the unit before, while its last product ran
                // O and own P: the last product is complete (with P over S, S(t) complete says so)
                if (C::OWN_P && nS > 0 && !(ok = wait_all(&bars->pv_done[x], nS - 1))) break;
                if (__any_sync(0xffffffffu, alpha != 1.f && l > 0.f)) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(tO + 32 * c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * alpha);
                        tmem_st32(tO + 32 * c, o);
                    }
                }
                tmem_st32(tP, pk);
                const float nb = (m == -INFINITY) ? 0.f : C::BIAS - m;
                weights<DT>(v2, sc, nb, ps, pk, 0);
                weights<DT>(v0, sc, nb, ps, pk, 16);
                tmem_st32(tP + 32, pk);
                tmem_wait_st();
                l = l * alpha + ((ps[0] + ps[1]) + (ps[2] + ps[3]));
                ++nS;
                tc_fence_before();
                mbar_arrive(&bars->p_full[x]);
                if (tile == r.kb1) break;
            }
            if (!ok) break;
            e = Pending{batch, r.head, r.row0, live ? l : 0.f, m};
            pending = true;
        }
        if (ok && pending) epilogue(true);
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
