// plan.cu -- block tables and slot maps of one serving step, built on the device.
//
// With a_r = lens[r], b_r = max(new[r], 0), o_r = sum_{i<r} b_i: request r holds ceil(a_r / s) pages of s
// positions and wants ceil((a_r + b_r) / s).  It fits unless a length is negative or a_r + b_r
// leaves 32 bits, it wants more than max_pages or o_r + b_r > tokens; with n_r = pages wanted less held (0 if it does not fit) and
// c_r = sum_{i<r} n_i, it is served when it fits and n_r = 0 or c_r + n_r <= free.  Its i-th new page
// is free_pages[free - 1 - (c_r + i)]: a page depends on prefix sums only, never on another request's
// result, so one launch does it all.
//
// Bound by latency (tens of kilobytes): every CTA computes both prefix sums over all requests for
// itself, in shared memory, which costs less than a second launch or a grid barrier; the tokens and
// the new pages are then dealt out over the CTAs, each finding its request by bisection.
#include "lm.h"
#include "plan.h"

namespace st {
namespace {

constexpr int THREADS = 1024;

// Inclusive prefix sum over the CTA, on top of `carry` (which becomes the total so far).
__device__ __forceinline__ int64_t scan(int64_t x, int64_t &carry, int64_t *warp_sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // the previous scan's sums are no longer read
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int64_t before = carry, all = carry;
#pragma unroll 8
    for (int w = 0; w < THREADS / 32; ++w) {
        const int64_t s = warp_sums[w];
        if (w < warp) before += s;
        all += s;
    }
    carry = all;
    return before + x;
}

// The request r whose run [first[r], first[r + 1]) holds x; first[] rises from 0 past x.
__device__ __forceinline__ int find(const int32_t *first, int n, int64_t x)
{
    int lo = 0, hi = n;  // first[lo] <= x < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int32_t clamp32(int64_t x) { return x > INT32_MAX ? INT32_MAX : static_cast<int32_t>(x); }

__global__ void __launch_bounds__(THREADS) plan_kernel(const __grid_constant__ PlanParams p)
{
    extern __shared__ int32_t sm[];
    __shared__ int64_t warp_sums[THREADS / 32];
    const int R = p.requests;
    int32_t *offset = sm;              // [R + 1] first token
    int32_t *taken = sm + R + 1;       // [R + 1] pages taken by earlier requests (served ones)
    int32_t *asked = sm + 2 * (R + 1); // [R] pages asked for by earlier requests; -1: not served
    const int64_t s = p.page_size;
    int64_t free = *p.free_count;
    free = free < 0 ? 0 : (free > p.free_capacity ? p.free_capacity : free);
    int64_t tok = 0, ask = 0, got = 0;
    for (int base = 0; base < R; base += THREADS) {
        const int r = base + threadIdx.x;
        const bool in = r < R;
        const int64_t a = in ? p.lens[r] : 0, bn = in ? p.new_tokens[r] : 0, b = bn > 0 ? bn : 0;
        const int64_t t1 = scan(b, tok, warp_sums);
        const int64_t held = a > 0 ? (a + s - 1) / s : 0, want = a >= 0 ? (a + b + s - 1) / s : 0;
        const bool fits = in && a >= 0 && bn >= 0 && want <= p.max_pages && t1 <= p.tokens &&
                          a + b <= INT32_MAX;
        const int64_t need = fits ? want - held : 0;
        const int64_t c1 = scan(need, ask, warp_sums);
        const bool served = fits && (need == 0 || c1 <= free);
        const int64_t g1 = scan(served ? need : 0, got, warp_sums);
        if (in) {
            offset[r] = clamp32(t1 - b);
            taken[r] = clamp32(g1 - (served ? need : 0));
            asked[r] = served ? clamp32(c1 - need) : -1;
            if (r == R - 1) {
                offset[R] = clamp32(t1);
                taken[R] = clamp32(g1);
            }
            if (blockIdx.x == 0) {
                p.lens_out[r] = static_cast<int32_t>(served ? a + b : a);
                p.status[r] = served ? 0 : 1;
                p.offsets[r] = clamp32(t1 - b);
                if (r == R - 1) {
                    p.offsets[R] = clamp32(t1);
                    *p.free_left = static_cast<int32_t>(free - g1);
                }
            }
        }
    }
    __syncthreads();
    const int64_t id = static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x, all = static_cast<int64_t>(gridDim.x) * THREADS;
    // new pages into the block tables (columns past those held: no CTA reads them)
    for (int64_t k = id; k < taken[R]; k += all) {
        const int r = find(taken, R, k);
        const int64_t i = k - taken[r], held = (static_cast<int64_t>(p.lens[r]) + s - 1) / s;
        p.block_table[r * p.table_stride + held + i] = p.free_pages[free - 1 - (asked[r] + i)];
    }
    for (int64_t t = id; t < p.tokens; t += all) {
        int32_t slot = -1, pos32 = -1;
        if (t < offset[R]) {
            const int r = find(offset, R, t);
            if (asked[r] >= 0) {
                const int64_t a = p.lens[r], pos = a + (t - offset[r]), held = (a + s - 1) / s, col = pos / s;
                const int64_t page = col < held ? p.block_table[r * p.table_stride + col]
                                                : p.free_pages[free - 1 - (asked[r] + col - held)];
                const int64_t at = page * s + (pos - col * s);
                pos32 = static_cast<int32_t>(pos);
                if (page >= 0 && at <= INT32_MAX) slot = static_cast<int32_t>(at);
            }
        }
        p.slots[t] = slot;
        p.positions[t] = pos32;
    }
}

std::atomic<uint64_t> configured{0};

}  // namespace

cudaError_t launch_plan(const PlanParams &p, cudaStream_t s)
{
    const int smem = 4 * (3 * p.requests + 2);
    cudaError_t e = allow_smem(plan_kernel, 4 * (3 * PLAN_MAX_REQUESTS + 2), configured);
    if (e != cudaSuccess) return e;
    // a CTA for every 4096 tokens (four a thread), 64 at most: each repeats the prefix sums
    int64_t grid = (p.tokens + 4 * THREADS - 1) / (4 * THREADS);
    grid = grid < 1 ? 1 : (grid > 64 ? 64 : grid);
    plan_kernel<<<static_cast<unsigned>(grid), THREADS, smem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace st
