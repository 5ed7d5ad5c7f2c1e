// window_tiles.cuh -- device pieces shared by the sliding-window kernels.
#pragma once
#include "elem.cuh"
#include "sm100.cuh"
#include "tiles.cuh"
#include "window.h"

namespace st {

// Instruction descriptor of kind::f16 with A and B of type DT (format 0: fp16, 1: bf16), fp32 D.
template <int DT>
__host__ __device__ constexpr uint32_t idesc16(int M, int N, bool a_mn, bool b_mn)
{
    const uint32_t f = DT == ST_BF16 ? 1u : 0u;
    return (1u << 4) | (f << 7) | (f << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// One lane of a converged warp, the same at every call.
__device__ __forceinline__ bool elect_one()
{
    uint32_t on;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
    return on != 0;
}

// Expect more bytes in the current phase, without arriving.
__device__ __forceinline__ void mbar_expect_tx(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// One 128-row tile of D columns by TMA (boxes of 64 columns), at row `row` of (head, batch).
template <int D>
__device__ __forceinline__ void tma_tile(const CUtensorMap *m, uint8_t *dst, uint64_t *bar, int32_t row, int32_t head, int32_t batch)
{
#pragma unroll
    for (int b = 0; b < D / 64; ++b) tma_load_4d(dst + b * 16384, m, bar, 64 * b, row, head, batch);
}

// The same tile by the whole warp with plain loads, rows `valid` and beyond as zeros: what lies past
// the end of a sequence (NaN included) must not enter a product, where a zero weight would not
// silence it.  The caller signals the tile's barrier after this.
template <int D>
__device__ __forceinline__ void load_tile_rows(const char *src, int64_t row_stride, int valid, uint8_t *dst)
{
    const int lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(dst);
#pragma unroll 8
    for (int i = lane; i < 128 * (D / 8); i += 32) {
        const int r = i / (D / 8), ch = i % (D / 8);
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (r < valid) x = *reinterpret_cast<const uint4 *>(src + r * row_stride + 16 * ch);
        st_shared_v4(base + (ch >> 3) * 16384 + sw128_off(r, ch & 7), x.x, x.y, x.z, x.w);
    }
    fence_proxy_async_smem();
    __syncwarp();
}

// Columns of a 64-key slice starting at key `base` that the query at position pos sees.
__device__ __forceinline__ uint64_t window_bits64(int32_t pos, int32_t window, int32_t sinks, int32_t base)
{
    const int32_t lo = window ? max(pos - window + 1, 0) : 0, s = min(sinks, pos + 1);
    return interval_bits64(lo - base, pos - base) | interval_bits64(-base, s - 1 - base);
}

}  // namespace st
