// elem.cuh -- 8-element vectors of the three element types, widened to fp32 and rounded back.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/st_attn.h"

namespace st {

// Eight consecutive elements as loaded: one 16-byte load for the 16-bit types, two for fp32.
template <int DT>
struct Vec8 {
    uint4 r[DT == ST_FP32 ? 2 : 1];
};

template <int DT>
__device__ __forceinline__ Vec8<DT> load8(const void *p)
{
    Vec8<DT> v;
    v.r[0] = static_cast<const uint4 *>(p)[0];
    if constexpr (DT == ST_FP32) v.r[1] = static_cast<const uint4 *>(p)[1];
    return v;
}

template <int DT>
__device__ __forceinline__ void store8(void *p, const Vec8<DT> &v)
{
    static_cast<uint4 *>(p)[0] = v.r[0];
    if constexpr (DT == ST_FP32) static_cast<uint4 *>(p)[1] = v.r[1];
}

template <int DT>
__device__ __forceinline__ void widen8(const Vec8<DT> &v, float (&x)[8])
{
    if constexpr (DT == ST_FP32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            x[4 * h] = __uint_as_float(v.r[h].x);
            x[4 * h + 1] = __uint_as_float(v.r[h].y);
            x[4 * h + 2] = __uint_as_float(v.r[h].z);
            x[4 * h + 3] = __uint_as_float(v.r[h].w);
        }
    } else {
        const uint32_t w[4] = {v.r[0].x, v.r[0].y, v.r[0].z, v.r[0].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (DT == ST_BF16) {
                x[2 * e] = __uint_as_float(w[e] << 16);
                x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[e]));
                x[2 * e] = f.x;
                x[2 * e + 1] = f.y;
            }
        }
    }
}

// Two fp32 values as a pair of 16-bit elements (round to nearest even; lo in the low half).
template <int DT>
__device__ __forceinline__ uint32_t pack16(float lo, float hi)
{
    uint32_t r;
    if constexpr (DT == ST_BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int DT>
__device__ __forceinline__ Vec8<DT> round8(const float (&x)[8])
{
    Vec8<DT> v;
    if constexpr (DT == ST_FP32) {
        v.r[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        v.r[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
    } else {
        v.r[0] = make_uint4(pack16<DT>(x[0], x[1]), pack16<DT>(x[2], x[3]), pack16<DT>(x[4], x[5]), pack16<DT>(x[6], x[7]));
    }
    return v;
}

}  // namespace st
