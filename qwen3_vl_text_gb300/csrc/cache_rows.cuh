// Eight elements of a head vector: bf16 and e4m3 packing shared by the kernels that fill a cache.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace h3 {

// Eight values divided by `scale` (IEEE division) and rounded to e4m3, saturating.
__device__ __forceinline__ uint2 quant8(const float (&x)[8], float scale) {
    uint32_t w[2];
    #pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 lo = make_float2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale));
        const float2 hi = make_float2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale));
        w[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3) |
               ((uint32_t)__nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3) << 16);
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(u[i]);
        x[2 * i + 1] = bf16_hi(u[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

}  // namespace h3
