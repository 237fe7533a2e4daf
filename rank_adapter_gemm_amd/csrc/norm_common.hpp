// Pieces shared by the norms: a row's reductions, z = x + residual and the FP8
// codes of a vector.
#pragma once

#include "common.hpp"
#include "fp8_common.hpp"

namespace lora {

// Reductions over the NT threads of one row (rows of 64 threads need no LDS).
// `slot` keeps two reductions of one row apart in LDS.
template <int NT, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float (*red)[NT / 64], int slot, int lane, int wave) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const float w = __shfl_xor(v, o, 64);
        v = MAX ? fmaxf(v, w) : v + w;
    }
    if constexpr (NT > 64) {
        if (lane == 0) red[slot][wave] = v;
        __syncthreads();
        v = red[slot][0];
#pragma unroll
        for (int i = 1; i < NT / 64; ++i) v = MAX ? fmaxf(v, red[slot][i]) : v + red[slot][i];
    }
    return v;
}

// z of one vector, in fp32; residual may be null.
template <int DT>
__device__ __forceinline__ void load_z(const void *x, const void *residual, int64_t at, float *z) {
    constexpr int VN = vec16<DT>::n;
    typedef typename elem<DT>::T E;
    vec16<DT>::widen(ldg16((const E *)x + at), z);
    if (residual) {
        float r[VN];
        vec16<DT>::widen(ldg16((const E *)residual + at), r);
#pragma unroll
        for (int i = 0; i < VN; ++i) z[i] += r[i];
    }
}

__device__ __forceinline__ uint2 codes_of(const float *yr, float inv) {
    return make_uint2(e4m3x4(yr[0] * inv, yr[1] * inv, yr[2] * inv, yr[3] * inv),
                      e4m3x4(yr[4] * inv, yr[5] * inv, yr[6] * inv, yr[7] * inv));
}

}  // namespace lora
