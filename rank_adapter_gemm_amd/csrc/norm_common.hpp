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

// Columns of part [groups][n] added up, in order within each of 16 strands and
// then over the strands: 64 columns a workgroup, 4 a thread.  The first d
// columns go to out0, the rest to out1 (either may be null), in type DT.
template <int DT>
__device__ __forceinline__ void column_sums(const float *part, int32_t groups, int64_t n, int32_t d,
                                            typename elem<DT>::T *out0, typename elem<DT>::T *out1, int64_t block) {
    __shared__ float s[16][64];
    const int strand = threadIdx.x >> 4;
    const int64_t c0 = block * 64, c = c0 + (threadIdx.x & 15) * 4;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < n)
#pragma unroll 8
        for (int g = strand; g < groups; g += 16) {
            const float4 f = *reinterpret_cast<const float4 *>(part + g * n + c);
            sum.x += f.x;
            sum.y += f.y;
            sum.z += f.z;
            sum.w += f.w;
        }
    *reinterpret_cast<float4 *>(&s[strand][(threadIdx.x & 15) * 4]) = sum;
    __syncthreads();
    const int64_t col = c0 + threadIdx.x;
    if (threadIdx.x >= 64 || col >= n) return;
    float f = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) f += s[i][threadIdx.x];
    typename elem<DT>::T *out = col < d ? out0 : out1;
    if (out) elem<DT>::store(out, col < d ? col : col - d, f);
}

}  // namespace lora
