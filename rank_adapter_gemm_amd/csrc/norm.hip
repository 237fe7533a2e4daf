// The step between two blocks: z = x + residual, y = z / sqrt(mean(z^2) + eps)
// * weight per row, and, for the FP8 base, the E4M3 codes and power-of-two
// scale of y's rows, so that the projections that follow need not read y
// again to quantize it.
//
// One pass over the data: a row is read once into registers (fp32), its sum
// of squares (and, for the codes, its largest rounded |y|) reduced across its
// threads, and every output written from the registers.  The sum z keeps its
// 32 bits for the norm; only what is stored is rounded, once per output.  The
// codes are those of y as stored (rounded to bf16), so they are bitwise what
// lora_quantize_rows_fp8 gives for it.
//
// Bound by its bytes (34811 x 4096 with codes, 1.28 GB: 226 us, 5.7 TB/s, more
// than a plain copy of 1 GiB reaches) and, for few rows, by one trip to memory
// and back: a row has as many threads as give each one or two of its 16-byte
// vectors, so that all of it is in flight at once (one row of 4096: 2.2 us).
#include "common.hpp"
#include "fp8_common.hpp"

namespace lora {

struct norm_args {
    const void *x, *residual, *weight;   // residual may be null
    void *residual_out, *y;              // each may be null (y only with codes)
    uint8_t *yq;                         // codes [T][d], with the scales
    float *ys;                           // scales [T]
    float eps, inv_d;
    int32_t T, d;
};

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

template <int DT>
__device__ __forceinline__ void load_z(const norm_args &a, int64_t at, float *z) {
    constexpr int VN = vec16<DT>::n;
    typedef typename elem<DT>::T E;
    vec16<DT>::widen(ldg16((const E *)a.x + at), z);
    if (a.residual) {
        float r[VN];
        vec16<DT>::widen(ldg16((const E *)a.residual + at), r);
#pragma unroll
        for (int i = 0; i < VN; ++i) z[i] += r[i];
    }
}

// The rounded y of one vector, as stored (and back in fp32 for the codes).
template <int DT>
__device__ __forceinline__ uint4 norm_vec(const float *z, float inv, const uint4 &wq, float *yr) {
    constexpr int VN = vec16<DT>::n;
    float w[VN], o[VN];
    vec16<DT>::widen(wq, w);
#pragma unroll
    for (int i = 0; i < VN; ++i) o[i] = z[i] * inv * w[i];
    const uint4 q = vec16<DT>::narrow(o);
    vec16<DT>::widen(q, yr);
    return q;
}

__device__ __forceinline__ uint2 codes_of(const float *yr, float inv) {
    return make_uint2(e4m3x4(yr[0] * inv, yr[1] * inv, yr[2] * inv, yr[3] * inv),
                      e4m3x4(yr[4] * inv, yr[5] * inv, yr[6] * inv, yr[7] * inv));
}

// NT threads per row, VPT 16-byte vectors of the row in each thread's
// registers; 256 / NT rows per workgroup where NT < 256.  VPT = 0: rows wider
// than the registers hold are read again for each pass (from cache), and
// written in the last pass only, so outputs may be the inputs' own buffers
// in either form.
template <int DT, int NT, int VPT, bool Q8>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT) k_add_rmsnorm(norm_args a) {
    static_assert(!Q8 || DT == LORA_BF16, "codes are of bf16 rows");
    static_assert(NT >= 256 || NT == 64, "a workgroup holds one row, or a row per wavefront");
    typedef typename elem<DT>::T E;
    constexpr int VN = vec16<DT>::n, RPB = NT < 256 ? 256 / NT : 1, W = NT / 64;
    __shared__ float red[2][W];
    const int tid = threadIdx.x % NT, lane = tid & 63, wave = tid >> 6;
    const int nvec = a.d / VN;
    for (int64_t t = (int64_t)blockIdx.x * RPB + threadIdx.x / NT; t < a.T; t += (int64_t)gridDim.x * RPB) {
        const int64_t row = t * a.d;
        float ss = 0.0f;
        if constexpr (VPT > 0) {
            float z[VPT][VN];
            uint4 wq[VPT];
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int c = tid + v * NT;
                if (c < nvec) {
                    load_z<DT>(a, row + (int64_t)c * VN, z[v]);
                    wq[v] = ldg16((const E *)a.weight + c * VN);
                }
            }
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int c = tid + v * NT;
                if (c < nvec) {
#pragma unroll
                    for (int i = 0; i < VN; ++i) ss = fmaf(z[v][i], z[v][i], ss);
                    if (a.residual_out) stg16((E *)a.residual_out + row + (int64_t)c * VN, vec16<DT>::narrow(z[v]));
                }
            }
            const float inv = 1.0f / sqrtf(row_reduce<NT, false>(ss, red, 0, lane, wave) * a.inv_d + a.eps);
            float m = 0.0f;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int c = tid + v * NT;
                if (c < nvec) {
                    const uint4 q = norm_vec<DT>(z[v], inv, wq[v], z[v]);
                    if (a.y) stg16((E *)a.y + row + (int64_t)c * VN, q);
#pragma unroll
                    for (int i = 0; i < VN; ++i) m = fmaxf(m, fabsf(z[v][i]));
                }
            }
            if constexpr (Q8) {
                const int e = scale_exp(row_reduce<NT, true>(m, red, 1, lane, wave));
                const float qi = exp2i(-e);
                if (tid == 0) a.ys[t] = exp2i(e);
#pragma unroll
                for (int v = 0; v < VPT; ++v) {
                    const int c = tid + v * NT;
                    if (c < nvec) *reinterpret_cast<uint2 *>(a.yq + row + (int64_t)c * 8) = codes_of(z[v], qi);
                }
            }
        } else {
            float z[VN];
            for (int c = tid; c < nvec; c += NT) {
                load_z<DT>(a, row + (int64_t)c * VN, z);
#pragma unroll
                for (int i = 0; i < VN; ++i) ss = fmaf(z[i], z[i], ss);
            }
            const float inv = 1.0f / sqrtf(row_reduce<NT, false>(ss, red, 0, lane, wave) * a.inv_d + a.eps);
            float qi = 0.0f;
            if constexpr (Q8) {
                float m = 0.0f;
                for (int c = tid; c < nvec; c += NT) {
                    load_z<DT>(a, row + (int64_t)c * VN, z);
                    norm_vec<DT>(z, inv, ldg16((const E *)a.weight + c * VN), z);
#pragma unroll
                    for (int i = 0; i < VN; ++i) m = fmaxf(m, fabsf(z[i]));
                }
                const int e = scale_exp(row_reduce<NT, true>(m, red, 1, lane, wave));
                qi = exp2i(-e);
                if (tid == 0) a.ys[t] = exp2i(e);
            }
            for (int c = tid; c < nvec; c += NT) {
                load_z<DT>(a, row + (int64_t)c * VN, z);
                if (a.residual_out) stg16((E *)a.residual_out + row + (int64_t)c * VN, vec16<DT>::narrow(z));
                const uint4 q = norm_vec<DT>(z, inv, ldg16((const E *)a.weight + c * VN), z);
                if (a.y) stg16((E *)a.y + row + (int64_t)c * VN, q);
                if constexpr (Q8) *reinterpret_cast<uint2 *>(a.yq + row + (int64_t)c * 8) = codes_of(z, qi);
            }
        }
        if constexpr (NT > 64) __syncthreads();          // `red` is reused by the next row
    }
}

template <int DT, bool Q8>
static lora_status_t launch_norm(const norm_args &a, hipStream_t s) {
    const int nvec = a.d / vec16<DT>::n;
    // A grid of at most 2^20 workgroups; each goes on to further rows.
    const int64_t cap = 1 << 20;
#define LORA_NORM(NTV, VPTV)                                                                            \
    do {                                                                                                \
        const int64_t rpb = NTV < 256 ? 256 / NTV : 1, n = (a.T + rpb - 1) / rpb;                       \
        hipLaunchKernelGGL((k_add_rmsnorm<DT, NTV, VPTV, Q8>), dim3((uint32_t)(n < cap ? n : cap)),     \
                           dim3(NTV < 256 ? 256 : NTV), 0, s, a);                                       \
    } while (0)
    // One vector a thread where nearly all threads have one (512 vectors, 34811
    // rows with codes 226 us and one row 2.2, with two a thread 230 and 2.8, with
    // eight 289 and 5.7), else two (386 vectors of fp32, 1111 rows: 7.0 us, with
    // one 7.7).
    if (nvec <= 64) LORA_NORM(64, 1);
    else if (nvec <= 128) LORA_NORM(64, 2);
    else if (nvec <= 256) LORA_NORM(256, 1);
    else if (nvec <= 448) LORA_NORM(256, 2);
    else if (nvec <= 512) LORA_NORM(512, 1);
    else if (nvec <= 896) LORA_NORM(512, 2);
    else if (nvec <= 1024) LORA_NORM(1024, 1);
    else if (nvec <= 2048) LORA_NORM(1024, 2);
    else if (nvec <= 4096) LORA_NORM(1024, 4);
    else LORA_NORM(1024, 0);
#undef LORA_NORM
    return hip_status(hipGetLastError());
}

lora_status_t launch_add_rmsnorm(const void *x, const void *residual, const void *weight, float eps, int32_t T,
                                 int32_t d, int32_t dtype, void *residual_out, void *y, uint8_t *yq, float *ys,
                                 hipStream_t s) {
    if (T <= 0) return LORA_OK;
    const norm_args a{x, residual, weight, residual_out, y, yq, ys, eps, 1.0f / (float)d, T, d};
    if (yq) return launch_norm<LORA_BF16, true>(a, s);
    return dtype == LORA_F32 ? launch_norm<LORA_F32, false>(a, s) : launch_norm<LORA_BF16, false>(a, s);
}

}  // namespace lora
