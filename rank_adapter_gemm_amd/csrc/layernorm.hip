// The layer norm between two blocks, and its backward pass:
//   z = x + residual,  y = (z - mean(z)) / sqrt(var(z) + eps) * weight + bias
// per row, with y's E4M3 codes and power-of-two scale where an FP8 base weight
// reads it.
//
// Forward: a row is read once into registers (fp32).  The variance is the mean
// of the squares of z - mean, a second reduction over the registers: the
// difference mean(z^2) - mean(z)^2 would lose the variance of rows far from 0.
// What is stored is rounded, once per output; the codes are those of y as stored.
// Bound by its bytes: 12345 x 8192 bf16 with codes, 910 MB, 162 us, 5.6 TB/s; one
// row of 4096 2.9 us, three reductions and a launch.
#include "norm_common.hpp"

namespace lora {

struct layernorm_args {
    const void *x, *residual, *weight, *bias;   // residual, bias: may be null
    void *residual_out, *y;                     // each may be null (y only with codes)
    uint8_t *yq;                                // codes [T][d], with the scales
    float *ys, *mean, *rstd;                    // [T]; mean and rstd may be null
    float eps, inv_d;
    int32_t T, d;
};

// The rounded y of one vector, as stored (and back in fp32 for the codes).
template <int DT>
__device__ __forceinline__ uint4 layernorm_vec(const float *z, float mean, float rstd, const uint4 &wq, const uint4 &bq,
                                               float *yr) {
    constexpr int VN = vec16<DT>::n;
    float w[VN], b[VN], o[VN];
    vec16<DT>::widen(wq, w);
    vec16<DT>::widen(bq, b);
#pragma unroll
    for (int i = 0; i < VN; ++i) o[i] = fmaf((z[i] - mean) * rstd, w[i], b[i]);
    const uint4 q = vec16<DT>::narrow(o);
    vec16<DT>::widen(q, yr);
    return q;
}

// NT threads per row, VPT 16-byte vectors of it in each thread's registers;
// VPT = 0: rows wider than the registers hold are read again for each pass and
// written in the last one only, so that outputs may be the inputs' own buffers
// in either form (as in k_add_rmsnorm).
template <int DT, int NT, int VPT, bool Q8>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT) k_add_layernorm(layernorm_args a) {
    static_assert(!Q8 || DT == LORA_BF16, "codes are of bf16 rows");
    static_assert(NT >= 256 || NT == 64, "a workgroup holds one row, or a row per wavefront");
    typedef typename elem<DT>::T E;
    constexpr int VN = vec16<DT>::n, RPB = NT < 256 ? 256 / NT : 1, W = NT / 64;
    __shared__ float red[3][W];
    const int tid = threadIdx.x % NT, lane = tid & 63, wave = tid >> 6;
    const int nvec = a.d / VN;
    auto load_b = [&](int c) { return a.bias ? ldg16((const E *)a.bias + c * VN) : make_uint4(0u, 0u, 0u, 0u); };
    for (int64_t t = (int64_t)blockIdx.x * RPB + threadIdx.x / NT; t < a.T; t += (int64_t)gridDim.x * RPB) {
        const int64_t row = t * a.d;
        float s = 0.0f, ss = 0.0f, m = 0.0f, qi = 0.0f;
        if constexpr (VPT > 0) {
            constexpr bool AHEAD = VPT <= 2;              // weight and bias with the row (else no register is left for them)
            float z[VPT][VN];
            uint4 wq[AHEAD ? VPT : 1], bq[AHEAD ? VPT : 1];
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int c = tid + v * NT;
                if (c < nvec) {
                    load_z<DT>(a.x, a.residual, row + (int64_t)c * VN, z[v]);
                    if constexpr (AHEAD) {
                        wq[v] = ldg16((const E *)a.weight + c * VN);
                        bq[v] = load_b(c);
                    }
                }
            }
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int c = tid + v * NT;
                if (c < nvec) {
#pragma unroll
                    for (int i = 0; i < VN; ++i) s += z[v][i];
                    if (a.residual_out) stg16((E *)a.residual_out + row + (int64_t)c * VN, vec16<DT>::narrow(z[v]));
                }
            }
            const float mean = row_reduce<NT, false>(s, red, 0, lane, wave) * a.inv_d;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
                if (tid + v * NT < nvec)
#pragma unroll
                    for (int i = 0; i < VN; ++i) ss = fmaf(z[v][i] - mean, z[v][i] - mean, ss);
            const float rstd = 1.0f / sqrtf(row_reduce<NT, false>(ss, red, 1, lane, wave) * a.inv_d + a.eps);
            if (a.mean && tid == 0) {
                a.mean[t] = mean;
                a.rstd[t] = rstd;
            }
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int c = tid + v * NT;
                if (c < nvec) {
                    if constexpr (!AHEAD) {
                        wq[0] = ldg16((const E *)a.weight + c * VN);
                        bq[0] = load_b(c);
                    }
                    const uint4 q = layernorm_vec<DT>(z[v], mean, rstd, wq[AHEAD ? v : 0], bq[AHEAD ? v : 0], z[v]);
                    if (a.y) stg16((E *)a.y + row + (int64_t)c * VN, q);
#pragma unroll
                    for (int i = 0; i < VN; ++i) m = fmaxf(m, fabsf(z[v][i]));
                }
            }
            if constexpr (Q8) {
                const int e = scale_exp(row_reduce<NT, true>(m, red, 2, lane, wave));
                qi = exp2i(-e);
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
                load_z<DT>(a.x, a.residual, row + (int64_t)c * VN, z);
#pragma unroll
                for (int i = 0; i < VN; ++i) s += z[i];
            }
            const float mean = row_reduce<NT, false>(s, red, 0, lane, wave) * a.inv_d;
            for (int c = tid; c < nvec; c += NT) {
                load_z<DT>(a.x, a.residual, row + (int64_t)c * VN, z);
#pragma unroll
                for (int i = 0; i < VN; ++i) ss = fmaf(z[i] - mean, z[i] - mean, ss);
            }
            const float rstd = 1.0f / sqrtf(row_reduce<NT, false>(ss, red, 1, lane, wave) * a.inv_d + a.eps);
            if (a.mean && tid == 0) {
                a.mean[t] = mean;
                a.rstd[t] = rstd;
            }
            if constexpr (Q8) {
                for (int c = tid; c < nvec; c += NT) {
                    load_z<DT>(a.x, a.residual, row + (int64_t)c * VN, z);
                    layernorm_vec<DT>(z, mean, rstd, ldg16((const E *)a.weight + c * VN), load_b(c), z);
#pragma unroll
                    for (int i = 0; i < VN; ++i) m = fmaxf(m, fabsf(z[i]));
                }
                const int e = scale_exp(row_reduce<NT, true>(m, red, 2, lane, wave));
                qi = exp2i(-e);
                if (tid == 0) a.ys[t] = exp2i(e);
            }
            for (int c = tid; c < nvec; c += NT) {
                load_z<DT>(a.x, a.residual, row + (int64_t)c * VN, z);
                if (a.residual_out) stg16((E *)a.residual_out + row + (int64_t)c * VN, vec16<DT>::narrow(z));
                const uint4 q = layernorm_vec<DT>(z, mean, rstd, ldg16((const E *)a.weight + c * VN), load_b(c), z);
                if (a.y) stg16((E *)a.y + row + (int64_t)c * VN, q);
                if constexpr (Q8) *reinterpret_cast<uint2 *>(a.yq + row + (int64_t)c * 8) = codes_of(z, qi);
            }
        }
        if constexpr (NT > 64) __syncthreads();          // `red` is reused by the next row
    }
}

template <int DT, bool Q8> static lora_status_t launch_forward(const layernorm_args &a, hipStream_t s) {
    const int nvec = a.d / vec16<DT>::n;
    const int64_t cap = 1 << 20;                          // workgroups; each goes on to further rows
#define LORA_NORM(NTV, VPTV)                                                                            \
    do {                                                                                                \
        const int64_t rpb = NTV < 256 ? 256 / NTV : 1, n = (a.T + rpb - 1) / rpb;                       \
        hipLaunchKernelGGL((k_add_layernorm<DT, NTV, VPTV, Q8>), dim3((uint32_t)(n < cap ? n : cap)),   \
                           dim3(NTV < 256 ? 256 : NTV), 0, s, a);                                       \
    } while (0)
    // as many threads as give each one or two vectors (the widths of k_add_rmsnorm)
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

lora_status_t launch_add_layernorm(const void *x, const void *residual, const void *weight, const void *bias, float eps,
                                   int32_t T, int32_t d, int32_t dtype, void *residual_out, void *y, uint8_t *yq,
                                   float *ys, float *mean, float *rstd, hipStream_t s) {
    if (T <= 0) return LORA_OK;
    const layernorm_args a{x, residual, weight, bias, residual_out, y, yq, ys, mean, rstd, eps, 1.0f / (float)d, T, d};
    if (yq) return launch_forward<LORA_BF16, true>(a, s);
    return dtype == LORA_F32 ? launch_forward<LORA_F32, false>(a, s) : launch_forward<LORA_BF16, false>(a, s);
}

// ---------------------------------------------------------------------------
// Backward: with h = (z - mean) rstd and a = dy * weight,
//   dx = rstd (a - mean(a) - h mean(a h)) + dresidual
//   dweight = sum over the rows of dy h,   dbias = sum of dy
// One pass over the data: a workgroup takes every G-th row; its threads own
// columns, and keep the sums for dweight and dbias of their columns in fp32
// registers from row to row.  They go to part [G][2][d] at the end, which a
// second kernel adds up, in a fixed order: no atomics, the same result each time.
// Bound by its bytes: 34811 x 4096 bf16 with dresidual, 1.14 GB, 200 us, 5.7 TB/s;
// with 512 workgroups of partial sums 222 us, with 1024 230.
// ---------------------------------------------------------------------------
struct layernorm_bwd_args {
    const void *dy, *dres, *z, *weight;         // dres may be null
    const float *mean, *rstd;
    void *dx;
    float *part;                                // [groups][2][d], or null: no weight gradients
    float inv_d;
    int32_t T, d;
};

// Sums of a and b over the row's NT threads; `red` holds two rows' in turn.
template <int NT>
__device__ __forceinline__ void row_reduce2(float &a, float &b, float (*red)[2], int lane, int wave) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        a += __shfl_xor(a, o, 64);
        b += __shfl_xor(b, o, 64);
    }
    if constexpr (NT > 64) {
        if (lane == 0) {
            red[wave][0] = a;
            red[wave][1] = b;
        }
        __syncthreads();
        a = red[0][0];
        b = red[0][1];
#pragma unroll
        for (int i = 1; i < NT / 64; ++i) {
            a += red[i][0];
            b += red[i][1];
        }
    }
}

// One vector's dx from what the row's sums gave.
template <int DT>
__device__ __forceinline__ void layernorm_dx(const float *dy, const float *h, const float *w, float rstd, float ma,
                                             float mah, float *dx) {
#pragma unroll
    for (int i = 0; i < vec16<DT>::n; ++i) dx[i] = rstd * (fmaf(dy[i], w[i], -ma) - h[i] * mah);
}

// A thread holds VPT vectors of the row as they came, and those of the next row,
// whose loads are under way during the reduction.
template <int DT, int NT, int VPT, bool RES, bool SUMS>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT) k_layernorm_bwd(layernorm_bwd_args a) {
    typedef typename elem<DT>::T E;
    constexpr int VN = vec16<DT>::n, RPB = NT < 256 ? 256 / NT : 1, W = NT / 64;
    __shared__ float red[2][W][2];
    const int tid = threadIdx.x % NT, lane = tid & 63, wave = tid >> 6;
    const int nvec = a.d / VN;
    const int64_t group = (int64_t)blockIdx.x * RPB + threadIdx.x / NT, groups = (int64_t)gridDim.x * RPB;
    float dw[VPT][VN] = {}, db[VPT][VN] = {};
    uint4 wq[VPT], next_y[VPT], next_z[VPT], next_r[RES ? VPT : 1];
    float next_mean = 0.0f, next_rstd = 0.0f;
    auto load_row = [&](int64_t t) {
        if (t >= a.T) return;
        next_mean = a.mean[t];
        next_rstd = a.rstd[t];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = tid + v * NT;
            if (c < nvec) {
                const int64_t at = t * a.d + (int64_t)c * VN;
                next_y[v] = ldg16((const E *)a.dy + at);
                next_z[v] = ldg16((const E *)a.z + at);
                if (RES) next_r[RES ? v : 0] = ldg16((const E *)a.dres + at);
            }
        }
    };
    load_row(group);
#pragma unroll
    for (int v = 0; v < VPT; ++v)
        if (tid + v * NT < nvec) wq[v] = ldg16((const E *)a.weight + (tid + v * NT) * VN);
    int turn = 0;
    for (int64_t t = group; t < a.T; t += groups, turn ^= 1) {
        uint4 yq[VPT], zq[VPT], rq[RES ? VPT : 1];
        const float mean = next_mean, rstd = next_rstd;
        float sa = 0.0f, sah = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            yq[v] = next_y[v];
            zq[v] = next_z[v];
            if (RES) rq[RES ? v : 0] = next_r[RES ? v : 0];
        }
        load_row(t + groups);
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (tid + v * NT < nvec) {
                float dy[VN], h[VN], w[VN];
                vec16<DT>::widen(yq[v], dy);
                vec16<DT>::widen(zq[v], h);
                vec16<DT>::widen(wq[v], w);
#pragma unroll
                for (int i = 0; i < VN; ++i) {
                    h[i] = (h[i] - mean) * rstd;
                    const float g = dy[i] * w[i];
                    sa += g;
                    sah = fmaf(g, h[i], sah);
                    if (SUMS) {
                        dw[v][i] = fmaf(dy[i], h[i], dw[v][i]);
                        db[v][i] += dy[i];
                    }
                }
            }
        row_reduce2<NT>(sa, sah, red[turn], lane, wave);
        sa *= a.inv_d;
        sah *= a.inv_d;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = tid + v * NT;
            // widened again: the compiler would hold the widened values, and has no registers for them
            if constexpr (VPT > 2)
                asm volatile("" : "+v"(yq[v].x), "+v"(yq[v].y), "+v"(yq[v].z), "+v"(yq[v].w), "+v"(zq[v].x), "+v"(zq[v].y),
                             "+v"(zq[v].z), "+v"(zq[v].w));
            if (c < nvec) {
                float dy[VN], h[VN], w[VN], o[VN];
                vec16<DT>::widen(yq[v], dy);
                vec16<DT>::widen(zq[v], h);
                vec16<DT>::widen(wq[v], w);
#pragma unroll
                for (int i = 0; i < VN; ++i) h[i] = (h[i] - mean) * rstd;
                layernorm_dx<DT>(dy, h, w, rstd, sa, sah, o);
                if (RES) {
                    float r[VN];
                    vec16<DT>::widen(rq[RES ? v : 0], r);
#pragma unroll
                    for (int i = 0; i < VN; ++i) o[i] += r[i];
                }
                stg16((E *)a.dx + t * a.d + (int64_t)c * VN, vec16<DT>::narrow(o));
            }
        }
    }
    if constexpr (SUMS) {
        float *part = a.part + group * 2 * a.d;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = tid + v * NT;
            if (c < nvec)
#pragma unroll
                for (int i = 0; i < VN; i += 4) {
                    *reinterpret_cast<float4 *>(part + c * VN + i) = make_float4(dw[v][i], dw[v][i + 1], dw[v][i + 2], dw[v][i + 3]);
                    *reinterpret_cast<float4 *>(part + a.d + c * VN + i) = make_float4(db[v][i], db[v][i + 1], db[v][i + 2], db[v][i + 3]);
                }
        }
    }
}

// Rows wider than the registers hold (dx only): read again for the second pass.
template <int DT> __global__ void __launch_bounds__(1024) k_layernorm_bwd_wide(layernorm_bwd_args a) {
    typedef typename elem<DT>::T E;
    constexpr int VN = vec16<DT>::n;
    __shared__ float red[2][16][2];
    const int tid = threadIdx.x, nvec = a.d / VN;
    int turn = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
        const float mean = a.mean[t], rstd = a.rstd[t];
        float dy[VN], h[VN], w[VN], sa = 0.0f, sah = 0.0f;
        auto load = [&](int c) {
            vec16<DT>::widen(ldg16((const E *)a.dy + t * a.d + (int64_t)c * VN), dy);
            vec16<DT>::widen(ldg16((const E *)a.z + t * a.d + (int64_t)c * VN), h);
            vec16<DT>::widen(ldg16((const E *)a.weight + (int64_t)c * VN), w);
#pragma unroll
            for (int i = 0; i < VN; ++i) h[i] = (h[i] - mean) * rstd;
        };
        for (int c = tid; c < nvec; c += 1024) {
            load(c);
#pragma unroll
            for (int i = 0; i < VN; ++i) {
                const float g = dy[i] * w[i];
                sa += g;
                sah = fmaf(g, h[i], sah);
            }
        }
        row_reduce2<1024>(sa, sah, red[turn], tid & 63, tid >> 6);
        for (int c = tid; c < nvec; c += 1024) {
            load(c);
            float o[VN];
            layernorm_dx<DT>(dy, h, w, rstd, sa * a.inv_d, sah * a.inv_d, o);
            if (a.dres) {
                float r[VN];
                vec16<DT>::widen(ldg16((const E *)a.dres + t * a.d + (int64_t)c * VN), r);
#pragma unroll
                for (int i = 0; i < VN; ++i) o[i] += r[i];
            }
            stg16((E *)a.dx + t * a.d + (int64_t)c * VN, vec16<DT>::narrow(o));
        }
    }
}

// dweight's and dbias's sums of such rows: a thread owns one vector of columns
// and strides the rows of its group (blockIdx.y).
template <int DT> __global__ void __launch_bounds__(256) k_layernorm_sums_wide(layernorm_bwd_args a) {
    typedef typename elem<DT>::T E;
    constexpr int VN = vec16<DT>::n;
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.d / VN) return;
    float dw[VN] = {}, db[VN] = {};
#pragma unroll 4
    for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
        float dy[VN], z[VN];
        vec16<DT>::widen(ldg16((const E *)a.dy + t * a.d + (int64_t)c * VN), dy);
        vec16<DT>::widen(ldg16((const E *)a.z + t * a.d + (int64_t)c * VN), z);
        const float mean = a.mean[t], rstd = a.rstd[t];
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            dw[i] = fmaf(dy[i], (z[i] - mean) * rstd, dw[i]);
            db[i] += dy[i];
        }
    }
    float *part = a.part + (int64_t)blockIdx.y * 2 * a.d + (int64_t)c * VN;
#pragma unroll
    for (int i = 0; i < VN; ++i) {
        part[i] = dw[i];
        part[a.d + i] = db[i];
    }
}

template <int DT>
__global__ void __launch_bounds__(256) k_column_sums(const float *part, int32_t groups, int64_t n, int32_t d,
                                                     typename elem<DT>::T *out0, typename elem<DT>::T *out1) {
    column_sums<DT>(part, groups, n, d, out0, out1, grid_index());
}

lora_status_t launch_column_sums(const float *part, int32_t groups, int64_t n, int32_t d, int32_t dtype, void *out0,
                                 void *out1, hipStream_t s) {
    const dim3 grid = grid_of((n + 63) / 64);
    if (dtype == LORA_F32)
        hipLaunchKernelGGL(k_column_sums<LORA_F32>, grid, dim3(256), 0, s, part, groups, n, d, (float *)out0,
                           (float *)out1);
    else
        hipLaunchKernelGGL(k_column_sums<LORA_BF16>, grid, dim3(256), 0, s, part, groups, n, d, (uint16_t *)out0,
                           (uint16_t *)out1);
    return hip_status(hipGetLastError());
}

// Groups of rows in the backward pass, each with a partial sum of each column to be
// written and read: a row each up to half the most, then that half, then 4 rows each up to
// the most.  512 threads a row and more: at most 256 (see above for more).  Narrower
// rows, whose threads have one or two vectors of them: at most 2048, whose sums pass the
// data up to 1024 rows.  Four such rows share a workgroup where 64 threads hold one (some
// groups are then without a row): 34811 x 512 bf16 32 us, with 512 groups 61, 256 108.
// Rows of 256 threads would gain by 512 groups: 1000 x 2048 15.1 us, then 11.2;
// 34811 x 2048 96, then 83, with 256 122.
constexpr int32_t kNormGroups = 256, kNormGroupsNarrow = 2048;

static int32_t norm_groups(int32_t T, int32_t most) {
    const int32_t few = most / 2, n = T / 4;
    return T < few ? T : n < few ? few : n < most ? n : most;
}

size_t layernorm_partial_bytes(int32_t T, int32_t d) {
    return align256((size_t)(norm_groups(T, kNormGroupsNarrow) + 3) * 2 * (size_t)d * 4);
}

template <int DT>
static lora_status_t launch_backward(const layernorm_bwd_args &a, void *dweight, void *dbias, hipStream_t s) {
    const int nvec = a.d / vec16<DT>::n;
    int32_t groups = 0;
#define LORA_BWD(NTV, VPTV)                                                                             \
    do {                                                                                                \
        constexpr int rpb = NTV < 256 ? 256 / NTV : 1;                                                  \
        const int n = (norm_groups(a.T, NTV < 512 ? kNormGroupsNarrow : kNormGroups) + rpb - 1) / rpb;  \
        const dim3 grid(n), block(NTV < 256 ? 256 : NTV);                                               \
        groups = n * rpb;                                                                               \
        if (a.part && a.dres) hipLaunchKernelGGL((k_layernorm_bwd<DT, NTV, VPTV, true, true>), grid, block, 0, s, a);   \
        else if (a.part) hipLaunchKernelGGL((k_layernorm_bwd<DT, NTV, VPTV, false, true>), grid, block, 0, s, a);       \
        else if (a.dres) hipLaunchKernelGGL((k_layernorm_bwd<DT, NTV, VPTV, true, false>), grid, block, 0, s, a);       \
        else hipLaunchKernelGGL((k_layernorm_bwd<DT, NTV, VPTV, false, false>), grid, block, 0, s, a);                  \
    } while (0)
    if (nvec <= 64) LORA_BWD(64, 1);
    else if (nvec <= 128) LORA_BWD(64, 2);
    else if (nvec <= 256) LORA_BWD(256, 1);
    else if (nvec <= 512) LORA_BWD(512, 1);
    else if (nvec <= 1024) LORA_BWD(1024, 1);
    else if (nvec <= 2048) LORA_BWD(512, 4);
    else {
        // the sums first: dx may be dy's or z's own buffer
        groups = norm_groups(a.T, kNormGroups);
        if (a.part)
            hipLaunchKernelGGL(k_layernorm_sums_wide<DT>, dim3((nvec + 255) / 256, groups), dim3(256), 0, s, a);
        hipLaunchKernelGGL(k_layernorm_bwd_wide<DT>, dim3(groups), dim3(1024), 0, s, a);
    }
#undef LORA_BWD
    const lora_status_t st = hip_status(hipGetLastError());
    if (st != LORA_OK || !a.part) return st;
    return launch_column_sums(a.part, groups, 2ll * a.d, a.d, DT, dweight, dbias, s);
}

lora_status_t launch_layernorm_backward(const void *dy, const void *dres, const void *z, const void *weight,
                                        const float *mean, const float *rstd, int32_t T, int32_t d, int32_t dtype,
                                        void *dx, void *dweight, void *dbias, float *part, hipStream_t s) {
    const layernorm_bwd_args a{dy, dres, z, weight, mean, rstd, dx, dweight || dbias ? part : nullptr, 1.0f / (float)d,
                               T, d};
    return dtype == LORA_F32 ? launch_backward<LORA_F32>(a, dweight, dbias, s)
                             : launch_backward<LORA_BF16>(a, dweight, dbias, s);
}

}  // namespace lora
