// The gated pair's part of the GEMM kernels: which columns a tile holds, the
// activations, the low-rank pass of both pools, the store of h = act(g) * u
// and the split-K reduction.
#pragma once

#include "gemm_common.hpp"

namespace lora {

// A launch numbers the columns of gate and up together, in groups of 64: 32
// columns of gate, then the same 32 of up.  So a wavefront of 64 columns
// holds both values of 32 columns of h in the same lanes' accumulators.
__device__ __forceinline__ int gated_col(int vcol) { return (vcol >> 6) * 32 + (vcol & 31); }
__device__ __forceinline__ bool gated_up(int vcol) { return (vcol & 32) != 0; }

// The logistic function of x; FINE uses the exact exponential and division
// (fp32 outputs), else one v_exp and one v_rcp (1 ulp each, far below bf16's
// step).  exp overflows to infinity for very negative x, which gives 0.
template <bool FINE> __device__ __forceinline__ float logistic(float x) {
    if (FINE) return 1.0f / (1.0f + expf(-x));
    return __builtin_amdgcn_rcpf(1.0f + __expf(-x));
}

template <int V> struct int_const { static constexpr int value = V; };

constexpr float kGeluTanhK = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluTanhC = 0.044715f;

// silu: x q, q = logistic(x).  gelu: x cdf(x), the normal distribution's cdf
// by erfc, which keeps the small values of negative x.  gelu_tanh: 0.5 x (1 +
// tanh(z)) = x logistic(2 z), z = sqrt(2/pi) (x + 0.044715 x^3).
template <bool FINE> __device__ __forceinline__ float act_value(int act, float x) {
    if (act == LORA_ACT_SILU) return x * logistic<FINE>(x);
    if (act == LORA_ACT_GELU) return x * (0.5f * erfcf(-0.70710678118654752f * x));
    return x * logistic<FINE>(kGeluTanhK * fmaf(kGeluTanhC * x * x, x, x));
}

// The low-rank terms of both pools: gate's into the even column blocks, up's
// into the odd ones.  col0: the wavefront's first column of h.
template <int RB, int CB, int RG, int KB, int RF>
__device__ __forceinline__ void gated_lora_pass(const gemm_args &g, f32x16_t (&acc)[RB][CB], const int32_t *s_t,
                                                const int32_t *s_id, int wrow0, int col0, int lane) {
    static_assert(CB % 2 == 0, "a wavefront holds whole pairs");
    gemm_args q = g;
    q.b = g.sl[0].b;
    q.scale = g.sl[0].scale;
    q.rank = g.sl[0].rank;
    q.row0 = g.sl[0].row0;
    lora_pass_impl<RB, CB / 2, RG, KB, RF, 2, 0>(q, acc, s_t, s_id, 0, wrow0, col0, lane);
    q.b = g.sl[1].b;
    q.scale = g.sl[1].scale;
    q.rank = g.sl[1].rank;
    q.row0 = g.sl[1].row0;
    q.v = g.v + g.sl[1].v_off;
    lora_pass_impl<RB, CB / 2, RG, KB, RF, 2, 1>(q, acc, s_t, s_id, 0, wrow0, col0, lane);
}

// The store: a wavefront's block of 32 rows goes through its LDS area once
// per output (h, and gate and up where they are kept), so that each lane
// writes 8 consecutive columns of a row, rounded once.
template <int BM, int BN, int WV, int WR, int RB, int CB>
__device__ __forceinline__ void gated_store_tile(const gemm_args &g, f32x16_t (&acc)[RB][CB], float *smem_f,
                                                 const int32_t *s_meta_t, int n0, int w, int lane) {
    constexpr int WM = BM / WR, WN = BN / (WV / WR), HN = WN / 2, SLD = HN + 4;
    static_assert(CB % 2 == 0 && WN % 64 == 0, "a wavefront holds whole pairs");
    const int wm = w / (WV / WR), wn = w % (WV / WR);
    const int N = g.N;
    constexpr int QN = HN / 8, RPP = 64 / QN, PASSES = 32 / RPP;
    float *stage = smem_f + w * 32 * SLD;
    const int q = lane % QN, rr = lane / QN;
    const int n = gated_col(n0 + wn * WN) + 8 * q;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        // every other column block, from OF on
        auto put = [&](uint16_t *out, auto of) {
            constexpr int OF = decltype(of)::value;
            __syncthreads();
#pragma unroll
            for (int p = 0; p < CB / 2; ++p)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    stage[(8 * (e >> 2) + 4 * (lane >> 5) + (e & 3)) * SLD + p * 32 + (lane & 31)] =
                        acc[rb][2 * p + OF][e];
            __syncthreads();
#pragma unroll
            for (int k = 0; k < PASSES; ++k) {
                const int32_t t = s_meta_t[wm * WM + rb * 32 + rr + RPP * k];
                if (t < 0 || n >= N) continue;
                const float *src = stage + (rr + RPP * k) * SLD + 8 * q;
                float f[8];
                *reinterpret_cast<float4 *>(f) = *reinterpret_cast<const float4 *>(src);
                *reinterpret_cast<float4 *>(f + 4) = *reinterpret_cast<const float4 *>(src + 4);
                stg16(out + (int64_t)t * N + n, vec16<LORA_BF16>::narrow(f));
            }
        };
        if (g.sl[0].y) {
            put(g.sl[0].y, int_const<0>{});
            put(g.sl[1].y, int_const<1>{});
        }
#pragma unroll
        for (int p = 0; p < CB / 2; ++p)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                acc[rb][2 * p][e] = act_value<false>(g.act, acc[rb][2 * p][e]) * acc[rb][2 * p + 1][e];
        put(g.y, int_const<0>{});
    }
}

// A split piece's fp32 partials, in the tile's own column order, columns past
// the last pair included (they hold zeros).
template <int BM, int BN, int WV, int WR, int RB, int CB>
__device__ __forceinline__ void gated_store_partial(const gemm_args &g, f32x16_t (&acc)[RB][CB], float *smem_f,
                                                    int n0, int w, int lane, int tidx, int split) {
    gemm_args q = g;
    q.N = g.n_tiles_n * BN;
    gemm_store_tile<BM, BN, WV, WR, true, false>(q, acc, smem_f, nullptr, n0, w, lane, tidx, split);
}

// 8 columns of one row of the low-rank term, for the reduction: o += s sum_j
// v[j] B[j][n..n+8], rank octets in order.
__device__ __forceinline__ void add_low_rank8(const gemm_args &g, const gemm_slice &sl, int32_t id, int64_t t, int n,
                                              float *o) {
    const int32_t rk = min(sl.rank[id], g.max_rank);
    if (rk <= 0) return;
    const float sc = sl.scale[id];
    const float *vrow = g.v + t * g.v_stride + sl.v_off;
    const uint16_t *b = sl.b + slot_row0(sl.row0, id, g.max_rank) * g.N + (int64_t)n * 8;
    float d[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int gg = 0; gg < (rk + 7) >> 3; ++gg) {
        float vv[8];
        *reinterpret_cast<float4 *>(vv) = *reinterpret_cast<const float4 *>(vrow + gg * 8);
        *reinterpret_cast<float4 *>(vv + 4) = *reinterpret_cast<const float4 *>(vrow + gg * 8 + 4);
        uint4 bq[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) bq[q] = ldg16(b + (int64_t)gg * g.N * 8 + q * 8);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            float bf[8];
            vec16<LORA_BF16>::widen(bq[q], bf);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[q] = fmaf(vv[e], bf[e], d[q]);
        }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) o[q] = fmaf(sc, d[q], o[q]);
}

// Split-K reduction of the gated tiles: a thread owns 8 columns of h of one
// row, sums both projections' partials in split order, adds both low-rank
// terms, and writes h (and gate and up where they are kept).
template <int BM, int BN>
__global__ void __launch_bounds__(256) k_gated_reduce(gemm_args g) {
    constexpr int HN = BN / 2, CPR = HN / 8, RW = 256 / CPR, CHUNKS = BM / RW;
    const int per = gridDim.x / kXcds, rem = gridDim.x % kXcds;
    const int xcd = blockIdx.x % kXcds;
    const int item = xcd * per + min(xcd, rem) + blockIdx.x / kXcds;   // whole tiles per XCD, as k_splitk_reduce
    const int tidx = item / CHUNKS, chunk = item % CHUNKS;
    int tm, tn;
    grouped_tile(g.tile_base + tidx, g.n_tiles_m, g.n_tiles_n, g.col_strips, tm, tn);
    const int r = chunk * RW + threadIdx.x / CPR, c = (threadIdx.x % CPR) * 8;
    const int p = tm * BM + r, n = tn * HN + c;
    if (p >= g.T || n >= g.N) return;
    const int32_t t = perm_row(g.perm, p, g.T);
    if (t < 0) return;
    const int cg = (c >> 5) * 64 + (c & 31);              // gate's column of the partial tile; up's is 32 on
    float o[2][8] = {};
    const float *src = g.partial + ((int64_t)tidx * g.splits * BM + r) * BN + cg;
    for (int s = 0; s < g.splits; ++s, src += BM * BN) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const float4 a = *reinterpret_cast<const float4 *>(src + 32 * m);
            const float4 b = *reinterpret_cast<const float4 *>(src + 32 * m + 4);
            o[m][0] += a.x; o[m][1] += a.y; o[m][2] += a.z; o[m][3] += a.w;
            o[m][4] += b.x; o[m][5] += b.y; o[m][6] += b.z; o[m][7] += b.w;
        }
    }
    const int32_t id = g.ids[t];
    if (id >= 0 && id < g.n_slots) {
        add_low_rank8(g, g.sl[0], id, t, n, o[0]);
        add_low_rank8(g, g.sl[1], id, t, n, o[1]);
    }
    const int64_t at = (int64_t)t * g.N + n;
    if (g.sl[0].y) {
        stg16(g.sl[0].y + at, vec16<LORA_BF16>::narrow(o[0]));
        stg16(g.sl[1].y + at, vec16<LORA_BF16>::narrow(o[1]));
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) o[0][e] = act_value<false>(g.act, o[0][e]) * o[1][e];
    stg16(g.y + at, vec16<LORA_BF16>::narrow(o[0]));
}

template <int BM, int BN> static void launch_gated_reduce(const gemm_args &g, hipStream_t s) {
    constexpr int RW = 256 / (BN / 16);
    hipLaunchKernelGGL((k_gated_reduce<BM, BN>), dim3(g.n_tiles * (BM / RW)), dim3(256), 0, s, g);
}

// Implemented beside their base GEMMs; g holds everything but the tile plan.
lora_status_t launch_gemm_gated(gemm_args &g, size_t partial_bytes, hipStream_t s);
lora_status_t launch_gemm_gated_fp8(gemm_args &g, size_t partial_bytes, hipStream_t s);

}  // namespace lora
