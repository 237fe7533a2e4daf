// dp of the linear layer's backward pass, and what it shares with the gated pair's.
#pragma once

#include "act.hpp"

namespace lora {

// What is left of a value beside its first bf16 part; an infinite or NaN value
// has no second part.
__device__ __forceinline__ float second_part(float rest) {
    return fabsf(rest) < __builtin_inff() ? rest : 0.0f;
}

// act and its derivative at x.
template <bool FINE> __device__ __forceinline__ void act_both(int act, float x, float &a, float &da) {
    if (act == LORA_ACT_SILU) {
        const float q = logistic<FINE>(x);
        a = x * q;
        da = fmaf(a, 1.0f - q, q);
    } else if (act == LORA_ACT_GELU) {
        const float cdf = 0.5f * erfcf(-0.70710678118654752f * x);
        a = x * cdf;
        // the density at x; exp(-x^2/2) is 0 long before x^2 overflows
        da = fmaf(x, 0.39894228040143268f * (FINE ? expf(-0.5f * x * x) : __expf(-0.5f * x * x)), cdf);
    } else {
        const float q = logistic<FINE>(kGeluTanhK * fmaf(kGeluTanhC * x * x, x, x));
        a = x * q;
        // q is 0 or 1 long before x^2 overflows, where 0 times its slope is 0
        da = fmaf(a * (1.0f - q), kGeluTanhK * fmaf(3.0f * kGeluTanhC, fminf(x * x, 1e30f), 1.0f), q);
    }
}

// ---------------------------------------------------------------------------
// dp of the linear layer, as k_gated_dact's dg, and the sums of its columns for
// dbias.  A cell of 256 threads takes 32 vectors of columns and a stretch of rows, every
// eighth of them a thread; the 8 strands are added through LDS to one partial sum
// per column and stretch.  WRITE = false: dp is dy itself, only its sums are made.
// Most of it latency; the segment build, which runs beside it, takes as long.
// ---------------------------------------------------------------------------
constexpr int kActVecs = 32, kActStrands = 8;

struct act_grad_args {
    const void *pre, *dy;
    void *dp;
    float *part;                       // [stretches][N]
    int32_t T, N, rows, act;
    int64_t lo;                        // bf16: from dp's first parts to its second
};

// Floats of LDS per cell.
template <int DT> constexpr int act_grad_lds() { return kActStrands * kActVecs * vec16<DT>::n; }

// Cell (bx, by) by 256 threads (tid) of a workgroup whose others do the same with
// theirs; past the last stretch there is nothing to do but the barrier.
template <int DT, bool WRITE, bool SUMS>
__device__ __forceinline__ void act_grad(const act_grad_args &g, int bx, int by, int tid, float *lds) {
    typedef typename elem<DT>::T E;
    constexpr int VN = vec16<DT>::n;
    const int vec = tid % kActVecs, strand = tid / kActVecs;
    const int n = (bx * kActVecs + vec) * VN;
    const int64_t t0 = (int64_t)by * g.rows, t1 = t0 + g.rows < g.T ? t0 + g.rows : g.T;
    float sum[VN] = {};
    if (n < g.N) {
#pragma unroll 2
        for (int64_t t = t0 + strand; t < t1; t += kActStrands) {
            const int64_t at = t * g.N + n;
            float d[VN];
            vec16<DT>::widen(ldg16((const E *)g.dy + at), d);
            if constexpr (WRITE) {
                float p[VN];
                vec16<DT>::widen(ldg16((const E *)g.pre + at), p);
#pragma unroll
                for (int e = 0; e < VN; ++e) {
                    float a, da;
                    act_both<DT == LORA_F32>(g.act, p[e], a, da);
                    d[e] *= da;
                }
                const uint4 q = vec16<DT>::narrow(d);
                stg16((E *)g.dp + at, q);
                if constexpr (DT == LORA_BF16) {
                    float h[VN];
                    vec16<DT>::widen(q, h);
#pragma unroll
                    for (int e = 0; e < VN; ++e) h[e] = second_part(d[e] - h[e]);
                    stg16((E *)g.dp + g.lo + at, vec16<DT>::narrow(h));
                }
            }
            if constexpr (SUMS)
#pragma unroll
                for (int e = 0; e < VN; ++e) sum[e] += d[e];
        }
    }
    if constexpr (SUMS) {
        float(*s)[kActVecs * VN] = reinterpret_cast<float(*)[kActVecs * VN]>(lds);
#pragma unroll
        for (int e = 0; e < VN; ++e) s[strand][vec * VN + e] = sum[e];
        __syncthreads();
        const int c = tid, col = bx * kActVecs * VN + c;
        if (c < kActVecs * VN && col < g.N && t0 < g.T) {
            float f = s[0][c];
#pragma unroll
            for (int i = 1; i < kActStrands; ++i) f += s[i][c];
            g.part[(int64_t)by * g.N + col] = f;
        }
    }
}

// A call's act_grad cells, run beside the segment build.  Rows of a stretch: about
// 1024 cells, of at least 2 rows a strand.
inline int32_t act_grad_rows(int32_t T, int32_t N, int32_t dtype) {
    const int cell = kActVecs * (dtype == LORA_F32 ? 4 : 8), tiles = (N + cell - 1) / cell, by = (1024 + tiles - 1) / tiles;
    int rows = (T + by - 1) / by;
    if (rows < 2 * kActStrands) rows = 2 * kActStrands;
    return (rows + kActStrands - 1) / kActStrands * kActStrands;
}

struct act_beside {
    act_grad_args args;
    int32_t dtype;
    bool write, sums;                  // dp is made, its columns' sums are made

    int32_t cols() const {
        const int cell = kActVecs * (dtype == LORA_F32 ? 4 : 8);
        return (args.N + cell - 1) / cell;
    }
    int32_t stretches() const { return (args.T + args.rows - 1) / args.rows; }
};

}  // namespace lora
