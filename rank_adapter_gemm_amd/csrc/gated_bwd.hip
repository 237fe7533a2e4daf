// Backward pass of the gated pair h = act(g) * u, base weights frozen:
//   dg = dh * u * act'(g),  du = dh * act(g)                        k_gated_dact
//   dv = s_a dg B_a^T   [T, r] for each of the two                  k_rank_grad
//   dx = dg Wg^T + du Wu^T + dv_g Ag_a^T + dv_u Au_a^T              k_gemm_nt / k_dx_f32
//   dA_a = sum over a's rows of x_t^T dv_t                          k_seg_outer
//   dB_a = s_a sum over a's rows of v_t^T dg_t,  v = x A_a          k_seg_outer
// Rows are visited in adapter order (the segment builder's perm), so every
// sum over an adapter's rows runs over neighbours, in row order, without
// atomics: results repeat bitwise.
#include "gated_common.hpp"

namespace lora {

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
        da = fmaf(a * (1.0f - q), kGeluTanhK * fmaf(3.0f * kGeluTanhC * x, x, 1.0f), q);
    }
}

// dg and du of 16 bytes of values per thread.  For bf16 they are rounded
// once: they are operands of bf16 matrix products, and their rounding enters
// each sum as one more rounding of an input would.
template <int DT>
__global__ void __launch_bounds__(256) k_gated_dact(const typename elem<DT>::T *gate, const typename elem<DT>::T *up,
                                                    const typename elem<DT>::T *dh, typename elem<DT>::T *dg,
                                                    typename elem<DT>::T *du, int64_t n_vec, int act) {
    constexpr int VN = vec16<DT>::n;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n_vec; i += gridDim.x * 256ll) {
        float g[VN], u[VN], h[VN];
        vec16<DT>::widen(ldg16(gate + i * VN), g);
        vec16<DT>::widen(ldg16(up + i * VN), u);
        vec16<DT>::widen(ldg16(dh + i * VN), h);
#pragma unroll
        for (int e = 0; e < VN; ++e) {
            float a, da;
            act_both<DT == LORA_F32>(act, g[e], a, da);
            g[e] = h[e] * u[e] * da;
            u[e] = h[e] * a;
        }
        stg16(dg + i * VN, vec16<DT>::narrow(g));
        stg16(du + i * VN, vec16<DT>::narrow(u));
    }
}

// ---------------------------------------------------------------------------
// dv.  One workgroup per row and projection: rank octet by octet, each thread
// strides the row's N values against the slot's B octets.
// ---------------------------------------------------------------------------
struct pair_pools {
    const void *a[2], *b[2];
    const float *scale[2];
    const int32_t *rank[2], *row0[2];
};

template <int DT>
__global__ void __launch_bounds__(256) k_rank_grad_rows(const typename elem<DT>::T *dy, int64_t dy_stride, int32_t T,
                                                        int32_t N, pair_pools pp, int32_t n_slots, int32_t R,
                                                        const int32_t *ids, float *dv) {
    typedef typename elem<DT>::T E;
    const int t = blockIdx.x, m = blockIdx.y;
    float *out = dv + (int64_t)t * 2 * R + m * R;
    const int32_t id = ids[t];
    const int32_t r = id >= 0 && id < n_slots ? min(pp.rank[m][id], R) : 0;
    const E *row = dy + m * dy_stride + (int64_t)t * N;
    __shared__ float red[4][8];
    for (int o = 0; o < R / 8; ++o) {
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (8 * o < r) {
            const E *b = (const E *)pp.b[m] + (slot_row0(pp.row0[m], id, R) + 8 * o) * N;
            for (int n = threadIdx.x; n < N; n += 256) {
                const float f = elem<DT>::load(row, n);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = fmaf(f, elem<DT>::load(b, (int64_t)n * 8 + e), acc[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int s = 32; s > 0; s >>= 1) acc[e] += __shfl_xor(acc[e], s, 64);
        __syncthreads();
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int e = 0; e < 8; ++e) red[threadIdx.x >> 6][e] = acc[e];
        __syncthreads();
        if (threadIdx.x < 8) {
            const int e = threadIdx.x, j = 8 * o + e;
            out[j] = j < r ? pp.scale[m][id] * ((red[0][e] + red[1][e]) + (red[2][e] + red[3][e])) : 0.0f;
        }
    }
}

// ---------------------------------------------------------------------------
// A of the batch's slots in rank octets, gate's ranks then up's: [segment][2R /
// 8][d_in][8], with the tables (row0, rank, scale) that make them one pool of
// max_rank 2R for the low-rank pass of the dx product.  dv holds the scales
// already, so the table's are 1.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) k_a_octets(pair_pools pp, const int32_t *seg_id, const int32_t *n_seg,
                                                  int32_t n_slots, int32_t K, int32_t R, uint16_t *oct,
                                                  int32_t *row0, int32_t *rank, float *scale) {
    const int i = blockIdx.x;
    if (i >= min(*n_seg, n_slots)) return;
    const int32_t id = seg_id[i];
    if (id < 0 || id >= n_slots) return;
    const int32_t r[2] = {min(pp.rank[0][id], R), min(pp.rank[1][id], R)};
    if (blockIdx.y == 0 && threadIdx.x == 0) {
        row0[id] = i * 2 * R;
        rank[id] = r[0] > 0 || r[1] > 0 ? 2 * R : 0;
        scale[id] = 1.0f;
    }
    const int k = blockIdx.y * 256 + threadIdx.x;
    if (k >= K) return;
    for (int o = 0; o < 2 * R / 8; ++o) {
        const int m = 8 * o >= R, j0 = 8 * o - m * R;
        const uint16_t *a = (const uint16_t *)pp.a[m] + (slot_row0(pp.row0[m], id, R) + j0) * K + k;
        uint32_t e[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) e[q] = j0 + q < r[m] ? a[(int64_t)q * K] : 0u;
        stg16(oct + (((int64_t)i * 2 * R / 8 + o) * K + k) * 8,
              make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16));
    }
}

// ---------------------------------------------------------------------------
// dx, bf16: rows of [dg, du] times rows of [Wg, Wu] (both contiguous along the
// sum, so both tiles are DMA'd rows with one swizzle and ds_read_b128
// fragments), the two projections one after the other along K.  Tiles,
// hand-off, low-rank pass, store and K split are those of the forward GEMM.
// ---------------------------------------------------------------------------
struct nt_args {
    const uint16_t *a[2], *w[2];       // [T][F], [N][F]
    int32_t F, Fp;                     // F rounded up to whole K steps
};

template <int BM, int BN, int NS, bool SPLIT, int WV, int WR>
__global__ void __launch_bounds__(WV * 64) k_gemm_nt(gemm_args g, nt_args nt) {
    constexpr int BK = 64, CH = BK / 8, WM = BM / WR, WN = BN / (WV / WR), RB = WM / 32, CB = WN / 32;
    constexpr int XSTAGE = BM * BK, STAGE = XSTAGE + BN * BK;
    constexpr int XI = BM * CH / (64 * WV), WI = BN * CH / (64 * WV);
    constexpr int EPI = WV * 32 * (WN + 4) * 4, LDS = NS * STAGE * 2 > EPI ? NS * STAGE * 2 : EPI;
    __shared__ __attribute__((aligned(1024))) uint16_t smem[LDS / 2];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int wm = w / (WV / WR), wn = w % (WV / WR);
    int tm, tn, split, tidx;
    tile_of(blockIdx.x, gridDim.x, g, tm, tn, split, tidx);
    const int m0 = tm * BM, n0 = tn * BN;
    const int N = g.N, T = g.T, F = nt.F;
    const int k_begin = SPLIT ? split * g.k_chunk : 0;
    const int k_end = SPLIT ? min(g.K, k_begin + g.k_chunk) : g.K;

    int64_t xrow[XI], wrow[WI];
    int xcol[XI], wcol[WI];
#pragma unroll
    for (int j = 0; j < XI; ++j) {
        const int c = (w * XI + j) * 64 + lane, r = c / CH, slot = c % CH, p = m0 + r;
        const int32_t t = p < T ? perm_row(g.perm, p, T) : -1;
        xrow[j] = t >= 0 ? (int64_t)t * F : -1;
        xcol[j] = 8 * (slot ^ swz_x<64>(r));
    }
#pragma unroll
    for (int j = 0; j < WI; ++j) {
        const int c = (w * WI + j) * 64 + lane, r = c / CH, slot = c % CH;
        wrow[j] = n0 + r < N ? (int64_t)(n0 + r) * F : -1;
        wcol[j] = 8 * (slot ^ swz_x<64>(r));
    }
    auto dma_stage = [&](int kt, int buf) {
        uint16_t *xs = smem + buf * STAGE, *wsm = xs + XSTAGE;
        const int k0 = k_begin + kt * BK;
        const bool second = k0 >= nt.Fp;                   // a step lies in one projection (Fp, k_begin: whole steps)
        const uint16_t *a = second ? nt.a[1] : nt.a[0], *wt = second ? nt.w[1] : nt.w[0];
        const int f0 = k0 - (second ? nt.Fp : 0);
#pragma unroll
        for (int j = 0; j < XI; ++j) {
            const int f = f0 + xcol[j];
            const void *src = xrow[j] >= 0 && f < F ? (const void *)(a + xrow[j] + f) : (const void *)g_zero16;
            dma16(src, xs + (w * XI + j) * 64 * 8);
        }
#pragma unroll
        for (int j = 0; j < WI; ++j) {
            const int f = f0 + wcol[j];
            const void *src = wrow[j] >= 0 && f < F ? (const void *)(wt + wrow[j] + f) : (const void *)g_zero16;
            dma16(src, wsm + (w * WI + j) * 64 * 8);
        }
    };

    f32x16_t acc[RB][CB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[rb][cb][e] = 0.0f;

    const int fr = lane & 31, fk = lane >> 5;
    constexpr int KS = BK / 16;
    bf16x8_t af[2][RB], bfr[2][CB];
    auto frag = [&](const uint16_t *base, int r, int ks) {
        return *reinterpret_cast<const bf16x8_t *>(base + r * BK + 8 * ((2 * ks + fk) ^ swz_x<64>(r)));
    };
    auto load_frags = [&](int buf, int ks, bf16x8_t *a, bf16x8_t *b) {
        const uint16_t *xs = smem + buf * STAGE, *wsm = xs + XSTAGE;
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) a[rb] = frag(xs, wm * WM + rb * 32 + fr, ks);
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) b[cb] = frag(wsm, wn * WN + cb * 32 + fr, ks);
    };
    auto mfmas = [&](const bf16x8_t *a, const bf16x8_t *b, int rb0, int rb1) {
#pragma unroll
        for (int rb = rb0; rb < rb1; ++rb)
#pragma unroll
            for (int cb = 0; cb < CB; ++cb)
                acc[rb][cb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[rb], b[cb], acc[rb][cb], 0, 0, 0);
    };
    constexpr int NREAD = RB + CB, PER = XI + WI;

    int32_t *s_meta_t = nullptr, *s_meta_id = nullptr;
    if constexpr (!SPLIT) {
        __shared__ int32_t s_t[BM], s_id[BM];
        s_meta_t = s_t;
        s_meta_id = s_id;
        for (int i = tid; i < BM; i += WV * 64) {
            const int p = m0 + i;
            const int32_t t = p < T ? perm_row(g.perm, p, T) : -1;
            int32_t id = -1;
            if (t >= 0) {
                const int32_t raw = g.ids[t];
                if (raw >= 0 && raw < g.n_slots && g.rank[raw] > 0) id = raw;
            }
            s_t[i] = t;
            s_id[i] = id;
        }
    }
    const int nk = (k_end - k_begin + BK - 1) / BK;
    static_assert((NS - 1) * PER <= 63, "vmcnt counts at most 63 loads");
    auto wait_stage = [&](int ahead) {
        if (ahead >= 3) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(3 * PER > 63 ? 63 : 3 * PER) : "memory");
        else if (ahead == 2) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * PER > 63 ? 63 : 2 * PER) : "memory");
        else if (ahead == 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(PER) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    };
#pragma unroll
    for (int st = 0; st < NS; ++st)
        if (st < nk) dma_stage(st, st);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if constexpr (!SPLIT)
        lora_pass_impl<RB, CB, (RB >= 2 ? 2 : 1), 1, (RB >= 2 ? 2 : 1)>(g, acc, s_meta_t, s_meta_id, n0, wm * WM,
                                                                      n0 + wn * WN, lane);
    wait_stage(min(NS - 1, nk - 1));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    load_frags(0, 0, af[0], bfr[0]);
    for (int kt = 0; kt < nk; ++kt) {
        const int buf = kt % NS;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const int cur = ks & 1, nxt = cur ^ 1;
            if (ks + 1 < KS) {
                load_frags(buf, ks + 1, af[nxt], bfr[nxt]);
                mfmas(af[cur], bfr[cur], 0, RB);
                sched_interleave<NREAD, RB * CB>();
            } else {
                // stage hand-off, as in k_gemm_bf16
                mfmas(af[cur], bfr[cur], 0, RB / 2);
                __builtin_amdgcn_sched_barrier(0);
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                wait_stage(min(NS - 2, nk - 2 - kt));
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
                if (kt + NS < nk) dma_stage(kt + NS, buf);
                __builtin_amdgcn_sched_barrier(0);
                load_frags((kt + 1) % NS, 0, af[nxt], bfr[nxt]);
                mfmas(af[cur], bfr[cur], RB / 2, RB);
                sched_interleave<NREAD, (RB - RB / 2) * CB>();
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    gemm_store_tile<BM, BN, WV, WR, SPLIT, false>(g, acc, reinterpret_cast<float *>(smem), s_meta_t, n0, w, lane,
                                                  tidx, split);
}

template <int BM, int BN, int NS, int WV, int WR, int NST, int WVT>
static void launch_nt_cfg(gemm_args g, const nt_args &nt, const gemm_plan &pl, hipStream_t s) {
    if (pl.n_dp > 0) {
        g.tile_base = 0;
        g.n_tiles = pl.n_dp;
        g.splits = 1;
        g.k_chunk = g.K;
        hipLaunchKernelGGL((k_gemm_nt<BM, BN, NS, false, WV, WR>), dim3(pl.n_dp), dim3(WV * 64), 0, s, g, nt);
    }
    if (pl.tail > 0) {
        g.tile_base = pl.n_dp;
        g.n_tiles = pl.tail;
        g.splits = pl.splits;
        g.k_chunk = pl.k_chunk;
        hipLaunchKernelGGL((k_gemm_nt<BM, BN, NST, true, WVT, WR>), dim3(pl.tail * pl.splits), dim3(WVT * 64), 0, s,
                           g, nt);
        hipLaunchKernelGGL((k_splitk_reduce<true, false, BM, BN>), dim3(pl.tail * (BM / (2048 / BN))), dim3(256), 0,
                           s, g);
    }
}

// ---------------------------------------------------------------------------
// dx, fp32: 64 x 64 tiles on v_mfma_f32_32x32x2_f32, the sum over F of dg then
// of du; the low-rank term from A's rows in the store.
// ---------------------------------------------------------------------------
struct dx_f32_args {
    const float *a[2], *w[2];
    float *dx;
    const float *dv;
    const int32_t *ids, *perm;
    int32_t T, F, N, n_slots, R, n_tiles_n;
};

__global__ void __launch_bounds__(256) k_dx_f32(dx_f32_args g, pair_pools pp) {
    constexpr int BK = 32, LD = 64 + 4;
    __shared__ __attribute__((aligned(16))) float s_a[BK][LD], s_w[BK][LD];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, wm = w >> 1, wn = w & 1;
    const int m0 = blockIdx.x / g.n_tiles_n * 64, n0 = blockIdx.x % g.n_tiles_n * 64;
    const int r = tid >> 2, kk = (tid & 3) * 8;
    const int32_t t_a = m0 + r < g.T ? perm_row(g.perm, m0 + r, g.T) : -1;
    const int64_t arow = (int64_t)(t_a < 0 ? 0 : t_a) * g.F;
    const bool wok = n0 + r < g.N;
    const int64_t wrow = (int64_t)(wok ? n0 + r : 0) * g.F;
    f32x16_t acc;
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
    for (int m = 0; m < 2; ++m)
        for (int f0 = 0; f0 < g.F; f0 += BK) {
            float4 ra[2], rw[2];
            const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
            const bool in = f0 + kk < g.F;                 // F is a multiple of 8
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                ra[i] = in && t_a >= 0 ? *reinterpret_cast<const float4 *>(g.a[m] + arow + f0 + kk + 4 * i) : zero;
                rw[i] = in && wok ? *reinterpret_cast<const float4 *>(g.w[m] + wrow + f0 + kk + 4 * i) : zero;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                s_a[kk + 4 * i + 0][r] = ra[i].x;
                s_a[kk + 4 * i + 1][r] = ra[i].y;
                s_a[kk + 4 * i + 2][r] = ra[i].z;
                s_a[kk + 4 * i + 3][r] = ra[i].w;
                s_w[kk + 4 * i + 0][r] = rw[i].x;
                s_w[kk + 4 * i + 1][r] = rw[i].y;
                s_w[kk + 4 * i + 2][r] = rw[i].z;
                s_w[kk + 4 * i + 3][r] = rw[i].w;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < BK; k += 2)
                acc = __builtin_amdgcn_mfma_f32_32x32x2f32(s_a[k + (lane >> 5)][wm * 32 + (lane & 31)],
                                                           s_w[k + (lane >> 5)][wn * 32 + (lane & 31)], acc, 0, 0, 0);
        }
    const int n = n0 + wn * 32 + (lane & 31);
    if (n >= g.N) return;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const int p = m0 + wm * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
        const int64_t t = p < g.T ? perm_row(g.perm, p, g.T) : -1;
        if (t < 0) continue;
        float val = acc[e];
        const int32_t id = g.ids[t];
        if (id >= 0 && id < g.n_slots)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int32_t rk = min(pp.rank[m][id], g.R);
                const float *a = (const float *)pp.a[m] + slot_row0(pp.row0[m], id, g.R) * g.N + n;
                const float *dv = g.dv + t * 2 * g.R + m * g.R;
                float d = 0.0f;
                for (int j = 0; j < rk; ++j) d = fmaf(dv[j], a[(int64_t)j * g.N], d);
                val += d;
            }
        g.dx[t * g.N + n] = val;
    }
}

// ---------------------------------------------------------------------------
// dA and dB: out[slot][j][n] = s sum over the slot's rows t of p[t][j] q[t][n].
// A workgroup takes 256 columns n of one slot, 8 ranks j at a time; slots
// without rows, and ranks past the slot's, get zeros.
// ---------------------------------------------------------------------------
struct outer_args {
    const void *q[2];                  // per projection: the rows' wide side
    const float *p;                    // [T][2R]
    const float *scale[2];             // null: p holds the scale
    const int32_t *rank[2];
    void *out[2];
    int64_t slot_stride, j_stride, n_stride;    // of out, in elements
    const int32_t *offsets, *perm;
    int32_t T, N, R, n_slots;
};

template <int DT> __global__ void __launch_bounds__(256) k_seg_outer(outer_args g) {
    typedef typename elem<DT>::T E;
    const int slot = blockIdx.x, m = blockIdx.z, n = blockIdx.y * 256 + threadIdx.x;
    if (n >= g.N) return;
    const int p0 = max(g.offsets[slot + 1], 0), p1 = min(g.offsets[slot + 2], g.T);
    const int32_t r = min(g.rank[m][slot], g.R);
    const E *q = (const E *)g.q[m];
    E *out = (E *)g.out[m] + slot * g.slot_stride + n * g.n_stride;
    const float sc = g.scale[m] ? g.scale[m][slot] : 1.0f;
    for (int j0 = 0; j0 < g.R; j0 += 8) {
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (j0 < r)
            for (int p = p0; p < p1; ++p) {
                const int64_t t = perm_row(g.perm, p, g.T);
                if (t < 0) continue;
                const float f = elem<DT>::load(q, t * g.N + n);
                const float *pv = g.p + t * 2 * g.R + m * g.R + j0;
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = fmaf(pv[e], f, acc[e]);
            }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            elem<DT>::store(out, (j0 + e) * g.j_stride, j0 + e < r ? sc * acc[e] : 0.0f);
    }
}

__global__ void __launch_bounds__(256) k_zero16(uint4 *p, int64_t n) {
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) p[i] = make_uint4(0u, 0u, 0u, 0u);
}

// ---------------------------------------------------------------------------
bwd_layout make_bwd_layout(int32_t T, int32_t n_slots, int32_t R, int32_t d_in, int32_t d_out, int32_t dtype) {
    bwd_layout B;
    B.L = make_ws_layout(T, n_slots, 2 * R, 0);
    const size_t t = (size_t)(T > 0 ? T : 1), eb = dtype == LORA_F32 ? 4 : 2;
    const size_t segs = (size_t)n_slots < t ? (size_t)n_slots : t;
    size_t o = B.L.total;
    B.dy = o;      o = align256(o + 2 * t * (size_t)d_out * eb);
    B.dv = o;      o = align256(o + 4 * t * 2 * (size_t)R);
    B.oct = o;     o = align256(o + (dtype == LORA_BF16 ? segs * 2 * (size_t)R * (size_t)d_in * 2 : 0));
    B.row0 = o;    o = align256(o + 4 * (size_t)n_slots);
    B.rank = o;    o = align256(o + 4 * (size_t)n_slots);
    B.scale = o;   o = align256(o + 4 * (size_t)n_slots);
    B.partial = o;
    const size_t tp = (t + 255) / 256 * 256, np = ((size_t)d_in + 255) / 256 * 256;
    const size_t need = dtype == LORA_BF16 && T > 0 ? 4 * (size_t)kMaxGemmSplit * tp * np : 0;
    B.total = align256(o + (need < kGemmPartialCap ? need : kGemmPartialCap));
    return B;
}

template <int DT>
static void launch_outer(outer_args g, hipStream_t s) {
    hipLaunchKernelGGL(k_seg_outer<DT>, dim3(g.n_slots, ceil_div(g.N, 256), 2), dim3(256), 0, s, g);
}

lora_status_t launch_zero(void *p, size_t bytes, hipStream_t s) {
    const int64_t n = (int64_t)(bytes / 16);
    if (n > 0)
        hipLaunchKernelGGL(k_zero16, dim3((uint32_t)(n < (4096 * 256) ? (n + 255) / 256 : 4096)), dim3(256), 0, s,
                           (uint4 *)p, n);
    return hip_status(hipGetLastError());
}

template <int DT> static lora_status_t backward(const gated_bwd_call &c, const bwd_layout &B, hipStream_t s) {
    typedef typename elem<DT>::T E;
    const lora_pool_t *p = c.pools;
    const int32_t T = c.T, K = p[0].d_in, F = p[0].d_out, R = p[0].max_rank, S = p[0].n_slots;
    const ws_layout &L = B.L;
    void *ws = c.ws;
    lora_status_t st = launch_segments(c.ids, T, S, L, ws, s, 1);
    if (st != LORA_OK) return st;
    const int32_t *perm = ws_ptr<int32_t>(ws, L.perm), *offsets = ws_ptr<int32_t>(ws, L.offsets);
    float *v = ws_ptr<float>(ws, L.v), *dv = ws_ptr<float>(ws, B.dv);
    E *dg = ws_ptr<E>(ws, B.dy), *du = dg + (int64_t)T * F;
    pair_pools pp;
    for (int m = 0; m < 2; ++m) {
        pp.a[m] = p[m].a;
        pp.b[m] = p[m].b;
        pp.scale[m] = p[m].scale;
        pp.rank[m] = p[m].rank;
        pp.row0[m] = p[m].row0;
    }
    const int64_t n_vec = (int64_t)T * F / vec16<DT>::n;
    hipLaunchKernelGGL(k_gated_dact<DT>, dim3((uint32_t)(n_vec < (1 << 24) ? (n_vec + 255) / 256 : 1 << 16)),
                       dim3(256), 0, s, (const E *)c.gate, (const E *)c.up, (const E *)c.dh, dg, du, n_vec, c.act);
    // v = x A (also records the bad ids); dv
    st = launch_shrink(c.x, T, p, 2, c.ids, true, v, L, ws, s);
    if (st != LORA_OK) return st;
    hipLaunchKernelGGL(k_rank_grad_rows<DT>, dim3(T, 2), dim3(256), 0, s, dg, (int64_t)T * F, T, F, pp, S, R, c.ids,
                       dv);
    if (c.dx && DT == LORA_F32) {
        dx_f32_args g{{(const float *)dg, (const float *)du}, {(const float *)c.W[0], (const float *)c.W[1]},
                      (float *)c.dx, dv, c.ids, perm, T, F, K, S, R, ceil_div(K, 64)};
        hipLaunchKernelGGL(k_dx_f32, dim3(ceil_div(T, 64) * g.n_tiles_n), dim3(256), 0, s, g, pp);
    } else if (c.dx) {
        uint16_t *oct = ws_ptr<uint16_t>(ws, B.oct);
        int32_t *row0 = ws_ptr<int32_t>(ws, B.row0), *rank = ws_ptr<int32_t>(ws, B.rank);
        float *scale = ws_ptr<float>(ws, B.scale);
        hipLaunchKernelGGL(k_a_octets, dim3(S < T ? S : T, ceil_div(K, 256)), dim3(256), 0, s, pp,
                           ws_ptr<int32_t>(ws, L.seg_id), ws_ptr<int32_t>(ws, L.n_seg), S, K, R, oct, row0, rank,
                           scale);
        nt_args nt{{(const uint16_t *)dg, (const uint16_t *)du}, {(const uint16_t *)c.W[0], (const uint16_t *)c.W[1]},
                   F, ceil_div(F, 64) * 64};
        gemm_args g{};
        g.y = (uint16_t *)c.dx;
        g.T = T;
        g.K = 2 * nt.Fp;
        g.N = K;
        g.perm = perm;
        g.b = oct;
        g.scale = scale;
        g.rank = rank;
        g.row0 = row0;
        g.n_slots = S;
        g.max_rank = 2 * R;
        g.ids = c.ids;
        g.v = dv;
        g.v_stride = 2 * R;
        g.partial = ws_ptr<float>(ws, B.partial);
        const gemm_plan pl = plan_gemm(T, g.K, g.N, c.ws_bytes - B.partial);
        g.n_tiles_m = ceil_div(T, pl.bm);
        g.n_tiles_n = ceil_div(g.N, pl.bn);
        g.col_strips = col_strips_pay(T, g.N, g.n_tiles_n);
        if (pl.bm == 256 && pl.bn == 256) launch_nt_cfg<256, 256, 2, 8, 2, 2, 8>(g, nt, pl, s);
        else if (pl.bm == 256 && pl.bn == 128) launch_nt_cfg<256, 128, 2, 8, 2, 2, 8>(g, nt, pl, s);
        else if (pl.bn == 128) launch_nt_cfg<128, 128, 2, 4, 2, 4, 8>(g, nt, pl, s);
        else launch_nt_cfg<128, 64, 2, 4, 2, 2, 4>(g, nt, pl, s);
    }
    if (c.dA[0]) {
        outer_args g{};
        g.offsets = offsets;
        g.perm = perm;
        g.T = T;
        g.R = R;
        g.n_slots = S;
        g.rank[0] = p[0].rank;
        g.rank[1] = p[1].rank;
        g.slot_stride = (int64_t)R * K;
        g.j_stride = 1;
        g.n_stride = R;
        g.q[0] = g.q[1] = c.x;
        g.p = dv;
        g.N = K;
        g.out[0] = c.dA[0];
        g.out[1] = c.dA[1];
        launch_outer<DT>(g, s);
        g.slot_stride = (int64_t)R * F;
        g.j_stride = F;
        g.n_stride = 1;
        g.q[0] = dg;
        g.q[1] = du;
        g.p = v;
        g.scale[0] = p[0].scale;
        g.scale[1] = p[1].scale;
        g.N = F;
        g.out[0] = c.dB[0];
        g.out[1] = c.dB[1];
        launch_outer<DT>(g, s);
    }
    return hip_status(hipGetLastError());
}

lora_status_t launch_gated_backward(const gated_bwd_call &c, const bwd_layout &B, hipStream_t s) {
    return c.pools[0].dtype == LORA_F32 ? backward<LORA_F32>(c, B, s) : backward<LORA_BF16>(c, B, s);
}

}  // namespace lora
