// Backward pass of the gated pair h = act(g) * u, base weights frozen:
//   dg = dh * u * act'(g),  du = dh * act(g)                        k_gated_dact
//   dv = s_a dg B_a^T   [T, r] for each of the two                  k_rank_grad
//   dx = dg Wg^T + du Wu^T + dv_g Ag_a^T + dv_u Au_a^T              k_gemm_nt / dx_f32
//   dA_a = sum over a's rows of x_t^T dv_t                          k_seg_outer
//   dB_a = s_a sum over a's rows of v_t^T dg_t,  v = x A_a          k_seg_outer
// Rows are visited in adapter order (the segment builder's perm), so every
// sum over an adapter's rows runs over neighbours, in row order, without
// atomics: results repeat bitwise.
#include "gated_common.hpp"

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

// dg and du of 16 bytes of values per thread.  bf16: two bf16 parts each, hi =
// bf16(f) and, `lo` values on, bf16(f - hi), together within 2^-17 of f.  The
// adapters' gradients take both (a sum over an adapter's few rows shows a
// rounding of dg: with hi alone their error against 64 bits was 1.3 to 1.8 times
// that of 32-bit products); dx, a sum over 2 d_out terms, takes hi, one more
// rounding of an operand, for half the matrix products (its error against 64
// bits is 1.2 to 1.43 times that of 32-bit products, over drawn sizes).
// Bound by its bytes: 2048 x 14336, 62 us, 6.6 TB/s.
template <int DT>
__global__ void __launch_bounds__(256) k_gated_dact(const typename elem<DT>::T *gate, const typename elem<DT>::T *up,
                                                    const typename elem<DT>::T *dh, typename elem<DT>::T *dg,
                                                    typename elem<DT>::T *du, int64_t lo, int64_t n_vec, int act) {
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
        const uint4 gq = vec16<DT>::narrow(g), uq = vec16<DT>::narrow(u);
        stg16(dg + i * VN, gq);
        stg16(du + i * VN, uq);
        if constexpr (DT == LORA_BF16) {
            float gh[VN], uh[VN];
            vec16<DT>::widen(gq, gh);
            vec16<DT>::widen(uq, uh);
#pragma unroll
            for (int e = 0; e < VN; ++e) {
                g[e] = second_part(g[e] - gh[e]);
                u[e] = second_part(u[e] - uh[e]);
            }
            stg16(dg + lo + i * VN, vec16<DT>::narrow(g));
            stg16(du + lo + i * VN, vec16<DT>::narrow(u));
        }
    }
}

// ---------------------------------------------------------------------------
// dv.  fp32: one workgroup per row and projection: rank octet by octet, each
// thread strides the row's N values against the slot's B octets (190 rows, 1384
// wide: 8 us, latency).
// ---------------------------------------------------------------------------
template <int DT>
__global__ void __launch_bounds__(256) k_rank_grad_rows(const typename elem<DT>::T *dy, int64_t dy_stride, int32_t T,
                                                        int32_t N, pair_pools pp, int32_t n_slots, int32_t R,
                                                        const int32_t *ids, float *dv) {
    typedef typename elem<DT>::T E;
    const int64_t wg = grid_index();
    if (wg >= 2ll * T) return;
    const int t = (int)(wg >> 1), m = (int)(wg & 1);
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

// bf16: a grouped product over adapter segments, as k_shrink_grouped, of up to
// 32 rows of dg (or du, blockIdx.z) with the adapter's B.  Both operands go
// global -> LDS by DMA, NS stages of 128 n; B's octets ([n][8 ranks], 16 bytes
// a column) lie in LDS as in memory and are read transposed
// (ds_read_b64_tr_b16: 4 n of 16 ranks per instruction).  Each of the 4
// wavefronts takes a 32-n quarter of every stage; N is split over blockIdx.y.
// Two stages for wide ranks, so that two workgroups fit a CU (64 ranks, 2048 rows
// of 14336: 57 us, with three stages 64; 16 ranks 46 and 40).
// Partial sums go to part[m][split][sorted position][R].  Bound by the bytes of
// dg's and du's parts (2048 rows of 14336: 43 us, 5.5 TB/s).
template <int RCH> struct rank_grad_cfg {
    static constexpr int BR = kShrinkRows, NR = RCH * 16, BK = 128, CH = BK / 8, NS = RCH > 2 ? 2 : 3;
    static constexpr int OCT = BK * 8 + 16;              // elements between octets (32 bytes apart in the banks)
    static constexpr int YST = BR * BK, STAGE = 2 * YST + (NR / 8) * OCT;   // dy's two parts, B
    static constexpr int YI = BR * CH / 256, BI = NR / 8 * BK / 256;   // DMA instructions per wave per stage
    static constexpr int RED = 4 * BR * (NR + 1);
    static constexpr int LDS_BYTES = NS * STAGE * 2 > RED * 4 ? NS * STAGE * 2 : RED * 4;
};

struct rank_grad_args {
    const uint16_t *dy;                // first and second parts: [2][2][T][N]
    int32_t T, N, R, n_slots, n_chunk;
    const int32_t *perm, *seg_id, *seg_start, *n_seg, *blk_start, *blk_seg;
    float *part;
};

template <int RCH> __global__ void __launch_bounds__(256) k_rank_grad(rank_grad_args g, pair_pools pp) {
    typedef rank_grad_cfg<RCH> C;
    constexpr int BR = C::BR, NR = C::NR, BK = C::BK, CH = C::CH, NS = C::NS, PER = 2 * C::YI + C::BI;
    __shared__ __attribute__((aligned(1024))) uint16_t smem[C::LDS_BYTES / 2];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, m = blockIdx.z;
    const int nseg = min(*g.n_seg, g.n_slots);
    if (nseg <= 0 || (int)blockIdx.x >= g.blk_start[nseg]) return;
    const int seg = g.blk_seg[blockIdx.x];
    if (seg < 0 || seg >= nseg) return;
    const int32_t id = g.seg_id[seg];
    if (id < 0 || id >= g.n_slots) return;
    const int64_t s0 = g.seg_start[seg], s1 = g.seg_start[seg + 1];
    const int64_t q0 = s0 + ((int64_t)blockIdx.x - g.blk_start[seg]) * BR;
    if (s0 < 0 || s1 > g.T || q0 < s0 || q0 >= s1) return;
    const int p0 = (int)q0, pend = (int)(s1 < q0 + BR ? s1 : q0 + BR);
    const int32_t rk = min(pp.rank[m][id], g.R);
    const int n_begin = blockIdx.y * g.n_chunk, n_end = min(g.N, n_begin + g.n_chunk);
    const int64_t lo = 2ll * g.T * g.N;
    const uint16_t *dy = g.dy + (int64_t)m * g.T * g.N;
    const uint16_t *b = (const uint16_t *)pp.b[m] + slot_row0(pp.row0[m], id, g.R) * g.N;

    int64_t yrow[C::YI];
    int ycol[C::YI];
#pragma unroll
    for (int j = 0; j < C::YI; ++j) {
        const int c = (wave * C::YI + j) * 64 + lane, r = c / CH, p = p0 + r;
        const int32_t t = p < pend ? perm_row(g.perm, p, g.T) : -1;
        yrow[j] = t >= 0 ? (int64_t)t * g.N : -1;
        ycol[j] = 8 * ((c % CH) ^ (r % CH));
    }
    auto dma_stage = [&](int kt, int buf) {
        uint16_t *ys = smem + buf * C::STAGE, *bs = ys + 2 * C::YST;
        const int k0 = n_begin + kt * BK;
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int j = 0; j < C::YI; ++j) {
                const int n = k0 + ycol[j];
                dma16(yrow[j] >= 0 && n < n_end ? (const void *)(dy + part * lo + yrow[j] + n) : (const void *)g_zero16,
                      ys + part * C::YST + (wave * C::YI + j) * 64 * 8);
            }
#pragma unroll
        for (int j = 0; j < C::BI; ++j) {                 // half an octet's 128 columns per instruction
            const int i = wave * C::BI + j, o = i >> 1, n = k0 + (i & 1) * 64 + lane;
            dma16(8 * o < rk && n < n_end ? (const void *)(b + ((int64_t)o * g.N + n) * 8) : (const void *)g_zero16,
                  bs + o * C::OCT + (i & 1) * 64 * 8);
        }
    };
    auto wait_stage = [&](int ahead) {
        if (ahead >= 2) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * PER) : "memory");
        else if (ahead == 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(PER) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    };
    f32x4_t acc[2][RCH];
#pragma unroll
    for (int rb = 0; rb < 2; ++rb)
#pragma unroll
        for (int rc = 0; rc < RCH; ++rc) acc[rb][rc] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const int l16 = lane & 15, kg = lane >> 4;
    const int nk = rk > 0 ? (n_end - n_begin + BK - 1) / BK : 0;
#pragma unroll
    for (int st = 0; st < NS - 1; ++st)
        if (st < nk) dma_stage(st, st);
    for (int kt = 0; kt < nk; ++kt) {
        wait_stage(min(NS - 2, nk - 1 - kt));
        // and this wave's reads of the stage before, whose buffer is refilled next
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (kt + NS - 1 < nk) dma_stage(kt + NS - 1, (kt + NS - 1) % NS);
        const uint16_t *ys = smem + (kt % NS) * C::STAGE, *bs = ys + 2 * C::YST;
        uint4 yq[2][2];
        bf16x8_t bq[RCH];
#pragma unroll
        for (int rb = 0; rb < 2; ++rb) {
            const int r = rb * 16 + l16;
#pragma unroll
            for (int part = 0; part < 2; ++part)
                yq[part][rb] = *reinterpret_cast<const uint4 *>(ys + part * C::YST + r * BK +
                                                                8 * ((4 * wave + kg) ^ (r % CH)));
        }
#pragma unroll
        for (int rc = 0; rc < RCH; ++rc) {
            // lane's address: n of its quarter's k group, ranks 4 (l16 & 3) .. + 3 of 16
            short4_t h[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int n = 32 * wave + 8 * kg + 4 * i + (l16 >> 2);
                const uint16_t *at = bs + (2 * rc + ((l16 & 3) >> 1)) * C::OCT + n * 8 + 4 * (l16 & 1);
                h[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4_t *)(reinterpret_cast<uintptr_t>(at)));
            }
            const short8_t hv = {h[0][0], h[0][1], h[0][2], h[0][3], h[1][0], h[1][1], h[1][2], h[1][3]};
            bq[rc] = __builtin_bit_cast(bf16x8_t, hv);
        }
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int rb = 0; rb < 2; ++rb)
#pragma unroll
                for (int rc = 0; rc < RCH; ++rc)
                    acc[rb][rc] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, yq[part][rb]),
                                                                          bq[rc], acc[rb][rc], 0, 0, 0);
    }
    __syncthreads();                                      // all waves done with the stages
    float (*red)[BR][NR + 1] = reinterpret_cast<float (*)[BR][NR + 1]>(smem);
#pragma unroll
    for (int rb = 0; rb < 2; ++rb)
#pragma unroll
        for (int rc = 0; rc < RCH; ++rc)
#pragma unroll
            for (int q = 0; q < 4; ++q) red[wave][rb * 16 + 4 * kg + q][rc * 16 + l16] = acc[rb][rc][q];
    __syncthreads();
    float *part = g.part + (int64_t)(m * gridDim.y + blockIdx.y) * g.T * g.R;
    for (int e = tid; e < BR * g.R; e += 256) {
        const int i = e / g.R, j = e % g.R;
        if (p0 + i < pend)
            part[(int64_t)(p0 + i) * g.R + j] = (red[0][i][j] + red[1][i][j]) + (red[2][i][j] + red[3][i][j]);
    }
}

// A of the batch's slots in rank octets, gate's ranks then up's: [segment][2R /
// 8][d_in][8], with the tables (row0, rank, scale) that make them one pool of
// max_rank 2R for the low-rank pass of the dx product.  dv holds the scales
// already, so the table's are 1.  Octet o of 256 values of d_in of segment i.
struct a_octets_args {
    const int32_t *seg_id, *n_seg;
    int32_t n_slots, K, R, k_blocks;
    uint16_t *oct;
    int32_t *row0, *rank;
    float *scale;
};

__device__ __forceinline__ void a_octets(const a_octets_args &g, const pair_pools &pp, int i, int kb, int o) {
    if (i >= min(*g.n_seg, g.n_slots)) return;
    const int32_t id = g.seg_id[i], R = g.R;
    if (id < 0 || id >= g.n_slots) return;
    const int m = 8 * o >= R, j0 = 8 * o - m * R;
    const int32_t r[2] = {min(pp.rank[0][id], R), min(pp.rank[1][id], R)};
    if (kb == 0 && o == 0 && threadIdx.x == 0) {
        g.row0[id] = i * 2 * R;
        g.rank[id] = r[0] > 0 || r[1] > 0 ? 2 * R : 0;
        g.scale[id] = 1.0f;
    }
    const int k = kb * 256 + threadIdx.x;
    if (k >= g.K) return;
    const uint16_t *a = (const uint16_t *)pp.a[m] + (slot_row0(pp.row0[m], id, R) + j0) * g.K + k;
    uint32_t e[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) e[q] = j0 + q < (m ? r[1] : r[0]) ? a[(int64_t)q * g.K] : 0u;
    stg16(g.oct + (((int64_t)i * 2 * R / 8 + o) * g.K + k) * 8,
          make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16));
}

// The rank vectors as the products that follow read them.  dv, fp32 [T][2R]
// in batch order: the partial sums added in split order, times the slot's
// scale; zero for rows without an adapter.  vt, bf16 [2][2][2R][Tp]: s v and
// dv, transposed, in adapter order with every segment's start on a multiple
// of 32 (its first work block), each value as two bf16 parts (hi = bf16(f),
// lo = bf16(f - hi): together within 2^-17 of f, far below the rounding of
// the bf16 gradients they add up to).  Places past a segment's rows are
// filled with zeros.  A workgroup: 32 positions of one work block and 8 ranks
// (blockIdx.y), or 32 rows of the base block (grid.x from n_work on), or, from
// first_octet on, A's octets, in the same launch because neither alone keeps
// the chip busy.  2048 rows: 7 us, latency.
struct rank_finish_args {
    const float *v, *part;
    int32_t n_split, T, R, n_slots, n_work, Tp;
    const int32_t *perm, *offsets, *seg_id, *seg_start, *n_seg, *blk_start, *blk_seg;
    float *dv;
    uint16_t *vt;
    int32_t *slot_blk;                 // [n_slots]: a segment's first work block, by its slot
    int32_t first_octet;
};

__global__ void __launch_bounds__(256) k_rank_finish(rank_finish_args g, a_octets_args oc, pair_pools pp) {
    constexpr int BR = kShrinkRows;
    const int R2 = 2 * g.R;
    if ((int)blockIdx.x >= g.first_octet) {
        const int item = (int)blockIdx.x - g.first_octet;
        a_octets(oc, pp, item / oc.k_blocks, item % oc.k_blocks, blockIdx.y);
        return;
    }
    if ((int)blockIdx.x >= g.n_work) {
        if (blockIdx.y) return;
        const int p0 = ((int)blockIdx.x - g.n_work) * BR, pend = min(min(g.offsets[1], p0 + BR), g.T);
        for (int e = threadIdx.x; e < BR * R2; e += 256) {
            const int p = p0 + e / R2;
            const int64_t t = p < pend ? perm_row(g.perm, p, g.T) : -1;
            if (t >= 0) g.dv[t * R2 + e % R2] = 0.0f;
        }
        return;
    }
    const int nseg = min(*g.n_seg, g.n_slots);
    if (nseg <= 0 || (int)blockIdx.x >= g.blk_start[nseg]) return;
    const int seg = g.blk_seg[blockIdx.x];
    if (seg < 0 || seg >= nseg) return;
    const int32_t id = g.seg_id[seg];
    if (id < 0 || id >= g.n_slots) return;
    if (threadIdx.x == 0 && blockIdx.y == 0 && (int)blockIdx.x == g.blk_start[seg]) g.slot_blk[id] = blockIdx.x;
    const int p0 = g.seg_start[seg] + ((int)blockIdx.x - g.blk_start[seg]) * BR;
    const int pend = min(min(g.seg_start[seg + 1], p0 + BR), g.T);
    const int i = threadIdx.x & 31, p = p0 + i;
    const int64_t t = p >= 0 && p < pend ? perm_row(g.perm, p, g.T) : -1;
    const int64_t at = (int64_t)blockIdx.x * BR + i;
    {
        const int j = blockIdx.y * 8 + (threadIdx.x >> 5), m = j >= g.R, jj = j - m * g.R;
        float f[2] = {0.0f, 0.0f};                        // s v, dv
        if (t >= 0 && jj < min(pp.rank[m][id], g.R)) {
            const float s = pp.scale[m][id];
            f[0] = s * g.v[t * R2 + j];
            const float *part = g.part + ((int64_t)m * g.n_split * g.T + p) * g.R + jj;
            for (int c = 0; c < g.n_split; ++c) f[1] += part[(int64_t)c * g.T * g.R];
            f[1] *= s;
        }
        if (t >= 0) g.dv[t * R2 + j] = f[1];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const uint32_t hi = f32_to_bf16_bits(f[w]);
            const float rest = second_part(f[w] - __uint_as_float(hi << 16));
            uint16_t *o = g.vt + (int64_t)w * 2 * R2 * g.Tp + (int64_t)j * g.Tp + at;
            o[0] = (uint16_t)hi;
            o[(int64_t)R2 * g.Tp] = (uint16_t)f32_to_bf16_bits(rest);
        }
    }
}

// ---------------------------------------------------------------------------
// dx, bf16: rows of [dg, du] times rows of [Wg, Wu] (both contiguous along the
// sum, so both tiles are DMA'd rows with one swizzle and ds_read_b128
// fragments), the two projections one after the other along K.  Tiles,
// hand-off, low-rank pass, store and K split are those of the forward GEMM, and
// so is the bound (LDS and matrix cores taking turns: 2048 x 28672 x 4096, 463
// us, 1039 TFLOP/s, and 16 us for the reduction).
// ---------------------------------------------------------------------------
struct nt_args {
    const uint16_t *a[2], *w[2];       // [T][F], [N][F]
    int32_t F, Fp;                     // F rounded up to whole K steps
    const int32_t *n_seg;
};

// Where a product split over K gets its low-rank term: on the matrix cores by
// the first piece of each tile where the adapters have 64 rows or more on
// average, else row by row in the reduction.  (2048 rows of 4 adapters, 8B
// sizes: pieces and reduction 475 us against 511 row by row; 777 rows of 24
// adapters of up to 40 ranks, 1048 x 2744: 80 against 50.)
__device__ __forceinline__ bool term_in_reduction(const gemm_args &g, const nt_args &nt) {
    return (int64_t)*nt.n_seg * 64 > g.T;
}

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

    __shared__ int32_t s_t[BM], s_id[BM];
    int32_t *s_meta_t = SPLIT ? nullptr : s_t;            // a piece stores every row of its partial tile
    const bool low_rank = !SPLIT || (split == 0 && !term_in_reduction(g, nt));
    if (low_rank) {
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
    if (low_rank)
        lora_pass_impl<RB, CB, (RB >= 2 ? 2 : 1), 1, (RB >= 2 ? 2 : 1), 1, 0, true>(g, acc, s_t, s_id, n0, wm * WM,
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

// The pieces' sums in split order; a thread owns 8 columns of one row.
template <int BM, int BN> __global__ void __launch_bounds__(256) k_nt_reduce(gemm_args g, nt_args nt) {
    constexpr int CPR = BN / 8, RW = 256 / CPR, CHUNKS = BM / RW;
    const int per = gridDim.x / kXcds, rem = gridDim.x % kXcds, xcd = blockIdx.x % kXcds;
    const int item = xcd * per + min(xcd, rem) + blockIdx.x / kXcds;   // whole tiles per XCD, as k_splitk_reduce
    const int tidx = item / CHUNKS, chunk = item % CHUNKS;
    int tm, tn;
    grouped_tile(g.tile_base + tidx, g.n_tiles_m, g.n_tiles_n, g.col_strips, tm, tn);
    const int r = chunk * RW + threadIdx.x / CPR, c = (threadIdx.x % CPR) * 8;
    const int p = tm * BM + r, n = tn * BN + c;
    const int64_t t = p < g.T ? perm_row(g.perm, p, g.T) : -1;
    // The low-rank sums: the row's threads read neighbouring columns of the
    // octets (16 bytes each), and hand them over in LDS.
    __shared__ float s_d[RW][BN];
    if (term_in_reduction(g, nt)) {                        // (uniform)
        const int32_t id = t >= 0 ? g.ids[t] : -1;
        const int32_t rk = id >= 0 && id < g.n_slots ? g.rank[id] : 0;
        const int lr = threadIdx.x / CPR, lc = threadIdx.x % CPR, nc = tn * BN + lc;
        float d[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        const float *vrow = g.v + (t < 0 ? 0 : t) * g.v_stride;
        const uint16_t *b = g.b + (rk > 0 ? (int64_t)g.row0[id] * g.N : 0) + (int64_t)nc * 8;
        // two octets at a time (rk is 2 max_rank, a multiple of 16)
        for (int j = 0; j < rk; j += 16, b += (int64_t)g.N * 16) {
            f32x4_t vv[2][2];
            uint4 bq[2][8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                vv[h][0] = *reinterpret_cast<const f32x4_t *>(vrow + j + 8 * h);
                vv[h][1] = *reinterpret_cast<const f32x4_t *>(vrow + j + 8 * h + 4);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    bq[h][q] = nc + CPR * q < g.N ? ldg16(b + (int64_t)h * g.N * 8 + CPR * q * 8)
                                                  : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    float bf[8];
                    vec16<LORA_BF16>::widen(bq[h][q], bf);
#pragma unroll
                    for (int e = 0; e < 8; ++e) d[q] = fmaf(vv[h][e >> 2][e & 3], bf[e], d[q]);
                }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) s_d[lr][lc + CPR * q] = d[q];
    }
    __syncthreads();
    if (t < 0 || n >= g.N) return;
    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const float *src = g.partial + ((int64_t)tidx * g.splits * BM + r) * BN + c;
    for (int s = 0; s < g.splits; ++s, src += BM * BN) {
        const float4 a = *reinterpret_cast<const float4 *>(src), b = *reinterpret_cast<const float4 *>(src + 4);
        o[0] += a.x; o[1] += a.y; o[2] += a.z; o[3] += a.w;
        o[4] += b.x; o[5] += b.y; o[6] += b.z; o[7] += b.w;
    }
    if (term_in_reduction(g, nt))
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] += s_d[threadIdx.x / CPR][c + q];
    stg16(g.y + t * g.N + n, vec16<LORA_BF16>::narrow(o));
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
        hipLaunchKernelGGL((k_nt_reduce<BM, BN>), dim3(pl.tail * (BM / (2048 / BN))), dim3(256), 0, s, g, nt);
    }
}

// The sum over both projections is long (twice d_out), so a grid that would
// not fill the chip with the largest tiles splits it over K rather than take
// smaller tiles (2048 x 28672 x 4096: 128 tiles in two pieces each against
// 256 tiles of 256 x 128).
static gemm_plan plan_dx(int T, int K, int N, size_t partial_bytes) {
    const int tiles = ceil_div(T, 256) * ceil_div(N, 256);
    if (tiles < 208 && K >= 8192 && T >= 256) {
        int splits = 256 / tiles;
        if (splits > kMaxGemmSplit) splits = kMaxGemmSplit;
        if (splits > K / 2048) splits = K / 2048;
        if (splits >= 2 && tiles * splits >= 208 && (size_t)splits * tiles * 256 * 256 * 4 <= partial_bytes) {
            const int kc = ceil_div(ceil_div(K, splits), 64) * 64;
            return gemm_plan{256, 256, 0, tiles, ceil_div(K, kc), kc};
        }
    }
    return plan_gemm(T, K, N, partial_bytes);
}

// ---------------------------------------------------------------------------
// dx, fp32: 64 x 64 tiles on v_mfma_f32_32x32x2_f32, the sum over dg's columns
// then du's (each in whole steps of 32); grids of few tiles split the steps.
// Threads that own 4 columns of a row then add the low-rank terms from A's rows.
// (190 x 2768 x 520: 14 us and 11 for the reduction, both latency; see
// k_dx_outer_f32.)
// ---------------------------------------------------------------------------
struct dx_f32_args {
    const float *a0, *a1, *w0, *w1;
    float *dx;
    const float *dv;
    const int32_t *ids, *perm;
    float *partial;                    // [tile][split][64][64]
    int32_t T, F, N, n_slots, R, n_tiles_n, splits, k_chunk;
};

__device__ __forceinline__ void dx_finish4(const dx_f32_args &g, const pair_pools &pp, int64_t t, int n,
                                           float (&o)[4]) {
    const int32_t id = g.ids[t];
    if (id >= 0 && id < g.n_slots) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int32_t rk = min(pp.rank[m][id], g.R);
            const float *a = (const float *)pp.a[m] + slot_row0(pp.row0[m], id, g.R) * g.N + n;
            const float *dv = g.dv + t * 2 * g.R + m * g.R;
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
            for (int j = 0; j < rk; ++j) {
                const float4 f = *reinterpret_cast<const float4 *>(a + (int64_t)j * g.N);
                const float s = dv[j];
                d[0] = fmaf(s, f.x, d[0]);
                d[1] = fmaf(s, f.y, d[1]);
                d[2] = fmaf(s, f.z, d[2]);
                d[3] = fmaf(s, f.w, d[3]);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) o[q] += d[q];
        }
    }
    *reinterpret_cast<float4 *>(g.dx + t * g.N + n) = make_float4(o[0], o[1], o[2], o[3]);
}

// Workgroup b of n.
template <bool SPLIT>
__device__ __forceinline__ void dx_f32(const dx_f32_args &g, const pair_pools &pp, int b, int n) {
    constexpr int BK = 32, NS = 3, AST = 64 * BK, STAGE = 2 * AST, LD = 64 + 4, PER = 4;
    __shared__ __attribute__((aligned(1024))) float smem[NS * STAGE];     // stages: [64][BK] of each; sums: [64][LD]
    static_assert(64 * LD <= NS * STAGE, "the sums fit the stages' LDS");
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, wm = w >> 1, wn = w & 1;
    int tm, tn, split;
    f32_tile(b, n, (g.T + 63) / 64, SPLIT ? g.splits : 1, tm, tn, split);
    const int tile = tm * g.n_tiles_n + tn, m0 = tm * 64, n0 = tn * 64;
    const int Fp = (g.F + BK - 1) / BK * BK;
    const int k_begin = split * g.k_chunk, k_end = min(2 * Fp, k_begin + g.k_chunk);
    // DMA: 16-byte chunk 256 j + tid of an operand is at row / 8, place % 8, and
    // holds the row's chunk place ^ (row % 8)
    int64_t arow[2], wrow[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int r = 32 * j + (tid >> 3);
        const int32_t t = m0 + r < g.T ? perm_row(g.perm, m0 + r, g.T) : -1;
        arow[j] = t >= 0 ? (int64_t)t * g.F : -1;
        wrow[j] = n0 + r < g.N ? (int64_t)(n0 + r) * g.F : -1;
    }
    const int kk = 4 * ((tid & 7) ^ ((tid >> 3) & 7));
    auto dma_stage = [&](int kt, int buf) {
        float *as = smem + buf * STAGE, *wsm = as + AST;
        const int k0 = k_begin + kt * BK;
        const bool second = k0 >= Fp;                      // a step lies in one projection
        const float *a = second ? g.a1 : g.a0, *wt = second ? g.w1 : g.w0;
        const int f = k0 - (second ? Fp : 0) + kk;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            dma16(arow[j] >= 0 && f < g.F ? (const void *)(a + arow[j] + f) : (const void *)g_zero16,
                  as + (256 * j + w * 64) * 4);
            dma16(wrow[j] >= 0 && f < g.F ? (const void *)(wt + wrow[j] + f) : (const void *)g_zero16,
                  wsm + (256 * j + w * 64) * 4);
        }
    };
    f32x16_t acc;
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
    const int nk = (k_end - k_begin + BK - 1) / BK;
#pragma unroll
    for (int st = 0; st < NS - 1; ++st)
        if (st < nk) dma_stage(st, st);
    for (int kt = 0; kt < nk; ++kt) {
        if (kt + 1 < nk) asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NS - 2) * PER) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // and this wave's reads of the stage refilled next
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (kt + NS - 1 < nk) dma_stage(kt + NS - 1, (kt + NS - 1) % NS);
        // product i takes k = i from the lower half-wavefront, 16 + i from the upper
        const float *as = smem + (kt % NS) * STAGE + (wm * 32 + (lane & 31)) * BK;
        const float *wsm = smem + (kt % NS) * STAGE + AST + (wn * 32 + (lane & 31)) * BK;
        float a[16], b[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = 4 * ((4 * (lane >> 5) + i) ^ (lane & 7));
            *reinterpret_cast<f32x4_t *>(a + 4 * i) = *reinterpret_cast<const f32x4_t *>(as + c);
            *reinterpret_cast<f32x4_t *>(b + 4 * i) = *reinterpret_cast<const f32x4_t *>(wsm + c);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], acc, 0, 0, 0);
    }
    float *part = SPLIT ? g.partial + ((int64_t)tile * g.splits + split) * 64 * 64 : nullptr;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const int i = wm * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3), c = wn * 32 + (lane & 31);
        if (SPLIT) part[i * 64 + c] = acc[e];
        else smem[i * LD + c] = acc[e];
    }
    if (SPLIT) return;
    __syncthreads();
    for (int i = tid; i < 64 * 16; i += 256) {
        const int c = (i & 15) * 4, p = m0 + (i >> 4), n = n0 + c;
        const int64_t t = p < g.T ? perm_row(g.perm, p, g.T) : -1;
        if (t < 0 || n >= g.N) continue;
        float o[4];
        *reinterpret_cast<float4 *>(o) = *reinterpret_cast<const float4 *>(smem + (i >> 4) * LD + c);
        dx_finish4(g, pp, t, n, o);
    }
}

__global__ void __launch_bounds__(256) k_dx_reduce_f32(dx_f32_args g, pair_pools pp) {
    const int tile = blockIdx.x >> 2, r = (blockIdx.x & 3) * 16 + (threadIdx.x >> 4), c = (threadIdx.x & 15) * 4;
    const int p = tile / g.n_tiles_n * 64 + r, n = tile % g.n_tiles_n * 64 + c;
    const int64_t t = p < g.T ? perm_row(g.perm, p, g.T) : -1;
    if (t < 0 || n >= g.N) return;
    float o[4] = {0.f, 0.f, 0.f, 0.f};
    const float *part = g.partial + (int64_t)tile * g.splits * 64 * 64 + r * 64 + c;
    for (int s = 0; s < g.splits; ++s, part += 64 * 64) {
        const float4 f = *reinterpret_cast<const float4 *>(part);
        o[0] += f.x; o[1] += f.y; o[2] += f.z; o[3] += f.w;
    }
    dx_finish4(g, pp, t, n, o);
}

// ---------------------------------------------------------------------------
// dA and dB, fp32: out[slot][j][n] = s sum over the slot's rows t of p[t][j]
// q[t][n].  A workgroup takes 256 columns n of one slot and projection, 16
// ranks j at a time; 64 rows' indices and rank values at a time lie in LDS,
// so that the loads of q do not wait for them.  dA's workgroups and dB's are
// one launch.  Slots without rows, and ranks past the slot's, get zeros.  (190
// rows of 6 slots, 520 and 1384 wide: 10 us, latency.)
// ---------------------------------------------------------------------------
struct outer_f32_args {
    const float *x, *dg, *du, *v, *dv;  // [T][K], [T][F], [T][F], [T][2R] (times the scale: dv), [T][2R]
    float *dA0, *dA1, *dB0, *dB1;
    const int32_t *offsets, *perm;
    int32_t T, K, F, R, n_slots, tiles_k, tiles_f;
};

__device__ __forceinline__ void seg_outer_f32(const outer_f32_args &g, const pair_pools &pp, int64_t wg) {
    constexpr int J = 16, U = 8, CH = 64;
    __shared__ __attribute__((aligned(16))) float s_p[CH][J];
    __shared__ int32_t s_row[CH];
    const int64_t n_a = 2ll * g.n_slots * g.tiles_k;
    const bool is_a = wg < n_a;
    const int tiles = is_a ? g.tiles_k : g.tiles_f;
    int item = (int)(is_a ? wg : wg - n_a);
    if (!is_a && item >= 2 * g.n_slots * tiles) return;
    const int tile = item % tiles;
    item /= tiles;
    const int m = item & 1, slot = item >> 1;
    const int N = is_a ? g.K : g.F, R = g.R, n = tile * 256 + threadIdx.x;
    const int p0 = max(g.offsets[slot + 1], 0), p1 = min(g.offsets[slot + 2], g.T);
    const int32_t r = min(m ? pp.rank[1][slot] : pp.rank[0][slot], R);
    const float *q = (is_a ? g.x : (m ? g.du : g.dg)) + (n < N ? n : 0);
    const float *pv = (is_a ? g.dv : g.v) + m * R;
    float *out = is_a ? (m ? g.dA1 : g.dA0) + ((int64_t)slot * N + n) * R : (m ? g.dB1 : g.dB0) + (int64_t)slot * R * N + n;
    const int64_t j_stride = is_a ? 1 : N;
    const float sc = is_a ? 1.0f : (m ? pp.scale[1][slot] : pp.scale[0][slot]);
    for (int j0 = 0; j0 < R; j0 += J) {
        float acc[J] = {};
        if (j0 < r)
            for (int p = p0; p < p1; p += CH) {
                const int rows = min(CH, p1 - p);
                __syncthreads();
                if ((int)threadIdx.x < CH)
                    s_row[threadIdx.x] = (int)threadIdx.x < rows ? perm_row(g.perm, p + threadIdx.x, g.T) : -1;
                {
                    const int i = threadIdx.x >> 2, j = (threadIdx.x & 3) * 4;
                    const int32_t t = i < rows ? perm_row(g.perm, p + i, g.T) : -1;
                    *reinterpret_cast<f32x4_t *>(&s_p[i][j]) = load4(t >= 0 && j0 + j < R, pv + (int64_t)t * 2 * R + j0 + j);
                }
                __syncthreads();
                for (int u0 = 0; u0 < rows; u0 += U) {
                    float f[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int64_t t = s_row[u0 + u];
                        f[u] = q[t < 0 ? 0 : t * N];
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        if (s_row[u0 + u] < 0) continue;  // (uniform) no row: whatever was read is not used
#pragma unroll
                        for (int e = 0; e < J; ++e) acc[e] = fmaf(s_p[u0 + u][e], f[u], acc[e]);
                    }
                }
            }
        if (n < N)
#pragma unroll
            for (int e = 0; e < J; ++e)
                if (j0 + e < R) out[(j0 + e) * j_stride] = j0 + e < r ? sc * acc[e] : 0.0f;
    }
}

// dx's tiles, then the adapters' gradients: neither needs the other, and
// together they fill more of the chip (190 rows, 520 and 1384 wide: 17 us,
// and 14 + 10 apart).
template <bool SPLIT>
__global__ void __launch_bounds__(256, 2) k_dx_outer_f32(dx_f32_args d, outer_f32_args o, pair_pools pp, int32_t n_dx) {
    const int64_t wg = grid_index();
    if (wg < n_dx) dx_f32<SPLIT>(d, pp, (int)wg, n_dx);
    else seg_outer_f32(o, pp, wg - n_dx);
}

// bf16, on the matrix cores: out[j][n] = sum_t vt[j][t] q[t][n] over a slot's
// rows, 32 rows a stage.  A workgroup takes 128 columns n, 32 per wavefront,
// and MB blocks of 32 ranks; q's rows (through perm) and both bf16 parts of
// vt's rows are DMA'd into a ring of stages, q read transposed as the base
// GEMM reads W.  One launch holds both gradients: the workgroups of dA (both
// projections' ranks at once, so x is read once) come first, then dB's.  Bound
// by the bytes of x and of dg's and du's parts (2048 rows of 4 slots, 4096 and
// 14336 wide: 43 us, 5.9 TB/s).
constexpr int kOuterCols = 128, kOuterRows = 1024;
struct seg_outer_args {
    const uint16_t *x, *dy, *vt;       // [T][K], [2][2][T][N] (both first parts, both second), see k_rank_finish
    uint16_t *dA[2], *dB[2];
    int32_t T, K, N, R, n_slots, Tp;
    const int32_t *perm, *offsets, *rank[2], *slot_blk;
    int32_t tiles_k, tiles_n;          // column tiles of x and of dy
};

template <int MB, int QP> struct outer_cfg {              // QP: parts of q
    static constexpr int BT = 32, NS = MB > 2 || QP > 1 ? 3 : 4;
    static constexpr int QST = BT * kOuterCols, PST = 32 * MB * BT, STAGE = QP * QST + 2 * PST;
    static constexpr int QI = QST / 8 / 256, PI = 2 * PST / 8 / 256;   // DMA instructions per wave per stage
};

// rank rows [0, nj) at vt + j Tp (and, 2 R Tp on, their second parts), rows p0..p1 of
// perm at places b0.., columns [n0, n0 + 128) of q [T][N] (QP = 2: and of its
// second part, q_lo on; the product of the second parts, 2^-16 of the whole, is
// left out).
template <int MB, int QP>
__device__ __forceinline__ void seg_outer_sum(f32x16_t (&acc)[MB], uint16_t *smem, int32_t *s_row,
                                              const seg_outer_args &g,
                                              const uint16_t *q, int64_t q_lo, int N, int n0, const uint16_t *vt, int nj,
                                              int p0, int p1, int64_t b0) {
    typedef outer_cfg<MB, QP> C;
    constexpr int BT = C::BT, NS = C::NS, QI = C::QI, PI = C::PI, PER = QP * QI + PI;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    auto dma_stage = [&](int kt, int buf) {
        uint16_t *qs = smem + buf * C::STAGE, *ps = qs + QP * C::QST;
#pragma unroll
        for (int j = 0; j < QI; ++j) {
            const int c = (wave * QI + j) * 64 + lane, r = c >> 4, col = n0 + 8 * ((c & 15) ^ swz_w<kOuterCols>(r));
            const int32_t t = s_row[kt * BT + r];
#pragma unroll
            for (int part = 0; part < QP; ++part)
                dma16(t >= 0 && col < N ? (const void *)(q + part * q_lo + (int64_t)t * N + col) : (const void *)g_zero16,
                      qs + part * C::QST + (wave * QI + j) * 64 * 8);
        }
#pragma unroll
        for (int j = 0; j < PI; ++j) {                    // rank rows of 4 chunks: first parts, then second parts
            const int c = (wave * PI + j) * 64 + lane, part = c / (32 * MB * 4), r = c / 4 % (32 * MB);
            const int ch = (c & 3) ^ ((r >> 1) & 3);
            dma16(r < nj ? (const void *)(vt + ((int64_t)part * 2 * g.R + r) * g.Tp + b0 + kt * BT + 8 * ch)
                         : (const void *)g_zero16,
                  ps + (wave * PI + j) * 64 * 8);
        }
    };
    auto wait_stage = [&](int ahead) {
        if (ahead >= 3) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(3 * PER) : "memory");
        else if (ahead == 2) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * PER) : "memory");
        else if (ahead == 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(PER) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    };
    const int fr = lane & 31, fk = lane >> 5, grp = lane >> 4, s16 = lane & 15;
    const int b_kofs = 8 * (grp >> 1) + (s16 >> 2), b_col = 32 * wave + 16 * (grp & 1) + 4 * (s16 & 3);
    // The rows' indices lie in LDS, kOuterRows at a time: a load of them in the
    // loop would wait for every stage in flight.
    for (; p0 < p1; p0 += kOuterRows, b0 += kOuterRows) {
    const int rows = min(p1 - p0, kOuterRows), nk = (rows + BT - 1) / BT;
    __syncthreads();
    for (int i = tid; i < nk * BT; i += 256) s_row[i] = i < rows ? perm_row(g.perm, p0 + i, g.T) : -1;
    __syncthreads();
#pragma unroll
    for (int st = 0; st < NS - 1; ++st)
        if (st < nk) dma_stage(st, st);
    for (int kt = 0; kt < nk; ++kt) {
        wait_stage(min(NS - 2, nk - 1 - kt));
        // and this wave's reads of the stage before, whose buffer is refilled next
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (kt + NS - 1 < nk) dma_stage(kt + NS - 1, (kt + NS - 1) % NS);
        const uint16_t *qs = smem + (kt % NS) * C::STAGE, *ps = qs + QP * C::QST;
#pragma unroll
        for (int ks = 0; ks < BT / 16; ++ks) {
            bf16x8_t bq[QP];
#pragma unroll
            for (int part = 0; part < QP; ++part) {
                short4_t h[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int k = 16 * ks + 4 * i + b_kofs;
                    const uint16_t *at = qs + part * C::QST + k * kOuterCols + 8 * ((b_col >> 3) ^ swz_w<kOuterCols>(k)) +
                                         (b_col & 7);
                    h[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4_t *)(reinterpret_cast<uintptr_t>(at)));
                }
                const short8_t hv = {h[0][0], h[0][1], h[0][2], h[0][3], h[1][0], h[1][1], h[1][2], h[1][3]};
                bq[part] = __builtin_bit_cast(bf16x8_t, hv);
            }
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    const int r = mb * 32 + fr, ch = (2 * ks + fk) ^ ((r >> 1) & 3);
                    const bf16x8_t a = *reinterpret_cast<const bf16x8_t *>(ps + part * C::PST + r * BT + 8 * ch);
                    acc[mb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, bq[0], acc[mb], 0, 0, 0);
                    if constexpr (QP > 1)
                        if (part == 0) acc[mb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, bq[QP - 1], acc[mb], 0, 0, 0);
                }
        }
    }
    }
}

template <int MBA, int MBB> __global__ void __launch_bounds__(256) k_seg_outer_mfma(seg_outer_args g) {
    constexpr int LA = outer_cfg<MBA, 1>::NS * outer_cfg<MBA, 1>::STAGE;
    constexpr int LB = outer_cfg<MBB, 2>::NS * outer_cfg<MBB, 2>::STAGE;
    __shared__ __attribute__((aligned(1024))) uint16_t smem[LA > LB ? LA : LB];
    __shared__ int32_t s_row[kOuterRows];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t wg = grid_index(), n_a = (int64_t)g.n_slots * g.tiles_k;
    const bool is_a = wg < n_a;
    int item = (int)(is_a ? wg : wg - n_a);
    const int tiles = is_a ? g.tiles_k : 2 * g.tiles_n;
    const int slot = item / tiles;
    if (slot >= g.n_slots) return;
    item -= slot * tiles;
    const int m = !is_a && item >= g.tiles_n, tile = item - m * g.tiles_n;
    const int n0 = tile * kOuterCols, N = is_a ? g.K : g.N;
    const int p0 = max(g.offsets[slot + 1], 0), p1 = min(g.offsets[slot + 2], g.T);
    const int64_t b0 = p1 > p0 ? (int64_t)g.slot_blk[slot] * kShrinkRows : 0;
    const int col = n0 + 32 * wave + (lane & 31), j4 = 4 * (lane >> 5);
    // ranks past the slot's get zeros whatever the rows hold
    const int R = g.R, rk[2] = {min(g.rank[0][slot], R), min(g.rank[1][slot], R)};
    if (is_a) {
        f32x16_t acc[MBA];
#pragma unroll
        for (int mb = 0; mb < MBA; ++mb)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[mb][e] = 0.0f;
        seg_outer_sum<MBA, 1>(acc, smem, s_row, g, g.x, 0, N, n0, g.vt + (int64_t)2 * 2 * R * g.Tp, 2 * R, p0, p1, b0);
        if (col >= N) return;
        // [slot][k][j]: a lane's accumulators hold groups of 4 neighbouring ranks of its k
#pragma unroll
        for (int mb = 0; mb < MBA; ++mb)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int j = mb * 32 + 8 * q + j4;
                if (j >= 2 * R) continue;
                const int jj = j < R ? j : j - R, r = j < R ? rk[0] : rk[1];
                uint16_t *out = (j < R ? g.dA[0] : g.dA[1]) + ((int64_t)slot * N + col) * R + jj;
                float f[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = jj + e < r ? acc[mb][4 * q + e] : 0.0f;
                *reinterpret_cast<uint2 *>(out) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
            }
    } else {
        f32x16_t acc[MBB];
#pragma unroll
        for (int mb = 0; mb < MBB; ++mb)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[mb][e] = 0.0f;
        seg_outer_sum<MBB, 2>(acc, smem, s_row, g, g.dy + (int64_t)m * g.T * N, 2ll * g.T * N, N, n0,
                              g.vt + (int64_t)m * R * g.Tp, R, p0, p1, b0);
        if (col >= N) return;
        uint16_t *out = (m ? g.dB[1] : g.dB[0]) + (int64_t)slot * R * N + col;
#pragma unroll
        for (int mb = 0; mb < MBB; ++mb)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int j = mb * 32 + 8 * (e >> 2) + j4 + (e & 3);
                if (j < R) out[(int64_t)j * N] = j < rk[m] ? (uint16_t)f32_to_bf16_bits(acc[mb][e]) : (uint16_t)0;
            }
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
    B.dy = o;      o = align256(o + (dtype == LORA_BF16 ? 4 : 2) * t * (size_t)d_out * eb);
    B.dv = o;      o = align256(o + 4 * t * 2 * (size_t)R);
    // transposed bf16 parts of s v and dv, every segment from a work block on
    B.vt = o;      o = align256(o + (dtype == LORA_BF16 ? 16 * (size_t)R * 32 * ((t + 31) / 32 + segs) : 0));
    B.oct = o;     o = align256(o + (dtype == LORA_BF16 ? segs * 2 * (size_t)R * (size_t)d_in * 2 : 0));
    B.row0 = o;    o = align256(o + 4 * (size_t)n_slots);
    B.slot_blk = o; o = align256(o + 4 * (size_t)n_slots);
    B.rank = o;    o = align256(o + 4 * (size_t)n_slots);
    B.scale = o;   o = align256(o + 4 * (size_t)n_slots);
    B.partial = o;
    const size_t tp = (t + 255) / 256 * 256, np = ((size_t)d_in + 255) / 256 * 256;
    const size_t need = T > 0 ? 4 * (size_t)kMaxGemmSplit * tp * np : 0;
    B.total = align256(o + (need < kGemmPartialCap ? need : kGemmPartialCap));
    return B;
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
    // k_rank_finish has its workgroups in one grid dimension, which holds fewer than 2^32 threads
    const int64_t finish = 2 * ceil_div(T, kShrinkRows) + (S < T ? S : T) * (1ll + (c.dx ? ceil_div(K, 256) : 0));
    if (DT == LORA_BF16 && finish * 256 >= 1ll << 32) return LORA_ERR_UNSUPPORTED;
    lora_status_t st = launch_segments(c.ids, T, S, L, ws, s, 1);
    if (st != LORA_OK) return st;
    const int32_t *perm = ws_ptr<int32_t>(ws, L.perm), *offsets = ws_ptr<int32_t>(ws, L.offsets);
    float *v = ws_ptr<float>(ws, L.v), *dv = ws_ptr<float>(ws, B.dv);
    E *dg = ws_ptr<E>(ws, B.dy), *du = dg + (int64_t)T * F;
    const pair_pools pp = make_pair_pools(p);
    const int64_t n_vec = (int64_t)T * F / vec16<DT>::n;
    hipLaunchKernelGGL(k_gated_dact<DT>, dim3((uint32_t)(n_vec < (1 << 24) ? (n_vec + 255) / 256 : 1 << 16)),
                       dim3(256), 0, s, (const E *)c.gate, (const E *)c.up, (const E *)c.dh, dg, du, 2ll * T * F, n_vec,
                       c.act);
    // v = x A (also records the bad ids); dv
    st = DT == LORA_F32 ? launch_shrink_pair(c.x, T, p, c.ids, v, ws_ptr<int32_t>(ws, L.header), s)
                        : launch_shrink(c.x, T, p, 2, c.ids, true, v, L, ws, s);
    if (st != LORA_OK) return st;
    const int32_t row_blocks = ceil_div(T, kShrinkRows), n_work = row_blocks + (S < T ? S : T), Tp = n_work * 32;
    uint16_t *vt = ws_ptr<uint16_t>(ws, B.vt);
    int32_t *slot_blk = ws_ptr<int32_t>(ws, B.slot_blk);
    if constexpr (DT == LORA_F32) {
        hipLaunchKernelGGL(k_rank_grad_rows<DT>, grid_of(2ll * T), dim3(256), 0, s, dg, (int64_t)T * F, T, F, pp, S, R,
                           c.ids, dv);
    } else {
        // about 1024 workgroups with work, of at least 512 columns
        int split = ceil_div(512, row_blocks + 1);
        if (split > kMaxKSplit) split = kMaxKSplit;
        if (split > F / 512) split = F / 512;
        if (split < 1) split = 1;
        const int n_chunk = ceil_div(ceil_div(F, split), 128) * 128;
        split = ceil_div(F, n_chunk);
        float *part = ws_ptr<float>(ws, L.partial);
        rank_grad_args g{(const uint16_t *)dg, T, F, R, S, n_chunk, perm, ws_ptr<int32_t>(ws, L.seg_id),
                         ws_ptr<int32_t>(ws, L.seg_start), ws_ptr<int32_t>(ws, L.n_seg),
                         ws_ptr<int32_t>(ws, L.blk_start), ws_ptr<int32_t>(ws, L.blk_seg), part};
        const dim3 grid(n_work, split, 2);
        switch ((R + 15) / 16) {
            case 1: hipLaunchKernelGGL(k_rank_grad<1>, grid, dim3(256), 0, s, g, pp); break;
            case 2: hipLaunchKernelGGL(k_rank_grad<2>, grid, dim3(256), 0, s, g, pp); break;
            case 3: hipLaunchKernelGGL(k_rank_grad<3>, grid, dim3(256), 0, s, g, pp); break;
            default: hipLaunchKernelGGL(k_rank_grad<4>, grid, dim3(256), 0, s, g, pp); break;
        }
        const int first_octet = n_work + row_blocks;
        const rank_finish_args f{v, part, split, T, R, S, n_work, Tp, perm, offsets, g.seg_id, g.seg_start, g.n_seg,
                                 g.blk_start, g.blk_seg, dv, vt, slot_blk, first_octet};
        const a_octets_args oc{g.seg_id, g.n_seg, S, K, R, ceil_div(K, 256), ws_ptr<uint16_t>(ws, B.oct),
                               ws_ptr<int32_t>(ws, B.row0), ws_ptr<int32_t>(ws, B.rank), ws_ptr<float>(ws, B.scale)};
        const int octets = c.dx ? (S < T ? S : T) * oc.k_blocks : 0;
        hipLaunchKernelGGL(k_rank_finish, dim3(first_octet + octets, 2 * R / 8), dim3(256), 0, s, f, oc, pp);
    }
    if constexpr (DT == LORA_F32) {
        dx_f32_args g{(const float *)dg, (const float *)du, (const float *)c.W[0], (const float *)c.W[1],
                      (float *)c.dx, dv, c.ids, perm, ws_ptr<float>(ws, B.partial), T, F, K, S, R, ceil_div(K, 64), 1, 0};
        const outer_f32_args o{(const float *)c.x, (const float *)dg, (const float *)du, v, dv,
                               (float *)c.dA[0], (float *)c.dA[1], (float *)c.dB[0], (float *)c.dB[1],
                               offsets, perm, T, K, F, R, c.dA[0] ? S : 0, ceil_div(K, 256), ceil_div(F, 256)};
        const int tiles = c.dx ? ceil_div(T, 64) * g.n_tiles_n : 0;
        if (c.dx) g.splits = f32_splits(tiles, 2 * ceil_div(F, 32) * 32, 64 * 64, c.ws_bytes - B.partial, g.k_chunk);
        const int n_dx = tiles * g.splits;
        const dim3 grid = grid_of(n_dx + 2ll * o.n_slots * (o.tiles_k + o.tiles_f));
        if (c.dx || c.dA[0]) {
            if (g.splits == 1) hipLaunchKernelGGL(k_dx_outer_f32<false>, grid, dim3(256), 0, s, g, o, pp, n_dx);
            else hipLaunchKernelGGL(k_dx_outer_f32<true>, grid, dim3(256), 0, s, g, o, pp, n_dx);
        }
        if (g.splits > 1) hipLaunchKernelGGL(k_dx_reduce_f32, dim3(tiles * 4), dim3(256), 0, s, g, pp);
    } else if (c.dx) {
        uint16_t *oct = ws_ptr<uint16_t>(ws, B.oct);
        int32_t *row0 = ws_ptr<int32_t>(ws, B.row0), *rank = ws_ptr<int32_t>(ws, B.rank);
        float *scale = ws_ptr<float>(ws, B.scale);
        nt_args nt{{(const uint16_t *)dg, (const uint16_t *)du}, {(const uint16_t *)c.W[0], (const uint16_t *)c.W[1]},
                   F, ceil_div(F, 64) * 64, ws_ptr<int32_t>(ws, L.n_seg)};
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
        const gemm_plan pl = plan_dx(T, g.K, g.N, c.ws_bytes - B.partial);
        g.n_tiles_m = ceil_div(T, pl.bm);
        g.n_tiles_n = ceil_div(g.N, pl.bn);
        g.col_strips = col_strips_pay(T, g.N, g.n_tiles_n);
        if (pl.bm == 256 && pl.bn == 256) launch_nt_cfg<256, 256, 2, 8, 2, 2, 8>(g, nt, pl, s);
        else if (pl.bm == 256 && pl.bn == 128) launch_nt_cfg<256, 128, 2, 8, 2, 2, 8>(g, nt, pl, s);
        else if (pl.bn == 128) launch_nt_cfg<128, 128, 2, 4, 2, 4, 8>(g, nt, pl, s);
        else launch_nt_cfg<128, 64, 2, 4, 2, 2, 4>(g, nt, pl, s);
    }
    if (c.dA[0] && DT == LORA_BF16) {
        seg_outer_args g{(const uint16_t *)c.x, (const uint16_t *)dg, vt,
                         {(uint16_t *)c.dA[0], (uint16_t *)c.dA[1]}, {(uint16_t *)c.dB[0], (uint16_t *)c.dB[1]},
                         T, K, F, R, S, Tp, perm, offsets, {p[0].rank, p[1].rank}, slot_blk, ceil_div(K, kOuterCols), ceil_div(F, kOuterCols)};
        const dim3 grid = grid_of((int64_t)S * (g.tiles_k + 2 * g.tiles_n));
        switch ((R + 15) / 16) {
            case 1: hipLaunchKernelGGL((k_seg_outer_mfma<1, 1>), grid, dim3(256), 0, s, g); break;
            case 2: hipLaunchKernelGGL((k_seg_outer_mfma<2, 1>), grid, dim3(256), 0, s, g); break;
            case 3: hipLaunchKernelGGL((k_seg_outer_mfma<3, 2>), grid, dim3(256), 0, s, g); break;
            default: hipLaunchKernelGGL((k_seg_outer_mfma<4, 2>), grid, dim3(256), 0, s, g); break;
        }
    }
    return hip_status(hipGetLastError());
}

lora_status_t launch_gated_backward(const gated_bwd_call &c, const bwd_layout &B, hipStream_t s) {
    return c.pools[0].dtype == LORA_F32 ? backward<LORA_F32>(c, B, s) : backward<LORA_BF16>(c, B, s);
}

}  // namespace lora
