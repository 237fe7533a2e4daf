// The linear layer with bias, activation and residual in fp32:
//   y = act(x W + bias + s_a (x A_a) B_a) + residual      per row, a = ids[t]
// (the bf16 and FP8 forms are instantiations of their base GEMMs).
//
// 32 rows x 128 columns per workgroup of 8 wavefronts on v_mfma_f32_32x32x2_f32, K
// in steps of 32 DMA'd into a ring of three stages; two wavefronts share 32 columns
// and take half of each step's k, so that a SIMD has two to choose from where a CU
// has one workgroup only, and a wavefront reads the next step's values from LDS
// while it multiplies.  The rows' low-rank terms are made before the first step,
// while the stages load.  Grids of few tiles split K; the sums go through LDS or
// the partial buffer to threads that own 4 columns of a row.
//
// 333 x 1032 x 2744, 5 adapters: 40 us (and 6 us for x A), of which 27 us are the
// steps (the same products without their loads 21 us) and the rest is what a launch
// of one workgroup a CU has before its first and after its last step.  4 wavefronts
// and no split 49 us, 4 split in two 30 us and 7 for the sums' launch.
#include "act_common.hpp"
#include "fp8_common.hpp"

namespace lora {

struct linear_f32_args {
    const float *x, *W, *b, *scale, *bias, *residual;
    const int32_t *rank, *row0, *ids, *perm;
    float *y, *pre;
    const float *v;
    float *partial;                    // [tile][split][32][128]
    int32_t T, K, N, n_slots, max_rank, v_stride, act, n_tiles_m, n_tiles_n, splits, k_chunk;
};

__device__ __forceinline__ row_term load_row_term(const linear_f32_args &g, int64_t t) {
    const int32_t id = t >= 0 ? g.ids[t] : -1;
    if (id < 0 || id >= g.n_slots) return row_term{0, 0, 0.0f};
    return row_term{min(g.rank[id], g.max_rank), (int32_t)slot_row0(g.row0, id, g.max_rank), g.scale[id]};
}

// The low-rank sums of the columns n = n0 + 32 q of NR rows (32 lanes share a row
// and read neighbouring columns); an octet's loads of all rows are in flight together.
template <int NR>
__device__ __forceinline__ void row_terms(const linear_f32_args &g, const row_term (&rt)[NR], const int64_t (&t)[NR],
                                          int n0, float (&d)[NR][4]) {
    int most = 0;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        most = max(most, rt[r].rank);
#pragma unroll
        for (int q = 0; q < 4; ++q) d[r][q] = 0.0f;
    }
    for (int j = 0; j < most; j += 8) {
        f32x4_t vv[NR][2], bb[NR][4][2];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const bool in = j < rt[r].rank;
            const float *b = g.b + ((int64_t)rt[r].row0 + j) * g.N + (int64_t)n0 * 8, *v = g.v + t[r] * g.v_stride + j;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                vv[r][h] = load4(in, v + 4 * h);
#pragma unroll
                for (int q = 0; q < 4; ++q) bb[r][q][h] = load4(in && n0 + 32 * q < g.N, b + 32 * q * 8 + 4 * h);
            }
        }
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 8; ++e) d[r][q] = fmaf(vv[r][e >> 2][e & 3], bb[r][q][e >> 2][e & 3], d[r][q]);
    }
}

// The epilogue of 4 neighbouring columns.
__device__ __forceinline__ void epilogue4(const linear_f32_args &g, int64_t t, int n, f32x4_t o) {
    const int64_t at = t * g.N + n;
    if (g.bias) {
        const f32x4_t b = *reinterpret_cast<const f32x4_t *>(g.bias + n);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += b[e];
    }
    if (g.pre) *reinterpret_cast<f32x4_t *>(g.pre + at) = o;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = act_or_none<true>(g.act, o[e]);
    if (g.residual) {
        const f32x4_t r = *reinterpret_cast<const f32x4_t *>(g.residual + at);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += r[e];
    }
    *reinterpret_cast<f32x4_t *>(g.y + at) = o;
}

// Until at most `ahead` (0 or 1) stages of PER loads are in flight.
template <int PER> __device__ __forceinline__ void wait_loads(int ahead) {
    if (ahead >= 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(PER) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <bool SPLIT> __global__ void __launch_bounds__(512) k_linear_f32(linear_f32_args g) {
    constexpr int BK = 32, NS = 3, XST = 32 * BK, STAGE = XST + BK * 128, WS = 128 + 4;
    __shared__ __attribute__((aligned(1024))) float smem[NS * STAGE];     // stages: x [32][BK], W [BK][128]; sums: [32][WS]
    static_assert(32 * WS <= NS * STAGE, "the sums fit the stages' LDS");
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, wc = w & 3, kh = w >> 2;
    int tm, tn, split;
    const int total = g.n_tiles_m * g.n_tiles_n * (SPLIT ? g.splits : 1);
    if (grid_index() >= total) return;
    f32_tile((int)grid_index(), total, g.n_tiles_m, SPLIT ? g.splits : 1, tm, tn, split);
    const int tile = tm * g.n_tiles_n + tn, m0 = tm * 32, n0 = tn * 128;
    const int N = g.N, T = g.T, k_begin = split * g.k_chunk, k_end = min(g.K, k_begin + g.k_chunk);
    // DMA, 16-byte chunks, two or three instructions a wavefront and stage.  W: chunk 512 j
    // + tid -> row k = 16 j + tid / 32, place tid % 32, which holds the columns' chunk
    // place, ^ 8 in every other 8 rows (the two half-wavefronts, 8 k apart, then read
    // different banks).  x: wavefronts 0 to 3, chunk tid -> row tid / 8, place tid %
    // 8, which holds the row's chunk place ^ swz_x(row).
    const int xr = (tid & 255) >> 3, xk = 4 * ((tid & 7) ^ swz_x<64>(xr));
    const int32_t t_x = m0 + xr < T ? perm_row(g.perm, m0 + xr, T) : -1;
    const float *xp = g.x + (int64_t)(t_x < 0 ? 0 : t_x) * g.K + xk;
    const int wr = tid >> 5, wcol = n0 + 4 * ((tid & 31) ^ (wr & 8));
    const bool wok = wcol < N;
    const float *wp = g.W + (int64_t)wr * N + (wok ? wcol : 0);
    auto dma_stage = [&](int kt, int buf) {
        float *xs = smem + buf * STAGE, *wsm = xs + XST;
        const int k0 = k_begin + kt * BK;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            dma16(wok && k0 + 16 * j + wr < k_end ? (const void *)(wp + (int64_t)(k0 + 16 * j) * N) : (const void *)g_zero16,
                  wsm + (512 * j + w * 64) * 4);
        if (w < 4) dma16(t_x >= 0 && k0 + xk < k_end ? (const void *)(xp + k0) : (const void *)g_zero16, xs + w * 64 * 4);
    };
    // product i of a step takes k = 16 kh + i from the lower half-wavefront and 8
    // more from the upper: a lane's 8 values of x are neighbours
    auto load_frags = [&](int buf, float (&a)[8], float (&b)[8]) {
        const float *xs = smem + buf * STAGE + (lane & 31) * BK, *wsm = smem + buf * STAGE + XST;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<f32x4_t *>(a + 4 * i) =
                *reinterpret_cast<const f32x4_t *>(xs + 4 * ((4 * kh + 2 * (lane >> 5) + i) ^ swz_x<64>(lane & 31)));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            b[i] = wsm[(16 * kh + 8 * (lane >> 5) + i) * 128 + ((32 * wc + (lane & 31)) ^ (lane & 32))];
    };
    f32x16_t acc;
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
    auto products = [&](const float (&a)[8], const float (&b)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], acc, 0, 0, 0);
    };
    const int nk = (k_end - k_begin + BK - 1) / BK;
    // later stages still in flight; a wavefront without x's instruction has two a stage
    auto wait_stage = [&](int ahead) {
        if (w < 4) wait_loads<3>(ahead);
        else wait_loads<2>(ahead);
    };
#pragma unroll
    for (int st = 0; st < NS; ++st)
        if (st < nk) dma_stage(st, st);
    // a thread's two rows of the tile, columns (tid & 31) + 32 q: their low-rank terms
    constexpr int NR = SPLIT ? 1 : 2;
    float d[NR][4];
    float sc[NR];
    if constexpr (!SPLIT) {
        row_term rt[NR];
        int64_t tr[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int p = m0 + (tid >> 5) + 16 * r;
            tr[r] = p < T ? perm_row(g.perm, p, T) : -1;
            rt[r] = load_row_term(g, tr[r]);
            sc[r] = rt[r].scale;
        }
        row_terms<NR>(g, rt, tr, n0 + (tid & 31), d);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    float a0[8], b0[8], a1[8], b1[8];
    load_frags(0, a0, b0);
    // The next stage is there for all and every wavefront has read this one, whose
    // place is filled anew; after the last step the next stage's values are read
    // and not used.
    auto step = [&](int kt, const float (&a)[8], const float (&b)[8], float (&an)[8], float (&bn)[8]) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        wait_stage(min(NS - 2, nk - 2 - kt));
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (kt + NS < nk) dma_stage(kt + NS, kt % NS);
        load_frags((kt + 1) % NS, an, bn);
        products(a, b);
        __builtin_amdgcn_sched_barrier(0);
    };
    for (int kt = 0; kt < nk; kt += 2) {
        step(kt, a0, b0, a1, b1);
        if (kt + 1 < nk) step(kt + 1, a1, b1, a0, b0);
    }
    __syncthreads();
    // the two halves' sums, the second half's wavefronts first
    auto place = [&](int e) {
        return (8 * (e >> 2) + 4 * (lane >> 5) + (e & 3)) * WS + wc * 32 + (lane & 31);
    };
    if (kh)
#pragma unroll
        for (int e = 0; e < 16; ++e) smem[place(e)] = acc[e];
    __syncthreads();
    if (!kh)
#pragma unroll
        for (int e = 0; e < 16; ++e) smem[place(e)] += acc[e];
    __syncthreads();
    if constexpr (SPLIT) {
        float *part = g.partial + ((int64_t)tile * g.splits + split) * 32 * 128;
        for (int i = tid; i < 32 * 32; i += 512)
            *reinterpret_cast<f32x4_t *>(part + 4 * i) =
                *reinterpret_cast<const f32x4_t *>(smem + (i >> 5) * WS + (i & 31) * 4);
    } else {
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float *at = smem + ((tid >> 5) + 16 * r) * WS + (tid & 31) + 32 * q;
                *at = fmaf(sc[r], d[r][q], *at);
            }
        __syncthreads();
        for (int i = tid; i < 32 * 32; i += 512) {
            const int r = i >> 5, c = (i & 31) * 4, n = n0 + c;
            const int64_t t = m0 + r < T ? perm_row(g.perm, m0 + r, T) : -1;
            if (t < 0 || n >= N) continue;
            epilogue4(g, t, n, *reinterpret_cast<const f32x4_t *>(smem + r * WS + c));
        }
    }
}

// The pieces' sums, in split order: 8 rows of one tile per workgroup.
__global__ void __launch_bounds__(256) k_linear_reduce_f32(linear_f32_args g) {
    const int tile = blockIdx.x >> 2, lr = threadIdx.x >> 5, r = (blockIdx.x & 3) * 8 + lr, c = (threadIdx.x & 31) * 4;
    const int p = tile / g.n_tiles_n * 32 + r, n0 = tile % g.n_tiles_n * 128, n = n0 + c;
    const int64_t t[1] = {p < g.T ? perm_row(g.perm, p, g.T) : -1};
    const row_term rt[1] = {load_row_term(g, t[0])};
    __shared__ float s_d[8][128];                         // the rows' low-rank sums
    float d[1][4];
    row_terms<1>(g, rt, t, n0 + (threadIdx.x & 31), d);
#pragma unroll
    for (int q = 0; q < 4; ++q) s_d[lr][(threadIdx.x & 31) + 32 * q] = d[0][q];
    __syncthreads();
    if (t[0] < 0 || n >= g.N) return;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
    const float *part = g.partial + (int64_t)tile * g.splits * 32 * 128 + r * 128 + c;
    for (int s = 0; s < g.splits; ++s, part += 32 * 128) {
        const f32x4_t f = *reinterpret_cast<const f32x4_t *>(part);
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] += f[q];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = fmaf(rt[0].scale, s_d[lr][c + q], o[q]);
    epilogue4(g, t[0], n, o);
}

// K ranges per tile, of at least 128 terms: the count whose time is least by this
// estimate -- rounds of 256 workgroups at 0.5 TFLOP/s each, 3 us a round beside
// them, and for split tiles the second launch and the partial sums written and read
// at 4 TB/s.
static int linear_f32_splits(int tiles, int K, size_t partial_bytes, int &k_chunk) {
    int best = 1;
    double best_us = 1e30;
    for (int s = 1; s <= kMaxGemmSplit && (s == 1 || s * 128 <= K); ++s) {
        const double sums = (double)s * tiles * 32 * 128 * 4;
        if (s > 1 && sums > (double)partial_bytes) break;
        const double us = ceil_div((int64_t)tiles * s, 256) * (2.0 * 32 * 128 * K / s / 0.5e6 + 3) +
                          (s > 1 ? 5 + 2 * sums / 4e6 : 0);
        if (us < best_us) {
            best = s;
            best_us = us;
        }
    }
    k_chunk = ceil_div(ceil_div(K, best), 32) * 32;
    return ceil_div(K, k_chunk);
}

// ---------------------------------------------------------------------------
// The bf16 layer of up to 64 rows, bound by the bytes of W: W goes from memory to
// the matrix cores without LDS.  A wavefront takes 128 columns and 32 k at a time:
// a lane reads 8 neighbouring columns of each of 8 rows of W (16 bytes each) and
// exchanges rows for columns in its registers (32 byte permutes for 128 bytes),
// which gives the B operands of 8 products whose columns are 8 apart; x's rows are
// the A operand as they lie.  The WV wavefronts of a workgroup share its K range,
// step by step, and add their sums through LDS; the K ranges' sums go to the
// partial buffer, and k_few_finish finishes them.  The first workgroups compute
// the rank vectors v = x A meanwhile, which only that second launch reads.
//
// One row, 14336 x 4096 (117 MB of W): 21 us, 5.6 TB/s, and 4 us for the second
// launch; a call 29 us.  4096 x 14336: 1 row 29 us, 64 rows 44; through LDS, by the
// tiles of the base GEMM, 70 and 80.
// ---------------------------------------------------------------------------
template <int MT, int WV>
__global__ void __launch_bounds__(WV * 64, WV == 4 ? 2 : 1) k_linear_few(gemm_args g, int32_t n_shrink) {
    constexpr int SLD = 128 + 4, BM = 16 * MT;
    __shared__ __attribute__((aligned(16))) float s_sum[WV / 2][BM][SLD];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, p = lane & 15, kg = lane >> 4;
    if ((int)blockIdx.x < n_shrink) {
        shrink_row<LORA_BF16, WV>(g.x, g.T, g.K, g.a, g.rank, g.row0, g.n_slots, g.max_rank, g.ids, g.vpart, g.err,
                                  blockIdx.x);
        return;
    }
    // neighbouring workgroups take neighbouring columns of one K range
    const int wg = (int)blockIdx.x - n_shrink, tn = wg % g.n_tiles_n, split = wg / g.n_tiles_n;
    const int N = g.N, K = g.K, T = g.T, n = tn * 128 + 8 * p;
    const int k_begin = split * g.k_chunk, k_end = min(K, k_begin + g.k_chunk);
    const uint16_t *wp = g.W + n;
    const bool n_ok = n < N;
    f32x4_t acc[MT][8];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int s = 0; s < 8; ++s) acc[m][s] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    uint4 wq[2][8], xq[2][MT];
    // K is a multiple of 8, so a lane's 8 rows are all in the range or none is
    auto load = [&](int k0, uint4 (&wr)[8], uint4 (&xr)[MT]) {
        const int k = k0 + 8 * kg;
        const bool in = k < k_end;
#pragma unroll
        for (int h = 0; h < 8; ++h) wr[h] = in && n_ok ? ldg16(wp + (int64_t)(k + h) * N) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int t = 16 * m + p;
            xr[m] = in && t < T ? ldg16(g.x + (int64_t)t * K + k) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    auto products = [&](const uint4 (&wr)[8], const uint4 (&xr)[MT]) {
        uint32_t r[8][4];
#pragma unroll
        for (int h = 0; h < 8; ++h) {
            r[h][0] = wr[h].x; r[h][1] = wr[h].y; r[h][2] = wr[h].z; r[h][3] = wr[h].w;
        }
#pragma unroll
        for (int s = 0; s < 8; ++s) {                     // column s of a lane's 8: its values of the 8 rows
            uint32_t o[4];
#pragma unroll
            for (int h = 0; h < 4; ++h)
                o[h] = __builtin_amdgcn_perm(r[2 * h + 1][s >> 1], r[2 * h][s >> 1], (s & 1) ? 0x07060302u : 0x05040100u);
            const bf16x8_t b = __builtin_bit_cast(bf16x8_t, make_uint4(o[0], o[1], o[2], o[3]));
#pragma unroll
            for (int m = 0; m < MT; ++m)
                acc[m][s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, xr[m]), b, acc[m][s], 0, 0, 0);
        }
    };
    constexpr int STRIDE = 32 * WV;
    int k0 = k_begin + 32 * w;
    load(k0, wq[0], xq[0]);
    for (; k0 < k_end; k0 += 2 * STRIDE) {
        load(k0 + STRIDE, wq[1], xq[1]);
        products(wq[0], xq[0]);
        load(k0 + 2 * STRIDE, wq[0], xq[0]);
        products(wq[1], xq[1]);
    }
    // the upper half of the wavefronts hands its sums to the lower, and so on
#pragma unroll
    for (int half = WV / 2; half >= 1; half /= 2) {
        if (w >= half && w < 2 * half)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float *at = &s_sum[w - half][16 * m + 4 * kg + e][8 * p];
                    *reinterpret_cast<f32x4_t *>(at) = f32x4_t{acc[m][0][e], acc[m][1][e], acc[m][2][e], acc[m][3][e]};
                    *reinterpret_cast<f32x4_t *>(at + 4) = f32x4_t{acc[m][4][e], acc[m][5][e], acc[m][6][e], acc[m][7][e]};
                }
        __syncthreads();
        if (w < half)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float *at = &s_sum[w][16 * m + 4 * kg + e][8 * p];
#pragma unroll
                    for (int s = 0; s < 8; ++s) acc[m][s][e] += at[s];
                }
        if (half > 1) __syncthreads();
    }
    if (w > 0) return;
    float *part = g.partial + ((int64_t)tn * g.splits + split) * BM * 128 + 8 * p;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 16 * m + 4 * kg + e;
            if (r >= T) continue;
            float *at = part + r * 128;
            *reinterpret_cast<f32x4_t *>(at) = f32x4_t{acc[m][0][e], acc[m][1][e], acc[m][2][e], acc[m][3][e]};
            *reinterpret_cast<f32x4_t *>(at + 4) = f32x4_t{acc[m][4][e], acc[m][5][e], acc[m][6][e], acc[m][7][e]};
        }
}

// The same on an FP8 base weight: 64 columns and 128 codes of k a wavefront and step;
// rows of wq and of xq lie along k, so a lane reads 32 codes of each of 4 columns and of
// each 16 rows as v_mfma_scale_f32_16x16x128_f8f6f4 takes them (lane l: A row and B
// column l % 16, k = 32 (l / 16) + 0..31, and their E8M0 scales).  4096 x 14336: 1
// row 19 us (35 by tiles), 16 rows 24, 32 rows 30.
typedef int few_i32x8_t __attribute__((ext_vector_type(8)));

template <int MT, int WV>
__global__ void __launch_bounds__(WV * 64) k_linear_few_fp8(gemm_args g, int32_t n_shrink) {
    constexpr int SLD = 64 + 4, BM = 16 * MT, CB = 4;
    __shared__ __attribute__((aligned(16))) float s_sum[WV / 2][BM][SLD];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, p = lane & 15, kg = lane >> 4;
    if ((int)blockIdx.x < n_shrink) {
        shrink_row<LORA_BF16, WV>(g.x, g.T, g.K, g.a, g.rank, g.row0, g.n_slots, g.max_rank, g.ids, g.vpart, g.err,
                                  blockIdx.x);
        return;
    }
    const int strips = 2 * g.n_tiles_n, wg = (int)blockIdx.x - n_shrink, strip = wg % strips, split = wg / strips;
    const int N = g.N, K = g.K, T = g.T, n0 = strip * 64;
    const int k_begin = split * g.k_chunk, k_end = min(K, k_begin + g.k_chunk);
    int esa[MT], esb[CB];
#pragma unroll
    for (int m = 0; m < MT; ++m) esa[m] = 16 * m + p < T ? e8m0_of(g.xs[16 * m + p]) : 127;
#pragma unroll
    for (int c = 0; c < CB; ++c) esb[c] = n0 + 16 * c + p < N ? e8m0_of(g.wsc[n0 + 16 * c + p]) : 127;
    f32x4_t acc[MT][CB];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < CB; ++c) acc[m][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    uint4 wq[2][CB][2], xq[2][MT][2];
    auto load = [&](int k0, uint4 (&wr)[CB][2], uint4 (&xr)[MT][2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = k0 + 32 * kg + 16 * h;          // K is a multiple of 16
#pragma unroll
            for (int c = 0; c < CB; ++c) {
                const int n = n0 + 16 * c + p;
                wr[c][h] = k < k_end && n < N ? ldg16(g.wq + (int64_t)n * K + k) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int t = 16 * m + p;
                xr[m][h] = k < k_end && t < T ? ldg16(g.xq + (int64_t)t * K + k) : make_uint4(0u, 0u, 0u, 0u);
            }
        }
    };
    auto operand = [](const uint4 (&q)[2]) {
        few_i32x8_t v;
        v[0] = (int)q[0].x; v[1] = (int)q[0].y; v[2] = (int)q[0].z; v[3] = (int)q[0].w;
        v[4] = (int)q[1].x; v[5] = (int)q[1].y; v[6] = (int)q[1].z; v[7] = (int)q[1].w;
        return v;
    };
    auto products = [&](const uint4 (&wr)[CB][2], const uint4 (&xr)[MT][2]) {
#pragma unroll
        for (int c = 0; c < CB; ++c)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                acc[m][c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(xr[m]), operand(wr[c]), acc[m][c], 0, 0,
                                                                             0, esa[m], 0, esb[c]);
    };
    constexpr int STRIDE = 128 * WV;
    int k0 = k_begin + 128 * w;
    load(k0, wq[0], xq[0]);
    for (; k0 < k_end; k0 += 2 * STRIDE) {
        load(k0 + STRIDE, wq[1], xq[1]);
        products(wq[0], xq[0]);
        load(k0 + 2 * STRIDE, wq[0], xq[0]);
        products(wq[1], xq[1]);
    }
#pragma unroll
    for (int half = WV / 2; half >= 1; half /= 2) {       // as in k_linear_few
        if (w >= half && w < 2 * half)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int c = 0; c < CB; ++c) s_sum[w - half][16 * m + 4 * kg + e][16 * c + p] = acc[m][c][e];
        __syncthreads();
        if (w < half)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int c = 0; c < CB; ++c) acc[m][c][e] += s_sum[w][16 * m + 4 * kg + e][16 * c + p];
        if (half > 1) __syncthreads();
    }
    if (w > 0) return;
    float *part = g.partial + ((int64_t)(strip >> 1) * g.splits + split) * BM * 128 + 64 * (strip & 1) + p;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 16 * m + 4 * kg + e;
            if (r >= T) continue;
#pragma unroll
            for (int c = 0; c < CB; ++c) part[r * 128 + 16 * c] = acc[m][c][e];
        }
}

// The K ranges' sums in their order, the row's low-rank term and the epilogue.  All of
// it is latency, so a thread has 4 neighbouring columns of a row only, and asks for
// everything as soon as its address is known: the partial sums, bias and residual with
// the row's id, then the slot's first two octets of B and of v with its rank (a padded
// slot has all its max_rank rows, a packed one at least 8).  16 x 4096, 8 ranges:
// with 8 columns a thread and 4 ranges ahead 7.0 us.
__global__ void __launch_bounds__(256) k_few_finish(gemm_args g, int32_t rows) {
    constexpr int PRE = 2;
    const int n = (blockIdx.x * 256 + threadIdx.x) * 4, t = blockIdx.y, N = g.N;
    if (n >= N) return;
    const int32_t id = g.ids[t];
    const float *part = g.partial + ((int64_t)(n >> 7) * g.splits * rows + t) * 128 + (n & 127);
    f32x4_t f[kMaxGemmSplit];
#pragma unroll
    for (int s = 0; s < kMaxGemmSplit; ++s) f[s] = load4(s < g.splits, part + (int64_t)s * rows * 128);
    const int64_t at = (int64_t)t * N + n;
    uint2 bias = make_uint2(0u, 0u), res = make_uint2(0u, 0u);
    if (g.bias) bias = *reinterpret_cast<const uint2 *>(g.bias + n);
    if (g.residual) res = *reinterpret_cast<const uint2 *>(g.residual + at);
    const bool in = id >= 0 && id < g.n_slots;
    const int32_t rk = in ? min(g.rank[id], g.max_rank) : 0;
    const float sc = in ? g.scale[id] : 0.0f;
    const uint16_t *b = g.b + ((in ? slot_row0(g.row0, id, g.max_rank) : 0) * N + (int64_t)n * 8);
    const float *v = g.v + (int64_t)t * g.v_stride;
    const int ahead = !in ? 0 : g.row0 ? 1 : min(PRE, g.max_rank / 8);
    uint4 bq[PRE][4];
    f32x4_t vq[PRE][2];
#pragma unroll
    for (int o = 0; o < PRE; ++o) {
        const bool ok = o < ahead;
#pragma unroll
        for (int q = 0; q < 4; ++q) bq[o][q] = ok ? ldg16(b + (int64_t)o * N * 8 + 8 * q) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int h = 0; h < 2; ++h) vq[o][h] = load4(ok, v + 8 * o + 4 * h);
    }
    float d[4] = {0.f, 0.f, 0.f, 0.f};
    auto octet = [&](const uint4 (&bw)[4], const f32x4_t (&vw)[2]) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float bf[8];
            vec16<LORA_BF16>::widen(bw[q], bf);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[q] = fmaf(vw[e >> 2][e & 3], bf[e], d[q]);
        }
    };
#pragma unroll
    for (int o = 0; o < PRE; ++o)
        if (o < ahead && 8 * o < rk) octet(bq[o], vq[o]);
    for (int o = ahead; 8 * o < rk; ++o) {
        uint4 bw[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) bw[q] = ldg16(b + (int64_t)o * N * 8 + 8 * q);
        const f32x4_t vw[2] = {*reinterpret_cast<const f32x4_t *>(v + 8 * o), *reinterpret_cast<const f32x4_t *>(v + 8 * o + 4)};
        octet(bw, vw);
    }
    f32x4_t o = f[0];
#pragma unroll
    for (int s = 1; s < kMaxGemmSplit; ++s)
        if (s < g.splits)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] += f[s][e];
    const float bf[4] = {bf16_lo(bias.x), bf16_hi(bias.x), bf16_lo(bias.y), bf16_hi(bias.y)};
    const float rf[4] = {bf16_lo(res.x), bf16_hi(res.x), bf16_lo(res.y), bf16_hi(res.y)};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (rk > 0) o[e] = fmaf(sc, d[e], o[e]);
        o[e] += bf[e];
    }
    if (g.pre) *reinterpret_cast<uint2 *>(g.pre + at) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = act_or_none<false>(g.act, o[e]) + rf[e];
    *reinterpret_cast<uint2 *>(g.y + at) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
}

template <int MT, int WV>
static lora_status_t launch_few(const gemm_args &g, hipStream_t s) {
    const int n_shrink = g.T * (g.max_rank / kRowRanks);
    if constexpr (MT < 4)
        if (g.xq)
            hipLaunchKernelGGL((k_linear_few_fp8<MT, WV>), dim3(n_shrink + 2 * g.n_tiles_n * g.splits), dim3(WV * 64), 0, s,
                               g, n_shrink);
    if (!g.xq)
        hipLaunchKernelGGL((k_linear_few<MT, WV>), dim3(n_shrink + g.n_tiles_n * g.splits), dim3(WV * 64), 0, s, g, n_shrink);
    hipLaunchKernelGGL(k_few_finish, dim3(ceil_div(g.N, 1024), g.T), dim3(256), 0, s, g, 16 * MT);
    return hip_status(hipGetLastError());
}

// K ranges per strip of columns (128, FP8 64), each of whole steps of the workgroup's
// wavefronts: the count whose time is least by this estimate -- rounds of 256
// workgroups that stream their part of W at a CU's 22 KB a microsecond, a
// microsecond a round beside that, and the partial sums written and read at 4 TB/s.
// (bf16, 4096 x 14336, 2 ranges: one row 29 us, 64 rows 45; 3 ranges 32 and 52; 5 29
// and 51.)
bool linear_few_plan(int32_t T, int32_t K, int32_t N, bool fp8, size_t partial_bytes, int &splits, int &k_chunk) {
    // FP8: from 33 rows on the tiles of the base GEMM are faster (4096 x 14336, 64 rows 38 us, here 43)
    if (T <= 0 || T > (fp8 ? 32 : kFewRows)) return false;
    const int tiles = ceil_div(N, 128), strips = fp8 ? 2 * tiles : tiles, rows = T <= 16 ? 16 : T <= 32 ? 32 : 64;
    const int step = (T <= 32 ? 8 : 4) * (fp8 ? 128 : 32);
    double best_us = 1e30;
    splits = 0;
    for (int s = 1; s <= kMaxGemmSplit && (s == 1 || s * step <= K); ++s) {
        const int chunk = ceil_div(ceil_div(K, s), step) * step;
        const double sums = (double)tiles * s * rows * 128 * 4;
        if (sums > (double)partial_bytes) break;
        const double us = ceil_div((int64_t)strips * s, 256) * (chunk * (fp8 ? 64.0 : 256.0) / 22e3 + 1) +
                          2 * sums * T / rows / 4e6;
        if (us < best_us) {
            best_us = us;
            splits = ceil_div(K, chunk);
            k_chunk = chunk;
        }
    }
    return splits > 0;
}

// v = x A of one pool, rows in their own order: a workgroup for four ranks of a row.
template <int DT>
__global__ void __launch_bounds__(256) k_shrink_one(const typename elem<DT>::T *x, int32_t T, int32_t d, const void *a,
                                                    const int32_t *rank, const int32_t *row0, int32_t n_slots, int32_t R,
                                                    const int32_t *ids, float *v, int32_t *err) {
    shrink_row<DT, 4>(x, T, d, a, rank, row0, n_slots, R, ids, v, err, grid_index());
}

lora_status_t launch_shrink_one(const void *x, int32_t T, const lora_pool_t &p, const int32_t *ids, float *v,
                                int32_t *err, hipStream_t s) {
    const dim3 grid = grid_of((int64_t)T * (p.max_rank / kRowRanks));
    if (p.dtype == LORA_F32)
        hipLaunchKernelGGL(k_shrink_one<LORA_F32>, grid, dim3(256), 0, s, (const float *)x, T, p.d_in, p.a, p.rank, p.row0,
                           p.n_slots, p.max_rank, ids, v, err);
    else
        hipLaunchKernelGGL(k_shrink_one<LORA_BF16>, grid, dim3(256), 0, s, (const uint16_t *)x, T, p.d_in, p.a, p.rank,
                           p.row0, p.n_slots, p.max_rank, ids, v, err);
    return hip_status(hipGetLastError());
}

lora_status_t launch_linear_few(const void *x, const void *W, const uint8_t *xq, const float *xs, const uint8_t *wq,
                                const float *wsc, void *y, int32_t T, const lora_pool_t &p, const int32_t *ids, float *v,
                                int32_t *err, float *partial, size_t partial_bytes, const epilogue &epi, hipStream_t s) {
    gemm_args g{};
    set_epilogue(g, &epi);
    if (!linear_few_plan(T, p.d_in, p.d_out, xq != nullptr, partial_bytes, g.splits, g.k_chunk)) return LORA_ERR_UNSUPPORTED;
    g.x = (const uint16_t *)x;
    g.W = (const uint16_t *)W;
    g.xq = xq;
    g.xs = xs;
    g.wq = wq;
    g.wsc = wsc;
    g.y = (uint16_t *)y;
    g.T = T;
    g.K = p.d_in;
    g.N = p.d_out;
    g.a = (const uint16_t *)p.a;
    g.b = (const uint16_t *)p.b;
    g.scale = p.scale;
    g.rank = p.rank;
    g.row0 = p.row0;
    g.n_slots = p.n_slots;
    g.max_rank = p.max_rank;
    g.ids = ids;
    g.v = v;
    g.vpart = v;
    g.v_stride = p.max_rank;
    g.err = err;
    g.partial = partial;
    g.n_tiles_m = 1;
    g.n_tiles_n = g.n_tiles = ceil_div(g.N, 128);
    if (T <= 16) return launch_few<1, 8>(g, s);
    if (T <= 32) return launch_few<2, 8>(g, s);
    return launch_few<4, 4>(g, s);
}

lora_status_t launch_linear_f32(const void *x, const void *W, void *y, int32_t T, const lora_pool_t &p,
                                const int32_t *ids, const float *v, int32_t v_stride, const int32_t *perm,
                                float *partial, size_t partial_bytes, const epilogue &epi, hipStream_t s) {
    linear_f32_args g{};
    g.x = (const float *)x;
    g.W = (const float *)W;
    g.b = (const float *)p.b;
    g.scale = p.scale;
    g.bias = (const float *)epi.bias;
    g.residual = (const float *)epi.residual;
    g.rank = p.rank;
    g.row0 = p.row0;
    g.ids = ids;
    g.perm = perm;
    g.y = (float *)y;
    g.pre = (float *)epi.pre;
    g.v = v;
    g.partial = partial;
    g.T = T;
    g.K = p.d_in;
    g.N = p.d_out;
    g.n_slots = p.n_slots;
    g.max_rank = p.max_rank;
    g.v_stride = v_stride;
    g.act = epi.act;
    g.n_tiles_m = ceil_div(T, 32);
    g.n_tiles_n = ceil_div(g.N, 128);
    const int64_t all = (int64_t)g.n_tiles_m * g.n_tiles_n;
    if (all > INT32_MAX) return LORA_ERR_UNSUPPORTED;
    const int tiles = (int)all;
    g.splits = linear_f32_splits(tiles, g.K, partial_bytes, g.k_chunk);
    if (g.splits == 1) {
        hipLaunchKernelGGL(k_linear_f32<false>, grid_of(tiles), dim3(512), 0, s, g);
    } else {
        hipLaunchKernelGGL(k_linear_f32<true>, dim3(tiles * g.splits), dim3(512), 0, s, g);
        hipLaunchKernelGGL(k_linear_reduce_f32, dim3(tiles * 4), dim3(256), 0, s, g);
    }
    return hip_status(hipGetLastError());
}

}  // namespace lora
