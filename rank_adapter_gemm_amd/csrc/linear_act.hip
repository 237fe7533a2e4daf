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
