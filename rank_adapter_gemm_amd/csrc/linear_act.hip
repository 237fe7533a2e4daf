// The linear layer with bias, activation and residual in fp32:
//   y = act(x W + bias + s_a (x A_a) B_a) + residual      per row, a = ids[t]
// (the bf16 and FP8 forms are instantiations of their base GEMMs).
//
// 32 rows x 128 columns per workgroup of 4 wavefronts on v_mfma_f32_32x32x2_f32, K
// in steps of 32 DMA'd into a ring of three stages, as the gated pair's fp32
// kernel; grids of few tiles split K, and the sums go through LDS or the partial
// buffer to threads that add the row's low-rank term and own 4 columns of a row.
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

// The low-rank sums of a row's columns n = n0 + 32 q (32 lanes share a row and read
// neighbouring columns).
__device__ __forceinline__ void row_term4(const linear_f32_args &g, const row_term &rt, int64_t t, int n0, float (&d)[4]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) d[q] = 0.0f;
    const float *b = g.b + (int64_t)rt.row0 * g.N + (int64_t)n0 * 8, *vrow = g.v + t * g.v_stride;
    for (int j = 0; j < rt.rank; j += 8, b += (int64_t)g.N * 8) {
        f32x4_t vv[2], bb[4][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            vv[h] = *reinterpret_cast<const f32x4_t *>(vrow + j + 4 * h);
#pragma unroll
            for (int q = 0; q < 4; ++q) bb[q][h] = load4(n0 + 32 * q < g.N, b + 32 * q * 8 + 4 * h);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 8; ++e) d[q] = fmaf(vv[e >> 2][e & 3], bb[q][e >> 2][e & 3], d[q]);
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

template <bool SPLIT> __global__ void __launch_bounds__(256, 2) k_linear_f32(linear_f32_args g) {
    constexpr int BK = 32, NS = 3, XST = 32 * BK, STAGE = XST + BK * 128, WS = 128 + 4, PER = 5;
    __shared__ __attribute__((aligned(1024))) float smem[NS * STAGE];     // stages: x [32][BK], W [BK][128]; sums: [32][WS]
    static_assert(32 * WS <= NS * STAGE, "the sums fit the stages' LDS");
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    int tm, tn, split;
    const int total = g.n_tiles_m * g.n_tiles_n * (SPLIT ? g.splits : 1);
    if (grid_index() >= total) return;
    f32_tile((int)grid_index(), total, g.n_tiles_m, SPLIT ? g.splits : 1, tm, tn, split);
    const int tile = tm * g.n_tiles_n + tn, m0 = tm * 32, n0 = tn * 128;
    const int N = g.N, T = g.T, k_begin = split * g.k_chunk, k_end = min(g.K, k_begin + g.k_chunk);
    __shared__ row_term s_term[SPLIT ? 1 : 32];
    if (!SPLIT && tid < 32) s_term[tid] = load_row_term(g, m0 + tid < T ? perm_row(g.perm, m0 + tid, T) : -1);
    // DMA, 16-byte chunks.  x: thread -> row tid / 8, place tid % 8, which holds
    // the row's chunk place ^ (row % 8).  W: chunk 256 j + tid -> row / 32, column chunk % 32.
    const int xr = tid >> 3, xk = 4 * ((tid & 7) ^ (xr & 7));
    const int32_t t_x = m0 + xr < T ? perm_row(g.perm, m0 + xr, T) : -1;
    const float *xp = g.x + (int64_t)(t_x < 0 ? 0 : t_x) * g.K + xk;
    const int wr = tid >> 5, wc = (tid & 31) * 4;
    const bool wok = n0 + wc < N;
    const float *wp = g.W + (int64_t)wr * N + (wok ? n0 + wc : 0);
    auto dma_stage = [&](int kt, int buf) {
        float *xs = smem + buf * STAGE, *wsm = xs + XST;
        const int k0 = k_begin + kt * BK;
        dma16(t_x >= 0 && k0 + xk < k_end ? (const void *)(xp + k0) : (const void *)g_zero16, xs + w * 64 * 4);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            dma16(wok && k0 + 8 * j + wr < k_end ? (const void *)(wp + (int64_t)(k0 + 8 * j) * N) : (const void *)g_zero16,
                  wsm + (256 * j + w * 64) * 4);
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
        // product i of a step takes k = i from the lower half-wavefront and
        // k = 16 + i from the upper: a lane's 16 values of x are neighbours
        const float *xs = smem + (kt % NS) * STAGE + (lane & 31) * BK;
        const float *wsm = smem + (kt % NS) * STAGE + XST + 16 * (lane >> 5) * 128 + w * 32 + (lane & 31);
        float a[16], b[16];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<f32x4_t *>(a + 4 * i) =
                *reinterpret_cast<const f32x4_t *>(xs + 4 * ((4 * (lane >> 5) + i) ^ (lane & 7)));
#pragma unroll
        for (int i = 0; i < 16; ++i) b[i] = wsm[i * 128];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], acc, 0, 0, 0);
    }
    float *part = SPLIT ? g.partial + ((int64_t)tile * g.splits + split) * 32 * 128 : nullptr;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const int r = 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3), c = w * 32 + (lane & 31);
        if (SPLIT) part[r * 128 + c] = acc[e];
        else smem[r * WS + c] = acc[e];
    }
    if (SPLIT) return;
    __syncthreads();
    for (int i = tid; i < 32 * 32; i += 256) {
        const int r = i >> 5, c = i & 31;
        const int64_t t = m0 + r < T ? perm_row(g.perm, m0 + r, T) : -1;
        if (t < 0 || s_term[r].rank <= 0) continue;
        float d[4];
        row_term4(g, s_term[r], t, n0 + c, d);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float *at = smem + r * WS + c + 32 * q;
            *at = fmaf(s_term[r].scale, d[q], *at);
        }
    }
    __syncthreads();
    for (int i = tid; i < 32 * 32; i += 256) {
        const int r = i >> 5, c = (i & 31) * 4, n = n0 + c;
        const int64_t t = m0 + r < T ? perm_row(g.perm, m0 + r, T) : -1;
        if (t < 0 || n >= N) continue;
        epilogue4(g, t, n, *reinterpret_cast<const f32x4_t *>(smem + r * WS + c));
    }
}

// The pieces' sums, in split order: 8 rows of one tile per workgroup.
__global__ void __launch_bounds__(256) k_linear_reduce_f32(linear_f32_args g) {
    const int tile = blockIdx.x >> 2, lr = threadIdx.x >> 5, r = (blockIdx.x & 3) * 8 + lr, c = (threadIdx.x & 31) * 4;
    const int p = tile / g.n_tiles_n * 32 + r, n0 = tile % g.n_tiles_n * 128, n = n0 + c;
    const int64_t t = p < g.T ? perm_row(g.perm, p, g.T) : -1;
    const row_term rt = load_row_term(g, t);
    __shared__ float s_d[8][128];                         // the rows' low-rank sums
    float d[4];
    row_term4(g, rt, t, n0 + (threadIdx.x & 31), d);
#pragma unroll
    for (int q = 0; q < 4; ++q) s_d[lr][(threadIdx.x & 31) + 32 * q] = d[q];
    __syncthreads();
    if (t < 0 || n >= g.N) return;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
    const float *part = g.partial + (int64_t)tile * g.splits * 32 * 128 + r * 128 + c;
    for (int s = 0; s < g.splits; ++s, part += 32 * 128) {
        const f32x4_t f = *reinterpret_cast<const f32x4_t *>(part);
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] += f[q];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = fmaf(rt.scale, s_d[lr][c + q], o[q]);
    epilogue4(g, t, n, o);
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
    g.splits = f32_splits(tiles, g.K, 32 * 128, partial_bytes, g.k_chunk);
    if (g.splits == 1) {
        hipLaunchKernelGGL(k_linear_f32<false>, grid_of(tiles), dim3(256), 0, s, g);
    } else {
        hipLaunchKernelGGL(k_linear_f32<true>, dim3(tiles * g.splits), dim3(256), 0, s, g);
        hipLaunchKernelGGL(k_linear_reduce_f32, dim3(tiles * 4), dim3(256), 0, s, g);
    }
    return hip_status(hipGetLastError());
}

}  // namespace lora
