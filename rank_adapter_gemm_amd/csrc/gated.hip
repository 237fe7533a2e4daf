// The gated feed-forward pair h = act(g) * u, g = x Wg + s_a (x Ag_a) Bg_a and u
// likewise: the launcher of the bf16 and FP8 kernels (the base GEMMs' gated
// instantiations, gemm.hip and gemm_fp8.hip) and the fp32 kernel.
#include "gated_common.hpp"

namespace lora {

// ---------------------------------------------------------------------------
// fp32: 32 rows x 64 columns of h per workgroup of 4 wavefronts, each with 32
// columns of one projection on v_mfma_f32_32x32x2_f32 (fp32 products and sums;
// the matrix cores' fp32 rate is twice the vector units').  Small tiles leave
// less of the chip idle in the last round, and several share a CU (333 x 1032
// x 2744: 64 us, 59 TFLOP/s; tiles of 64 rows, split over K, 83).  K in steps of
// 32, DMA'd into a ring of three stages (a step's products take less time than
// a load from HBM).  Grids of few tiles split K; the sums then go through LDS or
// the partial buffer to threads that add the row's low-rank terms and own 4
// columns of a row.  Bound by the products' rate and the waits between steps.
// ---------------------------------------------------------------------------
struct gated_f32_args {
    const float *x, *W[2], *b[2], *scale[2];
    const int32_t *rank[2], *row0[2];
    float *h, *keep[2];
    const int32_t *ids, *perm;
    const float *v;
    float *partial;                    // [tile][split][32][128]
    int32_t T, K, N, n_slots, max_rank, act, n_tiles_m, n_tiles_n, splits, k_chunk;
};

// What a row's low-rank terms need of its slot in both pools.
__device__ __forceinline__ row_slot load_row_slot(const gated_f32_args &g, int64_t t) {
    row_slot r{{0, 0}, {0, 0}, {0.f, 0.f}};
    const int32_t id = t >= 0 ? g.ids[t] : -1;
    if (id >= 0 && id < g.n_slots) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            r.rank[m] = min(g.rank[m][id], g.max_rank);
            r.row0[m] = (int32_t)slot_row0(g.row0[m], id, g.max_rank);
            r.scale[m] = g.scale[m][id];
        }
    }
    return r;
}

// Both low-rank sums of a row's columns n = n0 + 16 q (16 lanes share a row
// and read neighbouring columns); an octet's loads of both projections are in
// flight together.
__device__ __forceinline__ void low_rank4(const gated_f32_args &g, const row_slot &rs, int64_t t, int n0,
                                          float (&d)[2][4]) {
    const int oct = (max(rs.rank[0], rs.rank[1]) + 7) >> 3;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int q = 0; q < 4; ++q) d[m][q] = 0.0f;
    for (int gg = 0; gg < oct; ++gg) {
        f32x4_t vv[2][2], bb[2][4][2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const bool in = 8 * gg < rs.rank[m];
            const float *b = g.b[m] + (((int64_t)rs.row0[m] + 8 * gg) * g.N + (int64_t)n0 * 8);
            const float *vt = g.v + t * 2 * g.max_rank + m * g.max_rank + 8 * gg;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                vv[m][h] = load4(in, vt + 4 * h);
#pragma unroll
                for (int q = 0; q < 4; ++q) bb[m][q][h] = load4(in && n0 + 16 * q < g.N, b + 16 * q * 8 + 4 * h);
            }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 8; ++e) d[m][q] = fmaf(vv[m][e >> 2][e & 3], bb[m][q][e >> 2][e & 3], d[m][q]);
    }
}

// 4 neighbouring columns of one row from both projections' sums o.
__device__ __forceinline__ void gated_finish4(const gated_f32_args &g, int64_t t, int n, const float (&o)[2][4]) {
    const int64_t at = t * g.N + n;
    float4 h;
    h.x = act_value<true>(g.act, o[0][0]) * o[1][0];
    h.y = act_value<true>(g.act, o[0][1]) * o[1][1];
    h.z = act_value<true>(g.act, o[0][2]) * o[1][2];
    h.w = act_value<true>(g.act, o[0][3]) * o[1][3];
    *reinterpret_cast<float4 *>(g.h + at) = h;
    if (g.keep[0]) {
        *reinterpret_cast<float4 *>(g.keep[0] + at) = make_float4(o[0][0], o[0][1], o[0][2], o[0][3]);
        *reinterpret_cast<float4 *>(g.keep[1] + at) = make_float4(o[1][0], o[1][1], o[1][2], o[1][3]);
    }
}

template <bool SPLIT> __global__ void __launch_bounds__(256, 2) k_gated_f32(gated_f32_args g) {
    constexpr int BK = 32, NS = 3, XST = 32 * BK, STAGE = XST + BK * 128, WS = 128 + 4, PER = 5;
    __shared__ __attribute__((aligned(1024))) float smem[NS * STAGE];     // stages: x [32][BK], W [BK][128]; sums: [32][WS]
    static_assert(32 * WS <= NS * STAGE, "the sums fit the stages' LDS");
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    int tm, tn, split;
    const int total = g.n_tiles_m * g.n_tiles_n * (SPLIT ? g.splits : 1);
    if (grid_index() >= total) return;
    f32_tile((int)grid_index(), total, g.n_tiles_m, SPLIT ? g.splits : 1, tm, tn, split);
    const int tile = tm * g.n_tiles_n + tn, m0 = tm * 32, n0 = tn * 64;
    const int N = g.N, T = g.T, k_begin = split * g.k_chunk, k_end = min(g.K, k_begin + g.k_chunk);
    __shared__ row_slot s_slot[SPLIT ? 1 : 32];
    if (!SPLIT && tid < 32) s_slot[tid] = load_row_slot(g, m0 + tid < T ? perm_row(g.perm, m0 + tid, T) : -1);
    // DMA, 16-byte chunks.  x: thread -> row tid / 8, place tid % 8, which holds
    // the row's chunk place ^ (row % 8).  W: chunk 256 j + tid -> row / 32, gate's 16
    // chunks then up's.
    const int xr = tid >> 3, xk = 4 * ((tid & 7) ^ (xr & 7));
    const int32_t t_x = m0 + xr < T ? perm_row(g.perm, m0 + xr, T) : -1;
    const float *xp = g.x + (int64_t)(t_x < 0 ? 0 : t_x) * g.K + xk;
    const int wr = tid >> 5, wc = (tid & 15) * 4;
    const bool wok = n0 + wc < N;
    const float *wp = ((tid & 16) ? g.W[1] : g.W[0]) + (int64_t)wr * N + (wok ? n0 + wc : 0);
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
    for (int i = tid; i < 32 * 16; i += 256) {
        const int r = i >> 4, c = i & 15;
        const int64_t t = m0 + r < T ? perm_row(g.perm, m0 + r, T) : -1;
        if (t < 0 || max(s_slot[r].rank[0], s_slot[r].rank[1]) <= 0) continue;
        float d[2][4];
        low_rank4(g, s_slot[r], t, n0 + c, d);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float *at = smem + r * WS + 64 * m + c + 16 * q;
                *at = fmaf(s_slot[r].scale[m], d[m][q], *at);
            }
    }
    __syncthreads();
    for (int i = tid; i < 32 * 16; i += 256) {
        const int r = i >> 4, c = (i & 15) * 4, n = n0 + c;
        const int64_t t = m0 + r < T ? perm_row(g.perm, m0 + r, T) : -1;
        if (t < 0 || n >= N) continue;
        float o[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
            *reinterpret_cast<float4 *>(o[m]) = *reinterpret_cast<const float4 *>(smem + r * WS + 64 * m + c);
        gated_finish4(g, t, n, o);
    }
}

// The pieces' sums, in split order: 16 rows of one tile per workgroup.
__global__ void __launch_bounds__(256) k_gated_reduce_f32(gated_f32_args g) {
    const int tile = blockIdx.x >> 1, r = (blockIdx.x & 1) * 16 + (threadIdx.x >> 4), c = (threadIdx.x & 15) * 4;
    const int p = tile / g.n_tiles_n * 32 + r, n = tile % g.n_tiles_n * 64 + c;
    const int64_t t = p < g.T ? perm_row(g.perm, p, g.T) : -1;
    const row_slot rs = load_row_slot(g, t);
    __shared__ float s_d[2][16][64];                      // the rows' low-rank sums
    {
        float d[2][4];
        low_rank4(g, rs, t, tile % g.n_tiles_n * 64 + (threadIdx.x & 15), d);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int q = 0; q < 4; ++q) s_d[m][threadIdx.x >> 4][(threadIdx.x & 15) + 16 * q] = d[m][q];
    }
    __syncthreads();
    if (t < 0 || n >= g.N) return;
    float o[2][4] = {};
    const float *part = g.partial + (int64_t)tile * g.splits * 32 * 128 + r * 128 + c;
    for (int s = 0; s < g.splits; ++s, part += 32 * 128)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const float4 f = *reinterpret_cast<const float4 *>(part + 64 * m);
            o[m][0] += f.x; o[m][1] += f.y; o[m][2] += f.z; o[m][3] += f.w;
        }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int q = 0; q < 4; ++q) o[m][q] = fmaf(rs.scale[m], s_d[m][threadIdx.x >> 4][c + q], o[m][q]);
    gated_finish4(g, t, n, o);
}

// ---------------------------------------------------------------------------
// v = x A of both slices for rows in their own order.  A wavefront sums four
// ranks of one row and slice: the row's few workgroups spread over the chip
// (a single token's 2 x 16 ranks over 8 wavefronts, not one workgroup), and
// each lane has all its loads of a stretch of 8 vectors in flight.  x is read
// again for every four ranks, from cache.  Bound by latency: one token of 16
// ranks, 4096 wide, 9 us.
// ---------------------------------------------------------------------------
constexpr int kPairRanks = 4;

template <int DT>
__global__ void __launch_bounds__(256) k_shrink_pair(const typename elem<DT>::T *x, int32_t T, int32_t d, pair_pools pp,
                                                     int32_t n_slots, int32_t R, const int32_t *ids, float *v,
                                                     int32_t *err) {
    typedef typename elem<DT>::T E;
    constexpr int VN = vec16<DT>::n, U = 8;
    const int lane = threadIdx.x & 63;
    const int groups = 2 * R / kPairRanks;                // per row; R is a multiple of 8
    const int64_t item = grid_index() * 4 + (threadIdx.x >> 6);
    const int64_t t = item / groups;
    if (t >= T) return;
    const int j2 = (int)(item - t * groups) * kPairRanks, m = j2 >= R, j0 = j2 - m * R;
    const int32_t id = ids[t];
    const bool in = id >= 0 && id < n_slots;
    int32_t r = in ? min(pp.rank[m][id], R) : 0;
    const int32_t other = in ? pp.rank[1][id] : 1;
    float acc[kPairRanks] = {};
    // A padded slot has all its max_rank rows (zeros from its rank on), so its
    // loads need not wait for the rank; a packed one ends with its capacity.
    if (in && (!pp.row0[m] || j0 < r)) {
        const E *row = x + t * d, *a = (const E *)pp.a[m] + (slot_row0(pp.row0[m], id, R) + j0) * d;
        const int n = d / VN;
        for (int c0 = lane; c0 < n; c0 += 64 * U) {
            uint4 xq[U], aq[U][kPairRanks];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t c = (int64_t)min(c0 + 64 * u, n - 1) * VN;   // past the end: the last vector, not summed
                xq[u] = ldg16(row + c);
#pragma unroll
                for (int q = 0; q < kPairRanks; ++q) aq[u][q] = ldg16(a + q * (int64_t)d + c);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (c0 + 64 * u >= n) break;
                float xf[VN], af[VN];
                vec16<DT>::widen(xq[u], xf);
#pragma unroll
                for (int q = 0; q < kPairRanks; ++q) {
                    vec16<DT>::widen(aq[u][q], af);
#pragma unroll
                    for (int e = 0; e < VN; ++e) acc[q] = fmaf(xf[e], af[e], acc[q]);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < kPairRanks; ++q)
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) acc[q] += __shfl_xor(acc[q], o, 64);
    }
    if (lane == 0 && j2 == 0 && (id < -1 || id >= n_slots || (in && (r <= 0 || other <= 0))))
        flag_bad_row(err, (int32_t)t);
    if (lane == 0)
        *reinterpret_cast<float4 *>(v + t * 2 * R + j2) =
            make_float4(j0 < r ? acc[0] : 0.f, j0 + 1 < r ? acc[1] : 0.f, j0 + 2 < r ? acc[2] : 0.f,
                        j0 + 3 < r ? acc[3] : 0.f);
}

lora_status_t launch_shrink_pair(const void *x, int32_t T, const lora_pool_t *p, const int32_t *ids, float *v,
                                 int32_t *err, hipStream_t s) {
    const pair_pools pp = make_pair_pools(p);
    const int64_t items = (int64_t)T * (2 * p[0].max_rank / kPairRanks);
    const dim3 grid = grid_of((items + 3) / 4);
    if (p[0].dtype == LORA_F32)
        hipLaunchKernelGGL(k_shrink_pair<LORA_F32>, grid, dim3(256), 0, s, (const float *)x, T, p[0].d_in, pp,
                           p[0].n_slots, p[0].max_rank, ids, v, err);
    else
        hipLaunchKernelGGL(k_shrink_pair<LORA_BF16>, grid, dim3(256), 0, s, (const uint16_t *)x, T, p[0].d_in, pp,
                           p[0].n_slots, p[0].max_rank, ids, v, err);
    return hip_status(hipGetLastError());
}

lora_status_t launch_gated_forward(const gated_call &c, hipStream_t s) {
    const lora_pool_t *p = c.pools;
    if (p[0].dtype == LORA_F32) {
        gated_f32_args g{};
        g.x = (const float *)c.x;
        for (int m = 0; m < 2; ++m) {
            g.W[m] = (const float *)c.W[m];
            g.b[m] = (const float *)p[m].b;
            g.scale[m] = p[m].scale;
            g.rank[m] = p[m].rank;
            g.row0[m] = p[m].row0;
        }
        g.h = (float *)c.h;
        g.keep[0] = (float *)c.gate;
        g.keep[1] = (float *)c.up;
        g.ids = c.ids;
        g.perm = c.perm;
        g.v = c.v;
        g.T = c.T;
        g.K = p[0].d_in;
        g.N = p[0].d_out;
        g.n_slots = p[0].n_slots;
        g.max_rank = p[0].max_rank;
        g.act = c.act;
        g.n_tiles_n = ceil_div(g.N, 64);
        g.partial = c.partial;
        g.n_tiles_m = ceil_div(c.T, 32);
        const int tiles = g.n_tiles_m * g.n_tiles_n;
        g.splits = f32_splits(tiles, g.K, 32 * 128, c.partial_bytes, g.k_chunk);
        if (g.splits == 1) {
            hipLaunchKernelGGL(k_gated_f32<false>, grid_of(tiles), dim3(256), 0, s, g);
        } else {
            hipLaunchKernelGGL(k_gated_f32<true>, dim3(tiles * g.splits), dim3(256), 0, s, g);
            hipLaunchKernelGGL(k_gated_reduce_f32, dim3(tiles * 2), dim3(256), 0, s, g);
        }
        return hip_status(hipGetLastError());
    }
    gemm_args g{};
    g.x = (const uint16_t *)c.x;
    g.xq = c.xq;
    g.xs = c.xs;
    g.y = (uint16_t *)c.h;
    g.T = c.T;
    g.K = p[0].d_in;
    g.N = p[0].d_out;
    g.perm = c.perm;
    g.n_slots = p[0].n_slots;
    g.max_rank = p[0].max_rank;
    g.ids = c.ids;
    g.v = c.v;
    g.v_stride = 2 * p[0].max_rank;
    g.partial = c.partial;
    g.act = c.act;
    void *keep[2] = {c.gate, c.up};
    for (int m = 0; m < 2; ++m)
        g.sl[m] = gemm_slice{(const uint16_t *)c.W[m], (uint16_t *)keep[m], g.N, 0, (const uint16_t *)p[m].b,
                             p[m].scale, p[m].rank, p[m].row0, m * p[0].max_rank, c.wq[m], c.wsc[m]};
    return c.xq ? launch_gemm_gated_fp8(g, c.partial_bytes, s) : launch_gemm_gated(g, c.partial_bytes, s);
}

}  // namespace lora
