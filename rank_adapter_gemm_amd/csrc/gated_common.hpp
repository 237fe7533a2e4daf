// The gated pair's part of the GEMM kernels: which columns a tile holds, the
// activations, the low-rank pass of both pools, the store of h = act(g) * u
// and the split-K reduction.
#pragma once

#include "gemm_common.hpp"

namespace lora {

// Gate's and up's pools, by value.
struct pair_pools {
    const void *a[2], *b[2];
    const float *scale[2];
    const int32_t *rank[2], *row0[2];
};

inline pair_pools make_pair_pools(const lora_pool_t *p) {
    return pair_pools{{p[0].a, p[1].a}, {p[0].b, p[1].b}, {p[0].scale, p[1].scale}, {p[0].rank, p[1].rank},
                      {p[0].row0, p[1].row0}};
}

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

// A row's slot in both pools: what the per-row low-rank terms need of it.
struct row_slot {
    int32_t rank[2], row0[2];
    float scale[2];
};

// Whether the 32 rows of this thread's half-wavefront (one block of a tile's
// rows, one row a thread) name more than `most` adapters.
__device__ __forceinline__ bool many_adapters(int32_t id, int most) {
    const int sh = (threadIdx.x & 32);
    uint32_t pend = (uint32_t)(__ballot(id >= 0) >> sh);
    int n = 0;
    while (__any(pend != 0 && n <= most)) {
        const int32_t a = __shfl(id, pend ? __ffs((int)pend) - 1 + sh : 0, 64);
        const uint32_t same = (uint32_t)(__ballot(id == a) >> sh);
        n += pend != 0;
        pend &= ~same;
    }
    return n > most;
}

__device__ __forceinline__ row_slot load_row_slot(const gemm_args &g, int32_t id) {
    row_slot r{{0, 0}, {0, 0}, {0.f, 0.f}};
    if (id >= 0 && id < g.n_slots) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            r.rank[m] = min(g.sl[m].rank[id], g.max_rank);
            r.row0[m] = (int32_t)slot_row0(g.sl[m].row0, id, g.max_rank);
            r.scale[m] = g.sl[m].scale[id];
        }
    }
    return r;
}

// One projection's (M: gate's or up's) low-rank terms for kernels at their
// register limit.  The blocks' first adapters and ranks are loaded together,
// what is left of them one step at a time; a row's rank, place and scale come
// from LDS (a lookup in the pool would be one more trip to memory per adapter).
template <int RB, int CB, int M>
__device__ __forceinline__ void lora_pass_lean(const gemm_args &g, f32x16_t (&acc)[RB][CB * 2], const int32_t *s_t,
                                               const int32_t *s_id, const row_slot *s_slot, int wrow0, int wcol0,
                                               int lane) {
    gemm_args q = g;
    q.b = g.sl[M].b;
    q.v = g.v + g.sl[M].v_off;
    const int half = lane >> 5;
    float4 v0[RB], v1[RB];
    uint4 bq[RB][CB];
    uint32_t rest[RB];
    auto first_of = [&](int rb, uint32_t pend, int32_t &a, int32_t &ra, int32_t &ro, float &sa, uint32_t &rows) {
        const int row0 = wrow0 + rb * 32, f = __ffs((int)pend) - 1;
        a = uniform_i(s_id[row0 + f]);
        ra = uniform_i(s_slot[row0 + f].rank[M]);
        ro = uniform_i(s_slot[row0 + f].row0[M]);
        sa = __int_as_float(uniform_i(__float_as_int(s_slot[row0 + f].scale[M])));
        rows = (uint32_t)__ballot(s_id[row0 + (lane & 31)] == a);
    };
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        const int row = wrow0 + rb * 32 + (lane & 31);
        rest[rb] = (uint32_t)__ballot(s_id[row] >= 0);
        if (!rest[rb]) continue;
        int32_t a, ra, ro;
        float sa;
        uint32_t rows;
        first_of(rb, rest[rb], a, ra, ro, sa, rows);
        lora_step_load<CB>(q, a, ra, ro, s_id[row] == a, s_t[row], 0, half, wcol0, lane, v0[rb], v1[rb], bq[rb]);
    }
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        const int row = wrow0 + rb * 32 + (lane & 31);
        const uint32_t live = (uint32_t)__ballot(s_t[row] >= 0);
        for (uint32_t pend = rest[rb]; pend;) {
            int32_t a, ra, ro;
            float sa;
            uint32_t rows;
            first_of(rb, pend, a, ra, ro, sa, rows);
            const bool mine = (rows >> (lane & 31)) & 1u;
            for (int ks = 0; ks * 16 < ra; ++ks) {
                if (ks > 0 || pend != rest[rb])
                    lora_step_load<CB>(q, a, ra, ro, mine, s_t[row], ks, half, wcol0, lane, v0[rb], v1[rb], bq[rb]);
                lora_step_mfma<CB, 2, M>(acc[rb], sa, mine && 16 * ks + 8 * half < ra, v0[rb], v1[rb], bq[rb],
                                         (live & ~rows) != 0, rows);
            }
            pend &= ~rows;
        }
    }
}

// The low-rank terms of both pools on the matrix cores: gate's into the even
// column blocks, up's into the odd ones.  col0: the wavefront's first column of h.
template <int RB, int CB, int RG, int KB, int RF>
__device__ __forceinline__ void gated_lora_pass(const gemm_args &g, f32x16_t (&acc)[RB][CB], const int32_t *s_t,
                                                const int32_t *s_id, int wrow0, int col0, int lane) {
    static_assert(CB % 2 == 0, "a wavefront holds whole pairs");
    gemm_args q = g;
    q.b = g.sl[0].b;
    q.scale = g.sl[0].scale;
    q.rank = g.sl[0].rank;
    q.row0 = g.sl[0].row0;
    lora_pass_impl<RB, CB / 2, RG, KB, RF, 2, 0, true>(q, acc, s_t, s_id, 0, wrow0, col0, lane);
    q.b = g.sl[1].b;
    q.scale = g.sl[1].scale;
    q.rank = g.sl[1].rank;
    q.row0 = g.sl[1].row0;
    q.v = g.v + g.sl[1].v_off;
    lora_pass_impl<RB, CB / 2, RG, KB, RF, 2, 1, true>(q, acc, s_t, s_id, 0, wrow0, col0, lane);
}

// 4 fp32 values, zeros where not ok.  (A branch, not a choice between two
// values in memory, which would put the zeros and the result there.)
__device__ __forceinline__ f32x4_t load4(bool ok, const float *p) {
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    if (ok) v = *reinterpret_cast<const f32x4_t *>(p);
    return v;
}

// Both low-rank sums of one row, d[m][q] = sum_j v[j] B[j][n] of the 8 columns
// n = n0 + ST q below N: rank octets in order, both projections' loads of an octet
// in flight together.  ST is the number of lanes that share a row, so that
// neighbours read neighbouring columns (16 bytes each; a lane with 8
// neighbouring columns would touch a cache line of its own with every load:
// 2240 rows of which 192 single, FP8 4096 x 14336: 463 us).
template <int ST>
__device__ __forceinline__ void low_rank8(const gemm_args &g, const row_slot &rs, int64_t t, int n0,
                                          float (&d)[2][8]) {
    const int oct = (max(rs.rank[0], rs.rank[1]) + 7) >> 3;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int q = 0; q < 8; ++q) d[m][q] = 0.0f;
    for (int gg = 0; gg < oct; ++gg) {
        f32x4_t vv[2][2];
        uint4 bq[2][8];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const bool in = 8 * gg < rs.rank[m];
            const float *vrow = g.v + t * g.v_stride + g.sl[m].v_off + gg * 8;
            const uint16_t *b = g.sl[m].b + ((int64_t)rs.row0[m] + 8 * gg) * g.N + (int64_t)n0 * 8;
            vv[m][0] = load4(in, vrow);
            vv[m][1] = load4(in, vrow + 4);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                bq[m][q] = in && n0 + ST * q < g.N ? ldg16(b + ST * q * 8) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                float bf[8];
                vec16<LORA_BF16>::widen(bq[m][q], bf);
#pragma unroll
                for (int e = 0; e < 8; ++e) d[m][q] = fmaf(vv[m][e >> 2][e & 3], bf[e], d[m][q]);
            }
    }
}

// 8 columns of one row: gate and up stored where they are kept, and h.
__device__ __forceinline__ void gated_finish8(const gemm_args &g, int64_t t, int n, float (&o)[2][8]) {
    const int64_t at = t * g.N + n;
    if (g.sl[0].y) {
        stg16(g.sl[0].y + at, vec16<LORA_BF16>::narrow(o[0]));
        stg16(g.sl[1].y + at, vec16<LORA_BF16>::narrow(o[1]));
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) o[0][e] = act_value<false>(g.act, o[0][e]) * o[1][e];
    stg16(g.y + at, vec16<LORA_BF16>::narrow(o[0]));
}

// A tile row's part in the low-rank terms.  Blocks of 32 rows with few
// adapters (long segments) take them on the matrix cores, from s_id, an adapter
// after the other; the rows of other blocks each from their own adapter in
// the store, from s_slot.  The border was measured: 192 single tokens of 64
// adapters (FP8 base, 4096 x 14336) take 66 us row by row and 148 us block by
// block; the 70B-sized mixed batch (2 to 4 adapters of rank 8-64 a block)
// 4450, 4412 and 4212 us with a border of 1, 2 and 4, and no less with 8 or 16.
constexpr int kBlockAdapters = 4;

__device__ __forceinline__ void set_row(const gemm_args &g, int32_t id, bool per_row, int32_t &s_id, row_slot &s_slot) {
    const bool apart = per_row || many_adapters(id, kBlockAdapters);
    s_id = apart ? -1 : id;
    s_slot = load_row_slot(g, id);
}

// The store of a whole tile: the fp32 sums of WR * 32 rows at a time go
// through LDS, where the terms of rows that are not in the sums yet are added,
// and a thread then owns 8 neighbouring columns of gate, up and h of one row
// (16-byte stores, one rounding each).
template <int BM, int BN, int WV, int WR, int RB, int CB>
__device__ __forceinline__ void gated_store_tile(const gemm_args &g, f32x16_t (&acc)[RB][CB], float *smem_f,
                                                 const int32_t *s_t, const int32_t *s_id, const row_slot *s_slot, int n0,
                                                 int w, int lane) {
    constexpr int WM = BM / WR, WN = BN / (WV / WR), SLD = BN + 4, CPR = BN / 16, ITEMS = WR * 32 * CPR;
    const int wm = w / (WV / WR), wn = w % (WV / WR), tid = w * 64 + lane;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        __syncthreads();
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                smem_f[(wm * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3)) * SLD + wn * WN + cb * 32 + (lane & 31)] =
                    acc[rb][cb][e];
        __syncthreads();
        for (int i = tid; i < ITEMS; i += WV * 64) {
            const int r = i / CPR, c = i % CPR, row = (r >> 5) * WM + rb * 32 + (r & 31);
            if (s_t[row] < 0 || s_id[row] >= 0 || max(s_slot[row].rank[0], s_slot[row].rank[1]) <= 0) continue;
            float d[2][8];
            low_rank8<CPR>(g, s_slot[row], s_t[row], gated_col(n0) + c, d);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int cc = c + CPR * q;
                    float *at = smem_f + r * SLD + (cc >> 5) * 64 + (cc & 31) + 32 * m;
                    *at = fmaf(s_slot[row].scale[m], d[m][q], *at);
                }
        }
        __syncthreads();
        for (int i = tid; i < ITEMS; i += WV * 64) {
            const int r = i / CPR, c = (i % CPR) * 8, row = (r >> 5) * WM + rb * 32 + (r & 31);
            const int32_t t = s_t[row];
            const int n = gated_col(n0) + c;
            if (t < 0 || n >= g.N) continue;
            const float *src = smem_f + r * SLD + (c >> 5) * 64 + (c & 31);
            float o[2][8];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                *reinterpret_cast<float4 *>(o[m]) = *reinterpret_cast<const float4 *>(src + 32 * m);
                *reinterpret_cast<float4 *>(o[m] + 4) = *reinterpret_cast<const float4 *>(src + 32 * m + 4);
            }
            gated_finish8(g, t, n, o);
        }
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
    __shared__ float s_d[2][RW][HN];                      // the rows' low-rank sums
    const int32_t t = p < g.T ? perm_row(g.perm, p, g.T) : -1;
    const row_slot rs = load_row_slot(g, t >= 0 ? g.ids[t] : -1);
    const int lr = threadIdx.x / CPR, lc = threadIdx.x % CPR;
    {
        float d[2][8];
        low_rank8<CPR>(g, rs, t, tn * HN + lc, d);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int q = 0; q < 8; ++q) s_d[m][lr][lc + CPR * q] = d[m][q];
    }
    __syncthreads();
    if (t < 0 || n >= g.N) return;
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
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int q = 0; q < 8; ++q) o[m][q] = fmaf(rs.scale[m], s_d[m][lr][c + q], o[m][q]);
    gated_finish8(g, t, n, o);
}

template <int BM, int BN> static void launch_gated_reduce(const gemm_args &g, hipStream_t s) {
    constexpr int RW = 256 / (BN / 16);
    hipLaunchKernelGGL((k_gated_reduce<BM, BN>), dim3(g.n_tiles * (BM / RW)), dim3(256), 0, s, g);
}

// Workgroup b's tile and K range in the fp32 kernels: each XCD takes a
// contiguous run of (column tile, range, row tile), rows fastest, so the row
// tiles that read the same weights run together on one XCD's L2 (333 x 1032 x
// 2744: 69 us, and 71 with the rows spread over the XCDs).
__device__ __forceinline__ void f32_tile(int b, int total, int n_tiles_m, int splits, int &tm, int &tn, int &split) {
    const int per = total / kXcds, rem = total % kXcds, x = b % kXcds;
    const int v = x * per + min(x, rem) + b / kXcds;
    tm = v % n_tiles_m;
    split = v / n_tiles_m % splits;
    tn = v / n_tiles_m / splits;
}

// K ranges per tile of the fp32 kernels (tiles of `area` sums): the count whose
// time is least by this estimate -- rounds of 512 workgroups (two a CU, each at
// half a CU's 0.6 TFLOP/s) and the partial sums written and read at 4 TB/s.
// Ranges have at least 128 terms.
inline int f32_splits(int tiles, int K, int area, size_t partial_bytes, int &k_chunk) {
    int best = 1;
    double best_us = 1e30;
    for (int s = 1; s <= kMaxGemmSplit && (s == 1 || s * 128 <= K); ++s) {
        const double sums = (double)s * tiles * area * 4;
        if (s > 1 && sums > (double)partial_bytes) break;
        const double us = 2.0 * area * K / 0.3e6 * ceil_div((int64_t)tiles * s, 512) / s + (s > 1 ? 2 * sums / 4e6 : 0);
        if (us < best_us) {
            best = s;
            best_us = us;
        }
    }
    k_chunk = ceil_div(ceil_div(K, best), 32) * 32;
    return ceil_div(K, k_chunk);
}

// Implemented beside their base GEMMs; g holds everything but the tile plan.
lora_status_t launch_gemm_gated(gemm_args &g, size_t partial_bytes, hipStream_t s);
lora_status_t launch_gemm_gated_fp8(gemm_args &g, size_t partial_bytes, hipStream_t s);

}  // namespace lora
