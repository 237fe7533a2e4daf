// The linear layer with bias, activation and residual: its part of the GEMM
// kernels.  act is not linear, so every row's low-rank term is in its sums before
// the epilogue, on the matrix cores or row by row in the store, as in the gated pair.
#pragma once

#include "gated_common.hpp"

namespace lora {

// A row's slot: what the per-row low-rank term needs of it.
struct row_term {
    int32_t rank, row0;
    float scale;
};

// s_id: the row's adapter where its block's terms go through the matrix cores, -1
// where they are added in the store (from s_term), as set_row.
__device__ __forceinline__ void set_row_term(const gemm_args &g, int32_t id, int32_t &s_id, row_term &s_term) {
    s_id = many_adapters(id, kBlockAdapters) ? -1 : id;
    s_term = row_term{0, 0, 0.0f};
    if (id >= 0)
        s_term = row_term{min(g.rank[id], g.max_rank), (int32_t)slot_row0(g.row0, id, g.max_rank), g.scale[id]};
}

// The low-rank terms on the matrix cores for kernels at their register limit (as
// lora_pass_lean): a block of 32 rows and one of its adapters after the other, a
// row's rank, place and scale from LDS.
template <int RB, int CB>
__device__ __forceinline__ void act_pass_lean(const gemm_args &g, f32x16_t (&acc)[RB][CB], const int32_t *s_t,
                                              const int32_t *s_id, const row_term *s_term, int wrow0, int wcol0, int lane) {
    const int half = lane >> 5;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        const int row0 = wrow0 + rb * 32, row = row0 + (lane & 31);
        const uint32_t live = (uint32_t)__ballot(s_t[row] >= 0);
        for (uint32_t pend = (uint32_t)__ballot(s_id[row] >= 0); pend;) {
            const int f = row0 + __ffs((int)pend) - 1;
            const int32_t a = uniform_i(s_id[f]), ra = uniform_i(s_term[f].rank), ro = uniform_i(s_term[f].row0);
            const float sa = __int_as_float(uniform_i(__float_as_int(s_term[f].scale)));
            const uint32_t rows = (uint32_t)__ballot(s_id[row] == a);
            const bool mine = (rows >> (lane & 31)) & 1u;
            for (int ks = 0; ks * 16 < ra; ++ks) {
                float4 v0, v1;
                uint4 bq[CB];
                lora_step_load<CB>(g, a, ra, ro, mine, s_t[row], ks, half, wcol0, lane, v0, v1, bq);
                lora_step_mfma<CB, 1, 0>(acc[rb], sa, mine && 16 * ks + 8 * half < ra, v0, v1, bq, (live & ~rows) != 0,
                                         rows);
            }
            pend &= ~rows;
        }
    }
}

// The row's low-rank sums of the columns n0 + ST q, q = 0..7, below N (see low_rank8).
template <int ST>
__device__ __forceinline__ void row_term8(const gemm_args &g, const row_term &rt, int64_t t, int n0, float (&d)[8]) {
#pragma unroll
    for (int q = 0; q < 8; ++q) d[q] = 0.0f;
    const uint16_t *b = g.b + (int64_t)rt.row0 * g.N + (int64_t)n0 * 8;
    const float *vrow = g.v + t * g.v_stride;
    for (int j = 0; j < rt.rank; j += 8, b += (int64_t)g.N * 8) {
        const f32x4_t v[2] = {*reinterpret_cast<const f32x4_t *>(vrow + j), *reinterpret_cast<const f32x4_t *>(vrow + j + 4)};
        uint4 bq[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) bq[q] = n0 + ST * q < g.N ? ldg16(b + ST * q * 8) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            float bf[8];
            vec16<LORA_BF16>::widen(bq[q], bf);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[q] = fmaf(v[e >> 2][e & 3], bf[e], d[q]);
        }
    }
}

constexpr int kRowRanks = 4;

// Four ranks j0.. of one row's v = x A, by a workgroup of WV wavefronts that share the
// row's length (one wavefront to a row of 14336 values: 28 us, all of it latency).
// `item`: of T R / kRowRanks.  Records the row's id where it names no usable slot.
template <int DT, int WV>
__device__ __forceinline__ void shrink_row(const typename elem<DT>::T *x, int32_t T, int32_t d, const void *pool_a,
                                           const int32_t *rank, const int32_t *row0, int32_t n_slots, int32_t R,
                                           const int32_t *ids, float *v, int32_t *err, int64_t item) {
    typedef typename elem<DT>::T E;
    constexpr int VN = vec16<DT>::n, U = 4;
    __shared__ float s_v[WV][kRowRanks];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, groups = R / kRowRanks;
    const int64_t t = item / groups;
    if (t >= T) return;                                   // (the whole workgroup)
    const int j0 = (int)(item - t * groups) * kRowRanks;
    const int32_t id = ids[t];
    const bool in = id >= 0 && id < n_slots;
    const int32_t r = in ? min(rank[id], R) : 0;
    float acc[kRowRanks] = {};
    if (in && (!row0 || j0 < r)) {                        // as in k_shrink_pair
        const E *row = x + t * d, *a = (const E *)pool_a + (slot_row0(row0, id, R) + j0) * d;
        const int n = d / VN;
        for (int c0 = tid; c0 < n; c0 += 64 * WV * U) {
            uint4 xq[U], aq[U][kRowRanks];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t c = (int64_t)min(c0 + 64 * WV * u, n - 1) * VN;
                xq[u] = ldg16(row + c);
#pragma unroll
                for (int q = 0; q < kRowRanks; ++q) aq[u][q] = ldg16(a + q * (int64_t)d + c);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (c0 + 64 * WV * u >= n) break;
                float xf[VN], af[VN];
                vec16<DT>::widen(xq[u], xf);
#pragma unroll
                for (int q = 0; q < kRowRanks; ++q) {
                    vec16<DT>::widen(aq[u][q], af);
#pragma unroll
                    for (int e = 0; e < VN; ++e) acc[q] = fmaf(xf[e], af[e], acc[q]);
                }
            }
        }
    }
#pragma unroll
    for (int q = 0; q < kRowRanks; ++q)
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) acc[q] += __shfl_xor(acc[q], o, 64);
    if (lane == 0)
#pragma unroll
        for (int q = 0; q < kRowRanks; ++q) s_v[w][q] = acc[q];
    __syncthreads();
    if (tid < kRowRanks) {
        float f = s_v[0][tid];
#pragma unroll
        for (int u = 1; u < WV; ++u) f += s_v[u][tid];
        v[t * R + j0 + tid] = j0 + tid < r ? f : 0.0f;
    }
    if (tid == 0 && j0 == 0 && (id < -1 || id >= n_slots || (in && r <= 0))) flag_bad_row(err, (int32_t)t);
}

// The store of a whole tile: the fp32 sums of WR * 32 rows at a time go through
// LDS, where the terms that are not in them yet are added; a thread then owns 8
// neighbouring columns of one row (16-byte loads and stores, one rounding).  FP8,
// 192 rows of 64 adapters, 4096 x 14336: 43 us, of which the rows' terms are 12 (0.5
// MB of B a tile beside 0.9 MB of operands, at 33 KB / us into a CU; asked for
// further ahead they take the same).
template <int BM, int BN, int WV, int WR, int RB, int CB>
__device__ __forceinline__ void act_store_tile(const gemm_args &g, f32x16_t (&acc)[RB][CB], float *smem_f,
                                               const int32_t *s_t, const int32_t *s_id, const row_term *s_term,
                                               int n0) {
    constexpr int WM = BM / WR, WN = BN / (WV / WR), SLD = BN + 4, CPR = BN / 8, ITEMS = WR * 32 * CPR;
    constexpr int NT = WV * 64, PER = ITEMS / NT;
    static_assert(ITEMS % NT == 0, "whole rounds of the threads");
    const int tid = threadIdx.x, lane = tid & 63, w = uniform_i(tid >> 6), wm = w / (WV / WR), wn = w % (WV / WR);
    const int cc = (tid % CPR) * 8, n = n0 + cc;          // a thread's columns are the same in every round
    const uint4 bias = n < g.N ? load_bias8(g, n) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        // the residual's next values are under way while the sums are staged and finished
        auto row_of = [&](int k) {
            const int r = (tid + k * NT) / CPR;
            return n < g.N ? s_t[(r >> 5) * WM + rb * 32 + (r & 31)] : -1;
        };
        auto residual_of = [&](int k) {
            const int32_t t = k < PER ? row_of(k) : -1;
            return t >= 0 ? load_residual8(g, t, n) : make_uint4(0u, 0u, 0u, 0u);
        };
        uint4 next = residual_of(0);
        __syncthreads();
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                smem_f[(wm * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3)) * SLD + wn * WN + cb * 32 + (lane & 31)] =
                    acc[rb][cb][e];
        __syncthreads();
        for (int i = tid; i < ITEMS; i += NT) {
            const int r = i / CPR, c = i % CPR, row = (r >> 5) * WM + rb * 32 + (r & 31);
            if (s_t[row] < 0 || s_id[row] >= 0 || s_term[row].rank <= 0) continue;
            float d[8];
            row_term8<CPR>(g, s_term[row], s_t[row], n0 + c, d);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                float *at = smem_f + r * SLD + c + CPR * q;
                *at = fmaf(s_term[row].scale, d[q], *at);
            }
        }
        __syncthreads();
#pragma unroll 1                                           // (unrolled, the blocks' loop would not be)
        for (int k = 0; k < PER; ++k) {
            const int r = (tid + k * NT) / CPR, t = row_of(k);
            const uint4 res = next;
            next = residual_of(k + 1);
            if (t < 0) continue;
            float o[8];
            *reinterpret_cast<float4 *>(o) = *reinterpret_cast<const float4 *>(smem_f + r * SLD + cc);
            *reinterpret_cast<float4 *>(o + 4) = *reinterpret_cast<const float4 *>(smem_f + r * SLD + cc + 4);
            epilogue8(g, t, n, o, bias, res);
        }
    }
}

}  // namespace lora
