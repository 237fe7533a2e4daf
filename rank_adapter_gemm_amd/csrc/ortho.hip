// Orthogonalised updates: for each of n matrices G (an adapter slot's gradient of
// A, [d_in][r], or of B, [r][d_out])
//   X = G / (|G|_F + eps);  X <- c0 X + c1 (X X^T) X + c2 (X X^T)^2 X,  step by step
// (Newton-Schulz products: an odd polynomial of every singular value, the singular
// vectors kept).  The short side r is at most 128, so X is never formed: with M =
// X^T X (r x r, X taken with its long side down) a step is X <- X Q with Q = c0 I +
// c1 M + c2 M^2, and M <- M Q^2.  All are polynomials of the first M, so they
// commute, and the last X is G times one r x r matrix P:
//   k_ortho_gram    G^T G, split over the long side                 one read of G
//   k_ortho_poly    the pieces' sum, and the steps on r x r         a workgroup a matrix
//                   (r <= 16: k_ortho_apply does it)
//   k_ortho_apply   G P                                     one more read, one write
//
// Passes: M cannot say which way a direction that is not in X is to go.  Its
// eigenvalue there is a rounding, 2^-53 of either sign, and c0^2 times as large after
// each step; a negative one is not held back by the polynomial.  (On one M, rank 1 in 8 to
// 72 columns: 8 steps of 3.4445 up to 3e-7 off, 10 3e-4, 12 0.3, 16 5e5.)  So where the
// product of c0^2 would pass 2^22, 6 such steps, M is made anew from X itself, that is from G P
// (k_ortho_regram, one more read of G), and the next steps' matrix is joined to P by
// a product of all its tiles (k_ortho_join: P is symmetric but for roundings, and c0's
// product makes those large): 7 steps of 32 x 4096 x 16 take 28 us, 6 14.6.  What is
// left is c0's product times 2^-53, as with the steps on X in 64 bits; callers may ask
// for 2^30.
//
// 64 bits: small singular values are amplified, by c0 at every step (485-fold in 5
// steps of 3.4445), and an error e of M by up to 3e4 e relative to what those
// directions get.  32-bit sums of M (6e-8) would show in the result; 64-bit ones
// (v_mfma_f64_16x16x4_f64) do not.  So M, the steps and P are 64-bit, and G P is 64-bit
// products.  For bf16 G and P of at most 2^11, 6 such steps, it is exact bf16 products of P
// in three parts, summed in fp32: P's large values, where G has nothing, cancel there to
// 2^-24 2^11 of a row, a sixteenth of the result's half step.
//
// Tiles: W tiles of 16 indices of the short side hold it (W = 1, 2, 4, 8); only those
// on and under the diagonal are computed.  G goes from memory to the products
// without LDS: a lane reads neighbouring values of one row of G, and which index of
// the short side (or of the long one) stands at which place of a product is chosen
// to fit.  G [D][r] ("tall"): place p of tile s is index W p + s; G [r][D]: 16 s + p.
//
// 32 x 4096 x 16 bf16: 14 us, two launches of 7 and 8, latency.  8 x 64 x 14336
// fp32: 79 us: 17 for the sums, 36 for the steps, 28 for G P, all bound by the
// 64-bit products (64 clocks each; 9, 18 and 14 us of them at the full rate) and
// the reads before the first of them.
#include "gemm_common.hpp"

namespace lora {

typedef double f64x4_t __attribute__((ext_vector_type(4)));

// v_mfma_f64_16x16x4_f64, lane l: A row l % 16, B column l % 16, both k = l / 16;
// element e of the result is row 4 e + l / 16, column l % 16 (checked on the GPU).
__device__ __forceinline__ f64x4_t mfma64(double a, double b, f64x4_t c) {
    return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ int mfma64_row(int e, int lane) { return 4 * e + (lane >> 4); }

constexpr int ortho_tiles(int W) { return W * (W + 1) / 2; }
// Number of tile (a, b), a >= b.
__device__ __forceinline__ constexpr int ortho_tile(int a, int b) { return a * (a + 1) / 2 + b; }
// The short-side index at place p of tile s.
template <int W, bool TALL> __device__ __forceinline__ int ortho_index(int s, int p) {
    return TALL ? W * p + s : 16 * s + p;
}

struct ortho_args {
    const void *g;
    void *out;
    double *part;                      // [n][splits][tiles][64][4]: a tile's sums, lane by lane
    double *poly;                      // [n][16 W][16 W], zeros past r: these steps' matrix
    const double *before;              // k_ortho_regram, k_ortho_join: P of the steps before, transposed
    double *joined;                    // k_ortho_join: P of all steps, transposed
    double *inv;                       // [n]: 1 / (|G| + eps)
    int32_t D, n, r, splits, chunk;    // chunk: long-side indices per split, a multiple of 64
    int32_t rows, blocks;              // k_ortho_apply: long-side indices per workgroup, workgroups per matrix
    int32_t steps, first;              // first: the steps start at G
    float eps, scale;
    float coef[kMaxOrthoSteps][3];
};

// ---------------------------------------------------------------------------
// G^T G.  Eight wavefronts share a split's long side and add their sums through
// LDS in a fixed order.  Of 8 tiles a side a wavefront holds half the rows of
// tiles (0, 3, 4, 7 or 1, 2, 5, 6: 18 tiles each), and two of four share a part.
// ---------------------------------------------------------------------------
template <int W> __device__ __forceinline__ constexpr bool gram_owns(int half, int a) {
    return W < 8 || (((a + 1) >> 1) & 1) == half;
}
template <int W> __device__ __forceinline__ constexpr int gram_at(int half, int a, int b) {
    int n = 0;
    for (int i = 0; i < a; ++i) n += gram_owns<W>(half, i) ? i + 1 : 0;
    return n + b;
}

// 16-byte vector (or W * 2 or W * 4 bytes) of G, zeros where not ok.
template <int BYTES> __device__ __forceinline__ void load_bytes(const void *p, bool ok, uint32_t *q) {
    if constexpr (BYTES == 2) {
        q[0] = ok ? *(const uint16_t *)p : 0u;
    } else if constexpr (BYTES == 4) {
        q[0] = ok ? *(const uint32_t *)p : 0u;
    } else if constexpr (BYTES == 8) {
        const uint2 v = ok ? *(const uint2 *)p : make_uint2(0u, 0u);
        q[0] = v.x; q[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < BYTES / 16; ++i) {
            const uint4 v = ok ? ldg16((const char *)p + 16 * i) : make_uint4(0u, 0u, 0u, 0u);
            q[4 * i] = v.x; q[4 * i + 1] = v.y; q[4 * i + 2] = v.z; q[4 * i + 3] = v.w;
        }
    }
}
// Value i of such a vector.
template <int DT> __device__ __forceinline__ float value_of(const uint32_t *q, int i) {
    if (DT == LORA_F32) return __uint_as_float(q[i]);
    return (i & 1) ? bf16_hi(q[i >> 1]) : bf16_lo(q[i >> 1]);
}

// Wavefronts, and of those the ones that share a part's long side.
template <int W> struct gram_cfg {
    static constexpr int WAVES = W == 8 ? 4 : 8, KW = W == 8 ? 2 : 8;
};

template <int DT, int W, bool TALL, int HALF, int N>
__device__ __forceinline__ void gram_wave(const ortho_args &g, const typename elem<DT>::T *base, int begin, int end,
                                          int kw, int lane, f64x4_t (&acc)[N]) {
    constexpr int VN = vec16<DT>::n, KW = gram_cfg<W>::KW, EB = elem<DT>::bytes;
    // a wavefront reads U groups of STEP long-side indices at once: a value of W
    // short-side indices for each of 4 (tall), or 16 bytes of each tile's 16 rows
    constexpr int STEP = TALL ? 4 : 4 * VN, U = TALL ? 16 / W : 1;
    constexpr int WORDS = TALL ? (W * EB + 3) / 4 : 4 * W;
    const int p = lane & 15, kg = lane >> 4;
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = f64x4_t{0.0, 0.0, 0.0, 0.0};
    uint32_t q[2][U][WORDS];
    auto load = [&](int i0, uint32_t (&to)[U][WORDS]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (TALL) {
                const int i = i0 + 4 * u + kg;
                load_bytes<W * EB>(base + (int64_t)i * g.r + W * p, i < end && W * p < g.r, to[u]);
            } else {
                const int i = i0 + STEP * u + VN * kg;
#pragma unroll
                for (int s = 0; s < W; ++s)
                    load_bytes<16>(base + (int64_t)(16 * s + p) * g.D + i, i < end && 16 * s + p < g.r, to[u] + 4 * s);
            }
        }
    };
    auto products = [&](const uint32_t (&from)[U][WORDS]) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < (TALL ? 1 : VN); ++k) {
                double x[W];
#pragma unroll
                for (int s = 0; s < W; ++s) x[s] = (double)value_of<DT>(TALL ? from[u] : from[u] + 4 * s, TALL ? s : k);
#pragma unroll
                for (int a = 0; a < W; ++a)
                    if (gram_owns<W>(HALF, a))
#pragma unroll
                        for (int b = 0; b <= a; ++b)
                            acc[gram_at<W>(HALF, a, b)] = mfma64(x[a], x[b], acc[gram_at<W>(HALF, a, b)]);
            }
    };
    constexpr int STRIDE = KW * STEP * U;
    int i = begin + kw * STEP * U;
    load(i, q[0]);
    for (; i < end; i += 2 * STRIDE) {
        load(i + STRIDE, q[1]);
        products(q[0]);
        load(i + 2 * STRIDE, q[0]);
        products(q[1]);
    }
}

// The sums of the KW wavefronts (kw) that share a part: wavefront tile % KW adds up a
// tile, the others hand theirs over through LDS, then all add and store.
template <int W, int KW, int HALF, bool ADD, int N>
__device__ __forceinline__ void gram_sums(f64x4_t *part, const f64x4_t (&acc)[N], f64x4_t (*s_sum)[ortho_tiles(W)][64],
                                          int kw, int lane) {
#pragma unroll
    for (int a = 0; a < W; ++a)
        if (gram_owns<W>(HALF, a))
#pragma unroll
            for (int b = 0; b <= a; ++b) {
                const int tile = ortho_tile(a, b), to = tile % KW;
                f64x4_t f = acc[gram_at<W>(HALF, a, b)];
                if constexpr (!ADD) {
                    if (kw != to) s_sum[kw < to ? kw : kw - 1][tile][lane] = f;
                } else if (kw == to) {
#pragma unroll
                    for (int k = 0; k < KW - 1; ++k) f += s_sum[k][tile][lane];
                    part[tile * 64 + lane] = f;
                }
            }
}

// To split `item`'s place; the whole workgroup calls it.
template <int W, int KW, int N>
__device__ __forceinline__ void gram_finish(const ortho_args &g, const f64x4_t (&acc)[N],
                                            f64x4_t (*s_sum)[ortho_tiles(W)][64], int64_t item, int kw, int half, int lane) {
    f64x4_t *part = reinterpret_cast<f64x4_t *>(g.part) + item * ortho_tiles(W) * 64;
    if (W == 8 && half) gram_sums<W, KW, 1, false>(part, acc, s_sum, kw, lane);
    else gram_sums<W, KW, 0, false>(part, acc, s_sum, kw, lane);
    __syncthreads();
    if (W == 8 && half) gram_sums<W, KW, 1, true>(part, acc, s_sum, kw, lane);
    else gram_sums<W, KW, 0, true>(part, acc, s_sum, kw, lane);
}

template <int DT, int W, bool TALL>
__global__ void __launch_bounds__(gram_cfg<W>::WAVES * 64) k_ortho_gram(ortho_args g) {
    constexpr int NT = ortho_tiles(W), KW = gram_cfg<W>::KW, HALVES = gram_cfg<W>::WAVES / KW, N = NT / HALVES;
    __shared__ f64x4_t s_sum[KW - 1][NT][64];
    const int64_t item = grid_index();
    if (item >= (int64_t)g.n * g.splits) return;
    const int64_t mat = item / g.splits;
    const int split = (int)(item - mat * g.splits), lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int kw = wave / HALVES, half = wave % HALVES;
    const typename elem<DT>::T *base = (const typename elem<DT>::T *)g.g + mat * g.D * g.r;
    const int begin = split * g.chunk, end = min(g.D, begin + g.chunk);
    f64x4_t acc[N];
    if (half) gram_wave<DT, W, TALL, 1>(g, base, begin, end, kw, lane, acc);
    else gram_wave<DT, W, TALL, 0>(g, base, begin, end, kw, lane, acc);
    gram_finish<W, KW>(g, acc, s_sum, item, kw, half, lane);
}

// ---------------------------------------------------------------------------
// The steps on the r x r matrices, one workgroup a matrix.  All matrices are
// symmetric and commute, so a product is symmetric too, and only its tiles on and
// under the diagonal are computed.  Symmetry also makes a tile its own operand: the
// result's element e of a lane, X[16 a + 4 e + kg][16 b + p], is what the lane gives
// to product e as the right operand (k in a, column in b) and as the left one (row
// in b, k in a).  So a matrix of one tile stays in registers through all steps, and
// larger ones lie in LDS lane by lane, both triangles, one of them written across.
// ---------------------------------------------------------------------------
// Tile (a, b), a >= b, of P at its place in memory, and its mirror image.
template <int W, bool TALL>
__device__ __forceinline__ void poly_store(const ortho_args &g, int64_t mat, int a, int b, const f64x4_t &v, int lane) {
    double *poly = g.poly + mat * 256 * W * W;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = ortho_index<W, TALL>(a, mfma64_row(e, lane)), j = ortho_index<W, TALL>(b, lane & 15);
        const double f = i < g.r && j < g.r ? v[e] : 0.0;
        poly[i * 16 * W + j] = f;
        if (a != b) poly[j * 16 * W + i] = f;
    }
}

__device__ __forceinline__ double wave_sum64(double d) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) d += __shfl_xor(d, o, 64);
    return d;
}

// One of the tiles of product's operands after the other, four k at a time.
__device__ __forceinline__ f64x4_t mfma64_tile(const f64x4_t &x, const f64x4_t &y, f64x4_t c) {
#pragma unroll
    for (int s = 0; s < 4; ++s) c = mfma64(x[s], y[s], c);
    return c;
}

// The sum of a tile over the splits, in their order.
template <int NT> __device__ __forceinline__ f64x4_t poly_part(const ortho_args &g, int64_t mat, int tile, int lane) {
    const f64x4_t *part = reinterpret_cast<const f64x4_t *>(g.part) + (mat * g.splits * NT + tile) * 64 + lane;
    f64x4_t m = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 8
    for (int s = 0; s < g.splits; ++s) m += part[(int64_t)s * NT * 64];
    return m;
}

// 1 / (|G| + eps): from the trace of G^T G, or as the first steps left it.
__device__ __forceinline__ double poly_inv(const ortho_args &g, int64_t mat, double trace) {
    return g.first ? 1.0 / (sqrt(trace) + (double)g.eps) : g.inv[mat];
}

// One tile: P in a wavefront's registers, and 1 / (|G| + eps).  Few enough
// products for k_ortho_apply to do them itself, every workgroup of a matrix the
// same (as a launch of its own: 32 x 4096 x 16 15.9 us for 14.5), where one pass is all.
__device__ __forceinline__ f64x4_t poly_one(const ortho_args &g, int64_t mat, int lane, double &inv) {
    f64x4_t m = poly_part<1>(g, mat, 0, lane), one, pr;
    double d = 0.0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        one[e] = mfma64_row(e, lane) == (lane & 15) ? 1.0 : 0.0;
        d += one[e] * m[e];
    }
    inv = poly_inv(g, mat, wave_sum64(d));
    const f64x4_t zero = {0.0, 0.0, 0.0, 0.0};
    m *= inv * inv;
    pr = one;
    for (int step = 0; step < g.steps; ++step) {
        const f64x4_t q = (double)g.coef[step][0] * one + (double)g.coef[step][1] * m +
                          (double)g.coef[step][2] * mfma64_tile(m, m, zero);
        const f64x4_t t = mfma64_tile(m, q, zero);
        pr = step == 0 ? q : mfma64_tile(pr, q, zero);
        m = mfma64_tile(t, q, zero);
    }
    return pr;
}

// As a launch of its own, where several passes follow each other.
template <bool TALL> __global__ void __launch_bounds__(64) k_ortho_poly_one(ortho_args g) {
    const int64_t mat = grid_index();
    if (mat >= g.n) return;
    const int lane = threadIdx.x & 63;
    double inv;
    poly_store<1, TALL>(g, mat, 0, 0, poly_one(g, mat, lane, inv), lane);
    if (g.first && lane == 0) g.inv[mat] = inv;
}

// 2 or 4 tiles a side.  A step is three rounds with a barrier each: M M and from it
// Q; T = M Q and the new P = P Q; and the new M = T Q.  A wavefront has one tile of a
// product; of the second round's it has one of T and one of P, given out so that
// the four SIMDs have equally many.  Bound by the 64-bit products of one CU: 4
// tiles, 5 steps: 170 tiles, 64 clocks a product.
template <int W> struct poly_cfg {
    static constexpr int NT = ortho_tiles(W), WAVES = W == 4 ? 12 : 6;
};

template <int W, bool TALL> __global__ void __launch_bounds__(poly_cfg<W>::WAVES * 64) k_ortho_poly(ortho_args g) {
    constexpr int NT = poly_cfg<W>::NT;
    __shared__ f64x4_t s_m[W * W][64], s_q[W * W][64], s_t[W * W][64], s_p[W * W][64];
    __shared__ double s_trace[W];
    const int64_t mat = grid_index();
    if (mat >= g.n) return;
    const int lane = threadIdx.x & 63, wave = uniform_i(threadIdx.x >> 6), p = lane & 15, kg = lane >> 4;
    // wave's tile of M, Q and T, and its tile of P, or none (wavefronts 4 apart share a SIMD)
    const bool own = wave < NT, own_p = W == 4 ? wave < 8 || wave >= 10 : wave >= NT;
    const int tm = own ? wave : 0, tp = !own_p ? 0 : W == 4 ? (wave < 8 ? wave : wave - 2) : wave - NT;
    auto row_of = [](int tile) {
        int a = 0;
        while ((a + 1) * (a + 2) / 2 <= tile) ++a;
        return a;
    };
    const int ma = row_of(tm), mb = tm - ma * (ma + 1) / 2, pa = row_of(tp), pb = tp - pa * (pa + 1) / 2;
    auto put = [&](f64x4_t (*to)[64], int a, int b, const f64x4_t &v) {
        to[a * W + b][lane] = v;
        if (a != b)                                       // element e is row 4 e + kg, column p
#pragma unroll
            for (int e = 0; e < 4; ++e)
                reinterpret_cast<double *>(&to[b * W + a][16 * (p & 3) + 4 * e + kg])[p >> 2] = v[e];
    };
    auto product = [&](const f64x4_t (*x)[64], const f64x4_t (*y)[64], int a, int b) {
        f64x4_t c = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
        for (int k = 0; k < W; ++k) c = mfma64_tile(x[k * W + a][lane], y[k * W + b][lane], c);
        return c;
    };
    f64x4_t m = {0.0, 0.0, 0.0, 0.0}, one, r;
#pragma unroll
    for (int e = 0; e < 4; ++e) one[e] = ma == mb && mfma64_row(e, lane) == p ? 1.0 : 0.0;
    if (own) {
        m = poly_part<NT>(g, mat, tm, lane);
        if (ma == mb) {
            const double d = wave_sum64(one[0] * m[0] + one[1] * m[1] + one[2] * m[2] + one[3] * m[3]);
            if (lane == 0) s_trace[ma] = d;
        }
    }
    __syncthreads();
    double trace = s_trace[0];
#pragma unroll
    for (int i = 1; i < W; ++i) trace += s_trace[i];
    const double inv = poly_inv(g, mat, trace);
    if (g.first && threadIdx.x == 0) g.inv[mat] = inv;
    m *= inv * inv;
    if (own) put(s_m, ma, mb, m);
    __syncthreads();
    for (int step = 0; step < g.steps; ++step) {
        const bool last = step + 1 == g.steps;
        if (own) {
            const f64x4_t q = (double)g.coef[step][0] * one + (double)g.coef[step][1] * m +
                              (double)g.coef[step][2] * product(s_m, s_m, ma, mb);
            put(s_q, ma, mb, q);
            if (step == 0) put(s_p, ma, mb, q);
        }
        __syncthreads();
        if (step > 0 && own_p) r = product(s_p, s_q, pa, pb);
        if (last) break;
        if (own) put(s_t, ma, mb, product(s_m, s_q, ma, mb));
        __syncthreads();
        if (step > 0 && own_p) put(s_p, pa, pb, r);
        if (own) {
            m = product(s_t, s_q, ma, mb);
            put(s_m, ma, mb, m);
        }
        __syncthreads();
    }
    if (own_p) poly_store<W, TALL>(g, mat, pa, pb, g.steps > 1 ? r : s_p[pa * W + pb][lane], lane);
}

// 8 tiles a side: both triangles of four matrices would not fit in LDS, so the two
// factors of a product lie there, the tiles on and under the diagonal, in rows of 17
// values (both ways of reading a tile then spread over the banks); a wavefront has
// three tiles of each matrix.
template <bool TALL> __global__ void __launch_bounds__(768) k_ortho_poly8(ortho_args g) {
    constexpr int W = 8, NT = ortho_tiles(W), OWN = 3, TILE = 16 * 17;
    __shared__ double s_x[NT * TILE], s_y[NT * TILE];
    __shared__ double s_trace;
    const int64_t mat = grid_index();
    if (mat >= g.n) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, p = lane & 15, kg = lane >> 4;
    int ta[OWN], tb[OWN], tt[OWN];
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
        tt[o] = wave * OWN + o;
        int a = 0;
        while ((a + 1) * (a + 2) / 2 <= tt[o]) ++a;
        ta[o] = a;
        tb[o] = tt[o] - a * (a + 1) / 2;
    }
    f64x4_t m[OWN], pr[OWN], q[OWN], t[OWN];
    auto put = [&](double *s, const f64x4_t (&v)[OWN]) {
#pragma unroll
        for (int o = 0; o < OWN; ++o)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[tt[o] * TILE + mfma64_row(e, lane) * 17 + p] = v[o][e];
    };
    // own tiles of x y, both symmetric and commuting, so their product is too
    auto product = [&](const double *x, const double *y, f64x4_t (&to)[OWN]) {
#pragma unroll
        for (int o = 0; o < OWN; ++o) {
            f64x4_t c = {0.0, 0.0, 0.0, 0.0};
#pragma unroll(OWN > 1 ? 1 : W)
            for (int k = 0; k < W; ++k) {
                const double *xt = x + (ta[o] >= k ? ortho_tile(ta[o], k) : ortho_tile(k, ta[o])) * TILE;
                const double *yt = y + (k >= tb[o] ? ortho_tile(k, tb[o]) : ortho_tile(tb[o], k)) * TILE;
                const int xs = ta[o] >= k ? 17 : 1, xk = ta[o] >= k ? 1 : 17;   // strides of its row, of k
                const int ys = k >= tb[o] ? 1 : 17, yk = k >= tb[o] ? 17 : 1;
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    c = mfma64(xt[p * xs + (4 * s + kg) * xk], yt[p * ys + (4 * s + kg) * yk], c);
            }
            to[o] = c;
        }
    };
    auto one = [&](int o, int e) { return ta[o] == tb[o] && mfma64_row(e, lane) == p ? 1.0 : 0.0; };
#pragma unroll
    for (int o = 0; o < OWN; ++o) m[o] = f64x4_t{0.0, 0.0, 0.0, 0.0};
    const f64x4_t *part = reinterpret_cast<const f64x4_t *>(g.part) + mat * g.splits * NT * 64 + lane;
#pragma unroll 2
    for (int s = 0; s < g.splits; ++s, part += NT * 64)
#pragma unroll
        for (int o = 0; o < OWN; ++o) m[o] += part[tt[o] * 64];
    put(s_x, m);
    __syncthreads();
    if (wave == 0) {
        double d = 0.0;
        for (int i = lane; i < 16 * W; i += 64) d += s_x[ortho_tile(i >> 4, i >> 4) * TILE + (i & 15) * 18];
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) d += __shfl_xor(d, o, 64);
        if (lane == 0) s_trace = d;
    }
    __syncthreads();
    const double inv = poly_inv(g, mat, s_trace);
    if (g.first && threadIdx.x == 0) g.inv[mat] = inv;
#pragma unroll
    for (int o = 0; o < OWN; ++o)
#pragma unroll
        for (int e = 0; e < 4; ++e) m[o][e] *= inv * inv;
    for (int step = 0; step < g.steps; ++step) {
        const double c0 = g.coef[step][0], c1 = g.coef[step][1], c2 = g.coef[step][2];
        const bool last = step + 1 == g.steps;
        put(s_x, m);
        __syncthreads();
        product(s_x, s_x, t);
#pragma unroll
        for (int o = 0; o < OWN; ++o)
#pragma unroll
            for (int e = 0; e < 4; ++e) q[o][e] = c0 * one(o, e) + c1 * m[o][e] + c2 * t[o][e];
        put(s_y, q);
        __syncthreads();
        if (!last) product(s_x, s_y, t);                  // M Q
        __syncthreads();
        if (step == 0) {
#pragma unroll
            for (int o = 0; o < OWN; ++o) pr[o] = q[o];
        } else {
            put(s_x, pr);
            __syncthreads();
            product(s_x, s_y, pr);                        // P Q
            __syncthreads();
        }
        if (!last) {
            put(s_x, t);
            __syncthreads();
            product(s_x, s_y, m);                         // M Q Q
            __syncthreads();
        }
    }
#pragma unroll
    for (int o = 0; o < OWN; ++o) poly_store<W, TALL>(g, mat, ta[o], tb[o], pr[o], lane);
}

// P of the steps before and of these, P Q, by a wavefront a tile: transposed, Q P^T
// (Q is symmetric, what lies in memory is P^T).
template <int W> __global__ void __launch_bounds__(64) k_ortho_join(ortho_args g) {
    constexpr int LD = 16 * W;
    const int64_t item = grid_index(), mat = item / (W * W);
    if (mat >= g.n) return;
    const int tile = (int)(item - mat * (W * W)), lane = threadIdx.x & 63, p = lane & 15, kg = lane >> 4;
    const double *q = g.poly + (mat * LD + tile / W * 16 + p) * LD, *pt = g.before + mat * LD * LD + tile % W * 16 + p;
    f64x4_t c = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 8
    for (int k = 0; k < LD; k += 4) c = mfma64(q[k + kg], pt[(k + kg) * LD], c);
    double *out = g.joined + (mat * LD + tile / W * 16) * LD + tile % W * 16 + p;
#pragma unroll
    for (int e = 0; e < 4; ++e) out[mfma64_row(e, lane) * LD] = c[e];
}

// ---------------------------------------------------------------------------
// G P.  P lies in LDS (bf16: in three parts); the result's rows are P's, its
// columns long-side indices, so that a lane holds neighbouring values of the
// result in either layout.
// ---------------------------------------------------------------------------
// 4 neighbouring values, and back.
__device__ __forceinline__ f32x4_t load_4(const float *p) { return *reinterpret_cast<const f32x4_t *>(p); }
__device__ __forceinline__ f32x4_t load_4(const uint16_t *p) {
    const uint2 q = *reinterpret_cast<const uint2 *>(p);
    return f32x4_t{bf16_lo(q.x), bf16_hi(q.x), bf16_lo(q.y), bf16_hi(q.y)};
}
__device__ __forceinline__ void store_4(float *p, const f32x4_t &v) { *reinterpret_cast<f32x4_t *>(p) = v; }
__device__ __forceinline__ void store_4(uint16_t *p, const f32x4_t &v) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// 64-bit products.  tall: a block is 16 rows i of G, and a lane reads 4
// neighbouring values j of one; wide: 64 columns i, and a lane reads 4
// neighbouring ones of row j.
template <int W, bool TALL> struct apply_f64 {
    static constexpr int LD = 16 * W + 4, CB = TALL && W > 1 ? 2 : 1, R4 = TALL ? W : 4 * W, S = TALL ? 1 : 4;
    f32x4_t x[R4];

    template <typename E> __device__ __forceinline__ void load(const ortho_args &g, const E *in, int i0, int lane) {
        const int p = lane & 15, kg = lane >> 4, r = g.r;
#pragma unroll
        for (int k = 0; k < R4; ++k) {
            // tall: j = 16 k + 4 kg + (0..3) of row i0 + p; wide: row j = 4 k + kg, columns i0 + 4 p + (0..3)
            const int j = TALL ? 16 * k + 4 * kg : 4 * k + kg, i = TALL ? i0 + p : i0 + 4 * p;
            x[k] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            if (j < r && i < g.D) x[k] = load_4(in + (TALL ? (int64_t)i * r + j : (int64_t)j * g.D + i));
        }
    }
    // G's value in product k: of row (tall) p or column (wide) 4 p + s of the block, and j as P's in place 4 k + kg
    __device__ __forceinline__ double value(int k, int s) const { return (double)(TALL ? x[k >> 2][k & 3] : x[k][s]); }

    template <typename E>
    __device__ __forceinline__ void store(const ortho_args &g, E *out, const double *s_p, double factor, int i0, int lane) {
        const int p = lane & 15, kg = lane >> 4, r = g.r;
#pragma unroll 1                                           // (unrolled, the wide ones spill)
        for (int c0 = 0; c0 < W; c0 += CB) {
            f64x4_t acc[CB][S];
#pragma unroll
            for (int k = 0; k < R4; ++k) asm volatile("" : "+v"(x[k]));   // widened here, not once and kept
#pragma unroll
            for (int cb = 0; cb < CB; ++cb)
#pragma unroll
                for (int s = 0; s < S; ++s) acc[cb][s] = f64x4_t{0.0, 0.0, 0.0, 0.0};
#pragma unroll
            for (int k = 0; k < 4 * W; ++k)
#pragma unroll
                for (int cb = 0; cb < CB; ++cb) {
                    // the result's row 4 e + kg is the tile's column 4 kg + e where lanes store along it (tall)
                    const int c = 16 * (c0 + cb) + (TALL ? 4 * (p & 3) + (p >> 2) : p);
                    const double a = s_p[c * LD + 4 * k + kg];
#pragma unroll
                    for (int s = 0; s < S; ++s)
                        acc[cb][s] = mfma64(a, value(k, s), acc[cb][s]);
                }
#pragma unroll
            for (int cb = 0; cb < CB; ++cb) {
                if constexpr (TALL) {
                    const int c = 16 * (c0 + cb) + 4 * kg, i = i0 + p;
                    if (c < r && i < g.D)
                        store_4(out + (int64_t)i * r + c,
                                f32x4_t{(float)(factor * acc[cb][0][0]), (float)(factor * acc[cb][0][1]),
                                        (float)(factor * acc[cb][0][2]), (float)(factor * acc[cb][0][3])});
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int c = 16 * (c0 + cb) + mfma64_row(e, lane), i = i0 + 4 * p;
                        if (c < r && i < g.D)
                            store_4(out + (int64_t)c * g.D + i,
                                    f32x4_t{(float)(factor * acc[cb][0][e]), (float)(factor * acc[cb][S > 1 ? 1 : 0][e]),
                                            (float)(factor * acc[cb][S > 2 ? 2 : 0][e]),
                                            (float)(factor * acc[cb][S > 3 ? 3 : 0][e])});
                    }
                }
            }
        }
    }
};

// bf16 products: v_mfma_f32_16x16x32_bf16 (lane l: A row and B column l % 16, k = 8 (l / 16)
// + (0..7); the result's row 4 (l / 16) + e, column l % 16).  tall: a block is 16
// rows i, and a lane reads 8 neighbouring values of one; wide: 128 columns, and a
// lane reads 8 neighbouring columns of each of 8 rows j, and exchanges rows for
// columns in its registers.
template <int W, bool TALL> struct apply_bf16 {
    static constexpr int RP = W < 2 ? 32 : 16 * W, LD = RP + 8, PART = 16 * W * LD, KT = RP / 32;
    static constexpr int CB = W < 2 ? W : 2, S = TALL ? 1 : 8;
    uint4 x[KT][S];

    __device__ __forceinline__ void load(const ortho_args &g, const uint16_t *in, int i0, int lane) {
        const int p = lane & 15, kg = lane >> 4, r = g.r;
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            if constexpr (TALL) {
                const int j = 32 * k + 8 * kg, i = i0 + p;
                x[k][0] = j < r && i < g.D ? ldg16(in + (int64_t)i * r + j) : make_uint4(0u, 0u, 0u, 0u);
            } else {
                uint32_t w[8][4];                             // rows j = 32 k + 8 kg + (0..7), columns i0 + 8 p + (0..7)
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    const int j = 32 * k + 8 * kg + h, i = i0 + 8 * p;
                    const uint4 v = j < r && i < g.D ? ldg16(in + (int64_t)j * g.D + i) : make_uint4(0u, 0u, 0u, 0u);
                    w[h][0] = v.x; w[h][1] = v.y; w[h][2] = v.z; w[h][3] = v.w;
                }
#pragma unroll
                for (int s = 0; s < 8; ++s) {                 // column s of the 8: its values of the 8 rows
                    uint32_t o[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        o[h] = __builtin_amdgcn_perm(w[2 * h + 1][s >> 1], w[2 * h][s >> 1], (s & 1) ? 0x07060302u : 0x05040100u);
                    x[k][S > 1 ? s : 0] = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        }
    }

    __device__ __forceinline__ void store(const ortho_args &g, uint16_t *out, const uint16_t *s_p, int exponent, int i0,
                                          int lane) {
        const int p = lane & 15, kg = lane >> 4, r = g.r;
        auto scaled = [&](float f) { return ldexpf(f, exponent); };
#pragma unroll 1                                           // (unrolled, the wide ones spill)
        for (int c0 = 0; c0 < W; c0 += CB) {
            f32x4_t acc[CB][S];
#pragma unroll
            for (int cb = 0; cb < CB; ++cb)
#pragma unroll
                for (int s = 0; s < S; ++s) acc[cb][s] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int cb = 0; cb < CB; ++cb)
#pragma unroll
                    for (int part = 2; part >= 0; --part) {   // the small parts first
                        const bf16x8_t a = *reinterpret_cast<const bf16x8_t *>(s_p + part * PART + (16 * (c0 + cb) + p) * LD +
                                                                               32 * k + 8 * kg);
#pragma unroll
                        for (int s = 0; s < S; ++s)
                            acc[cb][s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8_t, x[k][s]),
                                                                                 acc[cb][s], 0, 0, 0);
                    }
#pragma unroll
            for (int cb = 0; cb < CB; ++cb) {
                if constexpr (TALL) {
                    const int c = 16 * (c0 + cb) + 4 * kg, i = i0 + p;
                    if (c < r && i < g.D)
                        *reinterpret_cast<uint2 *>(out + (int64_t)i * r + c) =
                            make_uint2(pack_bf16x2(scaled(acc[cb][0][0]), scaled(acc[cb][0][1])),
                                       pack_bf16x2(scaled(acc[cb][0][2]), scaled(acc[cb][0][3])));
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int c = 16 * (c0 + cb) + 4 * kg + e, i = i0 + 8 * p;
                        if (c >= r || i >= g.D) continue;
                        float f[8];
#pragma unroll
                        for (int s = 0; s < 8; ++s) f[s] = scaled(acc[cb][S > 1 ? s : 0][e]);
                        stg16(out + (int64_t)c * g.D + i, vec16<LORA_BF16>::narrow(f));
                    }
                }
            }
        }
    }
};

// scale / (|G| + eps) = times 2^exponent.  It need not be a number of 32 bits (a zero matrix
// and a small eps: up to 2^277), nor need G P be (G of up to 2^128, P of several
// hundred): the 32-bit sums are of G and times P, whose power of two brings G near 1 as
// far as P's parts allow, and the rest of the power goes to the result.
struct split_factor {
    double times;
    int exponent;
    __device__ __forceinline__ split_factor(float scale, double inv) {
        int e, to;
        (void)frexp(inv, &to);
        const double m = frexp((double)scale * inv, &e);
        to = to < -60 ? -60 : to > 60 ? 60 : to;
        times = ldexp(m, to);
        exponent = e - to;
    }
};

// Values j, j + 1 of row c of P, pair i of the matrix, to their place in LDS.
template <bool F64, int W, bool TALL, typename V> __device__ __forceinline__ void stage_pair(char *s_p, int i, V v) {
    const int c = i / (8 * W), j = 2 * (i % (8 * W));
    if constexpr (F64) {
        double *s = reinterpret_cast<double *>(s_p) + c * (16 * W + 4);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // tall: products take j = 16 k + 4 kg + s in the order of s, then kg
            const int jj = j + h;
            s[TALL ? (jj & ~15) + 4 * (jj & 3) + ((jj >> 2) & 3) : jj] = v[h];
        }
    } else {
        constexpr int LD = (W < 2 ? 32 : 16 * W) + 8;
        // three bf16 parts carry the value to 2^-27 (a part what the ones before leave, to 2^-9)
        uint32_t o[3] = {0u, 0u, 0u};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            double rest = v[h];
#pragma unroll
            for (int part = 0; part < 3; ++part) {
                const uint32_t b = f32_to_bf16_bits((float)rest) & 0xffffu;
                o[part] |= b << (16 * h);
                rest -= (double)__uint_as_float(b << 16);
            }
        }
#pragma unroll
        for (int part = 0; part < 3; ++part)
            *reinterpret_cast<uint32_t *>(reinterpret_cast<uint16_t *>(s_p) + part * 16 * W * LD + c * LD + j) = o[part];
    }
}

// All of P, read by 256 threads.
template <bool F64, int W, bool TALL> __device__ __forceinline__ void stage_poly(char *s_p, const double *p, double times) {
    typedef double f64x2_t __attribute__((ext_vector_type(2)));
    const f64x2_t *poly = reinterpret_cast<const f64x2_t *>(p);
    constexpr int PAIRS = 128 * W * W, STEP = PAIRS < 256 ? 1 : PAIRS < 256 * 8 ? PAIRS / 256 : 8;
    for (int i = threadIdx.x; i < PAIRS; i += 256 * STEP) {
        f64x2_t v[STEP];
#pragma unroll
        for (int u = 0; u < STEP; ++u) v[u] = poly[i + 256 * u];
#pragma unroll
        for (int u = 0; u < STEP; ++u) stage_pair<F64, W, TALL>(s_p, i + 256 * u, F64 ? v[u] : v[u] * times);
    }
}

// POLY: the one tile's steps are made here, P is not in memory.  F64: 64-bit products.
template <int DT, int W, bool TALL, bool POLY, bool F64> __global__ void __launch_bounds__(256) k_ortho_apply(ortho_args g) {
    typedef typename elem<DT>::T E;
    static_assert(F64 || DT == LORA_BF16, "fp32 has 64-bit products only");
    constexpr int RP = W < 2 ? 32 : 16 * W, BLOCK = TALL ? 16 : F64 ? 64 : 128;
    __shared__ __attribute__((aligned(16))) char s_p[F64 ? 16 * W * (16 * W + 4) * 8 : 3 * 16 * W * (RP + 8) * 2];
    const int64_t item = grid_index();
    if (item >= (int64_t)g.n * g.blocks) return;
    const int64_t mat = item / g.blocks;
    const int begin = (int)(item - mat * g.blocks) * g.rows, end = min(g.D, begin + g.rows);
    const E *in = (const E *)g.g + mat * g.D * g.r;
    E *out = (E *)g.out + mat * g.D * g.r;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    typename std::conditional<F64, apply_f64<W, TALL>, apply_bf16<W, TALL>>::type block;
    int i0 = begin + wave * BLOCK;
    if (i0 < end) block.load(g, in, i0, lane);            // under way while P is staged
    double inv;
    typedef double f64x2_t __attribute__((ext_vector_type(2)));
    if (W == 1 && !F64 && threadIdx.x < 16) {             // the products' k 16..31
        uint16_t *s = reinterpret_cast<uint16_t *>(s_p) + threadIdx.x * (RP + 8) + 16;
#pragma unroll
        for (int part = 0; part < 3; ++part)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<uint4 *>(s + part * 16 * W * (RP + 8) + 8 * h) = make_uint4(0u, 0u, 0u, 0u);
    }
    if constexpr (POLY) {
        static_assert(W == 1, "one tile");
        __shared__ __attribute__((aligned(16))) double s_tile[256];
        __shared__ double s_inv;
        if (wave == 0) {
            const f64x4_t pr = poly_one(g, mat, lane, inv);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = mfma64_row(e, lane), j = lane & 15;
                s_tile[16 * i + j] = i < g.r && j < g.r ? pr[e] : 0.0;
            }
            if (lane == 0) s_inv = inv;
        }
        __syncthreads();
        inv = s_inv;
        if (threadIdx.x < 128) {
            const f64x2_t v = reinterpret_cast<const f64x2_t *>(s_tile)[threadIdx.x];
            stage_pair<F64, W, TALL>(s_p, threadIdx.x, F64 ? v : v * split_factor(g.scale, inv).times);
        }
    } else {
        inv = g.inv[mat];
        const double times = F64 ? 1.0 : split_factor(g.scale, inv).times;
        stage_poly<F64, W, TALL>(s_p, g.poly + mat * 256 * W * W, times);
    }
    __syncthreads();
    const double factor = (double)g.scale * inv;
    const int exponent = split_factor(g.scale, inv).exponent;
    for (; i0 < end; i0 += 4 * BLOCK) {
        if constexpr (F64) block.store(g, out, reinterpret_cast<const double *>(s_p), factor, i0, lane);
        else block.store(g, out, reinterpret_cast<const uint16_t *>(s_p), exponent, i0, lane);
        if (i0 + 4 * BLOCK < end) block.load(g, in, i0 + 4 * BLOCK, lane);
    }
}

// ---------------------------------------------------------------------------
// (G P)^T G P, as k_ortho_gram's sums.  A block's G P comes out of the products (A: G's
// rows i, B: P's columns) with k = i of a product for the sums where its lanes have it.
// Four wavefronts share a split's blocks; of 8 tiles a side two of them make the same G P
// and half the sums each.
// ---------------------------------------------------------------------------
template <int DT, int W, bool TALL, int HALF, int N>
__device__ __forceinline__ void regram_wave(const ortho_args &g, const typename elem<DT>::T *in, const double *s_p,
                                            int begin, int end, int stride, int lane, f64x4_t (&acc)[N]) {
    typedef apply_f64<W, TALL> A;
    constexpr int BLOCK = TALL ? 16 : 64;
    const int p = lane & 15, kg = lane >> 4;
    A block;
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = f64x4_t{0.0, 0.0, 0.0, 0.0};
    for (int i0 = begin; i0 < end; i0 += stride * BLOCK) {
        block.load(g, in, i0, lane);
#pragma unroll 1                                           // (unrolled, the wide ones spill)
        for (int s = 0; s < A::S; ++s) {
            f64x4_t y[W];                                 // element e: i = 4 e + kg, column ortho_index(c, p)
#pragma unroll
            for (int c = 0; c < W; ++c) y[c] = f64x4_t{0.0, 0.0, 0.0, 0.0};
#pragma unroll
            for (int k = 0; k < 4 * W; ++k) {
                double x = block.value(k, 0);
                if constexpr (!TALL) x = s == 0 ? x : s == 1 ? block.value(k, 1) : s == 2 ? block.value(k, 2) : block.value(k, 3);
#pragma unroll
                for (int c = 0; c < W; ++c) y[c] = mfma64(x, s_p[ortho_index<W, TALL>(c, p) * A::LD + 4 * k + kg], y[c]);
                if constexpr (W > 2) asm volatile("" ::: "memory");   // P's values are read as they are wanted (all at once, they spill)
            }
#pragma unroll
            for (int a = 0; a < W; ++a)
                if (gram_owns<W>(HALF, a))
#pragma unroll
                    for (int b = 0; b <= a; ++b)
                        acc[gram_at<W>(HALF, a, b)] = mfma64_tile(y[a], y[b], acc[gram_at<W>(HALF, a, b)]);
        }
    }
}

template <int DT, int W, bool TALL> __global__ void __launch_bounds__(256) k_ortho_regram(ortho_args g) {
    constexpr int NT = ortho_tiles(W), HALVES = W == 8 ? 2 : 1, KW = 4 / HALVES, N = NT / HALVES;
    constexpr int P_BYTES = 16 * W * apply_f64<W, TALL>::LD * 8, SUMS = (KW - 1) * NT * 64 * 32;
    __shared__ __attribute__((aligned(32))) char smem[P_BYTES > SUMS ? P_BYTES : SUMS];
    const int64_t item = grid_index();
    if (item >= (int64_t)g.n * g.splits) return;
    const int64_t mat = item / g.splits;
    const int split = (int)(item - mat * g.splits), lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int kw = wave / HALVES, half = wave % HALVES;
    const typename elem<DT>::T *in = (const typename elem<DT>::T *)g.g + mat * g.D * g.r;
    stage_poly<true, W, TALL>(smem, g.before + mat * 256 * W * W, 1.0);
    __syncthreads();
    const double *s_p = reinterpret_cast<const double *>(smem);
    // a chunk is whole blocks, but for the last of G, whose loads stop at D
    const int begin = split * g.chunk + kw * (TALL ? 16 : 64), end = min(g.D, (split + 1) * g.chunk);
    f64x4_t acc[N];
    if (half) regram_wave<DT, W, TALL, 1>(g, in, s_p, begin, end, KW, lane, acc);
    else regram_wave<DT, W, TALL, 0>(g, in, s_p, begin, end, KW, lane, acc);
    __syncthreads();                                      // P's place is the sums' now
    gram_finish<W, KW>(g, acc, reinterpret_cast<f64x4_t(*)[NT][64]>(smem), item, kw, half, lane);
}

// ---------------------------------------------------------------------------
struct ortho_layout {
    int32_t r, D, W, splits, chunk;
    size_t part, poly, join[2], inv, total;
};

static ortho_layout make_ortho_layout(int32_t n, int32_t rows, int32_t cols) {
    ortho_layout L{};
    L.r = rows < cols ? rows : cols;
    L.D = rows < cols ? cols : rows;
    L.W = L.r <= 16 ? 1 : L.r <= 32 ? 2 : L.r <= 64 ? 4 : 8;
    // about a workgroup a CU over all matrices, of at least 256 indices (two of half the
    // wavefronts: twice the sums for k_ortho_poly to read, 32 x 4096 x 16 17.6 us for 15.9)
    int splits = ceil_div(256, n > 0 ? n : 1);
    if (splits > 32) splits = 32;
    if (splits > ceil_div(L.D, 256)) splits = ceil_div(L.D, 256);
    L.chunk = ceil_div(ceil_div(L.D, splits), 64) * 64;
    L.splits = ceil_div(L.D, L.chunk);
    size_t o = 0;
    L.part = o;   o = align256(o + (size_t)n * L.splits * ortho_tiles(L.W) * 256 * 8);
    L.poly = o;   o = align256(o + (size_t)n * 256 * L.W * L.W * 8);
    for (size_t &j : L.join) {
        j = o;    o = align256(o + (size_t)n * 256 * L.W * L.W * 8);
    }
    L.inv = o;    o = align256(o + (size_t)n * 8);
    L.total = o;
    return L;
}

size_t ortho_workspace_bytes(int32_t n, int32_t rows, int32_t cols) { return make_ortho_layout(n, rows, cols).total; }

struct ortho_steps {
    const float *coef;                 // [n][3], host
    int32_t n;
    double *join[2];                   // P of several passes, in turn
};

// The steps in passes (see the top): the first step of each, and their number.
constexpr double kPassGrowth = 0x1p22, kMostGrowth = 0x1p30, kPartsMost = 0x1p11, kPartsLeast = 0x1p-20;
static int ortho_passes(const float *coef, int steps, int (&first)[kMaxOrthoSteps + 1]) {
    int n = 0;
    double growth = 1.0;                                  // the largest product of c0^2 over steps of the pass up to here
    for (int i = 0; i < steps; ++i) {
        const double c = (double)coef[3 * i] * coef[3 * i], next = growth * c;
        if (i == 0 || next > kPassGrowth) {
            first[n++] = i;
            growth = c > 1.0 ? c : 1.0;
        } else {
            growth = next > 1.0 ? next : 1.0;
        }
    }
    first[n] = steps;
    return n;
}

bool ortho_steps_ok(const float *coef, int32_t steps) {
    double growth = 1.0;
    for (int i = 0; i < steps; ++i) {
        growth *= fabs((double)coef[3 * i]);
        if (growth > kMostGrowth) return false;
        if (growth < 1.0) growth = 1.0;
    }
    return true;
}

// What no value of P passes while X is below its bound: the product of the largest |c0 + c1 m
// + c2 m^2| of each step, m the squares of the singular values, at most 1 before the first.
static double ortho_bound(const float *coef, int steps) {
    double x = 1.0, bound = 1.0;                          // x: of the singular values
    for (int i = 0; i < steps; ++i) {
        const double c0 = coef[3 * i], c1 = coef[3 * i + 1], c2 = coef[3 * i + 2], most = x * x;
        auto q = [&](double m) { return fabs(c0 + m * (c1 + m * c2)); };
        double qs = fmax(q(0.0), q(most)), xs = x * q(most);
        auto look = [&](double m, bool turn_of_q) {       // where the derivative of q, or of x q, is zero
            if (!(m > 0.0 && m < most)) return;
            if (turn_of_q) qs = fmax(qs, q(m));
            else xs = fmax(xs, sqrt(m) * q(m));
        };
        look(-c1 / (2 * c2), true);
        const double root = sqrt(9 * c1 * c1 - 20 * c0 * c2);   // c0 + 3 c1 m + 5 c2 m^2 = 0
        look((-3 * c1 + root) / (10 * c2), false);
        look((-3 * c1 - root) / (10 * c2), false);
        if (c2 == 0.0) look(-c0 / (3 * c1), false);
        bound *= qs;
        x = xs;
    }
    return bound;
}

template <int DT, int W, bool TALL, bool POLY, bool F64> static void launch_apply(ortho_args g, hipStream_t s) {
    // about three workgroups a CU (two where each makes P), of whole rounds of their wavefronts' blocks
    constexpr int ROUND = 4 * (TALL ? 16 : F64 ? 64 : 128);
    int blocks = ceil_div(W == 1 ? 512 : 768, g.n);
    if (blocks > ceil_div(g.D, ROUND)) blocks = ceil_div(g.D, ROUND);
    g.rows = ceil_div(ceil_div(g.D, blocks), ROUND) * ROUND;
    g.blocks = ceil_div(g.D, g.rows);
    hipLaunchKernelGGL((k_ortho_apply<DT, W, TALL, POLY, F64>), grid_of((int64_t)g.n * g.blocks), dim3(256), 0, s, g);
}

template <int DT, int W, bool TALL> static void launch_ortho_cfg(ortho_args &g, const ortho_steps &c, hipStream_t s) {
    int first[kMaxOrthoSteps + 1];
    const int passes = ortho_passes(c.coef, c.n, first);
    double *const own = g.poly;
    // bf16 products of P's parts where they carry it, neither large nor near the smallest
    // numbers (5 steps of 32 x 4096 x 16: 14.4 us, by 64-bit products 15.1; 8 x 64 x 14336 61 and 80)
    bool parts = false;
    if (DT == LORA_BF16 && passes == 1) {
        const double bound = ortho_bound(c.coef, c.n);
        parts = bound <= kPartsMost && bound >= kPartsLeast;
    }
    for (int i = 0; i < passes; ++i) {
        g.first = i == 0;
        g.steps = first[i + 1] - first[i];
        for (int j = 0; j < 3 * g.steps; ++j) g.coef[j / 3][j % 3] = c.coef[3 * first[i] + j];
        if (i > 0) {
            g.before = g.poly;
            g.joined = c.join[i & 1];
            g.poly = own;
            hipLaunchKernelGGL((k_ortho_regram<DT, W, TALL>), grid_of((int64_t)g.n * g.splits), dim3(256), 0, s, g);
        } else {
            if (passes > 1) g.poly = c.join[0];
            hipLaunchKernelGGL((k_ortho_gram<DT, W, TALL>), grid_of((int64_t)g.n * g.splits),
                               dim3(gram_cfg<W>::WAVES * 64), 0, s, g);
        }
        if constexpr (W == 1) {
            if constexpr (DT == LORA_BF16)
                if (parts) return launch_apply<DT, W, TALL, true, false>(g, s);
            if (passes == 1) return launch_apply<DT, W, TALL, true, true>(g, s);
            hipLaunchKernelGGL(k_ortho_poly_one<TALL>, grid_of(g.n), dim3(64), 0, s, g);
        } else if constexpr (W == 8) {
            hipLaunchKernelGGL(k_ortho_poly8<TALL>, grid_of(g.n), dim3(768), 0, s, g);
        } else {
            hipLaunchKernelGGL((k_ortho_poly<W, TALL>), grid_of(g.n), dim3(poly_cfg<W>::WAVES * 64), 0, s, g);
        }
        if (i > 0) {
            hipLaunchKernelGGL(k_ortho_join<W>, grid_of((int64_t)g.n * W * W), dim3(64), 0, s, g);
            g.poly = g.joined;
        }
    }
    if constexpr (DT == LORA_BF16 && W > 1)
        if (parts) return launch_apply<DT, W, TALL, false, false>(g, s);
    launch_apply<DT, W, TALL, false, true>(g, s);
}

template <int DT, bool TALL> static void launch_ortho_w(ortho_args &g, const ortho_steps &c, int W, hipStream_t s) {
    if (W == 1) launch_ortho_cfg<DT, 1, TALL>(g, c, s);
    else if (W == 2) launch_ortho_cfg<DT, 2, TALL>(g, c, s);
    else if (W == 4) launch_ortho_cfg<DT, 4, TALL>(g, c, s);
    else launch_ortho_cfg<DT, 8, TALL>(g, c, s);
}

lora_status_t launch_orthogonalize(const void *in, int32_t n, int32_t rows, int32_t cols, int32_t dtype,
                                   const float *coef, int32_t steps, float eps, float scale, void *out, void *ws,
                                   hipStream_t s) {
    const ortho_layout L = make_ortho_layout(n, rows, cols);
    ortho_args g{};
    g.g = in;
    g.out = out;
    g.part = ws_ptr<double>(ws, L.part);
    g.poly = ws_ptr<double>(ws, L.poly);
    g.inv = ws_ptr<double>(ws, L.inv);
    g.D = L.D;
    g.n = n;
    g.r = L.r;
    g.splits = L.splits;
    g.chunk = L.chunk;
    g.eps = eps;
    g.scale = scale;
    const ortho_steps c{coef, steps, {ws_ptr<double>(ws, L.join[0]), ws_ptr<double>(ws, L.join[1])}};
    const bool tall = rows >= cols;
    if (dtype == LORA_F32) {
        if (tall) launch_ortho_w<LORA_F32, true>(g, c, L.W, s);
        else launch_ortho_w<LORA_F32, false>(g, c, L.W, s);
    } else {
        if (tall) launch_ortho_w<LORA_BF16, true>(g, c, L.W, s);
        else launch_ortho_w<LORA_BF16, false>(g, c, L.W, s);
    }
    return hip_status(hipGetLastError());
}

}  // namespace lora
