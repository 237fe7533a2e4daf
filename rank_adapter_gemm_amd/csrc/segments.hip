// a2 -- integer segment builder: histogram -> exclusive prefix sum -> stable
// scatter of row indices -> compaction of non-empty adapter segments.
//
// It produces what the SGMV routine of "Serving multiple LoRAs: segmented
// matrix multiplies and adapter scheduling" (section "Not merging the
// weights, computing in batches") obtains with a stable argsort by adapter id
// and consecutive-unique counts, and what lora_mixed_batch in "LoRAX, in
// depth" consumes as segment boundaries plus the owner of each segment.  The
// kernels never move x or y: later kernels index rows through `perm`, the
// offsets-instead-of-gather idea of "Multi-LoRA Serving 与 Adapter 隔离"
// (adapter ownership in one continuous batch).
//
// Key of row t: ids[t] + 1 (so "no adapter" = key 0 sorts first); ids outside
// [-1, n_slots) count as key 0 and are flagged in the error word.
//
// Three launches, all integer, no floating point:
//   1. per 1024-row tile, an LDS histogram of keys -> tile_hist[key][tile]
//   2. one workgroup: exclusive scan of tile_hist in (key, tile) order, so
//      entry (key, tile) becomes the first output position of that tile's rows
//      with that key; offsets[], the GEMM order's key bases (long segments
//      first, short ones last), then the compaction of non-empty keys >= 1
//   3. per tile, each row's rank among the earlier rows of its tile with the
//      same key (stable), perm[base + rank] = t, and its place in the GEMM
//      order.
// A batch of one tile takes one launch of one workgroup (k_seg_one): all of it
// is latency (64 slots, rows at random: 1024 rows 9.7 us, 1025 in three launches 13).
#include "act_grad.hpp"

namespace lora {

// Workspace header: the error word to "none"; with `all`, every other
// header word (the segment build's) to zero as well.
__global__ void k_ws_init(int32_t *header, int32_t all) {
    const int i = threadIdx.x;
    if (i == 0) header[0] = kErrNone;
    else if (all && i < 64) header[i] = 0;
}

__device__ __forceinline__ int32_t row_key(int32_t id, int32_t n_slots) {
    return (id >= -1 && id < n_slots) ? id + 1 : 0;
}

__global__ void __launch_bounds__(256) k_seg_hist(const int32_t *__restrict__ ids, int32_t T,
                                                  int32_t n_slots, int32_t *__restrict__ tile_hist,
                                                  int32_t n_tiles, int32_t *err) {
    extern __shared__ int32_t hist[];
    const int32_t nb = n_slots + 1, tile = blockIdx.x;
    for (int32_t k = threadIdx.x; k < nb; k += blockDim.x) hist[k] = 0;
    __syncthreads();
    const int32_t t0 = tile * kSegTile;
    const int32_t t1 = min(T, t0 + kSegTile);
    for (int32_t t = t0 + threadIdx.x; t < t1; t += blockDim.x) {
        const int32_t id = ids[t];
        if (!(id >= -1 && id < n_slots)) flag_bad_row(err, t);
        atomicAdd(&hist[row_key(id, n_slots)], 1);
    }
    __syncthreads();
    for (int32_t k = threadIdx.x; k < nb; k += blockDim.x)
        tile_hist[(size_t)k * n_tiles + tile] = hist[k];
}

// Block-wide exclusive scan of one value per thread (1024 threads = 16
// waves of 64).  Returns the exclusive prefix; *total gets the block sum.
__device__ __forceinline__ int32_t block_exclusive_scan(int32_t v, int32_t *s_wave, int32_t *total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int32_t inc = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t o = __shfl_up(inc, d, 64);
        if (lane >= d) inc += o;
    }
    if (lane == 63) s_wave[wave] = inc;
    __syncthreads();
    if (wave == 0) {
        const int nw = blockDim.x >> 6;
        int32_t w = (lane < nw) ? s_wave[lane] : 0;
        int32_t winc = w;
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) {
            const int32_t o = __shfl_up(winc, d, 64);
            if (lane >= d) winc += o;
        }
        if (lane < nw) s_wave[16 + lane] = winc - w;   // exclusive wave prefix
        if (lane == nw - 1) s_wave[32] = winc;
    }
    __syncthreads();
    const int32_t res = s_wave[16 + wave] + inc - v;
    *total = s_wave[32];
    __syncthreads();
    return res;
}

// Compaction of non-empty adapter keys (k >= 1) in ascending order, and the
// grouped shrink's work table: segment i covers work blocks [blk_start[i],
// blk_start[i+1]) of kShrinkRows rows each.  s_off: the keys' first output
// positions (s_off[nb] = T), in LDS; every thread of the block calls it.
__device__ void compact_segments(const int32_t *s_off, int32_t nb, int32_t T, int32_t *s_wave,
                                 int32_t *__restrict__ seg_id, int32_t *__restrict__ seg_start,
                                 int32_t *__restrict__ n_seg, int32_t *__restrict__ blk_start,
                                 int32_t *__restrict__ blk_seg) {
    int32_t seg_carry = 0, blk_carry = 0;
    for (int32_t k0 = 1; k0 < nb; k0 += blockDim.x) {
        const int32_t k = k0 + threadIdx.x;
        const int32_t len = (k < nb) ? (s_off[k + 1] - s_off[k]) : 0;
        const int32_t nonempty = len > 0;
        const int32_t nblk = (len + kShrinkRows - 1) / kShrinkRows;
        int32_t tot, btot;
        const int32_t idx = block_exclusive_scan(nonempty, s_wave, &tot) + seg_carry;
        const int32_t bidx = block_exclusive_scan(nblk, s_wave, &btot) + blk_carry;
        if (nonempty) {
            seg_id[idx] = k - 1;
            seg_start[idx] = s_off[k];
            blk_start[idx] = bidx;
            for (int32_t b = 0; b < nblk; ++b) blk_seg[bidx + b] = idx;
        }
        seg_carry += tot;
        blk_carry += btot;
    }
    if (threadIdx.x == 0) {
        seg_start[seg_carry] = T;
        blk_start[seg_carry] = blk_carry;
        *n_seg = seg_carry;
    }
}

// The GEMM's row order: the rows of the base block and of the segments of at
// least short_len rows, in sorted order, then the rows of the shorter
// segments, in sorted order (a stable partition of perm).  gbase[k] is the
// first GEMM position of key k's rows; srec lists the short segments in
// ascending key order as {key, first GEMM position, rows, 0}, then key 0 up
// to entry min(n_slots, T) (so the per-row expand reads one record per
// item); header[kHdrNLong] is the number of rows before the short ones and
// header[kHdrNShort] the number of short segments.  Every thread of the
// block calls it.
__device__ void gemm_order(const int32_t *s_off, int32_t nb, int32_t T, int32_t short_len, int32_t *s_wave,
                           int32_t *__restrict__ gbase, int4 *__restrict__ srec, int32_t *__restrict__ header) {
    if (short_len <= 1) {                                 // no segment is short: the sorted order itself
        for (int32_t k = threadIdx.x; k < nb; k += blockDim.x) gbase[k] = s_off[k];
        for (int32_t i = threadIdx.x; i < min(nb - 1, T); i += blockDim.x) srec[i] = make_int4(0, 0, 0, 0);
        if (threadIdx.x == 0) {
            header[kHdrNLong] = T;
            header[kHdrShortLen] = short_len;
            header[kHdrNShort] = 0;
        }
        return;
    }
    int32_t n_short = 0;
    for (int32_t k0 = 0; k0 < nb; k0 += blockDim.x) {
        const int32_t k = k0 + threadIdx.x;
        const int32_t len = (k < nb) ? (s_off[k + 1] - s_off[k]) : 0;
        int32_t tot;
        block_exclusive_scan((k >= 1 && len > 0 && len < short_len) ? len : 0, s_wave, &tot);
        n_short += tot;
    }
    const int32_t n_long = T - n_short;
    int32_t long_carry = 0, short_carry = 0, seg_carry = 0;
    for (int32_t k0 = 0; k0 < nb; k0 += blockDim.x) {
        const int32_t k = k0 + threadIdx.x;
        const int32_t len = (k < nb) ? (s_off[k + 1] - s_off[k]) : 0;
        const bool is_short = k >= 1 && len > 0 && len < short_len;
        int32_t lt, st, nt;
        const int32_t lp = block_exclusive_scan(is_short ? 0 : len, s_wave, &lt) + long_carry;
        const int32_t sp = block_exclusive_scan(is_short ? len : 0, s_wave, &st) + short_carry;
        const int32_t si = block_exclusive_scan(is_short ? 1 : 0, s_wave, &nt) + seg_carry;
        if (k < nb) gbase[k] = is_short ? n_long + sp : lp;
        if (is_short) srec[si] = make_int4(k, n_long + sp, len, 0);
        long_carry += lt;
        short_carry += st;
        seg_carry += nt;
    }
    const int32_t n_rec = min(nb - 1, T);
    for (int32_t i = seg_carry + threadIdx.x; i < n_rec; i += blockDim.x) srec[i] = make_int4(0, 0, 0, 0);
    if (threadIdx.x == 0) {
        header[kHdrNLong] = n_long;
        header[kHdrShortLen] = short_len;
        header[kHdrNShort] = seg_carry;
    }
}

// Each row's rank among the earlier rows of its tile with the same key
// (stable), one row a thread of a workgroup of kSegTile: every wavefront finds
// its lanes of equal keys, then the wavefronts take their turn at the running
// counts in LDS.  count[nb]: zeroed here; holds the tile's histogram
// afterwards.  key < 0: no row.  Every thread of the block calls it.
__device__ __forceinline__ int32_t tile_rank(int32_t key, int32_t nb, int32_t *count) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int32_t k = threadIdx.x; k < nb; k += blockDim.x) count[k] = 0;
    uint64_t same = 0, pend = __ballot(key >= 0);
    while (pend) {                                        // wave-uniform: one distinct key a round
        const int32_t k = __shfl(key, __ffsll((long long)pend) - 1, 64);
        const uint64_t m = __ballot(key == k);
        if (key == k) same = m;
        pend &= ~m;
    }
    const uint64_t below = same & ((1ull << lane) - 1);
    int32_t rank = __popcll(below);
    const bool first = same && below == 0;
    __syncthreads();
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) {
        if (w == wave && same) {
            rank += count[key];
            __builtin_amdgcn_wave_barrier();              // all lanes have read before the first of a key adds
            if (first) count[key] += __popcll(same);
        }
        __syncthreads();
    }
    return rank;
}

constexpr int kScanItems = 4;

__device__ __forceinline__ void seg_scan(int32_t *s_off, int32_t *__restrict__ tile_hist, int32_t n_slots,
                                                   int32_t n_tiles, int32_t T, int32_t short_len,
                                                   int32_t *__restrict__ offsets,
                                                   int32_t *__restrict__ seg_id,
                                                   int32_t *__restrict__ seg_start,
                                                   int32_t *__restrict__ n_seg,
                                                   int32_t *__restrict__ blk_start,
                                                   int32_t *__restrict__ blk_seg,
                                                   int32_t *__restrict__ gbase,
                                                   int4 *__restrict__ srec,
                                                   int32_t *__restrict__ header) {
    __shared__ int32_t s_wave[48];            // s_off: [n_slots + 2], LDS
    const int32_t nb = n_slots + 1;
    const int64_t N = (int64_t)nb * n_tiles;
    int32_t carry = 0;
    const int64_t chunk = (int64_t)blockDim.x * kScanItems;
    for (int64_t c0 = 0; c0 < N; c0 += chunk) {
        const int64_t e0 = c0 + (int64_t)threadIdx.x * kScanItems;
        int32_t vals[kScanItems], sum = 0;
#pragma unroll
        for (int q = 0; q < kScanItems; ++q) {
            vals[q] = (e0 + q < N) ? tile_hist[e0 + q] : 0;
            sum += vals[q];
        }
        int32_t tot;
        int32_t run = block_exclusive_scan(sum, s_wave, &tot) + carry;
#pragma unroll
        for (int q = 0; q < kScanItems; ++q) {
            const int64_t e = e0 + q;
            if (e < N) {
                tile_hist[e] = run;
                if (e % n_tiles == 0) s_off[e / n_tiles] = run;   // first tile of key e / n_tiles
            }
            run += vals[q];
        }
        carry += tot;
    }
    if (threadIdx.x == 0) s_off[nb] = T;
    __syncthreads();
    for (int32_t k = threadIdx.x; k <= nb; k += blockDim.x) offsets[k] = s_off[k];

    gemm_order(s_off, nb, T, short_len, s_wave, gbase, srec, header);
    compact_segments(s_off, nb, T, s_wave, seg_id, seg_start, n_seg, blk_start, blk_seg);
}

__global__ void __launch_bounds__(1024) k_seg_scan(int32_t *__restrict__ tile_hist, int32_t n_slots,
                                                   int32_t n_tiles, int32_t T, int32_t short_len,
                                                   int32_t *__restrict__ offsets,
                                                   int32_t *__restrict__ seg_id,
                                                   int32_t *__restrict__ seg_start,
                                                   int32_t *__restrict__ n_seg,
                                                   int32_t *__restrict__ blk_start,
                                                   int32_t *__restrict__ blk_seg,
                                                   int32_t *__restrict__ gbase,
                                                   int4 *__restrict__ srec,
                                                   int32_t *__restrict__ header) {
    extern __shared__ int32_t s_off[];
    seg_scan(s_off, tile_hist, n_slots, n_tiles, T, short_len, offsets, seg_id, seg_start, n_seg, blk_start, blk_seg,
             gbase, srec, header);
}

__global__ void __launch_bounds__(1024) k_seg_scatter(const int32_t *__restrict__ ids, int32_t T,
                                                      int32_t n_slots,
                                                      const int32_t *__restrict__ tile_hist,
                                                      int32_t n_tiles, int32_t *__restrict__ perm,
                                                      const int32_t *__restrict__ offsets,
                                                      const int32_t *__restrict__ gbase,
                                                      int32_t *__restrict__ gperm) {
    extern __shared__ int32_t s_count[];
    const int32_t t = blockIdx.x * kSegTile + threadIdx.x;
    const int32_t key = t < T ? row_key(ids[t], n_slots) : -1;
    const int32_t rank = tile_rank(key, n_slots + 1, s_count);
    if (key < 0) return;
    const int32_t pos = tile_hist[(size_t)key * n_tiles + blockIdx.x] + rank;
    perm[pos] = t;
    gperm[gbase[key] + (pos - offsets[key])] = t;        // same place within its key's block
}

// Batches of one tile: everything above by one workgroup, in one launch.
__device__ __forceinline__ void seg_one(int32_t *s_off, const int32_t *__restrict__ ids, int32_t T, int32_t n_slots,
                                                  int32_t short_len, int32_t *__restrict__ offsets,
                                                  int32_t *__restrict__ seg_id, int32_t *__restrict__ seg_start,
                                                  int32_t *__restrict__ n_seg, int32_t *__restrict__ blk_start,
                                                  int32_t *__restrict__ blk_seg, int32_t *gbase,
                                                  int4 *__restrict__ srec, int32_t *__restrict__ header,
                                                  int32_t *__restrict__ perm, int32_t *__restrict__ gperm,
                                                  int32_t *err) {
    __shared__ int32_t s_wave[48];            // s_off: [n_slots + 2], LDS: counts, then first positions
    const int32_t nb = n_slots + 1, t = threadIdx.x;
    const int32_t id = t < T ? ids[t] : -1;
    const int32_t key = t < T ? row_key(id, n_slots) : -1;
    if (t < T && !(id >= -1 && id < n_slots)) flag_bad_row(err, t);
    const int32_t rank = tile_rank(key, nb, s_off);
    int32_t carry = 0;
    for (int32_t k0 = 0; k0 < nb; k0 += blockDim.x) {
        const int32_t k = k0 + threadIdx.x;
        int32_t tot;
        const int32_t pos = block_exclusive_scan(k < nb ? s_off[k] : 0, s_wave, &tot) + carry;
        if (k < nb) s_off[k] = pos;
        carry += tot;
    }
    if (threadIdx.x == 0) s_off[nb] = T;
    __syncthreads();
    for (int32_t k = threadIdx.x; k <= nb; k += blockDim.x) offsets[k] = s_off[k];
    gemm_order(s_off, nb, T, short_len, s_wave, gbase, srec, header);
    compact_segments(s_off, nb, T, s_wave, seg_id, seg_start, n_seg, blk_start, blk_seg);
    __threadfence_block();                    // gbase was written by other threads of this block
    __syncthreads();
    if (key < 0) return;
    perm[s_off[key] + rank] = t;
    gperm[gbase[key] + rank] = t;
}

__global__ void __launch_bounds__(1024) k_seg_one(const int32_t *__restrict__ ids, int32_t T, int32_t n_slots,
                                                  int32_t short_len, int32_t *__restrict__ offsets,
                                                  int32_t *__restrict__ seg_id, int32_t *__restrict__ seg_start,
                                                  int32_t *__restrict__ n_seg, int32_t *__restrict__ blk_start,
                                                  int32_t *__restrict__ blk_seg, int32_t *gbase,
                                                  int4 *__restrict__ srec, int32_t *__restrict__ header,
                                                  int32_t *__restrict__ perm, int32_t *__restrict__ gperm,
                                                  int32_t *err) {
    extern __shared__ int32_t s_off[];
    seg_one(s_off, ids, T, n_slots, short_len, offsets, seg_id, seg_start, n_seg, blk_start, blk_seg, gbase, srec,
            header, perm, gperm, err);
}

// The one workgroup of the above, and beside it the cells of act_grad, four a
// workgroup, which need the chip and no segments (777 rows, 24 adapters, 2744
// columns through tanh GELU: 10 us, one after the other 8 and 12).
struct seg_one_args {
    const int32_t *ids;
    int32_t T;
    int32_t n_slots;
    int32_t short_len;
    int32_t *offsets;
    int32_t *seg_id;
    int32_t *seg_start;
    int32_t *n_seg;
    int32_t *blk_start;
    int32_t *blk_seg;
    int32_t *gbase;
    int4 *srec;
    int32_t *header;
    int32_t *perm;
    int32_t *gperm;
    int32_t *err;
};
struct seg_scan_args {
    int32_t *tile_hist;
    int32_t n_slots;
    int32_t n_tiles;
    int32_t T;
    int32_t short_len;
    int32_t *offsets;
    int32_t *seg_id;
    int32_t *seg_start;
    int32_t *n_seg;
    int32_t *blk_start;
    int32_t *blk_seg;
    int32_t *gbase;
    int4 *srec;
    int32_t *header;
};

template <int DT, bool WRITE, bool SUMS>
__device__ __forceinline__ void act_cells(const act_grad_args &g, int cols, int block, int32_t *lds) {
    const int quarter = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8), cell = block * 4 + quarter;
    act_grad<DT, WRITE, SUMS>(g, cell % cols, cell / cols, threadIdx.x & 255,
                              reinterpret_cast<float *>(lds) + quarter * act_grad_lds<DT>());
}

template <int DT, bool WRITE, bool SUMS>
__global__ void __launch_bounds__(1024) k_seg_one_act(seg_one_args a, act_grad_args g, int32_t cols) {
    extern __shared__ __attribute__((aligned(16))) int32_t s_lds[];
    if (blockIdx.x == 0)
        seg_one(s_lds, a.ids, a.T, a.n_slots, a.short_len, a.offsets, a.seg_id, a.seg_start, a.n_seg, a.blk_start,
                a.blk_seg, a.gbase, a.srec, a.header, a.perm, a.gperm, a.err);
    else
        act_cells<DT, WRITE, SUMS>(g, cols, blockIdx.x - 1, s_lds);
}

template <int DT, bool WRITE, bool SUMS>
__global__ void __launch_bounds__(1024) k_seg_scan_act(seg_scan_args a, act_grad_args g, int32_t cols) {
    extern __shared__ __attribute__((aligned(16))) int32_t s_lds[];
    if (blockIdx.x == 0)
        seg_scan(s_lds, a.tile_hist, a.n_slots, a.n_tiles, a.T, a.short_len, a.offsets, a.seg_id, a.seg_start, a.n_seg,
                 a.blk_start, a.blk_seg, a.gbase, a.srec, a.header);
    else
        act_cells<DT, WRITE, SUMS>(g, cols, blockIdx.x - 1, s_lds);
}

template <int DT, bool WRITE, bool SUMS>
static void launch_beside(const seg_one_args *one, const seg_scan_args &scan, const act_beside &act, size_t lds,
                          hipStream_t s) {
    const int cols = act.cols();
    const int64_t cells = (int64_t)cols * act.stretches();
    const size_t need = SUMS ? 4 * 4 * (size_t)act_grad_lds<DT>() : 0;
    if (lds < need) lds = need;
    const dim3 grid((uint32_t)(1 + (cells + 3) / 4));
    if (one) hipLaunchKernelGGL((k_seg_one_act<DT, WRITE, SUMS>), grid, dim3(1024), lds, s, *one, act.args, cols);
    else hipLaunchKernelGGL((k_seg_scan_act<DT, WRITE, SUMS>), grid, dim3(1024), lds, s, scan, act.args, cols);
}

template <int DT>
static void launch_beside_dt(const seg_one_args *one, const seg_scan_args &scan, const act_beside &act, size_t lds,
                             hipStream_t s) {
    if (act.write && act.sums) launch_beside<DT, true, true>(one, scan, act, lds, s);
    else if (act.write) launch_beside<DT, true, false>(one, scan, act, lds, s);
    else launch_beside<DT, false, true>(one, scan, act, lds, s);
}

lora_status_t launch_ws_init(void *ws, hipStream_t s, bool err_only) {
    hipLaunchKernelGGL(k_ws_init, dim3(1), dim3(64), 0, s, ws_ptr<int32_t>(ws, 0), err_only ? 0 : 1);
    return hip_status(hipGetLastError());
}

lora_status_t launch_segments(const int32_t *ids, int32_t T, int32_t n_slots, const ws_layout &L,
                              void *ws, hipStream_t s, int32_t short_len, const act_beside *act) {
    if (short_len < 1) short_len = 1;
    const int32_t n_tiles = (T + kSegTile - 1) / kSegTile;
    int32_t *err = ws_ptr<int32_t>(ws, L.header);
    int32_t *tile_hist = ws_ptr<int32_t>(ws, L.tile_hist);
    const size_t lds_hist = sizeof(int32_t) * (size_t)(n_slots + 1);
    const size_t lds_off = sizeof(int32_t) * (size_t)(n_slots + 2);
    const seg_scan_args scan{tile_hist, n_slots, n_tiles, T, short_len,
                       ws_ptr<int32_t>(ws, L.offsets), ws_ptr<int32_t>(ws, L.seg_id),
                       ws_ptr<int32_t>(ws, L.seg_start), ws_ptr<int32_t>(ws, L.n_seg),
                       ws_ptr<int32_t>(ws, L.blk_start), ws_ptr<int32_t>(ws, L.blk_seg),
                       ws_ptr<int32_t>(ws, L.gbase), ws_ptr<int4>(ws, L.srec), ws_ptr<int32_t>(ws, L.header)};
    auto beside = [&](const seg_one_args *one) {
        if (act->dtype == LORA_F32) launch_beside_dt<LORA_F32>(one, scan, *act, lds_off, s);
        else launch_beside_dt<LORA_BF16>(one, scan, *act, lds_off, s);
    };
    if (n_tiles == 1) {
        if (act) {
            const seg_one_args one{ids, T, n_slots, short_len,
                           ws_ptr<int32_t>(ws, L.offsets), ws_ptr<int32_t>(ws, L.seg_id),
                           ws_ptr<int32_t>(ws, L.seg_start), ws_ptr<int32_t>(ws, L.n_seg),
                           ws_ptr<int32_t>(ws, L.blk_start), ws_ptr<int32_t>(ws, L.blk_seg),
                           ws_ptr<int32_t>(ws, L.gbase), ws_ptr<int4>(ws, L.srec), ws_ptr<int32_t>(ws, L.header),
                           ws_ptr<int32_t>(ws, L.perm), ws_ptr<int32_t>(ws, L.gperm), err};
            beside(&one);
            return hip_status(hipGetLastError());
        }
        hipLaunchKernelGGL(k_seg_one, dim3(1), dim3(kSegTile), lds_off, s, ids, T, n_slots, short_len,
                           ws_ptr<int32_t>(ws, L.offsets), ws_ptr<int32_t>(ws, L.seg_id),
                           ws_ptr<int32_t>(ws, L.seg_start), ws_ptr<int32_t>(ws, L.n_seg),
                           ws_ptr<int32_t>(ws, L.blk_start), ws_ptr<int32_t>(ws, L.blk_seg),
                           ws_ptr<int32_t>(ws, L.gbase), ws_ptr<int4>(ws, L.srec), ws_ptr<int32_t>(ws, L.header),
                           ws_ptr<int32_t>(ws, L.perm), ws_ptr<int32_t>(ws, L.gperm), err);
        return hip_status(hipGetLastError());
    }
    hipLaunchKernelGGL(k_seg_hist, dim3(n_tiles), dim3(256), lds_hist, s, ids, T, n_slots,
                       tile_hist, n_tiles, err);
    if (act) beside(nullptr);
    else
        hipLaunchKernelGGL(k_seg_scan, dim3(1), dim3(1024), lds_off, s, tile_hist, n_slots, n_tiles, T, short_len,
                           ws_ptr<int32_t>(ws, L.offsets), ws_ptr<int32_t>(ws, L.seg_id),
                           ws_ptr<int32_t>(ws, L.seg_start), ws_ptr<int32_t>(ws, L.n_seg),
                           ws_ptr<int32_t>(ws, L.blk_start), ws_ptr<int32_t>(ws, L.blk_seg),
                           ws_ptr<int32_t>(ws, L.gbase), ws_ptr<int4>(ws, L.srec), ws_ptr<int32_t>(ws, L.header));
    hipLaunchKernelGGL(k_seg_scatter, dim3(n_tiles), dim3(kSegTile), lds_hist, s, ids, T, n_slots,
                       tile_hist, n_tiles, ws_ptr<int32_t>(ws, L.perm), ws_ptr<int32_t>(ws, L.offsets),
                       ws_ptr<int32_t>(ws, L.gbase), ws_ptr<int32_t>(ws, L.gperm));
    return hip_status(hipGetLastError());
}

}  // namespace lora
