// windows.cuh -- tiles over expert windows of ragged length, and the gated
// activation, for the experts' products (experts.cu: E4M3, dense.cu: bf16).
#pragma once

#include "moe.h"
#include "ptx.cuh"

namespace moe {

// A tile: TILE_M rows of one expert's window (from `row`, `valid` of them) by
// column tile n.
struct Tile {
    int p, n, row, valid;
};

// Tiles in the order (expert, n, rows), rows fastest: CTAs working side by
// side share a block of weights.  first_m[p] counts the row tiles before
// expert p; the expert is found by bisection from the last one on (tile indices
// only grow), not step by step: a few rows over hundreds of experts leave most
// of them empty (walking past them took 2 us of a single token's 46).
template <int TILE_M>
struct TileWalk {
    int p = 0;
    __device__ __forceinline__ Tile at(int tile, int n_tiles, const int* first_m, const int32_t* offsets,
                                       int P) {
        const int m_index = tile / n_tiles;
        if (first_m[p + 1] <= m_index) {
            int past = P;
            while (past - p > 1) {
                const int mid = (p + past) >> 1;
                if (first_m[mid] <= m_index)
                    p = mid;
                else
                    past = mid;
            }
        }
        const int m_tiles = first_m[p + 1] - first_m[p];
        const int local = tile - first_m[p] * n_tiles;
        Tile t;
        t.p = p;
        t.n = local / m_tiles;
        const int lo = offsets[p], hi = offsets[p + 1];
        t.row = lo + (local - t.n * m_tiles) * TILE_M;
        t.valid = min(TILE_M, hi - t.row);
        return t;
    }
};

// First row tile of every expert, in shared memory; returns their number.  A
// window that leaves the rows, runs backwards or starts before an earlier
// offset (it could share rows with an earlier window) counts as empty and is
// reported.  If `first` is given, the thread that holds the expert of the CTA's
// first tile leaves that tile there (the loading thread need not look it up).
// Whole CTA.
template <int THREADS, int TILE_M>
__device__ __forceinline__ int scan_windows(const int32_t* offsets, int P, int rows, int32_t* err, int* first_m,
                                            int* warp_total, int* warp_top, int n_tiles = 1, int4* first = nullptr) {
    constexpr int kWarps = THREADS / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (P + THREADS - 1) / THREADS;
    const int lo = min(P, (int)threadIdx.x * per), hi = min(P, lo + per);
    // With an expert a thread at most (P <= THREADS) its offsets are read once.
    const int a0 = lo < hi ? offsets[lo] : 0, b0 = lo < hi ? offsets[lo + 1] : 0;
    // the largest offset before this thread's first
    int top = a0;
    for (int p = lo + 1; p < hi; ++p) top = max(top, offsets[p]);
    int incl = top;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(kFull, incl, off);
        if (lane >= off) incl = max(incl, o);
    }
    if (lane == 31) warp_top[warp] = incl;
    top = __shfl_up_sync(kFull, incl, 1);
    if (lane == 0) top = 0;
    __syncthreads();
    top = max(top, __reduce_max_sync(kFull, lane < warp ? warp_top[lane] : 0));

    int sum = 0;
    for (int p = lo; p < hi; ++p) {
        const int a = p == lo ? a0 : offsets[p], b = p == lo ? b0 : offsets[p + 1];
        const bool ok = a >= top && b >= a && b <= rows;
        top = max(top, a);
        if (!ok && blockIdx.x == 0) set_error(err, MOE_DEVERR_WINDOW);
        const int m = ok ? (b - a + TILE_M - 1) / TILE_M : 0;
        first_m[p] = m;
        sum += m;
    }
    incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(kFull, incl, off);
        if (lane >= off) incl += o;
    }
    if (lane == 31) warp_total[warp] = incl;
    __syncthreads();
    const int mine = lane < kWarps ? warp_total[lane] : 0;
    const int total = __reduce_add_sync(kFull, mine);
    int run = __reduce_add_sync(kFull, lane < warp ? mine : 0) + incl - sum;
    const int m_first = (int)blockIdx.x / n_tiles;
    for (int p = lo; p < hi; ++p) {
        const int m = first_m[p];
        first_m[p] = run;
        if (first != nullptr && m_first >= run && m_first < run + m) {
            const int a = p == lo ? a0 : offsets[p], b = p == lo ? b0 : offsets[p + 1];
            const int local = (int)blockIdx.x - run * n_tiles, n = local / m, row = a + (local - n * m) * TILE_M;
            *first = make_int4(p, n, row, min(TILE_M, b - row));
        }
        run += m;
    }
    if (threadIdx.x == 0) first_m[P] = total;
    __syncthreads();
    return total;
}

// 1 / (1 + exp(-g)).  exp by 2^t with t = -g log2(e): the rounding of t makes its
// relative error |g| 2^-24, next to 2^-22 for the approximations; where |g| is
// large either exp(-g) or what it is multiplied into is negligible.  An overflow
// gives the limit 0.
__device__ __forceinline__ float sigmoid(float g) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}
__device__ __forceinline__ float gated(float g, float u) { return g * sigmoid(g) * u; }

}  // namespace moe
