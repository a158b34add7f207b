// Work list of a product grouped by expert, built by every CTA for itself from the row offsets.
#pragma once

#include "experts.h"

namespace k3 {

// Rows of a tile, TILE >> i for the i < PICK with the least cost, larger first: rounds of the `pairs` workers over
// `blocks` jobs a tile, times what a stage costs a worker (256 + rows cycles, see group_tc.cu).  Returns i.
template <int TILE, int PICK>
__device__ __forceinline__ int pick_tile(const int (&tiles)[PICK], int blocks, int pairs)
{
    int best = 0;
    uint64_t cost = 0;
#pragma unroll
    for (int i = 0; i < PICK; ++i) {
        const uint64_t c = (uint64_t)(((uint32_t)tiles[i] * blocks + pairs - 1) / (uint32_t)pairs) * (256 + (TILE >> i));
        if (i == 0 || c < cost) best = i, cost = c;
    }
    return best;
}

// All threads of the CTA (a multiple of 32): s_off[0 .. E] = the offsets, s_tile[0 .. E] = exclusive
// prefix of each expert's tiles of at most TILE rows (none for an empty expert), or of the pick of PICK
// widths from TILE down.  Returns false, after recording K3MOE_ERR_RANGE, when the offsets decrease or leave
// [0, rows].  s_tmp: PICK ints a warp.  The caller keeps tiles x blocks below 2^30.
template <int THREADS, int TILE, int PICK = 1>
__device__ __forceinline__ bool group_tiles(const int32_t *__restrict__ offsets, int E, int rows, int *s_off, int *s_tile,
                                            int *s_tmp, int *status, int blocks = 1, int pairs = 1)
{
    constexpr int WARPS = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    bool bad = false;
    for (int e = tid; e <= E; e += THREADS) {
        const int o = offsets[e];
        s_off[e] = o;
        bad |= o < 0 || o > rows;
    }
    __syncthreads();
    // thread i counts the tiles of experts [i per, (i + 1) per)
    const int per = (E + THREADS - 1) / THREADS, e0 = min(E, tid * per), e1 = min(E, e0 + per);
    int n[PICK] = {};
    for (int e = e0; e < e1; ++e) {
        const int c = s_off[e + 1] - s_off[e];
        bad |= c < 0;
#pragma unroll
        for (int i = 0; i < PICK; ++i) n[i] += (int)((uint32_t)(max(c, 0) + (TILE >> i) - 1) / (TILE >> i));
    }
#pragma unroll
    for (int i = 0; i < PICK; ++i) {
        const int sum = __reduce_add_sync(0xffffffffu, n[i]);
        if (lane == 0) s_tmp[w * PICK + i] = sum;
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) set_status(status, K3MOE_ERR_RANGE, -1);
        return false;
    }
    int warp_n[PICK], all[PICK];                             // of warp `lane`; of all
#pragma unroll
    for (int i = 0; i < PICK; ++i) {
        warp_n[i] = lane < WARPS ? s_tmp[lane * PICK + i] : 0;
        all[i] = PICK > 1 ? __reduce_add_sync(0xffffffffu, warp_n[i]) : 0;
    }
    const int best = PICK > 1 ? pick_tile<TILE, PICK>(all, blocks, pairs) : 0, tile = TILE >> best;
    int mine = n[0], others = warp_n[0];
#pragma unroll
    for (int i = 1; i < PICK; ++i)
        if (i == best) mine = n[i], others = warp_n[i];
    int at = mine;                                           // exclusive prefix over the warp, after the warps before it
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, at, d);
        if (lane >= d) at += v;
    }
    at += __reduce_add_sync(0xffffffffu, lane < w ? others : 0) - mine;
    for (int e = e0; e < e1; ++e) {
        s_tile[e] = at;
        at += (s_off[e + 1] - s_off[e] + tile - 1) / tile;
    }
    if (e1 == E && (e0 < E || tid == 0)) s_tile[E] = at;     // the last thread with experts (E > 0)
    __syncthreads();
    return true;
}

// All threads of the CTA: whether the offsets are non-decreasing within [0, rows] (else K3MOE_ERR_RANGE is recorded).
template <int THREADS>
__device__ __forceinline__ bool group_offsets_ok(const int32_t *__restrict__ offsets, int E, int rows, int *status)
{
    bool bad = false;
    for (int e = threadIdx.x; e < E; e += THREADS) {
        const int a = offsets[e], b = offsets[e + 1];
        bad |= a < 0 || b < a || b > rows;
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) set_status(status, K3MOE_ERR_RANGE, -1);
        return false;
    }
    return true;
}

// The expert holding tile index t: the last e with s_tile[e] <= t (empty experts share a prefix
// value, so the last of them is the one with tiles).
__device__ __forceinline__ int group_find(const int *s_tile, int E, int t)
{
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_tile[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

}  // namespace k3
