// Work list of a product grouped by expert, built by every CTA for itself from the row offsets.
#pragma once

#include "experts.h"

namespace k3 {

// All threads of the CTA (a multiple of 32): s_off[0 .. E] = the offsets, s_tile[0 .. E] = exclusive
// prefix of each expert's tiles of at most `tile` rows (none for an empty expert).  Returns false,
// after recording K3MOE_ERR_RANGE, when the offsets decrease or leave [0, rows].  s_tmp: 34 ints.
template <int THREADS>
__device__ __forceinline__ bool group_tiles(const int32_t *__restrict__ offsets, int E, int rows, int tile, int *s_off,
                                            int *s_tile, int *s_tmp, int *status)
{
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
    int n = 0;
    for (int e = e0; e < e1; ++e) {
        const int c = s_off[e + 1] - s_off[e];
        bad |= c < 0;
        n += c > 0 ? (c - 1) / tile + 1 : 0;
    }
    int sum = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += v;
    }
    if (lane == 31) s_tmp[w] = sum;
    if (__syncthreads_or(bad)) {
        if (tid == 0) set_status(status, K3MOE_ERR_RANGE, -1);
        return false;
    }
    int before = sum - n;
    for (int q = 0; q < w; ++q) before += s_tmp[q];
    for (int e = e0; e < e1; ++e) {
        s_tile[e] = before;
        const int c = s_off[e + 1] - s_off[e];
        before += c > 0 ? (c - 1) / tile + 1 : 0;
    }
    if (e1 == E && (e0 < E || tid == 0)) s_tile[E] = before;     // the last thread with experts (E > 0)
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
