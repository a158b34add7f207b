// Rows in expert order: the plan of a routing's pairs, the copy of the tokens' rows into it, the
// weighted sum back to tokens and that sum's gradient (k3moe_rows_*).  All are bound by HBM (or by
// launch latency at decode sizes): every byte is read or written once.
#include "experts.h"

namespace k3 {

// ------------------------------------------------------------------ plan
// Pairs p = t K + k in blocks of `per` pairs.  Their expert counts per block come first (one launch,
// skipped for a single block); then each block sums the counts of all blocks to the experts' offsets
// and its own first row of each expert, and numbers its pairs in order, PLAN_SUB at a time: each of
// the 32 warps numbers 64 consecutive pairs against its own counters, in two rounds of 32 in which
// lanes of the same expert find each other by match_any, and a scan over the warps' counters joins
// them.  Order is by pair alone, no atomics decide it.  Bound by latency: 16 x 16 pairs over 896 experts
// 4.2 us (one launch), 8192 x 16 pairs 10.2 us.
constexpr int PLAN_THREADS = 1024, PLAN_SUB = 2048, PLAN_BLOCKS = 128;

__device__ __forceinline__ int plan_expert(const int32_t *idx, int64_t p, int64_t n, int first, int E)
{
    if (p >= n) return -1;
    const uint32_t e = (uint32_t)idx[p] - (uint32_t)first;
    return e < (uint32_t)E ? (int)e : -1;
}

__global__ void __launch_bounds__(PLAN_THREADS) plan_count_kernel(const int32_t *__restrict__ idx, int64_t n, int64_t per,
                                                                  int first, int E, int32_t *__restrict__ counts)
{
    griddep_enter();
    __shared__ int hist[K3MOE_TRAIN_MAX_EXPERTS];
    const int tid = threadIdx.x;
    if (tid < E) hist[tid] = 0;
    __syncthreads();
    const int64_t p1 = min(n, (int64_t)(blockIdx.x + 1) * per);
    for (int64_t p = (int64_t)blockIdx.x * per + tid; p < p1; p += PLAN_THREADS) {
        const int e = plan_expert(idx, p, n, first, E);
        if (e >= 0) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    if (tid < E) counts[(size_t)blockIdx.x * E + tid] = hist[tid];
}

// counts NULL: one block, which counts its own pairs.
__global__ void __launch_bounds__(PLAN_THREADS) plan_place_kernel(const int32_t *__restrict__ idx, int64_t n, int64_t per,
                                                                  int first, int E,
                                                                  const int32_t *__restrict__ counts,
                                                                  int32_t *__restrict__ offsets,
                                                                  int32_t *__restrict__ pos)
{
    griddep_enter();
    extern __shared__ uint16_t whist[];                     // [32][E]
    __shared__ int base[K3MOE_TRAIN_MAX_EXPERTS], wsum[32];
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, nb = gridDim.x, b = blockIdx.x;
    int total = 0, before = 0;
    if (counts) {
        if (tid < E) {
#pragma unroll 8
            for (int q = 0; q < nb; ++q) {
                const int c = __ldg(counts + (size_t)q * E + tid);
                total += c;
                before += q < b ? c : 0;
            }
        }
    } else {
        if (tid < E) base[tid] = 0;
        __syncthreads();
        for (int64_t p = tid; p < n; p += PLAN_THREADS) {
            const int e = plan_expert(idx, p, n, first, E);
            if (e >= 0) atomicAdd(&base[e], 1);
        }
        __syncthreads();
        if (tid < E) total = base[tid];
        __syncthreads();
    }
    int sum = total;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += v;
    }
    if (lane == 31) wsum[w] = sum;
    __syncthreads();
    if (w == 0) {
        int v = wsum[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += u;
        }
        wsum[lane] = v;
    }
    __syncthreads();
    sum += w ? wsum[w - 1] : 0;
    if (tid < E) {
        base[tid] = sum - total + before;
        if (b == 0) {
            offsets[tid] = sum - total;
            if (tid == E - 1) offsets[E] = sum;
        }
    }
    const int64_t p1 = min(n, (int64_t)(b + 1) * per);
    uint16_t *mine = whist + w * E;
    for (int64_t s0 = (int64_t)b * per; s0 < p1; s0 += PLAN_SUB) {
        for (int i = tid; i < 32 * E; i += PLAN_THREADS) whist[i] = 0;
        __syncthreads();
        int e[2], rank[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            e[r] = plan_expert(idx, s0 + w * 64 + r * 32 + lane, p1, first, E);
            const uint32_t same = __match_any_sync(0xffffffffu, e[r]);
            rank[r] = e[r] >= 0 ? mine[e[r]] + __popc(same & ((1u << lane) - 1u)) : 0;
            __syncwarp();
            if (e[r] >= 0 && (same >> lane) == 1u) mine[e[r]] = (uint16_t)(rank[r] + 1);    // the last of its expert
            __syncwarp();
        }
        __syncthreads();
        int in_sub = 0;                                      // pairs of expert tid in this sub-block
        if (tid < E) {
#pragma unroll 8
            for (int q = 0; q < 32; ++q) {
                const int c = whist[q * E + tid];
                whist[q * E + tid] = (uint16_t)in_sub;
                in_sub += c;
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int64_t p = s0 + w * 64 + r * 32 + lane;
            if (p < p1) pos[p] = e[r] >= 0 ? base[e[r]] + mine[e[r]] + rank[r] : -1;
        }
        __syncthreads();
        if (tid < E) base[tid] += in_sub;
        // the next round's first barrier orders this before base is read again
    }
}

// ------------------------------------------------------------------ gather
// A CTA per token reads its row once and writes its K copies.  HBM writes bind it: 4096 x 16 rows of 3584
// bf16 take 79 us, 6.3 TB/s.
template <class T, int V>
__global__ void __launch_bounds__(256) rows_gather_kernel(const T *__restrict__ x, int64_t ldx,
                                                          const int32_t *__restrict__ pos, int T_, int K, int nv,
                                                          T *__restrict__ out, int64_t ldo, int n_rows, int *status)
{
    griddep_enter();
    // blockIdx.y: a share of the token's K copies, so that few tokens still fill the GPU
    const int k0 = (int)((long long)blockIdx.y * K / gridDim.y), k1 = (int)((long long)(blockIdx.y + 1) * K / gridDim.y);
    for (int t = blockIdx.x; t < T_; t += gridDim.x) {
        const int32_t *row = pos + (int64_t)t * K;
        for (int i = threadIdx.x; i < nv; i += blockDim.x) {
            const Vec<T, V> v = *reinterpret_cast<const Vec<T, V> *>(x + t * ldx + (int64_t)i * V);
#pragma unroll 4
            for (int k = k0; k < k1; ++k) {
                const int r = __ldg(row + k);
                if (r >= 0 && r < n_rows)
                    *reinterpret_cast<Vec<T, V> *>(out + r * ldo + (int64_t)i * V) = v;
                else if (r >= n_rows && i == 0)
                    set_status(status, K3MOE_ERR_RANGE, r);
            }
        }
    }
}

// ------------------------------------------------------------------ combine
// `split` warps per token, each with every split-th piece of 32 V columns, so that nothing but memory keeps a
// warp waiting: its lanes hold the token's rows and weights (32 at a time), and only rows that exist are
// loaded, eight in flight, summed in k order.  Reads of 512 bytes here and there bind it: 4096 x 16 rows of
// 3584 in 82 us, 6.1 TB/s (half of them missing 48 us, 5.5 TB/s); 16 tokens 3.2 us.
template <class T, int V>
__global__ void __launch_bounds__(256, 4) rows_combine_kernel(const T *__restrict__ y, int64_t ldy, int n_rows,
                                                           const int32_t *__restrict__ pos,
                                                           const float *__restrict__ wts, int T_, int K, int nv,
                                                           int split, T *__restrict__ z, int64_t ldz, int *status)
{
    griddep_enter();
    const int lane = threadIdx.x & 31;
    const int64_t work = (int64_t)T_ * split, step = (int64_t)gridDim.x * 8;
    for (int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); u < work; u += step) {
        const int t = (int)(u / split), first = (int)(u - (int64_t)t * split);
        int row = -1;
        float w = 0.f;
        auto table = [&](int kb) {
            row = -1;
            w = 0.f;
            if (kb + lane < K) {
                row = __ldg(pos + (int64_t)t * K + kb + lane);
                w = wts ? __ldg(wts + (int64_t)t * K + kb + lane) : 1.0f;
                if (row >= n_rows) {
                    set_status(status, K3MOE_ERR_RANGE, row);
                    row = -1;
                }
            }
        };
        table(0);
        for (int i = first * 32 + lane; i - lane < nv; i += split * 32) {
            const bool in = i < nv;
            float acc[V + (V == 1)] = {};
            for (int kb = 0; kb < K; kb += 32) {
                if (K > 32) table(kb);
                uint32_t live = __ballot_sync(0xffffffffu, row >= 0);
                while (live) {
                    Vec<T, V> v[8];
                    float f[8];
                    const int n = __popc(live);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int k = max(__ffs(live) - 1, 0);
                        live &= live - 1;
                        const int r = __shfl_sync(0xffffffffu, row, k);
                        f[j] = __shfl_sync(0xffffffffu, w, k);
                        if (in && j < n) v[j] = *reinterpret_cast<const Vec<T, V> *>(y + r * ldy + (int64_t)i * V);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < n && in)
#pragma unroll
                            for (int q = 0; q < V; q += 2) {
                                const float2 d = v[j].get2(q);
                                acc[q] = fmaf(f[j], d.x, acc[q]);
                                if (V > 1) acc[q + 1] = fmaf(f[j], d.y, acc[q + 1]);
                            }
                }
            }
            if (in) {
                Vec<T, V> o;
#pragma unroll
                for (int q = 0; q < V; q += 2) o.set2(q, acc[q], acc[q + 1]);
                *reinterpret_cast<Vec<T, V> *>(z + t * ldz + (int64_t)i * V) = o;
            }
        }
    }
}

// ------------------------------------------------------------------ combine's gradient
// Sums of eight values over the warp in nine shuffles: each of the first three steps halves the values a
// lane still holds.  Lane l ends with value l / 4 in v[0].
__device__ __forceinline__ void warp_sum8(float (&v)[8], int lane)
{
#pragma unroll
    for (int n = 4, d = 16; n > 0; n >>= 1, d >>= 1) {
        const bool up = lane & d;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < n) {
                const float give = up ? v[j] : v[j + n], keep = up ? v[j + n] : v[j];
                v[j] = keep + __shfl_xor_sync(0xffffffffu, give, d);
            }
    }
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
}

// CTA per token and eight pairs (or all its pairs, eight at a time): dz's row, the pairs' y rows read and
// their dy rows written (in that order by the same thread, so dy may be y), dot products summed per thread, warp and CTA in fixed order.  HBM
// binds it: 4096 x 16 rows of 3584 bf16 in 148 us, 6.5 TB/s.
template <class T, int V>
__global__ void __launch_bounds__(256, 3) rows_combine_grad_kernel(const T *__restrict__ dz, int64_t lddz, const T *y,
                                                                int64_t ldy, int n_rows,
                                                                const int32_t *__restrict__ pos,
                                                                const float *__restrict__ wts, int T_, int K, int nv,
                                                                T *dy, int64_t lddy, float *__restrict__ dw,
                                                                int *status)
{
    griddep_enter();
    __shared__ float part[8][8];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
    for (int t = blockIdx.x; t < T_; t += gridDim.x) {
        for (int kb = 8 * blockIdx.y; kb < K; kb += 8 * gridDim.y) {
            int r[8];
            float wt[8], acc[8] = {};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool in = kb + j < K;
                r[j] = in ? __ldg(pos + (int64_t)t * K + kb + j) : -1;
                wt[j] = in ? __ldg(wts + (int64_t)t * K + kb + j) : 0.f;
                if (r[j] >= n_rows) {
                    if (threadIdx.x == 0) set_status(status, K3MOE_ERR_RANGE, r[j]);
                    r[j] = -1;
                }
            }
            for (int i = threadIdx.x; i < nv; i += blockDim.x) {
                const Vec<T, V> d = *reinterpret_cast<const Vec<T, V> *>(dz + t * lddz + (int64_t)i * V);
                Vec<T, V> v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (r[j] >= 0) v[j] = *reinterpret_cast<const Vec<T, V> *>(y + r[j] * ldy + (int64_t)i * V);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (r[j] >= 0) {
                        Vec<T, V> o;
#pragma unroll
                        for (int q = 0; q < V; q += 2) {
                            const float2 f = d.get2(q), g = v[j].get2(q);
                            acc[j] = fmaf(f.y, g.y, fmaf(f.x, g.x, acc[j]));
                            o.set2(q, wt[j] * f.x, wt[j] * f.y);
                        }
                        *reinterpret_cast<Vec<T, V> *>(dy + r[j] * lddy + (int64_t)i * V) = o;
                    }
            }
            warp_sum8(acc, lane);
            if ((lane & 3) == 0) part[w][lane >> 2] = acc[0];
            __syncthreads();
            if (threadIdx.x < 8 && kb + threadIdx.x < K) {
                float s = 0.f;
                for (int q = 0; q < nw; ++q) s += part[q][threadIdx.x];
                dw[(int64_t)t * K + kb + threadIdx.x] = s;
            }
            __syncthreads();
        }
    }
}

// Threads for nv pieces a row: whole warps, at most 256, as few idle ones in the last pass as possible.
static int row_threads(int nv)
{
    const int passes = (nv + 255) / 256;
    return ((nv + passes - 1) / passes + 31) / 32 * 32;
}

}  // namespace k3

using namespace k3;

static int64_t plan_per(int64_t n)
{
    const int64_t per = (n + PLAN_BLOCKS - 1) / PLAN_BLOCKS;
    return per <= PLAN_SUB ? PLAN_SUB : (per + PLAN_SUB - 1) / PLAN_SUB * PLAN_SUB;
}

static bool plan_sizes_ok(int T, int K, int E)
{
    return T >= 0 && K >= 1 && E >= 1 && (int64_t)T * K < (1LL << 31);
}

extern "C" size_t k3moe_rows_plan_workspace_bytes(int T, int K, int n_experts)
{
    if (!plan_sizes_ok(T, K, n_experts) || n_experts > K3MOE_TRAIN_MAX_EXPERTS) return 0;
    const int64_t n = (int64_t)T * K, blocks = (n + plan_per(n) - 1) / plan_per(n);
    return 256 + sizeof(int32_t) * (size_t)blocks * n_experts;
}

extern "C" int k3moe_rows_plan(const int32_t *idx, int T, int K, int first_expert, int n_experts, int32_t *offsets,
                               int32_t *pos, void *workspace, size_t workspace_bytes, cudaStream_t st)
{
    if (!plan_sizes_ok(T, K, n_experts) || !offsets || (T > 0 && (!idx || !pos))) return K3MOE_ERR_ARG;
    if (first_expert < 0 || (int64_t)first_expert + n_experts > (1LL << 31) - 1) return K3MOE_ERR_ARG;
    if (n_experts > K3MOE_TRAIN_MAX_EXPERTS) return K3MOE_ERR_SHAPE;
    if (!workspace || workspace_bytes < k3moe_rows_plan_workspace_bytes(T, K, n_experts)) return K3MOE_ERR_WORKSPACE;
    if ((uintptr_t)workspace & 3) return K3MOE_ERR_ALIGN;
    const int64_t n = (int64_t)T * K, per = plan_per(n);
    const size_t nb = (size_t)n * 4, no = sizeof(int32_t) * ((size_t)n_experts + 1);
    const size_t nw = k3moe_rows_plan_workspace_bytes(T, K, n_experts);
    if (k3_overlap(idx, nb, pos, nb) || k3_overlap(idx, nb, offsets, no) || k3_overlap(pos, nb, offsets, no) ||
        k3_overlap(workspace, nw, idx, nb) || k3_overlap(workspace, nw, pos, nb) || k3_overlap(workspace, nw, offsets, no))
        return K3MOE_ERR_ALIAS;
    if (!k3_aligned({{idx, 4}, {offsets, 4}, {pos, 4}})) return K3MOE_ERR_ALIGN;
    const int blocks = n > 0 ? (int)((n + per - 1) / per) : 1;
    int32_t *counts = blocks > 1 ? static_cast<int32_t *>(workspace) : nullptr;
    static unsigned long long attr_set = 0;
    if (!k3_smem_attr(plan_place_kernel, 32 * K3MOE_TRAIN_MAX_EXPERTS * 2, attr_set)) return K3MOE_ERR_CUDA;
    if (counts) {
        k3_launch(plan_count_kernel, blocks, PLAN_THREADS, 0, st, idx, n, per, first_expert, n_experts, counts);
        k3_note_launch();
    }
    k3_launch(plan_place_kernel, blocks, PLAN_THREADS, (size_t)32 * n_experts * 2, st, idx, n, per, first_expert,
              n_experts, (const int32_t *)counts, offsets, pos);
    k3_note_launch();
    return cudaGetLastError() == cudaSuccess ? K3MOE_OK : K3MOE_ERR_CUDA;
}

static int rows_check(int T, int K, int D, int dtype, int n_rows)
{
    if (T < 0 || K < 1 || D < 1 || n_rows < 0 || (int64_t)T * K >= (1LL << 31)) return K3MOE_ERR_ARG;
    if (dtype != K3MOE_TYPE_BF16 && dtype != K3MOE_TYPE_F16) return K3MOE_ERR_UNSUPPORTED;
    return K3MOE_OK;
}

// 8 elements an access where all rows start on 16-byte boundaries and D is a multiple of 8, else one
template <class F>
static void with_types(int dtype, bool vec, F f)
{
    if (dtype == K3MOE_TYPE_BF16) {
        if (vec) f(__nv_bfloat16(), std::integral_constant<int, 8>());
        else f(__nv_bfloat16(), std::integral_constant<int, 1>());
    } else {
        if (vec) f(__half(), std::integral_constant<int, 8>());
        else f(__half(), std::integral_constant<int, 1>());
    }
}

extern "C" int k3moe_rows_gather(const void *x, int64_t ldx, const int32_t *pos, int T, int K, int D, int dtype,
                                 void *out, int64_t ldo, int n_rows, int32_t *status, cudaStream_t st)
{
    const int rc = rows_check(T, K, D, dtype, n_rows);
    if (rc) return rc;
    if (T > 0 && (!x || !pos || !status || (n_rows > 0 && !out))) return K3MOE_ERR_ARG;
    if (ldx < D || ldo < D) return K3MOE_ERR_ARG;
    const size_t no = k3_span(n_rows, D, ldo, dtype);
    if (k3_overlap(out, no, x, k3_span(T, D, ldx, dtype)) || k3_overlap(out, no, pos, (size_t)T * K * 4)) return K3MOE_ERR_ALIAS;
    if (!k3_aligned({{x, 2}, {out, 2}, {pos, 4}, {status, 4}})) return K3MOE_ERR_ALIGN;
    if (T == 0) return K3MOE_OK;
    const int sms = k3_num_sms();
    if (!sms) return K3MOE_ERR_CUDA;
    const bool vec = D % 8 == 0 && k3_rows16(x, ldx, dtype) && k3_rows16(out, ldo, dtype);
    with_types(dtype, vec, [&](auto t, auto v) {
        using Ty = decltype(t);
        constexpr int V = decltype(v)::value;
        const int nv = D / V, ky = T >= 4 * sms ? 1 : (int)std::min<int64_t>(K, (4 * sms + T - 1) / T);
        k3_launch(rows_gather_kernel<Ty, V>, dim3(T, ky), row_threads(nv), 0, st, (const Ty *)x, ldx, pos, T, K, nv,
                  (Ty *)out, ldo, n_rows, status);
    });
    k3_note_launch();
    return cudaGetLastError() == cudaSuccess ? K3MOE_OK : K3MOE_ERR_CUDA;
}

extern "C" int k3moe_rows_combine(const void *y, int64_t ldy, int n_rows, const int32_t *pos, const float *weights,
                                  int T, int K, int D, int dtype, void *z, int64_t ldz, int32_t *status,
                                  cudaStream_t st)
{
    const int rc = rows_check(T, K, D, dtype, n_rows);
    if (rc) return rc;
    if (T > 0 && (!z || !pos || !status || (n_rows > 0 && !y))) return K3MOE_ERR_ARG;
    if (ldy < D || ldz < D) return K3MOE_ERR_ARG;
    const size_t nz = k3_span(T, D, ldz, dtype), nt = (size_t)T * K * 4;
    if (k3_overlap(z, nz, y, k3_span(n_rows, D, ldy, dtype)) || k3_overlap(z, nz, pos, nt) || k3_overlap(z, nz, weights, weights ? nt : 0))
        return K3MOE_ERR_ALIAS;
    if (!k3_aligned({{y, 2}, {z, 2}, {pos, 4}, {weights, 4}, {status, 4}})) return K3MOE_ERR_ALIGN;
    if (T == 0) return K3MOE_OK;
    const int sms = k3_num_sms();
    if (!sms) return K3MOE_ERR_CUDA;
    const bool vec = D % 8 == 0 && k3_rows16(y, ldy, dtype) && k3_rows16(z, ldz, dtype);
    with_types(dtype, vec, [&](auto t, auto v) {
        using Ty = decltype(t);
        constexpr int V = decltype(v)::value;
        const int nv = D / V;
        // about four rounds of the 32 or so warps an SM holds (with one round 4096 tokens took 8 % longer)
        const int pieces = (nv + 31) / 32, split = (int)std::min<int64_t>(pieces, (128LL * sms + T - 1) / T);
        k3_launch(rows_combine_kernel<Ty, V>, (unsigned)std::min<int64_t>(((int64_t)T * split + 7) / 8, 1 << 20), 256, 0,
                  st, (const Ty *)y, ldy, n_rows, pos, weights, T, K, nv, split, (Ty *)z, ldz, status);
    });
    k3_note_launch();
    return cudaGetLastError() == cudaSuccess ? K3MOE_OK : K3MOE_ERR_CUDA;
}

extern "C" int k3moe_rows_combine_grad(const void *dz, int64_t lddz, const void *y, int64_t ldy, int n_rows,
                                       const int32_t *pos, const float *weights, int T, int K, int D, int dtype,
                                       void *dy, int64_t lddy, float *dweights, int32_t *status, cudaStream_t st)
{
    const int rc = rows_check(T, K, D, dtype, n_rows);
    if (rc) return rc;
    if (T > 0 && (!dz || !pos || !weights || !dweights || !status || (n_rows > 0 && (!y || !dy)))) return K3MOE_ERR_ARG;
    if (lddz < D || ldy < D || lddy < D) return K3MOE_ERR_ARG;
    const size_t ndy = k3_span(n_rows, D, lddy, dtype), ny = k3_span(n_rows, D, ldy, dtype), nz = k3_span(T, D, lddz, dtype);
    const size_t nt = (size_t)T * K * 4;
    const bool in_place = dy == y && lddy == ldy;
    if (k3_overlap(dy, ndy, dz, nz) || (!in_place && k3_overlap(dy, ndy, y, ny)) || k3_overlap(dy, ndy, pos, nt) ||
        k3_overlap(dy, ndy, weights, nt) || k3_overlap(dweights, nt, dy, ndy) || k3_overlap(dweights, nt, dz, nz) ||
        k3_overlap(dweights, nt, y, ny) || k3_overlap(dweights, nt, pos, nt) || k3_overlap(dweights, nt, weights, nt))
        return K3MOE_ERR_ALIAS;
    if (!k3_aligned({{dz, 2}, {y, 2}, {dy, 2}, {pos, 4}, {weights, 4}, {dweights, 4}, {status, 4}})) return K3MOE_ERR_ALIGN;
    if (T == 0) return K3MOE_OK;
    const bool vec = D % 8 == 0 && k3_rows16(dz, lddz, dtype) && k3_rows16(y, ldy, dtype) && k3_rows16(dy, lddy, dtype);
    with_types(dtype, vec, [&](auto t, auto v) {
        using Ty = decltype(t);
        constexpr int V = decltype(v)::value;
        // few tokens: a CTA for every eight pairs (16 tokens 7.0 -> 4.0 us); many: one for all of a token's
        // (4096 tokens: 7 % less; three CTAs an SM by registers: 13 % less than two)
        const int nv = D / V, ky = T < 4 * k3_num_sms() ? std::min(65535, (K + 7) / 8) : 1;
        k3_launch(rows_combine_grad_kernel<Ty, V>, dim3(T, ky), row_threads(nv), 0, st, (const Ty *)dz, lddz, (const Ty *)y, ldy,
                  n_rows, pos, weights, T, K, nv, (Ty *)dy, lddy, dweights, status);
    });
    k3_note_launch();
    return cudaGetLastError() == cudaSuccess ? K3MOE_OK : K3MOE_ERR_CUDA;
}
