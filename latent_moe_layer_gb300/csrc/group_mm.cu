// Products grouped by expert (k3moe_group_mm, _grad_x, _grad_w): argument checks, and the CUDA-core
// kernel of shapes and strides that the tensor-core kernels cannot take.
#include "experts.h"
#include "group_sched.cuh"

namespace k3 {

constexpr int GG_TILE = 64, GG_K = 16, GG_THREADS = 256;

// 64 x 64 outputs per CTA, 4 x 4 per thread, contraction in steps of 16 through shared memory, fp32
// sums in contraction order.  Any size, stride and alignment, at 19 TFLOP/s (65,536 rows, 3584 to 6144: shared
// memory and FMA issue bind it; the tensor-core kernels take 1.7 ms there, this one 152).  Tile rows m run over the output's
// contiguous axis for mm and grad_x (m = n_out / n_in index, columns = rows of x), and over n_out for
// grad_w (columns = n_in).
template <int MODE, class T, class O>
__global__ void __launch_bounds__(GG_THREADS) group_generic_kernel(const K3Group g)
{
    griddep_enter();
    __shared__ float sa[GG_K][GG_TILE + 1], sb[GG_K][GG_TILE + 1];
    __shared__ int s_off[K3MOE_TRAIN_MAX_EXPERTS + 1], s_tile[K3MOE_TRAIN_MAX_EXPERTS + 1], s_tmp[GG_THREADS / 32];
    if (!group_tiles<GG_THREADS, GG_TILE>(g.offsets, g.E, g.rows, s_off, s_tile, s_tmp, g.status)) return;
    const T *A = static_cast<const T *>(g.a), *B = static_cast<const T *>(g.b);
    O *out = static_cast<O *>(g.out);
    const int M = MODE == K3_GROUP_GRAD_X ? g.n_in : g.n_out;            // tile rows
    const int m_blocks = (M + GG_TILE - 1) / GG_TILE;
    const int c_blocks = MODE == K3_GROUP_GRAD_W ? (g.n_in + GG_TILE - 1) / GG_TILE : 1;
    const long long jobs = MODE == K3_GROUP_GRAD_W ? (long long)g.E * m_blocks * c_blocks
                                                   : (long long)s_tile[g.E] * m_blocks;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (long long job = blockIdx.x; job < jobs; job += gridDim.x) {
        const int m0 = (int)(job % m_blocks) * GG_TILE;
        int e, c0, c1, k1;                       // columns [c0, c1), contraction [0, k1)
        long long r0 = 0;
        if (MODE == K3_GROUP_GRAD_W) {
            e = (int)(job / m_blocks / c_blocks);
            c0 = (int)(job / m_blocks % c_blocks) * GG_TILE;
            c1 = min(g.n_in, c0 + GG_TILE);
            r0 = s_off[e];
            k1 = s_off[e + 1] - s_off[e];
        } else {
            const int t = (int)(job / m_blocks);
            e = group_find(s_tile, g.E, t);
            c0 = s_off[e] + (t - s_tile[e]) * GG_TILE;
            c1 = min(s_off[e + 1], c0 + GG_TILE);
            k1 = MODE == K3_GROUP_MM ? g.n_in : g.n_out;
        }
        float acc[4][4] = {};
        for (int k0 = 0; k0 < k1; k0 += GG_K) {
            for (int i = threadIdx.x; i < GG_K * GG_TILE; i += GG_THREADS) {
                // consecutive threads along the operand's contiguous axis
                const bool a_k = MODE == K3_GROUP_MM, b_k = MODE != K3_GROUP_GRAD_W;
                const int ka = a_k ? i % GG_K : i / GG_TILE, ma = a_k ? i / GG_K : i % GG_TILE;
                const int kb = b_k ? i % GG_K : i / GG_TILE, cb = b_k ? i / GG_K : i % GG_TILE;
                float va = 0.f, vb = 0.f;
                if (k0 + ka < k1 && m0 + ma < M) {
                    if (MODE == K3_GROUP_MM)
                        va = to_f32(B[e * g.stride_b + (m0 + ma) * g.ldb + k0 + ka]);
                    else if (MODE == K3_GROUP_GRAD_X)
                        va = to_f32(B[e * g.stride_b + (k0 + ka) * g.ldb + m0 + ma]);
                    else
                        va = to_f32(A[(r0 + k0 + ka) * g.lda + m0 + ma]);
                }
                if (k0 + kb < k1 && c0 + cb < c1) {
                    if (MODE == K3_GROUP_GRAD_W)
                        vb = to_f32(B[(r0 + k0 + kb) * g.ldb + c0 + cb]);
                    else
                        vb = to_f32(A[(int64_t)(c0 + cb) * g.lda + k0 + kb]);
                }
                sa[ka][ma] = va;
                sb[kb][cb] = vb;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < GG_K; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][tx + 16 * i], sb[k][ty + 16 * j], acc[i][j]);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int m = m0 + tx + 16 * i, c = c0 + ty + 16 * j;
                if (m >= M || c >= c1) continue;
                if (MODE == K3_GROUP_GRAD_W) {
                    O *o = out + e * g.stride_o + m * g.ldo + c;
                    *o = from_f32<O>(g.accumulate ? to_f32(*o) + acc[i][j] : acc[i][j]);
                } else {
                    out[c * g.ldo + m] = from_f32<O>(acc[i][j]);
                }
            }
    }
}

template <int MODE, class T, class O>
static int launch_generic(const K3Group &g, cudaStream_t st)
{
    const int sms = k3_num_sms();
    if (!sms) return K3MOE_ERR_CUDA;
    k3_launch(group_generic_kernel<MODE, T, O>, 4 * sms, GG_THREADS, 0, st, g);
    k3_note_launch();
    return cudaGetLastError() == cudaSuccess ? K3MOE_OK : K3MOE_ERR_CUDA;
}

template <int MODE>
static int dispatch_generic(const K3Group &g, cudaStream_t st)
{
    const bool bf = g.dtype == K3MOE_TYPE_BF16, f32 = g.out_dtype == K3MOE_TYPE_F32;
    if (bf) return f32 ? launch_generic<MODE, __nv_bfloat16, float>(g, st)
                       : launch_generic<MODE, __nv_bfloat16, __nv_bfloat16>(g, st);
    return f32 ? launch_generic<MODE, __half, float>(g, st) : launch_generic<MODE, __half, __half>(g, st);
}

}  // namespace k3

using namespace k3;

int k3_num_sms()
{
    static int sms[64] = {};
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev < 64 && sms[dev]) return sms[dev];
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 64) sms[dev] = n;
    return n;
}

int k3_group_generic(int mode, const K3Group &g, cudaStream_t st)
{
    switch (mode) {
    case K3_GROUP_MM: return dispatch_generic<K3_GROUP_MM>(g, st);
    case K3_GROUP_GRAD_X: return dispatch_generic<K3_GROUP_GRAD_X>(g, st);
    default: return dispatch_generic<K3_GROUP_GRAD_W>(g, st);
    }
}

// Checks shared by the three products; > 0: nothing to do.
static int group_check(const K3Group &g, int mode)
{
    if (g.E < 1 || g.rows < 0 || g.n_in < 1 || g.n_out < 1 || !g.offsets || !g.status) return K3MOE_ERR_ARG;
    if (g.E > K3MOE_TRAIN_MAX_EXPERTS) return K3MOE_ERR_SHAPE;
    if (g.dtype != K3MOE_TYPE_BF16 && g.dtype != K3MOE_TYPE_F16) return K3MOE_ERR_UNSUPPORTED;
    if (g.out_dtype != g.dtype && g.out_dtype != K3MOE_TYPE_F32) return K3MOE_ERR_UNSUPPORTED;
    if (mode == K3_GROUP_GRAD_W) {
        if (!g.out || (g.rows > 0 && (!g.a || !g.b))) return K3MOE_ERR_ARG;
        if (g.accumulate != 0 && g.accumulate != 1) return K3MOE_ERR_ARG;
        if (g.accumulate && g.out_dtype != K3MOE_TYPE_F32) return K3MOE_ERR_UNSUPPORTED;
        if (g.lda < g.n_out || g.ldb < g.n_in || g.ldo < g.n_in) return K3MOE_ERR_ARG;
        if (g.E > 1 && g.stride_o < (int64_t)(g.n_out - 1) * g.ldo + g.n_in) return K3MOE_ERR_ARG;
        const size_t no = k3_span(1, (g.E - 1) * g.stride_o + (int64_t)(g.n_out - 1) * g.ldo + g.n_in, 0, g.out_dtype);
        if (k3_overlap(g.out, no, g.a, k3_span(g.rows, g.n_out, g.lda, g.dtype)) ||
            k3_overlap(g.out, no, g.b, k3_span(g.rows, g.n_in, g.ldb, g.dtype)))
            return K3MOE_ERR_ALIAS;
        return K3MOE_OK;
    }
    const int in = mode == K3_GROUP_MM ? g.n_in : g.n_out, out = mode == K3_GROUP_MM ? g.n_out : g.n_in;
    if (g.rows > 0 && (!g.a || !g.b || !g.out)) return K3MOE_ERR_ARG;
    if (g.lda < in || g.ldo < out || g.ldb < g.n_in) return K3MOE_ERR_ARG;
    if (g.E > 1 && g.stride_b < 0) return K3MOE_ERR_ARG;      // 0: one weight for all groups
    const size_t no = k3_span(g.rows, out, g.ldo, g.out_dtype);
    const size_t nw = k3_span(1, (g.E - 1) * g.stride_b + (int64_t)(g.n_out - 1) * g.ldb + g.n_in, 0, g.dtype);
    if (k3_overlap(g.out, no, g.a, k3_span(g.rows, in, g.lda, g.dtype)) || k3_overlap(g.out, no, g.b, nw))
        return K3MOE_ERR_ALIAS;
    return g.rows == 0 ? 1 : K3MOE_OK;
}

static int group_run(const K3Group &g, int mode, cudaStream_t st)
{
    const int rc = group_check(g, mode);
    if (rc) return rc > 0 ? K3MOE_OK : rc;
    return k3_group_tc_fits(mode, g) ? k3_group_tc(mode, g, st) : k3_group_generic(mode, g, st);
}

extern "C" int k3moe_group_mm(const int32_t *offsets, int n_experts, int rows, int n_in, int n_out, const void *x,
                              int64_t ldx, const void *w, int64_t ldw, int64_t stride_w, int dtype, void *y,
                              int64_t ldy, int out_dtype, int32_t *status, cudaStream_t stream)
{
    const K3Group g = {offsets, n_experts, rows, n_in, n_out, x, ldx, w, ldw, stride_w, y, ldy, 0, dtype, out_dtype, 0,
                       status};
    return group_run(g, K3_GROUP_MM, stream);
}

extern "C" int k3moe_group_mm_grad_x(const int32_t *offsets, int n_experts, int rows, int n_in, int n_out,
                                     const void *dy, int64_t lddy, const void *w, int64_t ldw, int64_t stride_w,
                                     int dtype, void *dx, int64_t lddx, int out_dtype, int32_t *status,
                                     cudaStream_t stream)
{
    const K3Group g = {offsets, n_experts, rows, n_in, n_out, dy, lddy, w, ldw, stride_w, dx, lddx, 0, dtype,
                       out_dtype, 0, status};
    return group_run(g, K3_GROUP_GRAD_X, stream);
}

extern "C" int k3moe_group_mm_grad_w(const int32_t *offsets, int n_experts, int rows, int n_in, int n_out,
                                     const void *dy, int64_t lddy, const void *x, int64_t ldx, int dtype, void *dw,
                                     int64_t lddw, int64_t stride_dw, int out_dtype, int accumulate, int32_t *status,
                                     cudaStream_t stream)
{
    const K3Group g = {offsets, n_experts, rows, n_in, n_out, dy, lddy, x, ldx, 0, dw, lddw, stride_dw, dtype,
                       out_dtype, accumulate, status};
    return group_run(g, K3_GROUP_GRAD_W, stream);
}
