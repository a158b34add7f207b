// Products grouped by expert (k3moe_group_mm, _grad_x, _grad_w): argument checks, and the kernel of shapes
// and strides that the copy engine, which feeds the main kernel (group_tc.cu), cannot address.
#include "glu.cuh"
#include "group_sched.cuh"

namespace k3 {

constexpr int GG_TILE = 64, GG_K = 32, GG_THREADS = 256, GG_ROW = GG_K + 8;    // 80-byte rows: no bank is hit twice
// k steps summed by the tensor cores, which truncate, before the sum is added in fp32 (512 values, f16 256: see group_tc.cu)
template <class T> constexpr int GG_CHUNK = std::is_same<T, __half>::value ? 8 : 16;

template <class T>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2])
{
    if (std::is_same<T, __half>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// Four 8 x 8 blocks of 16-bit values: lane i gives the address of row i % 8 of block i / 8.
__device__ __forceinline__ void load_blocks(uint32_t (&r)[4], const void *row)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"((uint32_t)__cvta_generic_to_shared(row))
                 : "memory");
}

// 64 x 64 outputs per CTA, 32 x 16 a warp, the contraction in steps of 32 through shared memory; the next step's
// values are in flight meanwhile, one element a load, so any size, stride and alignment goes.  Those loads bind it:
// 4,099 rows over 8 experts, 1001 to 2003: 260 us, 63 TFLOP/s (fp32 sums on the CUDA cores: 820); the gradients 312 and 309.
// Tile rows x are output rows (tokens' rows; n_out for grad_w), columns y the output's contiguous axis.  The gated block's
// 64 columns are eight gate and the same eight up rows of the weights in turn, so that a thread's two accumulator pieces of a
// warp tile are both projections of the same elements.
template <int MODE, class T, class O>
__global__ void __launch_bounds__(GG_THREADS, 3) group_generic_kernel(const K3Group g, const K3GroupGlu unit)
{
    griddep_enter();
    constexpr bool W = MODE == K3_GROUP_GRAD_W, GLU = MODE == K3_GROUP_GLU || MODE == K3_GROUP_GLU_GRAD;
    constexpr bool X_K = !W, Y_K = MODE == K3_GROUP_MM || GLU;           // operands contiguous along the contraction
    constexpr int Y_TILE = GLU ? GG_TILE / 2 : GG_TILE;                  // output columns of a tile
    constexpr int LOADS = GG_TILE * GG_K / GG_THREADS;
    __shared__ __align__(16) uint16_t sx[2][GG_TILE][GG_ROW], sy[2][GG_TILE][GG_ROW];
    __shared__ int s_off[K3MOE_TRAIN_MAX_EXPERTS + 1], s_tile[K3MOE_TRAIN_MAX_EXPERTS + 1], s_tmp[GG_THREADS / 32];
    if (!group_tiles<GG_THREADS, GG_TILE>(g.offsets, g.E, g.rows, s_off, s_tile, s_tmp, g.status)) return;
    const uint16_t *A = static_cast<const uint16_t *>(g.a), *B = static_cast<const uint16_t *>(g.b);
    O *out = static_cast<O *>(g.out);
    const int NY = MODE == K3_GROUP_MM || GLU ? g.n_out : g.n_in;
    const int y_blocks = (NY + Y_TILE - 1) / Y_TILE, x_blocks = W ? (g.n_out + GG_TILE - 1) / GG_TILE : 1;
    const long long jobs = (W ? (long long)g.E * x_blocks : (long long)s_tile[g.E]) * y_blocks;
    const int lane = threadIdx.x & 31, wx = (threadIdx.x >> 5 & 1) * 32, wy = (threadIdx.x >> 6) * 16;
    for (long long job = blockIdx.x; job < jobs; job += gridDim.x) {
        const int y0 = (int)(job % y_blocks) * Y_TILE, t = (int)(job / y_blocks);
        int e, x0, x1, k1;                       // tile rows [x0, x1), contraction [0, k1)
        long long r0 = 0;
        if (W) {
            e = t / x_blocks;
            x0 = t % x_blocks * GG_TILE;
            x1 = g.n_out;
            r0 = s_off[e];
            k1 = s_off[e + 1] - s_off[e];
        } else {
            e = group_find(s_tile, g.E, t);
            x0 = s_off[e] + (t - s_tile[e]) * GG_TILE;
            x1 = s_off[e + 1];
            k1 = MODE == K3_GROUP_MM || GLU ? g.n_in : g.n_out;
        }
        const uint16_t *Be = B + (W ? r0 * g.ldb : e * g.stride_b), *Ae = A + (W ? r0 * g.lda : 0);
        uint16_t vx[LOADS], vy[LOADS];
        auto fetch = [&](int k0) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                // consecutive threads along the operand's contiguous axis
                const int at = threadIdx.x + i * GG_THREADS;
                const int kx = k0 + (X_K ? at % GG_K : at / GG_TILE), x = x0 + (X_K ? at / GG_K : at % GG_TILE);
                const int ky = k0 + (Y_K ? at % GG_K : at / GG_TILE), iy = Y_K ? at / GG_K : at % GG_TILE;
                const int y = y0 + (GLU ? iy / 16 * 8 + iy % 8 : iy), up = GLU && (iy & 8) ? NY : 0;
                vx[i] = kx < k1 && x < x1 ? Ae[X_K ? x * g.lda + kx : kx * g.lda + x] : (uint16_t)0;
                vy[i] = ky < k1 && y < NY ? Be[Y_K ? (y + up) * g.ldb + ky : ky * g.ldb + y] : (uint16_t)0;
            }
        };
        float acc[2][2][4] = {}, sum[2][2][4] = {};
        const int steps = (k1 + GG_K - 1) / GG_K;
        if (steps > 0) fetch(0);
        for (int s = 0; s < steps; ++s) {
            const int b = s & 1;
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const int at = threadIdx.x + i * GG_THREADS;
                sx[b][X_K ? at / GG_K : at % GG_TILE][X_K ? at % GG_K : at / GG_TILE] = vx[i];
                sy[b][Y_K ? at / GG_K : at % GG_TILE][Y_K ? at % GG_K : at / GG_TILE] = vy[i];
            }
            __syncthreads();                     // one a step: the other buffer was read before it
            if (s + 1 < steps) fetch((s + 1) * GG_K);
#pragma unroll
            for (int k = 0; k < GG_K; k += 16) {
                uint32_t fa[2][4], fy[4];
#pragma unroll
                for (int i = 0; i < 2; ++i) load_blocks(fa[i], &sx[b][wx + 16 * i + (lane & 15)][k + (lane >> 4) * 8]);
                load_blocks(fy, &sy[b][wy + (lane >> 4) * 8 + (lane & 7)][k + (lane >> 3 & 1) * 8]);
                const uint32_t fb[2][2] = {{fy[0], fy[1]}, {fy[2], fy[3]}};
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) mma_16816<T>(acc[i][j], fa[i], fb[j]);
            }
            if (s % GG_CHUNK<T> == GG_CHUNK<T> - 1 || s == steps - 1) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    (&sum[0][0][0])[i] += (&acc[0][0][0])[i];
                    (&acc[0][0][0])[i] = 0.f;
                }
            }
        }
        __syncthreads();                         // the next job writes the buffers
        if constexpr (GLU) {
            constexpr bool GRAD = MODE == K3_GROUP_GLU_GRAD;
#pragma unroll
            for (int i = 0; i < 4; ++i) {        // two elements of a row at a time
                const int x = x0 + wx + (i >> 1) * 16 + (lane >> 2) + (i & 1) * 8, y = y0 + wy / 2 + (lane & 3) * 2;
                if (x >= x1 || y >= NY) continue;
                const float *gs = &sum[i >> 1][0][2 * (i & 1)], *us = &sum[i >> 1][1][2 * (i & 1)];
                const F2 gv = {gs[0], gs[1]}, uv = {us[0], us[1]};
                F2 t = f2(unit.situ ? 1.0f : SILU_UNIT), o0, o1;
                const bool two = y + 1 < NY;
                if (GRAD) {
                    const T *d = static_cast<const T *>(unit.da) + x * unit.ldda + y;
                    t = mul2(t, {to_f32(d[0]), two ? to_f32(d[1]) : 0.f});
                }
                if (unit.situ) glu_two<K3MOE_ACT_SITU, GRAD, false>(gv, uv, t, unit.c, o0, o1);
                else glu_two<K3MOE_ACT_SILU, GRAD, false>(gv, uv, t, unit.c, o0, o1);
                O *o = out + x * g.ldo + y;
                o[0] = from_f32<O>(o0.x);
                if (two) o[1] = from_f32<O>(o0.y);
                if (GRAD) {
                    o[NY] = from_f32<O>(o1.x);
                    if (two) o[NY + 1] = from_f32<O>(o1.y);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int x = x0 + wx + (i >> 3) * 16 + (lane >> 2) + (i >> 1 & 1) * 8;
                const int y = y0 + wy + (i >> 2 & 1) * 8 + (lane & 3) * 2 + (i & 1);
                if (x >= x1 || y >= NY) continue;
                O *o = out + (W ? e * g.stride_o : 0) + x * g.ldo + y;
                const float v = (&sum[0][0][0])[i];
                *o = from_f32<O>(W && g.accumulate ? to_f32(*o) + v : v);
            }
        }
    }
}

template <int MODE, class T, class O>
static int launch_generic(const K3Group &g, cudaStream_t st, const K3GroupGlu &unit = {})
{
    const int sms = k3_num_sms();
    if (!sms) return K3MOE_ERR_CUDA;
    k3_launch(group_generic_kernel<MODE, T, O>, 3 * sms, GG_THREADS, 0, st, g, unit);
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

int k3_group_glu_generic(const K3Group &g, const K3GroupGlu &u, cudaStream_t st)
{
    if (g.dtype == K3MOE_TYPE_BF16)
        return u.da ? launch_generic<K3_GROUP_GLU_GRAD, __nv_bfloat16, __nv_bfloat16>(g, st, u)
                    : launch_generic<K3_GROUP_GLU, __nv_bfloat16, __nv_bfloat16>(g, st, u);
    return u.da ? launch_generic<K3_GROUP_GLU_GRAD, __half, __half>(g, st, u) : launch_generic<K3_GROUP_GLU, __half, __half>(g, st, u);
}

int k3_group_check(const K3Group &g, int mode)
{
    if (g.E < 1 || g.rows < 0 || g.n_in < 1 || g.n_out < 1 || !g.offsets || !g.status) return K3MOE_ERR_ARG;
    if (g.E > K3MOE_TRAIN_MAX_EXPERTS || std::max({g.rows, g.n_in, g.n_out}) > K3_GROUP_MAX_SIZE) return K3MOE_ERR_SHAPE;
    if (g.dtype != K3MOE_TYPE_BF16 && g.dtype != K3MOE_TYPE_F16) return K3MOE_ERR_UNSUPPORTED;
    if (g.out_dtype != g.dtype && g.out_dtype != K3MOE_TYPE_F32) return K3MOE_ERR_UNSUPPORTED;
    const size_t noff = sizeof(int32_t) * ((size_t)g.E + 1);
    const bool aligned = k3_aligned({{g.a, 2}, {g.b, 2}, {g.out, k3_type_bytes(g.out_dtype)}, {g.offsets, 4}, {g.status, 4}});
    if (mode == K3_GROUP_GRAD_W) {
        if (!g.out || (g.rows > 0 && (!g.a || !g.b))) return K3MOE_ERR_ARG;
        if (g.accumulate != 0 && g.accumulate != 1) return K3MOE_ERR_ARG;
        if (g.accumulate && g.out_dtype != K3MOE_TYPE_F32) return K3MOE_ERR_UNSUPPORTED;
        if (g.lda < g.n_out || g.ldb < g.n_in || g.ldo < g.n_in) return K3MOE_ERR_ARG;
        if (g.E > 1 && g.stride_o < (int64_t)(g.n_out - 1) * g.ldo + g.n_in) return K3MOE_ERR_ARG;
        const size_t no = k3_span(1, (g.E - 1) * g.stride_o + (int64_t)(g.n_out - 1) * g.ldo + g.n_in, 0, g.out_dtype);
        if (k3_overlap(g.out, no, g.a, k3_span(g.rows, g.n_out, g.lda, g.dtype)) ||
            k3_overlap(g.out, no, g.b, k3_span(g.rows, g.n_in, g.ldb, g.dtype)) || k3_overlap(g.out, no, g.offsets, noff))
            return K3MOE_ERR_ALIAS;
        return aligned ? K3MOE_OK : K3MOE_ERR_ALIGN;
    }
    const int in = mode == K3_GROUP_MM ? g.n_in : g.n_out, out = mode == K3_GROUP_MM ? g.n_out : g.n_in;
    if (g.rows > 0 && (!g.a || !g.b || !g.out)) return K3MOE_ERR_ARG;
    if (g.lda < in || g.ldo < out || g.ldb < g.n_in) return K3MOE_ERR_ARG;
    if (g.E > 1 && g.stride_b < 0) return K3MOE_ERR_ARG;      // 0: one weight for all groups
    const size_t no = k3_span(g.rows, out, g.ldo, g.out_dtype);
    const size_t nw = k3_span(1, (g.E - 1) * g.stride_b + (int64_t)(g.n_out - 1) * g.ldb + g.n_in, 0, g.dtype);
    if (k3_overlap(g.out, no, g.a, k3_span(g.rows, in, g.lda, g.dtype)) || k3_overlap(g.out, no, g.b, nw) ||
        k3_overlap(g.out, no, g.offsets, noff))
        return K3MOE_ERR_ALIAS;
    if (!aligned) return K3MOE_ERR_ALIGN;
    return g.rows == 0 ? 1 : K3MOE_OK;
}

static int group_run(const K3Group &g, int mode, cudaStream_t st)
{
    const int rc = k3_group_check(g, mode);
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
