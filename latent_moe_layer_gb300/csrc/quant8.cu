// Rows and weights to 8-bit floating point with a power-of-two scale for each block of 128 (k3moe_quant8_rows) or
// 128 x 128 (k3moe_quant8_weights).
//
// A block's scale is 2^k, k >= -127 the smallest with amax <= 2^k FMAX.  FMAX is 0.875 2^TOP in both formats (448 = 0.875
// 2^9, 57344 = 0.875 2^16), so with amax = 1.m 2^(E - 127) in fp32 the scale's byte is k + 127 = E + 1 - TOP, and one more
// where m is above 0.75: bits of amax, no logarithm.  x 2^-k is exact, so a code is rounded once.
//
// Bound by HBM: 65,536 x 3584 bf16 rows in 107 us (6.6 TB/s), weights of 28 experts of 3584 x 3072 into both orders from one
// read in 182 us (6.8 TB/s).  Rows off 16-byte boundaries are loaded element by element: 171 us for the 107.
#include <cuda_fp8.h>

#include "glu.cuh"

namespace k3 {

template <int KIND> constexpr int F8_TOP = KIND == K3MOE_F8_E4M3 ? 9 : 16;

template <class T> constexpr uint32_t INF16 = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;

// The largest finite size of eight values, as bits of T, and whether an infinity is among them.  The packed maximum passes
// over NaN; where it is infinite (or all of a place's values are NaN) the values are looked at one by one.
template <class T>
__device__ __forceinline__ uint32_t amax_bits(const Vec<T, 8> &v, bool &infinite)
{
    using T2 = std::conditional_t<std::is_same<T, __half>::value, __half2, __nv_bfloat162>;
    const T2 *p = reinterpret_cast<const T2 *>(v.w);
    const T2 m2 = __hmax2(__hmax2(__habs2(p[0]), __habs2(p[1])), __hmax2(__habs2(p[2]), __habs2(p[3])));
    const uint32_t w = *reinterpret_cast<const uint32_t *>(&m2);
    uint32_t m = max(w & 0x7FFFu, w >> 16 & 0x7FFFu);
    infinite = m >= INF16<T>;
    if (infinite) {
        m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = v.w[i] & 0x7FFFu, hi = v.w[i] >> 16 & 0x7FFFu;
            m = max(m, lo < INF16<T> ? lo : 0u);
            m = max(m, hi < INF16<T> ? hi : 0u);
        }
    }
    return m;
}
template <class T>
__device__ __forceinline__ float from_bits(uint32_t b)
{
    if (std::is_same<T, __half>::value) return __half2float(__ushort_as_half((unsigned short)b));
    return __uint_as_float(b << 16);
}

// The scale's byte from the largest finite size of a block.
template <int KIND>
__device__ __forceinline__ uint32_t scale_byte(float amax)
{
    const uint32_t b = __float_as_uint(amax);
    return (uint32_t)max(0, (int)(b >> 23) + 1 - F8_TOP<KIND> + ((b & 0x7FFFFFu) > 0x600000u));
}
// 2^-k; byte <= 247
__device__ __forceinline__ float unscale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Eight codes.  The conversion gives infinities the largest finite code: they become NaN (E4M3) or stay infinite (E5M2).
template <class T, int KIND>
__device__ __forceinline__ uint2 codes8(const Vec<T, 8> &v, float f, bool infinite)
{
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 e = v.get2(2 * i);
        const F2 x = mul2({e.x, e.y}, f2(f));
        c[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x.x, x.y), __NV_SATFINITE, KIND == K3MOE_F8_E4M3 ? __NV_E4M3 : __NV_E5M2);
    }
    if (infinite) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = v.w[i] & 0x7FFFu, hi = v.w[i] >> 16 & 0x7FFFu;
            if (lo == INF16<T>) c[i] = (c[i] & 0xFF80u) | (KIND == K3MOE_F8_E4M3 ? 0x7Fu : 0x7Cu);
            if (hi == INF16<T>) c[i] = (c[i] & 0x80FFu) | (KIND == K3MOE_F8_E4M3 ? 0x7F00u : 0x7C00u);
        }
    }
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// Eight elements from `p`, those from `n` on zero; whole pieces in one load where `vec`.
template <class T>
__device__ __forceinline__ Vec<T, 8> load8(const T *p, int n, bool vec)
{
    if (vec && n >= 8) return *reinterpret_cast<const Vec<T, 8> *>(p);
    Vec<T, 8> v = {};
    const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) v.w[i / 2] |= (uint32_t)q[i] << (16 * (i & 1));
    return v;
}
__device__ __forceinline__ void store8(uint8_t *p, uint2 c, int n, bool vec)
{
    if (vec && n >= 8) {
        *reinterpret_cast<uint2 *>(p) = c;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
}

// ------------------------------------------------------------------ rows
struct QuantRows {
    const void *x;
    int64_t ldx, ldc, lds;
    int rows, n, blocks;
    uint8_t *codes, *scales;
    int vec_x, vec_c;
    int64_t row_step;                                    // from a block to the next of the same lanes: row_step rows and block_step
    int block_step;                                      // blocks on, a row more where that is past the row's end
};

// Eight lanes a block of 128, lane l its pieces of eight elements l and l + 8 (half a warp with a piece a lane takes more
// instructions for the maximum), QR_UNROLL blocks in flight.  The blocks are walked without a division (with one a block,
// 65,536 x 3584 took 208 us).
constexpr int QR_THREADS = 256, QR_LANES = 8, QR_UNROLL = 2, QR_CTAS = 5;
template <class T, int KIND>
__global__ void __launch_bounds__(QR_THREADS, QR_CTAS) quant_rows_kernel(const QuantRows a)
{
    griddep_enter();
    const int lane = threadIdx.x & (QR_LANES - 1);
    const uint32_t first = (blockIdx.x * QR_THREADS + threadIdx.x) / QR_LANES;
    int64_t at = first / (uint32_t)a.blocks;             // the next block's row
    int block = (int)(first - (uint32_t)at * (uint32_t)a.blocks);
    // whole warps take part in every round: lanes without a block work on zeros
    while (__any_sync(0xffffffffu, at < a.rows)) {
        Vec<T, 8> v[QR_UNROLL][2];
        int64_t row[QR_UNROLL];
        int col[QR_UNROLL], n[QR_UNROLL];
#pragma unroll
        for (int u = 0; u < QR_UNROLL; ++u) {
            row[u] = at;
            col[u] = block * 128 + lane * 8;
            n[u] = at < a.rows ? a.n - col[u] : 0;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                v[u][h] = load8<T>(static_cast<const T *>(a.x) + (n[u] > 64 * h ? at * a.ldx + col[u] + 64 * h : 0), n[u] - 64 * h, a.vec_x);
            at += a.row_step;
            block += a.block_step;
            if (block >= a.blocks) block -= a.blocks, ++at;
        }
#pragma unroll
        for (int u = 0; u < QR_UNROLL; ++u) {
            bool infinite[2];
            uint32_t m = max(amax_bits<T>(v[u][0], infinite[0]), amax_bits<T>(v[u][1], infinite[1]));
#pragma unroll
            for (int o = QR_LANES / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            const uint32_t s = scale_byte<KIND>(from_bits<T>(m));
            if (n[u] > 0) {
                uint8_t *c = a.codes + row[u] * a.ldc + col[u];
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    store8(c + 64 * h, codes8<T, KIND>(v[u][h], unscale(s), infinite[h]), n[u] - 64 * h, a.vec_c);
                if (lane == 0) a.scales[row[u] * a.lds + (col[u] >> 7)] = (uint8_t)s;
            }
        }
    }
}

// ------------------------------------------------------------------ weights
struct QuantWeights {
    const void *w;
    int64_t ldw, stride_w, ldc, stride_c, ldt, stride_t;
    int E, N, K, nb, kb;
    uint8_t *codes, *codes_t, *scales;
    int vec_w, vec_c, vec_t;
};

// A CTA a 128 x 128 block.  A thread takes four rows at a time of eight columns, so that the transposed codes leave as words
// of four rows: word w of column c lies at w ^ 4 (c / 8 % 8) of the column's 32 words, which spreads the stores over the
// banks and keeps 16-byte pieces whole for the reads.
constexpr int QW_THREADS = 256;
template <class T, int KIND>
__global__ void __launch_bounds__(QW_THREADS) quant_weights_kernel(const QuantWeights a)
{
    griddep_enter();
    __shared__ __align__(16) uint32_t turn[128 * 32];
    __shared__ uint32_t s_max[QW_THREADS / 32];
    const int64_t tile = blockIdx.x;
    const int kb = (int)(tile % a.kb), nb = (int)(tile / a.kb % a.nb);
    const int64_t e = tile / a.kb / a.nb;
    const int n0 = nb * 128, k0 = kb * 128;
    const int cp = threadIdx.x & 15, rg = threadIdx.x >> 4;              // 8 columns; 4 rows from 4 rg and from 4 (rg + 16)
    const int cols = max(0, min(8, a.K - k0 - cp * 8));
    Vec<T, 8> v[2][4];
    uint32_t m = 0;
    bool infinite = false;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = n0 + 4 * (rg + 16 * h) + i, n = r < a.N ? cols : 0;
            v[h][i] = load8<T>(static_cast<const T *>(a.w) + (n > 0 ? e * a.stride_w + r * a.ldw + k0 + cp * 8 : 0), n, a.vec_w);
        }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            bool inf;
            m = max(m, amax_bits<T>(v[h][i], inf));
            infinite |= inf;
        }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < QW_THREADS / 32; ++i) m = max(m, s_max[i]);
    const uint32_t s = scale_byte<KIND>(from_bits<T>(m));
    const float f = unscale(s);
    if (threadIdx.x == 0) a.scales[tile] = (uint8_t)s;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint2 c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = n0 + 4 * (rg + 16 * h) + i;
            c[i] = codes8<T, KIND>(v[h][i], f, infinite);
            if (r < a.N && cols > 0) store8(a.codes + e * a.stride_c + r * a.ldc + k0 + cp * 8, c[i], cols, a.vec_c);
        }
        if (a.codes_t)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint32_t r0 = half ? c[0].y : c[0].x, r1 = half ? c[1].y : c[1].x;
                const uint32_t r2 = half ? c[2].y : c[2].x, r3 = half ? c[3].y : c[3].x;
                const uint32_t a01 = __byte_perm(r0, r1, 0x5140), b01 = __byte_perm(r0, r1, 0x7362);
                const uint32_t a23 = __byte_perm(r2, r3, 0x5140), b23 = __byte_perm(r2, r3, 0x7362);
                uint32_t *at = turn + (cp * 8 + half * 4) * 32 + ((rg + 16 * h) ^ (4 * (cp & 7)));
                at[0] = __byte_perm(a01, a23, 0x5410);
                at[32] = __byte_perm(a01, a23, 0x7632);
                at[64] = __byte_perm(b01, b23, 0x5410);
                at[96] = __byte_perm(b01, b23, 0x7632);
            }
    }
    if (!a.codes_t) return;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 128 * 8 / QW_THREADS; ++i) {
        const int at = threadIdx.x + i * QW_THREADS, c = at >> 3, q = at & 7, n = a.N - n0 - q * 16;
        if (k0 + c >= a.K || n <= 0) continue;
        const uint4 x = *reinterpret_cast<const uint4 *>(turn + c * 32 + ((4 * q) ^ (4 * (c / 8 & 7))));
        uint8_t *o = a.codes_t + e * a.stride_t + (k0 + c) * a.ldt + n0 + q * 16;
        if (a.vec_t && n >= 16) {
            *reinterpret_cast<uint4 *>(o) = x;
        } else {
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (j < n) o[j] = (uint8_t)(w[j / 4] >> (8 * (j & 3)));
        }
    }
}

template <class F>
static int by_type(int dtype, int kind, F f)
{
    auto go = [&](auto t) {
        using T = decltype(t);
        if (kind == K3MOE_F8_E4M3) f(t, std::integral_constant<int, K3MOE_F8_E4M3>());
        else f(T(), std::integral_constant<int, K3MOE_F8_E5M2>());
    };
    if (dtype == K3MOE_TYPE_BF16) go(__nv_bfloat16());
    else go(__half());
    k3_note_launch();
    return cudaGetLastError() == cudaSuccess ? K3MOE_OK : K3MOE_ERR_CUDA;
}

static bool bytes_by(const void *p, int64_t ld, int64_t stride, int n) { return ((uintptr_t)p | ld | stride) % n == 0; }

static bool bad_types(int dtype, int kind)
{
    return (dtype != K3MOE_TYPE_BF16 && dtype != K3MOE_TYPE_F16) || (kind != K3MOE_F8_E4M3 && kind != K3MOE_F8_E5M2);
}

}  // namespace k3

using namespace k3;

extern "C" int k3moe_quant8_rows(const void *x, int64_t ldx, int rows, int n, int dtype, int kind, uint8_t *codes, int64_t ldc,
                                 uint8_t *scales, int64_t lds, cudaStream_t stream)
{
    if (rows < 0 || n < 1 || (rows > 0 && (!x || !codes || !scales))) return K3MOE_ERR_ARG;
    if (bad_types(dtype, kind)) return K3MOE_ERR_UNSUPPORTED;
    if (n > INT32_MAX - 256) return K3MOE_ERR_SHAPE;         // columns are counted in 32 bits, blocks rounded up
    const int blocks = (int)(((int64_t)n + 127) / 128);
    if (ldx < n || ldc < n || lds < blocks) return K3MOE_ERR_ARG;
    const size_t nx = k3_span(rows, n, ldx, dtype), nc = rows ? (size_t)(rows - 1) * ldc + n : 0,
                 ns = rows ? (size_t)(rows - 1) * lds + blocks : 0;
    if (k3_overlap(codes, nc, x, nx) || k3_overlap(scales, ns, x, nx) || k3_overlap(codes, nc, scales, ns)) return K3MOE_ERR_ALIAS;
    if (!k3_aligned({{x, 2}})) return K3MOE_ERR_ALIGN;
    if (rows == 0) return K3MOE_OK;
    const int sms = k3_num_sms();
    if (!sms) return K3MOE_ERR_CUDA;
    const int64_t ctas = ((int64_t)rows * blocks + QR_THREADS / QR_LANES - 1) / (QR_THREADS / QR_LANES);
    const unsigned grid = (unsigned)std::min<int64_t>(ctas, QR_CTAS * (int64_t)sms);
    const int64_t step = (int64_t)grid * (QR_THREADS / QR_LANES);
    const QuantRows a = {x, ldx, ldc, lds, rows, n, blocks, codes, scales, k3_rows16(x, ldx, dtype), bytes_by(codes, ldc, 0, 8),
                         step / blocks, (int)(step % blocks)};
    return by_type(dtype, kind, [&](auto t, auto k) {
        k3_launch(quant_rows_kernel<decltype(t), decltype(k)::value>, grid, QR_THREADS, 0, stream, a);
    });
}

extern "C" int k3moe_quant8_weights(const void *w, int64_t ldw, int64_t stride_w, int n_experts, int n_out, int n_in, int dtype,
                                    int kind, uint8_t *codes, int64_t ldc, int64_t stride_c, uint8_t *codes_t, int64_t ldt,
                                    int64_t stride_t, uint8_t *scales, cudaStream_t stream)
{
    if (n_experts < 1 || n_out < 1 || n_in < 1 || !w || !codes || !scales) return K3MOE_ERR_ARG;
    if (bad_types(dtype, kind)) return K3MOE_ERR_UNSUPPORTED;
    if (ldw < n_in || ldc < n_in || (codes_t && ldt < n_out)) return K3MOE_ERR_ARG;
    const int64_t sw = (int64_t)(n_out - 1) * ldw + n_in, sc = (int64_t)(n_out - 1) * ldc + n_in,
                  stt = codes_t ? (int64_t)(n_in - 1) * ldt + n_out : 0;
    if (n_experts > 1 && (stride_w < 0 || stride_c < sc || (codes_t && stride_t < stt))) return K3MOE_ERR_ARG;
    if (n_out > INT32_MAX - 256 || n_in > INT32_MAX - 256) return K3MOE_ERR_SHAPE;
    const int nb = (int)(((int64_t)n_out + 127) / 128), kb = (int)(((int64_t)n_in + 127) / 128);
    const double tiles = (double)n_experts * nb * kb;
    if (tiles >= 2147483648.0) return K3MOE_ERR_SHAPE;
    const int64_t more = n_experts - 1;
    const size_t nw = (size_t)(more * stride_w + sw) * 2, nc = (size_t)(more * stride_c + sc),
                 nt = codes_t ? (size_t)(more * stride_t + stt) : 0, ns = (size_t)tiles;
    if (k3_overlap(codes, nc, w, nw) || k3_overlap(codes_t, nt, w, nw) || k3_overlap(scales, ns, w, nw) ||
        k3_overlap(codes, nc, codes_t, nt) || k3_overlap(codes, nc, scales, ns) || k3_overlap(codes_t, nt, scales, ns))
        return K3MOE_ERR_ALIAS;
    if (!k3_aligned({{w, 2}})) return K3MOE_ERR_ALIGN;
    const bool one = n_experts == 1;
    const QuantWeights a = {w, ldw, stride_w, ldc, stride_c, ldt, stride_t, n_experts, n_out, n_in, nb, kb, codes, codes_t, scales,
                            k3_rows16(w, ldw, dtype) && (one || stride_w * 2 % 16 == 0), bytes_by(codes, ldc, one ? 0 : stride_c, 8),
                            codes_t && bytes_by(codes_t, ldt, one ? 0 : stride_t, 16)};
    return by_type(dtype, kind, [&](auto t, auto k) {
        k3_launch(quant_weights_kernel<decltype(t), decltype(k)::value>, dim3((unsigned)tiles), QW_THREADS, 0, stream, a);
    });
}
