// Dropout from a counter-based generator (its mask is never stored: forward and gradient draw it
// again from seed, offset and the element's index), alone with a residual and inside the gated unit
// (k3moe_dropout, k3moe_glu_dropout, k3moe_glu_dropout_grad).
#include "experts.h"

namespace k3 {

struct DropArgs {
    uint32_t key[10][2];                  // the rounds' keys: seed + round x the generator's two increments
    uint32_t off0, off1;                  // offset
    uint32_t threshold;                   // keep where the word is at least this: floor(p 2^32)
    float scale;                          // 1 / (1 - p)
};

// Philox4x32-10 (Salmon, Moraes, Dror and Shaw 2011): ten rounds of two 32 x 32 -> 64-bit products.
__device__ __forceinline__ uint4 philox(uint64_t block, const DropArgs &a)
{
    uint32_t x0 = (uint32_t)block, x1 = (uint32_t)(block >> 32), x2 = a.off0, x3 = a.off1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p = (uint64_t)x0 * 0xD2511F53u, q = (uint64_t)x2 * 0xCD9E8D57u;
        x0 = (uint32_t)(q >> 32) ^ x1 ^ a.key[r][0];
        x1 = (uint32_t)q;
        x2 = (uint32_t)(p >> 32) ^ x3 ^ a.key[r][1];
        x3 = (uint32_t)p;
    }
    return make_uint4(x0, x1, x2, x3);
}

// factor[j] = scale where element i0 + j is kept, else 0; i0 a multiple of 4 when V is.
template <int V, bool DROP>
__device__ __forceinline__ void drop_factors(uint64_t i0, const DropArgs &a, float (&f)[V])
{
    if (!DROP) {
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = 1.0f;
    } else if (V % 4 == 0) {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            const uint4 r = philox((i0 + j) >> 2, a);
            f[j] = r.x >= a.threshold ? a.scale : 0.f;
            f[j + 1] = r.y >= a.threshold ? a.scale : 0.f;
            f[j + 2] = r.z >= a.threshold ? a.scale : 0.f;
            f[j + 3] = r.w >= a.threshold ? a.scale : 0.f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint4 r = philox((i0 + j) >> 2, a);
            const uint32_t q = (uint32_t)(i0 + j) & 3;
            f[j] = (q == 0 ? r.x : q == 1 ? r.y : q == 2 ? r.z : r.w) >= a.threshold ? a.scale : 0.f;
        }
    }
}

// ------------------------------------------------------------------ dropout with residual
template <class T, int V, bool DROP>
__global__ void __launch_bounds__(256) dropout_kernel(const T *x, const T *res, int64_t n, const DropArgs a, T *out)
{
    griddep_enter();
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < (n + V - 1) / V; i += step) {
        const int64_t i0 = i * V;
        float f[V];
        drop_factors<V, DROP>((uint64_t)i0, a, f);
        if (i0 + V <= n) {
            const Vec<T, V> v = *reinterpret_cast<const Vec<T, V> *>(x + i0);
            Vec<T, V> r = {}, o;
            if (res) r = *reinterpret_cast<const Vec<T, V> *>(res + i0);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                // a dropped element contributes 0 whatever it holds
                const float d = !DROP || f[j] != 0.f ? to_f32(v.v[j]) * f[j] : 0.f;
                o.v[j] = from_f32<T>(res ? d + to_f32(r.v[j]) : d);
            }
            *reinterpret_cast<Vec<T, V> *>(out + i0) = o;
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (i0 + j < n) {
                    const float d = !DROP || f[j] != 0.f ? to_f32(x[i0 + j]) * f[j] : 0.f;
                    out[i0 + j] = from_f32<T>(res ? d + to_f32(res[i0 + j]) : d);
                }
        }
    }
}

// ------------------------------------------------------------------ gated unit
// Results are rounded to 16 bits, so hardware exponential and reciprocal (a few 2^-22) suffice; an
// infinite exponential gives the exact limits 0 and 1.
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

// tanh x within 3e-7, relative also near 0: Lambert's continued fraction x / (1 + x^2 / (3 + x^2 / (5 + x^2 / (7 +
// x^2 / 9)))) as one quotient up to |x| = 1 (off by 6e-8 there), (e^2x - 1) / (e^2x + 1) beyond.
__device__ __forceinline__ float tanh_quotient(float x)
{
    const float x2 = x * x;
    float num = x * fmaf(x2, x2 + 105.0f, 945.0f), den = fmaf(x2, fmaf(15.0f, x2, 420.0f), 945.0f);
    if (fabsf(x) > 1.0f) {
        const float e = __expf(2.0f * fminf(fmaxf(x, -10.0f), 10.0f));      // tanh 10 is 1 in fp32
        num = e - 1.0f;
        den = e + 1.0f;
    }
    return x != x ? x : __fdividef(num, den);
}

// a(g, u) and its derivatives: SiLU a = g s u, or the soft-limited a = s f h with f = beta tanh(g /
// beta), h = linear_beta tanh(u / linear_beta), s = sigmoid(g).
template <int ACT>
__device__ __forceinline__ float glu_value(float g, float u, const K3Act &c)
{
    const float s = sigmoid(g);
    if (ACT == K3MOE_ACT_SILU) return g * s * u;
    return s * (c.beta * tanh_quotient(g * c.inv_beta)) * (c.linear_beta * tanh_quotient(u * c.inv_linear_beta));
}

template <int ACT>
__device__ __forceinline__ void glu_slopes(float g, float u, const K3Act &c, float &dg, float &du)
{
    const float s = sigmoid(g);
    if (ACT == K3MOE_ACT_SILU) {
        dg = u * (s + g * s * (1.0f - s));
        du = g * s;
    } else {
        const float tg = tanh_quotient(g * c.inv_beta), tu = tanh_quotient(u * c.inv_linear_beta);
        const float f = c.beta * tg, h = c.linear_beta * tu;
        dg = h * (s * (1.0f - s) * f + s * (1.0f - tg * tg));
        du = s * f * (1.0f - tu * tu);
    }
}

// Pieces of V elements over the [rows, width] matrix; piece i is row i / nv, column (i % nv) V.
template <class T, int V, int ACT, bool DROP, bool GRAD>
__global__ void __launch_bounds__(256) glu_kernel(const T *da, int64_t ldda, const T *gu, int64_t ldgu, int rows,
                                                  int width, const K3Act act, const DropArgs a, T *out, int64_t ldo)
{
    griddep_enter();
    const int nv = width / V;
    const int64_t total = (int64_t)rows * nv, step = (int64_t)gridDim.x * blockDim.x;
    int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    int64_t row = i / nv;
    int col = (int)(i - row * nv);
    const int64_t row_step = step / nv;
    const int col_step = (int)(step - row_step * nv);
    for (; i < total; i += step) {
        const T *src = gu + row * ldgu + (int64_t)col * V;
        const Vec<T, V> g = *reinterpret_cast<const Vec<T, V> *>(src);
        const Vec<T, V> u = *reinterpret_cast<const Vec<T, V> *>(src + width);
        Vec<T, V> d = {};
        if (GRAD) d = *reinterpret_cast<const Vec<T, V> *>(da + row * ldda + (int64_t)col * V);
        float f[V];
        drop_factors<V, DROP>((uint64_t)i * V, a, f);
        T *dst = out + row * ldo + (int64_t)col * V;
        if (GRAD) {
            Vec<T, V> og, ou;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float sg, su;
                glu_slopes<ACT>(to_f32(g.v[j]), to_f32(u.v[j]), act, sg, su);
                const float t = to_f32(d.v[j]) * f[j];
                const bool kept = !DROP || f[j] != 0.f;       // a dropped element contributes 0 whatever it holds
                og.v[j] = from_f32<T>(kept ? t * sg : 0.f);
                ou.v[j] = from_f32<T>(kept ? t * su : 0.f);
            }
            *reinterpret_cast<Vec<T, V> *>(dst) = og;
            *reinterpret_cast<Vec<T, V> *>(dst + width) = ou;
        } else {
            Vec<T, V> o;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float v = glu_value<ACT>(to_f32(g.v[j]), to_f32(u.v[j]), act) * f[j];
                o.v[j] = from_f32<T>(!DROP || f[j] != 0.f ? v : 0.f);
            }
            *reinterpret_cast<Vec<T, V> *>(dst) = o;
        }
        row += row_step;
        col += col_step;
        if (col >= nv) {
            col -= nv;
            ++row;
        }
    }
}

}  // namespace k3

using namespace k3;

static bool drop_args(double p, uint64_t seed, uint64_t offset, DropArgs &a)
{
    if (!(p >= 0.0 && p < 1.0)) return false;
    for (uint32_t r = 0; r < 10; ++r) {
        a.key[r][0] = (uint32_t)seed + r * 0x9E3779B9u;
        a.key[r][1] = (uint32_t)(seed >> 32) + r * 0xBB67AE85u;
    }
    a.off0 = (uint32_t)offset;
    a.off1 = (uint32_t)(offset >> 32);
    a.threshold = (uint32_t)(p * 4294967296.0);
    a.scale = (float)(1.0 / (1.0 - p));
    return true;
}

template <class F>
static void with_bool(bool b, F f)
{
    if (b) f(std::true_type());
    else f(std::false_type());
}

// enough CTAs of 256 threads for `pieces`, at most eight a multiprocessor (the loops stride the rest)
static int elementwise_grid(int64_t pieces, int sms)
{
    return (int)std::min<int64_t>((pieces + 255) / 256, (int64_t)8 * sms);
}

template <class T, int V>
static void launch_dropout(const void *x, const void *res, int64_t n, const DropArgs &a, void *out, int sms,
                           cudaStream_t st)
{
    with_bool(a.threshold != 0, [&](auto drop) {
        k3_launch(dropout_kernel<T, V, decltype(drop)::value>, elementwise_grid((n + V - 1) / V, sms), 256, 0, st,
                  (const T *)x, (const T *)res, n, a, (T *)out);
    });
}

extern "C" int k3moe_dropout(const void *x, const void *residual, int64_t n, int dtype, double p, uint64_t seed,
                             uint64_t offset, void *out, cudaStream_t st)
{
    DropArgs a;
    if (n < 0 || !drop_args(p, seed, offset, a) || (n > 0 && (!x || !out))) return K3MOE_ERR_ARG;
    if (dtype != K3MOE_TYPE_F32 && dtype != K3MOE_TYPE_BF16 && dtype != K3MOE_TYPE_F16) return K3MOE_ERR_UNSUPPORTED;
    const size_t nb = k3_span(1, n, n, dtype);
    if ((out != x && k3_overlap(out, nb, x, nb)) || (residual && out != residual && k3_overlap(out, nb, residual, nb)))
        return K3MOE_ERR_ALIAS;
    if (n == 0) return K3MOE_OK;
    const int sms = k3_num_sms();
    if (!sms) return K3MOE_ERR_CUDA;
    const bool vec = (((uintptr_t)x | (uintptr_t)residual | (uintptr_t)out) & 15) == 0;
    if (dtype == K3MOE_TYPE_F32)
        vec ? launch_dropout<float, 4>(x, residual, n, a, out, sms, st)
            : launch_dropout<float, 1>(x, residual, n, a, out, sms, st);
    else if (dtype == K3MOE_TYPE_BF16)
        vec ? launch_dropout<__nv_bfloat16, 8>(x, residual, n, a, out, sms, st)
            : launch_dropout<__nv_bfloat16, 1>(x, residual, n, a, out, sms, st);
    else
        vec ? launch_dropout<__half, 8>(x, residual, n, a, out, sms, st)
            : launch_dropout<__half, 1>(x, residual, n, a, out, sms, st);
    k3_note_launch();
    return cudaGetLastError() == cudaSuccess ? K3MOE_OK : K3MOE_ERR_CUDA;
}

template <class T, int V, bool GRAD>
static void launch_glu(const void *da, int64_t ldda, const void *gu, int64_t ldgu, int rows, int width,
                       const K3Act &act, const DropArgs &a, void *out, int64_t ldo, int sms, cudaStream_t st)
{
    with_bool(a.threshold != 0, [&](auto drop) {
        with_bool(act.kind == K3MOE_ACT_SITU, [&](auto situ) {
            constexpr int ACT = decltype(situ)::value ? K3MOE_ACT_SITU : K3MOE_ACT_SILU;
            k3_launch(glu_kernel<T, V, ACT, decltype(drop)::value, GRAD>,
                      elementwise_grid((int64_t)rows * (width / V), sms), 256, 0, st, (const T *)da, ldda,
                      (const T *)gu, ldgu, rows, width, act, a, (T *)out, ldo);
        });
    });
}

template <bool GRAD>
static int glu_run(const void *da, int64_t ldda, const void *gu, int64_t ldgu, int rows, int width, int dtype, int act,
                   float beta, float linear_beta, double p, uint64_t seed, uint64_t offset, void *out, int64_t ldo,
                   cudaStream_t st)
{
    DropArgs a;
    if (rows < 0 || width < 1 || width > (1 << 30) || !drop_args(p, seed, offset, a)) return K3MOE_ERR_ARG;
    if (rows > 0 && (!gu || !out || (GRAD && !da))) return K3MOE_ERR_ARG;
    if (ldgu < 2 * (int64_t)width || ldo < (GRAD ? 2 : 1) * (int64_t)width || (GRAD && ldda < width)) return K3MOE_ERR_ARG;
    if (act != K3MOE_ACT_SILU && act != K3MOE_ACT_SITU) return K3MOE_ERR_UNSUPPORTED;
    if (beta != beta || linear_beta != linear_beta) return K3MOE_ERR_ARG;
    if (dtype != K3MOE_TYPE_BF16 && dtype != K3MOE_TYPE_F16) return K3MOE_ERR_UNSUPPORTED;
    const size_t ngu = k3_span(rows, 2 * (int64_t)width, ldgu, dtype);
    const size_t no = k3_span(rows, (GRAD ? 2 : 1) * (int64_t)width, ldo, dtype);
    const bool in_place = GRAD && out == gu && ldo == ldgu;
    if ((!in_place && k3_overlap(out, no, gu, ngu)) || (GRAD && k3_overlap(out, no, da, k3_span(rows, width, ldda, dtype))))
        return K3MOE_ERR_ALIAS;
    if (rows == 0) return K3MOE_OK;
    const int sms = k3_num_sms();
    if (!sms) return K3MOE_ERR_CUDA;
    K3Act c;
    c.kind = act;
    c.beta = beta > 0.f ? beta : 4.0f;
    c.linear_beta = linear_beta > 0.f ? linear_beta : 25.0f;
    c.inv_beta = 1.0f / c.beta;
    c.inv_linear_beta = 1.0f / c.linear_beta;
    const bool vec = width % 8 == 0 && k3_rows16(gu, ldgu, dtype) && k3_rows16(out, ldo, dtype) &&
                     (!GRAD || k3_rows16(da, ldda, dtype));
    if (dtype == K3MOE_TYPE_BF16)
        vec ? launch_glu<__nv_bfloat16, 8, GRAD>(da, ldda, gu, ldgu, rows, width, c, a, out, ldo, sms, st)
            : launch_glu<__nv_bfloat16, 1, GRAD>(da, ldda, gu, ldgu, rows, width, c, a, out, ldo, sms, st);
    else
        vec ? launch_glu<__half, 8, GRAD>(da, ldda, gu, ldgu, rows, width, c, a, out, ldo, sms, st)
            : launch_glu<__half, 1, GRAD>(da, ldda, gu, ldgu, rows, width, c, a, out, ldo, sms, st);
    k3_note_launch();
    return cudaGetLastError() == cudaSuccess ? K3MOE_OK : K3MOE_ERR_CUDA;
}

extern "C" int k3moe_glu_dropout(const void *gu, int64_t ldgu, int rows, int width, int dtype, int act, float situ_beta,
                                 float situ_linear_beta, double p, uint64_t seed, uint64_t offset, void *a,
                                 int64_t lda, cudaStream_t stream)
{
    return glu_run<false>(nullptr, 0, gu, ldgu, rows, width, dtype, act, situ_beta, situ_linear_beta, p, seed, offset, a,
                          lda, stream);
}

extern "C" int k3moe_glu_dropout_grad(const void *da, int64_t ldda, const void *gu, int64_t ldgu, int rows, int width,
                                      int dtype, int act, float situ_beta, float situ_linear_beta, double p,
                                      uint64_t seed, uint64_t offset, void *dgu, int64_t lddgu, cudaStream_t stream)
{
    return glu_run<true>(da, ldda, gu, ldgu, rows, width, dtype, act, situ_beta, situ_linear_beta, p, seed, offset, dgu,
                         lddgu, stream);
}
