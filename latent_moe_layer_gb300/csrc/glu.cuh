// Arithmetic of the gated unit, for its own kernels (glu_dropout.cu) and the products that end in it (group_tc.cuh,
// group_mm.cu).
#pragma once

#include "experts.h"

namespace k3 {

// Results are rounded to 16 bits, so the hardware exponential and reciprocal suffice (2^-22 relative, and the rounding of
// the exponential's argument, 2^-24 of it); an infinite exponential gives the exact limits 0 and 1.
__device__ __forceinline__ float rcp_fast(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two fp32 values in one register pair; sums and products of both in one instruction.
struct F2 {
    float x, y;
};
__device__ __forceinline__ F2 f2(float v) { return {v, v}; }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\t"
        "mov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ F2 rcp2(F2 a) { return {rcp_fast(a.x), rcp_fast(a.y)}; }
// 2^-SHIFT (1 + exp(-v))
template <int SHIFT>
__device__ __forceinline__ F2 one_plus_exp_neg(F2 v)
{
    const F2 t = SHIFT ? fma2(v, f2(-1.4426950408889634f), f2((float)-SHIFT)) : mul2(v, f2(-1.4426950408889634f));
    float a, b;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(t.y));
    return fma2({a, b}, f2(1.0f), f2(1.0f / (1 << SHIFT)));
}
// SiLU takes its sigmoid as 2^10 s: s itself is a subnormal from -87.34 down, which the reciprocal flushes, and g s is not.
// So gates count down to -94.2 (the exponential alone leaves fp32 at -88.7); below, the unit is 0.  The other factor,
// dropout's, brings the 2^-10 along; products keep 14 bits where the result is bf16's smallest normal number, more above.
constexpr int SILU_SHIFT = 10;
constexpr float SILU_UNIT = 1.0f / (1 << SILU_SHIFT);

// The unit's constants.  tanh(x) = x (1 + TANH_N x^2) / (1 + TANH_D1 x^2 + TANH_D2 x^4) for |x| <= 1 within 7e-8 of
// itself: the quotient of these degrees with the smallest largest relative error there (fitted in fp64; 2.1e-7
// evaluated in fp32).  limit tanh(v / limit) takes them with limit's powers folded in, from v^2 itself.
constexpr double TANH_N = 0.09437645428558641, TANH_D1 = 0.4277082447645945, TANH_D2 = 0.009246752739316303;
struct SoftLimit {
    float limit, inv, small;              // 1 / limit; the quotient serves |v| <= small
    float n, d1, d2, neg_inv2;            // its coefficients; -1 / limit^2
};
struct GluArgs {
    SoftLimit g, u;
};
__device__ __forceinline__ void tanh_quotient(F2 v2, const SoftLimit &c, F2 &num, F2 &den)
{
    num = fma2(v2, f2(c.n), f2(1.0f));
    den = fma2(v2, fma2(v2, f2(c.d2), f2(c.d1)), f2(1.0f));
}
// tanh of any x, beyond 1 as (1 - t) / (1 + t) with t = e^-2|x|, and its derivative 1 - tanh^2 = 4 t / (1 + t)^2, which
// keeps its bits where the difference would have none left
__device__ __forceinline__ float tanh_any(float x, float &slope)
{
    const float v = x * x, num = fmaf(v, (float)TANH_N, 1.0f), den = fmaf(v, fmaf(v, (float)TANH_D2, (float)TANH_D1), 1.0f);
    const float t = expf(-2.0f * fabsf(x)), r = rcp_fast(1.0f + t);
    slope = 2.0f * t * r * (2.0f * r);
    return fabsf(x) <= 1.0f ? x * num * rcp_fast(den) : copysignf((1.0f - t) * r, x);
}

// sigmoid of any x as p q, a few 2^-22 of it: both stay normal numbers where the sigmoid itself is a subnormal; c is
// 1 - sigmoid, without the difference
__device__ __forceinline__ void sigmoid_any(float x, float &p, float &q, float &c)
{
    const float e = expf(-0.5f * fabsf(x)), r = rcp_fast(fmaf(e, e, 1.0f)), low = e * r;      // sigmoid(|x|) = r, of -|x| e low
    const bool neg = x < 0.0f;
    p = neg ? e : 1.0f;
    q = neg ? low : r;
    c = neg ? r : e * low;
}

// The unit a = s f(g) h(u), s = sigmoid(g), of two elements: SiLU f = g, h = u; SiTU f = beta tanh(g / beta),
// h = linear_beta tanh(u / linear_beta).  o0 = a t; GRAD: (o0, o1) = (da/dg, da/du) t.  SMALL: all tanh arguments
// are within [-1, 1] and |g| <= 60, so that the sigmoid and both tanh can share one reciprocal of a finite product.
template <int ACT, bool GRAD, bool SMALL>
__device__ __forceinline__ void glu_two(F2 g, F2 u, F2 t, const GluArgs &c, F2 &o0, F2 &o1)
{
    const F2 one = f2(1.0f), neg = f2(-1.0f);
    if (ACT == K3MOE_ACT_SILU) {
        // t has the factor SILU_UNIT
        const F2 s = rcp2(one_plus_exp_neg<SILU_SHIFT>(g)), gt = mul2(g, t);
        if (GRAD) {
            o0 = mul2(mul2(mul2(u, t), s), fma2(g, fma2(s, f2(-SILU_UNIT), one), one));    // u s (1 + g (1 - s))
            o1 = mul2(gt, s);
        } else {
            o0 = mul2(mul2(gt, u), s);
        }
        return;
    }
    if (SMALL) {
        F2 ng, dg, nu, du;
        tanh_quotient(mul2(g, g), c.g, ng, dg);
        tanh_quotient(mul2(u, u), c.u, nu, du);
        ng = mul2(ng, g);
        nu = mul2(nu, u);
        const F2 ds = one_plus_exp_neg<0>(g);
        if (GRAD) {
            // a reciprocal each: the pipe of products binds (one reciprocal of the product: 6 % more time)
            // da/dg = h s (f (1 - s) + 1 - (f / beta)^2), da/du = s f (1 - (h / linear_beta)^2)
            const F2 s = rcp2(ds), f = mul2(ng, rcp2(dg)), h = mul2(nu, rcp2(du)), st = mul2(s, t);
            o0 = mul2(mul2(h, st), fma2(f, fma2(f, f2(c.g.neg_inv2), fma2(s, neg, one)), one));
            o1 = mul2(mul2(f, st), fma2(mul2(h, f2(c.u.neg_inv2)), h, one));
        } else {
            o0 = mul2(mul2(ng, nu), mul2(rcp2(mul2(ds, mul2(dg, du))), t));
        }
    } else {
        F2 p, q, c1;                                     // s = p q, 1 - s
        sigmoid_any(g.x, p.x, q.x, c1.x);
        sigmoid_any(g.y, p.y, q.y, c1.y);
        F2 dg, du;                                       // 1 - tanh^2
        const F2 tg = {tanh_any(g.x * c.g.inv, dg.x), tanh_any(g.y * c.g.inv, dg.y)};
        const F2 tu = {tanh_any(u.x * c.u.inv, du.x), tanh_any(u.y * c.u.inv, du.y)};
        const F2 f = mul2(tg, f2(c.g.limit)), h = mul2(tu, f2(c.u.limit));
        if (GRAD) {
            o0 = mul2(mul2(mul2(h, p), mul2(q, t)), fma2(f, c1, dg));
            o1 = mul2(mul2(mul2(f, p), mul2(q, t)), du);
        } else {
            o0 = mul2(mul2(mul2(f, p), mul2(h, q)), t);
        }
    }
}

inline SoftLimit soft_limit(float limit, float largest)
{
    const double inv = 1.0 / (double)limit, inv2 = inv * inv;
    // beyond these limits the folded coefficients would leave fp32's range: all values by the general form
    const bool folds = limit >= 0x1p-20f && limit <= 0x1p20f;
    return {limit, (float)inv, folds ? std::min(limit, largest) : -1.0f, (float)(TANH_N * inv2), (float)(TANH_D1 * inv2),
            (float)(TANH_D2 * inv2 * inv2), (float)-inv2};
}

// The unit's constants, or the error of arguments that have none.
inline int glu_args(int act, float beta, float linear_beta, GluArgs &c)
{
    if (act != K3MOE_ACT_SILU && act != K3MOE_ACT_SITU) return K3MOE_ERR_UNSUPPORTED;
    // limits (0 and below: the defaults) whose reciprocal is a finite number that is not zero; NaN is neither
    for (const float limit : {beta, linear_beta})
        if (!(limit <= 0.f || (limit >= 0x1p-126f && limit <= 0x1p126f))) return K3MOE_ERR_ARG;
    c = {soft_limit(beta > 0.f ? beta : 4.0f, 60.0f), soft_limit(linear_beta > 0.f ? linear_beta : 25.0f, 0x1p20f)};
    return K3MOE_OK;
}

}  // namespace k3

// The gated block on a product: the unit, and the gradient's da (NULL: forward).
struct K3GroupGlu {
    int situ;
    k3::GluArgs c;
    const void *da;
    int64_t ldda;
};
int k3_group_glu_tc(const K3Group &g, const K3GroupGlu &u, cudaStream_t st);
int k3_group_glu_generic(const K3Group &g, const K3GroupGlu &u, cudaStream_t st);
