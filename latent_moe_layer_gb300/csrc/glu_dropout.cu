// Dropout from a counter-based generator (its mask is never stored: forward and gradient draw it
// again from seed, offset and the element's index), alone with a residual and inside the gated unit
// (k3moe_dropout, k3moe_glu_dropout, k3moe_glu_dropout_grad).
#include "experts.h"

namespace k3 {

constexpr uint32_t PHILOX_M0 = 0xD2511F53u, PHILOX_M1 = 0xCD9E8D57u, PHILOX_W0 = 0x9E3779B9u, PHILOX_W1 = 0xBB67AE85u;

struct DropArgs {
    uint32_t key[10][2];                  // the rounds' keys: seed + round x the generator's two increments
    uint32_t first[3];                    // what round 1 makes of the offset: hi(off0 M1) ^ key, lo(off0 M1), off1 ^ key
    uint64_t second;                      // M0 x first[0]: round 2's product where the element's high word is 0
    uint32_t threshold;                   // keep where the word is at least this: floor(p 2^32)
    float scale;                          // 1 / (1 - p)
};

// Philox4x32-10 (Salmon, Moraes, Dror and Shaw 2011): ten rounds of two 32 x 32 -> 64-bit products.  Counter
// (block, offset), key seed.  The products are what it costs (4 cycles each of the integer multiplier a
// warp), so those of rounds 1 and 2 that do not depend on the element come with the arguments; `p` is the
// first round's other product, (low word of block) x M0.
__device__ __forceinline__ uint4 philox(uint64_t p, uint32_t block_hi, const DropArgs &a)
{
    uint32_t x2 = (uint32_t)(p >> 32) ^ a.first[2], x3 = (uint32_t)p, x0, x1;
    p = a.second;
    if (block_hi) p = (uint64_t)(a.first[0] ^ block_hi) * PHILOX_M0;       // elements past 2^34
    uint64_t q = (uint64_t)x2 * PHILOX_M1;
    x0 = (uint32_t)(q >> 32) ^ a.first[1] ^ a.key[1][0];
    x1 = (uint32_t)q;
    x2 = (uint32_t)(p >> 32) ^ x3 ^ a.key[1][1];
    x3 = (uint32_t)p;
#pragma unroll
    for (int r = 2; r < 10; ++r) {
        p = (uint64_t)x0 * PHILOX_M0, q = (uint64_t)x2 * PHILOX_M1;
        x0 = (uint32_t)(q >> 32) ^ x1 ^ a.key[r][0];
        x1 = (uint32_t)q;
        x2 = (uint32_t)(p >> 32) ^ x3 ^ a.key[r][1];
        x3 = (uint32_t)p;
    }
    return make_uint4(x0, x1, x2, x3);
}

// word[j] = the random word of element i0 + j; i0 a multiple of V when V is 4 or 8.
template <int V>
__device__ __forceinline__ void drop_words(uint64_t i0, const DropArgs &a, uint32_t (&w)[V])
{
    const uint64_t block = i0 >> 2, p = (uint64_t)(uint32_t)block * PHILOX_M0;
    const uint32_t hi = (uint32_t)(block >> 32);
    if (V % 4 == 0) {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            const uint4 r = philox(p + (uint64_t)(j / 4) * PHILOX_M0, hi, a);      // block is even when V is 8
            w[j] = r.x, w[(j + 1) % V] = r.y, w[(j + 2) % V] = r.z, w[(j + 3) % V] = r.w;
        }
    } else {
        static_assert(V % 4 == 0 || V == 1, "whole blocks or one element");
        const uint4 r = philox(p, hi, a);
        const uint32_t q = (uint32_t)i0 & 3;
        w[0] = q == 0 ? r.x : q == 1 ? r.y : q == 2 ? r.z : r.w;
    }
}

// v where the element is kept, else 0 (whatever v holds)
template <bool DROP>
__device__ __forceinline__ float kept(float v, uint32_t word, const DropArgs &a)
{
    return !DROP || word >= a.threshold ? v : 0.f;
}

// ------------------------------------------------------------------ pipelined pieces
// With the generator a 16-bit piece costs about as much computing as HBM takes for its bytes, and warps that
// load, then compute, spend the sum of the two.  So there (RING) each thread copies its next piece of 16 bytes
// an input into shared memory ahead (cp.async; its own slots, so nothing is synchronised), which costs no
// registers: 58.7 M bf16 elements take a fifth less.  Without the generator, and for fp32, direct loads are 3-5 %
// faster (its computing hides behind the bytes).
constexpr int PIPE = 2, PIPE_THREADS = 256;

__device__ __forceinline__ void cp_async16(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Runs work(i, values) over this thread's pieces i0, i0 + step, ... < total; addr gives the inputs' addresses of
// the next piece, in order.
template <class T, int V, int NIN, bool RING, class Addr, class Work>
__device__ __forceinline__ void for_pieces(int64_t i0, int64_t step, int64_t total, Addr addr, Work work)
{
    if constexpr (RING) {
        static_assert(V * sizeof(T) == 16, "16-byte pieces");
        __shared__ uint4 ring[PIPE][NIN][PIPE_THREADS];
        const int tid = threadIdx.x;
        int64_t ahead = i0;
        auto fetch = [&](int slot) {
            if (ahead < total) {
                const T *p[NIN];
                addr(p);
#pragma unroll
                for (int j = 0; j < NIN; ++j)
                    cp_async16(&ring[slot][j][tid], p[j]);
            }
            cp_async_commit();
            ahead += step;
        };
#pragma unroll
        for (int s = 0; s < PIPE - 1; ++s) fetch(s);
        int slot = 0;
        for (int64_t i = i0; i < total; i += step) {
            fetch((slot + PIPE - 1) % PIPE);
            cp_async_wait<PIPE - 1>();
            Vec<T, V> in[NIN];
#pragma unroll
            for (int j = 0; j < NIN; ++j) in[j] = *reinterpret_cast<const Vec<T, V> *>(&ring[slot][j][tid]);
            work(i, in);
            slot = (slot + 1) % PIPE;
        }
    } else {
        for (int64_t i = i0; i < total; i += step) {
            const T *p[NIN];
            addr(p);
            Vec<T, V> in[NIN];
#pragma unroll
            for (int j = 0; j < NIN; ++j)
                in[j] = *reinterpret_cast<const Vec<T, V> *>(p[j]);
            work(i, in);
        }
    }
}

// ------------------------------------------------------------------ dropout with residual
// 58.7 M fp32 elements with a residual in 107 us (6.6 TB/s, HBM binds); in bf16 55 us (6.4 TB/s) and 52 us
// without the residual (4.5 TB/s: the generator binds).
template <class T, int V, bool DROP, bool RES>
__global__ void __launch_bounds__(PIPE_THREADS) dropout_kernel(const T *x, const T *res, int64_t n, const DropArgs a,
                                                               T *out)
{
    griddep_enter();
    const int64_t step = (int64_t)gridDim.x * PIPE_THREADS, i0 = (int64_t)blockIdx.x * PIPE_THREADS + threadIdx.x;
    const int64_t whole = n / V;
    int64_t at = i0 * V;
    for_pieces<T, V, 1 + RES, DROP && V == 8>(
        i0, step, whole,
        [&](const T *(&p)[1 + RES]) {
            p[0] = x + at;
            if (RES) p[RES] = res + at;
            at += step * V;
        },
        [&](int64_t i, const Vec<T, V>(&in)[1 + RES]) {
            uint32_t w[V] = {};
            if (DROP) drop_words<V>((uint64_t)i * V, a, w);
            Vec<T, V> o;
#pragma unroll
            for (int j = 0; j < V; j += 2) {
                float2 d = in[0].get2(j);
                d = {kept<DROP>(d.x * a.scale, w[j], a), kept<DROP>(d.y * a.scale, w[V == 1 ? 0 : j + 1], a)};
                if (RES) {
                    const float2 r = in[RES].get2(j);
                    d = {d.x + r.x, d.y + r.y};
                }
                o.set2(j, d.x, d.y);
            }
            *reinterpret_cast<Vec<T, V> *>(out + i * V) = o;
        });
    // the elements after the last whole piece, one a thread
    const int64_t i = whole * V + i0;
    if (i < n) {
        uint32_t w[1] = {};
        if (DROP) drop_words<1>((uint64_t)i, a, w);
        const float d = kept<DROP>(to_f32(x[i]) * a.scale, w[0], a);
        out[i] = from_f32<T>(RES ? d + to_f32(res[i]) : d);
    }
}

// ------------------------------------------------------------------ gated unit
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

// Whether all |v| <= limit (no NaN): packed maxima for the 16-bit types.
template <class T, int V>
__device__ __forceinline__ bool all_within(const Vec<T, V> &v, float limit)
{
    if constexpr (V == 8) {
        using T2 = std::conditional_t<std::is_same<T, __half>::value, __half2, __nv_bfloat162>;
        const T2 *p = reinterpret_cast<const T2 *>(v.w);
        const T2 m = __hmax2_nan(__hmax2_nan(__habs2(p[0]), __habs2(p[1])), __hmax2_nan(__habs2(p[2]), __habs2(p[3])));
        const float2 e = unpack2<T>(*reinterpret_cast<const uint32_t *>(&m));
        return e.x <= limit && e.y <= limit;
    } else {
        return fabsf(v.get2(0).x) <= limit;
    }
}

// V outputs from loaded inputs g, u (and the output's gradient).  Where all values are finite (SMALL) a dropped
// element's factor is cleared; elsewhere its results are, since 0 x NaN is not 0.
template <class T, int V, int ACT, bool DROP, bool GRAD, bool SMALL>
__device__ __forceinline__ void glu_piece(const Vec<T, V> (&in)[2 + GRAD], const uint32_t (&w)[V], const GluArgs &act,
                                          const DropArgs &a, Vec<T, V> &o0, Vec<T, V> &o1)
{
    constexpr bool FACTOR = DROP && SMALL && ACT == K3MOE_ACT_SITU, RESULT = DROP && !FACTOR;
#pragma unroll
    for (int j = 0; j < V; j += 2) {
        const int k = V == 1 ? 0 : j + 1;
        const float2 g = in[0].get2(j), u = in[1].get2(j);
        F2 v0, v1, t = f2(ACT == K3MOE_ACT_SILU ? a.scale * SILU_UNIT : a.scale);
        if (GRAD) {
            const float2 d = in[1 + GRAD].get2(j);
            t = mul2({d.x, d.y}, t);
        }
        t = {kept<FACTOR>(t.x, w[j], a), kept<FACTOR>(t.y, w[k], a)};
        glu_two<ACT, GRAD, SMALL>({g.x, g.y}, {u.x, u.y}, t, act, v0, v1);
        o0.set2(j, kept<RESULT>(v0.x, w[j], a), kept<RESULT>(v0.y, w[k], a));
        if (GRAD) o1.set2(j, kept<RESULT>(v1.x, w[j], a), kept<RESULT>(v1.y, w[k], a));
    }
}

// From a thread's piece to its next: `col` pieces further in the row, and a row more where that is past the row's
// end (nv pieces).  The addresses move by bytes[0], or by bytes[1] with that row more.
struct GluWalk {
    int64_t gu[2], da[2], out[2];
    int col, nv;
    __device__ __forceinline__ bool next(int &c) const
    {
        c += col;
        const bool over = c >= nv;
        if (over) c -= nv;
        return over;
    }
};
template <class P>
__device__ __forceinline__ void move_on(P *&p, const int64_t (&bytes)[2], bool over)
{
    p = reinterpret_cast<P *>(reinterpret_cast<uintptr_t>(p) + (over ? bytes[1] : bytes[0]));
}

// Pieces of V elements over the [rows, width] matrix; piece i is row i / nv, column (i % nv) V.  About 100 of the
// warp instructions per 8 elements are the generator's; the arithmetic pipes bind next to HBM.  32,768 x 3072 bf16,
// p = 0.1, back to back: SiLU 106 us (5.7 TB/s; without dropout 90 us, 6.7 TB/s), SiTU 146 us, the gradients 152 and 182
// us.  CTAs an SM (registers) by measurement: more cost registers that spill, fewer leave latency open.  SiLU's gradient
// took 187 us with the 72 registers of three CTAs, its forward without dropout 96 with the 54 of four.
template <int ACT, bool DROP, bool GRAD>
constexpr int glu_ctas() { return ACT == K3MOE_ACT_SILU ? (GRAD || DROP ? 4 : 5) : GRAD ? 3 : 4; }
template <class T, int V, int ACT, bool DROP, bool GRAD>
__global__ void __launch_bounds__(PIPE_THREADS, glu_ctas<ACT, DROP, GRAD>())
    glu_kernel(const T *da, int64_t ldda, const T *gu, int64_t ldgu, int rows, int width, const GluArgs act,
               const DropArgs a, const GluWalk walk, T *out, int64_t ldo)
{
    griddep_enter();
    const int nv = walk.nv;
    const int64_t total = (int64_t)rows * nv, step = (int64_t)gridDim.x * PIPE_THREADS;
    const int64_t i0 = (int64_t)blockIdx.x * PIPE_THREADS + threadIdx.x;
    const int64_t row = i0 / nv;
    int col = (int)(i0 - row * nv), out_col = col;       // of the piece being fetched; of the one being computed
    const T *gu_at = gu + row * ldgu + (int64_t)col * V, *da_at = GRAD ? da + row * ldda + (int64_t)col * V : nullptr;
    T *out_at = out + row * ldo + (int64_t)col * V;
    for_pieces<T, V, 2 + GRAD, DROP && V == 8>(
        i0, step, total,
        [&](const T *(&p)[2 + GRAD]) {
            p[0] = gu_at;
            p[1] = gu_at + width;
            if (GRAD) p[1 + GRAD] = da_at;
            const bool over = walk.next(col);
            move_on(gu_at, walk.gu, over);
            if (GRAD) move_on(da_at, walk.da, over);
        },
        [&](int64_t i, const Vec<T, V>(&in)[2 + GRAD]) {
            uint32_t w[V] = {};
            if (DROP) drop_words<V>((uint64_t)i * V, a, w);
            Vec<T, V> o0, o1;
            // one branch a piece: tanh arguments beyond 1 (or NaN) are rare
            const bool small = ACT == K3MOE_ACT_SILU ||
                               (all_within<T, V>(in[0], act.g.small) && all_within<T, V>(in[1], act.u.small));
            if (small) glu_piece<T, V, ACT, DROP, GRAD, true>(in, w, act, a, o0, o1);
            else glu_piece<T, V, ACT, DROP, GRAD, false>(in, w, act, a, o0, o1);
            *reinterpret_cast<Vec<T, V> *>(out_at) = o0;
            if (GRAD) *reinterpret_cast<Vec<T, V> *>(out_at + width) = o1;
            move_on(out_at, walk.out, walk.next(out_col));
        });
}

}  // namespace k3

using namespace k3;

static bool drop_args(double p, uint64_t seed, uint64_t offset, DropArgs &a)
{
    if (!(p >= 0.0 && p < 1.0)) return false;
    for (uint32_t r = 0; r < 10; ++r) {
        a.key[r][0] = (uint32_t)seed + r * PHILOX_W0;
        a.key[r][1] = (uint32_t)(seed >> 32) + r * PHILOX_W1;
    }
    const uint64_t q = (uint64_t)(uint32_t)offset * PHILOX_M1;
    a.first[0] = (uint32_t)(q >> 32) ^ a.key[0][0];
    a.first[1] = (uint32_t)q;
    a.first[2] = (uint32_t)(offset >> 32) ^ a.key[0][1];
    a.second = (uint64_t)a.first[0] * PHILOX_M0;
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

// CTAs for `pieces`: as many as are resident at once (the loops stride the rest, since a second, partly filled round
// of CTAs costs as much as a full one), and no more than `few` an SM where each thread then has 64 pieces or more.
// `fit` is the kernel's own memory.
template <class F>
static unsigned resident_grid(F kern, int64_t pieces, int sms, int &fit, int few = 32)
{
    int n = fit;
    if (!n) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, PIPE_THREADS, 0) != cudaSuccess || n < 1) n = 1;
        fit = n;
    }
    if (pieces >= (int64_t)64 * PIPE_THREADS * few * sms) n = std::min(n, few);
    return (unsigned)std::min<int64_t>((pieces + PIPE_THREADS - 1) / PIPE_THREADS, (int64_t)n * sms);
}

template <class T, int V>
static void launch_dropout(const void *x, const void *res, int64_t n, const DropArgs &a, void *out, int sms,
                           cudaStream_t st)
{
    with_bool(a.threshold != 0, [&](auto drop) {
        with_bool(res != nullptr, [&](auto with_res) {
            auto kern = dropout_kernel<T, V, decltype(drop)::value, decltype(with_res)::value>;
            static int fit = 0;
            k3_launch(kern, resident_grid(kern, (n + V - 1) / V, sms, fit), PIPE_THREADS, 0, st, (const T *)x,
                      (const T *)res, n, a, (T *)out);
        });
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
                       bool is_situ, const GluArgs &act, const DropArgs &a, void *out, int64_t ldo, int sms,
                       cudaStream_t st)
{
    with_bool(a.threshold != 0, [&](auto drop) {
        with_bool(is_situ, [&](auto situ) {
            constexpr int ACT = decltype(situ)::value ? K3MOE_ACT_SITU : K3MOE_ACT_SILU;
            auto kern = glu_kernel<T, V, ACT, decltype(drop)::value, GRAD>;
            static int fit = 0;
            GluWalk walk;
            walk.nv = width / V;
            // SiLU's gradient with the generator is bound by HBM, which serves long runs of its five streams better from
            // fewer CTAs: 152 us with 2 an SM, 187 with 3 (32,768 x 3072); at 5,003 rows all that fit are 6 % faster
            constexpr int FEW = GRAD && V == 8 && decltype(drop)::value && ACT == K3MOE_ACT_SILU ? 2 : 32;
            const unsigned grid = resident_grid(kern, (int64_t)rows * walk.nv, sms, fit, FEW);
            const int64_t step = (int64_t)grid * PIPE_THREADS, row_step = step / walk.nv;
            walk.col = (int)(step - row_step * walk.nv);
            auto moves = [&](int64_t ld, int64_t (&bytes)[2]) {
                bytes[0] = (row_step * ld + (int64_t)walk.col * V) * (int64_t)sizeof(T);
                bytes[1] = bytes[0] + (ld - (int64_t)walk.nv * V) * (int64_t)sizeof(T);
            };
            moves(ldgu, walk.gu);
            moves(ldda, walk.da);
            moves(ldo, walk.out);
            k3_launch(kern, grid, PIPE_THREADS, 0, st, (const T *)da, ldda, (const T *)gu, ldgu, rows, width, act, a, walk,
                      (T *)out, ldo);
        });
    });
}

static SoftLimit soft_limit(float limit, float largest)
{
    const double inv = 1.0 / (double)limit, inv2 = inv * inv;
    // beyond these limits the folded coefficients would leave fp32's range: all values by the general form
    const bool folds = limit >= 0x1p-20f && limit <= 0x1p20f;
    return {limit, (float)inv, folds ? std::min(limit, largest) : -1.0f, (float)(TANH_N * inv2), (float)(TANH_D1 * inv2),
            (float)(TANH_D2 * inv2 * inv2), (float)-inv2};
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
    // limits (0 and below: the defaults) whose reciprocal is a finite number that is not zero; NaN is neither
    for (const float limit : {beta, linear_beta})
        if (!(limit <= 0.f || (limit >= 0x1p-126f && limit <= 0x1p126f))) return K3MOE_ERR_ARG;
    if (dtype != K3MOE_TYPE_BF16 && dtype != K3MOE_TYPE_F16) return K3MOE_ERR_UNSUPPORTED;
    const size_t ngu = k3_span(rows, 2 * (int64_t)width, ldgu, dtype);
    const size_t no = k3_span(rows, (GRAD ? 2 : 1) * (int64_t)width, ldo, dtype);
    const bool in_place = GRAD && out == gu && ldo == ldgu;
    if ((!in_place && k3_overlap(out, no, gu, ngu)) || (GRAD && k3_overlap(out, no, da, k3_span(rows, width, ldda, dtype))))
        return K3MOE_ERR_ALIAS;
    if (rows == 0) return K3MOE_OK;
    const int sms = k3_num_sms();
    if (!sms) return K3MOE_ERR_CUDA;
    const bool situ = act == K3MOE_ACT_SITU;
    const GluArgs c = {soft_limit(beta > 0.f ? beta : 4.0f, 60.0f), soft_limit(linear_beta > 0.f ? linear_beta : 25.0f, 0x1p20f)};
    const bool vec = width % 8 == 0 && k3_rows16(gu, ldgu, dtype) && k3_rows16(out, ldo, dtype) &&
                     (!GRAD || k3_rows16(da, ldda, dtype));
    if (dtype == K3MOE_TYPE_BF16)
        vec ? launch_glu<__nv_bfloat16, 8, GRAD>(da, ldda, gu, ldgu, rows, width, situ, c, a, out, ldo, sms, st)
            : launch_glu<__nv_bfloat16, 1, GRAD>(da, ldda, gu, ldgu, rows, width, situ, c, a, out, ldo, sms, st);
    else
        vec ? launch_glu<__half, 8, GRAD>(da, ldda, gu, ldgu, rows, width, situ, c, a, out, ldo, sms, st)
            : launch_glu<__half, 1, GRAD>(da, ldda, gu, ldgu, rows, width, situ, c, a, out, ldo, sms, st);
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
