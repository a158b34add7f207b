// Norms around a block (k3moe_rms_norm, k3moe_norm_residual and their gradients): the norm after the block with
// its gate, the residual and the norm before the next block in one pass over the rows.
//
//   h = alpha res + gate * (gain * y rs(y)),   n = next_gain * h rs(h),   rs(v) = 1 / sqrt(mean v^2 + eps)
//
// and with v' = v rs(v), from dh and dn:
//   t     = dh + rs(h) (next_gain dn - h' mean(next_gain dn h'))        dnext_gain = sum over rows of dn h'
//   dres  = alpha t,   dgate = t gain y',   s = gate t,                 dgain = sum over rows of s y'
//   dy    = rs(y) (gain s - y' mean(gain s y'))
// The means are computed again from y and h, which the gradient reads anyway: nothing is kept for it but h.  rms_norm
// is the second half alone (h = x given).
#include "experts.h"

namespace k3 {

constexpr int NORM_GATE_NONE = K3MOE_GATE_NONE, NORM_GATE_ROW = K3MOE_GATE_ROW, NORM_GATE_FULL = K3MOE_GATE_FULL;

struct NormArgs {
    // forward: y, res, gate (or x in y); gradient: dh, dn, y, h, gate
    const void *y, *res, *gate, *dh, *dn, *hin;
    int64_t ld_y, ld_res, ld_gate, ld_dh, ld_dn, ld_hin;
    const void *gain, *next_gain;                        // NULL: ones
    int gain_f32, gate_kind, next;
    float scale, eps, inv_d;
    int rows, D, group;                                  // group: threads a row
    void *h, *n, *dgate;                                 // gradient: h = dy, n = dres (without POST: n = dx)
    int64_t ld_h, ld_n, ld_dgate;
    float *part;                                         // [dgain, dnext_gain][row groups of the grid][D]
};

__device__ __forceinline__ void norm_cp16(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
                 : "memory");
}

// V gains from element i.
template <class T, int V>
__device__ __forceinline__ void load_gain(const void *p, int f32, int i, float (&g)[V])
{
    if (!p) {
#pragma unroll
        for (int j = 0; j < V; ++j) g[j] = 1.0f;
    } else if (f32) {
        const float *q = static_cast<const float *>(p) + i;
        if constexpr (V % 4 == 0) {
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                const float4 x = __ldg(reinterpret_cast<const float4 *>(q + j));
                g[j] = x.x, g[j + 1] = x.y, g[j + 2] = x.z, g[j + 3] = x.w;
            }
        } else {
            g[0] = __ldg(q);
        }
    } else {
        const Vec<T, V> x = *reinterpret_cast<const Vec<T, V> *>(static_cast<const T *>(p) + i);
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            const float2 e = x.get2(j);
            g[j] = e.x;
            if (V > 1) g[(j + 1) % V] = e.y;
        }
    }
}

// Sums over the threads of a row (its warps of the CTA, all of them in the same order: every thread gets the same bits).
// Two buffers in turn, so that one barrier a sum is enough.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int group, float *buf, int &turn)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (group == 32) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = group >> 5, first = (int)threadIdx.x / group * warps;
    float *b = buf + turn * 32 * 3;
    turn ^= 1;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) b[warp * 3 + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane < warps ? b[(first + lane) * 3 + i] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

// Whether the next row's pieces fit in shared memory (not those of the widest fp32 rows).
template <int V, int SLOTS>
constexpr bool norm_ring() { return V > 1 && SLOTS * 16 + 1024 <= kMaxSmem; }

// A group of threads holds a row in registers, P pieces of V elements a thread, and walks over the rows.  With 16-byte
// pieces every thread copies its pieces of the next row into shared memory (its own slots: nothing is synchronised) as
// soon as all of this row's are in registers.
template <class T, int V, int P, bool GRAD, bool POST, int MAXT, int CTAS>
__global__ void __launch_bounds__(MAXT, CTAS) norm_kernel(const NormArgs a)
{
    griddep_enter();
    constexpr int NIN = GRAD ? (POST ? 5 : 3) : (POST ? 3 : 1);
    constexpr bool RING = norm_ring<V, NIN * P * MAXT>();
    extern __shared__ uint4 ring[];
    __shared__ float buf[2 * 32 * 3];
    const int group = a.group, g = (int)threadIdx.x / group, t = (int)threadIdx.x - g * group;
    const int per = (int)blockDim.x / group, pieces = a.D / V;
    int turn = 0;
    // the inputs in the order of their slots, NULL where there is none
    const void *src[NIN];
    int64_t ld[NIN];
    if constexpr (GRAD) {
        src[0] = a.dn, ld[0] = a.ld_dn;
        src[1] = a.hin, ld[1] = a.ld_hin;
        src[2] = a.dh, ld[2] = a.ld_dh;
        if constexpr (POST) {
            src[3] = a.y, ld[3] = a.ld_y;
            src[4] = a.gate_kind == NORM_GATE_FULL ? a.gate : nullptr, ld[4] = a.ld_gate;
        }
    } else {
        src[0] = a.y, ld[0] = a.ld_y;
        if constexpr (POST) {
            src[1] = a.res, ld[1] = a.ld_res;
            src[2] = a.gate_kind == NORM_GATE_FULL ? a.gate : nullptr, ld[2] = a.ld_gate;
        }
    }
    auto piece = [&](int p) { return p * group + t; };
    auto slot = [&](int k, int p) { return ring + (k * P + p) * blockDim.x + threadIdx.x; };
    auto fetch = [&](int64_t row) {
        if constexpr (RING) {
            if (row < a.rows) {
#pragma unroll
                for (int k = 0; k < NIN; ++k)
                    if (src[k])
#pragma unroll
                        for (int p = 0; p < P; ++p)
                            if (piece(p) < pieces) norm_cp16(slot(k, p), static_cast<const T *>(src[k]) + row * ld[k] + piece(p) * V);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    float acc[GRAD ? 2 : 1][GRAD ? P * V : 1] = {};
    const int64_t step = (int64_t)gridDim.x * per;
    fetch((int64_t)blockIdx.x * per + g);
    for (int64_t base = (int64_t)blockIdx.x * per; base < a.rows; base += step) {
        const int64_t row = base + g;
        const bool on = row < a.rows;
        Vec<T, V> in[NIN][P] = {};
        if constexpr (RING) asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
        for (int k = 0; k < NIN; ++k)
            if (src[k] && on)
#pragma unroll
                for (int p = 0; p < P; ++p)
                    if (piece(p) < pieces) {
                        if constexpr (RING) in[k][p] = *reinterpret_cast<const Vec<T, V> *>(slot(k, p));
                        else in[k][p] = *reinterpret_cast<const Vec<T, V> *>(static_cast<const T *>(src[k]) + row * ld[k] + piece(p) * V);
                    }
        const float row_gate = POST && a.gate_kind == NORM_GATE_ROW && on ? static_cast<const float *>(a.gate)[row] : 1.0f;
        auto put = [&](void *out, int64_t ldo, int p, const Vec<T, V> &v) {
            if (on && piece(p) < pieces) *reinterpret_cast<Vec<T, V> *>(static_cast<T *>(out) + row * ldo + piece(p) * V) = v;
        };
        if constexpr (!GRAD) {
            float ss[1] = {};
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int j = 0; j < V; j += 2) {
                    const float2 y = in[0][p].get2(j);
                    ss[0] = fmaf(y.x, y.x, fmaf(y.y, y.y, ss[0]));
                }
            row_sum(ss, group, buf, turn);
            fetch(row + step);
            float r = rsqrtf(fmaf(ss[0], a.inv_d, a.eps));
            if constexpr (POST) {
                float h[P][V];
                float s2[1] = {};
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    float gain[V];
                    if (piece(p) < pieces) load_gain<T, V>(a.gain, a.gain_f32, piece(p) * V, gain);
                    Vec<T, V> o;
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        const int k = V == 1 ? 0 : j + 1;
                        const float2 y = in[0][p].get2(j), x = in[1][p].get2(j), m = in[2][p].get2(j);
                        const bool full = a.gate_kind == NORM_GATE_FULL;
                        const float h1 = fmaf(a.scale, x.y, (full ? m.y : row_gate) * (y.y * r * gain[k]));
                        h[p][k] = h1;
                        h[p][j] = fmaf(a.scale, x.x, (full ? m.x : row_gate) * (y.x * r * gain[j]));
                        o.set2(j, h[p][j], h1);
                        if (piece(p) < pieces) s2[0] = fmaf(h[p][j], h[p][j], V > 1 ? fmaf(h1, h1, s2[0]) : s2[0]);
                    }
                    put(a.h, a.ld_h, p, o);
                }
                if (a.next) {
                    row_sum(s2, group, buf, turn);
                    r = rsqrtf(fmaf(s2[0], a.inv_d, a.eps));
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        float gain[V];
                        if (piece(p) < pieces) load_gain<T, V>(a.next_gain, a.gain_f32, piece(p) * V, gain);
                        Vec<T, V> o;
#pragma unroll
                        for (int j = 0; j < V; j += 2) {
                            const int k = V == 1 ? 0 : j + 1;
                            o.set2(j, h[p][j] * r * gain[j], h[p][k] * r * gain[k]);
                        }
                        put(a.n, a.ld_n, p, o);
                    }
                }
            } else {
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    float gain[V];
                    if (piece(p) < pieces) load_gain<T, V>(a.next_gain, a.gain_f32, piece(p) * V, gain);
                    Vec<T, V> o;
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        const int k = V == 1 ? 0 : j + 1;
                        const float2 x = in[0][p].get2(j);
                        o.set2(j, x.x * r * gain[j], x.y * r * gain[k]);
                    }
                    put(a.n, a.ld_n, p, o);
                }
            }
        } else {
            // mean squares of h and y, and <next_gain dn, h>
            float s[3] = {};
#pragma unroll
            for (int p = 0; p < P; ++p) {
                if (a.next) {
                    float gain[V];
                    if (piece(p) < pieces) load_gain<T, V>(a.next_gain, a.gain_f32, piece(p) * V, gain);
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        const float2 d = in[0][p].get2(j), h = in[1][p].get2(j);
                        s[0] = fmaf(h.x, h.x, fmaf(h.y, h.y, s[0]));
                        if (piece(p) < pieces) s[1] = fmaf(d.x * gain[j], h.x, V > 1 ? fmaf(d.y * gain[(j + 1) % V], h.y, s[1]) : s[1]);
                    }
                }
                if constexpr (POST)
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        const float2 y = in[3][p].get2(j);
                        s[2] = fmaf(y.x, y.x, fmaf(y.y, y.y, s[2]));
                    }
            }
            row_sum(s, group, buf, turn);
            fetch(row + step);
            const float rh = a.next ? rsqrtf(fmaf(s[0], a.inv_d, a.eps)) : 0.0f, mh = s[1] * a.inv_d * rh * rh;
            const float ry = POST ? rsqrtf(fmaf(s[2], a.inv_d, a.eps)) : 0.0f;
            float u[1] = {};
            float gt[POST ? P : 1][V];                   // gain t, before the gate
#pragma unroll
            for (int p = 0; p < P; ++p) {
                float gain[V], post[V];
                if (a.next && piece(p) < pieces) load_gain<T, V>(a.next_gain, a.gain_f32, piece(p) * V, gain);
                if (POST && piece(p) < pieces) load_gain<T, V>(a.gain, a.gain_f32, piece(p) * V, post);
                Vec<T, V> o, og;
#pragma unroll
                for (int j = 0; j < V; j += 2) {
                    float w[2], wg[2] = {};
                    const float2 d = in[0][p].get2(j), h = in[1][p].get2(j), e = in[2][p].get2(j);
#pragma unroll
                    for (int i = 0; i < (V == 1 ? 1 : 2); ++i) {
                        float v = i ? e.y : e.x;
                        if (a.next) {
                            const float dn = i ? d.y : d.x, hv = i ? h.y : h.x;
                            v += rh * fmaf(-hv, mh, dn * gain[j + i]);
                            acc[1][p * V + j + i] = fmaf(dn, hv * rh, acc[1][p * V + j + i]);
                        }
                        if constexpr (POST) {
                            const float2 yy = in[3][p].get2(j), mm = in[4][p].get2(j);
                            const float yh = (i ? yy.y : yy.x) * ry, m = a.gate_kind == NORM_GATE_FULL ? (i ? mm.y : mm.x) : row_gate;
                            w[i] = a.scale * v;
                            acc[0][p * V + j + i] = fmaf(m * v, yh, acc[0][p * V + j + i]);
                            if (piece(p) < pieces) {
                                const float q = post[j + i] * v;
                                wg[i] = q * yh;
                                const float c = a.gate_kind == NORM_GATE_FULL ? m * q : q;
                                gt[p][j + i] = c;
                                u[0] = fmaf(c, yh, u[0]);
                            }
                        } else {
                            w[i] = v;
                        }
                    }
                    o.set2(j, w[0], V == 1 ? 0.0f : w[1 % (V == 1 ? 1 : 2)]);
                    if (POST) og.set2(j, wg[0], wg[1]);
                }
                put(a.n, a.ld_n, p, o);
                if (POST && a.gate_kind == NORM_GATE_FULL) put(a.dgate, a.ld_dgate, p, og);
            }
            if constexpr (POST) {
                row_sum(u, group, buf, turn);
                if (a.gate_kind == NORM_GATE_ROW && t == 0 && on) static_cast<float *>(a.dgate)[row] = u[0];
                const float m = u[0] * a.inv_d * ry, f = a.gate_kind == NORM_GATE_ROW ? row_gate * ry : ry;
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    Vec<T, V> o;
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        const int k = V == 1 ? 0 : j + 1;
                        const float2 y = in[3][p].get2(j);
                        o.set2(j, f * fmaf(-y.x, m, gt[p][j]), f * fmaf(-y.y, m, gt[p][k]));
                    }
                    put(a.h, a.ld_h, p, o);
                }
            }
        }
    }
    if constexpr (GRAD) {
        // rows that are not there added nothing
        const int64_t groups = (int64_t)gridDim.x * per, mine = (int64_t)blockIdx.x * per + g;
#pragma unroll
        for (int k = POST ? 0 : 1; k < 2; ++k) {
            if (k == 1 && !a.next) break;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                if (piece(p) >= pieces) continue;
                float *o = a.part + (k * groups + mine) * a.D + piece(p) * V;
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = acc[k][p * V + j];
            }
        }
    }
}

// Column sums of the row groups' parts, in a fixed order: 32 columns a CTA, 16 rows of threads.
__global__ void __launch_bounds__(512) norm_gain_kernel(const float *part, int groups, int D, float *dgain, float *dnext)
{
    griddep_enter();
    __shared__ float s[16][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = (int)blockIdx.x * 32 + x;
    float *out = blockIdx.y ? dnext : dgain;
    const float *p = part + (int64_t)blockIdx.y * groups * D;
    float v = 0.0f;
    if (out && c < D)
        for (int i = y; i < groups; i += 16) v += p[(int64_t)i * D + c];
    s[y][x] = v;
    __syncthreads();
    if (out && y == 0 && c < D) {
#pragma unroll
        for (int i = 1; i < 16; ++i) v += s[i][x];
        out[c] = v;
    }
}

// Threads a row and rows a CTA: 16 elements a thread (a warp where a row has at most 512).
constexpr int NORM_ELEMS = 16;
static int norm_group(int D) { return std::max(32, (int)(((int64_t)D + 32 * NORM_ELEMS - 1) / (32 * NORM_ELEMS)) * 32); }
static int norm_rows(int group) { return group >= 128 ? 1 : 256 / group; }
// Row groups of a gradient's grid at most, each with sums of its own.
static int64_t norm_groups(int64_t rows, int D)
{
    const int per = norm_rows(norm_group(D));
    return std::min<int64_t>((rows + per - 1) / per, per > 1 ? 304 : 608) * per;
}

template <class T, int V, bool GRAD, bool POST, int MAXT>
static int launch_norm(NormArgs a, float *dgain, float *dnext, cudaStream_t st)
{
    constexpr int P = NORM_ELEMS / V;
    constexpr int NIN = GRAD ? (POST ? 5 : 3) : (POST ? 3 : 1);
    constexpr int CTAS = GRAD || MAXT > 512 ? 1 : 2;
    auto kern = norm_kernel<T, V, P, GRAD, POST, MAXT, CTAS>;
    const int per = norm_rows(a.group), threads = a.group * per, sms = k3_num_sms();
    if (!sms) return K3MOE_ERR_CUDA;
    constexpr bool RING = norm_ring<V, NIN * P * MAXT>();
    const int smem = RING ? NIN * P * threads * 16 : 0;
    static unsigned long long attr_set = 0;
    if (RING && !k3_smem_attr(kern, NIN * P * MAXT * 16, attr_set)) return K3MOE_ERR_CUDA;
    static int fits[33] = {};                            // CTAs an SM by warps a row
    int fit = fits[a.group / 32];
    if (!fit) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kern, threads, smem) != cudaSuccess || fit < 1) return K3MOE_ERR_CUDA;
        fits[a.group / 32] = fit;
    }
    int64_t grid = std::min<int64_t>(((int64_t)a.rows + per - 1) / per, (int64_t)fit * sms);
    if (GRAD) grid = std::min<int64_t>(grid, norm_groups(a.rows, a.D) / per);
    if (grid > 0) {
        k3_launch(kern, dim3((unsigned)grid), threads, smem, st, a);
        k3_note_launch();
    }
    if (GRAD && ((POST && dgain) || (a.next && dnext))) {
        k3_launch(norm_gain_kernel, dim3((unsigned)((a.D + 31) / 32), 2), 512, 0, st, (const float *)a.part,
                  (int)(grid * per), a.D, POST ? dgain : nullptr, a.next ? dnext : nullptr);
        k3_note_launch();
    }
    return cudaGetLastError() == cudaSuccess ? K3MOE_OK : K3MOE_ERR_CUDA;
}

template <class T, int V, bool GRAD>
static int launch_sized(const NormArgs &a, bool post, float *dgain, float *dnext, cudaStream_t st)
{
    if constexpr (V > 1)
        if (a.group <= 512)
            return post ? launch_norm<T, V, GRAD, true, 512>(a, dgain, dnext, st) : launch_norm<T, V, GRAD, false, 512>(a, dgain, dnext, st);
    return post ? launch_norm<T, V, GRAD, true, 1024>(a, dgain, dnext, st) : launch_norm<T, V, GRAD, false, 1024>(a, dgain, dnext, st);
}

template <bool GRAD>
static int launch_typed(NormArgs a, bool post, int dtype, bool vec, float *dgain, float *dnext, cudaStream_t st)
{
    a.group = norm_group(a.D);
    a.inv_d = 1.0f / (float)a.D;
    if (dtype == K3MOE_TYPE_F32)
        return vec ? launch_sized<float, 4, GRAD>(a, post, dgain, dnext, st) : launch_sized<float, 1, GRAD>(a, post, dgain, dnext, st);
    if (dtype == K3MOE_TYPE_BF16)
        return vec ? launch_sized<__nv_bfloat16, 8, GRAD>(a, post, dgain, dnext, st)
                   : launch_sized<__nv_bfloat16, 1, GRAD>(a, post, dgain, dnext, st);
    return vec ? launch_sized<__half, 8, GRAD>(a, post, dgain, dnext, st) : launch_sized<__half, 1, GRAD>(a, post, dgain, dnext, st);
}

// Checks shared by the calls.
struct NormMatrix {
    const void *p;
    int64_t ld;
    bool out, wanted;
};
static int norm_check(int rows, int D, int dtype, int gain_dtype, float eps, std::initializer_list<NormMatrix> ms, bool &vec)
{
    if (rows < 0 || D < 1 || !(eps > 0.0f && eps <= 3.0e38f)) return K3MOE_ERR_ARG;
    if (D > K3MOE_NORM_MAX_WIDTH) return K3MOE_ERR_SHAPE;
    if (dtype != K3MOE_TYPE_F32 && dtype != K3MOE_TYPE_BF16 && dtype != K3MOE_TYPE_F16) return K3MOE_ERR_UNSUPPORTED;
    if (gain_dtype != K3MOE_TYPE_F32 && gain_dtype != dtype) return K3MOE_ERR_UNSUPPORTED;
    vec = (D * k3_type_bytes(dtype)) % 16 == 0;
    for (const NormMatrix &m : ms) {
        if (!m.p && (!m.wanted || rows == 0)) continue;
        if (!m.p || m.ld < D) return K3MOE_ERR_ARG;
        vec = vec && k3_rows16(m.p, m.ld, dtype);
        if (!m.out) continue;
        // an output may be an input itself: a row is in registers before any of it is written
        const size_t nb = k3_span(rows, D, m.ld, dtype);
        for (const NormMatrix &o : ms) {
            if (&o == &m || !o.p) continue;
            if (!o.out && o.p == m.p && o.ld == m.ld) continue;
            if (k3_overlap(m.p, nb, o.p, k3_span(rows, D, o.ld, dtype))) return K3MOE_ERR_ALIAS;
        }
    }
    return K3MOE_OK;
}
// Vectors (gains, row gates, gradients' sums, workspace) apart from every output.
struct NormVector {
    const void *p;
    size_t bytes;
    bool out;
};
static bool norm_apart(int rows, int D, int dtype, std::initializer_list<NormMatrix> ms, std::initializer_list<NormVector> vs)
{
    for (const NormVector &v : vs) {
        if (!v.p) continue;
        for (const NormMatrix &m : ms)
            if (m.p && (m.out || v.out) && k3_overlap(v.p, v.bytes, m.p, k3_span(rows, D, m.ld, dtype))) return false;
        for (const NormVector &w : vs)
            if (&w != &v && w.p && (w.out || v.out) && k3_overlap(v.p, v.bytes, w.p, w.bytes)) return false;
    }
    return true;
}
static bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace k3

using namespace k3;

extern "C" int k3moe_rms_norm(const void *x, int64_t ldx, const void *gain, int gain_dtype, float eps, int rows, int D,
                              int dtype, void *out, int64_t ldo, cudaStream_t stream)
{
    bool vec = false;
    const std::initializer_list<NormMatrix> ms = {{x, ldx, false, true}, {out, ldo, true, true}};
    const int rc = norm_check(rows, D, dtype, gain_dtype, eps, ms, vec);
    if (rc) return rc;
    if (!norm_apart(rows, D, dtype, ms, {{gain, (size_t)D * k3_type_bytes(gain_dtype), false}})) return K3MOE_ERR_ALIAS;
    if (rows == 0) return K3MOE_OK;
    NormArgs a = {};
    a.y = x, a.ld_y = ldx;
    a.next_gain = gain, a.gain_f32 = gain_dtype == K3MOE_TYPE_F32, a.next = 1;
    a.eps = eps, a.rows = rows, a.D = D;
    a.n = out, a.ld_n = ldo;
    return launch_typed<false>(a, false, dtype, vec && aligned16(gain), nullptr, nullptr, stream);
}

extern "C" int k3moe_norm_residual(const void *y, int64_t ldy, const void *residual, int64_t ldr, const void *gain,
                                   const void *next_gain, int gain_dtype, const void *gate, int64_t ldgate, int gate_kind,
                                   float residual_scale, float eps, int rows, int D, int dtype, void *h, int64_t ldh, void *n,
                                   int64_t ldn, cudaStream_t stream)
{
    if (gate_kind != NORM_GATE_NONE && gate_kind != NORM_GATE_ROW && gate_kind != NORM_GATE_FULL) return K3MOE_ERR_ARG;
    if ((gate_kind == NORM_GATE_NONE) != !gate && (gate || rows > 0)) return K3MOE_ERR_ARG;
    const bool full = gate_kind == NORM_GATE_FULL;
    bool vec = false;
    const std::initializer_list<NormMatrix> ms = {{y, ldy, false, true}, {residual, ldr, false, true},
                                                  {full ? gate : nullptr, ldgate, false, full}, {h, ldh, true, true},
                                                  {n, ldn, true, false}};
    const int rc = norm_check(rows, D, dtype, gain_dtype, eps, ms, vec);
    if (rc) return rc;
    const size_t ng = (size_t)D * k3_type_bytes(gain_dtype);
    if (!norm_apart(rows, D, dtype, ms, {{gain, ng, false}, {next_gain, ng, false},
                                         {gate_kind == NORM_GATE_ROW ? gate : nullptr, (size_t)rows * 4, false}}))
        return K3MOE_ERR_ALIAS;
    if (rows == 0) return K3MOE_OK;
    NormArgs a = {};
    a.y = y, a.ld_y = ldy;
    a.res = residual, a.ld_res = ldr;
    a.gate = gate, a.ld_gate = ldgate, a.gate_kind = gate_kind;
    a.gain = gain, a.next_gain = next_gain, a.gain_f32 = gain_dtype == K3MOE_TYPE_F32, a.next = n != nullptr;
    a.scale = residual_scale, a.eps = eps, a.rows = rows, a.D = D;
    a.h = h, a.ld_h = ldh;
    a.n = n, a.ld_n = ldn;
    return launch_typed<false>(a, true, dtype, vec && aligned16(gain) && aligned16(next_gain), nullptr, nullptr, stream);
}

extern "C" size_t k3moe_norm_grad_workspace_bytes(int rows, int D)
{
    return rows < 0 || D < 1 || D > K3MOE_NORM_MAX_WIDTH ? 0 : (size_t)std::max<int64_t>(1, norm_groups(rows, D)) * D * 2 * sizeof(float);
}

extern "C" int k3moe_rms_norm_grad(const void *dy, int64_t lddy, const void *x, int64_t ldx, const void *gain, int gain_dtype,
                                   const void *add, int64_t ldadd, float eps, int rows, int D, int dtype, void *dx,
                                   int64_t lddx, float *dgain, void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    bool vec = false;
    const std::initializer_list<NormMatrix> ms = {{dy, lddy, false, true}, {x, ldx, false, true}, {add, ldadd, false, false},
                                                  {dx, lddx, true, true}};
    const int rc = norm_check(rows, D, dtype, gain_dtype, eps, ms, vec);
    if (rc) return rc;
    const size_t need = k3moe_norm_grad_workspace_bytes(rows, D);
    if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 3)) return K3MOE_ERR_WORKSPACE;
    if (!norm_apart(rows, D, dtype, ms, {{gain, (size_t)D * k3_type_bytes(gain_dtype), false}, {dgain, (size_t)D * 4, true},
                                         {workspace, need, true}}))
        return K3MOE_ERR_ALIAS;
    NormArgs a = {};
    a.dn = dy, a.ld_dn = lddy;
    a.hin = x, a.ld_hin = ldx;
    a.dh = add, a.ld_dh = ldadd;
    a.next_gain = gain, a.gain_f32 = gain_dtype == K3MOE_TYPE_F32, a.next = 1;
    a.eps = eps, a.rows = rows, a.D = D;
    a.n = dx, a.ld_n = lddx;
    a.part = static_cast<float *>(workspace);
    return launch_typed<true>(a, false, dtype, vec && aligned16(gain), nullptr, dgain, stream);
}

extern "C" int k3moe_norm_residual_grad(const void *dh, int64_t lddh, const void *dn, int64_t lddn, const void *y, int64_t ldy,
                                        const void *h, int64_t ldh, const void *gain, const void *next_gain, int gain_dtype,
                                        const void *gate, int64_t ldgate, int gate_kind, float residual_scale, float eps,
                                        int rows, int D, int dtype, void *dy, int64_t lddy, void *dresidual, int64_t lddr,
                                        void *dgate, int64_t lddgate, float *dgain, float *dnext_gain, void *workspace,
                                        size_t workspace_bytes, cudaStream_t stream)
{
    if (gate_kind != NORM_GATE_NONE && gate_kind != NORM_GATE_ROW && gate_kind != NORM_GATE_FULL) return K3MOE_ERR_ARG;
    const bool full = gate_kind == NORM_GATE_FULL, by_row = gate_kind == NORM_GATE_ROW;
    if ((gate_kind == NORM_GATE_NONE) != !gate && (gate || rows > 0)) return K3MOE_ERR_ARG;
    if ((gate_kind == NORM_GATE_NONE) != !dgate && (dgate || rows > 0)) return K3MOE_ERR_ARG;
    if (rows > 0 && !dh && !dn) return K3MOE_ERR_ARG;
    if (rows > 0 && !dn && dnext_gain) return K3MOE_ERR_ARG;
    bool vec = false;
    const std::initializer_list<NormMatrix> ms = {
        {dh, lddh, false, false}, {dn, lddn, false, false}, {y, ldy, false, true}, {h, ldh, false, dn != nullptr},
        {full ? gate : nullptr, ldgate, false, full}, {dy, lddy, true, true}, {dresidual, lddr, true, true},
        {full ? dgate : nullptr, lddgate, true, full}};
    const int rc = norm_check(rows, D, dtype, gain_dtype, eps, ms, vec);
    if (rc) return rc;
    const size_t need = k3moe_norm_grad_workspace_bytes(rows, D);
    if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 3)) return K3MOE_ERR_WORKSPACE;
    const size_t ng = (size_t)D * k3_type_bytes(gain_dtype);
    if (!norm_apart(rows, D, dtype, ms, {{gain, ng, false}, {next_gain, ng, false}, {by_row ? gate : nullptr, (size_t)rows * 4, false},
                                         {by_row ? dgate : nullptr, (size_t)rows * 4, true}, {dgain, (size_t)D * 4, true},
                                         {dnext_gain, (size_t)D * 4, true}, {workspace, need, true}}))
        return K3MOE_ERR_ALIAS;
    NormArgs a = {};
    a.dh = dh, a.ld_dh = lddh;
    a.dn = dn, a.ld_dn = lddn;
    a.y = y, a.ld_y = ldy;
    a.hin = dn ? h : nullptr, a.ld_hin = ldh;
    a.gate = gate, a.ld_gate = ldgate, a.gate_kind = gate_kind;
    a.gain = gain, a.next_gain = next_gain, a.gain_f32 = gain_dtype == K3MOE_TYPE_F32, a.next = dn || dnext_gain;
    a.scale = residual_scale, a.eps = eps, a.rows = rows, a.D = D;
    a.h = dy, a.ld_h = lddy;
    a.n = dresidual, a.ld_n = lddr;
    a.dgate = dgate, a.ld_dgate = lddgate;
    a.part = static_cast<float *>(workspace);
    return launch_typed<true>(a, true, dtype, vec && aligned16(gain) && aligned16(next_gain), dgain, dnext_gain, stream);
}
