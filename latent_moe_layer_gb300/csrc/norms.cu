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
//
// One read of every input, one write of every output: HBM should bind, and does forwards (8192 x 7168 bf16 with an
// elementwise gate and the next norm: 95-99 us, 5.9-6.2 TB/s; 16,384 x 3584: 92 us).  The gradient (162 and 156 us, 5.8 and
// 6.0 TB/s) is near what its instructions take: two dependent sums a row over all of a CTA's warps, some 450 warp
// instructions for eight elements of five inputs.  16 rows of 7168 take 6 us, a launch.
#include "glu.cuh"

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
    float *part;                                         // [dgain, dnext_gain][CTAs][D]
};

__device__ __forceinline__ void norm_cp16(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
                 : "memory");
}

// V elements from column c of a row of D.  LOOSE: element by element, zeros past the row's end.
template <class T, int V, bool LOOSE>
__device__ __forceinline__ Vec<T, V> load_piece(const T *row, int c, int D)
{
    if constexpr (!LOOSE) return *reinterpret_cast<const Vec<T, V> *>(row + c);
    Vec<T, V> v = {};
#pragma unroll
    for (int j = 0; j < V; j += 2) {
        const float x = c + j < D ? to_f32(row[c + j]) : 0.0f, y = c + j + 1 < D ? to_f32(row[c + j + 1]) : 0.0f;
        v.set2(j, x, y);                                     // (exact: the type's own values)
    }
    return v;
}
template <class T, int V, bool LOOSE>
__device__ __forceinline__ void store_piece(T *row, int c, int D, const Vec<T, V> &v)
{
    if constexpr (!LOOSE) {
        *reinterpret_cast<Vec<T, V> *>(row + c) = v;
    } else {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            const float2 e = v.get2(j);
            if (c + j < D) row[c + j] = from_f32<T>(e.x);
            if (c + j + 1 < D) row[c + j + 1] = from_f32<T>(e.y);
        }
    }
}

// V gains from column c; any gain past the last.
template <class T, int V, bool LOOSE>
__device__ __forceinline__ void load_gain(const void *p, int f32, int c, int D, F2 (&g)[V / 2])
{
    if (!p) {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) g[j] = f2(1.0f);
    } else if (LOOSE) {
        auto at = [&](int i) {
            i = min(i, D - 1);
            return f32 ? static_cast<const float *>(p)[i] : to_f32(static_cast<const T *>(p)[i]);
        };
#pragma unroll
        for (int j = 0; j < V / 2; ++j) g[j] = {at(c + 2 * j), at(c + 2 * j + 1)};
    } else if (f32) {
        const float *q = static_cast<const float *>(p) + c;
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            const float4 x = __ldg(reinterpret_cast<const float4 *>(q + j));
            g[j / 2] = {x.x, x.y}, g[j / 2 + 1] = {x.z, x.w};
        }
    } else {
        const Vec<T, V> x = *reinterpret_cast<const Vec<T, V> *>(static_cast<const T *>(p) + c);
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            const float2 e = x.get2(j);
            g[j / 2] = {e.x, e.y};
        }
    }
}
template <class T, int V>
__device__ __forceinline__ F2 pair_of(const Vec<T, V> &v, int j)
{
    const float2 e = v.get2(j);
    return {e.x, e.y};
}
__device__ __forceinline__ F2 neg2(F2 a) { return {-a.x, -a.y}; }

// Sums of N values over a warp, all of them at once: the lanes split over the values as they halve (6 shuffles for four
// values instead of 20).  Value i is left in lanes 8 i .. 8 i + 7 (N = 1: in all).
template <int N>
__device__ __forceinline__ float warp_sums(const float (&v)[N], int lane)
{
    float k;
    if constexpr (N == 1) {
        k = v[0];
        k += __shfl_xor_sync(0xffffffffu, k, 16);
        k += __shfl_xor_sync(0xffffffffu, k, 8);
    } else {
        const float v2 = N > 2 ? v[N > 2 ? 2 : 0] : 0.0f, v3 = N > 3 ? v[N > 3 ? 3 : 0] : 0.0f;
        const bool high = lane & 16, odd = lane & 8;
        const float k0 = (high ? v2 : v[0]) + __shfl_xor_sync(0xffffffffu, high ? v[0] : v2, 16);
        const float k1 = (high ? v3 : v[1]) + __shfl_xor_sync(0xffffffffu, high ? v[1] : v3, 16);
        k = (odd ? k1 : k0) + __shfl_xor_sync(0xffffffffu, odd ? k0 : k1, 8);
    }
    k += __shfl_xor_sync(0xffffffffu, k, 4);
    k += __shfl_xor_sync(0xffffffffu, k, 2);
    k += __shfl_xor_sync(0xffffffffu, k, 1);
    return k;
}
template <int N>
__device__ __forceinline__ void spread_sums(float k, float (&v)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = N == 1 ? k : __shfl_sync(0xffffffffu, k, 8 * i);
}

// Sums over the threads of a row (its warps of the CTA, all of them in the same order: every thread gets the same bits).
// Two buffers in turn, so that one barrier a sum is enough.
template <bool ONE, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int group, float4 *buf, int &turn)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (!ONE && group < 32) {
        for (int o = group >> 1; o; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        return;
    }
    float k = warp_sums(v, lane);
    if (ONE || group > 32) {
        const int warps = group >> 5, first = ONE ? 0 : (int)threadIdx.x / group * warps;
        float4 *b = buf + turn * 32;
        turn ^= 1;
        if (N == 1 ? lane == 0 : (lane & 7) == 0) reinterpret_cast<float *>(b + warp)[N == 1 ? 0 : lane >> 3] = k;
        __syncthreads();
        float w[N] = {};
        if (lane < warps) {
            const float4 q = b[first + lane];
            w[0] = q.x;
            if constexpr (N > 1) w[1] = q.y;
            if constexpr (N > 2) w[2] = q.z;
            if constexpr (N > 3) w[3] = q.w;
        }
        k = warp_sums(w, lane);
    }
    spread_sums(k, v);
}

// The inputs in the order of their slots, NULL where there is none: read from the arguments (constant memory) where they are
// used, as registers are what a gradient is short of.
template <bool GRAD>
__device__ __forceinline__ const void *norm_src(const NormArgs &a, int k)
{
    if (GRAD) return k == 0 ? a.dn : k == 1 ? a.hin : k == 2 ? a.dh : k == 3 ? a.y : a.gate_kind == NORM_GATE_FULL ? a.gate : nullptr;
    return k == 0 ? a.y : k == 1 ? a.res : a.gate_kind == NORM_GATE_FULL ? a.gate : nullptr;
}
template <bool GRAD>
__device__ __forceinline__ int64_t norm_ld(const NormArgs &a, int k)
{
    if (GRAD) return k == 0 ? a.ld_dn : k == 1 ? a.ld_hin : k == 2 ? a.ld_dh : k == 3 ? a.ld_y : a.ld_gate;
    return k == 0 ? a.ld_y : k == 1 ? a.ld_res : a.ld_gate;
}

// Whether the rows of a call follow each other through steps of their own (see the gradient's loop); its gains are kept in
// shared memory, as the two rows' pieces leave the L1 too little room for them (`slots`, `gains`: bytes of either).
constexpr bool norm_piped(bool grad, bool post, bool one, int slots, int gains)
{
    return grad && post && one && 2 * slots + gains + 1024 <= kMaxSmem;
}
// Rows' pieces that a thread keeps in flight in shared memory: two rows where they fit, else one or none (wide fp32 rows).
template <bool LOOSE, int BYTES>
constexpr int norm_slots() { return LOOSE ? 0 : std::min(2, (kMaxSmem - 1024) / BYTES); }

// A group of threads holds a row, P pieces of V elements a thread, and walks over the rows (ONE: the group is the CTA, so that
// rows' addresses are the same for all its threads).  With 16-byte pieces every thread copies its pieces of the next row into
// shared memory (its own slots: nothing is synchronised): with two slots while this row is worked on, with one when all
// of this row's pieces have been used (a slot is never written while a load of it may be under way).
template <class T, int V, int P, bool GRAD, bool POST, int MAXT, int CTAS, bool ONE, bool LOOSE>
__global__ void __launch_bounds__(MAXT, CTAS) norm_kernel(const NormArgs a)
{
    griddep_enter();
    constexpr int NIN = GRAD ? (POST ? 5 : 3) : (POST ? 3 : 1), H = V / 2;
    constexpr int SLOTS = norm_slots<LOOSE, NIN * P * MAXT * 16>();
    constexpr bool PIPED = !LOOSE && norm_piped(GRAD, POST, ONE, NIN * P * MAXT * 16, 2 * P * V * MAXT * 4);
    extern __shared__ uint4 ring[];
    __shared__ float4 buf[2 * 32];
    const int group = ONE ? (int)blockDim.x : a.group, g = ONE ? 0 : (int)threadIdx.x / group, t = (int)threadIdx.x - g * group;
    const int per = ONE ? 1 : (int)blockDim.x / group, pieces = (a.D + V - 1) / V;
    int turn = 0;
    auto piece = [&](int p) { return p * group + t; };
    auto gain_at = [&](int p) { return min(piece(p), pieces - 1) * V; };         // any gain where the elements are zeros
    // PIPED: this thread's gains (0: gain, 1: next_gain), after the slots
    auto gain_slot = [&](int k, int p, int q) {
        return reinterpret_cast<float4 *>(ring + 2 * NIN * P * blockDim.x) + ((k * P + p) * (V / 4) + q) * blockDim.x + threadIdx.x;
    };
    auto gains = [&](int k, int p, F2 (&g)[H]) {
        if constexpr (PIPED) {
#pragma unroll
            for (int q = 0; q < V / 4; ++q) {
                const float4 x = *gain_slot(k, p, q);
                g[2 * q] = {x.x, x.y}, g[2 * q + 1] = {x.z, x.w};
            }
        } else {
            load_gain<T, V, LOOSE>(k ? a.next_gain : a.gain, a.gain_f32, gain_at(p), a.D, g);
        }
    };
    auto slot = [&](int s, int k, int p) { return ring + ((s * NIN + k) * P + p) * blockDim.x + threadIdx.x; };
    auto fetch = [&](int64_t row, int s) {
        if (row < a.rows) {
#pragma unroll
            for (int k = 0; k < NIN; ++k)
                if (norm_src<GRAD>(a, k))
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        if (piece(p) < pieces) norm_cp16(slot(s, k, p), static_cast<const T *>(norm_src<GRAD>(a, k)) + row * norm_ld<GRAD>(a, k) + piece(p) * V);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    F2 acc[GRAD ? 2 : 1][GRAD ? P : 1][H] = {};
    const int64_t step = (int64_t)gridDim.x * per;
    const bool full = POST && a.gate_kind == NORM_GATE_FULL;
    auto put = [&](bool on, int64_t row, void *out, int64_t ldo, int p, const Vec<T, V> &v) {
        if (on && piece(p) < pieces) store_piece<T, V, LOOSE>(static_cast<T *>(out) + row * ldo, piece(p) * V, a.D, v);
    };
    auto gate_of = [&](int64_t row, bool on) {
        return POST && a.gate_kind == NORM_GATE_ROW && on ? static_cast<const float *>(a.gate)[row] : 1.0f;
    };
    // The gradient's steps on a row whose pieces in(k, p) gives.  Pieces past the row's end are zeros.
    // 1: mean squares of h and y, and <next_gain dn, h>
    auto grad_sums = [&](auto in, float &s0, float &s1, float &s2) {
        F2 hh = f2(0.0f), dh = f2(0.0f), yy = f2(0.0f);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if (a.next) {
                F2 gain[H];
                gains(1, p, gain);
                const Vec<T, V> dv = in(0, p), hv = in(1, p);
#pragma unroll
                for (int j = 0; j < H; ++j) {
                    const F2 h = pair_of(hv, 2 * j);
                    hh = fma2(h, h, hh);
                    dh = fma2(mul2(pair_of(dv, 2 * j), gain[j]), h, dh);
                }
            }
            if constexpr (POST) {
                const Vec<T, V> yv = in(3, p);
#pragma unroll
                for (int j = 0; j < H; ++j) {
                    const F2 y = pair_of(yv, 2 * j);
                    yy = fma2(y, y, yy);
                }
            }
        }
        s0 = hh.x + hh.y, s1 = dh.x + dh.y, s2 = yy.x + yy.y;
    };
    // 2: t, dresidual and dgate (or dx), the gains' sums; gt = gain gate t (a gate by row comes in at the end) and <gt, y'>
    auto grad_middle = [&](auto in, bool on, int64_t row, float rh, float mean, float ry, float row_gate, auto &gt) {
        const F2 rh2 = f2(rh), ry2 = f2(ry), mh = f2(-mean * rh * rh), scale = f2(a.scale), rg = f2(row_gate);
        F2 us = f2(0.0f);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            F2 v[H];
            const Vec<T, V> ev = in(2, p);
#pragma unroll
            for (int j = 0; j < H; ++j) v[j] = pair_of(ev, 2 * j);
            if (a.next) {
                F2 gain[H];
                gains(1, p, gain);
                const Vec<T, V> dv = in(0, p), hv = in(1, p);
#pragma unroll
                for (int j = 0; j < H; ++j) {
                    const F2 dn = pair_of(dv, 2 * j), h = pair_of(hv, 2 * j);
                    v[j] = fma2(rh2, fma2(h, mh, mul2(dn, gain[j])), v[j]);
                    acc[1][p][j] = fma2(dn, mul2(h, rh2), acc[1][p][j]);
                }
            }
            Vec<T, V> o;
            if constexpr (POST) {
                // what follows is loaded after that is done, for its registers
                asm volatile("" ::: "memory");
#pragma unroll
                for (int j = 0; j < H; ++j) {
                    const F2 w = mul2(scale, v[j]);
                    o.set2(2 * j, w.x, w.y);
                }
                put(on, row, a.n, a.ld_n, p, o);
                F2 gain[H];
                gains(0, p, gain);
                const Vec<T, V> yv = in(3, p);
                // (one test a piece: inside the loop both sides would run)
                if (full) {
                    const Vec<T, V> mv = in(4, p);
                    Vec<T, V> og;
#pragma unroll
                    for (int j = 0; j < H; ++j) {
                        const F2 yh = mul2(pair_of(yv, 2 * j), ry2), q = mul2(gain[j], v[j]), m = pair_of(mv, 2 * j);
                        const F2 wg = mul2(q, yh), mv2 = mul2(m, v[j]);
                        og.set2(2 * j, wg.x, wg.y);
                        acc[0][p][j] = fma2(mv2, yh, acc[0][p][j]);
                        gt[p][j] = mul2(m, q);
                        us = fma2(m, wg, us);
                    }
                    put(on, row, a.dgate, a.ld_dgate, p, og);
                } else {
#pragma unroll
                    for (int j = 0; j < H; ++j) {
                        const F2 yh = mul2(pair_of(yv, 2 * j), ry2);
                        acc[0][p][j] = fma2(mul2(rg, v[j]), yh, acc[0][p][j]);
                        gt[p][j] = mul2(gain[j], v[j]);
                        us = fma2(gt[p][j], yh, us);
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < H; ++j) o.set2(2 * j, v[j].x, v[j].y);
                put(on, row, a.n, a.ld_n, p, o);
            }
        }
        return us.x + us.y;
    };
    // 3: dy, and a row's dgate
    auto grad_last = [&](auto in, bool on, int64_t row, float u, float ry, float row_gate, auto &gt) {
        if (a.gate_kind == NORM_GATE_ROW && t == 0 && on) static_cast<float *>(a.dgate)[row] = u;
        const F2 m = f2(-u * a.inv_d * ry), f = f2(row_gate * ry);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const Vec<T, V> yv = in(3, p);
            Vec<T, V> o;
#pragma unroll
            for (int j = 0; j < H; ++j) {
                const F2 d = mul2(f, fma2(pair_of(yv, 2 * j), m, gt[p][j]));
                o.set2(2 * j, d.x, d.y);
            }
            put(on, row, a.h, a.ld_h, p, o);
        }
    };
    F2 gt[GRAD && POST ? P : 1][H];
    if constexpr (SLOTS == 2) {
        // what no copy will write is read as zeros
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
#pragma unroll
            for (int k = 0; k < NIN; ++k)
#pragma unroll
                for (int p = 0; p < P; ++p)
                    if (!norm_src<GRAD>(a, k) || piece(p) >= pieces) *slot(s, k, p) = make_uint4(0, 0, 0, 0);
    }
    if constexpr (PIPED) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int p = 0; p < P; ++p) {
                F2 g[H];
                load_gain<T, V, LOOSE>(k ? a.next_gain : a.gain, a.gain_f32, gain_at(p), a.D, g);
#pragma unroll
                for (int q = 0; q < V / 4; ++q) *gain_slot(k, p, q) = make_float4(g[2 * q].x, g[2 * q].y, g[2 * q + 1].x, g[2 * q + 1].y);
            }
        // Step 1 of the next row goes with step 2 of this one, so that a row costs one barrier and one reduction of all sums.
        auto rows_of = [&](int s) {
            return [&, s](int k, int p) { return *reinterpret_cast<const Vec<T, V> *>(slot(s, k, p)); };
        };
        int64_t row = blockIdx.x;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) fetch(row + s * step, s);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        float s[3];
        grad_sums(rows_of(0), s[0], s[1], s[2]);
        row_sum<ONE>(s, group, buf, turn);
        for (int at = 0; row < a.rows; row += step) {
            const float rh = a.next ? rsqrtf(fmaf(s[0], a.inv_d, a.eps)) : 0.0f, ry = rsqrtf(fmaf(s[2], a.inv_d, a.eps));
            const float row_gate = gate_of(row, true);
            const int next = at ^ 1;
            float w[4];
            w[0] = grad_middle(rows_of(at), true, row, rh, s[1] * a.inv_d, ry, row_gate, gt);
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            grad_sums(rows_of(next), w[1], w[2], w[3]);              // past the last row: whatever the slot holds, unused
            row_sum<ONE>(w, group, buf, turn);
            grad_last(rows_of(at), true, row, w[0], ry, row_gate, gt);
            fetch(row + SLOTS * step, at);
            s[0] = w[1], s[1] = w[2], s[2] = w[3];
            at = next;
        }
    } else {
        int at = 0;                                              // the slot of this row
        if (SLOTS > 0) fetch((int64_t)blockIdx.x * per + g, 0);
        for (int64_t base = (int64_t)blockIdx.x * per; base < a.rows; base += step) {
            const int64_t row = base + g;
            const bool on = ONE || row < a.rows;
            // the row's pieces: in their slot while the next row's are copied into the other, else in registers
            constexpr bool HELD = SLOTS != 2;
            Vec<T, V> held[HELD ? NIN : 1][HELD ? P : 1] = {};
            if constexpr (SLOTS == 2) {
                fetch(row + step, at ^ 1);
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            } else if constexpr (SLOTS == 1) {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            }
            if constexpr (HELD) {
#pragma unroll
                for (int k = 0; k < NIN; ++k)
                    if (norm_src<GRAD>(a, k) && on)
#pragma unroll
                        for (int p = 0; p < P; ++p)
                            if (piece(p) < pieces) {
                                if constexpr (SLOTS > 0) held[k][p] = *reinterpret_cast<const Vec<T, V> *>(slot(0, k, p));
                                else held[k][p] = load_piece<T, V, LOOSE>(static_cast<const T *>(norm_src<GRAD>(a, k)) + row * norm_ld<GRAD>(a, k), piece(p) * V, a.D);
                            }
            }
            auto in = [&](int k, int p) {
                if constexpr (HELD) {
                    return held[k][p];
                } else {
                    Vec<T, V> v = {};
                    if (on) v = *reinterpret_cast<const Vec<T, V> *>(slot(at, k, p));
                    return v;
                }
            };
            const float row_gate = gate_of(row, on);
            if constexpr (!GRAD) {
                F2 sq = f2(0.0f);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const Vec<T, V> yv = in(0, p);
#pragma unroll
                    for (int j = 0; j < H; ++j) {
                        const F2 y = pair_of(yv, 2 * j);
                        sq = fma2(y, y, sq);
                    }
                }
                float ss[1] = {sq.x + sq.y};
                row_sum<ONE>(ss, group, buf, turn);
                float r = rsqrtf(fmaf(ss[0], a.inv_d, a.eps));
                if constexpr (POST) {
                    F2 h[P][H], s2 = f2(0.0f);
                    const F2 scale = f2(a.scale);
                    r *= row_gate;
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        F2 gain[H];
                        gains(0, p, gain);
                        const Vec<T, V> yv = in(0, p), xv = in(1, p);
                        // (one test a piece: inside the loop both sides would run)
#pragma unroll
                        for (int j = 0; j < H; ++j) gain[j] = mul2(gain[j], f2(r));
                        if (full) {
                            const Vec<T, V> mv = in(2, p);
#pragma unroll
                            for (int j = 0; j < H; ++j) gain[j] = mul2(gain[j], pair_of(mv, 2 * j));
                        }
                        Vec<T, V> o;
#pragma unroll
                        for (int j = 0; j < H; ++j) {
                            h[p][j] = fma2(pair_of(yv, 2 * j), gain[j], mul2(scale, pair_of(xv, 2 * j)));
                            o.set2(2 * j, h[p][j].x, h[p][j].y);
                            s2 = fma2(h[p][j], h[p][j], s2);
                        }
                        put(on, row, a.h, a.ld_h, p, o);
                    }
                    if (SLOTS == 1) fetch(row + step, 0);
                    if (a.next) {
                        float s[1] = {s2.x + s2.y};
                        row_sum<ONE>(s, group, buf, turn);
                        r = rsqrtf(fmaf(s[0], a.inv_d, a.eps));
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            F2 gain[H];
                            gains(1, p, gain);
                            Vec<T, V> o;
#pragma unroll
                            for (int j = 0; j < H; ++j) {
                                const F2 n = mul2(mul2(h[p][j], f2(r)), gain[j]);
                                o.set2(2 * j, n.x, n.y);
                            }
                            put(on, row, a.n, a.ld_n, p, o);
                        }
                    }
                } else {
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        F2 gain[H];
                        gains(1, p, gain);
                        const Vec<T, V> xv = in(0, p);
                        Vec<T, V> o;
#pragma unroll
                        for (int j = 0; j < H; ++j) {
                            const F2 n = mul2(mul2(pair_of(xv, 2 * j), f2(r)), gain[j]);
                            o.set2(2 * j, n.x, n.y);
                        }
                        put(on, row, a.n, a.ld_n, p, o);
                    }
                    if (SLOTS == 1) fetch(row + step, 0);
                }
            } else {
                float s[3];
                grad_sums(in, s[0], s[1], s[2]);
                row_sum<ONE>(s, group, buf, turn);
                const float rh = a.next ? rsqrtf(fmaf(s[0], a.inv_d, a.eps)) : 0.0f;
                const float ry = POST ? rsqrtf(fmaf(s[2], a.inv_d, a.eps)) : 0.0f;
                float u[1] = {grad_middle(in, on, row, rh, s[1] * a.inv_d, ry, row_gate, gt)};
                if (SLOTS == 1) fetch(row + step, 0);
                if constexpr (POST) {
                    row_sum<ONE>(u, group, buf, turn);
                    grad_last(in, on, row, u[0], ry, row_gate, gt);
                }
            }
            if (SLOTS == 2) at ^= 1;
        }
    }
    if constexpr (GRAD) {
        // rows that are not there added nothing; a CTA's groups are added up before its sums leave it
        float *all = reinterpret_cast<float *>(ring);
        if constexpr (!ONE) __syncthreads();
#pragma unroll
        for (int k = POST ? 0 : 1; k < 2; ++k) {
            if (k == 1 && !a.next) break;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                if (piece(p) >= pieces) continue;
                float *o = (ONE ? a.part + (k * (int64_t)gridDim.x + blockIdx.x) * a.D : all + (k * per + g) * a.D) + piece(p) * V;
#pragma unroll
                for (int j = 0; j < H; ++j) {
                    if (!LOOSE || piece(p) * V + 2 * j < a.D) o[2 * j] = acc[k][p][j].x;
                    if (!LOOSE || piece(p) * V + 2 * j + 1 < a.D) o[2 * j + 1] = acc[k][p][j].y;
                }
            }
        }
        if constexpr (!ONE) {
            __syncthreads();
            for (int i = threadIdx.x; i < 2 * a.D; i += blockDim.x) {
                const int k = i >= a.D, c = i - k * a.D;
                if (k ? !a.next : !POST) continue;
                float sum = 0.0f;
                for (int q = 0; q < per; ++q) sum += all[(k * per + q) * a.D + c];
                a.part[(k * (int64_t)gridDim.x + blockIdx.x) * a.D + c] = sum;
            }
        }
    }
}

// Column sums of the CTAs' parts, in a fixed order: 32 columns a CTA, 16 rows of threads.
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

// Elements a thread: 16; 8 for norm_residual's gradient up to 8192 columns, which keeps the sums of two gains and more in
// registers.
static int norm_group(int D, int elems)
{
    int n = (D + elems - 1) / elems;
    if (n > 16) return (n + 31) / 32 * 32;
    int group = 4;                                       // a part of a warp
    while (group < n) group *= 2;
    return group;
}
// Threads a row at most where a CTA has several rows.  64, 96 and 128 (67 M elements, bf16): norm_residual_grad of 1024 columns
// 203, 203, 226 us; rms_norm_grad of 768 columns 134, 120, 120, of 1536 146, 112, 111, of 1024 111, 111, 122; norm_residual of
// 1536 columns 106, 111, 111, of 2048 102, 102, 112.
constexpr int NORM_NARROW = 96;
static int norm_rows(int group) { return group > NORM_NARROW ? 1 : 256 / group; }
// CTAs of a gradient's grid at most, each with sums of its own.
static int64_t norm_parts(int64_t rows) { return std::min<int64_t>(rows, 608); }

template <class T, int V, int ELEMS, bool GRAD, bool POST, int MAXT, int CTAS, bool ONE, bool LOOSE>
static int launch_norm(NormArgs a, float *dgain, float *dnext, cudaStream_t st)
{
    constexpr int P = ELEMS / V;
    constexpr int NIN = GRAD ? (POST ? 5 : 3) : (POST ? 3 : 1);
    constexpr int SLOTS = norm_slots<LOOSE, NIN * P * MAXT * 16>();
    a.group = norm_group(a.D, ELEMS);
    const int per = ONE ? 1 : norm_rows(a.group), threads = a.group * per, sms = k3_num_sms();
    auto kern = norm_kernel<T, V, P, GRAD, POST, MAXT, CTAS, ONE, LOOSE>;
    if (!sms) return K3MOE_ERR_CUDA;
    constexpr bool PIPED = !LOOSE && norm_piped(GRAD, POST, ONE, NIN * P * MAXT * 16, 2 * P * V * MAXT * 4);
    constexpr int PER_THREAD = SLOTS * NIN * P * 16 + (PIPED ? 2 * P * V * 4 : 0);
    const int smem = std::max(PER_THREAD * threads, GRAD && !ONE ? 2 * per * a.D * 4 : 0);
    static unsigned long long attr_set = 0;
    if (SLOTS && !k3_smem_attr(kern, PER_THREAD * MAXT, attr_set)) return K3MOE_ERR_CUDA;
    static int fits[33] = {};                            // CTAs an SM by warps of a CTA
    int fit = fits[threads / 32];
    if (!fit) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kern, threads, smem) != cudaSuccess || fit < 1) return K3MOE_ERR_CUDA;
        fits[threads / 32] = fit;
    }
    int64_t grid = std::min<int64_t>(((int64_t)a.rows + per - 1) / per, (int64_t)fit * sms);
    if (GRAD) grid = std::min<int64_t>(grid, norm_parts(a.rows));
    if (grid > 0) {
        k3_launch(kern, dim3((unsigned)grid), threads, smem, st, a);
        k3_note_launch();
    }
    if (GRAD && ((POST && dgain) || (a.next && dnext))) {
        k3_launch(norm_gain_kernel, dim3((unsigned)((a.D + 31) / 32), 2), 512, 0, st, (const float *)a.part,
                  (int)grid, a.D, POST ? dgain : nullptr, a.next ? dnext : nullptr);
        k3_note_launch();
    }
    return cudaGetLastError() == cudaSuccess ? K3MOE_OK : K3MOE_ERR_CUDA;
}

template <class T, int V, bool GRAD, bool POST, bool LOOSE>
static int launch_sized(const NormArgs &a, float *dgain, float *dnext, cudaStream_t st)
{
    auto go = [&](auto elems, auto threads, auto ctas, auto one) {
        return launch_norm<T, V, elems.value, GRAD, POST, threads.value, ctas.value, one.value, LOOSE>(a, dgain, dnext, st);
    };
    using std::integral_constant;
    const integral_constant<int, 8> e8;
    const integral_constant<int, 16> e16;
    const std::true_type one;
    const std::false_type several;
    // (threads, CTAs an SM) that the registers are counted for
    if constexpr (GRAD && POST) {
        // A thread wants 72 registers, so an SM holds 28 warps: two CTAs of at most 14 (448 threads, 3584 columns), which in
        // fp32 leaves room for two rows in shared memory, or one of at most 28 (896 threads, 7168 columns).  Wider rows take
        // 1024 threads of 64 registers, which spill 52 bytes (fp32 72).  67 M elements (fp32 half), 448 | 896 | 1024 threads: bf16 1024
        // columns 203 | 203 | 248 us, 3584: 175 | 175 | 207, 5120: 198 with 896, 218 with 1024, 7168: 182 and 220; fp32 1024
        // columns 172 | 195 | 219, 3584: 170 | 172 | 179, 7168: 183 and 192.  (4096 columns, one CTA of 512 threads where 64
        // registers would hold two: 217 and 200, fp32 196 and 174.)
        if (a.D <= NORM_NARROW * 8) return go(e8, integral_constant<int, 256>(), integral_constant<int, 3>(), several);
        if constexpr (!LOOSE) {
            if (a.D <= 3584) return go(e8, integral_constant<int, 448>(), integral_constant<int, 2>(), one);
            if (a.D <= 7168) return go(e8, integral_constant<int, 896>(), integral_constant<int, 1>(), one);
        }
        if (a.D <= 8192) return go(e8, integral_constant<int, 1024>(), integral_constant<int, 1>(), one);
    } else {
        // (65,536 x 512 forwards: 22 us with 16 elements a thread, 30 with 8; 131,072 x 64: 27 and 7)
        if (a.D <= (GRAD ? NORM_NARROW * 8 : 256)) return go(e8, integral_constant<int, 256>(), integral_constant<int, GRAD ? 3 : 4>(), several);
        if (a.D <= NORM_NARROW * 16) return go(e16, integral_constant<int, 256>(), integral_constant<int, GRAD ? 3 : 4>(), several);
        if (a.D <= 8192) return go(e16, integral_constant<int, 512>(), integral_constant<int, 2>(), one);
    }
    return go(e16, integral_constant<int, 1024>(), integral_constant<int, 1>(), one);
}

template <class T, int V, bool GRAD>
static int launch_post(const NormArgs &a, bool post, bool vec, float *dgain, float *dnext, cudaStream_t st)
{
    if (post) return vec ? launch_sized<T, V, GRAD, true, false>(a, dgain, dnext, st) : launch_sized<T, V, GRAD, true, true>(a, dgain, dnext, st);
    return vec ? launch_sized<T, V, GRAD, false, false>(a, dgain, dnext, st) : launch_sized<T, V, GRAD, false, true>(a, dgain, dnext, st);
}

template <bool GRAD>
static int launch_typed(NormArgs a, bool post, int dtype, bool vec, float *dgain, float *dnext, cudaStream_t st)
{
    a.inv_d = 1.0f / (float)a.D;
    if (dtype == K3MOE_TYPE_F32) return launch_post<float, 4, GRAD>(a, post, vec, dgain, dnext, st);
    if (dtype == K3MOE_TYPE_BF16) return launch_post<__nv_bfloat16, 8, GRAD>(a, post, vec, dgain, dnext, st);
    return launch_post<__half, 8, GRAD>(a, post, vec, dgain, dnext, st);
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
// Vectors (gains, row gates, gradients' sums, workspace) apart from every output; all pointers at their elements' bytes.
struct NormVector {
    const void *p;
    size_t bytes;
    bool out;
    int element;
};
static int norm_vectors(int rows, int D, int dtype, std::initializer_list<NormMatrix> ms, std::initializer_list<NormVector> vs)
{
    bool aligned = true;
    for (const NormMatrix &m : ms) aligned = aligned && k3_aligned({{m.p, k3_type_bytes(dtype)}});
    for (const NormVector &v : vs) {
        if (!v.p) continue;
        aligned = aligned && k3_aligned({{v.p, v.element}});
        for (const NormMatrix &m : ms)
            if (m.p && (m.out || v.out) && k3_overlap(v.p, v.bytes, m.p, k3_span(rows, D, m.ld, dtype))) return K3MOE_ERR_ALIAS;
        for (const NormVector &w : vs)
            if (&w != &v && w.p && (w.out || v.out) && k3_overlap(v.p, v.bytes, w.p, w.bytes)) return K3MOE_ERR_ALIAS;
    }
    return aligned ? K3MOE_OK : K3MOE_ERR_ALIGN;
}
static bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace k3

using namespace k3;

extern "C" int k3moe_rms_norm(const void *x, int64_t ldx, const void *gain, int gain_dtype, float eps, int rows, int D,
                              int dtype, void *out, int64_t ldo, cudaStream_t stream)
{
    bool vec = false;
    const std::initializer_list<NormMatrix> ms = {{x, ldx, false, true}, {out, ldo, true, true}};
    int rc = norm_check(rows, D, dtype, gain_dtype, eps, ms, vec);
    if (rc) return rc;
    const int eg = k3_type_bytes(gain_dtype);
    if ((rc = norm_vectors(rows, D, dtype, ms, {{gain, (size_t)D * eg, false, eg}}))) return rc;
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
    int rc = norm_check(rows, D, dtype, gain_dtype, eps, ms, vec);
    if (rc) return rc;
    const int eg = k3_type_bytes(gain_dtype);
    const size_t ng = (size_t)D * eg;
    if ((rc = norm_vectors(rows, D, dtype, ms, {{gain, ng, false, eg}, {next_gain, ng, false, eg},
                                                {gate_kind == NORM_GATE_ROW ? gate : nullptr, (size_t)rows * 4, false, 4}})))
        return rc;
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
    return rows < 0 || D < 1 || D > K3MOE_NORM_MAX_WIDTH ? 0 : (size_t)std::max<int64_t>(1, norm_parts(rows)) * D * 2 * sizeof(float);
}

extern "C" int k3moe_rms_norm_grad(const void *dy, int64_t lddy, const void *x, int64_t ldx, const void *gain, int gain_dtype,
                                   const void *add, int64_t ldadd, float eps, int rows, int D, int dtype, void *dx,
                                   int64_t lddx, float *dgain, void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    bool vec = false;
    const std::initializer_list<NormMatrix> ms = {{dy, lddy, false, true}, {x, ldx, false, true}, {add, ldadd, false, false},
                                                  {dx, lddx, true, true}};
    int rc = norm_check(rows, D, dtype, gain_dtype, eps, ms, vec);
    if (rc) return rc;
    const size_t need = k3moe_norm_grad_workspace_bytes(rows, D);
    if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 3)) return K3MOE_ERR_WORKSPACE;
    const int eg = k3_type_bytes(gain_dtype);
    if ((rc = norm_vectors(rows, D, dtype, ms, {{gain, (size_t)D * eg, false, eg}, {dgain, (size_t)D * 4, true, 4},
                                                {workspace, need, true, 4}})))
        return rc;
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
    int rc = norm_check(rows, D, dtype, gain_dtype, eps, ms, vec);
    if (rc) return rc;
    const size_t need = k3moe_norm_grad_workspace_bytes(rows, D);
    if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 3)) return K3MOE_ERR_WORKSPACE;
    const int eg = k3_type_bytes(gain_dtype);
    const size_t ng = (size_t)D * eg;
    if ((rc = norm_vectors(rows, D, dtype, ms, {{gain, ng, false, eg}, {next_gain, ng, false, eg},
                                                {by_row ? gate : nullptr, (size_t)rows * 4, false, 4},
                                                {by_row ? dgate : nullptr, (size_t)rows * 4, true, 4}, {dgain, (size_t)D * 4, true, 4},
                                                {dnext_gain, (size_t)D * 4, true, 4}, {workspace, need, true, 4}})))
        return rc;
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
