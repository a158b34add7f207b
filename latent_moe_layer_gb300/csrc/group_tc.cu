// Products grouped by expert on the tensor cores (k3moe_group_mm, _grad_x, _grad_w): tcgen05 over CTA
// pairs, TMA-fed, persistent.
//
// One tile is D[256 x N] (+)= A[256 x c] B[N x c]^T, c the contraction, fp32 accumulators in TMEM:
//   mm       A = W_e rows (c = n_in contiguous),       B = x rows,  N = up to 256 of the expert's rows
//   grad_x   A = W_e columns (c = n_out, MN-major),    B = dy rows, N as above
//   grad_w   A = dy columns (c = rows, MN-major),      B = x columns (MN-major), N = 256
// The weights are the M side in mm and grad_x, so a group's raggedness costs at most 15 padding columns
// (N is a multiple of 16), its rows past the end are columns that are computed and not stored, and NaN or
// infinities there reach nothing else.  In grad_w the rows are the contraction: the rows of the last
// 16-row step that lie beyond the group (the next expert's) are set to zero in shared memory first.
//
// Each CTA of the pair loads its 128 rows of A and its half of B, 64 contraction values a stage: 32 KB
// of shared-memory writes per CTA feed a 256 x 256 x 64 step, half of what two single-CTA tiles of
// 128 x 256 need.  An SM takes in 64 bytes a cycle, so a stage costs max(2 N, 256 + N) cycles: the tensor
// cores bind at N = 256, the intake below.  Two accumulator sets (2 x 256 TMEM columns) let the epilogue
// of one tile overlap the next tile's MMAs.
//
// Where a call has few tiles, two or four pairs share a tile's contraction and add up their parts through
// distributed shared memory (SPLIT below).
//
// Measured, bf16: 57,344 rows over 28 experts, 3584 to 6144: 1.27-1.34 ms, 1.9-2.0 PFLOP/s (513 cycles a stage, 512
// are the MMAs'); 8192^3 in one group 0.574 ms, 1.92 PFLOP/s; 65,536 rows over 112 experts 1.64-1.71 ms (467
// cycles a stage at N = 192 to 208), 1.9-2.0 ms under the power cap; 251 rows over 112 experts 0.63-0.65 ms, the
// weights at 6.8 TB/s; grad_w of 16,381 rows over 56 experts, 3584 x 3072 in fp32: 0.54-0.57 ms, of which the stores
// alone take 0.43 (5.7 TB/s); 1 row, 6144 to 64, 9.7 us (22.5 with one pair).
#include <cudaTypedefs.h>

#include "experts.h"
#include "group_sched.cuh"
#include "pair.cuh"

namespace k3 {

constexpr int GT_BK = 64, GT_TILE_M = 256, GT_TILE_N = 256;
// mm, grad_x: row tiles of at most 256, 128, 64 or 32 rows, so that a few large experts still fill the GPU
constexpr int GT_TILE_PICKS = 4;
constexpr int GT_A_BYTES = 128 * GT_BK * 2, GT_STAGE = 2 * GT_A_BYTES;
// The tensor core truncates what it adds, always towards zero: products of one sign lose 3.2e-9 of their sum a
// contraction value in bf16 and 6.3e-9 in f16, whose products have more bits (products of random sign 1.2e-9).  grad_w,
// and mm and grad_x with an fp32 output, therefore add up parts of 512 (f16: 256) values in fp32 registers: an error of
// 1.7e-6 of the sum at any length.  mm and grad_x with a 16-bit output do so from GT_LONG values on: below, the loss is at
// most 1/9 of the f16 output's own half unit in the last place (bf16: 1/100).  Parts cost fp32 outputs 1-11 % in bf16
// (2,047 rows over 14 experts, 3584 to 3584: 71 -> 73 us; 16,384 over 112, 3584 to 6144: 820 -> 845); for 16-bit ones it
// would be 67 -> 71 and 792 -> 819 us, and in f16 60 -> 82.
constexpr int GT_PART_BF16 = 3, GT_PART_F16 = 2;                        // log2 of a part's stages
constexpr int GT_LONG = 8192;
// mm, grad_x: bytes of activation rows whose tiles pass under one block of weights before the next block
constexpr int64_t GT_L2_ROWS = 32 << 20;

template <int MODE, bool FOLD>
struct GroupSmem {
    static constexpr int NS = MODE == K3_GROUP_GRAD_W ? 5 : 6;
    // grad_w's epilogue keeps 64 sums a thread and writes every value in fp32: four warps a TMEM quarter
    static constexpr int EPI_WARPS = MODE == K3_GROUP_GRAD_W ? 16 : 8;
    static constexpr int THREADS = 96 + 32 * EPI_WARPS;                 // TMA, MMA, tails, epilogue
    static constexpr int OFF_OUT = NS * GT_STAGE;
    // output staging of a warp: grad_w one 4 KB box, else 16 rows x 32 16-bit values
    static constexpr int OUT_WARP = MODE == K3_GROUP_GRAD_W ? 4096 : 1024;
    static constexpr int OUT_BYTES = EPI_WARPS * OUT_WARP;
    static constexpr int OFF_BAR = OFF_OUT + OUT_BYTES;
    static constexpr int N_BAR = 3 * NS + 5;                            // full, empty, tail; tfull, tempty x 2; drain
    static constexpr int OFF_INT = OFF_BAR + N_BAR * 8 + 8;
    // grad_w needs no tile table and reads the offsets from memory, which leaves room for its fifth stage
    static constexpr int N_INT = MODE == K3_GROUP_GRAD_W ? 0 : 2 * (K3MOE_TRAIN_MAX_EXPERTS + 1) + GT_TILE_PICKS * THREADS / 32;
    static constexpr int BYTES = OFF_INT + N_INT * 4 + 1024;
    static_assert(BYTES <= kMaxSmem, "shared memory");
};

struct GroupMaps {
    CUtensorMap a;           // mm: box 64 x 128 rows; grad_x, grad_w: box 64 x 64, or two of them (wide)
    CUtensorMap b[5];        // mm, grad_x: boxes of 128, 64, 32, 16, 8 rows; grad_w: b[0] as a
    CUtensorMap out;         // grad_w
};

struct GroupTcArgs {
    const int32_t *offsets;
    int E, rows, M, Nc;      // M: the tile-row extent; Nc: grad_w's column extent (n_in)
    int K;                   // contraction of mm and grad_x
    int l2_rows;             // rows of GT_L2_ROWS bytes
    int pairs;               // clusters of the launch
    int expert_coord;        // 0: one weight for all experts
    int wide_a, wide_b;      // MN-major operands whose width is a multiple of 64: both 64 x 64 boxes in one copy
    int bf16, accumulate;
    int part;                // FOLD: log2 of a part's stages
    int out16;               // mm, grad_x: output rows on 16-byte boundaries
    void *out;
    int64_t ldo, stride_o;
    int *status;
};

struct GroupJob {
    int m0, c0, n, steps, last;      // first row and column of the tile; columns; stages; contraction values of the last stage
};

// A CTA pair's walk over the tiles: job indexes first, first + stride, ...  An expert's tiles are
// consecutive, so that what they share stays in L2.
template <int MODE>
struct GroupWalk {
    const GroupTcArgs &a;
    const int *s_off, *s_tile;
    const int mb, cb, jobs, stride;
    int job, e = -1, begin = 0, end = 0, off0 = 0, rows = 0;     // the current expert, its job range and rows

    __device__ __forceinline__ GroupWalk(const GroupTcArgs &a_, const int *so, const int *st, int mb_, int cb_, int jobs_)
        : a(a_), s_off(so), s_tile(st), mb(mb_), cb(cb_), jobs(jobs_), stride((int)ncluster_x()), job((int)cluster_id_x())
    {
        enter();
    }
    __device__ __forceinline__ bool valid() const { return job < jobs; }
    __device__ __forceinline__ void next()
    {
        job += stride;
        enter();
    }
    __device__ __forceinline__ void enter()
    {
        if (job < end || job >= jobs) return;
        if (MODE == K3_GROUP_GRAD_W) {
            e = job / (mb * cb);
            begin = e * mb * cb;
            end = begin + mb * cb;
        } else {
            // the next expert as a rule, a search where experts are smaller than the stride
            if (e + 1 < a.E && job < s_tile[e + 2] * mb) ++e;
            else e = group_find(s_tile, a.E, job / mb);
            begin = s_tile[e] * mb;
            end = s_tile[e + 1] * mb;
        }
        off0 = s_off[e];
        rows = s_off[e + 1] - off0;
    }
    __device__ __forceinline__ GroupJob get() const
    {
        GroupJob j;
        int w = job - begin;
        if (MODE == K3_GROUP_GRAD_W) {
            j.m0 = (w / cb) * GT_TILE_M;
            j.c0 = (w % cb) * GT_TILE_N;
            j.n = GT_TILE_N;
            j.steps = (rows + GT_BK - 1) / GT_BK;
            j.last = rows - (j.steps - 1) * GT_BK;
        } else {
            // row tiles (in groups that fit the L2) next to each other on the same block of weights
            int t = s_tile[e + 1] - s_tile[e], first = 0;
            const int all = t;
            if (rows > a.l2_rows) {
                const int group = max(1, (int)((int64_t)a.l2_rows * t / rows)), g = w / (group * mb);
                first = g * group;
                w -= first * mb;
                t = min(group, t - first);
            }
            j.m0 = (w / t) * GT_TILE_M;
            const int i = first + w % t;
            // an expert's tiles differ by at most 16 rows: 585 rows are 208 + 192 + 185, not 256 + 256 + 73
            const int units = (rows + 15) >> 4, u = units / all, more = units - u * all;
            j.c0 = off0 + 16 * (i * u + min(i, more));
            j.n = min(16 * (u + (i < more)), off0 + rows - j.c0);
            j.steps = (a.K + GT_BK - 1) / GT_BK;
            j.last = a.K - (j.steps - 1) * GT_BK;
        }
        return j;
    }
};

// `rows` (a multiple of 8, at most 128) rows of B from row `row`: boxes of 128 .. 8 rows, largest first.
__device__ __forceinline__ void load_rows(const CUtensorMap *maps, uint32_t dst, uint32_t bar, int k, int row, int rows)
{
#pragma unroll
    for (int i = 0; i < 5; ++i) {
        const int box = 128 >> i;
        if (rows & box) {
            tma_load_2d_pair(dst, maps + i, bar, k, row);
            dst += box * 128;
            row += box;
        }
    }
}

// (a, b) += (c, d), both sums in one instruction.  Sums that begin at zero and take a part in eight columns at a time leave
// no register spilled, which the issuing loop would pay (251 rows over 112 experts, fp32 output: 745 us with 16, 734 with 8).
__device__ __forceinline__ void add2(float &a, float &b, uint32_t c, uint32_t d)
{
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tadd.rn.f32x2 x, x, y;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "r"(c), "r"(d));
}

// FOLD: parts of the contraction are added up in registers; grad_w always, see GT_LONG.
// CUT: grad_w's rows end inside 16 bytes (a variant of its own for the registers it costs).
// SPLIT: the pairs of a cluster of 2 SPLIT CTAs share one tile's contraction, for calls of few tiles.  The
// caller gives every tile a cluster of its own: each pair leaves its part of the sum in its shared memory (the ring
// is done with), and the pairs add up the parts of a share of the tile each, in a fixed order, and store it.
template <int MODE, class O, bool CUT, int SPLIT, bool FOLD>
__global__ void __launch_bounds__(GroupSmem<MODE, FOLD>::THREADS, 1)
    group_tc_kernel(const __grid_constant__ GroupMaps maps, const GroupTcArgs args)
{
    using SM = GroupSmem<MODE, FOLD>;
    constexpr int NS = SM::NS;
    constexpr bool W = MODE == K3_GROUP_GRAD_W;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint64_t *full = (uint64_t *)(smem + SM::OFF_BAR), *empty = full + NS, *tail = empty + NS;
    uint64_t *tfull = tail + NS, *tempty = tfull + 2, *drain = tempty + 2;
    uint32_t *tmem_holder = (uint32_t *)(drain + 1);
    volatile int *abort_flag = (volatile int *)(tmem_holder + 1);
    int *s_int = (int *)(smem + SM::OFF_INT), *s_tile = s_int + K3MOE_TRAIN_MAX_EXPERTS + 1;
    const int *s_off = W ? args.offsets : s_int;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // this CTA's place in its pair, the pair's place in the cluster, the cluster rank of the pair's even CTA
    const uint32_t rank = cluster_ctarank() & 1, pair = SPLIT > 1 ? cluster_ctarank() >> 1 : 0, lead = 2 * pair;
    // FOLD: parts of the stages s0 .. s1 - 1 (parts begin at multiples of their length)
    auto parts = [&](int s0, int s1) {
        const int up = (s1 + (1 << args.part) - 1) >> args.part;
        return SPLIT == 1 ? up : s1 > s0 ? up - (s0 >> args.part) : 0;
    };
    // its stages of a job
    auto first_stage = [&](const GroupJob &j) { return SPLIT == 1 ? 0 : (int)((uint32_t)j.steps * pair / SPLIT); };
    auto end_stage = [&](const GroupJob &j) { return SPLIT == 1 ? j.steps : (int)((uint32_t)j.steps * (pair + 1) / SPLIT); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(smem_u32(full + i), 2);            // both CTAs' loads (or their zeroed tails)
            mbar_init(smem_u32(empty + i), 1);
            mbar_init(smem_u32(tail + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(tfull + i), 1);
            mbar_init(smem_u32(tempty + i), 2 * SM::EPI_WARPS);
        }
        mbar_init(smem_u32(drain), 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == 0 && lane < (W ? 2 : 6)) prefetch_tmap(lane == 0 ? &maps.a : &maps.b[lane - 1]);
    cluster_sync();                                      // barriers of both CTAs before any remote arrival

    // all of the above may run while the previous kernel of the stream finishes; tensor memory may not
    // be taken before, as that kernel may still have to
    griddep_enter();
    if (warp == 1) tmem_alloc_pair(smem_u32(tmem_holder), 512);
    tc_fence_before();                                   // the CTA-wide barriers below publish the address
    const int mb = (args.M + GT_TILE_M - 1) / GT_TILE_M, cb = W ? (args.Nc + GT_TILE_N - 1) / GT_TILE_N : 1;
    const bool offsets_ok =
        W ? group_offsets_ok<SM::THREADS>(args.offsets, args.E, args.rows, args.status)
          : group_tiles<SM::THREADS, GT_TILE_N, GT_TILE_PICKS>(args.offsets, args.E, args.rows, s_int, s_tile,
                                                               s_tile + K3MOE_TRAIN_MAX_EXPERTS + 1, args.status, mb,
                                                               args.pairs);
    // every CTA reads the same offsets, so all agree on a refusal
    const int jobs = !offsets_ok ? 0 : W ? args.E * mb * cb : s_tile[args.E] * mb;

    tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    // mm, grad_x: a warp's 32 output columns (one a lane) of 16 rows, from fp32
    auto store16 = [&](const GroupJob &j, int m0, int c, const uint32_t (&v)[16], uint8_t *box) {
        const int m = m0 + lane;
        if (sizeof(O) == 2 && args.out16) {
            // a lane holds one output column of 16 rows: turned in shared memory, two rows to a word,
            // into 16-byte pieces of rows (stored as they are, 64 bytes an instruction, a tile's
            // outputs took 6 us)
            using T = std::conditional_t<sizeof(O) == 2, O, __half>;
            uint32_t *st = reinterpret_cast<uint32_t *>(box);
            __syncwarp();                                    // the previous pieces have been read
#pragma unroll
            for (int i = 0; i < 8; ++i)
                st[i * 32 + lane] = pack2<T>(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
            __syncwarp();
            // lane: rows 2 p and 2 p + 1, columns m0 + 8 (lane % 4) .. + 7; odd pairs read their halves in the
            // other order, which keeps the banks apart
            const int p = lane >> 2, m8 = m0 + (lane & 3) * 8, odd = p & 1;
            const uint4 *src = reinterpret_cast<const uint4 *>(st + p * 32 + (lane & 3) * 8);
            const uint4 x = src[odd], y = src[1 - odd], a = odd ? y : x, b = odd ? x : y;
            const uint4 row[2] = {{__byte_perm(a.x, a.y, 0x5410), __byte_perm(a.z, a.w, 0x5410),
                                   __byte_perm(b.x, b.y, 0x5410), __byte_perm(b.z, b.w, 0x5410)},
                                  {__byte_perm(a.x, a.y, 0x7632), __byte_perm(a.z, a.w, 0x7632),
                                   __byte_perm(b.x, b.y, 0x7632), __byte_perm(b.z, b.w, 0x7632)}};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (c + 2 * p + i >= j.n) continue;
                O *o = static_cast<O *>(args.out) + (int64_t)(j.c0 + c + 2 * p + i) * args.ldo + m8;
                if (m8 + 8 <= args.M) {
                    *reinterpret_cast<uint4 *>(o) = row[i];
                } else {
                    const O *e = reinterpret_cast<const O *>(row + i);
#pragma unroll
                    for (int q8 = 0; q8 < 8; ++q8)
                        if (m8 + q8 < args.M) o[q8] = e[q8];
                }
            }
        } else if (m < args.M) {
            O *o = static_cast<O *>(args.out) + (int64_t)(j.c0 + c) * args.ldo + m;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (c + i < j.n) o[i * args.ldo] = from_f32<O>(__uint_as_float(v[i]));
        }
    };

    // grad_w: 32 rows and CW columns (128 bytes a row); fill(h, v) gives the lane's row at columns h .. h + 15
    constexpr int CW = 128 / (int)sizeof(O);
    auto store_box = [&](const GroupJob &j, int e, int m0, int c, uint8_t *box, auto fill) {
        // a box that crosses the last column of rows that end inside 16 bytes: the copy engine
        // would write those 16 bytes whole, so its values are stored one by one
        const bool cut = CUT && j.c0 + c + CW > args.Nc;
        if (m0 < args.M && j.c0 + c < args.Nc) {                         // else wholly outside
            if (!cut && lane == 0) bulk_wait_read<0>();                  // the box's previous store has read it
            __syncwarp();
#pragma unroll
            for (int h = 0; h < CW; h += 16) {
                uint32_t v[16] = {};
                fill(h, v);
                if (cut) {
                    O *o = static_cast<O *>(args.out) + e * args.stride_o + (int64_t)(m0 + lane) * args.ldo + j.c0 + c + h;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (m0 + lane < args.M && j.c0 + c + h + i < args.Nc)
                            o[i] = from_f32<O>(__uint_as_float(v[i]) + (args.accumulate ? to_f32(o[i]) : 0.f));
                    continue;
                }
                // 16-byte pieces at the 128-byte swizzle's place: piece p of row r at p ^ (r % 8)
#pragma unroll
                for (int p = 0; p < (int)sizeof(O); ++p) {
                    uint4 w;
                    if (sizeof(O) == 4) {
                        const uint32_t *f = v + (4 * p & 15);
                        w = make_uint4(f[0], f[1], f[2], f[3]);
                    } else {
                        Vec<std::conditional_t<sizeof(O) == 4, __half, O>, 8> o;
#pragma unroll
                        for (int i = 0; i < 8; i += 2)
                            o.set2(i, __uint_as_float(v[(8 * p + i) & 15]), __uint_as_float(v[(8 * p + i + 1) & 15]));
                        w = make_uint4(o.w[0], o.w[1], o.w[2], o.w[3]);
                    }
                    const int piece = h * (int)sizeof(O) / 16 + p;
                    *reinterpret_cast<uint4 *>(box + lane * 128 + ((piece ^ (lane & 7)) << 4)) = w;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (!cut && lane == 0) {
                if (args.accumulate) tma_add_3d(&maps.out, smem_u32(box), j.c0 + c, m0, e);
                else tma_store_3d(&maps.out, smem_u32(box), j.c0 + c, m0, e);
                bulk_commit();
            }
        }
    };
    // SPLIT: 16 columns from c of row `row` into this pair's part of the sum, [n / 4][128][4]
    auto put_part = [&](int c, int row, const uint32_t (&v)[16]) {
        uint4 *at = reinterpret_cast<uint4 *>(smem) + c / 4 * 128 + row;
#pragma unroll
        for (int i = 0; i < 4; ++i) at[i * 128] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    };
    // SPLIT: the sum of the pairs' parts at 16 columns from c, row `row` of this CTA's; its own part first, then the next
    // pair's, so that no CTA is asked by all at once
    auto add_parts = [&](int c, int row, uint32_t (&v)[16]) {
        const uint32_t at = (c / 4 * 128 + row) * 16;
        float sum[16];
#pragma unroll
        for (int p = 0; p < SPLIT; ++p) {
            const uint32_t from = cluster_addr(smem_u32(smem), 2 * ((pair + p) % SPLIT) + rank) + at;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 x = p ? ld_cluster_f32x4(from + k * 2048) : *reinterpret_cast<const float4 *>(smem + at + k * 2048);
                sum[4 * k] = p ? sum[4 * k] + x.x : x.x;
                sum[4 * k + 1] = p ? sum[4 * k + 1] + x.y : x.y;
                sum[4 * k + 2] = p ? sum[4 * k + 2] + x.z : x.z;
                sum[4 * k + 3] = p ? sum[4 * k + 3] + x.w : x.w;
            }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(sum[k]);
    };

    // The producer and issuer warps run their loops as whole warps, one elected lane doing the work.
    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer (each CTA its half)
        const bool one = elect_one();
        const uint32_t full0 = cluster_addr(smem_u32(full), lead);
        RingPos<NS> p, t;                                // stages; tails
        uint32_t issued = 0;
        bool ok = true;
        for (GroupWalk<MODE> walk(args, s_off, s_tile, mb, cb, jobs); walk.valid() && ok; walk.next()) {
            const GroupJob j = walk.get();
            const int half = W ? 128 : ((j.n + 15) & ~15) / 2;           // this CTA's share of B's rows
            const int m = j.m0 + 128 * (int)rank, e = args.expert_coord * walk.e;
            const int c = j.c0 + half * (int)rank, r0 = walk.off0;
            const uint32_t bytes = GT_A_BYTES + half * 128;
            const int s1 = end_stage(j);
            for (int s = first_stage(j); s < s1; ++s, ++issued, p.next()) {
                if (!pair_wait(smem_u32(empty + p.slot), p.phase ^ 1, abort_flag, args.status, 61)) {
                    ok = false;
                    break;
                }
                const uint32_t a_dst = smem_u32(smem) + p.slot * GT_STAGE, b_dst = a_dst + GT_A_BYTES;
                uint32_t bar = full0 + p.slot * 8;
                const bool tailed = W && s == j.steps - 1 && (j.last & 15);
                if (tailed) bar = smem_u32(tail + t.slot);
                const int k = s * GT_BK;
                if (one) {
                    // the tail warp zeroes a tail's foreign rows before it arrives for this CTA
                    if (tailed) mbar_expect_tx(bar, bytes);
                    else mbar_expect_tx_cluster(bar, bytes);
                    if (MODE == K3_GROUP_MM) {
                        tma_load_3d_pair(a_dst, &maps.a, bar, k, m, e);
                    } else if (MODE == K3_GROUP_GRAD_X) {
                        if (args.wide_a) {
                            tma_load_4d_pair(a_dst, &maps.a, bar, 0, k, m / 64, e);
                        } else {
                            tma_load_3d_pair(a_dst, &maps.a, bar, m, k, e);
                            tma_load_3d_pair(a_dst + GT_A_BYTES / 2, &maps.a, bar, m + 64, k, e);
                        }
                    }
                    if (!W) {
                        load_rows(maps.b, b_dst, bar, k, c, half);
                    } else {
                        if (args.wide_a) {
                            tma_load_3d_pair(a_dst, &maps.a, bar, 0, r0 + k, m / 64);
                        } else {
                            tma_load_2d_pair(a_dst, &maps.a, bar, m, r0 + k);
                            tma_load_2d_pair(a_dst + GT_A_BYTES / 2, &maps.a, bar, m + 64, r0 + k);
                        }
                        if (args.wide_b) {
                            tma_load_3d_pair(b_dst, &maps.b[0], bar, 0, r0 + k, c / 64);
                        } else {
                            tma_load_2d_pair(b_dst, &maps.b[0], bar, c, r0 + k);
                            tma_load_2d_pair(b_dst + GT_A_BYTES / 2, &maps.b[0], bar, c + 64, r0 + k);
                        }
                    }
                }
                __syncwarp();
                if (tailed) t.next();
            }
        }
        // the last releases of this CTA's slots land before it may exit: a slot's next use would wait for them
        for (uint32_t q = 0; ok && q < min(issued, (uint32_t)NS); ++q, p.next()) {
            if (issued < (uint32_t)NS && q == 0) p.slot = 0, p.phase = 1;
            ok = pair_wait(smem_u32(empty + p.slot), p.phase ^ 1, abort_flag, args.status, 62);
        }
        if (!ok) {
            // given up: the copies in flight land before the shared memory is given back.  The even CTA waits
            // for the stages that both announced; what only one of them did is far past its latency in 1 ms.
            if (rank == 0) drain_ring(full, issued, NS);
            const uint64_t t0 = globaltimer();
            while (globaltimer() - t0 < 1000000) __nanosleep(1000);
        }
    } else if (warp == 1 && rank == 0) {
        // ------------------------------------------------------------ MMA issuer (even CTA, for both)
        const uint32_t major = (MODE == K3_GROUP_MM ? 0 : IDESC_A_MN) | (W ? IDESC_B_MN : 0);
        // a step of 16 contraction values: 32 bytes along a K-major row, 16 rows of 128 bytes MN-major
        constexpr int a_step = MODE == K3_GROUP_MM ? 2 : 128, b_step = W ? 128 : 2;
        const uint32_t a0 = smem_u32(smem);
        const uint64_t ad0 = MODE == K3_GROUP_MM ? smem_desc_sw128(a0) : smem_desc_mn_sw128(a0, GT_A_BYTES / 2);
        const uint64_t bd0 = W ? smem_desc_mn_sw128(a0 + GT_A_BYTES, GT_A_BYTES / 2) : smem_desc_sw128(a0 + GT_A_BYTES);
        const bool one = elect_one();
        const int part_mask = (1 << args.part) - 1;
        RingPos<NS> p;
        RingPos<2> acc;
        bool ok = true;
        for (GroupWalk<MODE> walk(args, s_off, s_tile, mb, cb, jobs); walk.valid() && ok; walk.next()) {
            const GroupJob j = walk.get();
            const uint32_t idesc = idesc_f16(GT_TILE_M, (j.n + 15) & ~15, args.bf16) | major;
            const int s0 = first_stage(j), s1 = end_stage(j);
            for (int s = s0; s < s1; ++s, p.next()) {
                const bool begin = s == s0 || (FOLD && (s & part_mask) == 0), last = s == j.steps - 1;
                const bool end = s == s1 - 1 || (FOLD && (s & part_mask) == part_mask);
                if (begin) {
                    ok = pair_wait(smem_u32(tempty + acc.slot), acc.phase ^ 1, abort_flag, args.status, 63);
                    tc_fence_after();
                }
                ok = ok && pair_wait(smem_u32(full + p.slot), p.phase, abort_flag, args.status, 64);
                if (!ok) break;
                // a tail was written by threads of either CTA, not by the copy engine
                if (W && last && (j.last & 15)) mbar_try_wait_cluster(smem_u32(full + p.slot), p.phase);
                tc_fence_after();
                const uint32_t d = tmem + acc.slot * GT_TILE_N;
                const uint64_t ad = ad0 + p.slot * (GT_STAGE / 16), bd = bd0 + p.slot * (GT_STAGE / 16);
                const int kk_n = last ? (j.last + 15) >> 4 : GT_BK / 16;
                if (one) {
#pragma unroll
                    for (int kk = 0; kk < GT_BK / 16; ++kk)
                        if (kk < kk_n)
                            tc_mma_f16_pair(d, ad + a_step * kk, bd + b_step * kk, idesc, (!begin || kk > 0) ? 1u : 0u);
                    tc_commit_pair(smem_u32(empty + p.slot), lead);
                    if (end) tc_commit_pair(smem_u32(tfull + acc.slot), lead);
                }
                __syncwarp();
                if (end) acc.next();
            }
        }
        // every issued MMA completes before TMEM is released
        if (one) tc_commit_pair(smem_u32(drain), lead);
        __syncwarp();
        mbar_wait(smem_u32(drain), 0, 0xFFFFFFFFu);
    } else if (W && warp == 2) {
        // ------------------------------------------------------------ tails of the groups (each CTA its half)
        RingPos<NS> t;
        uint32_t it = 0;
        for (GroupWalk<MODE> walk(args, s_off, s_tile, mb, cb, jobs); walk.valid(); walk.next()) {
            const GroupJob j = walk.get();
            it += end_stage(j) - first_stage(j);
            if (j.steps == 0 || !(j.last & 15) || pair != SPLIT - 1) continue;       // the last pair has the last stage
            const int slot = (it - 1) % NS;
            if (!pair_wait(smem_u32(tail + t.slot), t.phase, abort_flag, args.status, 65)) break;
            t.next();
            // rows last .. last rounded up to 16 of the four 64 x 64 boxes, eight lanes a row: a row is 128
            // bytes, whatever the swizzle
            uint8_t *st = smem + slot * GT_STAGE + (lane >> 3) * (GT_A_BYTES / 2) + (lane & 7) * 16;
            for (int r = j.last; r & 15; ++r) *reinterpret_cast<uint4 *>(st + r * 128) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_u32(full + slot), lead));
        }
    } else if (warp >= 3) {
        // ------------------------------------------------------------ epilogue (each CTA its 128 rows)
        constexpr int PARTS = SM::EPI_WARPS / 4, COLS = GT_TILE_N / PARTS;
        const int q = warp & 3, part = (warp - 3) >> 2;                  // TMEM lanes 32q .. 32q + 31
        const uint32_t tbase = tmem + ((uint32_t)(32 * q) << 16);
        const uint32_t tempty0 = cluster_addr(smem_u32(tempty), lead);
        RingPos<2> acc;
        uint8_t *box = smem + SM::OFF_OUT + (warp - 3) * SM::OUT_WARP;
        bool ok = true;
        for (GroupWalk<MODE> walk(args, s_off, s_tile, mb, cb, jobs); walk.valid() && ok; walk.next()) {
            const GroupJob j = walk.get();
            const int m0 = j.m0 + 128 * (int)rank + 32 * q;
            if (W) {
                const int s0 = first_stage(j), s1 = end_stage(j);
                const int chunks = parts(s0, s1);
                if (j.steps == 0 && args.accumulate) continue;           // an expert without rows: nothing, or zeros
                float sum[COLS] = {};
                for (int ch = 0; ch < chunks; ++ch) {
                    ok = pair_wait(smem_u32(tfull + acc.slot), acc.phase, abort_flag, args.status, 66);
                    if (!ok) break;
                    tc_fence_after();
                    if (SPLIT == 1 && chunks == 1) break;                // stored from TMEM below
#pragma unroll
                    for (int g = 0; g < COLS / 8; ++g) {
                        uint32_t v[8];
                        tmem_ld8(tbase + acc.slot * GT_TILE_N + part * COLS + 8 * g, v);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 8; i += 2) add2(sum[8 * g + i], sum[8 * g + i + 1], v[i], v[i + 1]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(tempty0 + acc.slot * 8);
                    acc.next();
                }
                if (!ok) break;
                if (SPLIT > 1) {
                    float4 *mine = reinterpret_cast<float4 *>(smem) + part * COLS / 4 * 128 + 32 * q + lane;
#pragma unroll
                    for (int g = 0; g < COLS / 4; ++g)
                        if (j.c0 + part * COLS + 4 * g < args.Nc)
                            mine[g * 128] = chunks ? make_float4(sum[4 * g], sum[4 * g + 1], sum[4 * g + 2], sum[4 * g + 3]) : float4{};
                    continue;
                }
#pragma unroll
                for (int g0 = 0; g0 < COLS; g0 += CW)
                    store_box(j, walk.e, m0, part * COLS + g0, box, [&](int h, uint32_t (&v)[16]) {
                        if (chunks == 1) {
                            tmem_ld16(tbase + acc.slot * GT_TILE_N + part * COLS + g0 + h, v);
                            tc_wait_ld();
                        } else if (chunks > 1) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(sum[g0 + h + i]);
                        }
                    });
                if (chunks != 1) continue;
            } else if (FOLD) {
                // the warp's columns are 16 (part + PARTS i) .. + 15, so that narrow tiles occupy all warps
                const int chunks = parts(first_stage(j), end_stage(j));
                float sum[COLS] = {};
                for (int ch = 0; ch < chunks; ++ch) {
                    ok = pair_wait(smem_u32(tfull + acc.slot), acc.phase, abort_flag, args.status, 66);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int g = 0; g < COLS / 16; ++g) {
                        const int c = 16 * (part + PARTS * g);
                        if (c >= j.n) break;
#pragma unroll
                        for (int h = 0; h < 16; h += 8) {
                            uint32_t v[8];
                            tmem_ld8(tbase + acc.slot * GT_TILE_N + c + h, v);
                            tc_wait_ld();
#pragma unroll
                            for (int i = 0; i < 8; i += 2) add2(sum[16 * g + h + i], sum[16 * g + h + i + 1], v[i], v[i + 1]);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(tempty0 + acc.slot * 8);
                    acc.next();
                }
                if (!ok) break;
#pragma unroll
                for (int g = 0; g < COLS / 16; ++g) {
                    const int c = 16 * (part + PARTS * g);
                    if (c >= j.n) break;
                    uint32_t v[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(sum[16 * g + i]);
                    if (SPLIT > 1) put_part(c, 32 * q + lane, v);
                    else store16(j, m0, c, v, box);
                }
                continue;
            } else {
                ok = pair_wait(smem_u32(tfull + acc.slot), acc.phase, abort_flag, args.status, 66);
                if (!ok) break;
                tc_fence_after();
                for (int c = 16 * part; c < j.n; c += 16 * PARTS) {
                    uint32_t v[16];
                    tmem_ld16(tbase + acc.slot * GT_TILE_N + c, v);
                    tc_wait_ld();
                    if (SPLIT > 1) put_part(c, 32 * q + lane, v);
                    else store16(j, m0, c, v, box);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty0 + acc.slot * 8);
            acc.next();
        }
    }
    if (SPLIT > 1) {
        tc_fence_before();
        __syncthreads();
        cluster_sync();                                  // every pair's part is in its shared memory
        const GroupWalk<MODE> walk(args, s_off, s_tile, mb, cb, jobs);
        if (warp >= 3 && walk.valid()) {
            const GroupJob j = walk.get();
            uint8_t *box = smem + SM::OFF_OUT + (warp - 3) * SM::OUT_WARP;
            // pieces of 32 rows of the accumulator, dealt out over the pairs' warps
            const int width = W ? CW : 16, pieces = W && j.steps == 0 && args.accumulate ? 0 : (j.n + width - 1) / width * 4;
            for (int i = (warp - 3) * SPLIT + (int)pair; i < pieces; i += SPLIT * SM::EPI_WARPS) {
                const int row = 32 * (i & 3), c = (i >> 2) * width, m0 = j.m0 + 128 * (int)rank + row;
                if (W) {
                    store_box(j, walk.e, m0, c, box, [&](int h, uint32_t (&v)[16]) { add_parts(c + h, row + lane, v); });
                } else {
                    uint32_t v[16];
                    add_parts(c, row + lane, v);
                    store16(j, m0, c, v, box);
                }
            }
        }
    }
    if (W && warp >= 3 && lane == 0) bulk_wait<0>();
    tc_fence_before();
    __syncthreads();
    // the issuer's last commit arrives in both CTAs: the other one waits for it too before it may exit
    if (rank == 1 && threadIdx.x == 32) mbar_wait(smem_u32(drain), 0, 0xFFFFFFFFu);
    cluster_sync();                                      // no arrival or MMA of the pair is outstanding past this
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ------------------------------------------------------------------ host
typedef PFN_cuTensorMapEncodeTiled_v12000 EncodeFn;

static EncodeFn encode_fn()
{
    static EncodeFn fn = nullptr;
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = (EncodeFn)p;
    }
    return fn;
}

static bool encode(CUtensorMap *m, int type, const void *base, int nd, const int64_t (&dim)[4], const int64_t (&stride)[3],
                   const int (&box)[4])
{
    EncodeFn fn = encode_fn();
    if (!fn) return false;
    const int es = k3_type_bytes(type);
    const CUtensorMapDataType dt = type == K3MOE_TYPE_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : type == K3MOE_TYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                             : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    cuuint64_t d[4], st[3];
    cuuint32_t b[4], one[4] = {1, 1, 1, 1};
    for (int i = 0; i < nd; ++i) {
        d[i] = (cuuint64_t)dim[i];
        b[i] = (cuuint32_t)box[i];
        if (i + 1 < nd) st[i] = (cuuint64_t)(stride[i] * es);
    }
    return fn(m, dt, nd, const_cast<void *>(base), d, st, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Map over `n2` matrices of [rows, cols] (n2 = 0: two dimensions), 128-byte swizzle, 128-byte box rows.
static bool encode_rows(CUtensorMap *m, int type, const void *base, int64_t cols, int64_t rows, int64_t n2, int64_t ld,
                        int64_t stride2, int box_rows)
{
    return encode(m, type, base, n2 > 0 ? 3 : 2, {cols, rows, n2, 1}, {ld, stride2, 0},
                  {128 / k3_type_bytes(type), box_rows, 1, 1});
}

// The same matrices of 16-bit elements as [n2][cols / 64][rows][64], where that is whole: a box of two blocks is
// what an MN-major operand of 128 columns wants in one copy (grad_w of 57,344 rows over 28 experts: 1.53 ms, 1.56 with
// two copies an operand).
static bool encode_wide(CUtensorMap *m, int type, const void *base, int64_t cols, int64_t rows, int64_t n2, int64_t ld,
                        int64_t stride2)
{
    return encode(m, type, base, n2 > 0 ? 4 : 3, {64, rows, cols / 64, n2}, {ld, 64, stride2}, {64, 64, 2, 1});
}

// Clusters of 2 SPLIT CTAs that are on the GPU together (0: an error).
template <int MODE, class O, bool CUT, int SPLIT, bool FOLD>
static int fit_clusters(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&attr)[2], cudaStream_t st)
{
    using SM = GroupSmem<MODE, FOLD>;
    auto kern = group_tc_kernel<MODE, O, CUT, SPLIT, FOLD>;
    static unsigned long long attr_set = 0;
    if (!k3_smem_attr(kern, SM::BYTES, attr_set)) return 0;
    const int sms = k3_num_sms();
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {2 * SPLIT, 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(sms / (2 * SPLIT) * (2 * SPLIT));
    cfg.blockDim = SM::THREADS;
    cfg.dynamicSmemBytes = SM::BYTES;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (SPLIT == 1) return sms / 2;
    static int fit = 0;
    if (!fit) {
        int n = 0;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        cfg.numAttrs = 2;
        fit = n > 0 ? n : -1;
    }
    return std::max(fit, 0);
}

template <int MODE, class O, bool FOLD, bool CUT = false, int SPLIT = 1>
static int launch_tc(const GroupMaps &maps, GroupTcArgs a, int64_t max_jobs, cudaStream_t st)
{
    if constexpr (MODE == K3_GROUP_GRAD_W && !CUT)
        if (a.Nc * sizeof(O) % 16) return launch_tc<MODE, O, FOLD, true>(maps, a, max_jobs, st);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    const int fit = fit_clusters<MODE, O, CUT, SPLIT, FOLD>(cfg, attr, st);
    if (fit < 1) return K3MOE_ERR_CUDA;
    a.pairs = (int)std::min<int64_t>(max_jobs, fit);
    cfg.gridDim = dim3(2 * SPLIT * (unsigned)a.pairs);
    cudaLaunchKernelEx(&cfg, group_tc_kernel<MODE, O, CUT, SPLIT, FOLD>, maps, a);
    k3_note_launch();
    return cudaGetLastError() == cudaSuccess ? K3MOE_OK : K3MOE_ERR_CUDA;
}

// mm, grad_x: most tiles of the widest kind: at most one partly filled one an expert with rows.
static int64_t widest_tiles(const GroupTcArgs &a)
{
    return ((int64_t)a.rows / GT_TILE_N + std::min(a.E, a.rows)) * ((a.M + GT_TILE_M - 1) / GT_TILE_M);
}

// mm, grad_x: cycles that a call takes on `clusters` clusters of `split` pairs beyond its launch, its rows spread evenly
// and its tiles chosen as the kernel does.  Measured on 33 shapes of one to 2,048 rows and 256 to 6144 contraction values,
// the sum is within 10 %: a stage costs 256 + n cycles and not less than 370, a tile's end 26 n; adding up the parts
// 1,600 and, as the network between SMs brings 8 bytes a cycle, 66 for each column that comes from another pair.
static int64_t tile_cycles(const GroupTcArgs &a, int split, int clusters)
{
    const int64_t mb = (a.M + GT_TILE_M - 1) / GT_TILE_M, steps = (a.K + GT_BK - 1) / GT_BK;
    const int64_t live = std::min(a.E, a.rows), each = (a.rows + live - 1) / live;
    int64_t best = 0, n = 0, rounds = 0;
    for (int i = 0; i < GT_TILE_PICKS; ++i) {
        const int64_t tile = GT_TILE_N >> i, tiles = (each + tile - 1) / tile, r = (live * tiles * mb + clusters - 1) / clusters;
        if (i == 0 || r * (256 + tile) < best) {
            best = r * (256 + tile);
            rounds = r;
            n = ((each + tiles - 1) / tiles + 15) & ~(int64_t)15;
        }
    }
    return rounds * ((steps + split - 1) / split) * std::max<int64_t>(370, 256 + n) + 26 * n +
           (split > 1 ? 1600 + 66 * n * (split - 1) / split : 0);
}

// One pair a tile, or two or four where every tile then has a cluster of its own (whatever the offsets hold) and
// that is faster: 1 row, 6144 to 64: 9.8 us with four, 14.5 with two, 22.8 with one; 16 experts of a row, 4096 to 512:
// 12.7 with two, 17.1 with one; 1,024 rows, 1024 to 512: 10.8, 8.4, 8.0.
template <int MODE, class O, bool FOLD>
static int launch_rows(const GroupMaps &maps, const GroupTcArgs &a, int64_t max_jobs, cudaStream_t st)
{
    const int64_t tiles = widest_tiles(a), steps = (a.K + GT_BK - 1) / GT_BK;
    const int pairs = k3_num_sms() / 2;
    if (tiles <= pairs / 2) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[2];
        int64_t best = tile_cycles(a, 1, pairs);
        int split = 1;
        const int fit[2] = {fit_clusters<MODE, O, false, 2, FOLD>(cfg, attr, st),
                            fit_clusters<MODE, O, false, 4, FOLD>(cfg, attr, st)};
        for (int i = 0; i < 2; ++i) {
            if (tiles > fit[i] || steps < (2 << i)) continue;            // each pair has a stage
            const int64_t c = tile_cycles(a, 2 << i, fit[i]);
            if (c < best) best = c, split = 2 << i;
        }
        if (split == 4) return launch_tc<MODE, O, FOLD, false, 4>(maps, a, max_jobs, st);
        if (split == 2) return launch_tc<MODE, O, FOLD, false, 2>(maps, a, max_jobs, st);
    }
    return launch_tc<MODE, O, FOLD>(maps, a, max_jobs, st);
}

// grad_w the same way, its rows spread evenly: 550 cycles a stage, 500 and 40 a column for the parts.  One expert,
// 2048 x 256, 32,768 rows: 62 us with four pairs a tile, 97 with two, 168 with one; 1,500 rows, 256 x 256: 16.9, 18.9, 21.0;
// 1,000 rows: 17 with any.
template <class O>
static int launch_grad_w(const GroupMaps &maps, const GroupTcArgs &a, int64_t jobs, cudaStream_t st)
{
    constexpr int MODE = K3_GROUP_GRAD_W;
    const int pairs = k3_num_sms() / 2;
    if (jobs <= pairs / 2 && a.Nc * sizeof(O) % 16 == 0) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[2];
        const int64_t steps = (((int64_t)a.rows + a.E - 1) / a.E + GT_BK - 1) / GT_BK, n = std::min(a.Nc, GT_TILE_N);
        const int fit[2] = {fit_clusters<MODE, O, false, 2, true>(cfg, attr, st),
                            fit_clusters<MODE, O, false, 4, true>(cfg, attr, st)};
        int64_t best = steps * 550;
        int split = 1;
        for (int i = 0; i < 2; ++i) {
            const int k = 2 << i;
            const int64_t c = (steps + k - 1) / k * 550 + 500 + 40 * n * (k - 1) / k;
            if (jobs <= fit[i] && c < best) best = c, split = k;
        }
        if (split == 4) return launch_tc<MODE, O, true, false, 4>(maps, a, jobs, st);
        if (split == 2) return launch_tc<MODE, O, true, false, 2>(maps, a, jobs, st);
    }
    return launch_tc<MODE, O, true>(maps, a, jobs, st);
}

template <int MODE, class O>
static int launch_mode(const GroupMaps &maps, const GroupTcArgs &a, int64_t max_jobs, cudaStream_t st)
{
    if constexpr (MODE == K3_GROUP_GRAD_W) return launch_grad_w<O>(maps, a, max_jobs, st);
    else if (a.K > (sizeof(O) == 4 ? GT_BK << a.part : GT_LONG)) return launch_rows<MODE, O, true>(maps, a, max_jobs, st);
    else return launch_rows<MODE, O, false>(maps, a, max_jobs, st);
}

template <int MODE>
static int launch_typed(const GroupMaps &maps, const GroupTcArgs &a, int out_type, int64_t max_jobs, cudaStream_t st)
{
    if (k3_num_sms() < 2) return K3MOE_ERR_CUDA;
    if (out_type == K3MOE_TYPE_F32) return launch_mode<MODE, float>(maps, a, max_jobs, st);
    if (out_type == K3MOE_TYPE_BF16) return launch_mode<MODE, __nv_bfloat16>(maps, a, max_jobs, st);
    return launch_mode<MODE, __half>(maps, a, max_jobs, st);
}

}  // namespace k3

using namespace k3;

bool k3_group_tc_fits(int mode, const K3Group &g)
{
    if (mode == K3_GROUP_GRAD_W)
        return g.rows > 0 && k3_rows16(g.a, g.lda, g.dtype) && k3_rows16(g.b, g.ldb, g.dtype) &&
               k3_rows16(g.out, g.ldo, g.out_dtype) && (g.E == 1 || (g.stride_o * k3_type_bytes(g.out_dtype)) % 16 == 0);
    return k3_rows16(g.a, g.lda, g.dtype) && k3_rows16(g.b, g.ldb, g.dtype) && (g.E == 1 || (g.stride_b * 2) % 16 == 0);
}

int k3_group_tc(int mode, const K3Group &g, cudaStream_t st)
{
    GroupMaps maps;
    GroupTcArgs a = {};
    a.offsets = g.offsets;
    a.E = g.E;
    a.rows = g.rows;
    a.bf16 = g.dtype == K3MOE_TYPE_BF16;
    a.part = a.bf16 ? GT_PART_BF16 : GT_PART_F16;
    a.accumulate = g.accumulate;
    a.out = g.out;
    a.ldo = g.ldo;
    a.stride_o = g.stride_o;
    a.status = g.status;
    bool ok = true;
    if (mode == K3_GROUP_GRAD_W) {
        a.M = g.n_out;
        a.Nc = g.n_in;
        a.expert_coord = 1;
        const int64_t so = g.E > 1 ? g.stride_o : (int64_t)g.n_out * g.ldo;
        a.wide_a = g.n_out % 64 == 0;
        a.wide_b = g.n_in % 64 == 0;
        ok = (a.wide_a ? encode_wide(&maps.a, g.dtype, g.a, g.n_out, g.rows, 0, g.lda, 0)
                       : encode_rows(&maps.a, g.dtype, g.a, g.n_out, g.rows, 0, g.lda, 0, 64)) &&
             (a.wide_b ? encode_wide(&maps.b[0], g.dtype, g.b, g.n_in, g.rows, 0, g.ldb, 0)
                       : encode_rows(&maps.b[0], g.dtype, g.b, g.n_in, g.rows, 0, g.ldb, 0, 64)) &&
             encode_rows(&maps.out, g.out_dtype, g.out, g.n_in, g.n_out, g.E, g.ldo, so, 32);
        for (int i = 1; i < 5; ++i) maps.b[i] = maps.b[0];
        if (!ok) return K3MOE_ERR_CUDA;
        const int64_t jobs = (int64_t)g.E * ((a.M + GT_TILE_M - 1) / GT_TILE_M) * ((a.Nc + GT_TILE_N - 1) / GT_TILE_N);
        if (jobs >= (1LL << 30)) return K3MOE_ERR_SHAPE;
        return launch_typed<K3_GROUP_GRAD_W>(maps, a, g.out_dtype, jobs, st);
    }
    const bool mm = mode == K3_GROUP_MM;
    a.M = mm ? g.n_out : g.n_in;
    a.K = mm ? g.n_in : g.n_out;
    // one weight for all experts: a single matrix at coordinate 0
    a.expert_coord = g.E > 1 && g.stride_b > 0;
    a.l2_rows = (int)std::max<int64_t>(GT_TILE_N, GT_L2_ROWS / ((int64_t)a.K * 2));
    const int64_t nw = a.expert_coord ? g.E : 1, sw = a.expert_coord ? g.stride_b : (int64_t)g.n_out * g.ldb;
    a.wide_a = !mm && g.n_in % 64 == 0;
    ok = a.wide_a ? encode_wide(&maps.a, g.dtype, g.b, g.n_in, g.n_out, nw, g.ldb, sw)
                  : encode_rows(&maps.a, g.dtype, g.b, g.n_in, g.n_out, nw, g.ldb, sw, mm ? 128 : 64);
    for (int i = 0; i < 5; ++i) ok = ok && encode_rows(&maps.b[i], g.dtype, g.a, a.K, g.rows, 0, g.lda, 0, 128 >> i);
    maps.out = maps.a;
    a.out16 = k3_rows16(g.out, g.ldo, g.out_dtype);
    if (!ok) return K3MOE_ERR_CUDA;
    // at most one partly filled tile an expert with rows, in the narrowest tiles
    const int64_t jobs = ((int64_t)g.rows / (GT_TILE_N >> (GT_TILE_PICKS - 1)) + std::min(g.E, g.rows)) *
                         ((a.M + GT_TILE_M - 1) / GT_TILE_M);
    if (jobs >= (1LL << 30)) return K3MOE_ERR_SHAPE;
    return mm ? launch_typed<K3_GROUP_MM>(maps, a, g.out_dtype, jobs, st)
              : launch_typed<K3_GROUP_GRAD_X>(maps, a, g.out_dtype, jobs, st);
}
