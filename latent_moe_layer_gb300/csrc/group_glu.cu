// The gated block's projections and unit in one pass, and their gradient (k3moe_group_glu, _grad): argument checks and the
// launches of group_tc.cuh's kernel whose tiles hold the gate and the up rows of the same columns.
//
// A tile's 256 weight rows are 16 gate rows and the 16 up rows of the same columns in turn, so that both projections of an
// output lie in one warp's quarter of the accumulator, 16 lanes apart: the warp's halves swap eight columns each (8 shuffles
// a 256 outputs) and nothing else of the product changes.  (Gate and up in accumulators of their own need twice the TMEM
// columns a row, which halves the tile's rows and with it the use of an operand; 64 rows of either in turn need an
// exchange between warps through shared memory.)  The gradient computes the projections again, 2 rows n_in 2 width
// operations, instead of reading 4 bytes an element of them that the forward pass would have had to write.
//
// dgu leaves in the operands' 16 bits, as grad_x and grad_w take it: their results lie 2.3e-3 (bf16; f16 2.9e-4) of their norm
// from 64 bits, against 1.66e-3 (2.1e-4) of the outputs' own rounding with dgu in fp32.
//
// Bound as the products: 251 rows over 112 experts, 3584 to 3072: 650 us, the weights at 6.8 TB/s (product and unit
// apart: 650 + 5); 32,768 rows over 56 experts 889 us, 1.62 PFLOP/s, in short runs (apart: 880 + 94) and 998-1,045 under the
// power cap.  One pass saves memory, not time, where there is a backward pass: 16,381 rows over 28 experts take 437 us and 471
// for the gradient, with stored projections (group_mm, the unit, the unit's gradient) 457 + 50 + 76.
#include "group_tc.cuh"

using namespace k3;

namespace k3 {

// Boxes of 16 gate rows and the same 16 up rows in turn: [E][width / 16][2][16][n_in], where width is whole blocks; else the
// matrices as they are, a box of 16 rows at a time.
static bool encode_glu(GroupMaps &maps, GroupTcArgs &a, const K3Group &g, int64_t nw, int64_t sw)
{
    a.wide_a = g.n_out % 16 == 0;
    if (!a.wide_a) return encode_rows(&maps.a, g.dtype, g.b, g.n_in, 2 * (int64_t)g.n_out, nw, g.ldb, sw, 16);
    return encode<5>(&maps.a, g.dtype, g.b, 5, {g.n_in, 16, 2, g.n_out / 16, nw}, {g.ldb, g.n_out * g.ldb, 16 * g.ldb, sw},
                     {64, 16, 2, 4, 1});
}

}  // namespace k3

int k3_group_glu_tc(const K3Group &g, const K3GroupGlu &u, cudaStream_t st)
{
    GroupMaps maps;
    GroupGluTcArgs a = {};
    a.offsets = g.offsets;
    a.E = g.E;
    a.rows = g.rows;
    a.M = g.n_out;
    a.K = g.n_in;
    a.bf16 = g.dtype == K3MOE_TYPE_BF16;
    a.part = a.bf16 ? GT_PART_BF16 : GT_PART_F16;
    a.out = g.out;
    a.ldo = g.ldo;
    a.status = g.status;
    a.situ = u.situ;
    a.glu = u.c;
    a.da = u.da;
    a.ldda = u.ldda;
    a.da16 = u.da && k3_rows16(u.da, u.ldda, g.dtype);
    // both halves of a gradient's row in 16-byte pieces
    a.out16 = k3_rows16(g.out, g.ldo, g.dtype) && (!u.da || g.n_out % 8 == 0);
    a.expert_coord = g.E > 1 && g.stride_b > 0;
    a.l2_rows = (int)std::max<int64_t>(GT_TILE_MAX, GT_L2_ROWS / ((int64_t)a.K * 2));
    const int64_t nw = a.expert_coord ? g.E : 1, sw = a.expert_coord ? g.stride_b : 2 * (int64_t)g.n_out * g.ldb;
    bool ok = encode_glu(maps, a, g, nw, sw);
    for (int i = 0; i < 5; ++i) ok = ok && encode_rows(&maps.b[i], g.dtype, g.a, a.K, g.rows, 0, g.lda, 0, 128 >> i);
    maps.out = maps.a;
    if (!ok || k3_num_sms() < 2) return K3MOE_ERR_CUDA;
    const int64_t jobs = most_tiles<K3_GROUP_GLU>(a, GT_TILE_MAX >> (GT_TILE_PICKS - 1));
    if (jobs >= (1LL << 30)) return K3MOE_ERR_SHAPE;
    if (u.da) return a.bf16 ? launch_mode<K3_GROUP_GLU_GRAD, __nv_bfloat16>(maps, a, jobs, st)
                            : launch_mode<K3_GROUP_GLU_GRAD, __half>(maps, a, jobs, st);
    return a.bf16 ? launch_mode<K3_GROUP_GLU, __nv_bfloat16>(maps, a, jobs, st) : launch_mode<K3_GROUP_GLU, __half>(maps, a, jobs, st);
}

// g: as of a product with 2 width outputs, whose weights they are; the output's own width is checked here.
static int glu_run(K3Group g, int act, float beta, float linear_beta, const void *da, int64_t ldda, bool grad, cudaStream_t st)
{
    const int width = g.n_out;
    if (width < 1 || width > (1 << 29)) return K3MOE_ERR_ARG;
    const int64_t ldo = g.ldo;
    const int cols = grad ? 2 * width : width;
    if (ldo < cols || (grad && g.rows > 0 && (!da || ldda < width))) return K3MOE_ERR_ARG;
    K3GroupGlu u = {act == K3MOE_ACT_SITU, {}, grad ? da : nullptr, ldda};
    if (const int rc = glu_args(act, beta, linear_beta, u.c)) return rc;
    // the products' checks for [rows, 2 width]; an output of half that width spans less
    g.n_out = 2 * width;
    K3Group full = g;
    full.out = nullptr;
    full.ldo = g.n_out;
    full.rows = 0;
    int rc = k3_group_check(full, K3_GROUP_MM);
    if (rc < 0) return rc;
    if (g.rows > K3_GROUP_MAX_SIZE) return K3MOE_ERR_SHAPE;
    if (g.rows < 0 || (g.rows > 0 && (!g.a || !g.b || !g.out)) || g.lda < g.n_in) return K3MOE_ERR_ARG;
    const size_t no = k3_span(g.rows, cols, ldo, g.dtype);
    const size_t nw = k3_span(1, (g.E - 1) * g.stride_b + (int64_t)(g.n_out - 1) * g.ldb + g.n_in, 0, g.dtype);
    if (k3_overlap(g.out, no, g.a, k3_span(g.rows, g.n_in, g.lda, g.dtype)) || k3_overlap(g.out, no, g.b, nw) ||
        k3_overlap(g.out, no, g.offsets, sizeof(int32_t) * ((size_t)g.E + 1)) ||
        (grad && k3_overlap(g.out, no, da, k3_span(g.rows, width, ldda, g.dtype))))
        return K3MOE_ERR_ALIAS;
    if (!k3_aligned({{g.out, 2}, {da, 2}})) return K3MOE_ERR_ALIGN;                      // (the others: above)
    if (g.rows == 0) return K3MOE_OK;
    g.n_out = width;
    const bool fits = k3_rows16(g.a, g.lda, g.dtype) && k3_rows16(g.b, g.ldb, g.dtype) && (g.E == 1 || (g.stride_b * 2) % 16 == 0);
    return fits ? k3_group_glu_tc(g, u, st) : k3_group_glu_generic(g, u, st);
}

extern "C" int k3moe_group_glu(const int32_t *offsets, int n_experts, int rows, int n_in, int width, const void *x, int64_t ldx,
                               const void *w, int64_t ldw, int64_t stride_w, int dtype, int act, float situ_beta,
                               float situ_linear_beta, void *a, int64_t lda, int32_t *status, cudaStream_t stream)
{
    const K3Group g = {offsets, n_experts, rows, n_in, width, x, ldx, w, ldw, stride_w, a, lda, 0, dtype, dtype, 0, status};
    return glu_run(g, act, situ_beta, situ_linear_beta, nullptr, 0, false, stream);
}

extern "C" int k3moe_group_glu_grad(const int32_t *offsets, int n_experts, int rows, int n_in, int width, const void *da,
                                    int64_t ldda, const void *x, int64_t ldx, const void *w, int64_t ldw, int64_t stride_w,
                                    int dtype, int act, float situ_beta, float situ_linear_beta, void *dgu, int64_t lddgu,
                                    int32_t *status, cudaStream_t stream)
{
    const K3Group g = {offsets, n_experts, rows, n_in, width, x, ldx, w, ldw, stride_w, dgu, lddgu, 0, dtype, dtype, 0, status};
    return glu_run(g, act, situ_beta, situ_linear_beta, da, ldda, true, stream);
}
