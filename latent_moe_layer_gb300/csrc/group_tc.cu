// Products grouped by expert on the tensor cores (k3moe_group_mm, _grad_x, _grad_w): launches of group_tc.cuh's kernel.
#include "group_tc.cuh"

namespace k3 {

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
        const int64_t jobs = (int64_t)g.E * ((a.M + GT_TILE_M - 1) / GT_TILE_M) * ((a.Nc + GT_TILE_MAX - 1) / GT_TILE_MAX);
        if (jobs >= (1LL << 30)) return K3MOE_ERR_SHAPE;
        return launch_typed<K3_GROUP_GRAD_W>(maps, a, g.out_dtype, jobs, st);
    }
    const bool mm = mode == K3_GROUP_MM;
    a.M = mm ? g.n_out : g.n_in;
    a.K = mm ? g.n_in : g.n_out;
    // one weight for all experts: a single matrix at coordinate 0
    a.expert_coord = g.E > 1 && g.stride_b > 0;
    a.l2_rows = (int)std::max<int64_t>(GT_TILE_MAX, GT_L2_ROWS / ((int64_t)a.K * 2));
    const int64_t nw = a.expert_coord ? g.E : 1, sw = a.expert_coord ? g.stride_b : (int64_t)g.n_out * g.ldb;
    a.wide_a = !mm && g.n_in % 64 == 0;
    ok = a.wide_a ? encode_wide(&maps.a, g.dtype, g.b, g.n_in, g.n_out, nw, g.ldb, sw)
                  : encode_rows(&maps.a, g.dtype, g.b, g.n_in, g.n_out, nw, g.ldb, sw, mm ? 128 : 64);
    for (int i = 0; i < 5; ++i) ok = ok && encode_rows(&maps.b[i], g.dtype, g.a, a.K, g.rows, 0, g.lda, 0, 128 >> i);
    maps.out = maps.a;
    a.out16 = k3_rows16(g.out, g.ldo, g.out_dtype);
    if (!ok) return K3MOE_ERR_CUDA;
    // at most one partly filled tile an expert with rows, in the narrowest tiles
    const int64_t jobs = ((int64_t)g.rows / (GT_TILE_MAX >> (GT_TILE_PICKS - 1)) + std::min(g.E, g.rows)) *
                         ((a.M + GT_TILE_M - 1) / GT_TILE_M);
    if (jobs >= (1LL << 30)) return K3MOE_ERR_SHAPE;
    return mm ? launch_typed<K3_GROUP_MM>(maps, a, g.out_dtype, jobs, st)
              : launch_typed<K3_GROUP_GRAD_X>(maps, a, g.out_dtype, jobs, st);
}
