// Products of 8-bit operands with a scale for each block of 128, grouped by expert (k3moe_group_mm8): argument checks and the
// launch of group_tc.cuh's kernel with block-scaled MMAs.
//
// The scales are powers of two, so the tensor cores apply them (kind::mxf8f6f4, a scale for each 32 values: the four MMAs of a
// 128-value stage read the same byte) and a tile's sum stays in TMEM from end to end.  fp32 scales would take every stage's
// partial sums through registers: 256 x 240 values read and added in each 480 cycles.  A stage has the bytes of a 16-bit
// one (128 a row) and twice its products in the same time; tiles are 240 rows wide at most, as two accumulators leave 32
// columns for scales.  A warp of each CTA lays the scales out in shared memory (a word a row for four stages), tcgen05.cp
// copies them to tensor memory.
//
// 8192^3 in one group 307 us, 3.58 PFLOP/s (resident operands: 525 cycles a stage of 240 rows, 4.3 PFLOP/s; here about
// 580); 65,536 rows over 112 experts, 3584 to 6144, 957 us, 3.02 PFLOP/s (28 stages a tile: some 900 cycles a tile pass
// before its first MMAs); 251 rows over 112 experts with their quantising 328 us, the weights at 6.8 TB/s.  What truncation
// costs: at most 2e-6 of the sum of the products' sizes with fp32 outputs, which add up parts of 512 values.
#include "group_tc.cuh"

using namespace k3;

extern "C" int k3moe_group_mm8(const int32_t *offsets, int n_experts, int rows, int n_in, int n_out, const uint8_t *x, int64_t ldx,
                               int x_kind, const uint8_t *x_scales, int64_t ldxs, const uint8_t *w, int64_t ldw, int64_t stride_w,
                               int w_kind, const uint8_t *w_scales, int64_t sse, int64_t sso, int64_t ssi, void *y, int64_t ldy,
                               int out_dtype, int32_t *status, cudaStream_t stream)
{
    const int E = n_experts;
    if (E < 1 || rows < 0 || n_in < 1 || n_out < 1 || !offsets || !status) return K3MOE_ERR_ARG;
    if (E > K3MOE_TRAIN_MAX_EXPERTS || std::max({rows, n_in, n_out}) > K3_GROUP_MAX_SIZE) return K3MOE_ERR_SHAPE;
    for (const int kind : {x_kind, w_kind})
        if (kind != K3MOE_F8_E4M3 && kind != K3MOE_F8_E5M2) return K3MOE_ERR_UNSUPPORTED;
    if (out_dtype != K3MOE_TYPE_F32 && out_dtype != K3MOE_TYPE_BF16 && out_dtype != K3MOE_TYPE_F16) return K3MOE_ERR_UNSUPPORTED;
    if (rows > 0 && (!x || !x_scales || !w || !w_scales || !y)) return K3MOE_ERR_ARG;
    const int64_t blocks = ((int64_t)n_in + 127) / 128, w_blocks = ((int64_t)n_out + 127) / 128;
    if (ldx < n_in || ldw < n_in || ldy < n_out || ldxs < blocks) return K3MOE_ERR_ARG;
    if ((E > 1 && (stride_w < 0 || sse < 0)) || sso < 0 || ssi < 0) return K3MOE_ERR_ARG;
    // the copy engine's boundaries, and words of four x scales
    const int64_t strides = ldx | ldw | (E > 1 ? stride_w : 0);
    if (((uintptr_t)x | (uintptr_t)w | (uint64_t)strides) & 15 || ((uintptr_t)x_scales | (uint64_t)ldxs) & 3) return K3MOE_ERR_UNSUPPORTED;
    const int64_t more = E - 1;
    const size_t no = k3_span(rows, n_out, ldy, out_dtype), nx = rows ? (size_t)((rows - 1) * ldx + n_in) : 0,
                 nxs = rows ? (size_t)((rows - 1) * ldxs + blocks) : 0,
                 nw = (size_t)(more * stride_w + (n_out - 1) * ldw + n_in),
                 nws = (size_t)(more * sse + (w_blocks - 1) * sso + (blocks - 1) * ssi + 1);
    if (k3_overlap(y, no, x, nx) || k3_overlap(y, no, x_scales, nxs) || k3_overlap(y, no, w, nw) || k3_overlap(y, no, w_scales, nws) ||
        k3_overlap(y, no, offsets, sizeof(int32_t) * ((size_t)E + 1)))
        return K3MOE_ERR_ALIAS;
    if (!k3_aligned({{y, k3_type_bytes(out_dtype)}, {offsets, 4}, {status, 4}})) return K3MOE_ERR_ALIGN;
    if (rows == 0) return K3MOE_OK;
    GroupMaps maps;
    GroupMm8Args a = {};
    a.offsets = offsets;
    a.E = E;
    a.rows = rows;
    a.M = n_out;
    a.K = n_in;
    a.part = GT_PART_F8;
    a.out = y;
    a.ldo = ldy;
    a.out16 = k3_rows16(y, ldy, out_dtype);
    a.status = status;
    a.xs = x_scales;
    a.ldxs = ldxs;
    a.xs16 = (((uintptr_t)x_scales | (uint64_t)ldxs) & 15) == 0;
    a.ws = w_scales;
    a.sse = E > 1 ? sse : 0;
    a.sso = sso;
    a.ssi = ssi;
    a.blocks = (int)blocks;
    // the instruction descriptor's element types: 0 E4M3, 1 E5M2
    a.a_type = w_kind == K3MOE_F8_E5M2;
    a.b_type = x_kind == K3MOE_F8_E5M2;
    a.expert_coord = E > 1 && stride_w > 0;
    a.l2_rows = (int)std::max<int64_t>(GT_TILE_MAX, GT_L2_ROWS / (int64_t)n_in);
    bool ok = encode_rows(&maps.a, GT_BYTES, w, n_in, n_out, a.expert_coord ? E : 1, ldw, a.expert_coord ? stride_w : (int64_t)n_out * ldw, 128);
    for (int i = 0; i < 5; ++i) ok = ok && encode_rows(&maps.b[i], GT_BYTES, x, n_in, rows, 0, ldx, 0, 128 >> i);
    maps.out = maps.a;
    if (!ok || k3_num_sms() < 2) return K3MOE_ERR_CUDA;
    const int64_t jobs = most_tiles<K3_GROUP_MM8>(a, group_tile(K3_GROUP_MM8) >> (GT_TILE_PICKS - 1));
    if (jobs >= (1LL << 30)) return K3MOE_ERR_SHAPE;
    if (out_dtype == K3MOE_TYPE_F32) return launch_mode<K3_GROUP_MM8, float>(maps, a, jobs, stream);
    if (out_dtype == K3MOE_TYPE_BF16) return launch_mode<K3_GROUP_MM8, __nv_bfloat16>(maps, a, jobs, stream);
    return launch_mode<K3_GROUP_MM8, __half>(maps, a, jobs, stream);
}
