// Internal declarations of the expert training operators (rows.cu, glu_dropout.cu,
// group_mm.cu, group_tc.cu).
#pragma once

#include <algorithm>
#include <type_traits>

#include "k3moe_internal.h"

namespace k3 {

// 16-bit and fp32 element types by K3MOE_TYPE_* code.
template <int TYPE> struct TypeOf;
template <> struct TypeOf<K3MOE_TYPE_F32> { using t = float; };
template <> struct TypeOf<K3MOE_TYPE_BF16> { using t = __nv_bfloat16; };
template <> struct TypeOf<K3MOE_TYPE_F16> { using t = __half; };

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Two values rounded together (one conversion instruction for the 16-bit types).
__device__ __forceinline__ void store2(float *o, float a, float b) { o[0] = a, o[1] = b; }
__device__ __forceinline__ void store2(__nv_bfloat16 *o, float a, float b)
{
    *reinterpret_cast<__nv_bfloat162 *>(o) = __floats2bfloat162_rn(a, b);
}
__device__ __forceinline__ void store2(__half *o, float a, float b)
{
    *reinterpret_cast<__half2 *>(o) = __floats2half2_rn(a, b);
}

// V consecutive elements as one aligned access (V sizeof(T) = 2 to 32 bytes).
template <class T, int V>
struct alignas(V * sizeof(T) > 16 ? 16 : V * sizeof(T)) Vec {
    T v[V];
};

}  // namespace k3

inline int k3_type_bytes(int type) { return type == K3MOE_TYPE_F32 ? 4 : 2; }

// Bytes spanned by n rows of `len` elements with leading dimension ld.
inline size_t k3_span(int64_t n, int64_t len, int64_t ld, int type)
{
    return n > 0 && len > 0 ? (size_t)((n - 1) * ld + len) * k3_type_bytes(type) : 0;
}

inline bool k3_overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return na && nb && x < y + nb && y < x + na;
}

// Rows that may be read in 16-byte pieces: base and leading dimension.
inline bool k3_rows16(const void *p, int64_t ld, int type)
{
    return ((uintptr_t)p & 15) == 0 && (ld * k3_type_bytes(type)) % 16 == 0;
}

// Streaming multiprocessors of the current device (cached per device), 0 on failure.
int k3_num_sms();

// One product grouped by expert.  mm: a = x, out = y; grad_x: a = dy, out = dx; grad_w: a = dy,
// b = x, out = dw.
enum K3GroupMode { K3_GROUP_MM = 0, K3_GROUP_GRAD_X = 1, K3_GROUP_GRAD_W = 2 };
struct K3Group {
    const int32_t *offsets;
    int E, rows, n_in, n_out;
    const void *a;
    int64_t lda;
    const void *b;               // mm, grad_x: w; grad_w: x
    int64_t ldb, stride_b;
    void *out;
    int64_t ldo, stride_o;       // stride_o: grad_w's expert stride
    int dtype, out_dtype, accumulate;
    int *status;
};
int k3_group_generic(int mode, const K3Group &g, cudaStream_t st);
// Whether the tensor-core kernels take it (every row on a 16-byte boundary), and their launch.
bool k3_group_tc_fits(int mode, const K3Group &g);
int k3_group_tc(int mode, const K3Group &g, cudaStream_t st);
