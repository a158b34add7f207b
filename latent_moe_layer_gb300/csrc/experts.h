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

// Two values of a 16-bit type in a register, low half first.
template <class T> __device__ __forceinline__ float2 unpack2(uint32_t w);
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t w)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <class T> __device__ __forceinline__ uint32_t pack2(float a, float b);      // rounded to nearest even
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b)
{
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// A piece of memory of V elements: 16 bytes kept as words until they are used (16-bit values held one to a
// register cost the bf16 kernels up to 40 registers), or one element.
template <class T, int V>
struct alignas(16) Vec {
    static_assert(V * sizeof(T) == 16, "16 bytes, or one element");
    uint32_t w[4];
    // elements j and j + 1, j even
    __device__ __forceinline__ float2 get2(int j) const
    {
        if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[j]), __uint_as_float(w[j + 1]));
        else return unpack2<T>(w[j / 2]);
    }
    __device__ __forceinline__ void set2(int j, float a, float b)
    {
        if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(a), w[j + 1] = __float_as_uint(b);
        else w[j / 2] = pack2<T>(a, b);
    }
};
template <class T>
struct Vec<T, 1> {
    T v;
    __device__ __forceinline__ float2 get2(int) const { return make_float2(to_f32(v), 0.f); }
    __device__ __forceinline__ void set2(int, float a, float) { v = from_f32<T>(a); }
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
