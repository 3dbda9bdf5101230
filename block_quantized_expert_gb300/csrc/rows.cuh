// rows.cuh -- vectors of 1 to 8 elements of one row in fp32, for the kernels
// that take rows in fp32, bf16 or fp16 (moe_dtype).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// C elements of T moved in words of at most 16 bytes.
template <typename T, int C>
struct alignas(sizeof(T) * C < 16 ? sizeof(T) * C : 16) Chunk {
    T v[C];
};

template <typename T, int C>
__device__ __forceinline__ Chunk<T, C> load_chunk(const T* p) {
    return *reinterpret_cast<const Chunk<T, C>*>(p);
}

template <typename T, int C>
__device__ __forceinline__ void store_chunk(T* p, const float (&f)[C]) {
    Chunk<T, C> c;
#pragma unroll
    for (int i = 0; i < C; ++i) c.v[i] = from_f32<T>(f[i]);
    *reinterpret_cast<Chunk<T, C>*>(p) = c;
}

inline int dtype_size(moe_dtype d) { return d == MOE_F32 ? 4 : 2; }
inline bool dtype_ok(moe_dtype d) { return d == MOE_F32 || d == MOE_BF16 || d == MOE_F16; }

// Alignment (a power of two up to 16) that every row of `base` with this
// stride in bytes shares.
inline unsigned row_align(const void* base, long long stride_bytes) {
    const unsigned long long a = (unsigned long long)(uintptr_t)base | (unsigned long long)stride_bytes | 16ull;
    return (unsigned)(a & (~a + 1));
}

}  // namespace moe
