// rows.cuh -- vectors of 1 to 8 elements of one row in fp32, for the kernels
// that take rows in fp32, bf16 or fp16 (moe_dtype).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

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

// 16-bit types two at a time, in one conversion.
template <typename T, int C>
__device__ __forceinline__ Chunk<T, C> pack_chunk(const float (&f)[C]) {
    Chunk<T, C> c;
    if constexpr (sizeof(T) == 2 && C % 2 == 0) {
#pragma unroll
        for (int i = 0; i < C; i += 2) {
            if constexpr (std::is_same<T, __half>::value)
                *reinterpret_cast<__half2*>(&c.v[i]) = __floats2half2_rn(f[i], f[i + 1]);
            else
                *reinterpret_cast<__nv_bfloat162*>(&c.v[i]) = __floats2bfloat162_rn(f[i], f[i + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) c.v[i] = from_f32<T>(f[i]);
    }
    return c;
}

// The other way: 16-bit types by words (as single elements the compiler gives each bf16 a
// register of its own).
template <typename T, int C>
__device__ __forceinline__ void unpack_chunk(const Chunk<T, C>& c, float (&f)[C]) {
    if constexpr (sizeof(T) == 2 && C % 2 == 0) {
#pragma unroll
        for (int i = 0; i < C; i += 2) {
            if constexpr (std::is_same<T, __half>::value) {
                const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&c.v[i]));
                f[i] = v.x;
                f[i + 1] = v.y;
            } else {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(&c.v[i]);
                f[i] = __uint_as_float(w << 16);
                f[i + 1] = __uint_as_float(w & 0xFFFF0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) f[i] = to_f32(c.v[i]);
    }
}

template <typename T, int C>
__device__ __forceinline__ void store_chunk(T* p, const float (&f)[C]) {
    *reinterpret_cast<Chunk<T, C>*>(p) = pack_chunk<T, C>(f);
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
