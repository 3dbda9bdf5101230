// row_codes.cuh -- codes of a row in 8-bit integers with one scale, for the kernels
// that make them (moe_quantize_rows, moe_norm_rows).
#pragma once

#include <cmath>

#include "rows.cuh"

namespace moe {

// Codes of C values v, |v| <= m: rint of the quotient 127 v / m as fp32 rounds
// it.  c = 127 / m has two roundings and v c is taken exactly, within 2^-15 of
// that quotient, so where it is further than 2^-13 from half way between two
// integers it rounds the same; a chunk with a value that is not, one chunk in
// 512, is divided.  Adding 1.5 * 2^23 rounds to an integer and leaves it in the
// low bits.  `by` is not 1 for rows of extreme size, which are all divided.
template <int C>
__device__ __forceinline__ Chunk<int8_t, C> quant_codes(const float (&v)[C], float c, float m, float by) {
    constexpr float kBig = 12582912.f;
    float near = by == 1.f ? 0.f : 1.f, n[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        n[i] = __fmaf_rn(v[i], c, kBig);
        near = fmaxf(near, fabsf(__fmaf_rn(v[i], c, kBig - n[i])));
    }
    if (near > 0.5f - 0x1p-13f) {
#pragma unroll
        for (int i = 0; i < C; ++i) n[i] = __fadd_rn(__fdiv_rn(__fmul_rn(v[i] * by, 127.f), m), kBig);
    }
    Chunk<int8_t, C> out;
    if constexpr (C % 4 == 0) {
#pragma unroll
        for (int i = 0; i < C; i += 4) {
            const uint32_t lo = __byte_perm(__float_as_uint(n[i]), __float_as_uint(n[i + 1]), 0x0040);
            const uint32_t hi = __byte_perm(__float_as_uint(n[i + 2]), __float_as_uint(n[i + 3]), 0x0040);
            reinterpret_cast<uint32_t*>(out.v)[i / 4] = __byte_perm(lo, hi, 0x5410);
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) out.v[i] = (int8_t)__float_as_int(n[i]);
    }
    return out;
}

// Largest magnitude of a chunk as bits, in which infinities and NaN are above all
// numbers: 16-bit types two at a time (both halves of the result), fp32 alone.
template <typename A, int C>
__device__ __forceinline__ uint32_t top_bits(const Chunk<A, C>& c, uint32_t top) {
    if constexpr (sizeof(A) == 2 && C % 2 == 0) {
#pragma unroll
        for (int i = 0; i < C; i += 2)
            top = __vmaxu2(top, *reinterpret_cast<const uint32_t*>(&c.v[i]) & 0x7FFF7FFFu);
    } else if constexpr (sizeof(A) == 2) {
        top = __vmaxu2(top, *reinterpret_cast<const uint16_t*>(&c.v[0]) & 0x7FFFu);
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) top = max(top, *reinterpret_cast<const uint32_t*>(&c.v[i]) & 0x7FFFFFFFu);
    }
    return top;
}

// The warp's largest magnitude, as bits of fp32, from its threads' top_bits.
template <typename A>
__device__ __forceinline__ uint32_t warp_most(uint32_t top) {
    if (sizeof(A) == 2) {
        const uint16_t h = (uint16_t)max(top & 0xFFFFu, top >> 16);
        top = __float_as_uint(to_f32(*reinterpret_cast<const A*>(&h)));
    }
    return __reduce_max_sync(0xFFFFFFFFu, top);
}

// The block's; part: one word a warp.
template <typename A>
__device__ __forceinline__ float block_most(uint32_t top, uint32_t* part) {
    top = warp_most<A>(top);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
    __syncthreads();
    top = part[0];
    for (int a = 1; a < (int)(blockDim.x >> 5); ++a) top = max(top, part[a]);
    return __uint_as_float(top);
}

// What the codes of a row with this largest magnitude need.
struct RowScale {
    float scale;      // most / 127; NaN for a row with an infinity or a NaN
    bool live;        // a finite row, not all zeros
    float by, m, c127;  // 127 v must not overflow, nor may 1 / m: v by / m by
};

__device__ __forceinline__ RowScale row_scale(float most) {
    RowScale r;
    r.live = most > 0.f && most < INFINITY;
    r.by = most > 0x1p119f ? 0x1p-8f : most < 0x1p-100f ? 0x1p100f : 1.f;
    r.m = most * r.by;
    r.c127 = __fmul_rn(127.f, __frcp_rn(r.m));
    r.scale = most < INFINITY ? __fdiv_rn(most, 127.f) : NAN;
    return r;
}

}  // namespace moe
