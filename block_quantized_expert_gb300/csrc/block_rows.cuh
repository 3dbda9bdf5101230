// block_rows.cuh -- scale bytes of blocks of 4-bit codes in fp32.
#pragma once

#include "common.cuh"

namespace moe {

// UE8M0 byte; 255 is NaN (common.cuh's form is for scales that the layer made).
__device__ __forceinline__ float ue8m0_value(uint32_t c) {
    return c == 255u ? __uint_as_float(0x7FC00000u) : ue8m0_to_f32(c);
}

template <bool kNv>
__device__ __forceinline__ float block_scale(uint32_t c) {
    return kNv ? e4m3_to_f32(c) : ue8m0_value(c);
}

}  // namespace moe
