// int_product.cuh -- what the kernels of moe_expert_product share: the call's
// arguments and the segments of the sorted positions.
#pragma once

#include "layer.h"
#include "rows.cuh"

namespace moe {

struct Product {
    const int8_t* q; long long qs; int rows; const float* scale; int K;
    const int8_t* wq; const float* w_scale; int E, N;
    const int32_t* offsets; const int32_t* row_src; int k;
    int R; void* out; long long os;
    unsigned long long wait_ns;  // limit of every wait of the tensor-core form
    int stall;                   // its copies never arrive (test of that limit)
};

// Segment bound of expert e, held inside [0, R] whatever the offsets are.
__device__ __forceinline__ int segment_at(const Product& a, int e) {
    return min(max(a.offsets ? a.offsets[e] : (e ? a.R : 0), 0), a.R);
}

// Row of q that position p reads, or -1.
__device__ __forceinline__ int source_row(const Product& a, int p) {
    const int r = a.row_src ? (a.row_src[p] < 0 ? -1 : a.row_src[p] / a.k) : p;
    return r < a.rows ? r : -1;
}

// The tensor-core form (int_product_tc.cu): K and qs multiples of 16, q and wq
// 16-byte aligned.
bool product_tc_fits(const Product& a);
// Its sticky error flag (common.cuh), taken (read and cleared in one step) after the
// stream's work.
cudaError_t product_flag(uint32_t* flag, cudaStream_t s);
cudaError_t launch_product_tc(const Product& a, moe_dtype out, cudaStream_t s);

}  // namespace moe
