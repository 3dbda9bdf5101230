// block_product.cuh -- what the kernels of moe_block_product share: the call's
// arguments and the segments of the sorted positions.
#pragma once

#include "block_rows.cuh"
#include "layer.h"
#include "rows.cuh"

namespace moe {

struct BlockProduct {
    const uint8_t* q; long long qs; int rows; const uint8_t* s; const float* scale; int K;
    const uint8_t* wq; const uint8_t* ws; const float* w_scale; int E, N;
    const int32_t* offsets; const int32_t* row_src; int k;
    int R; void* out; long long os;
    unsigned long long wait_ns;  // limit of every wait of the tensor-core form
    int stall;                   // its copies never arrive (test of that limit)
};

// Segment bound of expert e, held inside [0, R] whatever the offsets are.
__device__ __forceinline__ int segment_at(const BlockProduct& a, int e) {
    return min(max(a.offsets ? a.offsets[e] : (e ? a.R : 0), 0), a.R);
}

// Row of q that position p reads, or -1.
__device__ __forceinline__ int source_row(const BlockProduct& a, int p) {
    const int r = a.row_src ? (a.row_src[p] < 0 ? -1 : a.row_src[p] / a.k) : p;
    return r < a.rows ? r : -1;
}

// The tensor-core form (block_product_tc.cu): q and wq 16-byte aligned, qs a multiple of 16.
cudaError_t launch_block_product_tc(const BlockProduct& a, bool nv, moe_dtype out, cudaStream_t s);
// Whether it takes a call with pairs of CTAs (else one CTA a tile) on a GPU of `sms` SMs.
bool block_product_pairs(int E, int R, int K, int N, int sms);
// Where the current device has its sticky error flag (common.cuh).
cudaError_t block_product_flag_at(uint32_t** flag);

}  // namespace moe
