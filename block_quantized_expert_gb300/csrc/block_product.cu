// block_product.cu -- rows in blocks of 4-bit codes times experts in the same
// blocks over the sorted segments (moe_block_product; C entry at the end).
//
//   out[p, n] = scale[r] w_scale[e, n] sum_i v[r, i] w[e, n, i]
//
// for the positions p of expert e's segment, r the row that position p reads, v
// and w the blocks' values (code times block scale).
#include <atomic>
#include <type_traits>

#include "block_product.cuh"
#include "entry.h"

namespace moe {
namespace {

// One block a tile of 64 positions of one segment x 64 channels, 32 of K at a time
// as fp32 through shared memory, 4 x 4 sums a thread.
template <typename O, bool kNv>
__global__ void __launch_bounds__(256) k_block_product_any(const BlockProduct a) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int kTile = 64;
    __shared__ int sm_e, sm_j;
    __shared__ float xs[kTile][33], ws[kTile][33];
    __shared__ int src[kTile];
    const int tid = threadIdx.x;
    if (tid == 0) {
        int left = blockIdx.y;
        sm_e = -1;
        for (int e = 0; e < a.E; ++e) {
            const int n = (max(segment_at(a, e + 1) - segment_at(a, e), 0) + kTile - 1) / kTile;
            if (left < n) {
                sm_e = e;
                sm_j = left;
                break;
            }
            left -= n;
        }
    }
    __syncthreads();
    const int e = sm_e, n0 = blockIdx.x * kTile;
    if (e < 0) return;
    const int p0 = segment_at(a, e) + kTile * sm_j;
    const int count = min(kTile, segment_at(a, e + 1) - p0);
    if (tid < kTile) src[tid] = tid < count ? source_row(a, p0 + tid) : -1;
    __syncthreads();
    // this thread brings eight elements of one row
    const int lr = tid >> 2, lc = (tid & 3) * 8, tx = tid & 15, ty = tid >> 4;
    const int blocks = a.K / (kNv ? 16 : 32);
    auto bring = [&](float (&row)[33], const uint8_t* q, const uint8_t* s, int k) {
        const float f = q ? block_scale<kNv>(s[(k + lc) / (kNv ? 16 : 32)]) : 0.f;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const uint32_t c = q ? q[(k + lc + i) / 2] : 0u;
            row[lc + i] = q ? e2m1_to_f32(c & 15u) * f : 0.f;
            row[lc + i + 1] = q ? e2m1_to_f32(c >> 4) * f : 0.f;
        }
    };
    const bool has_x = src[lr] >= 0, has_w = n0 + lr < a.N;
    const uint8_t* xq = has_x ? a.q + src[lr] * a.qs : nullptr;
    const uint8_t* xb = has_x ? a.s + (long long)src[lr] * blocks : nullptr;
    const long long wr = (long long)e * a.N + n0 + lr;
    const uint8_t* wq = has_w ? a.wq + wr * (a.K / 2) : nullptr;
    const uint8_t* wb = has_w ? a.ws + wr * blocks : nullptr;
    float acc[4][4] = {};
    for (int k = 0; k < a.K; k += 32) {
        bring(xs[lr], xq, xb, k);
        bring(ws[lr], wq, wb, k);
        __syncthreads();
#pragma unroll 8
        for (int c = 0; c < 32; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[ty + 16 * i][c], ws[tx + 16 * j][c], acc[i][j]);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int p = ty + 16 * i;
        if (p >= count) continue;
        const float s = src[p] < 0 ? 0.f : a.scale ? a.scale[src[p]] : 1.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + tx + 16 * j;
            if (n < a.N)
                reinterpret_cast<O*>(a.out)[(long long)(p0 + p) * a.os + n] =
                    from_f32<O>(acc[i][j] * s * (a.w_scale ? a.w_scale[(long long)e * a.N + n] : 1.f));
        }
    }
}

// Positions past the last segment are written as zeros.
template <typename O>
__global__ void __launch_bounds__(256) k_block_tail(const BlockProduct a) {
    pdl_launch_dependents();
    pdl_wait();
    for (long long p = segment_at(a, a.E) + (long long)blockIdx.x; p < a.R; p += gridDim.x)
        for (int n = threadIdx.x; n < a.N; n += blockDim.x) reinterpret_cast<O*>(a.out)[p * a.os + n] = from_f32<O>(0.f);
}

template <typename O>
cudaError_t product_o(const BlockProduct& a, bool nv, cudaStream_t s) {
    const long long tiles = (long long)a.R / 64 + (a.E < a.R ? a.E : a.R);  // at most one partly filled tile an expert
    const dim3 grid((a.N + 63) / 64, (unsigned)tiles);
    cudaError_t e = launch_pdl(nv ? k_block_product_any<O, true> : k_block_product_any<O, false>, grid, dim3(256), 0, s, a);
    if (e == cudaSuccess && a.offsets) e = launch_pdl(k_block_tail<O>, dim3(a.R < 152 ? a.R : 152), dim3(256), 0, s, a);
    return e;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_block_product(const uint8_t* q, long long q_stride, int q_rows, const uint8_t* s,
                                        const float* scale, int K, int format, const uint8_t* wq, const uint8_t* ws,
                                        const float* w_scale, int n_experts, int N, const int32_t* offsets,
                                        const int32_t* row_src, int top_k, int R, void* out, moe_dtype out_dtype,
                                        long long out_stride, moe_stream_t stream) {
    const char* what = "moe_block_product";
    if (!dtype_ok(out_dtype)) return refuse(MOE_ERR_INVALID_ARG, "%s: unknown dtype", what);
    if (format != MOE_WEIGHTS_MXFP4 && format != MOE_WEIGHTS_NVFP4)
        return refuse(MOE_ERR_INVALID_ARG, "%s: unknown format", what);
    if (K < 32 || K > 131072 || K % 32 != 0)
        return refuse(MOE_ERR_INVALID_ARG, "%s: K must be a multiple of 32 in [32, 131072]", what);
    if (N < 1 || N > (1 << 20)) return refuse(MOE_ERR_INVALID_ARG, "%s: N must be in [1, 2^20]", what);
    if (n_experts < 1 || n_experts > kMaxExperts)
        return refuse(MOE_ERR_INVALID_ARG, "%s: n_experts must be in [1, 1024]", what);
    if (R < 0 || R > (1 << 20) || q_rows < 0) return refuse(MOE_ERR_INVALID_ARG, "%s: R must be in [0, 2^20]", what);
    if (!row_src && q_rows < R) return refuse(MOE_ERR_INVALID_ARG, "%s: q has fewer rows than out", what);
    if (row_src && (top_k < 1 || top_k > kMaxTopK))
        return refuse(MOE_ERR_INVALID_ARG, "%s: top_k must be in [1, 8]", what);
    if (!offsets && n_experts != 1) return refuse(MOE_ERR_INVALID_ARG, "%s: several experts need offsets", what);
    if (q_stride < K / 2 || out_stride < N || q_stride > kMostStride || out_stride > kMostStride)
        return refuse(MOE_ERR_INVALID_ARG, "%s: a row stride is below the row or above 2^40", what);
    if (q_stride % 16 != 0) return refuse(MOE_ERR_INVALID_ARG, "%s: q_stride must be a multiple of 16", what);
    if (R == 0) return MOE_OK;
    if (!q || !s || !wq || !ws || !out) return refuse(MOE_ERR_INVALID_ARG, "%s: NULL pointer", what);
    if ((uintptr_t)q % 16 || (uintptr_t)wq % 16)
        return refuse(MOE_ERR_INVALID_ARG, "%s: q and wq must be aligned to 16 bytes", what);
    if ((uintptr_t)out % dtype_size(out_dtype))
        return refuse(MOE_ERR_INVALID_ARG, "%s: out is not aligned to its elements", what);
    const BlockProduct a{q, q_stride, q_rows, s, scale, K, wq, ws, w_scale, n_experts, N, offsets, row_src, top_k, R, out,
                         out_stride, 2000000000ull, 0};
    cudaStream_t str = (cudaStream_t)stream;
    const bool nv = format == MOE_WEIGHTS_NVFP4;
    cudaError_t e;
    if (out_dtype == MOE_F32) e = product_o<float>(a, nv, str);
    else if (out_dtype == MOE_BF16) e = product_o<__nv_bfloat16>(a, nv, str);
    else e = product_o<__half>(a, nv, str);
    return status_of(e, what);
}
