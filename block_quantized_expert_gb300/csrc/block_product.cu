// block_product.cu -- rows in blocks of 4-bit codes times experts in the same
// blocks over the sorted segments (moe_block_product; C entry at the end).
//
//   out[p, n] = scale[r] w_scale[e, n] sum_i v[r, i] w[e, n, i]
//
// for the positions p of expert e's segment, r the row that position p reads, v
// and w the blocks' values (code times block scale).
#include "block_product.cuh"
#include "entry.h"
#include "int_product.cuh"

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
    BlockProduct a{q, q_stride, q_rows, s, scale, K, wq, ws, w_scale, n_experts, N, offsets, row_src, top_k, R, out,
                         out_stride, 2000000000ull, 0};
    cudaStream_t str = (cudaStream_t)stream;
    const bool nv = format == MOE_WEIGHTS_NVFP4;
    if (take_product_stall()) {
        a.stall = 1;
        a.wait_ns = 5000000ull;
    }
    return status_of(launch_block_product_tc(a, nv, out_dtype, str), what);
}
