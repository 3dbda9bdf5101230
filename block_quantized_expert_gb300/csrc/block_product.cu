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

namespace moe {
namespace {

// ---------------------------------------------------------------- few rows --
// Single tokens: a warp takes kChan channels of one expert for up to kFew positions of
// its segment, lane l the 32 elements (16 bytes of codes) from 32 l, 32 l + 1024, ...
// Codes turn into fp16 by the hardware's converter; the products of 16 of them are summed
// in pairs in fp16, exactly (eight products of at most 36 in steps of a quarter: 1152 of
// 2048), then scaled and summed in fp32, and joined by shuffles.  Bound by the latency of its loads with
// few warps to hide it: one row of 4096 x 4096 has 10 % of the warps that fit, issues in 15 % of
// its cycles and fills no pipe past 18 %.  Block (x, p): channels 4 kChan x .. of the segment
// of position p, if p is the first of its kFew.
constexpr int kFew = 2, kChan = 4;

// 8 codes to 4 x 2 values in fp16.
__device__ __forceinline__ void codes_to_f16(uint32_t w, __half2 (&o)[4]) {
    uint32_t r[4];
    asm("{\n.reg .b8 b0, b1, b2, b3;\nmov.b32 {b0, b1, b2, b3}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\ncvt.rn.f16x2.e2m1x2 %1, b1;\n"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\ncvt.rn.f16x2.e2m1x2 %3, b3;\n}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = *reinterpret_cast<const __half2*>(&r[i]);
}

// The scales of a lane's 32 elements: two bytes, or one for both.
template <bool kNv>
__device__ __forceinline__ float2 lane_scales(const uint8_t* s, int at) {
    if (kNv) {
        const uint32_t lo = s[2 * at], hi = s[2 * at + 1];  // (rows of scales need not be aligned)
        const __half2 h = __half2(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)lo, __NV_E4M3)),
                                  __half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)hi, __NV_E4M3)));
        return __half22float2(h);
    }
    const float f = ue8m0_value(s[at]);
    return make_float2(f, f);
}

template <typename O, bool kNv>
__global__ void __launch_bounds__(128) k_block_product_few(const BlockProduct a) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ int sm_e, sm_begin, sm_end;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, p = blockIdx.y;
    if (threadIdx.x == 0) sm_e = -1;
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += 128) {
        const int b = segment_at(a, e), n = segment_at(a, e + 1);
        if (b <= p && p < n) {  // (offsets that are not in order may name several: any one)
            sm_e = e;
            sm_begin = b;
            sm_end = n;
        }
    }
    __syncthreads();
    const int e = sm_e, n0 = (blockIdx.x * 4 + warp) * kChan;
    if (e < 0) {  // past the last segment: zeros
        if (p >= segment_at(a, a.E) && lane < kChan && n0 + lane < a.N)
            reinterpret_cast<O*>(a.out)[(long long)p * a.os + n0 + lane] = from_f32<O>(0.f);
        return;
    }
    if ((p - sm_begin) % kFew != 0 || n0 >= a.N) return;
    const int rows = min(kFew, sm_end - p), pieces = a.K / 32, blocks = a.K / (kNv ? 16 : 32);
    int src[kFew];
#pragma unroll
    for (int r = 0; r < kFew; ++r) src[r] = r < rows ? source_row(a, p + r) : -1;
    const uint8_t *w[kChan], *ws[kChan];
#pragma unroll
    for (int c = 0; c < kChan; ++c) {
        const long long n = (long long)e * a.N + min(n0 + c, a.N - 1);
        w[c] = a.wq + n * (a.K / 2);
        ws[c] = a.ws + n * blocks;
    }
    float acc[kChan][kFew] = {};
    uint4 v[kChan];
    float2 s[kChan];
    auto load = [&](int i) {
        if (i >= pieces) return;
#pragma unroll
        for (int c = 0; c < kChan; ++c) {
            v[c] = __ldcs(reinterpret_cast<const uint4*>(w[c]) + i);
            s[c] = lane_scales<kNv>(ws[c], i);
        }
    };
    load(lane);
    for (int i = lane; i < pieces; i += 32) {
        uint4 now[kChan];
        float2 by[kChan];
#pragma unroll
        for (int c = 0; c < kChan; ++c) {
            now[c] = v[c];
            by[c] = s[c];
        }
        load(i + 32);
#pragma unroll
        for (int r = 0; r < kFew; ++r) {
            if (r >= rows) break;
            if (src[r] < 0) {  // no row: zeros, which a channel with a NaN byte still makes NaN
#pragma unroll
                for (int c = 0; c < kChan; ++c) acc[c][r] = fmaf(0.f, by[c].x, fmaf(0.f, by[c].y, acc[c][r]));
                continue;
            }
            const uint4 x = reinterpret_cast<const uint4*>(a.q + src[r] * a.qs)[i];
            const float2 xs = lane_scales<kNv>(a.s + (long long)src[r] * blocks, i);
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int c = 0; c < kChan; ++c) {
                const uint32_t ww[4] = {now[c].x, now[c].y, now[c].z, now[c].w};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    __half2 sum = __float2half2_rn(0.f);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        __half2 fx[4], fw[4];
                        codes_to_f16(xw[2 * h + j], fx);
                        codes_to_f16(ww[2 * h + j], fw);
#pragma unroll
                        for (int u = 0; u < 4; ++u) sum = __hfma2(fx[u], fw[u], sum);
                    }
                    const float2 f = __half22float2(sum);
                    acc[c][r] = fmaf(f.x + f.y, h ? xs.y * by[c].y : xs.x * by[c].x, acc[c][r]);
                }
            }
        }
    }
#pragma unroll
    for (int c = 0; c < kChan; ++c) {
        if (n0 + c >= a.N) break;
        const float cs = a.w_scale ? a.w_scale[(long long)e * a.N + n0 + c] : 1.f;
#pragma unroll
        for (int r = 0; r < kFew; ++r) {
            if (r >= rows) break;
            const float sum = warp_sum(acc[c][r]), rs = src[r] < 0 ? 0.f : a.scale ? a.scale[src[r]] : 1.f;
            if (lane == 0) reinterpret_cast<O*>(a.out)[(long long)(p + r) * a.os + n0 + c] = from_f32<O>(sum * rs * cs);
        }
    }
}

// Here and on the tensor cores, NVFP4, us (each call's weights from HBM):
//   K x N         one position   two of one expert   two of two experts
//   4096 x 4096   6.6            10.0 / 8.6          7.8 / 9.7
//   2048 x 4096   4.4             6.3 / 6.8          5.1 / 7.6
//   4096 x 1024   5.4             7.3 / 8.6          5.9 / 8.8
//   512 x 512     2.4             3.1 / 5.3          2.6 / 5.6
// MXFP4 at 4096 x 4096 10.9 / 8.0 and 9.1 / 9.0: two positions of one large expert alone lose, and which
// experts they are of is on the device.  One position of 4096 x 4096 takes 8.6 on the tensor cores; four take 11.3
// and 8.6 with two positions a warp, six of six experts 17.2 and 16.1.
bool few_rows(int R) { return R <= 2; }

cudaError_t launch_few(const BlockProduct& a, bool nv, moe_dtype out, cudaStream_t s) {
    const dim3 grid((a.N + 4 * kChan - 1) / (4 * kChan), a.R);
    auto run = [&](auto type) {
        using O = decltype(type);
        return launch_pdl(nv ? k_block_product_few<O, true> : k_block_product_few<O, false>, grid, dim3(128), 0, s, a);
    };
    if (out == MOE_F32) return run(float());
    if (out == MOE_BF16) return run(__nv_bfloat16());
    return run(__half());
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
    if (q_stride < K / 2 || out_stride < N || q_stride >= kMostStride || out_stride > kMostStride)
        return refuse(MOE_ERR_INVALID_ARG, "%s: a row stride is below the row or above 2^40 (q_stride: from 2^40 up)", what);
    if (q_stride % 16 != 0) return refuse(MOE_ERR_INVALID_ARG, "%s: q_stride must be a multiple of 16", what);
    if (R == 0) return MOE_OK;
    if (!q || !s || !wq || !ws || !out) return refuse(MOE_ERR_INVALID_ARG, "%s: NULL pointer", what);
    if ((uintptr_t)q % 16 || (uintptr_t)wq % 16)
        return refuse(MOE_ERR_INVALID_ARG, "%s: q and wq must be aligned to 16 bytes", what);
    if ((uintptr_t)out % dtype_size(out_dtype))
        return refuse(MOE_ERR_INVALID_ARG, "%s: out is not aligned to its elements", what);
    if (!aligned4(scale, w_scale, offsets, row_src))
        return refuse(MOE_ERR_INVALID_ARG, "%s: scale, w_scale, offsets or row_src is not aligned to its elements", what);
    BlockProduct a{q, q_stride, q_rows, s, scale, K, wq, ws, w_scale, n_experts, N, offsets, row_src, top_k, R, out,
                   out_stride, 2000000000ull, 0};
    cudaStream_t str = (cudaStream_t)stream;
    const bool nv = format == MOE_WEIGHTS_NVFP4;
    if (few_rows(R)) return status_of(launch_few(a, nv, out_dtype, str), what);
    if (take_product_stall()) {
        a.stall = 1;
        a.wait_ns = 5000000ull;
    }
    return status_of(launch_block_product_tc(a, nv, out_dtype, str), what);
}

extern "C" int moe_test_block_product_form(int n_experts, int R, int K, int N, int num_sms) {
    if (n_experts < 1 || R < 1 || K < 1 || N < 1 || num_sms < 2) return -1;
    return few_rows(R) ? 0 : block_product_pairs(n_experts, R, K, N, num_sms) ? 2 : 1;
}
