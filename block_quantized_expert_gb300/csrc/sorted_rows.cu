// sorted_rows.cu -- token rows to and from the experts' order, and the
// gradients on the way back (moe_dispatch, moe_combine, their backward forms
// and moe_route_backward; C entries at the end).
//
// A row r = t * k + j is slot j of token t; row_dst[r] is its position among
// the R = T * k sorted rows, or -1.  Every kernel walks tokens, not positions:
// a token's row is then read once for its k slots (dispatch), its k sorted
// rows are joined without atomics in a fixed order (combine), and one pass
// over y gives both dy and dw (combine_backward).  A position outside [0, R)
// counts as an empty slot.  All of it is bound by HBM; offsets are 64 bits.
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "layer.h"
#include "route.cuh"
#include "rows.cuh"

namespace moe {

namespace {

// ---------------------------------------------------------------- dispatch --
// xs[row_dst[t, j]] = x[t], in words of V: types do not matter to a copy.
// Reads T H, writes R H elements.
template <typename V>
__global__ void __launch_bounds__(128) k_dispatch(const char* __restrict__ x, long long x_pitch, int T, int k,
                                                  int words, const int32_t* __restrict__ placed,
                                                  const int32_t* __restrict__ row_dst, char* __restrict__ xs,
                                                  long long xs_pitch) {
    pdl_launch_dependents();
    pdl_wait();
    const long long R = (long long)T * k;
    for (long long t = blockIdx.x; t < T; t += gridDim.x) {
        const V* src = reinterpret_cast<const V*>(x + t * x_pitch);
        for (int c = threadIdx.x; c < words; c += blockDim.x) {
            const V v = src[c];
            for (int j = 0; j < k; ++j) {
                const long long p = row_dst[t * k + j];
                if (p >= 0 && p < R) reinterpret_cast<V*>(xs + p * xs_pitch)[c] = v;
            }
        }
    }
    // positions past the last placed row
    const V zero = V();
    for (long long p = max(*placed, 0) + (long long)blockIdx.x; p < R; p += gridDim.x)
        for (int c = threadIdx.x; c < words; c += blockDim.x) reinterpret_cast<V*>(xs + p * xs_pitch)[c] = zero;
}

// ----------------------------------------------------------------- combine --
// out[t] = sum_j w[t, j] y[row_dst[t, j]] over the filled slots in ascending
// position, which is ascending expert id, the order of the layer's own
// combine; w = NULL stands for ones (the gradient of dispatch).  The sum is
// held in fp32 and rounded once.
template <typename A, typename O, int C>
__global__ void __launch_bounds__(128) k_combine_rows(const A* __restrict__ y, long long ys,
                                                      const float* __restrict__ w, int T, int k, int H,
                                                      const int32_t* __restrict__ row_dst, O* __restrict__ out,
                                                      long long os) {
    pdl_launch_dependents();
    pdl_wait();
    const long long R = (long long)T * k;
    for (long long t = blockIdx.x; t < T; t += gridDim.x) {
        long long pos[kMaxTopK];
        float wt[kMaxTopK];
        int m = 0;  // filled slots, kept sorted by position
        for (int j = 0; j < k; ++j) {
            const long long p = row_dst[t * k + j];
            if (p < 0 || p >= R) continue;
            int a = m++;
            for (; a > 0 && pos[a - 1] > p; --a) {
                pos[a] = pos[a - 1];
                wt[a] = wt[a - 1];
            }
            pos[a] = p;
            wt[a] = w ? w[t * k + j] : 1.f;
        }
        for (int c = threadIdx.x * C; c < H; c += blockDim.x * C) {
            float acc[C];
#pragma unroll
            for (int i = 0; i < C; ++i) acc[i] = 0.f;
            for (int a = 0; a < m; ++a) {
                const Chunk<A, C> v = load_chunk<A, C>(y + pos[a] * ys + c);
#pragma unroll
                for (int i = 0; i < C; ++i) acc[i] += wt[a] * to_f32(v.v[i]);
            }
            store_chunk<O, C>(out + t * os + c, acc);
        }
    }
}

// -------------------------------------------------------- combine_backward --
// dy[row_dst[t, j]] = w[t, j] dout[t] and dw[t, j] = <dout[t], y[row_dst[t, j]]>
// (0 for an empty slot): one block a token, dout[t] read once; the dot products
// are fp32 sums joined by shuffles and then in warp order.
template <typename A, typename O, int C>
__global__ void __launch_bounds__(256) k_combine_backward(const O* __restrict__ dout, long long ds,
                                                          const A* __restrict__ y, long long ys,
                                                          const float* __restrict__ w, int T, int k, int H,
                                                          const int32_t* __restrict__ placed,
                                                          const int32_t* __restrict__ row_dst, A* __restrict__ dy,
                                                          long long dys, float* __restrict__ dw) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float part[8][kMaxTopK];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const long long R = (long long)T * k;
    for (long long t = blockIdx.x; t < T; t += gridDim.x) {
        float dot[kMaxTopK];
#pragma unroll
        for (int j = 0; j < kMaxTopK; ++j) dot[j] = 0.f;
        for (int c = threadIdx.x * C; c < H; c += blockDim.x * C) {
            const Chunk<O, C> d = load_chunk<O, C>(dout + t * ds + c);
#pragma unroll
            for (int j = 0; j < kMaxTopK; ++j) {
                if (j >= k) break;
                const long long p = row_dst[t * k + j];
                if (p < 0 || p >= R) continue;
                const float wt = w[t * k + j];
                const Chunk<A, C> v = load_chunk<A, C>(y + p * ys + c);
                float g[C];
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    const float f = to_f32(d.v[i]);
                    dot[j] += f * to_f32(v.v[i]);
                    g[i] = wt * f;
                }
                store_chunk<A, C>(dy + p * dys + c, g);
            }
        }
#pragma unroll
        for (int j = 0; j < kMaxTopK; ++j) {
            const float s = warp_sum(dot[j]);
            if (lane == 0) part[warp][j] = s;
        }
        __syncthreads();
        if (threadIdx.x < (unsigned)k) {
            float s = 0.f;
            for (int a = 0; a < warps; ++a) s += part[a][threadIdx.x];
            dw[t * k + threadIdx.x] = s;
        }
        __syncthreads();
    }
    float zero[C];
#pragma unroll
    for (int i = 0; i < C; ++i) zero[i] = 0.f;
    for (long long p = max(*placed, 0) + (long long)blockIdx.x; p < R; p += gridDim.x)
        for (int c = threadIdx.x * C; c < H; c += blockDim.x * C) store_chunk<A, C>(dy + p * dys + c, zero);
}

// ---------------------------------------------------------- route_backward --
// w_j = w_scale s_j / S, S = sum of s over the kept slots, s = sqrt(softplus(l)):
//   dl_j = (w_scale / S^2) sum_i s_i (dw_j - dw_i) * sigmoid(l_j) / (2 s_j),
// the differences taken first, so that one kept slot gives exactly 0.  Below
// l = -17, sigmoid(l) / (2 s) is exp(l / 2) / 2 to less than fp32's rounding.
// One warp a token; the row of E gradients is written once, zeros and all.
__global__ void __launch_bounds__(128) k_route_backward(const float* __restrict__ logits,
                                                        const int32_t* __restrict__ ids,
                                                        const float* __restrict__ dw, int T, int E, int k,
                                                        float w_scale, float* __restrict__ dlogits) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr unsigned kAll = 0xFFFFFFFFu;
    const int lane = threadIdx.x & 31;
    const long long step = (long long)gridDim.x * (blockDim.x >> 5);
    for (long long t = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); t < T; t += step) {
        const int id = lane < k ? ids[t * k + lane] : -1;
        const bool kept = id >= 0 && id < E;
        const float l = kept ? logits[t * E + id] : 0.f;
        const float g = kept ? dw[t * k + lane] : 0.f;
        const float s = kept ? sqrt_softplus(l) : 0.f;
        float total = 0.f, against = 0.f;
        for (int i = 0; i < k; ++i) {
            const float si = __shfl_sync(kAll, s, i), gi = __shfl_sync(kAll, g, i);
            if (__shfl_sync(kAll, (int)kept, i)) {
                total += si;
                against += si * (g - gi);
            }
        }
        float d = 0.f;
        if (kept && total > 0.f) {
            const float slope = l < -17.f ? 0.5f * expf(0.5f * l) : 1.f / (1.f + expf(-l)) / (2.f * s);
            d = w_scale / total / total * against * slope;
        }
        int at[kMaxTopK];
        float val[kMaxTopK];
#pragma unroll
        for (int j = 0; j < kMaxTopK; ++j) {
            at[j] = __shfl_sync(kAll, id, j);
            val[j] = __shfl_sync(kAll, d, j);
        }
        float* row = dlogits + t * E;
        for (int e = lane; e < E; e += 32) {
            float v = 0.f;
#pragma unroll
            for (int j = 0; j < kMaxTopK; ++j)
                if (at[j] == e) v += val[j];
            row[e] = v;
        }
    }
}

// ----------------------------------------------------------------- entries --
moe_status fail(moe_status st, const char* fmt, ...) {
    char buf[200];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    set_thread_error(buf);
    return st;
}

moe_status launched(cudaError_t e, const char* what) {
    return e == cudaSuccess ? MOE_OK : fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// The checks that every entry shares; MOE_OK with *empty set for T = 0.
moe_status check_rows(const char* what, int T, int top_k, int hidden) {
    if (top_k < 1 || top_k > kMaxTopK) return fail(MOE_ERR_INVALID_ARG, "%s: top_k must be in [1, 8]", what);
    if (T < 0 || (long long)T * top_k > (1LL << 30))
        return fail(MOE_ERR_INVALID_ARG, "%s: T must be >= 0 and T * top_k at most 2^30", what);
    if (hidden < 1 || hidden > (1 << 24)) return fail(MOE_ERR_INVALID_ARG, "%s: hidden must be in [1, 2^24]", what);
    return MOE_OK;
}

moe_status check_types(const char* what, moe_dtype a, moe_dtype o) {
    if (!dtype_ok(a) || !dtype_ok(o)) return fail(MOE_ERR_INVALID_ARG, "%s: unknown dtype", what);
    if (o != a && o != MOE_F32)
        return fail(MOE_ERR_INVALID_ARG, "%s: the token side must have the sorted side's dtype or MOE_F32", what);
    return MOE_OK;
}

// A side's base and stride in elements of `size` bytes.
moe_status check_side(const char* what, const char* name, const void* p, long long stride, int hidden, int size) {
    if (!p) return fail(MOE_ERR_INVALID_ARG, "%s: %s is NULL", what, name);
    if ((uintptr_t)p % size) return fail(MOE_ERR_INVALID_ARG, "%s: %s is not aligned to its elements", what, name);
    if (stride < hidden) return fail(MOE_ERR_INVALID_ARG, "%s: the stride of %s is below hidden", what, name);
    if (stride > (1LL << 40)) return fail(MOE_ERR_INVALID_ARG, "%s: the stride of %s is above 2^40", what, name);
    return MOE_OK;
}

unsigned blocks_for(long long n) { return (unsigned)(n < (1LL << 30) ? n : (1LL << 30)); }

// Calls f.template operator()<A, O, C>() for the types and the widest C that the
// rows allow: whole 16-byte words of A, else pairs, else single elements.
template <typename A, typename O, typename F>
cudaError_t by_width(unsigned align_a, unsigned align_o, int hidden, F&& f) {
    constexpr int W = 16 / (int)sizeof(A);
    auto fits = [&](int c) {
        const unsigned ob = c * (unsigned)sizeof(O) < 16 ? c * (unsigned)sizeof(O) : 16;
        return hidden % c == 0 && align_a >= c * sizeof(A) && align_o >= ob;
    };
    if (fits(W)) return f.template operator()<A, O, W>();
    if (fits(2)) return f.template operator()<A, O, 2>();
    return f.template operator()<A, O, 1>();
}

template <typename F>
cudaError_t by_type(moe_dtype a, moe_dtype o, unsigned align_a, unsigned align_o, int hidden, F&& f) {
    if (a == MOE_F32) return by_width<float, float>(align_a, align_o, hidden, f);
    if (a == MOE_BF16)
        return o == MOE_F32 ? by_width<__nv_bfloat16, float>(align_a, align_o, hidden, f)
                            : by_width<__nv_bfloat16, __nv_bfloat16>(align_a, align_o, hidden, f);
    return o == MOE_F32 ? by_width<__half, float>(align_a, align_o, hidden, f)
                        : by_width<__half, __half>(align_a, align_o, hidden, f);
}

struct CombineLaunch {
    const void* y; long long ys; const float* w; int T, k, H; const int32_t* row_dst; void* out; long long os;
    cudaStream_t s;
    template <typename A, typename O, int C>
    cudaError_t operator()() const {
        return launch_pdl(k_combine_rows<A, O, C>, dim3(blocks_for(T)), dim3(128), 0, s, (const A*)y, ys, w, T, k, H,
                          row_dst, (O*)out, os);
    }
};

struct CombineBackwardLaunch {
    const void* dout; long long ds; const void* y; long long ys; const float* w; int T, k, H;
    const int32_t *placed, *row_dst; void* dy; long long dys; float* dw; cudaStream_t s;
    template <typename A, typename O, int C>
    cudaError_t operator()() const {
        return launch_pdl(k_combine_backward<A, O, C>, dim3(blocks_for(T)), dim3(256), 0, s, (const O*)dout, ds,
                          (const A*)y, ys, w, T, k, H, placed, row_dst, (A*)dy, dys, dw);
    }
};

template <typename V>
cudaError_t dispatch_words(const void* x, long long xp, int T, int k, int bytes, const int32_t* placed,
                           const int32_t* row_dst, void* xs, long long xsp, cudaStream_t s) {
    return launch_pdl(k_dispatch<V>, dim3(blocks_for(T)), dim3(128), 0, s, (const char*)x, xp, T, k,
                      bytes / (int)sizeof(V), placed, row_dst, (char*)xs, xsp);
}

moe_status combine(const char* what, const void* y, moe_dtype dtype, long long y_stride, const float* w, int T,
                   int top_k, int hidden, const int32_t* row_dst, void* out, moe_dtype out_dtype,
                   long long out_stride, moe_stream_t stream) {
    moe_status st = check_rows(what, T, top_k, hidden);
    if (st == MOE_OK) st = check_types(what, dtype, out_dtype);
    if (st != MOE_OK || T == 0) return st;
    st = check_side(what, "the sorted side", y, y_stride, hidden, dtype_size(dtype));
    if (st == MOE_OK) st = check_side(what, "the token side", out, out_stride, hidden, dtype_size(out_dtype));
    if (st == MOE_OK && !row_dst) st = fail(MOE_ERR_INVALID_ARG, "%s: row_dst is NULL", what);
    if (st != MOE_OK) return st;
    const CombineLaunch f{y, y_stride, w, T, top_k, hidden, row_dst, out, out_stride, (cudaStream_t)stream};
    return launched(by_type(dtype, out_dtype, row_align(y, y_stride * dtype_size(dtype)),
                            row_align(out, out_stride * dtype_size(out_dtype)), hidden, f), what);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_dispatch(const void* x, moe_dtype dtype, long long x_stride, int T, int top_k, int hidden,
                                   const int32_t* offsets, int n_experts, const int32_t* row_dst, void* xs,
                                   long long xs_stride, moe_stream_t stream) {
    const char* what = "moe_dispatch";
    moe_status st = check_rows(what, T, top_k, hidden);
    if (st == MOE_OK) st = check_types(what, dtype, dtype);
    if (st == MOE_OK && (n_experts < 1 || n_experts > kMaxExperts))
        st = fail(MOE_ERR_INVALID_ARG, "%s: n_experts must be in [1, 1024]", what);
    if (st != MOE_OK || T == 0) return st;
    const int size = dtype_size(dtype);
    st = check_side(what, "x", x, x_stride, hidden, size);
    if (st == MOE_OK) st = check_side(what, "xs", xs, xs_stride, hidden, size);
    if (st == MOE_OK && (!offsets || !row_dst)) st = fail(MOE_ERR_INVALID_ARG, "%s: offsets or row_dst is NULL", what);
    if (st != MOE_OK) return st;
    const unsigned ax = row_align(x, x_stride * size), as = row_align(xs, xs_stride * size);
    const unsigned al = ax < as ? ax : as;
    const int bytes = hidden * size;
    const int32_t* placed = offsets + n_experts;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (al >= 16 && bytes % 16 == 0)
        e = dispatch_words<uint4>(x, x_stride * size, T, top_k, bytes, placed, row_dst, xs, xs_stride * size, s);
    else if (al >= 4 && bytes % 4 == 0)
        e = dispatch_words<uint32_t>(x, x_stride * size, T, top_k, bytes, placed, row_dst, xs, xs_stride * size, s);
    else
        e = dispatch_words<uint16_t>(x, x_stride * size, T, top_k, bytes, placed, row_dst, xs, xs_stride * size, s);
    return launched(e, what);
}

extern "C" moe_status moe_dispatch_backward(const void* dxs, moe_dtype dtype, long long dxs_stride, int T, int top_k,
                                            int hidden, const int32_t* row_dst, void* dx, moe_dtype dx_dtype,
                                            long long dx_stride, moe_stream_t stream) {
    return combine("moe_dispatch_backward", dxs, dtype, dxs_stride, nullptr, T, top_k, hidden, row_dst, dx, dx_dtype,
                   dx_stride, stream);
}

extern "C" moe_status moe_combine(const void* y, moe_dtype dtype, long long y_stride, const float* w, int T, int top_k,
                                  int hidden, const int32_t* row_dst, void* out, moe_dtype out_dtype,
                                  long long out_stride, moe_stream_t stream) {
    if (!w && T > 0) return fail(MOE_ERR_INVALID_ARG, "moe_combine: w is NULL");
    return combine("moe_combine", y, dtype, y_stride, w, T, top_k, hidden, row_dst, out, out_dtype, out_stride,
                   stream);
}

extern "C" moe_status moe_combine_backward(const void* dout, moe_dtype dout_dtype, long long dout_stride,
                                           const void* y, moe_dtype dtype, long long y_stride, const float* w, int T,
                                           int top_k, int hidden, const int32_t* offsets, int n_experts,
                                           const int32_t* row_dst, void* dy, long long dy_stride, float* dw,
                                           moe_stream_t stream) {
    const char* what = "moe_combine_backward";
    moe_status st = check_rows(what, T, top_k, hidden);
    if (st == MOE_OK) st = check_types(what, dtype, dout_dtype);
    if (st == MOE_OK && (n_experts < 1 || n_experts > kMaxExperts))
        st = fail(MOE_ERR_INVALID_ARG, "%s: n_experts must be in [1, 1024]", what);
    if (st != MOE_OK || T == 0) return st;
    const int size = dtype_size(dtype), dsize = dtype_size(dout_dtype);
    st = check_side(what, "dout", dout, dout_stride, hidden, dsize);
    if (st == MOE_OK) st = check_side(what, "y", y, y_stride, hidden, size);
    if (st == MOE_OK) st = check_side(what, "dy", dy, dy_stride, hidden, size);
    if (st == MOE_OK && (!w || !dw || !offsets || !row_dst))
        st = fail(MOE_ERR_INVALID_ARG, "%s: w, dw, offsets or row_dst is NULL", what);
    if (st != MOE_OK) return st;
    const unsigned ay = row_align(y, y_stride * size), ad = row_align(dy, dy_stride * size);
    const CombineBackwardLaunch f{dout, dout_stride, y, y_stride, w, T, top_k, hidden, offsets + n_experts, row_dst,
                                  dy, dy_stride, dw, (cudaStream_t)stream};
    return launched(by_type(dtype, dout_dtype, ay < ad ? ay : ad, row_align(dout, dout_stride * dsize), hidden, f),
                    what);
}

extern "C" moe_status moe_route_backward(const float* logits, const int32_t* ids, const float* dw, int T, int n_experts,
                                         int top_k, float w_scale, float* dlogits, moe_stream_t stream) {
    const char* what = "moe_route_backward";
    moe_status st = check_rows(what, T, top_k, 1);
    if (st == MOE_OK && (n_experts < top_k || n_experts > kMaxExperts))
        st = fail(MOE_ERR_INVALID_ARG, "%s: n_experts must be in [top_k, 1024]", what);
    if (st == MOE_OK && !std::isfinite(w_scale)) st = fail(MOE_ERR_INVALID_ARG, "%s: w_scale must be finite", what);
    if (st != MOE_OK || T == 0) return st;
    if (!logits || !ids || !dw || !dlogits) return fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer", what);
    return launched(launch_pdl(k_route_backward, dim3(blocks_for((T + 3LL) / 4)), dim3(128), 0, (cudaStream_t)stream,
                               logits, ids, dw, T, n_experts, top_k, w_scale, dlogits), what);
}
