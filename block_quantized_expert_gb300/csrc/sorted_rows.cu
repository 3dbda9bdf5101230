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
//
// No input is `const __restrict__`: a kernel starts while the one in front of it
// may still be writing that input, and the qualifier would promise data that stays
// as it is for the whole kernel, which allows loads before the wait or by the
// read-only path.  The outputs keep __restrict__, so loads still pass stores.
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "layer.h"
#include "route.cuh"
#include "rows.cuh"

namespace moe {

namespace {

// A token's filled slots: pos[a] and wt[a] for a < m, in ascending position;
// w = nullptr stands for ones.
struct Slots {
    int m;
    int pos[kMaxTopK];
    float wt[kMaxTopK];
};

// Written by one warp: lane j < k ranks its own position among the others.  The
// block synchronises before it reads them.
__device__ __forceinline__ void find_slots(Slots& s, const int32_t* row_dst, const float* w, long long t, int k, int R) {
    constexpr unsigned kAll = 0xFFFFFFFFu;
    const int lane = threadIdx.x & 31;
    const int p = lane < k ? row_dst[t * k + lane] : -1;
    const bool on = p >= 0 && p < R;
    const float wj = on && w ? w[t * k + lane] : 1.f;
    const unsigned filled = __ballot_sync(kAll, on);
    int rank = 0;
#pragma unroll
    for (int i = 0; i < kMaxTopK; ++i) {
        const int q = __shfl_sync(kAll, p, i);
        if (((filled >> i) & 1u) && (q < p || (q == p && i < lane))) ++rank;
    }
    if (on) {
        s.pos[rank] = p;
        s.wt[rank] = wj;
    }
    if (lane == 0) s.m = __popc(filled);
}

// ---------------------------------------------------------------- dispatch --
// xs[row_dst[t, j]] = x[t], in words of V: types do not matter to a copy.
// Block (t, y) moves the words y * 128 + i, + 128 gridDim.y, ... of token t, one
// word a thread.  Reads T H, writes R H elements; at T = 8192, k = 6, H = 4096,
// bf16: 71.7 us, 6.6 TB/s (four words a thread: 73.6).
template <typename V>
__global__ void __launch_bounds__(128) k_dispatch(const char* x, long long x_pitch, int T, int k,
                                                  int words, const int32_t* placed,
                                                  const int32_t* row_dst, char* __restrict__ xs,
                                                  long long xs_pitch) {
    pdl_launch_dependents();
    pdl_wait();
    const int R = T * k, first = blockIdx.y * 128 + threadIdx.x, step = gridDim.y * 128;
    const long long t = blockIdx.x;
    const V* src = reinterpret_cast<const V*>(x + t * x_pitch);
    for (int c = first; c < words; c += step) {
        const V v = src[c];
#pragma unroll
        for (int j = 0; j < kMaxTopK; ++j) {
            if (j >= k) break;
            const int p = row_dst[t * k + j];
            if (p >= 0 && p < R) reinterpret_cast<V*>(xs + (long long)p * xs_pitch)[c] = v;
        }
    }
    // positions past the last placed row
    const V zero = V();
    for (long long p = max(*placed, 0) + t; p < R; p += gridDim.x)
        for (int c = first; c < words; c += step) reinterpret_cast<V*>(xs + p * xs_pitch)[c] = zero;
}

// ----------------------------------------------------------------- combine --
// out[t] = sum_j w[t, j] y[row_dst[t, j]] over the filled slots in ascending
// position, which is ascending expert id, the order of the layer's own
// combine; w = NULL stands for ones (the gradient of dispatch).  Two rows of a
// chunk are on their way at a time; the sum is held in fp32 and rounded once.
// T = 8192, k = 6, H = 4096, bf16: 80 us to fp32 and 71.5 us to bf16, 6.6 to 6.7
// TB/s.  Four rows at a time take 83 and 74 us, all eight 88 and 79 (their
// registers leave fewer blocks on an SM).  With one chunk a thread instead of four
// those 88 and 79 were 115 and 101: a block waits for its token's positions first.
template <typename A, typename O, int C, int U>
__global__ void __launch_bounds__(128) k_combine_rows(const A* y, long long ys,
                                                      const float* w, int T, int k, int H,
                                                      const int32_t* row_dst, O* __restrict__ out,
                                                      long long os) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ Slots s;
    const long long t = blockIdx.x;
    if (threadIdx.x < 32) find_slots(s, row_dst, w, t, k, T * k);
    __syncthreads();
    const int m = s.m;
    O* dst = out + t * os;
    for (int c0 = (blockIdx.y * 128 * U + threadIdx.x) * C; c0 < H; c0 += gridDim.y * 128 * U * C) {
        float acc[U][C];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < C; ++i) acc[u][i] = 0.f;
#pragma unroll
        for (int h = 0; h < kMaxTopK; h += 2) {
            if (h >= m) break;
            Chunk<A, C> v[2][U];
#pragma unroll
            for (int a = 0; a < 2; ++a)
                if (h + a < m) {
                    const A* row = y + s.pos[h + a] * ys + c0;
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (c0 + u * 128 * C < H) v[a][u] = load_chunk<A, C>(row + u * 128 * C);
                }
#pragma unroll
            for (int a = 0; a < 2; ++a)
                if (h + a < m) {
                    const float wt = s.wt[h + a];
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int i = 0; i < C; ++i) acc[u][i] += wt * to_f32(v[a][u].v[i]);
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + u * 128 * C < H) store_chunk<O, C>(dst + c0 + u * 128 * C, acc[u]);
    }
}

// -------------------------------------------------------- combine_backward --
// dy[row_dst[t, j]] = w[t, j] dout[t] and dw[t, j] = <dout[t], y[row_dst[t, j]]>
// (0 for an empty slot).  kGroup warps a slot walk its row of y once, U chunks on
// their way at a time; the slots of a token stand next to each other, so that
// dout[t] comes from L1 but once.  The dot product is a fp32 sum a lane, joined
// by shuffles, then in warp order.  T = 8192, k = 6, H = 4096, bf16: 130 us, with the
// router's gradient 135, 6.5 TB/s (one block a token with the k rows of a chunk in
// flight: 154 to 270).
template <typename A, typename O, int C, int U, int kGroup>
__global__ void __launch_bounds__(kGroup == 8 ? 256 : 128) k_combine_backward(const O* dout, long long ds,
                                                          const A* y, long long ys,
                                                          const float* w, int T, int k, int H,
                                                          const int32_t* placed,
                                                          const int32_t* row_dst, A* __restrict__ dy,
                                                          long long dys, float* __restrict__ dw) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int kWarps = kGroup == 8 ? 8 : 4;  // of a block
    __shared__ float part[kWarps];
    constexpr int kStep = 32 * kGroup * C;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int first = (threadIdx.x % (32 * kGroup)) * C;
    const int R = T * k;
    const long long r = (long long)blockIdx.x * (kWarps / kGroup) + warp / kGroup;  // slot
    const int p = r < R ? row_dst[r] : -1;
    const bool on = p >= 0 && p < R;
    float dot = 0.f;
    if (on) {
        const float wt = w[r];
        const O* drow = dout + (long long)((int)r / k) * ds;
        const A* yrow = y + p * ys;
        A* grow = dy + p * dys;
        for (int c0 = first; c0 < H; c0 += U * kStep) {
            Chunk<O, C> d[U];
            Chunk<A, C> v[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + u * kStep < H) {
                    v[u] = load_chunk<A, C>(yrow + c0 + u * kStep);
                    d[u] = load_chunk<O, C>(drow + c0 + u * kStep);
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + u * kStep < H) {
                    float g[C];
#pragma unroll
                    for (int i = 0; i < C; ++i) {
                        const float f = to_f32(d[u].v[i]);
                        dot += f * to_f32(v[u].v[i]);
                        g[i] = wt * f;
                    }
                    store_chunk<A, C>(grow + c0 + u * kStep, g);
                }
        }
    }
    dot = warp_sum(dot);
    if (kGroup > 1) {
        if (lane == 0) part[warp] = dot;
        __syncthreads();
        dot = 0.f;
        for (int a = 0; a < kGroup; ++a) dot += part[warp / kGroup * kGroup + a];
    }
    if (r < R && threadIdx.x % (32 * kGroup) == 0) dw[r] = dot;
    float zero[C];
#pragma unroll
    for (int i = 0; i < C; ++i) zero[i] = 0.f;
    for (long long q = max(*placed, 0) + r; q < R; q += (long long)gridDim.x * (kWarps / kGroup))
        for (int c = first; c < H; c += kStep) store_chunk<A, C>(dy + q * dys + c, zero);
}

// ---------------------------------------------------------- route_backward --
// w_j = w_scale s_j / S, S = sum of s over the kept slots, s = sqrt(softplus(l)):
//   dl_j = (w_scale / S^2) sum_i s_i (dw_j - dw_i) * sigmoid(l_j) / (2 s_j),
// the differences taken first, so that one kept slot gives exactly 0.  S may be as
// small as 1e-38 and S^2 is then 0 in fp32, so the shares p_i = s_i / S stand for
// s_i and the slope is divided by S once: all factors stay near 1.
//   dl_j = w_scale sum_i p_i (dw_j - dw_i) * sigmoid(l_j) / (2 s_j S)
// Below l = -17, s is exp(l / 2) and sigmoid(l) / (2 s) half of that, to less than
// fp32's rounding (its square, exp(l), is subnormal below -87).  Below -174 exp(l / 2)
// itself is, and s counts as 0.
// One warp a token: the row of zeros, then the k gradients into it.
__global__ void __launch_bounds__(128) k_route_backward(const float* logits,
                                                        const int32_t* ids,
                                                        const float* dw, int T, int E, int k,
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
        const float s = !kept || l < -174.f ? 0.f : l < -17.f ? expf(0.5f * l) : sqrt_softplus(l);
        float total = 0.f, against = 0.f;
        for (int i = 0; i < k; ++i) total += __shfl_sync(kAll, s, i);
        const float p = total != 0.f ? s / total : 0.f;  // (NaN stays NaN)
        const unsigned on = __ballot_sync(kAll, kept);
        for (int i = 0; i < k; ++i) {
            const float pi = __shfl_sync(kAll, p, i), gi = __shfl_sync(kAll, g, i);
            if ((on >> i) & 1u) against += pi * (g - gi);
        }
        float d = 0.f;
        if (kept && s != 0.f) d = w_scale * against * (l < -17.f ? 0.5f * p : 0.5f / ((1.f + expf(-l)) * s * total));
        // an id that stands twice: its first slot writes the sum
        float sum = 0.f;
        bool before = false;
#pragma unroll
        for (int j = 0; j < kMaxTopK; ++j) {
            const bool same = __shfl_sync(kAll, id, j) == id;
            const float v = __shfl_sync(kAll, d, j);
            if (same) sum += v;
            before |= same && j < lane;
        }
        float* row = dlogits + t * E;
        if (E % 4 == 0 && (uintptr_t)dlogits % 16 == 0) {
            for (int e = 4 * lane; e < E; e += 128) *reinterpret_cast<float4*>(row + e) = make_float4(0.f, 0.f, 0.f, 0.f);
        } else {
            for (int e = lane; e < E; e += 32) row[e] = 0.f;
        }
        __syncwarp();  // the zeros stand before the gradients
        if (kept && !before) row[id] = sum;
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

// The checks that every entry shares.
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

// Blocks of 128 threads along one token's `chunks` in the combine: four times U
// chunks a thread where there are tokens enough to fill the GPU, else U (one token
// of 4096 fp32: 8 blocks).
unsigned parts_for(int T, int chunks, int U) {
    const int per = (T >= 1024 ? 512 : 128) * U;
    const int n = (chunks + per - 1) / per;
    return (unsigned)(n < 65535 ? n : 65535);
}

// Calls f.template operator()<A, O, C, U>() for the types and the widest C that
// the rows allow: whole 16-byte words of A, else pairs, else single elements; of
// the narrow ones a thread has U on the way at once.
template <typename A, typename O, typename F>
cudaError_t by_width(unsigned align_a, unsigned align_o, int hidden, F&& f) {
    constexpr int W = 16 / (int)sizeof(A);
    auto fits = [&](int c) {
        const unsigned ob = c * (unsigned)sizeof(O) < 16 ? c * (unsigned)sizeof(O) : 16;
        return hidden % c == 0 && align_a >= c * sizeof(A) && align_o >= ob;
    };
    if (fits(W)) return f.template operator()<A, O, W, 1>();
    if (fits(2)) return f.template operator()<A, O, 2, 2>();
    return f.template operator()<A, O, 1, 4>();
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
    template <typename A, typename O, int C, int U>
    cudaError_t operator()() const {
        return launch_pdl(k_combine_rows<A, O, C, U>, dim3(T, parts_for(T, H / C, U)), dim3(128), 0, s, (const A*)y, ys,
                          w, T, k, H, row_dst, (O*)out, os);
    }
};

struct CombineBackwardLaunch {
    const void* dout; long long ds; const void* y; long long ys; const float* w; int T, k, H;
    const int32_t *placed, *row_dst; void* dy; long long dys; float* dw; cudaStream_t s;
    template <typename A, typename O, int C, int U>
    cudaError_t operator()() const {
        // eight warps a slot where there are slots too few to fill the GPU with fewer (150 SMs
        // of 16 slots); with two warps and one chunk in flight a thread the long batch takes
        // 130 us, with one or four 134 (one slot a block of 64: 130, but 6.7 for 5.1 us at 1024
        // tokens of 1024), with fewer warps on an SM 165 and more
        const long long R = (long long)T * k;
        return R < 2400 ? launch<A, O, C, 2 * U, 8>((unsigned)R) : launch<A, O, C, U, 2>((unsigned)((R + 1) / 2));
    }
    template <typename A, typename O, int C, int U, int kGroup>
    cudaError_t launch(unsigned blocks) const {
        return launch_pdl(k_combine_backward<A, O, C, U, kGroup>, dim3(blocks), dim3(kGroup == 8 ? 256 : 128), 0, s,
                          (const O*)dout, ds, (const A*)y, ys, w, T, k, H, placed, row_dst, (A*)dy, dys, dw);
    }
};

template <typename V>
cudaError_t dispatch_words(const void* x, long long xp, int T, int k, int bytes, const int32_t* placed,
                           const int32_t* row_dst, void* xs, long long xsp, cudaStream_t s) {
    const int words = bytes / (int)sizeof(V), parts = (words + 127) / 128;
    return launch_pdl(k_dispatch<V>, dim3(T, parts < 65535 ? parts : 65535), dim3(128), 0, s, (const char*)x, xp, T, k, words,
                      placed, row_dst, (char*)xs, xsp);
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
    return launched(launch_pdl(k_route_backward, dim3((T + 3) / 4), dim3(128), 0, (cudaStream_t)stream,
                               logits, ids, dw, T, n_experts, top_k, w_scale, dlogits), what);
}
