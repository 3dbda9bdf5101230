// int_product.cu -- rows in 8-bit integers with one scale each
// (moe_quantize_rows) and their product with 8-bit integer experts over the
// sorted segments (moe_expert_product; C entries at the end).
//
//   out[p, n] = scale[r] w_scale[e, n] sum_i q[r, i] wq[e, n, i]
//
// for the positions p of expert e's segment, r the row that position p reads.
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "int_product.cuh"

namespace moe {
namespace {

// ----------------------------------------------------------- quantize_rows --
// v = x, or silu(x[c]) * x[K + c] of a gated row of 2 K (expf and IEEE
// division).  scale = max|v| / 127 and q = rint(127 v / max|v|): dividing the
// exact 127 v (for bf16 and fp16 x) by the maximum, not v by the rounded scale,
// keeps values half way between two codes half way.  A maximum above 2^119 is
// scaled down first (127 v would overflow).  A row with an infinity or a NaN
// gets scale NaN, so that its products are NaN, and codes 0.
template <typename A, int C, bool kGated>
__device__ __forceinline__ void quant_load(const A* row, int K, int c, float (&v)[C]) {
    const Chunk<A, C> a = load_chunk<A, C>(row + c);
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = to_f32(a.v[i]);
    if (kGated) {
        const Chunk<A, C> u = load_chunk<A, C>(row + K + c);
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = __fmul_rn(__fdiv_rn(v[i], 1.f + expf(-v[i])), to_f32(u.v[i]));
    }
}

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

// One block a row.  kKeep chunks of C values a thread stay in registers between
// the maximum and the codes; kKeep = 0: rows of any length, read (and gated)
// twice.  x is not __restrict__: the kernel in front may still write it when this one
// starts (sorted_rows.cu).
template <typename A, int C, bool kGated, int kKeep>
__global__ void __launch_bounds__(256, kGated ? 4 : 6) k_quantize_rows(const A* x, long long xs, int K,
                                                       int8_t* __restrict__ q, long long qs,
                                                       float* __restrict__ scale) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ uint32_t part[8];
    const long long row_at = blockIdx.x;
    const A* row = x + row_at * xs;
    const int first = threadIdx.x * C, step = blockDim.x * C;
    // what stays: the row's own words, or the gated values
    constexpr int kHeld = kKeep ? kKeep : 1;
    Chunk<A, C> raw[kHeld];
    float gated[kGated ? kHeld : 1][C];
    uint32_t top = 0;
    auto take = [&](int n, int c) {
        if (kGated) {
            quant_load<A, C, true>(row, K, c, gated[kGated ? n : 0]);
#pragma unroll
            for (int i = 0; i < C; ++i) top = max(top, __float_as_uint(gated[kGated ? n : 0][i]) & 0x7FFFFFFFu);
        } else {
            raw[n] = load_chunk<A, C>(row + c);
            top = top_bits<A, C>(raw[n], top);
        }
    };
    if (kKeep) {
#pragma unroll
        for (int n = 0; n < kKeep; ++n)
            if (first + n * step < K) take(n, first + n * step);
    } else {
        for (int c = first; c < K; c += step) take(0, c);
    }
    if (!kGated && sizeof(A) == 2) {  // to the bits of that magnitude in fp32
        const uint16_t h = (uint16_t)max(top & 0xFFFFu, top >> 16);
        top = __float_as_uint(to_f32(*reinterpret_cast<const A*>(&h)));
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
    __syncthreads();
    top = part[0];
    for (int a = 1; a < (int)(blockDim.x >> 5); ++a) top = max(top, part[a]);
    const float most = __uint_as_float(top);
    const bool live = most > 0.f && most < INFINITY;
    // 127 v must not overflow, nor may 1 / m
    const float by = most > 0x1p119f ? 0x1p-8f : most < 0x1p-100f ? 0x1p100f : 1.f;
    const float m = most * by, c127 = __fmul_rn(127.f, __frcp_rn(m));
    if (threadIdx.x == 0) scale[row_at] = most < INFINITY ? __fdiv_rn(most, 127.f) : NAN;
    auto put = [&](int n, int c) {
        float v[C];
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = kGated ? gated[kGated ? n : 0][i] : to_f32(raw[n].v[i]);
        Chunk<int8_t, C> out = {};
        if (live) out = quant_codes(v, c127, m, by);
        *reinterpret_cast<Chunk<int8_t, C>*>(q + row_at * qs + c) = out;
    };
    if (kKeep) {
#pragma unroll
        for (int n = 0; n < kKeep; ++n)
            if (first + n * step < K) put(n, first + n * step);
    } else {
        for (int c = first; c < K; c += step) {
            take(0, c);
            put(0, c);
        }
    }
}

// ---------------------------------------------------------------- few rows --
// Single tokens: a warp takes kChan channels of one expert for up to kFew
// positions of its segment, lane l the bytes 16 l, 16 l + 512, ... of K; products
// by __dp4a, exact 32-bit integer sums (sum_to_f32), joined by shuffles.  Bound by the weights,
// each read once for every kFew positions: T = 1 with six of 256 experts, K = N =
// 4096: 19 us, 5.3 TB/s.  Block (x, p): channels 16 x .. of the segment of position p, if p
// is the first of its kFew.
constexpr int kFew = 4, kChan = 4;

// A sum of up to 131072 products of codes in fp32.  They lie in [-2^31 + 2^24, 2^31]:
// the least 32-bit integer is not among them, and stands for 2^31, which only K =
// 131072 with every code -128 reaches.
__device__ __forceinline__ float sum_to_f32(int sum) { return sum == INT_MIN ? 0x1p31f : (float)sum; }

template <typename O>
__global__ void __launch_bounds__(128) k_product_few(const Product a) {
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
    const int rows = min(kFew, sm_end - p);
    const int8_t* q[kFew];
    float s[kFew];
#pragma unroll
    for (int r = 0; r < kFew; ++r) {
        const int src = r < rows ? source_row(a, p + r) : -1;
        q[r] = a.q + (long long)max(src, 0) * a.qs + lane * 16;
        s[r] = src >= 0 ? a.scale[src] : 0.f;
    }
    const int8_t* w[kChan];
#pragma unroll
    for (int c = 0; c < kChan; ++c) w[c] = a.wq + ((long long)e * a.N + min(n0 + c, a.N - 1)) * a.K + lane * 16;
    int acc[kChan][kFew] = {};
    auto add = [&](const uint4 (&v)[kChan], int k) {
#pragma unroll
        for (int r = 0; r < kFew; ++r) {
            if (r >= rows) break;
            const uint4 x = *reinterpret_cast<const uint4*>(q[r] + k);
#pragma unroll
            for (int c = 0; c < kChan; ++c) {
                acc[c][r] = __dp4a((int)x.x, (int)v[c].x, acc[c][r]);
                acc[c][r] = __dp4a((int)x.y, (int)v[c].y, acc[c][r]);
                acc[c][r] = __dp4a((int)x.z, (int)v[c].z, acc[c][r]);
                acc[c][r] = __dp4a((int)x.w, (int)v[c].w, acc[c][r]);
            }
        }
    };
    int k = 0;
    for (; k + 1024 <= a.K; k += 1024) {  // two steps of every channel on their way
        uint4 v[2][kChan];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < kChan; ++c) v[h][c] = __ldcs(reinterpret_cast<const uint4*>(w[c] + k + 512 * h));
        add(v[0], k);
        add(v[1], k + 512);
    }
    for (; k + lane * 16 < a.K; k += 512) {
        uint4 v[kChan];
#pragma unroll
        for (int c = 0; c < kChan; ++c) v[c] = __ldcs(reinterpret_cast<const uint4*>(w[c] + k));
        add(v, k);
    }
    __syncwarp();
#pragma unroll
    for (int c = 0; c < kChan; ++c) {
        if (n0 + c >= a.N) break;
        const float cs = a.w_scale[(long long)e * a.N + n0 + c];
#pragma unroll
        for (int r = 0; r < kFew; ++r) {
            if (r >= rows) break;
            const int sum = __reduce_add_sync(0xFFFFFFFFu, acc[c][r]);
            if (lane == 0)
                reinterpret_cast<O*>(a.out)[(long long)(p + r) * a.os + n0 + c] = from_f32<O>(sum_to_f32(sum) * s[r] * cs);
        }
    }
}

// ---------------------------------------------------------------- any size --
// Any K, stride and alignment: one block a tile of 64 positions of one segment x
// 64 channels, 64 bytes of K at a time through shared memory, 4 x 4 sums a thread
// by __dp4a (exact 32-bit integers): 8192 rows, K = N = 1000, 166 us (bound by the
// issue of loads and sums, 0.1 PFLOP/s).  kWords: K, stride and bases allow four codes a
// load, else they come one by one (777 rows, K = 1101, N = 1001: 78 us for 35 at K = 1100).
template <bool kWords>
__device__ __forceinline__ int codes4(const int8_t* row, int c, int K) {
    if (row == nullptr || c >= K) return 0;
    if (kWords) return *reinterpret_cast<const int*>(row + c);
    uint32_t v = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (c + i < K) v |= (uint32_t)(uint8_t)row[c + i] << (8 * i);
    return (int)v;
}

template <typename O, bool kWords>
__global__ void __launch_bounds__(256) k_product_any(const Product a) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int kTile = 64;
    __shared__ int sm_e, sm_j;
    __shared__ int xs[kTile][17], ws[kTile][17];  // 16 words of four codes a row
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
    // this thread brings word lw of rows lr, lr + 16, ... and sums channels tx + 16 j, positions ty + 16 i
    const int lw = tid & 15, lr = tid >> 4, tx = tid & 15, ty = tid >> 4;
    const int8_t *xrow[4], *wrow[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = lr + 16 * i;
        xrow[i] = src[r] >= 0 ? a.q + src[r] * a.qs : nullptr;
        wrow[i] = n0 + r < a.N ? a.wq + ((long long)e * a.N + n0 + r) * a.K : nullptr;
    }
    int acc[4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += 64) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            xs[lr + 16 * i][lw] = codes4<kWords>(xrow[i], k0 + 4 * lw, a.K);
            ws[lr + 16 * i][lw] = codes4<kWords>(wrow[i], k0 + 4 * lw, a.K);
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            int x[4], w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = xs[ty + 16 * i][c];
                w[i] = ws[tx + 16 * i][c];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(x[i], w[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int p = ty + 16 * i;
        if (p >= count) continue;
        const float s = src[p] >= 0 ? a.scale[src[p]] : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + tx + 16 * j;
            if (n < a.N)
                reinterpret_cast<O*>(a.out)[(long long)(p0 + p) * a.os + n] =
                    from_f32<O>(sum_to_f32(acc[i][j]) * s * a.w_scale[(long long)e * a.N + n]);
        }
    }
}

// Positions past the last segment are written as zeros.
template <typename O>
__global__ void __launch_bounds__(256) k_product_tail(const Product a) {
    pdl_launch_dependents();
    pdl_wait();
    for (long long p = segment_at(a, a.E) + (long long)blockIdx.x; p < a.R; p += gridDim.x)
        for (int n = threadIdx.x; n < a.N; n += blockDim.x) reinterpret_cast<O*>(a.out)[p * a.os + n] = from_f32<O>(0.f);
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

template <typename A, int C, int kKeep>
cudaError_t quantize_c(bool gated, const void* x, long long xs, long long rows, int K, int8_t* q, long long qs,
                       float* scale, cudaStream_t s) {
    const int each = kKeep ? kKeep : 1, chunks = (K + C * each - 1) / (C * each);
    const int threads = chunks >= 256 ? 256 : (chunks + 31) / 32 * 32;
    auto* f = gated ? k_quantize_rows<A, C, true, kKeep> : k_quantize_rows<A, C, false, kKeep>;
    return launch_pdl(f, dim3((unsigned)rows), dim3(threads), 0, s, (const A*)x, xs, K, q, qs, scale);
}

// The widest chunk that the rows allow.  Many rows: four chunks a thread and so
// more rows on an SM at once; few rows: more threads for each.
template <typename A>
cudaError_t quantize_a(bool gated, const void* x, long long xs, long long rows, int K, int8_t* q, long long qs,
                       float* scale, cudaStream_t s) {
    constexpr int W = 16 / (int)sizeof(A);
    const unsigned ax = row_align(x, xs * (long long)sizeof(A)), aq = row_align(q, qs);
    if (K % W == 0 && ax >= 16 && aq >= (unsigned)W) {
        if (rows >= 1024 && K <= 1024 * W) return quantize_c<A, W, 4>(gated, x, xs, rows, K, q, qs, scale, s);
        if (K <= 256 * W) return quantize_c<A, W, 1>(gated, x, xs, rows, K, q, qs, scale, s);
        if (K <= 512 * W) return quantize_c<A, W, 2>(gated, x, xs, rows, K, q, qs, scale, s);
        if (K <= 1024 * W) return quantize_c<A, W, 4>(gated, x, xs, rows, K, q, qs, scale, s);
        return quantize_c<A, W, 0>(gated, x, xs, rows, K, q, qs, scale, s);
    }
    if (K % 2 == 0 && ax >= 2 * sizeof(A) && aq >= 2 && K <= 8192)
        return quantize_c<A, 2, 16>(gated, x, xs, rows, K, q, qs, scale, s);
    return quantize_c<A, 1, 0>(gated, x, xs, rows, K, q, qs, scale, s);
}

// Whether the CUDA cores stream the weights for every kFew positions.  At K = N =
// 4096 they take 6.5 us for one position and 11 for 8 of one expert where the
// tensor-core form takes 19; 16 positions of one expert 20 for 19.5, of four 22 for
// 21, but of 16 experts 47 for 65.
bool few_rows(const Product& a) { return a.R <= 8 || (a.R <= 16 && a.R <= a.E); }

std::atomic<bool> g_stall_next{false};  // moe_test_stall_next_product

template <typename O>
cudaError_t product_o(const Product& a, cudaStream_t s) {
    if (product_tc_fits(a))
        return launch_pdl(k_product_few<O>, dim3((a.N + 4 * kChan - 1) / (4 * kChan), a.R), dim3(128), 0, s, a);
    // at most one partly filled tile an expert
    const long long tiles = (long long)a.R / 64 + (a.E < a.R ? a.E : a.R);
    if (tiles > 65535) return cudaErrorInvalidConfiguration;
    const bool words = a.K % 4 == 0 && a.qs % 4 == 0 && (uintptr_t)a.q % 4 == 0 && (uintptr_t)a.wq % 4 == 0;
    auto* f = words ? k_product_any<O, true> : k_product_any<O, false>;
    cudaError_t e = launch_pdl(f, dim3((a.N + 63) / 64, (unsigned)tiles), dim3(256), 0, s, a);
    if (e == cudaSuccess && a.offsets) e = launch_pdl(k_product_tail<O>, dim3(a.R < 152 ? a.R : 152), dim3(256), 0, s, a);
    return e;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_quantize_rows(const void* x, moe_dtype dtype, long long x_stride, int gated, int rows, int K,
                                        int8_t* q, long long q_stride, float* scale, moe_stream_t stream) {
    const char* what = "moe_quantize_rows";
    if (!dtype_ok(dtype)) return fail(MOE_ERR_INVALID_ARG, "%s: unknown dtype", what);
    if (rows < 0 || rows > (1 << 30)) return fail(MOE_ERR_INVALID_ARG, "%s: rows must be in [0, 2^30]", what);
    if (K < 1 || K > 131072) return fail(MOE_ERR_INVALID_ARG, "%s: K must be in [1, 131072]", what);
    if (x_stride < (gated ? 2LL : 1LL) * K || q_stride < K || x_stride > (1LL << 40) || q_stride > (1LL << 40))
        return fail(MOE_ERR_INVALID_ARG, "%s: a row stride is below the row or above 2^40", what);
    if (rows == 0) return MOE_OK;
    if (!x || !q || !scale) return fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer", what);
    if ((uintptr_t)x % dtype_size(dtype)) return fail(MOE_ERR_INVALID_ARG, "%s: x is not aligned to its elements", what);
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (dtype == MOE_F32) e = quantize_a<float>(gated != 0, x, x_stride, rows, K, q, q_stride, scale, s);
    else if (dtype == MOE_BF16) e = quantize_a<__nv_bfloat16>(gated != 0, x, x_stride, rows, K, q, q_stride, scale, s);
    else e = quantize_a<__half>(gated != 0, x, x_stride, rows, K, q, q_stride, scale, s);
    return launched(e, what);
}

extern "C" moe_status moe_expert_product(const int8_t* q, long long q_stride, int q_rows, const float* scale, int K,
                                         const int8_t* wq, const float* w_scale, int n_experts, int N,
                                         const int32_t* offsets, const int32_t* row_src, int top_k, int R, void* out,
                                         moe_dtype out_dtype, long long out_stride, moe_stream_t stream) {
    const char* what = "moe_expert_product";
    if (!dtype_ok(out_dtype)) return fail(MOE_ERR_INVALID_ARG, "%s: unknown dtype", what);
    if (K < 1 || K > 131072) return fail(MOE_ERR_INVALID_ARG, "%s: K must be in [1, 131072]", what);
    if (N < 1 || N > (1 << 20)) return fail(MOE_ERR_INVALID_ARG, "%s: N must be in [1, 2^20]", what);
    if (n_experts < 1 || n_experts > kMaxExperts)
        return fail(MOE_ERR_INVALID_ARG, "%s: n_experts must be in [1, 1024]", what);
    if (R < 0 || R > (1 << 20) || q_rows < 0) return fail(MOE_ERR_INVALID_ARG, "%s: R must be in [0, 2^20]", what);
    if (!row_src && q_rows < R) return fail(MOE_ERR_INVALID_ARG, "%s: q has fewer rows than out", what);
    if (row_src && (top_k < 1 || top_k > kMaxTopK))
        return fail(MOE_ERR_INVALID_ARG, "%s: top_k must be in [1, 8]", what);
    if (!offsets && n_experts != 1) return fail(MOE_ERR_INVALID_ARG, "%s: several experts need offsets", what);
    if (q_stride < K || out_stride < N || q_stride > (1LL << 40) || out_stride > (1LL << 40))
        return fail(MOE_ERR_INVALID_ARG, "%s: a row stride is below the row or above 2^40", what);
    if (R == 0) return MOE_OK;
    if (!q || !scale || !wq || !w_scale || !out) return fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer", what);
    if ((uintptr_t)out % dtype_size(out_dtype))
        return fail(MOE_ERR_INVALID_ARG, "%s: out is not aligned to its elements", what);
    Product a{q, q_stride, q_rows, scale, K, wq, w_scale, n_experts, N, offsets, row_src, top_k, R, out,
              out_stride, 2000000000ull, 0};
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (product_tc_fits(a) && !few_rows(a)) {
        if (g_stall_next.exchange(false)) {
            a.stall = 1;
            a.wait_ns = 5000000ull;
        }
        e = launch_product_tc(a, out_dtype, s);
    }
    else if (out_dtype == MOE_F32) e = product_o<float>(a, s);
    else if (out_dtype == MOE_BF16) e = product_o<__nv_bfloat16>(a, s);
    else e = product_o<__half>(a, s);
    return launched(e, what);
}

extern "C" moe_status moe_check_product(moe_stream_t stream) {
    const char* what = "moe_check_product";
    uint32_t flag = 0;
    const cudaError_t e = product_flag(&flag, (cudaStream_t)stream);
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    if (flag) return fail(MOE_ERR_TIMEOUT, "%s: a device-side wait of moe_expert_product ran out", what);
    return MOE_OK;
}

extern "C" moe_status moe_test_stall_next_product(void) {
    g_stall_next = true;
    return MOE_OK;
}
