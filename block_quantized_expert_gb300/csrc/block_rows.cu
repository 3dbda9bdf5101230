// block_rows.cu -- rows to blocks of 4-bit codes and back (moe_quantize_blocks,
// moe_dequantize_blocks; C entries at the end).
//
// A block's elements are e2m1 codes times one scale, two codes a byte, the even
// element in the low half:
//   MXFP4  32 elements, 2^(floor(log2 amax) - 2) as a UE8M0 byte
//   NVFP4  16 elements, s = e4m3 of amax / 6 / g as a byte; element = code s g
// g is one scale a row: given, or the least power of two from amax(row) / 2688
// up.  2688 = 6 * 448, so no s passes 448; and with a power of two s g has four
// bits, so that the quotients amax / 6 / g and v / (s g), which fp32 rounds once,
// fall on a value half way between two codes exactly where the real ones do.
// With amax / 2688 itself one value in 500 of 16-bit rows is within 2^-24 of half way.
#include <cmath>
#include <type_traits>

#include "block_rows.cuh"
#include "entry.h"
#include "rows.cuh"

namespace moe {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kUnit = 16;  // elements of one thread's turn: an NVFP4 block, half an MXFP4 one

template <typename A>
struct Quantize {
    const A* x;
    long long xs;
    int rows, K;
    uint8_t* q;
    long long qs;
    uint8_t* s;     // [rows][K / 32] or [rows][K / 16]
    float* scale;   // NVFP4: g of every row
    bool given;     // scale is read
};

// 16 elements; kWide: 16-byte words.
template <typename A, bool kWide>
__device__ __forceinline__ void load_unit(const A* p, float (&v)[kUnit]) {
    if (kWide) {
        constexpr int W = 16 / (int)sizeof(A);
#pragma unroll
        for (int n = 0; n < kUnit; n += W) {
            const Chunk<A, W> c = load_chunk<A, W>(p + n);
#pragma unroll
            for (int i = 0; i < W; ++i) v[n + i] = to_f32(c.v[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kUnit; ++i) v[i] = to_f32(p[i]);
    }
}

// silu(x[c]) * x[K + c] of a gated row, each operation rounded by itself.
template <typename A, bool kGated, bool kWide>
__device__ __forceinline__ void take_unit(const A* row, int K, int c, float (&v)[kUnit]) {
    load_unit<A, kWide>(row + c, v);
    if (kGated) {
        float u[kUnit];
        load_unit<A, kWide>(row + K + c, u);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) v[i] = __fmul_rn(__fdiv_rn(v[i], 1.f + expf(-v[i])), u[i]);
    }
}

__device__ __forceinline__ uint32_t unit_top(const float (&v)[kUnit]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kUnit; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return top;
}

// 16 quotients to codes.
__device__ __forceinline__ uint2 pack_unit(const float (&y)[kUnit]) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        asm("{\n.reg .b8 a, b, c, d;\n"
            "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\ncvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
            "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\ncvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
            "mov.b32 %0, {a, b, c, d};\n}"
            : "=r"(w[h])
            : "f"(y[8 * h]), "f"(y[8 * h + 1]), "f"(y[8 * h + 2]), "f"(y[8 * h + 3]), "f"(y[8 * h + 4]), "f"(y[8 * h + 5]),
              "f"(y[8 * h + 6]), "f"(y[8 * h + 7]));
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void store_codes(uint8_t* p, uint2 w) {
    if ((uintptr_t)p % 8 == 0) {
        *reinterpret_cast<uint2*>(p) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p[i] = (uint8_t)(w.x >> (8 * i));
            p[4 + i] = (uint8_t)(w.y >> (8 * i));
        }
    }
}

// The block's scale byte and the codes of this thread's 16 elements.  A block with an infinity
// or a NaN gets the byte of NaN and codes 0.
template <bool kNv>
__device__ __forceinline__ uint2 unit_codes(const float (&v)[kUnit], uint32_t top, float g, uint8_t& byte) {
    const float amax = __uint_as_float(top);
    float y[kUnit];
    if (kNv) {
        if (!(amax < INFINITY)) {
            byte = 0x7F;
            return make_uint2(0, 0);
        }
        const float t = __fdiv_rn(__fdiv_rn(amax, 6.f), g);
        byte = t > 0.f ? (uint8_t)__nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3) : 0;
        const float d = __fmul_rn(e4m3_to_f32(byte), g);
        if (!(d > 0.f)) return make_uint2(0, 0);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) y[i] = __fdiv_rn(v[i], d);
    } else {
        if (!(amax < INFINITY)) {
            byte = 0xFF;
            return make_uint2(0, 0);
        }
        const int e = (int)(top >> 23) - 129;  // floor(log2 amax) - 2; amax of 0 or below 2^-126: -129
        const int x = e < -127 ? -127 : e;
        byte = (uint8_t)(x + 127);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) y[i] = scale_pow2(v[i], x);
    }
    return pack_unit(y);
}

// The least power of two from amax / 2688 = amax / (1.3125 * 2^11) up, at least 2^-126.
__device__ __forceinline__ float row_power(uint32_t top) {
    const int e = (int)(top >> 23) - 127 - 11 + ((top & 0x7FFFFFu) > 0x280000u);
    return __uint_as_float((uint32_t)(max(e, -126) + 127) << 23);
}

// kRow threads a row, `blockDim.x / kRow` rows a block (kRow = 0: the block).  NVFP4
// with scales of its own needs the row's maximum first: up to kKeep units a thread
// stay in registers, kKeep = 0 reads the row twice.
template <typename A, bool kNv, bool kGated, bool kWide, int kKeep>
__global__ void __launch_bounds__(256) k_quantize_blocks(const Quantize<A> a) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ uint32_t part[8];
    const long long t = blockIdx.x;
    const A* row = a.x + t * a.xs;
    const int units = a.K / kUnit, blocks = a.K / (kNv ? 16 : 32);
    constexpr int kHeld = kKeep ? kKeep : 1;
    float v[kHeld][kUnit];
    uint32_t tops[kHeld];
    float g = 1.f;
    const int first = threadIdx.x, step = blockDim.x;
    if (kNv && !a.given) {
        uint32_t top = 0;
        if (kKeep) {
#pragma unroll
            for (int n = 0; n < kHeld; ++n)
                if (first + n * step < units) {
                    take_unit<A, kGated, kWide>(row, a.K, (first + n * step) * kUnit, v[n]);
                    tops[n] = unit_top(v[n]);
                    top = max(top, tops[n]);
                }
        } else {
            for (int u = first; u < units; u += step) {
                take_unit<A, kGated, kWide>(row, a.K, u * kUnit, v[0]);
                top = max(top, unit_top(v[0]));
            }
        }
        top = __reduce_max_sync(kAll, top);
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
        __syncthreads();
        top = part[0];
        for (int i = 1; i < (int)(blockDim.x >> 5); ++i) top = max(top, part[i]);
        const bool fine = top < 0x7F800000u;
        g = top == 0 ? 0.f : fine ? row_power(top) : NAN;
        if (threadIdx.x == 0) a.scale[t] = g;
    } else if (kNv) {
        g = a.scale[t];
    }
    const bool held = kKeep && kNv && !a.given;
    auto put = [&](const float (&f)[kUnit], uint32_t top, int u) {
        if (!kNv) top = max(top, __shfl_xor_sync(kAll, top, 1));
        if (u >= units) return;
        uint8_t byte;
        const uint2 w = unit_codes<kNv>(f, top, g, byte);
        store_codes(a.q + t * a.qs + u * 8, w);
        if (kNv) a.s[t * blocks + u] = byte;
        else if (u % 2 == 0) a.s[t * blocks + u / 2] = byte;
    };
    if (held) {
#pragma unroll
        for (int n = 0; n < kHeld; ++n) put(v[n], tops[n], first + n * step);
    } else {
        for (int u0 = 0; u0 < units; u0 += step) {  // (whole warps, for the exchange between halves)
            const int u = u0 + first;
            uint32_t top = 0;
            if (u < units) {
                take_unit<A, kGated, kWide>(row, a.K, u * kUnit, v[0]);
                top = unit_top(v[0]);
            }
            put(v[0], top, u);
        }
    }
}

// ------------------------------------------------------------------- back --
template <typename O>
struct Dequantize {
    const uint8_t* q;
    long long qs;
    const uint8_t* s;
    const float* scale;  // NULL: ones
    long long rows;
    int K;
    O* x;
    long long xs;
};

// (code s) g, one rounding in fp32 and one to the rows' type.
template <typename O, bool kNv, bool kWide>
__global__ void __launch_bounds__(256) k_dequantize_blocks(const Dequantize<O> a) {
    pdl_launch_dependents();
    pdl_wait();
    const int units = a.K / kUnit;
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < a.rows * units; i += gridDim.x * 256LL) {
        const long long t = i / units;
        const int u = (int)(i - t * units);
        const uint8_t* p = a.q + t * a.qs + u * 8;
        uint32_t w[2] = {0, 0};
        if ((uintptr_t)p % 8 == 0) {
            const uint2 both = *reinterpret_cast<const uint2*>(p);
            w[0] = both.x;
            w[1] = both.y;
        } else {
            for (int b = 0; b < 8; ++b) w[b >> 2] |= (uint32_t)p[b] << (8 * (b & 3));
        }
        const float s = kNv ? e4m3_to_f32(a.s[t * units + u]) : ue8m0_value(a.s[t * (units / 2) + u / 2]);
        const float g = a.scale ? a.scale[t] : 1.f;
        constexpr int W = kWide ? 16 / (int)sizeof(O) : 1;
        O* to = a.x + t * a.xs + u * kUnit;
#pragma unroll
        for (int c = 0; c < kUnit; c += W) {
            float f[W];
#pragma unroll
            for (int j = 0; j < W; ++j) f[j] = e2m1_to_f32(w[(c + j) >> 3] >> (4 * ((c + j) & 7)) & 15u) * s * g;
            store_chunk<O, W>(to + c, f);
        }
    }
}

// ----------------------------------------------------------------- launches --
template <typename A, bool kNv, bool kGated, bool kWide>
cudaError_t quantize_w(const Quantize<A>& a, cudaStream_t s) {
    const int units = a.K / kUnit;
    const bool two = kNv && !a.given;  // passes
    const int each = two && units > 256 ? (units <= 512 ? 2 : 4) : 1;
    const int per = (units + each - 1) / each, threads = per >= 256 ? 256 : (per + 31) / 32 * 32;
    auto* f = !two || units <= 256 ? k_quantize_blocks<A, kNv, kGated, kWide, 1>
              : units <= 512       ? k_quantize_blocks<A, kNv, kGated, kWide, 2>
              : units <= 1024      ? k_quantize_blocks<A, kNv, kGated, kWide, 4>
                                   : k_quantize_blocks<A, kNv, kGated, kWide, 0>;
    return launch_pdl(f, dim3(a.rows), dim3(threads), 0, s, a);
}

template <typename A>
cudaError_t quantize_a(const Quantize<A>& a, bool nv, bool gated, cudaStream_t s) {
    const bool wide = row_align(a.x, a.xs * (long long)sizeof(A)) >= 16 && (!gated || a.K * sizeof(A) % 16 == 0);
    auto run = [&](auto n, auto g) {
        return wide ? quantize_w<A, decltype(n)::value, decltype(g)::value, true>(a, s)
                    : quantize_w<A, decltype(n)::value, decltype(g)::value, false>(a, s);
    };
    if (nv) return gated ? run(std::true_type(), std::true_type()) : run(std::true_type(), std::false_type());
    return gated ? run(std::false_type(), std::true_type()) : run(std::false_type(), std::false_type());
}

template <typename O>
cudaError_t dequantize_o(const Dequantize<O>& a, bool nv, cudaStream_t s) {
    const bool wide = row_align(a.x, a.xs * (long long)sizeof(O)) >= 16;
    const long long blocks = (a.rows * (a.K / kUnit) + 255) / 256;
    const dim3 grid((unsigned)(blocks < 152 * 32 ? blocks : 152 * 32));
    auto* f = nv ? (wide ? k_dequantize_blocks<O, true, true> : k_dequantize_blocks<O, true, false>)
                 : (wide ? k_dequantize_blocks<O, false, true> : k_dequantize_blocks<O, false, false>);
    return launch_pdl(f, grid, dim3(256), 0, s, a);
}

moe_status check_blocks(const char* what, moe_dtype dtype, int rows, int K, int format) {
    if (!dtype_ok(dtype)) return refuse(MOE_ERR_INVALID_ARG, "%s: unknown dtype", what);
    if (format != MOE_WEIGHTS_MXFP4 && format != MOE_WEIGHTS_NVFP4)
        return refuse(MOE_ERR_INVALID_ARG, "%s: unknown format", what);
    if (rows < 0 || rows > (1 << 30)) return refuse(MOE_ERR_INVALID_ARG, "%s: rows must be in [0, 2^30]", what);
    if (K < 32 || K > 131072 || K % 32 != 0)
        return refuse(MOE_ERR_INVALID_ARG, "%s: K must be a multiple of 32 in [32, 131072]", what);
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_quantize_blocks(const void* x, moe_dtype dtype, long long x_stride, int gated, int rows, int K,
                                          int format, uint8_t* q, long long q_stride, uint8_t* s, float* scale,
                                          int scale_given, moe_stream_t stream) {
    const char* what = "moe_quantize_blocks";
    moe_status st = check_blocks(what, dtype, rows, K, format);
    if (st != MOE_OK) return st;
    if (x_stride < (gated ? 2LL : 1LL) * K || q_stride < K / 2 || x_stride > kMostStride || q_stride > kMostStride)
        return refuse(MOE_ERR_INVALID_ARG, "%s: a row stride is below the row or above 2^40", what);
    if (rows == 0) return MOE_OK;
    const bool nv = format == MOE_WEIGHTS_NVFP4;
    if (!x || !q || !s || (nv && !scale)) return refuse(MOE_ERR_INVALID_ARG, "%s: NULL pointer", what);
    if (!nv && scale) return refuse(MOE_ERR_INVALID_ARG, "%s: MXFP4 rows have no scale", what);
    if ((uintptr_t)x % dtype_size(dtype)) return refuse(MOE_ERR_INVALID_ARG, "%s: x is not aligned to its elements", what);
    cudaStream_t str = (cudaStream_t)stream;
    auto run = [&](auto type) {
        using A = decltype(type);
        return quantize_a<A>({(const A*)x, x_stride, rows, K, q, q_stride, s, scale, scale_given != 0}, nv, gated != 0, str);
    };
    cudaError_t e;
    if (dtype == MOE_F32) e = run(float());
    else if (dtype == MOE_BF16) e = run(__nv_bfloat16());
    else e = run(__half());
    return status_of(e, what);
}

extern "C" moe_status moe_dequantize_blocks(const uint8_t* q, long long q_stride, const uint8_t* s, const float* scale,
                                            int rows, int K, int format, void* x, moe_dtype dtype, long long x_stride,
                                            moe_stream_t stream) {
    const char* what = "moe_dequantize_blocks";
    moe_status st = check_blocks(what, dtype, rows, K, format);
    if (st != MOE_OK) return st;
    if (x_stride < K || q_stride < K / 2 || x_stride > kMostStride || q_stride > kMostStride)
        return refuse(MOE_ERR_INVALID_ARG, "%s: a row stride is below the row or above 2^40", what);
    if (rows == 0) return MOE_OK;
    if (!x || !q || !s) return refuse(MOE_ERR_INVALID_ARG, "%s: NULL pointer", what);
    if ((uintptr_t)x % dtype_size(dtype)) return refuse(MOE_ERR_INVALID_ARG, "%s: x is not aligned to its elements", what);
    cudaStream_t str = (cudaStream_t)stream;
    const bool nv = format == MOE_WEIGHTS_NVFP4;
    auto run = [&](auto type) {
        using O = decltype(type);
        return dequantize_o<O>({q, q_stride, s, scale, rows, K, (O*)x, x_stride}, nv, str);
    };
    cudaError_t e;
    if (dtype == MOE_F32) e = run(float());
    else if (dtype == MOE_BF16) e = run(__nv_bfloat16());
    else e = run(__half());
    return status_of(e, what);
}
