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
//
// 65536 x 4096 bf16 to codes: 122 us in NVFP4 (5.6 TB/s), 96 in MXFP4 (7.0); back 101 and 98
// (6.8; MXFP4 with a row scale 102).  Gated, 49152 x 2048: 127 and 104 (4.0 TB/s), bound by the
// issue of the gate's and the codes' arithmetic (75 and 79 % of all slots), as NVFP4 is in part
// (65 %).  With given scales 188: a division for each element.
#include <cmath>
#include <type_traits>

#include "block_rows.cuh"
#include "entry.h"
#include "row_codes.cuh"

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
__device__ __forceinline__ void load_unit(const A* p, Chunk<A, kUnit>& c) {
    if (kWide) {
        constexpr int W = 16 / (int)sizeof(A);
#pragma unroll
        for (int n = 0; n < kUnit; n += W) *reinterpret_cast<Chunk<A, W>*>(&c.v[n]) = load_chunk<A, W>(p + n);
    } else {
#pragma unroll
        for (int i = 0; i < kUnit; ++i) c.v[i] = p[i];
    }
}

// 1 / v within one unit: a quotient x r corrected by its exact remainder, q - (q v - x) r
// (Markstein's correction), is then off by 2^-46 before it is rounded.  In this order of signs
// it keeps that of a zero.
__device__ __forceinline__ float reciprocal(float v) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// 16 values of a row: its own, held in its type until they are used, or silu(x[c]) *
// x[K + c].
template <typename A, bool kGated>
struct Unit {
    Chunk<A, kUnit> raw;
    __device__ __forceinline__ void values(float (&f)[kUnit]) const { unpack_chunk(raw, f); }
    template <bool kWide>
    __device__ __forceinline__ uint32_t take(const A* row, int, int c) {
        load_unit<A, kWide>(row + c, raw);
        const uint32_t top = top_bits<A, kUnit>(raw, 0);
        if (sizeof(A) == 4) return top;
        const uint16_t h = (uint16_t)max(top & 0xFFFFu, top >> 16);
        return __float_as_uint(to_f32(*reinterpret_cast<const A*>(&h)));
    }
};

template <typename A>
struct Unit<A, true> {
    float v[kUnit];
    __device__ __forceinline__ void values(float (&f)[kUnit]) const {
#pragma unroll
        for (int i = 0; i < kUnit; ++i) f[i] = v[i];
    }
    template <bool kWide>
    __device__ __forceinline__ uint32_t take(const A* row, int K, int c) {
        Chunk<A, kUnit> g, u;
        load_unit<A, kWide>(row + c, g);
        load_unit<A, kWide>(row + K + c, u);
        float gate[kUnit];
        unpack_chunk(g, gate);
        unpack_chunk(u, v);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
            const float x = gate[i], d = 1.f + expf(-x), r = reciprocal(d), q = __fmul_rn(x, r);
            // (past 2^120 a remainder could be 0 * infinity)
            const float y = d < 0x1p120f ? __fmaf_rn(-r, __fmaf_rn(q, d, -x), q) : __fdiv_rn(x, d);
            v[i] = __fmul_rn(y, v[i]);
            top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        }
        return top;
    }
};

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

// What the blocks of a row share: g, and where g is a power of two well inside fp32's
// range (and the row's maximum with it), its reciprocal, else 0.
struct RowPower {
    float g, by;
};

// The block's scale byte and the codes of this thread's 16 elements.  A block with an infinity
// or a NaN gets the byte of NaN and codes 0.
//
// With a power of two for g the quotients amax / 6 and v / (s g) are products with a
// reciprocal, corrected by their exact remainders: off by 2^-46 before they are rounded, which
// changes no code, for a value half way between two has an exact quotient, and one that is not
// is 2^-24 of it away at least.  Given scales, and rows at the ends of the range, are divided.
template <bool kNv, typename U>
__device__ __forceinline__ uint2 unit_codes(const U& v, uint32_t top, RowPower p, uint8_t& byte) {
    float y[kUnit];
    v.values(y);
    if (!(__uint_as_float(top) < INFINITY)) {
        byte = kNv ? 0x7F : 0xFF;
        return make_uint2(0, 0);
    }
    if (kNv) {
        const float amax = __uint_as_float(top);
        if (p.by != 0.f) {
            constexpr float kSixth = 1.f / 6.f;
            const float q6 = __fmul_rn(amax, kSixth), t = __fmaf_rn(__fmaf_rn(-6.f, q6, amax), kSixth, q6) * p.by;
            byte = (uint8_t)__nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
            const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(byte, __NV_E4M3)));
            if (s == 0.f) return make_uint2(0, 0);
            const float d = s * p.g, r = reciprocal(s) * p.by;
#pragma unroll
            for (int i = 0; i < kUnit; ++i) {
                const float x = y[i], q = __fmul_rn(x, r);
                y[i] = __fmaf_rn(-r, __fmaf_rn(q, d, -x), q);
            }
        } else {
            const float t = __fdiv_rn(__fdiv_rn(amax, 6.f), p.g);
            byte = t > 0.f ? (uint8_t)__nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3) : 0;
            const float d = __fmul_rn(e4m3_to_f32(byte), p.g);
            if (!(d > 0.f)) return make_uint2(0, 0);
#pragma unroll
            for (int i = 0; i < kUnit; ++i) y[i] = __fdiv_rn(y[i], d);
        }
    } else {
        const int e = (int)(top >> 23) - 129;  // floor(log2 amax) - 2; amax of 0 or below 2^-126: -129
        const int x = e < -127 ? -127 : e;
        byte = (uint8_t)(x + 127);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) y[i] = scale_pow2(y[i], x);
    }
    return pack_unit(y);
}

// The least power of two from amax / 2688 = amax / (1.3125 * 2^11) up, at least 2^-126.
__device__ __forceinline__ float row_power(uint32_t top) {
    const int e = (int)(top >> 23) - 127 - 11 + ((top & 0x7FFFFFu) > 0x280000u);
    return __uint_as_float((uint32_t)(max(e, -126) + 127) << 23);
}

// A block a row, or with kWarp (short rows) a warp a row.  NVFP4 with scales of its own
// needs the row's maximum first: up to kKeep units a thread stay in registers, kKeep = 0
// reads the row twice.
template <typename A, bool kNv, bool kGated, bool kWide, bool kWarp, int kKeep>
__global__ void __launch_bounds__(256) k_quantize_blocks(const Quantize<A> a) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ uint32_t part[8];
    const long long t = kWarp ? blockIdx.x * 8LL + (threadIdx.x >> 5) : blockIdx.x;
    if (t >= a.rows) return;
    const A* row = a.x + t * a.xs;
    const int units = a.K / kUnit, blocks = a.K / (kNv ? 16 : 32);
    constexpr int kHeld = kKeep ? kKeep : 1;
    Unit<A, kGated> v[kHeld];
    uint32_t tops[kHeld];
    RowPower g = {1.f, 0.f};
    const int first = kWarp ? threadIdx.x & 31 : threadIdx.x, step = kWarp ? 32 : blockDim.x;
    const bool own = kNv && !a.given;
    if (own) {
        uint32_t top = 0;
        if (kKeep) {
#pragma unroll
            for (int n = 0; n < kHeld; ++n)
                if (first + n * step < units) {
                    tops[n] = v[n].template take<kWide>(row, a.K, (first + n * step) * kUnit);
                    top = max(top, tops[n]);
                }
        } else {
            for (int u = first; u < units; u += step) top = max(top, v[0].template take<kWide>(row, a.K, u * kUnit));
        }
        top = __reduce_max_sync(kAll, top);
        if (!kWarp) {
            if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
            __syncthreads();
            const int lane = threadIdx.x & 31;
            top = __reduce_max_sync(kAll, lane < (int)(blockDim.x >> 5) ? part[lane] : 0u);
        }
        g.g = top == 0 ? 0.f : top < 0x7F800000u ? row_power(top) : NAN;
        // (2^-70 to 2^110: what is 2^-20 of it and less has code 0 whatever its remainder)
        if (top >= 0x1C800000u && top <= 0x76800000u) g.by = __uint_as_float(0x7F000000u - __float_as_uint(g.g));
        if (first == 0) a.scale[t] = g.g;
    } else if (kNv) {
        g.g = a.scale[t];
    }
    auto put = [&](const Unit<A, kGated>& f, uint32_t top, int u) {
        if (!kNv) top = max(top, __shfl_xor_sync(kAll, top, 1));
        if (u >= units) return;
        uint8_t byte;
        const uint2 w = unit_codes<kNv>(f, top, g, byte);
        store_codes(a.q + t * a.qs + u * 8, w);
        if (kNv) a.s[t * blocks + u] = byte;
        else if (u % 2 == 0) a.s[t * blocks + u / 2] = byte;
    };
    if (kKeep && own) {
#pragma unroll
        for (int n = 0; n < kHeld; ++n) put(v[n], tops[n], first + n * step);
    } else {
        for (int u0 = 0; u0 < units; u0 += step) {  // (whole warps, for the exchange between halves)
            const int u = u0 + first;
            uint32_t top = 0;
            if (u < units) top = v[0].template take<kWide>(row, a.K, u * kUnit);
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

// 16 elements; kWide: 32-byte words (in 16-byte ones each store of a warp leaves half of every
// sector to the next: 137 us for 65536 x 4096 to bf16).
template <typename O, bool kWide>
__device__ __forceinline__ void store_unit(O* p, const float (&f)[kUnit]) {
    const Chunk<O, kUnit> c = pack_chunk<O, kUnit>(f);
    if (kWide) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(c.v);
#pragma unroll
        for (int i = 0; i < (int)sizeof(c) / 4; i += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                         ::"l"(reinterpret_cast<uint32_t*>(p) + i), "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]),
                           "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7]) : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < kUnit; ++i) p[i] = c.v[i];
    }
}

// (code s) g, one rounding in fp32 and one to the rows' type.  blockDim.y rows a block,
// blockDim.x threads each, four units a thread on their way at once.  NVFP4: code times
// e4m3 has six bits at most and is exact in fp16; MXFP4: code times s, a power of two, is exact
// in fp32 up to 2^125 (in subnormals, too), and from there on s lends g three bits.  s g is not
// formed: it can overflow, or lose bits, where code s g does neither.
template <typename O, bool kNv, bool kWide>
__global__ void __launch_bounds__(256) k_dequantize_blocks(const Dequantize<O> a) {
    pdl_launch_dependents();
    pdl_wait();
    const int units = a.K / kUnit;
    const long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= a.rows) return;
    const float g = a.scale ? a.scale[t] : 1.f;
    const uint8_t* q = a.q + t * a.qs;
    const uint8_t* s = a.s + t * (kNv ? units : units / 2);
    O* x = a.x + t * a.xs;
    const bool whole = (uintptr_t)q % 8 == 0;
    for (int u0 = threadIdx.x; u0 < units; u0 += 4 * blockDim.x) {
        uint32_t w[4][2], byte[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int u = u0 + n * blockDim.x;
            if (u >= units) break;
            w[n][0] = w[n][1] = 0;
            if (whole) {
                const uint2 both = *reinterpret_cast<const uint2*>(q + u * 8);
                w[n][0] = both.x;
                w[n][1] = both.y;
            } else {
                for (int b = 0; b < 8; ++b) w[n][b >> 2] |= (uint32_t)q[u * 8 + b] << (8 * (b & 3));
            }
            byte[n] = s[kNv ? u : u / 2];
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int u = u0 + n * blockDim.x;
            if (u >= units) break;
            float f[kUnit];
            const __half2 sh = __half2half2(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte[n], __NV_E4M3)));
            const float e8 = ue8m0_value(byte[n]);
            const bool lend = !kNv && byte[n] > 252u;
            const float by = lend && fabsf(g) < 0x1p125f ? 8.f * g : g, p = lend ? 0.125f * e8 : e8;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t c[4];
                asm("{\n.reg .b8 b0, b1, b2, b3;\nmov.b32 {b0, b1, b2, b3}, %4;\n"
                    "cvt.rn.f16x2.e2m1x2 %0, b0;\ncvt.rn.f16x2.e2m1x2 %1, b1;\n"
                    "cvt.rn.f16x2.e2m1x2 %2, b2;\ncvt.rn.f16x2.e2m1x2 %3, b3;\n}"
                    : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3]) : "r"(w[n][h]));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    __half2 v2 = *reinterpret_cast<const __half2*>(&c[i]);
                    if (kNv) v2 = __hmul2(v2, sh);
                    float2 v = __half22float2(v2);
                    if (!kNv) v = make_float2(v.x * p, v.y * p);
                    f[8 * h + 2 * i] = v.x * by;
                    f[8 * h + 2 * i + 1] = v.y * by;
                }
            }
            store_unit<O, kWide>(x + u * kUnit, f);
        }
    }
}

// ----------------------------------------------------------------- launches --
template <typename A, bool kNv, bool kGated, bool kWide>
cudaError_t quantize_w(const Quantize<A>& a, cudaStream_t s) {
    const int units = a.K / kUnit;
    const bool two = kNv && !a.given;  // passes
    if (units <= 64) {  // a warp a row
        const dim3 warps((unsigned)((a.rows + 7LL) / 8));
        if (!two || units <= 32) return launch_pdl(k_quantize_blocks<A, kNv, kGated, kWide, true, 1>, warps, dim3(256), 0, s, a);
        return launch_pdl(k_quantize_blocks<A, kNv, kGated, kWide, true, 2>, warps, dim3(256), 0, s, a);
    }
    // Two units a thread where there are rows enough to fill the GPU with half the threads (65536 x
    // 4096 bf16: 122 us for 137; one row 1.9 for 1.5; gated rows, bound by their arithmetic, 133 for 127).
    const bool halves = a.rows >= 1024 && !kGated;
    const int each = !two ? 1 : units > 512 ? 4 : units > 256 || (halves && units > 128) ? 2 : 1;
    const int per = (units + each - 1) / each, threads = per >= 256 ? 256 : (per + 31) / 32 * 32;
    auto* f = two && units > 1024 ? k_quantize_blocks<A, kNv, kGated, kWide, false, 0>
              : each == 4         ? k_quantize_blocks<A, kNv, kGated, kWide, false, 4>
              : each == 2         ? k_quantize_blocks<A, kNv, kGated, kWide, false, 2>
                                  : k_quantize_blocks<A, kNv, kGated, kWide, false, 1>;
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
    const bool wide = ((uintptr_t)a.x | (unsigned long long)(a.xs * (long long)sizeof(O))) % 32 == 0;
    const int units = a.K / kUnit, x = units < 1024 ? (units + 3) / 4 : 256, y = 256 / x;  // four units a thread
    const dim3 grid((unsigned)((a.rows + y - 1) / y));
    auto* f = nv ? (wide ? k_dequantize_blocks<O, true, true> : k_dequantize_blocks<O, true, false>)
                 : (wide ? k_dequantize_blocks<O, false, true> : k_dequantize_blocks<O, false, false>);
    return launch_pdl(f, grid, dim3(x, y), 0, s, a);
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
    if (!aligned4(scale)) return refuse(MOE_ERR_INVALID_ARG, "%s: scale is not aligned to its elements", what);
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
    if (!aligned4(scale)) return refuse(MOE_ERR_INVALID_ARG, "%s: scale is not aligned to its elements", what);
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
