// norm_rows.cu -- the root-mean-square norm in front of an expert layer, with the
// residual's addition and 8-bit codes (moe_norm_rows), and its gradient
// (moe_norm_rows_backward; C entries at the end).
//
//   h = x + residual, rounded to the rows' type;  r = 1 / sqrt(mean h^2 + eps)
//   y = h r gamma, rounded to the rows' type
//
// and with g = dy gamma, dh the gradient that reaches h by the residual's way:
//
//   dx = dh + r (g - h r^2 mean(g h)),   dgamma = sum_t dy h r
//
// The mean is over the h that the stream holds, so that the gradient, which has
// only that h, is the gradient of what was computed.  Sums are fp32 in a fixed
// order: equal calls give equal bits.  As in sorted_rows.cu no input is
// `const __restrict__`; here h may be x or residual itself, too.
#include <cmath>
#include <type_traits>

#include "entry.h"
#include "row_codes.cuh"

namespace moe {
namespace {

// Sum over the block, the same in every thread; `part` is free again after the
// next __syncthreads.
__device__ __forceinline__ float block_sum(float v, float* part) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < (int)(blockDim.x >> 5); ++i) v += part[i];
    return v;
}

template <typename A>
struct Norm {
    const A *x, *residual;
    long long xs, rs;
    const void* gamma;
    int T, H;
    float eps;
    A *h, *y;  // either may be NULL
    long long hs, ys;
    float* rstd;  // may be NULL
    int8_t* q;    // NULL: no codes
    long long qs;
    float* scale;
};

// One block a row, or with kWarp a warp.  kKeep chunks of C elements a thread stay in
// registers from the sum to the codes; kKeep = 0: rows of any length, read again for each pass (from h
// where it is written: it may lie over an input).  Bound by HBM where rows move in 16-byte
// words: 8192 x 4096 bf16 with a residual 41.3 us, 6.5 TB/s, 32768 rows 154, 7.0; with codes
// 54.5; without a residual 27, 5.0, where L1 is busy to 68 % (each block reads gamma, in fp32 twice its
// row's bytes) and the issue slots to 58; in single elements (H = 4095) 132.
template <typename A, typename G, int C, int kKeep, int kMost, bool kWarp>
__global__ void __launch_bounds__(kMost, kMost > 256 ? 1 : kKeep == 2 ? 8 : 6) k_norm_rows(const Norm<A> a) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float part[32];
    __shared__ uint32_t tops[32];
    const long long t = kWarp ? blockIdx.x * 8LL + (threadIdx.x >> 5) : blockIdx.x;
    if (kWarp && t >= a.T) return;
    const int lane = kWarp ? threadIdx.x & 31 : threadIdx.x;
    const int first = lane * C, step = kWarp ? 32 * C : blockDim.x * C, H = a.H;
    const A* x = a.x + t * a.xs;
    const G* gamma = reinterpret_cast<const G*>(a.gamma);
    constexpr int kHeld = kKeep ? kKeep : 1;
    Chunk<A, C> held[kHeld];
    auto each = [&](auto&& f) {
        if (kKeep) {
#pragma unroll
            for (int n = 0; n < kHeld; ++n)
                if (first + n * step < H) f(held[n], first + n * step);
        } else {
            for (int c = first; c < H; c += step) f(held[0], c);
        }
    };
    auto add = [&](Chunk<A, C>& v, const Chunk<A, C>& r) {
        float f[C], g[C];
        unpack_chunk(v, f);
        unpack_chunk(r, g);
#pragma unroll
        for (int i = 0; i < C; ++i) f[i] += g[i];
        v = pack_chunk<A, C>(f);
    };
    float sum = 0.f;
    each([&](Chunk<A, C>& v, int c) {
        v = load_chunk<A, C>(x + c);
        if (a.residual) add(v, load_chunk<A, C>(a.residual + t * a.rs + c));
        if (a.h) *reinterpret_cast<Chunk<A, C>*>(a.h + t * a.hs + c) = v;
        float f[C];
        unpack_chunk(v, f);
#pragma unroll
        for (int i = 0; i < C; ++i) sum = fmaf(f[i], f[i], sum);
    });
    const float r = 1.f / sqrtf((kWarp ? warp_sum(sum) : block_sum(sum, part)) / (float)H + a.eps);
    if (lane == 0 && a.rstd) a.rstd[t] = r;
    // y of a chunk of h, in place
    auto scaled = [&](Chunk<A, C>& v, int c) {
        float f[C], g[C];
        unpack_chunk(load_chunk<G, C>(gamma + c), g);
        unpack_chunk(v, f);
#pragma unroll
        for (int i = 0; i < C; ++i) f[i] = f[i] * r * g[i];
        v = pack_chunk<A, C>(f);
    };
    const A* from = a.h ? a.h + t * a.hs : x;
    auto again = [&](Chunk<A, C>& v, int c) {  // kKeep = 0: h of the row once more
        v = load_chunk<A, C>(from + c);
        if (a.residual && !a.h) add(v, load_chunk<A, C>(a.residual + t * a.rs + c));
    };
    uint32_t top = 0;
    each([&](Chunk<A, C>& v, int c) {
        if (!kKeep) again(v, c);
        scaled(v, c);
        if (a.y) *reinterpret_cast<Chunk<A, C>*>(a.y + t * a.ys + c) = v;
        if (a.q) top = top_bits<A, C>(v, top);
    });
    if (!a.q) return;
    const float most = kWarp ? __uint_as_float(warp_most<A>(top)) : block_most<A>(top, tops);
    const RowScale by = row_scale(most);
    if (lane == 0) a.scale[t] = by.scale;
    each([&](Chunk<A, C>& v, int c) {
        if (!kKeep) {
            if (a.y) {
                v = load_chunk<A, C>(a.y + t * a.ys + c);
            } else {
                again(v, c);
                scaled(v, c);
            }
        }
        float f[C];
        unpack_chunk(v, f);
        Chunk<int8_t, C> out = {};
        if (by.live) out = quant_codes(f, by.c127, by.m, by.by);
        *reinterpret_cast<Chunk<int8_t, C>*>(a.q + t * a.qs + c) = out;
    });
}

// ---------------------------------------------------------------- gradient --
template <typename A>
struct NormBack {
    const A *dy, *dh, *h;  // dh may be NULL
    long long dys, dhs, hs;
    const void* gamma;
    const float* rstd;
    int T, H;
    A* dx;
    long long dxs;
    float* part;  // [gridDim.x][H] sums of dy h r over a block's rows, or NULL
};

// A chunk's share of the row's dot product sum(g h r) and of dgamma.
template <typename A, typename G, int C>
__device__ __forceinline__ void back_dot(const Chunk<A, C>& dy, const Chunk<A, C>& h, const Chunk<G, C>& gamma, float r,
                                         float& dot, float (&dgamma)[C]) {
    float v[C], w[C], g[C];
    unpack_chunk(dy, v);
    unpack_chunk(h, w);
    unpack_chunk(gamma, g);
#pragma unroll
    for (int i = 0; i < C; ++i) {
        w[i] *= r;
        dot = fmaf(v[i] * g[i], w[i], dot);
        dgamma[i] = fmaf(v[i], w[i], dgamma[i]);
    }
}

// A chunk of dx; mean of g h r.
template <typename A, typename G, int C>
__device__ __forceinline__ void back_dx(const Chunk<A, C>& dy, const Chunk<A, C>& h, const Chunk<G, C>& gamma,
                                        const Chunk<A, C>& dh, bool has_dh, float r, float mean, A* dx) {
    float f[C], w[C], g[C];
    unpack_chunk(dy, f);
    unpack_chunk(h, w);
    unpack_chunk(gamma, g);
#pragma unroll
    for (int i = 0; i < C; ++i) f[i] = fmaf(-w[i], r * mean, f[i] * g[i]);
    if (has_dh) {
        unpack_chunk(dh, w);
#pragma unroll
        for (int i = 0; i < C; ++i) f[i] = fmaf(r, f[i], w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) f[i] *= r;
    }
    store_chunk<A, C>(dx, f);
}

// A block walks rows t, t + gridDim.x, ... ; a thread's columns stay the same, so
// its share of dgamma is summed in registers and written once.  With kWarp each of its
// eight warps walks rows of its own, and the warps' shares are summed in their order.
template <typename A, typename G, int C, int kKeep, int kMost, bool kWarp>
__global__ void __launch_bounds__(kMost, kMost == 256 ? (kWarp && kKeep > 2 ? 2 : 3) : 1) k_norm_backward(const NormBack<A> a) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float part[2][32];
    const int warp = threadIdx.x >> 5, H = a.H;
    const int first = (kWarp ? threadIdx.x & 31 : threadIdx.x) * C, step = kWarp ? 32 * C : blockDim.x * C;
    Chunk<G, C> gamma[kKeep];
    float dgamma[kKeep][C] = {};
#pragma unroll
    for (int n = 0; n < kKeep; ++n)
        if (first + n * step < H) gamma[n] = load_chunk<G, C>(reinterpret_cast<const G*>(a.gamma) + first + n * step);
    int turn = 0;
    const long long start = kWarp ? blockIdx.x * 8LL + warp : blockIdx.x, rows = kWarp ? gridDim.x * 8LL : gridDim.x;
    for (long long t = start; t < a.T; t += rows, turn ^= 1) {
        Chunk<A, C> dy[kKeep], h[kKeep], dh[kKeep];
        const float r = a.rstd[t];
#pragma unroll
        for (int n = 0; n < kKeep; ++n) {
            const int c = first + n * step;
            if (c >= H) continue;
            dy[n] = load_chunk<A, C>(a.dy + t * a.dys + c);
            h[n] = load_chunk<A, C>(a.h + t * a.hs + c);
            if (a.dh) dh[n] = load_chunk<A, C>(a.dh + t * a.dhs + c);
        }
        float dot = 0.f;
#pragma unroll
        for (int n = 0; n < kKeep; ++n)
            if (first + n * step < H) back_dot(dy[n], h[n], gamma[n], r, dot, dgamma[n]);
        const float mean = (kWarp ? warp_sum(dot) : block_sum(dot, part[turn])) / (float)H;  // of g h r
#pragma unroll
        for (int n = 0; n < kKeep; ++n)
            if (first + n * step < H) back_dx(dy[n], h[n], gamma[n], dh[n], a.dh != nullptr, r, mean, a.dx + t * a.dxs + first + n * step);
    }
    if (!a.part) return;
    if constexpr (kWarp) {
        __shared__ alignas(32) float sums[8][kKeep * 32 * C];
#pragma unroll
        for (int n = 0; n < kKeep; ++n)
            if (first + n * step < H) store_chunk<float, C>(&sums[warp][first + n * step], dgamma[n]);
        __syncthreads();
        for (int c = threadIdx.x; c < H; c += blockDim.x) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) sum += sums[w][c];
            a.part[(long long)blockIdx.x * H + c] = sum;
        }
    } else {
#pragma unroll
        for (int n = 0; n < kKeep; ++n)
            if (first + n * step < H) store_chunk<float, C>(a.part + (long long)blockIdx.x * H + first + n * step, dgamma[n]);
    }
}

// The same for rows in 16-byte words, with the rows on their way held in shared memory, not in
// registers: a thread copies its own chunks of kDepth rows ahead and reads them back itself, so
// no barrier is between them.  A block an SM, of kGroups groups of threads with a row each, whose
// shares of dgamma meet in shared memory.  8192 x 4096 bf16 with dh: 45.6 us, 5.9 TB/s, dgamma's
// passes over 2.5 MB of parts within; with the rows in registers 52 (8192 wide: 50 and 69).
// Two groups and 128 registers there (three: 57; three blocks an SM 46.8; three rows ahead
// 46.2), three groups with half the chunks (8192 x 2048: 28.3; three blocks an SM 33, four groups 34).
template <typename A, typename G, int kKeep, int kDepth, int kGroups>
__global__ void __launch_bounds__(256 * kGroups, 1) k_norm_backward_ring(const NormBack<A> a) {
    constexpr int C = 16 / (int)sizeof(A);
    extern __shared__ __align__(16) uint4 ring[];  // [kDepth][3][kKeep][blockDim.x]
    __shared__ float part[2][kGroups][8];
    pdl_launch_dependents();
    pdl_wait();
    const int threads = blockDim.x / kGroups, group = threadIdx.x / threads, id = threadIdx.x % threads;
    const int first = id * C, step = threads * C, H = a.H;
    const long long start = (long long)blockIdx.x * kGroups + group, rows = (long long)gridDim.x * kGroups;
    Chunk<G, C> gamma[kKeep];
    float dgamma[kKeep][C] = {};
#pragma unroll
    for (int n = 0; n < kKeep; ++n)
        if (first + n * step < H) gamma[n] = load_chunk<G, C>(reinterpret_cast<const G*>(a.gamma) + first + n * step);
    auto at = [&](int slot, int which, int n) { return ((slot * 3 + which) * kKeep + n) * (int)blockDim.x + (int)threadIdx.x; };
    auto ahead = [&](long long t, int slot) {
        if (t < a.T) {
#pragma unroll
            for (int n = 0; n < kKeep; ++n) {
                const int c = first + n * step;
                if (c >= H) continue;
                const A* from[3] = {a.dy + t * a.dys + c, a.h + t * a.hs + c, a.dh ? a.dh + t * a.dhs + c : nullptr};
#pragma unroll
                for (int w = 0; w < 3; ++w)
                    if (from[w])
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                                     ::"r"((uint32_t)__cvta_generic_to_shared(&ring[at(slot, w, n)])), "l"(from[w]) : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kDepth; ++i) ahead(start + i * rows, i);
    int turn = 0, slot = 0;
    for (long long t = start; t < a.T; t += rows, turn ^= 1) {
        const float r = a.rstd[t];
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
        Chunk<A, C> dy[kKeep], h[kKeep], dh[kKeep];
#pragma unroll
        for (int n = 0; n < kKeep; ++n) {
            if (first + n * step >= H) continue;
            *reinterpret_cast<uint4*>(&dy[n]) = ring[at(slot, 0, n)];
            *reinterpret_cast<uint4*>(&h[n]) = ring[at(slot, 1, n)];
            if (a.dh) *reinterpret_cast<uint4*>(&dh[n]) = ring[at(slot, 2, n)];
        }
        ahead(t + kDepth * rows, slot);
        slot = slot + 1 == kDepth ? 0 : slot + 1;
        float dot = 0.f;
#pragma unroll
        for (int n = 0; n < kKeep; ++n)
            if (first + n * step < H) back_dot(dy[n], h[n], gamma[n], r, dot, dgamma[n]);
        dot = warp_sum(dot);
        if (id % 32 == 0) part[turn][group][id / 32] = dot;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(threads) : "memory");  // the group's own
        dot = 0.f;
        for (int i = 0; i < threads / 32; ++i) dot += part[turn][group][i];
        const float mean = dot / (float)H;  // of g h r
#pragma unroll
        for (int n = 0; n < kKeep; ++n)
            if (first + n * step < H) back_dx(dy[n], h[n], gamma[n], dh[n], a.dh != nullptr, r, mean, a.dx + t * a.dxs + first + n * step);
    }
    if (!a.part) return;
    // the groups' shares of dgamma, summed in their order: the ring has room for them
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    float* sums = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int n = 0; n < kKeep; ++n)
        if (first + n * step < H) store_chunk<float, C>(sums + group * H + first + n * step, dgamma[n]);
    __syncthreads();
    for (int c = threadIdx.x; c < H; c += blockDim.x) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) sum += sums[i * H + c];
        a.part[(long long)blockIdx.x * H + c] = sum;
    }
}

// Rows of any length: dx alone, a block a row, read twice.
template <typename A, typename G>
__global__ void __launch_bounds__(1024) k_norm_backward_long(const NormBack<A> a) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float part[32];
    const long long t = blockIdx.x;
    const A *dy = a.dy + t * a.dys, *h = a.h + t * a.hs;
    const G* gamma = reinterpret_cast<const G*>(a.gamma);
    const float r = a.rstd[t];
    float dot = 0.f;
    for (int c = threadIdx.x; c < a.H; c += blockDim.x) dot = fmaf(to_f32(dy[c]) * to_f32(gamma[c]), to_f32(h[c]) * r, dot);
    const float mean = block_sum(dot, part) / (float)a.H;
    for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
        float f = r * (to_f32(dy[c]) * to_f32(gamma[c]) - to_f32(h[c]) * r * mean);
        if (a.dh) f += to_f32(a.dh[t * a.dhs + c]);
        a.dx[t * a.dxs + c] = from_f32<A>(f);
    }
}

// Their dgamma: block (x, y) sums 256 columns over the rows y, y + gridDim.y, ...
template <typename A>
__global__ void __launch_bounds__(256) k_dgamma_long(const NormBack<A> a) {
    pdl_launch_dependents();
    pdl_wait();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.H) return;
    float sum = 0.f;
    for (long long t = blockIdx.y; t < a.T; t += gridDim.y)
        sum = fmaf(to_f32(a.dy[t * a.dys + c]), to_f32(a.h[t * a.hs + c]) * a.rstd[t], sum);
    a.part[(long long)blockIdx.y * a.H + c] = sum;
}

// dgamma[c] = the parts' sum: 32 columns a block, each warp a part in turn.
__global__ void __launch_bounds__(1024) k_join_parts(const float* part, int parts, int H, float* dgamma) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float sums[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (c < H)
        for (int p = warp; p < parts; p += 32) sum += part[(long long)p * H + c];
    sums[warp][lane] = sum;
    __syncthreads();
    sum = warp_sum(sums[lane][warp]);
    if (lane == 0 && blockIdx.x * 32 + warp < H) dgamma[blockIdx.x * 32 + warp] = sum;
}

// ----------------------------------------------------------------- launches --
// Numbers of blocks here are measured on, and meant for, 152 SMs; every form is right with any.
// Blocks of the gradient at most: three an SM of 256 threads, and more of the smaller ones
// (8192 x 1024 bf16: 29 us with 456, 20 with 912).
// Rows past 16384 are long whatever their type.
constexpr int kLongParts = 16;
int most_parts(int H) { return H <= 2048 ? 912 : H <= 16384 ? 456 : kLongParts; }

// Short rows take a warp each: the GPU starts a block in about 1 ns, so that 65536 rows of any
// width took 67 us and more (of 64 bf16: 11.4 now, 1024: 45).  The warp pays with more chunks a
// lane where rows are few: 1024 x 1024 bf16 2.6 us by blocks and 3.0 by warps, 2048 rows
// 4.4 and 4.3, 8192 8.8 and 7.5.  The gradient's blocks walk rows, and there the warps win as long as
// a lane has 16 columns (8192 x 256 bf16: 6.4 us for 10.3, 65536: 29 for 81; 8192 x 512
// fp32 15.5 for 18.4, but x 1024 bf16, 32 columns, 27.6 for 20.3); 456 blocks of them (912:
// 7.9 us for the first, 304: 7.0).
constexpr int kWarpRows = 2048, kWarpBlocks = 456;

int threads_for(int chunks) { return (chunks + 31) / 32 * 32; }

// Few rows, all of them on the GPU at once: a thread a chunk (1000 x 2048 bf16: 3.0 us; 3.9 with two
// chunks, 4.4 with four).  Many: two chunks a thread and eight blocks of 256 an SM (8192 x 4096 bf16
// 26.9 us and with a residual 41.3; four chunks 28.2 and 42.2, one 33 and 43), or four for
// fp32 rows without a residual (32768 x 2048: 79 us for 89) and for long rows.
constexpr long long kAtOnce = 152 * 2048;
template <typename A, typename G, int C>
cudaError_t norm_c(const Norm<A>& a, cudaStream_t s) {
    const int chunks = (a.H + C - 1) / C;
    if (chunks <= 32 || (chunks <= 128 && a.T >= kWarpRows)) {
        const dim3 grid((a.T + 7) / 8);
        if (chunks <= 32) return launch_pdl(k_norm_rows<A, G, C, 1, 256, true>, grid, dim3(256), 0, s, a);
        if (chunks <= 64) return launch_pdl(k_norm_rows<A, G, C, 2, 256, true>, grid, dim3(256), 0, s, a);
        return launch_pdl(k_norm_rows<A, G, C, 4, 256, true>, grid, dim3(256), 0, s, a);
    }
    if (chunks <= 128 || (chunks <= 512 && (long long)a.T * chunks <= kAtOnce))
        return launch_pdl(k_norm_rows<A, G, C, 1, 512, false>, dim3(a.T), dim3(threads_for(chunks)), 0, s, a);
    if (chunks <= 512 && (sizeof(A) == 2 || a.residual))
        return launch_pdl(k_norm_rows<A, G, C, 2, 256, false>, dim3(a.T), dim3(threads_for((chunks + 1) / 2)), 0, s, a);
    if (chunks <= 1024) return launch_pdl(k_norm_rows<A, G, C, 4, 256, false>, dim3(a.T), dim3(threads_for((chunks + 3) / 4)), 0, s, a);
    if (chunks <= 4096) return launch_pdl(k_norm_rows<A, G, C, 4, 1024, false>, dim3(a.T), dim3(threads_for((chunks + 3) / 4)), 0, s, a);
    return launch_pdl(k_norm_rows<A, G, C, 0, 1024, false>, dim3(a.T), dim3(1024), 0, s, a);
}

template <typename A, typename G, int kKeep, int kDepth, int kGroups>
cudaError_t back_ring(const NormBack<A>& a, int parts, int threads, cudaStream_t s) {
    auto* kernel = k_norm_backward_ring<A, G, kKeep, kDepth, kGroups>;
    const int smem = kDepth * 3 * kKeep * kGroups * threads * 16;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    return e != cudaSuccess ? e : launch_pdl(kernel, dim3(parts), dim3(kGroups * threads), smem, s, a);
}

template <typename A, typename G, int C>
cudaError_t back_c(const NormBack<A>& a, float* dgamma, cudaStream_t s) {
    const int chunks = (a.H + C - 1) / C;
    const int most = most_parts(a.H);
    int parts = a.T < most ? a.T : most;
    cudaError_t e = cudaSuccess;
    if (a.T == 0) {
    } else if (chunks <= 128 && a.H <= 512) {
        parts = a.T < 8 * kWarpBlocks ? (a.T + 7) / 8 : kWarpBlocks;
        const dim3 grid(parts);
        if (chunks <= 32) e = launch_pdl(k_norm_backward<A, G, C, 1, 256, true>, grid, dim3(256), 0, s, a);
        else if (chunks <= 64) e = launch_pdl(k_norm_backward<A, G, C, 2, 256, true>, grid, dim3(256), 0, s, a);
        else if constexpr (C <= 4) e = launch_pdl(k_norm_backward<A, G, C, 4, 256, true>, grid, dim3(256), 0, s, a);
    } else if (C == 16 / (int)sizeof(A) && a.T > 456 && chunks > 128 && chunks <= 1024) {
        parts = 152;
        if (chunks <= 256) e = back_ring<A, G, 1, 3, 3>(a, parts, threads_for(chunks), s);
        else if (chunks <= 512) e = back_ring<A, G, 2, 2, 2>(a, parts, threads_for((chunks + 1) / 2), s);
        else e = back_ring<A, G, 4, 2, 1>(a, parts, threads_for((chunks + 3) / 4), s);
    } else if (chunks <= 2048) {
        const dim3 grid(parts);
        if (chunks <= 256) e = launch_pdl(k_norm_backward<A, G, C, 1, 256, false>, grid, dim3(threads_for(chunks)), 0, s, a);
        else if (chunks <= 512) e = launch_pdl(k_norm_backward<A, G, C, 2, 256, false>, grid, dim3(threads_for((chunks + 1) / 2)), 0, s, a);
        else if (chunks <= 1024) e = launch_pdl(k_norm_backward<A, G, C, 2, 512, false>, grid, dim3(threads_for((chunks + 1) / 2)), 0, s, a);
        else e = launch_pdl(k_norm_backward<A, G, C, 4, 512, false>, grid, dim3(threads_for((chunks + 3) / 4)), 0, s, a);
    } else {
        // dgamma first: dx may lie over dy
        parts = parts < kLongParts ? parts : kLongParts;
        if (a.part) e = launch_pdl(k_dgamma_long<A>, dim3((a.H + 255) / 256, parts), dim3(256), 0, s, a);
        if (e == cudaSuccess) e = launch_pdl(k_norm_backward_long<A, G>, dim3(a.T), dim3(1024), 0, s, a);
    }
    if (e == cudaSuccess && dgamma)
        e = launch_pdl(k_join_parts, dim3((a.H + 31) / 32), dim3(1024), 0, s, (const float*)a.part, parts, a.H, dgamma);
    return e;
}

// The widest chunk that every row of every operand allows (16 bytes of A; gamma's
// rows are one row of another type).
template <typename A, typename G, typename F>
cudaError_t by_chunk(unsigned align, const void* gamma, int H, F&& f) {
    constexpr int W = 16 / (int)sizeof(A);
    const uintptr_t g = (uintptr_t)gamma;
    if (H % W == 0 && align >= 16 && g % 16 == 0) return f(std::integral_constant<int, W>());
    if (H % 2 == 0 && align >= 2 * sizeof(A) && g % (2 * sizeof(G)) == 0) return f(std::integral_constant<int, 2>());
    return f(std::integral_constant<int, 1>());
}

unsigned least(unsigned a, unsigned b) { return a < b ? a : b; }

template <typename A, typename G>
cudaError_t norm_ag(const Norm<A>& a, cudaStream_t s) {
    constexpr long long z = sizeof(A);
    unsigned al = row_align(a.x, a.xs * z);
    if (a.residual) al = least(al, row_align(a.residual, a.rs * z));
    if (a.h) al = least(al, row_align(a.h, a.hs * z));
    if (a.y) al = least(al, row_align(a.y, a.ys * z));
    if (a.q) al = least(al, (unsigned)z * row_align(a.q, a.qs));  // a code for each element
    return by_chunk<A, G>(al, a.gamma, a.H, [&](auto c) { return norm_c<A, G, decltype(c)::value>(a, s); });
}

template <typename A, typename G>
cudaError_t back_ag(NormBack<A> a, float* dgamma, cudaStream_t s) {
    constexpr long long z = sizeof(A);
    unsigned al = least(row_align(a.dy, a.dys * z), row_align(a.h, a.hs * z));
    al = least(al, row_align(a.dx, a.dxs * z));
    if (a.dh) al = least(al, row_align(a.dh, a.dhs * z));
    return by_chunk<A, G>(al, a.gamma, a.H, [&](auto c) { return back_c<A, G, decltype(c)::value>(a, dgamma, s); });
}

moe_status check_norm(const char* what, moe_dtype dtype, moe_dtype gamma_dtype, int T, int H) {
    if (!dtype_ok(dtype)) return refuse(MOE_ERR_INVALID_ARG, "%s: unknown dtype", what);
    if (gamma_dtype != dtype && gamma_dtype != MOE_F32)
        return refuse(MOE_ERR_INVALID_ARG, "%s: gamma's dtype must be the rows' or MOE_F32", what);
    if (T < 0 || T > (1 << 24)) return refuse(MOE_ERR_INVALID_ARG, "%s: T must be in [0, 2^24]", what);
    if (H < 1 || H > 131072) return refuse(MOE_ERR_INVALID_ARG, "%s: hidden must be in [1, 131072]", what);
    return MOE_OK;
}

// A matrix of rows; `needed`: it may not be NULL.
moe_status check_matrix(const char* what, const char* name, const void* p, long long stride, int H, int size, bool needed) {
    if (!p) return needed ? refuse(MOE_ERR_INVALID_ARG, "%s: %s is NULL", what, name) : MOE_OK;
    if (stride < H || stride > kMostStride)
        return refuse(MOE_ERR_INVALID_ARG, "%s: the row stride of %s is below the row or above 2^40", what, name);
    if ((uintptr_t)p % size) return refuse(MOE_ERR_INVALID_ARG, "%s: %s is not aligned to its elements", what, name);
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_norm_rows(const void* x, moe_dtype dtype, long long x_stride, const void* residual,
                                    long long residual_stride, const void* gamma, moe_dtype gamma_dtype, int T, int hidden,
                                    float eps, void* h, long long h_stride, void* y, long long y_stride, float* rstd,
                                    int8_t* q, long long q_stride, float* scale, moe_stream_t stream) {
    const char* what = "moe_norm_rows";
    moe_status st = check_norm(what, dtype, gamma_dtype, T, hidden);
    if (st == MOE_OK && !(eps >= 0.f && std::isfinite(eps)))
        st = refuse(MOE_ERR_INVALID_ARG, "%s: eps must be finite and not negative", what);
    if (st != MOE_OK || T == 0) return st;
    const int z = dtype_size(dtype);
    st = check_matrix(what, "x", x, x_stride, hidden, z, true);
    if (st == MOE_OK) st = check_matrix(what, "residual", residual, residual_stride, hidden, z, false);
    if (st == MOE_OK) st = check_matrix(what, "h", h, h_stride, hidden, z, false);
    if (st == MOE_OK) st = check_matrix(what, "y", y, y_stride, hidden, z, q == nullptr);
    if (st == MOE_OK) st = check_matrix(what, "q", q, q_stride, hidden, 1, false);
    if (st == MOE_OK) st = check_matrix(what, "gamma", gamma, hidden, hidden, dtype_size(gamma_dtype), true);
    if (st == MOE_OK && (q == nullptr) != (scale == nullptr))
        st = refuse(MOE_ERR_INVALID_ARG, "%s: of q and scale one is NULL", what);
    if (st == MOE_OK && !aligned4(rstd, scale))
        st = refuse(MOE_ERR_INVALID_ARG, "%s: rstd or scale is not aligned to its elements", what);
    if (st != MOE_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    auto run = [&](auto type) {
        using A = decltype(type);
        const Norm<A> a{(const A*)x, (const A*)residual, x_stride, residual_stride, gamma, T, hidden, eps, (A*)h, (A*)y,
                        h_stride, y_stride, rstd, q, q_stride, scale};
        return gamma_dtype == MOE_F32 ? norm_ag<A, float>(a, s) : norm_ag<A, A>(a, s);
    };
    cudaError_t e;
    if (dtype == MOE_F32) e = run(float());
    else if (dtype == MOE_BF16) e = run(__nv_bfloat16());
    else e = run(__half());
    return status_of(e, what);
}

extern "C" size_t moe_norm_scratch_bytes(int T, int hidden) {
    if (T < 0 || T > (1 << 24) || hidden < 1 || hidden > 131072) return 0;
    const int most = most_parts(hidden);
    return (size_t)(T < 1 ? 1 : T < most ? T : most) * hidden * sizeof(float);
}

extern "C" moe_status moe_norm_rows_backward(const void* dy, moe_dtype dtype, long long dy_stride, const void* dh,
                                             long long dh_stride, const void* h, long long h_stride, const void* gamma,
                                             moe_dtype gamma_dtype, const float* rstd, int T, int hidden, void* dx,
                                             long long dx_stride, float* dgamma, void* scratch, size_t scratch_bytes,
                                             moe_stream_t stream) {
    const char* what = "moe_norm_rows_backward";
    moe_status st = check_norm(what, dtype, gamma_dtype, T, hidden);
    if (st != MOE_OK) return st;
    if (dgamma && (!scratch || scratch_bytes < moe_norm_scratch_bytes(T, hidden)))
        return refuse(MOE_ERR_INVALID_ARG, "%s: scratch is NULL or below moe_norm_scratch_bytes", what);
    if (dgamma && (uintptr_t)scratch % 16) return refuse(MOE_ERR_INVALID_ARG, "%s: scratch is not aligned to 16 bytes", what);
    if (!aligned4(rstd, dgamma)) return refuse(MOE_ERR_INVALID_ARG, "%s: rstd or dgamma is not aligned to its elements", what);
    if (T == 0 && !dgamma) return MOE_OK;
    const int z = dtype_size(dtype);
    if (T > 0) {
        st = check_matrix(what, "dy", dy, dy_stride, hidden, z, true);
        if (st == MOE_OK) st = check_matrix(what, "dh", dh, dh_stride, hidden, z, false);
        if (st == MOE_OK) st = check_matrix(what, "h", h, h_stride, hidden, z, true);
        if (st == MOE_OK) st = check_matrix(what, "dx", dx, dx_stride, hidden, z, true);
        if (st == MOE_OK) st = check_matrix(what, "gamma", gamma, hidden, hidden, dtype_size(gamma_dtype), true);
        if (st == MOE_OK && !rstd) st = refuse(MOE_ERR_INVALID_ARG, "%s: rstd is NULL", what);
        if (st != MOE_OK) return st;
    }
    cudaStream_t s = (cudaStream_t)stream;
    auto run = [&](auto type) {
        using A = decltype(type);
        const NormBack<A> a{(const A*)dy, (const A*)dh, (const A*)h, dy_stride, dh_stride, h_stride, gamma, rstd, T,
                            hidden, (A*)dx, dx_stride, dgamma ? (float*)scratch : nullptr};
        return gamma_dtype == MOE_F32 ? back_ag<A, float>(a, dgamma, s) : back_ag<A, A>(a, dgamma, s);
    };
    cudaError_t e;
    if (dtype == MOE_F32) e = run(float());
    else if (dtype == MOE_BF16) e = run(__nv_bfloat16());
    else e = run(__half());
    return status_of(e, what);
}
