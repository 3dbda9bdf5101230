// int_product_tc.cu -- the product with 8-bit integer experts on the tensor
// cores (moe_expert_product).
//
// This part's tensor cores have no fast 8-bit integer form, but an 8-bit integer is
// exact in fp16, a product of two is exact in fp32 and so is a sum of them up
// to 2^24: the codes are turned into fp16 on the way to tcgen05.mma.kind::f16
// with fp32 accumulators.  For K up to 1024 no sum passes 2^24, at K = 16384 a mean
// |q wq| of 1024 with signs that agree is enough.  Past it the accumulator rounds once
// in every 16 products, in all within 2^-23 (2 + K / 16) of the sum of |q wq|.
//
// One CTA per SM walks tiles of 128 output channels (A, one tensor-memory lane
// a channel) x up to kCap positions of one segment (B), K in units of 128:
//   kAGroups warpgroups  codes of one channel a thread -> fp16 -> tensor memory
//                        (the A operand: it takes no shared-memory bandwidth from B)
//   kBGroups x 4 warps   token codes: global -> registers, a few units ahead and
//                        across tiles -> fp16 -> shared memory, rows of 128 bytes,
//                        128-byte swizzle; a gather costs nothing here
//   kEpiWarps warps      accumulators -> scales -> out
//   1 warp               TMA of 128 channels x 128 bytes of codes into a ring
//   1 warp               the MMAs
//   1 warp               token rows and scales of up to kTabs tiles ahead
// The groups of one kind take the units in turn, two units in the making at once.
//
// Measured at K = N = 4096 (bf16 out), the copy rate being 6.78 TB/s and cuBLAS's bf16
// rate 1909 TFLOP/s: 3000 rows over some 231 of 256 experts 630 us, 6.2 TB/s of
// weights; 49152 rows over 256 experts 1.29 ms, 1.28 PFLOP/s, where a fixed 14 us a
// round (a tile's 32 units of weights, whatever its rows) weighs on tiles of 150
// rows; 8192 rows of one expert 155 us, 1.77 PFLOP/s.
#include <cuda.h>

#include <cmath>
#include <mutex>

#include "int_product.cuh"
#include "tc_ptx.cuh"

namespace moe {

namespace {

using namespace tc;

constexpr int kRawBytes = 128 * 128;  // one ring slot of weight codes

// Narrow tiles are bound by the stream of weights: a long ring, one CTA a tile.
// Wide ones are bound by the MMA and by the turning of codes: a pair of CTAs (a
// cluster of two on one MMA, cta_group::2) takes 256 channels x 256 positions; each
// turns its own 128 channels and one half of the positions, half of what a CTA
// alone would turn for the same products.
template <bool kPair_>
struct Cfg {
    static constexpr bool kPair = kPair_;
    static constexpr int kCtas = kPair ? 2 : 1;
    static constexpr int kCap = kPair ? 256 : 64;           // positions of a tile
    static constexpr int kRows = kCap / kCtas;              // of them in this CTA's shared memory
    static constexpr int kUnit = 128;                       // K of one unit
    static constexpr int kSlots = 4;                        // units in flight to the MMA
    static constexpr int kRaw = kPair ? 4 : 8;              // weight ring
    static constexpr int kAGroups = 2;
    static constexpr int kBGroups = 2;
    static constexpr int kBWarps = 4;                       // warps of one token group
    static constexpr int kLanes = kUnit / 16;               // lanes that share a token's unit
    static constexpr int kPass = kBWarps * 32 / kLanes;     // token rows a group moves at once
    static constexpr int kPasses = kRows / kPass;
    static constexpr int kAhead = kPair ? 1 : 2;            // units of token codes held in registers
    static constexpr int kTabs = 4;                         // tiles whose token rows are looked up
    static constexpr int kSubBytes = kRows * 128;           // 64 of K of all its positions in fp16
    static constexpr int kBBytes = kSubBytes * (kUnit / 64);
    static constexpr int kACols = kUnit / 2;                // tensor-memory columns of one unit
    static constexpr int kACol = 512 - kACols * kSlots;
    static constexpr int kAccs = kPair ? 1 : 2;             // accumulators of a tile
    static constexpr int kBufs = kPair ? 1 : 2;             // tiles in tensor memory
    static constexpr int kBFirst = 4 * kAGroups;
    static constexpr int kEpi = kBFirst + kBGroups * kBWarps;   // first epilogue warp; then TMA, MMA, rows
    static constexpr int kEpiWarps = kPair ? 8 : 4;
    static constexpr int kTma = kEpi + kEpiWarps, kMma = kTma + 1, kLook = kMma + 1;
    static constexpr int kThreads = (kLook + 1) * 32;
    static constexpr int kSmem = 1024 + kSlots * kBBytes + kRaw * kRawBytes;
    // Units are counted through all tiles of a CTA and the groups take them in turn, so a
    // slot of either ring always belongs to the same group: one that met every other use
    // of a slot could take the phase before last, of the same parity, for its own.
    static_assert(kRaw % kAGroups == 0 && kSlots % kAGroups == 0 && kSlots % kBGroups == 0, "rings");
    static_assert(kRows % kPass == 0 && kCap % 32 == 0 && kBufs * kAccs * kCap <= kACol, "tensor memory");
};

// One lane of the warp, the same one each time: 1 there, 0 elsewhere.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t r;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xFFFFFFFF;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r;
}

// D[tmem] (+)= A[tmem] B[smem]^T, fp16 operands, fp32 accumulators; called by the
// whole warp, issued by the lane with `on`.  Under an `if` on the lane instead,
// the operands are no longer uniform over the warp and an issue takes 147
// cycles whatever N is; so it takes 35 to 60 for N <= 64 and N / 2 above (measured).
template <bool kPair>
__device__ __forceinline__ void mma_f16_ts(uint32_t on, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
    if (kPair)
        asm volatile(
            "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}"
            ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(on)
            : "memory");
    else
        asm volatile(
            "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
            ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(on)
            : "memory");
}

// Arrives on the barrier (of both CTAs of a pair) when the MMAs so far are done.
template <bool kPair>
__device__ __forceinline__ void mma_commit_by(uint32_t on, uint32_t bar) {
    if (kPair)
        asm volatile(
            "{\n.reg .pred q;\n.reg .b16 m;\nmov.b16 m, 3;\nsetp.ne.b32 q, %1, 0;\n"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n}"
            ::"r"(bar), "r"(on)
            : "memory");
    else
        asm volatile(
            "{\n.reg .pred q;\nsetp.ne.b32 q, %1, 0;\n"
            "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar), "r"(on)
            : "memory");
}

// Arrives on the pair's first CTA's barrier at the same place as `bar` here.  What
// it orders (this CTA's shared and tensor memory, read by the pair's MMA) is local
// and fenced for the MMA before; with release.cluster instead every arrival waits
// for a fence over the cluster, about 2000 cycles a unit (measured, all else equal:
// 2260 us for the 49152 rows of 256 experts at K = N = 4096, and 1570 without).
__device__ __forceinline__ void mbar_arrive_first(uint32_t bar) {
    asm volatile(
        "{\n.reg .b32 r;\nmapa.shared::cluster.u32 r, %0, 0;\n"
        "mbarrier.arrive.shared::cluster.b64 _, [r];\n}" ::"r"(bar) : "memory");
}

// mbar_wait for phases that come late as a rule (and, in a pair, from threads of
// the other CTA as well): the thread is suspended for up to 100 us at a time, so
// that polling leaves the issue slots to the others (677 us for 684 at 3000 rows).
template <bool kPair>
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    if (kPair)
        asm volatile(
            "{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
            "selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok) : "r"(bar), "r"(parity), "r"(100000u) : "memory");
    else
        asm volatile(
            "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
            "selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok) : "r"(bar), "r"(parity), "r"(100000u) : "memory");
    return ok != 0;
}

// One look, without suspension.
template <bool kPair>
__device__ __forceinline__ bool test_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    if (kPair)
        asm volatile(
            "{\n.reg .pred p;\nmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
            "selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    else
        asm volatile(
            "{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
            "selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}

template <bool kPair>
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
    if (try_wait<kPair>(bar, parity)) return true;
    const uint64_t t0 = globaltimer();
    while (!try_wait<kPair>(bar, parity))
        if (*abort || globaltimer() - t0 > limit_ns) return false;
    return true;
}

__device__ __forceinline__ void pair_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <bool kPair>
__device__ __forceinline__ void tmem_alloc_all(uint32_t slot) {
    if (!kPair) return tmem_alloc(slot, 512);
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(slot) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

template <bool kPair>
__device__ __forceinline__ void tmem_free_all(uint32_t taddr) {
    if (!kPair) return tmem_dealloc(taddr, 512);
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(taddr) : "memory");
}

// 32 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
          "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
          "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Four codes to two words of two fp16: with the sign bit turned, byte b = code
// + 128 under the high byte 0x64 reads 1024 + b, from which 1152 is taken; all exact.
__device__ __forceinline__ void codes_to_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = v ^ 0x80808080u;
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), bias);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
}

// 16 bytes; volatile, so that it is issued here and not at its use.
__device__ __forceinline__ void ld_ahead(uint4& v, const int8_t* p) {
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
}

__device__ __forceinline__ void st_shared16(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

struct Tile {
    int e, n0, p0, count;
};

__device__ uint32_t g_product_err;   // sticky, taken by moe_check_product
__device__ uint32_t g_product_seen;  // what the check under way has taken

// Reads and clears the flag in one step: what is raised after it stays for the next.
__global__ void k_take_flag() { g_product_seen = atomicExch(&g_product_err, 0u); }

template <bool kPair, typename O>
__global__ void __launch_bounds__(Cfg<kPair>::kThreads, 1) k_product_tc(const Product a, const __grid_constant__ CUtensorMap wmap) {
    using C = Cfg<kPair>;
    constexpr int kCap = C::kCap;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[2 * C::kRaw + 2 * C::kSlots + 4 + 2 * C::kTabs];
    __shared__ uint32_t token_at[C::kTabs][C::kRows];  // where a tile's rows of q start, in 16 bytes
    __shared__ int token_passes[C::kTabs];
    __shared__ __align__(8) float token_scale[C::kTabs][kCap];
    __shared__ int first[kMaxExperts + 1];  // token tiles before each expert
    __shared__ int begin[kMaxExperts + 1];  // its segment
    __shared__ int scan[32];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    constexpr unsigned kAll = 0xFFFFFFFFu;
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = kPair ? blockIdx.x & 1 : 0;  // in the pair
    const int first_tile = blockIdx.x / C::kCtas, tile_step = gridDim.x / C::kCtas;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t b_base = base, raw_base = base + C::kSlots * C::kBBytes;
    const uint32_t bar0 = smem_u32(bars);
    auto raw_full = [&](int i) { return bar0 + 8u * i; };
    auto raw_empty = [&](int i) { return bar0 + 8u * (C::kRaw + i); };
    auto full = [&](int i) { return bar0 + 8u * (2 * C::kRaw + i); };
    auto empty = [&](int i) { return bar0 + 8u * (2 * C::kRaw + C::kSlots + i); };
    auto d_full = [&](int i) { return bar0 + 8u * (2 * C::kRaw + 2 * C::kSlots + i); };
    auto d_empty = [&](int i) { return bar0 + 8u * (2 * C::kRaw + 2 * C::kSlots + 2 + i); };
    auto tab_full = [&](int i) { return bar0 + 8u * (2 * C::kRaw + 2 * C::kSlots + 4 + i); };
    auto tab_empty = [&](int i) { return bar0 + 8u * (2 * C::kRaw + 2 * C::kSlots + 4 + C::kTabs + i); };
    volatile int* abort = &abort_flag;
    if (tid == 0) {
        for (int i = 0; i < C::kRaw; ++i) {
            mbar_init(raw_full(i), 1);
            mbar_init(raw_empty(i), 4);
        }
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(full(i), C::kCtas * (4 + C::kBWarps));
            mbar_init(empty(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(d_full(i), 1);
            mbar_init(d_empty(i), C::kCtas * C::kEpiWarps);
        }
        for (int i = 0; i < C::kTabs; ++i) {
            mbar_init(tab_full(i), 1);
            mbar_init(tab_empty(i), C::kBGroups * C::kBWarps + C::kEpiWarps);
        }
        abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&wmap);
    }
    // all 512 columns: they start at address 0, which the code below relies on
    if (warp == C::kMma) tmem_alloc_all<kPair>(smem_u32(&tmem_slot));
    pdl_wait();

    // token tiles of every expert: ceil(count / kCap) of nearly equal size
    {
        int mine = 0;
        const int per = (a.E + C::kThreads - 1) / C::kThreads;
        for (int i = 0; i < per; ++i) {
            const int e = tid * per + i;
            if (e <= a.E) begin[e] = segment_at(a, e);
            if (e < a.E) mine += (max(segment_at(a, e + 1) - begin[e], 0) + kCap - 1) / kCap;
        }
        if (tid == 0) begin[a.E] = segment_at(a, a.E);
        int run = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kAll, run, o);
            if (lane >= o) run += v;
        }
        if (lane == 31) scan[warp] = run;
        __syncthreads();
        int before = run - mine;
        for (int i = 0; i < warp; ++i) before += scan[i];
        for (int i = 0; i < per; ++i) {
            const int e = tid * per + i;
            if (e < a.E) {
                first[e] = before;
                before += (max(begin[e + 1] - begin[e], 0) + kCap - 1) / kCap;
                if (e == a.E - 1) first[a.E] = before;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (kPair) pair_sync();  // the other CTA's barriers are ready
    tc_fence_after();
    const int m_tiles = (a.N + 128 * C::kCtas - 1) / (128 * C::kCtas);
    const int tiles = first[a.E] * m_tiles;  // below 2^28: R <= 2^20, N <= 2^20
    const int units = (a.K + C::kUnit - 1) / C::kUnit;
    const int my_tiles = first_tile < tiles ? (tiles - first_tile + tile_step - 1) / tile_step : 0;

    // Tile t: the channels of one token tile follow each other.
    auto tile_at = [&](int t) {
        const int tt = t / m_tiles;
        int lo = 0, hi = a.E - 1;  // last e with first[e] <= tt
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= tt) lo = mid; else hi = mid - 1;
        }
        Tile w;
        w.e = lo;
        w.n0 = ((t - tt * m_tiles) * C::kCtas + rank) * 128;
        const int count = begin[lo + 1] - begin[lo], n = first[lo + 1] - first[lo];
        const int step = n < 8 ? ((count + n - 1) / n + 15) / 16 * 16 : kCap;  // at most kCap
        w.p0 = begin[lo] + (tt - first[lo]) * step;
        w.count = min(step, begin[lo + 1] - w.p0);
        return w;
    };
    // Accumulator columns of so many positions; each CTA of a pair holds one half.
    auto columns = [&](int count) { return (count + 16 * C::kCtas - 1) / (16 * C::kCtas) * (16 * C::kCtas); };
    auto arrive_full = [&](int i) {
        if (kPair) mbar_arrive_first(full(i)); else mbar_arrive(full(i));
    };
    auto release = [&](int b) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            if (kPair) mbar_arrive_first(d_empty(b)); else mbar_arrive(d_empty(b));
        }
    };
    bool ok = true;

    if (warp == C::kTma) {
        // ------------------------------------------------- weight codes (TMA) --
        int i = 0;
        for (int t = first_tile; t < tiles && ok; t += tile_step) {
            const Tile w = tile_at(t);
            for (int k0 = 0; k0 < a.K && ok; k0 += 128, ++i) {
                const int s = i % C::kRaw;
                ok = __all_sync(kAll, wait_for<false>(raw_empty(s), ((i / C::kRaw) & 1) ^ 1, abort, a.wait_ns));
                if (ok && lane == 0) {
                    mbar_arrive_expect_tx(raw_full(s), kRawBytes);
                    if (!a.stall) tma_load_2d(raw_base + s * kRawBytes, &wmap, k0, w.e * a.N + w.n0, raw_full(s));
                }
                __syncwarp();
            }
        }
    } else if (warp == C::kLook) {
        // --------------------------------------- rows and scales of the tiles --
        int n = 0;
        for (int t = first_tile; t < tiles && ok; t += tile_step, ++n) {
            const Tile w = tile_at(t);
            const int i = n % C::kTabs, half = columns(w.count) / C::kCtas;
            ok = __all_sync(kAll, wait_for<false>(tab_empty(i), ((n / C::kTabs) & 1) ^ 1, abort, a.wait_ns));
            if (!ok) break;
            for (int c = lane; c < kCap; c += 32) {
                const int r = c < w.count ? source_row(a, w.p0 + c) : -1;
                token_scale[i][c] = r >= 0 ? a.scale[r] : 0.f;
                // this CTA's half; positions without a row read any: none of their sums is
                // used but times 0
                const int row = c - rank * half;
                if (row >= 0 && row < C::kRows) token_at[i][row] = (uint32_t)(max(r, 0) * (a.qs >> 4));
            }
            if (lane == 0) token_passes[i] = (half + C::kPass - 1) / C::kPass;
            __syncwarp();
            if (lane == 0) mbar_arrive(tab_full(i));
        }
    } else if (warp == C::kMma) {
        // ------------------------------------------------------------- MMA --
        // (the first CTA of a pair issues for both)
        // Narrow: N is always kCap, which costs no more than a smaller N and keeps the
        // instruction's word a constant, and the steps take turns on two accumulators: one
        // that waits for itself takes 51 cycles a step, two 35 (measured).  The
        // epilogue adds the two.
        // The next unit is looked for between the steps of this one: a look, its vote and
        // fence take about 300 cycles, which the MMAs' queue would not cover.
        const uint32_t on = elect_lane();
        const uint64_t b0 = desc_sw128(b_base);
        int s = 0, n = 0;
        uint32_t phase = 0;
        bool ready = false;  // unit s has been seen
        for (int t = first_tile; t < tiles && ok && rank == 0; t += tile_step, ++n) {
            // (the reduction's result is known to be uniform, a value from memory is not)
            const uint32_t cols = kPair ? __reduce_max_sync(kAll, columns(tile_at(t).count)) : kCap;
            const uint32_t idesc = (1u << 4) | ((cols >> 3) << 17) | ((128u * C::kCtas >> 4) << 24);
            const int b = n % C::kBufs;
            const uint32_t d = __reduce_max_sync(kAll, (uint32_t)(b * C::kAccs * kCap));
            ok = __all_sync(kAll, wait_for<kPair>(d_empty(b), ((n / C::kBufs) & 1) ^ 1, abort, a.wait_ns));
            tc_fence_after();
            for (int k = a.K; k > 0 && ok; k -= C::kUnit) {
                if (!ready) {
                    ok = __all_sync(kAll, wait_for<kPair>(full(s), phase, abort, a.wait_ns));
                    if (!ok) break;
                    tc_fence_after();
                }
                const int su = __reduce_max_sync(kAll, s);  // uniform: 652 to 629 us at 3000 rows
                const uint64_t bd = b0 + (uint64_t)(su * (C::kBBytes >> 4));
                const uint32_t ad = C::kACol + su * C::kACols, fresh = k == a.K, done = empty(su);
                auto step = [&](int i) {
                    mma_f16_ts<kPair>(on, d + (i % C::kAccs) * kCap, ad + i * 8,
                                      bd + (uint64_t)((i >> 2) * (C::kSubBytes >> 4) + (i & 3) * 2), idesc,
                                      i >= C::kAccs || !fresh);
                };
                if (++s == C::kSlots) {
                    s = 0;
                    phase ^= 1;
                }
                if (k >= C::kUnit) {
                    const bool seen = test_wait<kPair>(full(s), phase);
#pragma unroll
                    for (int i = 0; i < C::kUnit / 32; ++i) step(i);
                    ready = __all_sync(kAll, seen);
                    if (ready) tc_fence_after();
#pragma unroll
                    for (int i = C::kUnit / 32; i < C::kUnit / 16; ++i) step(i);
                } else {
                    for (int i = 0; i * 16 < k; ++i) step(i);
                    ready = false;
                }
                mma_commit_by<kPair>(on, done);
            }
            if (ok) mma_commit_by<kPair>(on, d_full(b));
        }
    } else if (warp < C::kBFirst) {
        // --------------------------------------------- weights to tensor memory --
        const int lanes = (warp & 3) * 32, r = lanes + lane, group = warp >> 2;
        const uint32_t lane_at = (uint32_t)lanes << 16;
        const int all_units = my_tiles * units;
        for (int g = group; g < all_units && ok; g += C::kAGroups) {
            const int rs = g % C::kRaw, s = g % C::kSlots;
            ok = __all_sync(kAll, wait_for<false>(raw_full(rs), (g / C::kRaw) & 1, abort, a.wait_ns));
            if (!ok) break;
            const uint32_t row = raw_base + rs * kRawBytes + r * 128;
#pragma unroll
            for (int h = 0; h < C::kUnit / 64; ++h) {
                uint4 v[4];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(v[c].x), "=r"(v[c].y), "=r"(v[c].z), "=r"(v[c].w)
                                 : "r"(row + (((4 * h + c) ^ (r & 7)) << 4)) : "memory");
                uint32_t f[32];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    codes_to_f16(v[c].x, f[8 * c], f[8 * c + 1]);
                    codes_to_f16(v[c].y, f[8 * c + 2], f[8 * c + 3]);
                    codes_to_f16(v[c].z, f[8 * c + 4], f[8 * c + 5]);
                    codes_to_f16(v[c].w, f[8 * c + 6], f[8 * c + 7]);
                }
                if (h == 0) {
                    ok = __all_sync(kAll, wait_for<kPair>(empty(s), ((g / C::kSlots) & 1) ^ 1, abort, a.wait_ns));
                    if (!ok) break;
                    tc_fence_after();
                }
                tmem_st32(lane_at + C::kACol + s * C::kACols + 32 * h, f);
            }
            if (!ok) break;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                // the codes are let go of only here, where the stores that need them are
                // done: after an arrival right behind the loads, the compiler may still
                // sink a load below it, into the slot's next filling (seen)
                mbar_arrive(raw_empty(rs));
                arrive_full(s);
            }
        }
    } else if (warp < C::kEpi) {
        // ------------------------------------------- tokens to shared memory --
        const int group = (warp - C::kBFirst) / C::kBWarps, bw = (warp - C::kBFirst) % C::kBWarps;
        // lane: 16 codes of one of four rows; eight neighbouring lanes hold 64 of K of two
        // rows, whose stores meet all banks once
        static_assert(C::kLanes == 8, "lanes of a row");
        const int sub = (lane & 3) + ((lane >> 4) << 2), row0 = bw * 4 + ((lane >> 2) & 3);
        const uint32_t at = b_base + (sub >> 2) * C::kSubBytes + row0 * 128;
        const uint32_t lo = at + (((2 * (sub & 3)) ^ (row0 & 7)) << 4), hi = at + (((2 * (sub & 3) + 1) ^ (row0 & 7)) << 4);
        const int8_t* q = a.q + sub * 16;
        // the stream of this group's units runs kAhead ahead, over the ends of tiles; a
        // warp lets go of a tile's table when it has read the next one
        int at_t = first_tile, at_u = group, at_n = 0, at_passes = 0;
        uint32_t src[C::kPasses];
        auto next_rows = [&]() {
            if (at_t >= tiles) return;
            const int i = at_n % C::kTabs;
            ok = __all_sync(kAll, wait_for<false>(tab_full(i), (at_n / C::kTabs) & 1, abort, a.wait_ns));
            if (!ok) return;
#pragma unroll
            for (int p = 0; p < C::kPasses; ++p) src[p] = token_at[i][p * C::kPass + row0];
            at_passes = token_passes[i];
            __syncwarp();
            if (lane == 0 && at_n > 0) mbar_arrive(tab_empty((at_n - 1) % C::kTabs));
        };
        auto to_tile = [&]() {  // (a tile may be shorter than the groups' turn)
            while (at_u >= units && at_t < tiles && ok) {
                at_u -= units;
                at_t += tile_step;
                ++at_n;
                next_rows();
            }
        };
        auto load = [&](uint4 (&v)[C::kPasses], int& passes) {
            if (at_t >= tiles || !ok) return;
            const int k = at_u * C::kUnit;
            passes = at_passes;
            const int8_t* at = q + k;
            if (k + C::kUnit <= a.K) {
#pragma unroll
                for (int i = 0; i < C::kPasses; ++i) ld_ahead(v[i], at + (uint64_t)src[i] * 16);
            } else {  // past K the weights are zeros, so the codes may be anything
#pragma unroll
                for (int i = 0; i < C::kPasses; ++i)
                    if (k + sub * 16 < a.K) ld_ahead(v[i], at + (uint64_t)src[i] * 16);
            }
            at_u += C::kBGroups;
            to_tile();
        };
        uint4 buf[C::kAhead][C::kPasses];
        int passes[C::kAhead];
        next_rows();
        to_tile();
#pragma unroll
        for (int j = 0; j < C::kAhead; ++j) load(buf[j], passes[j]);
        const int all_units = my_tiles * units;
        int g = group;
        while (g < all_units && ok) {
#pragma unroll
            for (int j = 0; j < C::kAhead; ++j) {
                if (g >= all_units || !ok) break;
                const int s = g % C::kSlots;
                ok = __all_sync(kAll, wait_for<kPair>(empty(s), ((g / C::kSlots) & 1) ^ 1, abort, a.wait_ns));
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < C::kPasses; ++i) {
                    if (i >= passes[j]) break;
                    uint32_t f[8];
                    codes_to_f16(buf[j][i].x, f[0], f[1]);
                    codes_to_f16(buf[j][i].y, f[2], f[3]);
                    codes_to_f16(buf[j][i].z, f[4], f[5]);
                    codes_to_f16(buf[j][i].w, f[6], f[7]);
                    const uint32_t to = s * C::kBBytes + i * C::kPass * 128;  // kPass % 8 == 0: the swizzle stays
                    st_shared16(lo + to, f[0], f[1], f[2], f[3]);
                    st_shared16(hi + to, f[4], f[5], f[6], f[7]);
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) arrive_full(s);
                load(buf[j], passes[j]);
                g += C::kBGroups;
            }
        }
    } else {
        // -------------------------------------------------------- epilogue --
        // warp e of the kEpiWarps: lanes (e % 4) * 32, every (kEpiWarps / 4)-th 32 columns
        constexpr int kParts = C::kEpiWarps / 4, kMine = kCap / 32 / kParts;
        const int ew = (warp - C::kEpi) & 3, part = (warp - C::kEpi) >> 2, et = tid - C::kEpi * 32;
        O* out = reinterpret_cast<O*>(a.out);
        const bool pairs = a.N % 2 == 0 && a.os % 2 == 0 && (uintptr_t)a.out % 4 == 0;
        for (long long p = begin[a.E] + (long long)blockIdx.x; p < a.R; p += gridDim.x)
            for (int n = et; n < a.N; n += 32 * C::kEpiWarps) out[p * a.os + n] = from_f32<O>(0.f);
        int n = 0;
        for (int t = first_tile; t < tiles && ok; t += tile_step, ++n) {
            const Tile w = tile_at(t);
            const int b = n % C::kBufs;
            const float* scale = token_scale[n % C::kTabs];
            const int ch = w.n0 + ew * 32 + lane;
            const float cs = ch < a.N ? a.w_scale[(long long)w.e * a.N + ch] : 0.f;
            ok = __all_sync(kAll, wait_for<false>(tab_full(n % C::kTabs), (n / C::kTabs) & 1, abort, a.wait_ns));
            if (!ok) break;
            ok = __all_sync(kAll, wait_for<kPair>(d_full(b), (n / C::kBufs) & 1, abort, a.wait_ns));
            if (!ok) break;
            tc_fence_after();
            O* dst = out + (long long)w.p0 * a.os + ch;
            const int last = (w.count - 1) / 32;  // the accumulator is free when its columns are in registers
            bool held = true;
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const int c0 = 32 * (i * kParts + part);
                if (c0 >= w.count) break;
                uint32_t v[32];
                const uint32_t acc = ((uint32_t)(ew * 32) << 16) + b * C::kAccs * kCap + c0;
                tmem_ld32(acc, v);
                if (C::kAccs == 2 && a.K > 16) {  // (of one step of K there is one accumulator only)
#pragma unroll
                    for (int h = 0; h < 32; h += 16) {
                        uint32_t v2[16];
                        tmem_ld16(acc + kCap + h, v2);
                        tmem_ld_wait();
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            v[h + c] = __float_as_uint(__uint_as_float(v[h + c]) + __uint_as_float(v2[c]));
                    }
                }
                tmem_ld_wait();
                if (i * kParts + part + kParts > last) {
                    release(b);
                    held = false;
                }
                const bool whole = c0 + 32 <= w.count && w.n0 + 128 <= a.N;
                if (sizeof(O) == 2 && pairs) {
                    // neighbouring lanes swap: the even one stores both channels of an even
                    // position, the odd one those of the next
                    const bool odd = lane & 1;
                    O* at = dst + (long long)(c0 + odd) * a.os - odd;
                    auto put = [&](int c, bool on) {
                        const float2 s = *reinterpret_cast<const float2*>(&scale[c0 + c]);
                        const float x = __uint_as_float(v[c]) * s.x * cs, y = __uint_as_float(v[c + 1]) * s.y * cs;
                        const float z = __shfl_xor_sync(kAll, odd ? x : y, 1);
                        const float f[2] = {odd ? z : x, odd ? y : z};
                        if (on) store_chunk<O, 2>(at, f);
                        at += 2 * a.os;
                    };
                    if (whole) {
#pragma unroll
                        for (int c = 0; c < 32; c += 2) put(c, true);
                    } else {
#pragma unroll
                        for (int c = 0; c < 32; c += 2) put(c, c0 + c + odd < w.count && ch < a.N);
                    }
                    continue;
                }
                O* at = dst + (long long)c0 * a.os;
                auto put = [&](int c, bool on) {
                    if (on) *at = from_f32<O>(__uint_as_float(v[c]) * scale[c0 + c] * cs);
                    at += a.os;
                };
                if (whole) {
#pragma unroll
                    for (int c = 0; c < 32; ++c) put(c, true);
                } else {
#pragma unroll
                    for (int c = 0; c < 32; ++c) put(c, c0 + c < w.count && ch < a.N);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(tab_empty(n % C::kTabs));
            if (held) release(b);
        }
    }
    if (!ok) {
        *abort = 1;
        raise_flag(&g_product_err, ERR_TIMEOUT);
        spin_ns(20000000ull);  // copies in flight land
    }
    tc_fence_before();
    __syncthreads();
    if (kPair) pair_sync();  // neither CTA leaves while the other may still reach it
    if (warp == C::kMma) {
        tc_fence_after();
        tmem_free_all<kPair>(tmem_slot);
    }
    if (kPair) pair_sync();
}

// Map over the codes of all experts, [rows][K]: boxes of 128 bytes x 128 rows, 128-byte swizzle.
bool map_weights(CUtensorMap* m, const int8_t* wq, uint64_t K, uint64_t rows) {
    using Encode = decltype(&cuTensorMapEncodeTiled);
    static const Encode encode = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e =
            cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found);
        return e == cudaSuccess && found == cudaDriverEntryPointSuccess ? reinterpret_cast<Encode>(p) : nullptr;
    }();
    if (!encode) return false;
    const cuuint64_t dims[2] = {K, rows}, strides[1] = {K};
    const cuuint32_t box[2] = {128, 128}, step[2] = {1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(wq), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// `most`: tiles at most; the grid is no larger than what runs at the same time.
template <bool kPair, typename O>
cudaError_t launch_kind(const Product& a, long long most, int dev, const CUtensorMap& map, cudaStream_t s) {
    using C = Cfg<kPair>;
    static std::mutex lock;
    static int fits[64] = {};  // tiles in flight, once looked up
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C::kCtas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    {
        std::lock_guard<std::mutex> hold(lock);
        n = dev < 64 ? fits[dev] : 0;
        if (!n) {
            cudaError_t e = cudaFuncSetAttribute(k_product_tc<kPair, O>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
            // (a pair needs two SMs of one cluster of them: not every SM finds a partner)
            cfg.gridDim = dim3(C::kCtas);
            if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, k_product_tc<kPair, O>, &cfg);
            if (e != cudaSuccess) return e;
            if (n < 1) return cudaErrorInvalidConfiguration;
            if (dev < 64) fits[dev] = n;
        }
    }
    cfg.gridDim = dim3((unsigned)(most < n ? most : n) * C::kCtas);
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_product_tc<kPair, O>, a, map);
}

template <typename O>
cudaError_t launch_o(const Product& a, const CUtensorMap& map, cudaStream_t s) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // Narrow or wide tiles, by rounds over the GPU times what a round takes.  A segment of
    // m positions has about m / cap + 1/2 tiles (those of the dense product are known) and
    // at least one.  Rounds measured at K = 4096: narrow 14.0 us with 12 positions a tile,
    // 15.3 with 31, 17.4 with 62; wide 15.6, 15.8 and 16.7, then 18.6 with 100, 20.4 with
    // 150, 22.6 with 200.  So 32 experts of 31 positions take 107 us narrow and 110 wide, of
    // 62 122 and 117, of 100 194 and 130; one of 256 19 and 27, of 512 32 and 28.
    // The segments themselves are on the device, and are taken as equal here: 3000 rows on 8
    // of 256 experts run narrow, at 146 us where the wide form takes 83.
    const double segs = a.E < a.R ? a.E : a.R;
    auto cost = [&](int cap, int channels, int at_once, double base, double a_row) {
        const double mean = a.R / segs, each = a.E == 1 ? (a.R + cap - 1) / cap : mean / cap + 0.5;
        const double n = each > 1 ? each : 1;
        return std::ceil(segs * n * ((a.N + channels - 1) / channels) / at_once) * (base + a_row * mean / n);
    };
    auto most = [&](int cap, int channels) {  // tiles
        return (a.R / cap + (long long)segs) * ((a.N + channels - 1) / channels);
    };
    if (cost(256, 256, sms / 2, 14.2, 0.042) < cost(64, 128, sms, 13.1, 0.068))
        return launch_kind<true, O>(a, most(256, 256), dev, map, s);
    return launch_kind<false, O>(a, most(64, 128), dev, map, s);
}

}  // namespace

cudaError_t product_flag(uint32_t* flag, cudaStream_t s) {
    static std::mutex lock;  // one check at a time: they share g_product_seen
    std::lock_guard<std::mutex> hold(lock);
    k_take_flag<<<1, 1, 0, s>>>();
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) e = cudaMemcpyFromSymbolAsync(flag, g_product_seen, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, s);
    const cudaError_t done = cudaStreamSynchronize(s);
    return e == cudaSuccess ? done : e;
}

bool product_tc_fits(const Product& a) {
    return a.rows > 0 && a.K % 16 == 0 && a.qs % 16 == 0 && a.rows * (a.qs / 16) < 0xFFFFFFFFLL && (uintptr_t)a.q % 16 == 0 && (uintptr_t)a.wq % 16 == 0;
}

cudaError_t launch_product_tc(const Product& a, moe_dtype out, cudaStream_t s) {
    CUtensorMap map;
    if (!map_weights(&map, a.wq, (uint64_t)a.K, (uint64_t)a.E * a.N)) return cudaErrorInvalidValue;
    if (out == MOE_F32) return launch_o<float>(a, map, s);
    if (out == MOE_BF16) return launch_o<__nv_bfloat16>(a, map, s);
    return launch_o<__half>(a, map, s);
}

}  // namespace moe
