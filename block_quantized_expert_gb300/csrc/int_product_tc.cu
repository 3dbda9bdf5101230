// int_product_tc.cu -- the product with 8-bit integer experts on the tensor
// cores (moe_expert_product).
//
// This part's tensor cores have no fast 8-bit integer form, but an 8-bit integer is
// exact in fp16, a product of two is exact in fp32 and so is a sum of them up
// to 2^24: the codes are turned into fp16 on the way to tcgen05.mma.kind::f16
// with fp32 accumulators.  A sum passes 2^24 only for K > 1024 and codes that
// nearly all are extreme and agree in sign; it is then rounded like any fp32 sum.
//
// One CTA per SM walks tiles of 128 output channels (A, one tensor-memory lane
// a channel) x up to kCap positions of one segment (B), K in units:
//   kAGroups warpgroups  codes of one channel a thread -> fp16 -> tensor memory
//                        (the A operand: it takes no shared-memory bandwidth from B)
//   kBGroups x 4 or 8    token codes: global -> registers, a few units ahead and
//   warps                across tiles -> fp16 -> shared memory, rows of 128 bytes,
//                        128-byte swizzle; a gather costs nothing here
//   4 warps              accumulators -> scales -> out, while the next tile is
//                        summed (two accumulators)
//   1 warp               TMA of 128 channels x 128 bytes of codes into a ring
//   1 warp               the MMAs (N = the tile's rows rounded to 16)
// The groups of one kind take the units in turn.
#include <cuda.h>

#include <mutex>

#include "int_product.cuh"
#include "tc_ptx.cuh"

namespace moe {

bool make_byte_map(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint32_t box_rows);

namespace {

using namespace tc;

constexpr int kRawBytes = 128 * 128;  // one ring slot of weight codes
constexpr uint64_t kWaitNs = 2000000000ull;

// Narrow tiles are bound by the stream of weights: long units (fewer waits a
// byte) and a long ring.  Wide ones are bound by the MMA: 192 positions are
// the most of which two accumulators and four units fit tensor memory.
template <int kCap_>
struct Cfg {
    static constexpr int kCap = kCap_;
    static constexpr bool kWide = kCap > 64;
    static constexpr int kUnit = kWide ? 64 : 128;         // K of one unit
    static constexpr int kSlots = 4;                       // units in flight to the MMA
    static constexpr int kRaw = kWide ? 4 : 8;             // weight ring
    static constexpr int kPerRaw = 128 / kUnit;            // units in one of its slots
    static constexpr int kAGroups = 2;
    static constexpr int kBGroups = 2;
    static constexpr int kBWarps = kWide ? 8 : 4;          // warps of one token group
    static constexpr int kLanes = kUnit / 16;              // lanes that share a token's unit
    static constexpr int kPass = kBWarps * 32 / kLanes;    // token rows a group moves at once
    static constexpr int kPasses = kCap / kPass;
    static constexpr int kAhead = kWide ? 1 : 2;           // units of token codes held in registers
    static constexpr int kSubBytes = kCap * 128;           // 64 of K of all tokens in fp16
    static constexpr int kBBytes = kSubBytes * (kUnit / 64);
    static constexpr int kACols = kUnit / 2;               // tensor-memory columns of one unit
    static constexpr int kACol = 512 - kACols * kSlots;
    static constexpr int kDCols = kCap;
    static constexpr int kBFirst = 4 * kAGroups;
    static constexpr int kEpi = kBFirst + kBGroups * kBWarps;  // first epilogue warp; then TMA, then MMA
    static constexpr int kThreads = (kEpi + 6) * 32;
    static constexpr int kSmem = 1024 + kSlots * kBBytes + kRaw * kRawBytes;
    static_assert(kCap % kPass == 0 && kCap % 32 == 0 && 2 * kDCols <= kACol, "tensor memory");
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
// cycles whatever N is; so it takes 60 for N <= 64 and N / 2 above (measured).
__device__ __forceinline__ void mma_f16_ts(uint32_t on, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(on)
        : "memory");
}

__device__ __forceinline__ void mma_commit_by(uint32_t on, uint32_t bar) {
    asm volatile(
        "{\n.reg .pred q;\nsetp.ne.b32 q, %1, 0;\n"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar), "r"(on)
        : "memory");
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

// 16 bytes, or zeros; volatile, so that it is issued here and not at its use.
__device__ __forceinline__ void ld_ahead(uint4& v, const int8_t* p, bool on) {
    asm volatile(
        "{\n.reg .pred q;\nsetp.ne.b32 q, %5, 0;\nmov.b32 %0, 0;\nmov.b32 %1, 0;\nmov.b32 %2, 0;\nmov.b32 %3, 0;\n"
        "@q ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w) : "l"(p), "r"((int)on));
}

__device__ __forceinline__ void st_shared16(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

struct Tile {
    int e, n0, p0, count;
};

__device__ uint32_t g_product_err;

template <int kCap, typename O>
__global__ void __launch_bounds__(Cfg<kCap>::kThreads, 1) k_product_tc(const Product a, const __grid_constant__ CUtensorMap wmap) {
    using C = Cfg<kCap>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[2 * C::kRaw + 2 * C::kSlots + 4];
    __shared__ int first[kMaxExperts + 1];  // token tiles before each expert
    __shared__ int begin[kMaxExperts + 1];  // its segment
    __shared__ int scan[32];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    constexpr unsigned kAll = 0xFFFFFFFFu;
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t b_base = base, raw_base = base + C::kSlots * C::kBBytes;
    const uint32_t bar0 = smem_u32(bars);
    auto raw_full = [&](int i) { return bar0 + 8u * i; };
    auto raw_empty = [&](int i) { return bar0 + 8u * (C::kRaw + i); };
    auto full = [&](int i) { return bar0 + 8u * (2 * C::kRaw + i); };
    auto empty = [&](int i) { return bar0 + 8u * (2 * C::kRaw + C::kSlots + i); };
    auto d_full = [&](int i) { return bar0 + 8u * (2 * C::kRaw + 2 * C::kSlots + i); };
    auto d_empty = [&](int i) { return bar0 + 8u * (2 * C::kRaw + 2 * C::kSlots + 2 + i); };
    volatile int* abort = &abort_flag;
    if (tid == 0) {
        for (int i = 0; i < C::kRaw; ++i) {
            mbar_init(raw_full(i), 1);
            mbar_init(raw_empty(i), 4 * C::kPerRaw);
        }
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(full(i), 4 + C::kBWarps);
            mbar_init(empty(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(d_full(i), 1);
            mbar_init(d_empty(i), 4);
        }
        abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&wmap);
    }
    // all 512 columns: they start at address 0, which the code below relies on
    if (warp == C::kEpi + 5) tmem_alloc(smem_u32(&tmem_slot), 512);
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
    tc_fence_after();
    const int m_tiles = (a.N + 127) / 128;
    const int tiles = first[a.E] * m_tiles;  // below 2^28: R <= 2^20, N <= 2^20 and m_tiles tiles a token tile
    const int units = (a.K + C::kUnit - 1) / C::kUnit;

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
        w.n0 = (t - tt * m_tiles) * 128;
        const int count = begin[lo + 1] - begin[lo], n = first[lo + 1] - first[lo];
        const int step = n < 8 ? ((count + n - 1) / n + 15) / 16 * 16 : kCap;  // at most kCap
        w.p0 = begin[lo] + (tt - first[lo]) * step;
        w.count = min(step, begin[lo + 1] - w.p0);
        return w;
    };
    bool ok = true;

    if (warp == C::kEpi + 4) {
        // ------------------------------------------------- weight codes (TMA) --
        if (lane == 0) {
            int i = 0;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const Tile w = tile_at(t);
                for (int k0 = 0; k0 < a.K; k0 += 128, ++i) {
                    const int s = i % C::kRaw;
                    ok = mbar_wait(raw_empty(s), ((i / C::kRaw) & 1) ^ 1, kWaitNs, abort);
                    if (!ok) break;
                    mbar_arrive_expect_tx(raw_full(s), kRawBytes);
                    tma_load_2d(raw_base + s * kRawBytes, &wmap, k0, w.e * a.N + w.n0, raw_full(s));
                }
            }
        }
    } else if (warp == C::kEpi + 5) {
        // ------------------------------------------------------------- MMA --
        const uint32_t on = elect_lane();
        int g = 0, n = 0;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++n) {
            const uint32_t cols = (tile_at(t).count + 15) / 16 * 16;
            const uint32_t idesc = (1u << 4) | ((cols >> 3) << 17) | ((128u >> 4) << 24);
            const int b = n & 1;
            const uint32_t d = b * C::kDCols;
            ok = __all_sync(kAll, mbar_wait(d_empty(b), ((n >> 1) & 1) ^ 1, kWaitNs, abort));
            tc_fence_after();
            for (int u = 0; u < units && ok; ++u, ++g) {
                const int s = g % C::kSlots;
                ok = __all_sync(kAll, mbar_wait(full(s), (g / C::kSlots) & 1, kWaitNs, abort));
                if (!ok) break;
                // the loaders' stores, seen through the barrier, before the MMA's own reads; the
                // fence stands here because there it would wait for the loads that run ahead
                fence_async_shared();
                tc_fence_after();
                const uint64_t bd = desc_sw128(b_base + s * C::kBBytes);
                const uint32_t ad = C::kACol + s * C::kACols;
                if (a.K - u * C::kUnit >= C::kUnit) {
#pragma unroll
                    for (int i = 0; i < C::kUnit / 16; ++i)
                        mma_f16_ts(on, d, ad + i * 8, bd + (uint64_t)((i >> 2) * (C::kSubBytes >> 4) + (i & 3) * 2), idesc,
                                   (u | i) != 0);
                } else {
                    for (int i = 0; i < (a.K - u * C::kUnit + 15) / 16; ++i)
                        mma_f16_ts(on, d, ad + i * 8, bd + (uint64_t)((i >> 2) * (C::kSubBytes >> 4) + (i & 3) * 2), idesc,
                                   (u | i) != 0);
                }
                mma_commit_by(on, empty(s));
            }
            if (ok) mma_commit_by(on, d_full(b));
        }
    } else if (warp < C::kBFirst) {
        // --------------------------------------------- weights to tensor memory --
        // (with two units a ring slot, each of them frees half of it)
        const int lanes = (warp & 3) * 32, r = lanes + lane, group = warp >> 2;
        const uint32_t lane_at = (uint32_t)lanes << 16;
        int i0 = 0, g0 = 0;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x, i0 += (units + C::kPerRaw - 1) / C::kPerRaw, g0 += units) {
            for (int u = group; u < units; u += C::kAGroups) {
                const int i = i0 + u / C::kPerRaw, rs = i % C::kRaw, g = g0 + u, s = g % C::kSlots;
                const int part = u % C::kPerRaw;
                ok = __all_sync(kAll, mbar_wait(raw_full(rs), (i / C::kRaw) & 1, kWaitNs, abort));
                if (!ok) break;
                const uint32_t row = raw_base + rs * kRawBytes + r * 128;
                uint4 v[C::kUnit / 16];
#pragma unroll
                for (int c = 0; c < C::kUnit / 16; ++c)
                    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(v[c].x), "=r"(v[c].y), "=r"(v[c].z), "=r"(v[c].w)
                                 : "r"(row + (((C::kUnit / 16 * part + c) ^ (r & 7)) << 4)));
#pragma unroll
                for (int h = 0; h < C::kUnit / 64; ++h) {
                    uint32_t f[32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        codes_to_f16(v[4 * h + c].x, f[8 * c], f[8 * c + 1]);
                        codes_to_f16(v[4 * h + c].y, f[8 * c + 2], f[8 * c + 3]);
                        codes_to_f16(v[4 * h + c].z, f[8 * c + 4], f[8 * c + 5]);
                        codes_to_f16(v[4 * h + c].w, f[8 * c + 6], f[8 * c + 7]);
                    }
                    if (h == 0) {
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(raw_empty(rs));
                            if (C::kPerRaw == 2 && u == units - 1 && part == 0) mbar_arrive(raw_empty(rs));  // no second unit
                        }
                        ok = __all_sync(kAll, mbar_wait(empty(s), ((g / C::kSlots) & 1) ^ 1, kWaitNs, abort));
                        if (!ok) break;
                        tc_fence_after();
                    }
                    tmem_st32(lane_at + C::kACol + s * C::kACols + 32 * h, f);
                }
                if (!ok) break;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(full(s));
            }
        }
    } else if (warp < C::kEpi) {
        // ------------------------------------------- tokens to shared memory --
        const int group = (warp - C::kBFirst) / C::kBWarps, bw = (warp - C::kBFirst) % C::kBWarps;
        const int sub = lane % C::kLanes, row0 = bw * (32 / C::kLanes) + lane / C::kLanes;
        // where lane's 16 codes of row row0 go: two 16-byte pieces, in an order that
        // keeps the eight lanes of a store on eight banks
        const uint32_t at = b_base + (sub >> 2) * C::kSubBytes + row0 * 128;
        const uint32_t lo = at + (((2 * (sub & 3)) ^ (row0 & 7)) << 4), hi = at + (((2 * (sub & 3) + 1) ^ (row0 & 7)) << 4);
        const bool odd = sub >= 4;
        // the stream of this group's units runs kAhead ahead, over the ends of tiles
        int at_t = blockIdx.x, at_u = group;
        const int8_t* src[C::kPasses];
        auto rows_of = [&](int t) {
            if (t >= tiles) return;
            const Tile w = tile_at(t);
#pragma unroll
            for (int i = 0; i < C::kPasses; ++i) {
                const int row = i * C::kPass + row0;
                const int r = row < w.count ? source_row(a, w.p0 + row) : -1;
                src[i] = r >= 0 ? a.q + (long long)r * a.qs + sub * 16 : nullptr;
            }
        };
        auto load = [&](uint4 (&v)[C::kPasses]) {
            if (at_t >= tiles) return;
            const int k = at_u * C::kUnit;
#pragma unroll
            for (int i = 0; i < C::kPasses; ++i) ld_ahead(v[i], src[i] + k, src[i] != nullptr && k + sub * 16 < a.K);
            at_u += C::kBGroups;
            if (at_u >= units) {
                at_u = group;
                at_t += gridDim.x;
                rows_of(at_t);
            }
        };
        if (group < units) {
            uint4 buf[C::kAhead][C::kPasses];
            rows_of(at_t);
#pragma unroll
            for (int j = 0; j < C::kAhead; ++j) load(buf[j]);
            int t = blockIdx.x, u = group, g0 = 0;
            int passes = t < tiles ? (tile_at(t).count + C::kPass - 1) / C::kPass : 0;
            while (t < tiles && ok) {
#pragma unroll
                for (int j = 0; j < C::kAhead; ++j) {
                    if (t >= tiles || !ok) break;
                    const int g = g0 + u, s = g % C::kSlots;
                    ok = __all_sync(kAll, mbar_wait(empty(s), ((g / C::kSlots) & 1) ^ 1, kWaitNs, abort));
                    if (!ok) break;
#pragma unroll
                    for (int i = 0; i < C::kPasses; ++i) {
                        if (i >= passes) break;
                        uint32_t f[8];
                        codes_to_f16(buf[j][i].x, f[0], f[1]);
                        codes_to_f16(buf[j][i].y, f[2], f[3]);
                        codes_to_f16(buf[j][i].z, f[4], f[5]);
                        codes_to_f16(buf[j][i].w, f[6], f[7]);
                        const uint32_t to = s * C::kBBytes + i * C::kPass * 128;  // kPass % 8 == 0: the swizzle stays
                        st_shared16((odd ? hi : lo) + to, odd ? f[4] : f[0], odd ? f[5] : f[1], odd ? f[6] : f[2],
                                    odd ? f[7] : f[3]);
                        st_shared16((odd ? lo : hi) + to, odd ? f[0] : f[4], odd ? f[1] : f[5], odd ? f[2] : f[6],
                                    odd ? f[3] : f[7]);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full(s));
                    load(buf[j]);
                    u += C::kBGroups;
                    if (u >= units) {
                        u = group;
                        t += gridDim.x;
                        g0 += units;
                        if (t < tiles) passes = (tile_at(t).count + C::kPass - 1) / C::kPass;
                    }
                }
            }
        }
    } else {
        // -------------------------------------------------------- epilogue --
        const int ew = warp - C::kEpi, et = tid - C::kEpi * 32;
        O* out = reinterpret_cast<O*>(a.out);
        for (long long p = begin[a.E] + (long long)blockIdx.x; p < a.R; p += gridDim.x)
            for (int n = et; n < a.N; n += 128) out[p * a.os + n] = from_f32<O>(0.f);
        int n = 0;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++n) {
            const Tile w = tile_at(t);
            const int b = n & 1;
            float rs[kCap / 32];  // lane i: scale of rows i, 32 + i, ...
#pragma unroll
            for (int i = 0; i < kCap / 32; ++i) {
                const int c = 32 * i + lane, r = c < w.count ? source_row(a, w.p0 + c) : -1;
                rs[i] = r >= 0 ? a.scale[r] : 0.f;
            }
            const int ch = w.n0 + ew * 32 + lane;
            const float cs = ch < a.N ? a.w_scale[(long long)w.e * a.N + ch] : 0.f;
            ok = __all_sync(kAll, mbar_wait(d_full(b), (n >> 1) & 1, kWaitNs, abort));
            if (!ok) break;
            tc_fence_after();
            O* dst = out + (long long)w.p0 * a.os + ch;
#pragma unroll
            for (int i = 0; i < kCap / 32; ++i) {
                const int c0 = 32 * i;
                if (c0 >= w.count) break;
                uint32_t v[32];
                tmem_ld32(((uint32_t)(ew * 32) << 16) + b * C::kDCols + c0, v);
                tmem_ld_wait();
                if (c0 + 32 >= w.count) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(d_empty(b));
                }
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const float s = __shfl_sync(kAll, rs[i], c);
                    if (c0 + c < w.count && ch < a.N)
                        dst[(long long)(c0 + c) * a.os] = from_f32<O>(__uint_as_float(v[c]) * s * cs);
                }
            }
        }
    }
    if (!ok) {
        *abort = 1;
        raise_flag(&g_product_err, ERR_TIMEOUT);
        spin_ns(20000000ull);  // copies in flight land
    }
    tc_fence_before();
    __syncthreads();
    if (warp == C::kEpi + 5) {
        tc_fence_after();
        tmem_dealloc(tmem_slot, 512);
    }
}

template <int kCap, typename O>
cudaError_t launch_cap(const Product& a, int grid, const CUtensorMap& map, cudaStream_t s) {
    static std::mutex lock;
    static bool ready[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> hold(lock);
        if (dev >= 64 || !ready[dev]) {
            e = cudaFuncSetAttribute(k_product_tc<kCap, O>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<kCap>::kSmem);
            if (e != cudaSuccess) return e;
            if (dev < 64) ready[dev] = true;
        }
    }
    return launch_pdl(k_product_tc<kCap, O>, dim3(grid), dim3(Cfg<kCap>::kThreads), Cfg<kCap>::kSmem, s, a, map);
}

template <typename O>
cudaError_t launch_o(const Product& a, const CUtensorMap& map, cudaStream_t s) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const long long most = ((long long)a.R / 64 + (a.E < a.R ? a.E : a.R)) * ((a.N + 127) / 128);  // tiles, at most
    const int grid = (int)(most < sms ? most : sms);
    // Few rows an expert: short accumulators and a longer ring of weights.
    return (long long)a.R <= 40LL * a.E ? launch_cap<64, O>(a, grid, map, s) : launch_cap<192, O>(a, grid, map, s);
}

}  // namespace

bool product_tc_fits(const Product& a) {
    return a.K % 16 == 0 && a.qs % 16 == 0 && (uintptr_t)a.q % 16 == 0 && (uintptr_t)a.wq % 16 == 0;
}

cudaError_t launch_product_tc(const Product& a, moe_dtype out, cudaStream_t s) {
    CUtensorMap map;
    if (!make_byte_map(&map, a.wq, (uint64_t)a.K, (uint64_t)a.E * a.N, 128)) return cudaErrorInvalidValue;
    if (out == MOE_F32) return launch_o<float>(a, map, s);
    if (out == MOE_BF16) return launch_o<__nv_bfloat16>(a, map, s);
    return launch_o<__half>(a, map, s);
}

}  // namespace moe
