// block_product_tc.cu -- the product of rows and experts in blocks of 4-bit codes on
// the tensor cores (moe_block_product): tcgen05.mma.kind::mxf4nvf4 (e4m3 scales of 16
// elements) and kind::mxf4 (UE8M0 scales of 32), fp32 accumulators.
//
// A CTA (or a pair of CTAs on one MMA, cta_group::2) walks tiles of 128 (256) output
// channels (A, one tensor-memory lane a channel) x up to kCap positions of one
// segment (B), K in units of 256, 128 bytes of codes a row:
//   4 or 6 warps  TMA, in four or two teams that take units in turn: a box of 128 channels'
//                 codes, and the positions' rows, four at a time by row_src (tile::gather4) or 16
//                 where positions are rows.  A lane issues a copy in some 130 cycles and
//                 a unit's wait, expectation and copies follow each other, so one warp's copies took 2.2
//                 times as long, and all six on each unit 584 us for 549 (49152 rows below)
//   4 warps       block scales of both sides, from their rows in global memory through
//                 registers into the 512-byte atoms that tcgen05.cp takes to tensor memory, in
//                 batches of 64 bytes a row (in pieces of a unit, 16 bytes, 708 us for 667, in
//                 sectors by one lane a row 656 for 620; two batches of 32 bytes in flight 646
//                 for 549, two of 64 in the narrow form 346 for 332)
//   1 warp        the copies of the scales and the MMAs, four of K = 64 a unit
//   4 warps       accumulators -> row and channel scales -> out, two accumulators in turn
//   1 warp        rows and row scales of up to kTabs tiles ahead
//
// Measured at K = N = 4096, bf16 out, the copy rate being 6.78 TB/s: 3000 rows over some 234 of
// 256 experts 312 us in MXFP4, 332 in NVFP4, 6.8 and 6.7 TB/s; 49152 rows over 256 experts 514 and
// 549 us, 3.2 and 3.0 PFLOP/s; 8192 rows of one expert 53 and 63 us, 5.2 and 4.4 PFLOP/s (what the tensor cores
// give in fp4 is not measured here; 13.5 is the nominal rate).
// The narrow form is bound by the stream of weights; six rows of six experts (16 us) are two
// rounds of tiles, each some 5 us whatever a tile's height (of 64 channels 20 us in all, of
// 32 33), of which the scales' loads are 0.5, the MMAs 0.2 and the copies' issue 0.5.
// The wide one has no single bound left: without the weights' boxes 49152 rows take 9 to 17 %
// less, without the scales' loads 4 to 7, without the stores 4 to 7, with one MMA of four 4.
#include <cuda.h>

#include <cmath>
#include <mutex>

#include "block_product.cuh"
#include "tc_pair.cuh"

namespace moe {

namespace {

using namespace tc;

template <bool kPair_, bool kNv_>
struct Cfg {
    static constexpr bool kPair = kPair_, kNv = kNv_;
    static constexpr int kCtas = kPair ? 2 : 1;
    static constexpr int kCap = kPair ? 224 : 64;        // positions of a tile
    static constexpr int kRows = kCap / kCtas;           // of them in this CTA's shared memory
    static constexpr int kUnit = 256;                    // K of one unit
    static constexpr int kABytes = 128 * 128;
    static constexpr int kBBytes = kRows * 128;
    static constexpr int kWords = kNv ? 4 : 2;           // 4-byte words of a row's scales of a unit: an atom each
    static constexpr int kHalves = (kCap + 127) / 128;   // 128-row parts of the positions' scales
    static constexpr int kStage = kABytes + kBBytes;
    static constexpr int kStages = kPair ? 5 : 7;
    // Scales come in batches of 64 bytes a row, four units or eight; the units of two batches
    // lie apart by a few banks more than their atoms, so that the stores of one row's meet
    // other banks.
    static constexpr int kBatch = 16 / kWords, kSfBufs = 2;
    static constexpr int kSfStride = kWords * (1 + kHalves) * 512 + 8 * kWords;
    static constexpr int kTabs = 4;                      // tiles whose rows are looked up
    static constexpr int kSfCol = 2 * kCap;              // tensor memory: two accumulators, scales
    static constexpr int kSfA = 4 * kWords, kSfB = 4 * kWords * kHalves;
    static constexpr int kSfWarps = 4, kEpiWarps = 4;
    static constexpr int kEpi = kSfWarps;                // warps: scales, epilogue, TMA, MMA, rows
    static constexpr int kTmaWarps = kPair ? 6 : 4, kTeams = kPair ? 2 : 4;  // teams take units in turn
    static constexpr int kPer = kTmaWarps / kTeams, kGroups = (kRows / 4 + kPer - 1) / kPer;  // warps of a team, copies of a warp
    static constexpr int kTma = kEpi + kEpiWarps, kMma = kTma + kTmaWarps, kLook = kMma + 1;
    static constexpr int kThreads = (kLook + 1) * 32;
    static constexpr int kSmem = 1024 + kStages * kStage + kSfBufs * kBatch * kSfStride;
    static_assert(kSfCol + kSfA + kSfB <= 512 && kCap % (16 * kCtas) == 0 && kBBytes % 1024 == 0, "tensor memory");
    static_assert(kSfWarps == 4 && kTeams <= kStages && kTmaWarps % kTeams == 0 && kGroups <= 32, "roles");
};

// D[tmem] (+)= (A sfa)(B sfb)^T over K = 64, both operands in shared memory; issued
// by the lane with `on` (under an `if` on the lane the operands are not uniform and an issue
// takes far longer).
template <bool kPair, bool kNv>
__device__ __forceinline__ void mma_fp4(uint32_t on, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate) {
#define MOE_MMA_FP4(group, kind)                                                                          \
    asm volatile(                                                                                         \
        "{\n.reg .pred p, q;\nsetp.ne.b32 p, %6, 0;\nsetp.ne.b32 q, %7, 0;\n"                             \
        "@q tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, [%4], [%5], p;\n}"          \
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(on)                \
        : "memory")
    if (kPair && kNv) MOE_MMA_FP4("2", "mxf4nvf4.block_scale.scale_vec::4X");
    if (kPair && !kNv) MOE_MMA_FP4("2", "mxf4.block_scale.scale_vec::2X");
    if (!kPair && kNv) MOE_MMA_FP4("1", "mxf4nvf4.block_scale.scale_vec::4X");
    if (!kPair && !kNv) MOE_MMA_FP4("1", "mxf4.block_scale.scale_vec::2X");
#undef MOE_MMA_FP4
}

// 512 bytes (32 lanes x 16) into four columns, replicated into the four lane quarters; in
// a pair both CTAs copy from their own shared memory.
template <bool kPair>
__device__ __forceinline__ void copy_scales(uint32_t on, uint32_t col, uint64_t desc) {
    if (kPair)
        asm volatile("{\n.reg .pred q;\nsetp.ne.b32 q, %2, 0;\n@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n}"
                     ::"r"(col), "l"(desc), "r"(on) : "memory");
    else
        asm volatile("{\n.reg .pred q;\nsetp.ne.b32 q, %2, 0;\n@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n}"
                     ::"r"(col), "l"(desc), "r"(on) : "memory");
}

// A box of the map, and four rows of one, 128 bytes of each from byte x, into this CTA's
// shared memory; the bytes count on `bar`, which for a pair is the first CTA's.  A row
// past the map reads as zeros.
template <bool kPair>
__device__ __forceinline__ void load_box(uint32_t dst, const void* map, int x, int y, uint32_t bar) {
    if (kPair)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
    else
        tma_load_2d(dst, map, x, y, bar);
}

template <bool kPair>
__device__ __forceinline__ void gather_rows(uint32_t dst, const void* map, int x, int4 y, uint32_t bar) {
    if (kPair)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
            ::"r"(dst), "l"(map), "r"(x), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w), "r"(bar) : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
            ::"r"(dst), "l"(map), "r"(x), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w), "r"(bar) : "memory");
}

// The address of the pair's first CTA's shared memory at the same place.
__device__ __forceinline__ uint32_t in_first(uint32_t at) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(at));
    return r;
}

__device__ __forceinline__ void arrive_expect_in(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void st_shared4(uint32_t at, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

struct Tile {
    int e, n0, p0, count;
};

__device__ uint32_t g_block_err;   // sticky, taken by moe_check_product

// 16 scale bytes of one row from byte `at` on, zeros from byte `all` on: no row (nullptr)
// is all zeros.  bytes: 16, 4 or 2 where every row's pieces of that size are whole and aligned.
// Small pieces cost: six of 64 experts for each of 500 and of 8192 tokens, N = 2880, MXFP4, 47.5 and 200 us at
// K = 2560 (80 bytes a row), 53 and 240 at 2816 (88, in fours), 96 and 496 at 2880 (90, in twos).
__device__ __forceinline__ void load_scales(uint32_t (&w)[4], const uint8_t* row, int at, int all, int bytes) {
    w[0] = w[1] = w[2] = w[3] = 0;
    if (row == nullptr || at >= all) return;
    row += at;
    if (bytes == 16) {
        asm volatile("ld.global.L2::256B.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(row));
        return;
    }
    const int n = all - at;
    if (bytes == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (4 * i < n) w[i] = *reinterpret_cast<const uint32_t*>(row + 4 * i);
        return;
    }
    if (bytes == 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (2 * i < n) w[i / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(row + 2 * i) << (16 * (i & 1));
        return;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < n) w[i / 4] |= (uint32_t)row[i] << (8 * (i & 3));
}

template <bool kPair, bool kNv, typename O>
__global__ void __launch_bounds__(Cfg<kPair, kNv>::kThreads, 1)
    k_block_product_tc(const BlockProduct a, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap qmap) {
    using C = Cfg<kPair, kNv>;
    constexpr int kCap = C::kCap, kSpan = kNv ? 16 : 32;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[2 * C::kStages + 2 * C::kSfBufs + 4 + 2 * C::kTabs];
    __shared__ __align__(16) int token_row[C::kTabs][kCap];  // rows of q, or `none`
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
    const int none = max(a.rows, 1);              // a row past the map of q: zeros
    const int first_tile = blockIdx.x / C::kCtas, tile_step = gridDim.x / C::kCtas;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sf_base = base + C::kStages * C::kStage;
    const uint32_t bar0 = smem_u32(bars);
    // (of a pair the first CTA's are used)
    auto landed = [&](int i) { return bar0 + 8u * i; };                     // codes
    auto empty = [&](int i) { return bar0 + 8u * (C::kStages + i); };
    auto scaled = [&](int i) { return bar0 + 8u * (2 * C::kStages + i); };  // a batch of scales
    auto sf_empty = [&](int i) { return bar0 + 8u * (2 * C::kStages + C::kSfBufs + i); };
    constexpr int kOther = 2 * (C::kStages + C::kSfBufs);
    auto d_full = [&](int i) { return bar0 + 8u * (kOther + i); };
    auto d_empty = [&](int i) { return bar0 + 8u * (kOther + 2 + i); };
    auto tab_full = [&](int i) { return bar0 + 8u * (kOther + 4 + i); };
    auto tab_empty = [&](int i) { return bar0 + 8u * (kOther + 4 + C::kTabs + i); };
    volatile int* abort = &abort_flag;
    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(landed(i), C::kCtas);
            mbar_init(empty(i), 1);
        }
        for (int i = 0; i < C::kSfBufs; ++i) {
            mbar_init(scaled(i), C::kCtas * C::kSfWarps);
            mbar_init(sf_empty(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(d_full(i), 1);
            mbar_init(d_empty(i), C::kCtas * C::kEpiWarps);
        }
        for (int i = 0; i < C::kTabs; ++i) {
            mbar_init(tab_full(i), 1);
            mbar_init(tab_empty(i), C::kTmaWarps + C::kSfWarps + C::kEpiWarps);
        }
        abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&wmap);
        prefetch_tmap(&qmap);
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
    auto release = [&](int b) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            if (kPair) mbar_arrive_first(d_empty(b)); else mbar_arrive(d_empty(b));
        }
    };
    auto leave_tab = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(tab_empty(i));
    };
    bool ok = true;

    if (warp >= C::kTma && warp < C::kTma + C::kTmaWarps) {
        // ------------------------------------------------------ codes (TMA) --
        // A team's first warp brings the weights; the positions' rows, four a copy, are shared out
        // over its warps.
        const int team = (warp - C::kTma) / C::kPer, part = (warp - C::kTma) % C::kPer;
        const int group = lane * C::kPer + part, units = (a.K + C::kUnit - 1) / C::kUnit;
        const bool boxes = a.row_src == nullptr;  // the map's are 16 rows then
        int s = team, next = team, n = 0;  // next: unit of this team, counted from the tile's first
        uint32_t phase = 1;
        for (int t = first_tile; t < tiles && ok; t += tile_step, ++n) {
            const Tile w = tile_at(t);
            const int tab = n % C::kTabs, half = columns(w.count) / C::kCtas;
            ok = __all_sync(kAll, wait_for<false>(tab_full(tab), (n / C::kTabs) & 1, abort, a.wait_ns));
            if (!ok) break;
            const bool mine = !boxes && lane < C::kGroups && 4 * group < half, box = boxes && 16 * group < half;
            int4 y = make_int4(none, none, none, none);
            if (mine) y = *reinterpret_cast<const int4*>(&token_row[tab][rank * half + 4 * group]);
            leave_tab(tab);
            for (; next < units && ok; next += C::kTeams) {
                ok = __all_sync(kAll, wait_for<kPair>(empty(s), phase, abort, a.wait_ns));
                if (!ok) break;
                const int su = __reduce_max_sync(kAll, s), x = next * (C::kUnit / 2);
                const uint32_t st = base + su * C::kStage, bar = kPair ? in_first(landed(su)) : landed(su);
                if (part == 0 && lane == 0) {
                    if (kPair) arrive_expect_in(bar, C::kABytes + half * 128);
                    else mbar_arrive_expect_tx(bar, C::kABytes + half * 128);
                    if (!a.stall) load_box<kPair>(st, &wmap, x, w.e * a.N + w.n0, bar);
                }
                __syncwarp();
                if (mine) gather_rows<kPair>(st + C::kABytes + group * 512, &qmap, x, y, bar);
                if (box) load_box<kPair>(st + C::kABytes + group * 2048, &qmap, x, w.p0 + rank * half + 16 * group, bar);
                s += C::kTeams;
                if (s >= C::kStages) {
                    s -= C::kStages;
                    phase ^= 1;
                }
            }
            next -= units;
        }
    } else if (warp == C::kLook) {
        // --------------------------------------- rows and scales of the tiles --
        int n = 0;
        for (int t = first_tile; t < tiles && ok; t += tile_step, ++n) {
            const Tile w = tile_at(t);
            const int i = n % C::kTabs;
            ok = __all_sync(kAll, wait_for<false>(tab_empty(i), ((n / C::kTabs) & 1) ^ 1, abort, a.wait_ns));
            if (!ok) break;
            for (int c = lane; c < kCap; c += 32) {
                const int r = c < w.count ? source_row(a, w.p0 + c) : -1;
                token_scale[i][c] = r < 0 ? 0.f : a.scale ? a.scale[r] : 1.f;
                token_row[i][c] = r < 0 ? none : r;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(tab_full(i));
        }
    } else if (warp == C::kMma) {
        // ------------------------------------------------------------- MMA --
        // (the first CTA of a pair issues for both)
        // The loops run by values that the compiler knows to be uniform over the warp (kernel
        // arguments and reductions; what comes from memory is not), so that stages' addresses are,
        // and the next unit is looked for between this one's issues: a wait, its vote and fence
        // take longer than the MMAs of a few positions.
        const uint32_t on = elect_lane();
        const int mine = __reduce_max_sync(kAll, rank == 0 && first_tile < tiles ? (tiles - first_tile + tile_step - 1) / tile_step : 0);
        const int units = (a.K + C::kUnit - 1) / C::kUnit;
        int s = 0, buf = 0;  // stage, buffer of scales
        uint32_t phase = 0, sf_phase = 0;
        bool ready = false;    // stage s has been seen
        for (int n = 0; n < mine && ok; ++n) {
            const uint32_t cols = __reduce_max_sync(kAll, columns(tile_at(first_tile + n * tile_step).count));
            // e2m1 both, N >> 3, UE8M0 scales: bit 23, M >> 4
            const uint32_t idesc = (1u << 7) | (1u << 10) | ((cols >> 3) << 17) | ((kNv ? 0u : 1u) << 23) | ((128u * C::kCtas >> 4) << 24);
            const int b = n & 1;
            const uint32_t d = b * kCap;
            ok = __all_sync(kAll, wait_for<kPair>(d_empty(b), ((n >> 1) & 1) ^ 1, abort, a.wait_ns));
            tc_fence_after();
            int unit = 0;  // of the batch
            for (int u = 0; u < units && ok; ++u) {
                if (unit == 0) ok = __all_sync(kAll, wait_for<kPair>(scaled(buf), sf_phase, abort, a.wait_ns));
                if (!ready) ok = ok && __all_sync(kAll, wait_for<kPair>(landed(s), phase, abort, a.wait_ns));
                if (!ok) break;
                tc_fence_after();
                const uint32_t st = base + s * C::kStage, sf = sf_base + (buf * C::kBatch + unit) * C::kSfStride, done = empty(s);
                const uint64_t ad = desc_sw128(st), bd = desc_sw128(st + C::kABytes), fd = desc_sf(sf);
                const int steps = min(a.K - u * C::kUnit + 63, 256) / 64;
                if (++s == C::kStages) {
                    s = 0;
                    phase ^= 1;
                }
                const bool seen = test_wait<kPair>(landed(s), phase);
#pragma unroll
                for (int j = 0; j < C::kWords; ++j) {
                    copy_scales<kPair>(on, C::kSfCol + 4 * j, fd + 32 * j);
#pragma unroll
                    for (int h = 0; h < C::kHalves; ++h)
                        if (h == 0 || cols > 128)
                            copy_scales<kPair>(on, C::kSfCol + C::kSfA + 4 * (j * C::kHalves + h),
                                               fd + 32 * (C::kWords * (1 + h) + j));
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j >= steps) break;
                    const int word = kNv ? j : j / 2;
                    const uint32_t id = kNv ? 0u : (j & 1) * 2u;  // which half of a word's bytes
                    mma_fp4<kPair, kNv>(on, d, ad + 2 * j, bd + 2 * j, idesc | (id << 4) | (id << 29), C::kSfCol + 4 * word,
                                        C::kSfCol + C::kSfA + 4 * word * C::kHalves, j > 0 || u > 0);
                }
                mma_commit_by<kPair>(on, done);
                if (++unit == C::kBatch || u == units - 1) {
                    mma_commit_by<kPair>(on, sf_empty(buf));
                    unit = 0;
                    if (++buf == C::kSfBufs) {
                        buf = 0;
                        sf_phase ^= 1;
                    }
                }
                ready = __all_sync(kAll, seen);
            }
            if (ok) mma_commit_by<kPair>(on, d_full(b));
        }
    } else if (warp < C::kSfWarps) {
        // ---------------------------------------------------- block scales --
        // Four neighbouring lanes hold 64 bytes of one row, a batch: whole sectors, and stores
        // that meet all banks once.  A warp's eight rows are r, r + 32, .. and r + 1, r + 33, ..
        // of 128, four such eights a warp, of the channels and of each half of the positions.
        constexpr int kParts = 1 + C::kHalves;
        const int piece = lane & 3, r0 = ((lane >> 2) & 3) * 32 + (lane >> 4) + 2 * warp;
        const int blocks = a.K / kSpan;
        const uintptr_t low = (uintptr_t)a.s | (uintptr_t)a.ws | (uintptr_t)blocks;
        const int bytes = low % 16 == 0 ? 16 : low % 4 == 0 ? 4 : low % 2 == 0 ? 2 : 1;
        uint32_t v[kParts][4][4];
        const uint8_t* rows[kParts][4];
        int at_t = first_tile, at_b = 0, at_n = 0;
        // the loads run a batch ahead of the stores, over the ends of tiles
        auto load = [&]() {
            if (at_t >= tiles || !ok) return;
            if (at_b == 0) {
                const Tile w = tile_at(at_t);
                const int tab = at_n % C::kTabs;
                ok = __all_sync(kAll, wait_for<false>(tab_full(tab), (at_n / C::kTabs) & 1, abort, a.wait_ns));
                if (!ok) return;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = r0 + 8 * i;
                    rows[0][i] = w.n0 + r < a.N ? a.ws + ((long long)w.e * a.N + w.n0 + r) * blocks : nullptr;
#pragma unroll
                    for (int h = 0; h < C::kHalves; ++h) {
                        const int src = r + 128 * h < kCap ? token_row[tab][r + 128 * h] : none;
                        rows[1 + h][i] = src != none ? a.s + (long long)src * blocks : nullptr;
                    }
                }
                leave_tab(tab);
            }
#pragma unroll
            for (int p = 0; p < kParts; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i) load_scales(v[p][i], rows[p][i], at_b + 16 * piece, blocks, bytes);
            at_b += 64;
            if (at_b >= blocks) {
                at_b = 0;
                at_t += tile_step;
                ++at_n;
            }
        };
        int buf = 0;
        uint32_t phase = 1;
        load();
        const int all = first_tile < tiles ? (tiles - first_tile + tile_step - 1) / tile_step * ((blocks + 63) / 64) : 0;
        for (int batch = 0; batch < all && ok; ++batch) {
            ok = __all_sync(kAll, wait_for<kPair>(sf_empty(buf), phase, abort, a.wait_ns));
            if (!ok) break;
            const uint32_t to = sf_base + buf * C::kBatch * C::kSfStride + (r0 & 31) * 16 + (r0 >> 5) * 4;
#pragma unroll
            for (int p = 0; p < kParts; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int unit = piece * (4 / C::kWords) + j / C::kWords;
                        st_shared4(to + unit * C::kSfStride + (p * C::kWords + j % C::kWords) * 512 + i * 128, v[p][i][j]);
                    }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) {
                if (kPair) mbar_arrive_first(scaled(buf)); else mbar_arrive(scaled(buf));
            }
            if (++buf == C::kSfBufs) {
                buf = 0;
                phase ^= 1;
            }
            load();
        }
    } else {
        // -------------------------------------------------------- epilogue --
        const int ew = warp - C::kEpi, et = tid - C::kEpi * 32;  // ew: lanes 32 ew .. of tensor memory
        static_assert(C::kEpi % 4 == 0 && C::kEpiWarps == 4, "a warp reads its own quarter of the lanes");
        O* out = reinterpret_cast<O*>(a.out);
        const bool pairs = a.N % 2 == 0 && a.os % 2 == 0 && (uintptr_t)a.out % 4 == 0;
        for (long long p = begin[a.E] + (long long)blockIdx.x; p < a.R; p += gridDim.x)
            for (int n = et; n < a.N; n += 32 * C::kEpiWarps) out[p * a.os + n] = from_f32<O>(0.f);
        int n = 0;
        for (int t = first_tile; t < tiles && ok; t += tile_step, ++n) {
            const Tile w = tile_at(t);
            const int b = n & 1;
            const float* scale = token_scale[n % C::kTabs];
            const int ch = w.n0 + ew * 32 + lane;
            const float cs = ch < a.N && a.w_scale ? a.w_scale[(long long)w.e * a.N + ch] : 1.f;
            ok = __all_sync(kAll, wait_for<false>(tab_full(n % C::kTabs), (n / C::kTabs) & 1, abort, a.wait_ns));
            if (!ok) break;
            ok = __all_sync(kAll, wait_for<kPair>(d_full(b), (n >> 1) & 1, abort, a.wait_ns));
            if (!ok) break;
            tc_fence_after();
            O* dst = out + (long long)w.p0 * a.os + ch;
#pragma unroll 1
            for (int c0 = 0; c0 < w.count; c0 += 32) {
                uint32_t v[32];
                tmem_ld32(((uint32_t)(ew * 32) << 16) + b * kCap + c0, v);
                tmem_ld_wait();
                if (c0 + 32 >= w.count) release(b);  // the accumulator is free when its columns are in registers
                const bool whole = c0 + 32 <= w.count && w.n0 + ew * 32 + 32 <= a.N;
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
            leave_tab(n % C::kTabs);
        }
    }
    if (!ok) {
        *abort = 1;
        raise_flag(&g_block_err, ERR_TIMEOUT);
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

// Map over rows of codes, bytes of one row adjacent: boxes of 128 bytes x `rows_at_once`
// rows, 128-byte swizzle.
bool map_codes(CUtensorMap* m, const uint8_t* q, uint64_t bytes, uint64_t rows, uint64_t stride, uint32_t rows_at_once) {
    using Encode = decltype(&cuTensorMapEncodeTiled);
    static const Encode encode = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e =
            cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found);
        return e == cudaSuccess && found == cudaDriverEntryPointSuccess ? reinterpret_cast<Encode>(p) : nullptr;
    }();
    if (!encode) return false;
    const cuuint64_t dims[2] = {bytes, rows}, strides[1] = {stride};
    const cuuint32_t box[2] = {128, rows_at_once}, step[2] = {1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(q), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// `most`: tiles at most; the grid is no larger than what runs at the same time.
template <bool kPair, bool kNv, typename O>
cudaError_t launch_kind(const BlockProduct& a, long long most, int dev, const CUtensorMap& wmap, const CUtensorMap& qmap,
                        cudaStream_t s) {
    using C = Cfg<kPair, kNv>;
    auto* kernel = k_block_product_tc<kPair, kNv, O>;
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
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
            // (a pair needs two SMs of one cluster of them: not every SM finds a partner)
            cfg.gridDim = dim3(C::kCtas);
            if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
            if (e != cudaSuccess) return e;
            if (n < 1) return cudaErrorInvalidConfiguration;
            if (dev < 64) fits[dev] = n;
        }
    }
    cfg.gridDim = dim3((unsigned)(most < n ? most : n) * C::kCtas);
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a, wmap, qmap);
}

template <bool kNv, typename O>
cudaError_t launch_o(const BlockProduct& a, const CUtensorMap& wmap, const CUtensorMap& qmap, cudaStream_t s) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    auto most = [&](int cap, int channels) {  // tiles
        return (a.R / cap + (long long)(a.E < a.R ? a.E : a.R)) * ((a.N + channels - 1) / channels);
    };
    if (block_product_pairs(a.E, a.R, a.K, a.N, sms))
        return launch_kind<true, kNv, O>(a, most(Cfg<true, kNv>::kCap, 256), dev, wmap, qmap, s);
    return launch_kind<false, kNv, O>(a, most(Cfg<false, kNv>::kCap, 128), dev, wmap, qmap, s);
}

}  // namespace

// Narrow or wide tiles, by rounds over the GPU times what a round takes, in us.  A segment
// of m positions has about m / cap + 1/2 tiles (those of the dense product are known) and at
// least one; it is taken as equal to the others, for the segments are on the device.
// Measured at K = 4096 in NVFP4, narrow and wide: 256 rows of one expert 10.1 and 12.5, 300 14.0
// and 13.7, 1024 23 and 21; 32 experts of 32 rows 56 and 57, of 64 66 and 59; at K = 2048 and
// 256 experts of 24 rows 216 and 211 (MXFP4 181 and 190), of 48 272 and 228 (216 and 204); 777
// rows at K = 1120, N = 1001 10.3 and 17.3.
bool block_product_pairs(int E, int R, int K, int N, int sms) {
    static_assert(Cfg<true, true>::kCap == Cfg<true, false>::kCap && Cfg<false, true>::kCap == Cfg<false, false>::kCap, "one rule");
    const double segs = E < R ? E : R;
    auto cost = [&](int cap, int channels, int at_once, double fixed, double base, double a_row) {
        const double mean = R / segs, each = E == 1 ? (R + cap - 1) / cap : mean / cap + 0.5;
        const double n = each > 1 ? each : 1;
        const double rounds = std::ceil(segs * n * ((N + channels - 1) / channels) / at_once);
        return fixed + rounds * (base + a_row * mean / n) * K / 4096;
    };
    return cost(Cfg<true, true>::kCap, 256, sms / 2, 5.8, 7.4, 0.01) < cost(Cfg<false, true>::kCap, 128, sms, 4.3, 6.6, 0);
}

cudaError_t block_product_flag_at(uint32_t** flag) { return cudaGetSymbolAddress((void**)flag, g_block_err); }

cudaError_t launch_block_product_tc(const BlockProduct& a, bool nv, moe_dtype out, cudaStream_t s) {
    CUtensorMap wmap, qmap;
    const uint64_t bytes = (uint64_t)a.K / 2;
    if (!map_codes(&wmap, a.wq, bytes, (uint64_t)a.E * a.N, bytes, 128) ||
        !map_codes(&qmap, a.q, bytes, (uint64_t)(a.rows > 0 ? a.rows : 1), (uint64_t)a.qs, a.row_src ? 1 : 16))
        return cudaErrorInvalidValue;
    auto run = [&](auto type) {
        using O = decltype(type);
        return nv ? launch_o<true, O>(a, wmap, qmap, s) : launch_o<false, O>(a, wmap, qmap, s);
    };
    if (out == MOE_F32) return run(float());
    if (out == MOE_BF16) return run(__nv_bfloat16());
    return run(__half());
}

}  // namespace moe
