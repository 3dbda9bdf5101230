// permute.h -- the counting sort by expert with bookkeeping of the caller's
// (route_permute.cu), for the entry points without a layer.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

namespace moe {

// CTAs (of 1024 rows) of the sort over several, 0 where one CTA sorts alone.
inline int perm_ctas(int R) { return R > 8 * 1024 ? (R + 1023) / 1024 : 0; }
// perm_cnt: perm_ctas(T k) * E words; the rest as launch_permute_raw.
cudaError_t launch_permute_rows(const int32_t* ids, int T, int k, int E, int32_t* offsets, int32_t* row_src,
                                int32_t* row_dst, int32_t* counts, int32_t* poff, int32_t* tile_scan,
                                int32_t* chunk_scan, int32_t* row_pos, int32_t* pos_row, int32_t* perm_cnt,
                                cudaStream_t s);

}  // namespace moe
