// The kernels of the attention over a paged cache, between the plan and the kernels' files.
#pragma once

#include "kernels.h"
#include "tmap.h"

namespace fastar {

// The tensor map of a bf16 pool: (channel, slot, head, page), boxes of 64 channels and `rows` slots.
inline bool make_pool_tmap(CUtensorMap* m, const PagedAttnArgs& a, const void* pool, int d, int rows) {
  const uint64_t dims[4] = {(uint64_t)d, (uint64_t)1 << a.pool.page_shift, (uint64_t)a.Hkv, (uint64_t)a.pool.pages};
  // (a dimension of one element: any stride will do but 0)
  const uint64_t strides[3] = {(uint64_t)a.pool.rs * 2, (uint64_t)(a.Hkv > 1 ? a.pool.hs : d) * 2, (uint64_t)a.pool.ps * 2};
  return make_tmap_bf16_4d(m, pool, dims, strides, 64, rows);
}

constexpr int kF32Rows = 32, kF32Keys = 64;
cudaError_t launch_paged_attn_f32(int d, const PagedAttnArgs& a, cudaStream_t s);
// bf16, up to kFewRows rows a KV head
constexpr int kFewRows = 32, kFewWarps = 4;
cudaError_t launch_paged_attn_few(int d, const PagedAttnArgs& a, cudaStream_t s);
// bf16; alone: at d = 128 single CTAs, for up to 128 rows; the rows of an item
int paged_tc_rows(int d, bool alone);
size_t paged_tc_cut_bytes();            // a share's entry of PagedAttnArgs::cuts
cudaError_t launch_paged_attn_tc(int d, const PagedAttnArgs& a, bool alone, cudaStream_t s);

}  // namespace fastar
