// The kernels of the attention over a paged cache, between the plan and the kernels' files.
#pragma once

#include "kernels.h"

namespace fastar {

constexpr int kF32Rows = 32, kF32Keys = 64;
cudaError_t launch_paged_attn_f32(int d, const PagedAttnArgs& a, cudaStream_t s);
// bf16, up to kFewRows rows a KV head
constexpr int kFewRows = 32, kFewWarps = 4;
cudaError_t launch_paged_attn_few(int d, const PagedAttnArgs& a, cudaStream_t s);
// bf16; alone: at d = 128 single CTAs, for up to 128 rows
cudaError_t launch_paged_attn_tc(int d, const PagedAttnArgs& a, bool alone, cudaStream_t s);

}  // namespace fastar
