// kda_paged_launch.h - internal launchers behind kda_paged.h (not part of the public header).
#pragma once

#include "kda_launch.h"
#include "kda_paged.h"

namespace kda {

cudaError_t launch_paged_plan(const kda_plan_params& p, cudaStream_t s);

// wide: 16-byte accesses (every row 16-byte aligned, head_dim a multiple of 16, the turned part in whole runs of 8 pairs).
cudaError_t launch_rope_append(const kda_rope_params& p, bool wide, cudaStream_t s);

// One warp per (row, query head) on the CUDA cores: any cache.
cudaError_t launch_paged_attention_simt(const kda_attention_params& p, cudaStream_t s);

}  // namespace kda
