// kda_paged_launch.h - internal launchers behind kda_paged.h (not part of the public header).
#pragma once

#include "kda_launch.h"
#include "kda_paged.h"

namespace kda {

cudaError_t launch_paged_plan(const kda_plan_params& p, cudaStream_t s);

// wide: 16-byte accesses (every row 16-byte aligned, head_dim a multiple of 16, the turned part in whole runs of 8 pairs).
cudaError_t launch_rope_append(const kda_rope_params& p, bool wide, cudaStream_t s);

// A block of eight warps per (row, query head) on the CUDA cores: any cache.
cudaError_t launch_paged_attention_simt(const kda_attention_params& p, cudaStream_t s);

// One side of a paged cache as a tensor map for copies of 64 columns of `box` tokens (kda_tmap.cu).
cudaError_t pages_tensor_map(const kda_pages& g, const kda_paged_cache& c, int box, CUtensorMap* out);

// Whether the tensor-core kernel takes this cache (head_dim, page size, alignment).
bool paged_attention_on_tensor_cores(const kda_paged_cache& c);

// Workspace bytes of that kernel for parts of items, on `ctas` CTAs, after the zeroed counters.
size_t paged_attention_parts_bytes(int head_dim, int ctas);

// Attention on the tensor cores, persistent on `ctas` CTAs (one an SM); cudaErrorNotSupported, with nothing launched,
// when the cache's strides have no tensor map, a stride of q or out is 2^31 or more, or the work is past 32 bits.
cudaError_t launch_paged_attention_tc(const kda_attention_params& p, void* workspace, int ctas, cudaStream_t s);

}  // namespace kda
