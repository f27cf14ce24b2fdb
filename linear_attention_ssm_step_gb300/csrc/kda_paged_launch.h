// kda_paged_launch.h - internal launchers behind kda_paged.h (not part of the public header).
#pragma once

#include "kda_launch.h"
#include "kda_paged_fp8.h"

namespace kda {

cudaError_t launch_paged_plan(const kda_plan_params& p, cudaStream_t s);

// wide: 16-byte accesses (every row 16-byte aligned, head_dim a multiple of 16, the turned part in whole runs of 8 pairs).
cudaError_t launch_rope_append(const kda_rope_params& p, bool wide, cudaStream_t s);

// A block of eight warps per (row, query head) on the CUDA cores: any cache, in 8 bits where there are scales.
cudaError_t launch_paged_attention_simt(const kda_attention_params& p, const kda_paged_scales* scales, cudaStream_t s);

// q_wide: as `wide` above, for q and q_out. lane_elems: key and value elements that a lane takes of a row at a time, 4
// (head_dim 128) or 2 (64) where all rows allow it, 0 for any others.
cudaError_t launch_rope_append_fp8(const kda_rope_params& p, const kda_paged_scales& sc, bool q_wide, int lane_elems,
                                   cudaStream_t s);

// wide: 16 codes at a time (head_dim a multiple of 16, every row on 16 bytes).
cudaError_t launch_paged_read_fp8(const kda_read_params& p, const kda_paged_scales& sc, bool wide, cudaStream_t s);

// One side of a paged cache as a tensor map for copies of 64 columns of `box` tokens (kda_tmap.cu).
cudaError_t pages_tensor_map(const kda_pages& g, const kda_paged_cache& c, int box, CUtensorMap* out);

// One side of a cache in 8 bits (head_dim 64 or 128) for copies of whole heads of `box` tokens.
cudaError_t code_pages_tensor_map(const kda_pages& g, const kda_paged_cache& c, int box, CUtensorMap* out);

// Whether the tensor-core kernel takes this cache (head_dim, page size, alignment), of bf16 or in 8 bits.
bool paged_attention_on_tensor_cores(const kda_paged_cache& c, bool fp8);

// Workspace bytes of that kernel for parts of items, on `ctas` CTAs, after the zeroed counters.
size_t paged_attention_parts_bytes(int head_dim, int ctas);

// Rows of an item (4, 8, 16 or 32) in the kernel for few rows over a cache in 8 bits; 0: the requests bring too many. That
// kernel's launcher; as launch_paged_attention_tc, which calls it.
int paged_attention_few_rows(const kda_attention_params& p);
cudaError_t launch_paged_attention_fp8_rows(const kda_attention_params& p, const kda_paged_scales& sc, int rows,
                                            void* workspace, int ctas, cudaStream_t s);

// Attention on the tensor cores, persistent on `ctas` CTAs (one an SM); cudaErrorNotSupported, with nothing launched,
// when the cache's strides have no tensor map, a stride of q or out is 2^31 or more, or the work is past 32 bits.
// scales: of a cache in 8 bits, or NULL.
cudaError_t launch_paged_attention_tc(const kda_attention_params& p, const kda_paged_scales* scales, void* workspace,
                                      int ctas, cudaStream_t s);

}  // namespace kda
