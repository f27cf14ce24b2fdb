// kda_paged.cuh - what the paged-attention kernels share.
#pragma once

#include "kda_device.cuh"
#include "kda_paged.h"

namespace kda {

// The kernels of a step follow one another closely (plan, then per layer append and attention), and the small ones are
// over in a few microseconds, so each is launched to be brought in while the kernel before it ends (launch_early), and
// waits here until everything before it in the stream is done and visible, before it touches memory. Called one after
// another: the append of 256 rows 6.2 -> 3.9 us, the plan of 256 requests 6.2 -> 3.5. (Signalling the next kernel at the
// start instead of at the end was slower, 4.7 us for the append: its waiting CTAs are in the way.)
__device__ __forceinline__ void earlier_work() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// One request's rows and keys after the checks: n rows from row0 on, kv keys,
// row j at position kv - n + j. A request with bad row bounds has n = 0.
struct AttnRequest {
  int row0, n, kv;
  unsigned bad;  // KDA_ERR_* bits
};

__device__ __forceinline__ AttnRequest attn_request(const kda_attention_params& p, int r) {
  AttnRequest q{p.cu_new[r], 0, p.kv_len[r], 0u};
  const int end = p.cu_new[r + 1];
  if (q.row0 < 0 || end < q.row0 || end > p.num_tokens)
    q.bad |= KDA_ERR_SEQLENS;
  else
    q.n = end - q.row0;
  if (q.kv < 0 || q.kv > (long long)p.table_width * p.cache.page_size) {
    q.bad |= KDA_ERR_LENGTHS;
    q.kv = 0;
  }
  return q;
}

// The first key a row at position pos sees (window 0: all before it).
__device__ __forceinline__ int first_key(int pos, int window) {
  return window > 0 && pos >= window ? pos - window + 1 : 0;
}

// Launches a kernel that begins with earlier_work(), allowing it to be brought in early.
template <typename... Params, typename... Args>
inline cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

}  // namespace kda
