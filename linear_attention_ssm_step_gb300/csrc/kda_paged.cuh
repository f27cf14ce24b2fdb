// kda_paged.cuh - what the paged-attention kernels share.
#pragma once

#include "kda_device.cuh"
#include "kda_paged.h"

namespace kda {

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

}  // namespace kda
