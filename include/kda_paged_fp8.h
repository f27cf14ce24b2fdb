/*
 * kda_paged_fp8.h - the paged calls of kda_paged.h on a cache held in 8 bits:
 * keys and values quantised as they are written, attention over them, and
 * reading them back.
 *
 * Format. One byte per element, the E4M3 code of kda_fp8.h (largest finite
 * magnitude 448; the codes 0x7F and 0xFF are NaN), in pages of any strides as
 * in kda_paged.h, and one fp32 scale for each block of KDA_FP8_SCALE_TOKENS
 * consecutive tokens of a page and head, keys and values apart. A page of
 * page_size tokens has ceil(page_size / KDA_FP8_SCALE_TOKENS) blocks, the last
 * of them shorter where that leaves a rest. The cache holds code * scale.
 * Scales are powers of two from 2^-40 to 2^40; the calls that read take any
 * positive number in that range (and give undefined numbers, but nothing
 * else, outside it), the append takes powers of two alone where it continues a
 * block.
 *
 * The calls take the parameters of their 16-bit forms, with these differences:
 *   - kda_paged_cache.k and .v point to uint8 codes; their strides are in
 *     elements, which are bytes; a pointer needs no alignment;
 *   - the scales travel in a kda_paged_scales.
 * kda_paged_plan hands out the pages of such a cache too. The conventions of
 * kda_paged.h hold for everything else.
 */
#ifndef KDA_GB300_KDA_PAGED_FP8_H
#define KDA_GB300_KDA_PAGED_FP8_H

#include "kda_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_FP8_SCALE_TOKENS 16

/* The scales of one side of a cache: that of (page, block, head) at page * page_stride + block * block_stride +
   head * head_stride elements. Strides >= 0 and below 2^31. */
typedef struct {
  float* ptr;
  int64_t page_stride, block_stride, head_stride;
} kda_page_scales;

typedef struct {
  kda_page_scales k, v;
} kda_paged_scales;

/*
 * kda_rope_append on a cache in 8 bits: q_out as there; k (turned, in fp32)
 * and v quantised straight from fp32 to codes.
 *
 * The rows of one call that fall into one block are taken together. For each
 * side and head, with m the largest magnitude among them and e the smallest
 * integer in [-40, 40] with m * 2^-e <= 448 (40 if there is none):
 *   - where the first of the rows stands at the block's first token, the block
 *     begins anew: its scale becomes 2^e, whatever was there;
 *   - else it holds earlier tokens, and its scale becomes the larger of 2^e
 *     and the old one; if that is 2^e, the codes of the tokens before the
 *     first row are rounded anew, code <- rne(code * old / 2^e);
 *   - the rows' codes are rne(x / scale), round to nearest even.
 * A scale thus grows only while its block fills, and a token of it is rounded
 * again each time it does. Codes behind the rows are left as they are, and
 * count with the new scale. Numbers past 448 * 2^40 saturate there, infinite
 * ones too; NaN becomes a NaN code and does not count in m.
 *
 * Rows of one block must follow one another in the call, row t + 1 at
 * slots[t] + 1 (kda_paged_plan's rows of a request do). Rows among them that
 * are not stored (a negative position, slot -1 or outside the cache) stand for
 * the tokens in between, whose codes are left as they are and count with the
 * new scale. Where rows of a block come in any other order, or a slot twice,
 * that block's codes and scales are undefined. At most 2^30 rows a call.
 * k is turned with sines and cosines good to 2^-20, far below the rounding of a
 * code; q as in kda_rope_append.
 */
kda_status kda_rope_append_fp8(const kda_rope_params* p, const kda_paged_scales* s, void* stream);

/*
 * kda_paged_attention over a cache in 8 bits: the same formulas on the values
 * code * scale. Scores, maxima, sums and outputs are kept in fp32, out is
 * rounded to bf16 once. On the tensor cores
 *   - a query enters as two E4M3 numbers by a power of two for its row and
 *     head, exact within 2^9 of the largest magnitude of its head and off by
 *     less than 2^-17 of that below;
 *   - a weight, times its key's value scale, enters as fp16, by a power of two
 *     for the row that follows its largest; its sum does not. So it is off by up
 *     to 2^-11 of itself, and at the least by 2^-31 of the row's largest (2^-35
 *     for few rows): n small ones beside a large one by up to n times that.
 * Scores of 2^23 or more in magnitude, which fp32 holds no better than to a
 * whole number, may give infinite or NaN numbers in the kernel for chunks.
 * A query with an infinite or NaN number gives NaN in out and lse. NaN codes
 * that a row sees act as NaN does in kda_paged_attention.
 *
 * head_dim 64 or 128 with a page size that is a power of two from 16 on and
 * cache rows on 16 bytes (pointers, and strides that are multiples of 16) runs
 * on the tensor cores, any other cache on the CUDA cores. The workspace is
 * kda_paged_attention's, and the two calls may take turns with one.
 *
 * lse is off by up to 2^-21 of the largest |log2| of a value scale beside what
 * its terms' rounding in fp32 makes.
 *
 * Calls with up to 32 rows (new tokens times query heads of a key-value head) a
 * request on average (num_tokens over num_requests, idle ones too) run in a
 * kernel for few rows, others in one for chunks. A step that mixes decode tokens
 * and chunks is faster as two calls, one for each.
 */
kda_status kda_paged_attention_fp8(const kda_attention_params* p, const kda_paged_scales* s, void* workspace,
                                   size_t workspace_bytes, void* stream);

/*
 * Cached tokens read back as packed bf16 rows. Request r has rows cu_rows[r] ..
 * cu_rows[r+1]-1, n of them, and row j takes token kv_len[r] - n + j:
 *   k_out[row][h] = bf16(code * scale) of keys, v_out likewise of values,
 * exact for scales that are powers of two. n = kv_len reads a whole request;
 * cu_new reads the tokens of a step. A row in front of token 0, or of a page
 * outside [0, num_pages) (KDA_ERR_PAGES), gives zeros. Bounds, lengths and rows
 * that no request covers or several do: as in kda_paged_attention (but rows of
 * requests in order are written whatever other requests hold). NaN codes read
 * as NaN.
 */
typedef struct {
  int32_t num_requests; /* 0..KDA_MAX_REQUESTS */
  int32_t num_tokens;   /* rows of k_out and v_out, >= 0 */
  void* k_out;          /* bf16 [num_tokens][cache.num_heads][head_dim] */
  int64_t k_out_b_stride, k_out_h_stride;
  void* v_out;
  int64_t v_out_b_stride, v_out_h_stride;
  const int32_t* cu_rows; /* [num_requests + 1] */
  const int32_t* kv_len;  /* [num_requests] */
  const int32_t* table;   /* [num_requests][table_width] */
  int64_t table_stride;
  int32_t table_width;    /* >= 1; table_width * cache.page_size <= 2^31 - 256 */
  kda_paged_cache cache;  /* read */
  uint32_t* error_word;   /* optional */
} kda_read_params;

kda_status kda_paged_read_fp8(const kda_read_params* p, const kda_paged_scales* s, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_GB300_KDA_PAGED_FP8_H */
