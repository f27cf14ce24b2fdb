/*
 * kda_paged.h - paged attention beside the KDA step: the page plan of a step,
 * rotary positions with the append to the cache, and the attention of each
 * request's new tokens over its cached ones.
 *
 * A hybrid decoder puts layers of ordinary attention between its KDA layers.
 * Such a layer keeps keys and values in pages of page_size tokens that any
 * request can own. One serving step runs
 *
 *   kda_paged_plan       once: pages for the new tokens, block table, slots
 *   kda_rope_append      per attention layer: q and k turned, k and v stored
 *   kda_paged_attention  per attention layer
 *
 * on the packed rows of all requests (request r owns rows cu_new[r] ..
 * cu_new[r+1]-1, as kda_prefill's cu_seqlens), whether they bring one token
 * (decode), a few (speculative verify) or a chunk of a prompt (prefill).
 *
 * The conventions of kda.h hold: device pointers owned by the caller, nothing
 * allocated or synchronized, kernels on `stream` only, host-side validation
 * before any launch, kda_last_error(), error words that kernels OR bits into,
 * strides in elements, bf16 tensors with the last dimension contiguous.
 * Where arguments must not overlap, rows of heads (q, k, v and q_out, q and
 * out) may lie beside one another in the rows, or in the heads, of one buffer
 * of a common stride; any others are taken to overlap where their ranges from
 * the first byte to the last do.
 * Every call is deterministic and can be captured in a CUDA graph.
 */
#ifndef KDA_GB300_KDA_PAGED_H
#define KDA_GB300_KDA_PAGED_H

#include <stddef.h>

#include "kda.h"
#include "kda_prefill.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bits ORed into error_word besides those of kda.h and kda_prefill.h. */
#define KDA_ERR_PAGES 16u   /* the free pages ran out, or a page or slot number is outside the cache */
#define KDA_ERR_LENGTHS 32u /* a request's lengths are negative or longer than its block table or the rows */

/* Requests one kda_paged_plan or kda_paged_attention call takes. */
#define KDA_MAX_REQUESTS 4096

/* One side (keys or values) of a paged cache: bf16, element (page, token, head,
   c) at page * page_stride + token * token_stride + head * head_stride + c. Any
   order of the strides (tokens before heads, heads before tokens, keys and
   values of a page side by side) works. */
typedef struct {
  void* ptr;
  int64_t page_stride, token_stride, head_stride;
} kda_pages;

typedef struct {
  kda_pages k, v;
  int32_t num_pages; /* >= 0; num_pages * page_size < 2^31 */
  int32_t page_size; /* tokens a page, >= 1 */
  int32_t num_heads; /* key-value heads, >= 1 */
  int32_t head_dim;
} kda_paged_cache;

/*
 * The page plan of a step: for every request, pages for its new tokens, then
 * where each packed row stands and is stored.
 *
 * Request r has cached[r] tokens in the cache and brings new_len[r]. With
 * have = ceil(cached / page_size) and need = ceil((cached + new) / page_size)
 * - have, table entries [0, have) are read and entries [have, have + need)
 * are written, from the top of the free list: the i-th page handed out in this
 * call, counted through the requests in order, is free_pages[*free_count - 1
 * - i]. Then for row t = cu_new[r] + j:
 *   positions[t] = cached[r] + j
 *   slots[t]     = table[r][positions[t] / page_size] * page_size + positions[t] % page_size
 *   kv_len[r]    = cached[r] + new_len[r]
 * cu_new is the exclusive sum of new_len (2^31 - 1 where it is larger); *free_count_out is *free_count minus
 * the pages handed out.
 *
 * Admission. A request is turned down when its lengths are negative or exceed
 * table_width * page_size, when its rows end past num_tokens
 * (KDA_ERR_LENGTHS), or when it needs pages and the running sum of needs up to
 * it exceeds *free_count (KDA_ERR_PAGES; the running sum goes on, so that every
 * later request that needs pages is turned down too). It then gets no pages,
 * kv_len 0 (attention gives its rows zeros), and its rows have position and
 * slot -1; they still count in cu_new (a negative new_len counts as 0). Rows
 * past the last request's (up to num_tokens, for calls padded to a fixed size)
 * get -1 too. A page number outside [0, num_pages), in the table or the free
 * list, gives slot -1 and KDA_ERR_PAGES. *free_count outside [0,
 * free_capacity] is taken as the nearer bound.
 *
 * Pages come back through the caller: the plan counts tokens, so a page past
 * ceil(cached / page_size) is no longer the request's, and its table entry is
 * written again when the request grows. After a step a request holds the
 * first ceil(kv_len / page_size) entries of its row. Where fewer tokens are
 * kept (drafts that a verify step rejects: cached < kv_len), the entries from
 * ceil(cached / page_size) on go back to the end of the free list, and their
 * number onto *free_count, before the next plan; all of them do when a
 * request ends. free_pages needs the room: free_capacity of num_pages always
 * has it.
 */
typedef struct {
  int32_t num_requests; /* 0..KDA_MAX_REQUESTS */
  int32_t num_tokens;   /* rows of positions and slots, >= 0 */
  int32_t page_size, num_pages;
  const int32_t* cached;     /* [num_requests] */
  const int32_t* new_len;    /* [num_requests] */
  int32_t* table;            /* [num_requests][table_width], updated in place */
  int64_t table_stride;      /* elements between requests, >= table_width */
  int32_t table_width;       /* >= 1; table_width * page_size <= 2^31 - 256 */
  const int32_t* free_pages; /* [free_capacity] */
  int32_t free_capacity;     /* >= 0 */
  const int32_t* free_count; /* [1] */
  int32_t* free_count_out;   /* [1], not free_count itself */
  int32_t* cu_new;           /* [num_requests + 1] */
  int32_t* kv_len;           /* [num_requests] */
  int32_t* positions;        /* [num_tokens] */
  int32_t* slots;            /* [num_tokens] */
  uint32_t* error_word;      /* optional */
} kda_plan_params;

kda_status kda_paged_plan(const kda_plan_params* p, void* stream);

/*
 * Rotary positions, and the append to the cache. For every row t with
 * positions[t] >= 0, in fp32, rounded to bf16 once:
 *   q_out[t][h] = rope(q[t][h]);  cache.k[slot][h] = rope(k[t][h]);  cache.v[slot][h] = v[t][h]
 * where rope turns the first rotary_dim values of a head, pair i by the angle
 * positions[t] * f_i: (x, y) -> mscale * (x cos - y sin, y cos + x sin). Pair i
 * is (2i, 2i+1) when interleaved, else (i, i + rotary_dim/2). The other values
 * of the head pass unchanged. A row with a negative position is skipped whole;
 * a row with slot -1 only turns q; any other slot outside the cache does so
 * too, with KDA_ERR_PAGES. Two rows with the same slot are undefined.
 *
 * freqs: device uint64 [rotary_dim / 2], f_i as a fraction of a whole turn per
 * position in units of 2^-64 (kda_rope_freqs fills a host array). positions[t]
 * * freqs[i] modulo 2^64 is the exact phase, at any position; a product of
 * fp32 radians would be off by 2^-24 of the angle, 0.008 radians at 131072.
 *
 * q_out may be q itself (same pointer and strides); otherwise it must overlap
 * none of q, k, v, and the cache must overlap none of them.
 */
typedef struct {
  int32_t num_tokens;  /* >= 0 */
  int32_t num_q_heads; /* >= 1 */
  int32_t rotary_dim;  /* even, 0..head_dim */
  int32_t interleaved;
  float mscale;        /* finite; scales the turned part (long-context attention factor), 1 for none */
  kda_view q, k, v;    /* bf16 [num_tokens][heads][head_dim]; t_stride unused */
  void* q_out;         /* bf16 [num_tokens][num_q_heads][head_dim] */
  int64_t q_out_b_stride, q_out_h_stride;
  const int32_t* positions; /* [num_tokens] */
  const int32_t* slots;     /* [num_tokens] */
  const uint64_t* freqs;    /* [rotary_dim / 2], 8-byte aligned */
  kda_paged_cache cache;    /* head_dim 1..256; written */
  uint32_t* error_word;     /* optional */
} kda_rope_params;

kda_status kda_rope_append(const kda_rope_params* p, void* stream);

/* How kda_rope_freqs scales the frequencies f_i = base^(-2i/rotary_dim) for
   contexts `factor` times the original. */
#define KDA_ROPE_PLAIN 0  /* not at all */
#define KDA_ROPE_LINEAR 1 /* f_i / factor: positions interpolated */
#define KDA_ROPE_BASE 2   /* base * factor^(rotary_dim / (rotary_dim - 2)): the slowest pair slowed by factor, the
                             fastest kept; rotary_dim > 2 */
#define KDA_ROPE_PARTS 3  /* by parts: with r = f_i * original_len / 2pi turns in the original context and
                             w = clamp((r - low) / (high - low), 0, 1): w f_i + (1 - w) f_i / factor */

/* Fills the HOST array freqs[rotary_dim / 2] for kda_rope_append. A host function: no CUDA call. KDA_EINVAL unless
   rotary_dim is even, 2..256, base > 1, factor >= 1 and finite, and, for KDA_ROPE_PARTS, original_len > 0 and
   0 <= low < high (finite). */
kda_status kda_rope_freqs(uint64_t* freqs, int32_t rotary_dim, double base, int32_t scaling, double factor,
                          double original_len, double low, double high);

/*
 * Attention of the new tokens over the paged cache (which already holds their
 * keys and values). Request r has rows cu_new[r] .. cu_new[r+1]-1 and kv_len[r]
 * tokens in the cache, the last of them being its rows: row j stands at
 * p = kv_len - n + j and sees the keys max(0, p - window + 1) .. p (window 0:
 * all from 0). Query head h reads key-value head h / (num_q_heads /
 * cache.num_heads). Per row and head
 *   out = sum_j softmax_j(scale q.k_j) v_j,  lse = log sum_j exp(scale q.k_j)
 * A row that sees no key (p < 0, so kv_len < n) gives zeros and lse -inf.
 * Scores, maxima, sums and outputs are kept in fp32; the weights enter the
 * product with v as bf16 (their sum does not); out is rounded to bf16 once.
 *
 * Keys and values of tokens at or past kv_len do not enter any result, whatever
 * they hold, nor do keys a row does not see enter that row's scores. Infinite
 * and NaN numbers that a row does see act as the formulas say: a score of -inf
 * is a weight of 0; where all the scores are -inf, out is NaN (0 / 0) and lse
 * -inf; a score of +inf or NaN makes out and lse NaN. An infinite or NaN number
 * of a value below kv_len makes infinite or NaN its dimension of out in the
 * rows that see it, and may make it NaN in other rows of the request.
 *
 * Pages are found through table[r][token / page_size]; entries of pages no row
 * sees are not read. A page outside [0, num_pages) counts as keys and values
 * of zero, with KDA_ERR_PAGES. Bounds cu_new out of order or past num_tokens
 * skip the request (KDA_ERR_SEQLENS); a kv_len negative or over table_width *
 * page_size counts as 0 (KDA_ERR_LENGTHS). Rows no request covers are not
 * written; rows that several requests cover are undefined, and where the
 * requests together hold more than num_tokens rows, every row is
 * (KDA_ERR_SEQLENS).
 *
 * head_dim 64 or 128 with a page size that is a power of two from 16 on and
 * 16-byte aligned cache rows (pointers, and strides that are multiples of 8)
 * runs on the tensor cores; any other cache (head_dim 1..256) on the CUDA
 * cores, slower (as do strides of q or out of 2^31 elements or more, and work
 * past 2^31 tiles of 256 rows by 128 keys).
 *
 * workspace: kda_paged_attention_workspace_bytes(head_dim) bytes of device
 * memory, 16-byte aligned, the caller's own, overlapping no other argument.
 * Its first KDA_ATTENTION_WORKSPACE_ZEROED bytes must be zero when it is first
 * used; every call leaves them zero for the next (after KDA_ERR_TIMEOUT, clear
 * them again; out is then unspecified). Calls in flight at once need a
 * workspace each.
 */
#define KDA_ATTENTION_WORKSPACE_ZEROED 4096

typedef struct {
  int32_t num_requests; /* 0..KDA_MAX_REQUESTS */
  int32_t num_tokens;   /* rows of q and out, >= 0 */
  int32_t num_q_heads;  /* a multiple of cache.num_heads, at most 128 times it */
  int32_t window;       /* keys a row sees at most; 0: no limit */
  float scale;          /* finite, > 0 */
  kda_view q;           /* bf16 [num_tokens][num_q_heads][head_dim]; t_stride unused */
  void* out;            /* bf16 [num_tokens][num_q_heads][head_dim] */
  int64_t out_b_stride, out_h_stride;
  float* lse;           /* optional fp32 [num_tokens][num_q_heads] */
  const int32_t* cu_new; /* [num_requests + 1] */
  const int32_t* kv_len; /* [num_requests] */
  const int32_t* table;  /* [num_requests][table_width] */
  int64_t table_stride;
  int32_t table_width;   /* >= 1; table_width * cache.page_size <= 2^31 - 256 */
  kda_paged_cache cache; /* read */
  uint32_t* error_word;  /* optional */
} kda_attention_params;

kda_status kda_paged_attention(const kda_attention_params* p, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes on the current device; 0 without one or for head_dim outside 1..256. */
size_t kda_paged_attention_workspace_bytes(int32_t head_dim);

#ifdef __cplusplus
}
#endif

#endif /* KDA_GB300_KDA_PAGED_H */
