// kda_paged_api.cu - the C ABI of include/kda_paged.h: host-side argument
// validation, the choice of kernel and dispatch.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <numeric>

#include "kda_error.h"
#include "kda_paged.h"
#include "kda_paged_launch.h"

namespace {

using kda::fail;
using kda::ok;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Byte extent [lo, hi) of a buffer or strided tensor.
struct Extent {
  uintptr_t lo = 0, hi = 0;
};

Extent bytes_extent(const void* p, size_t bytes) {
  Extent e;
  e.lo = reinterpret_cast<uintptr_t>(p);
  e.hi = e.lo + bytes;
  return e;
}

// Rows of heads: [n][heads][dim] bf16.
Extent rows_extent(const void* p, int64_t n, int64_t b_stride, int64_t heads, int64_t h_stride, int64_t dim) {
  return n < 1 ? Extent() : bytes_extent(p, (size_t)((n - 1) * b_stride + (heads - 1) * h_stride + dim) * 2);
}

Extent pages_extent(const kda_pages& g, const kda_paged_cache& c) {
  if (c.num_pages < 1) return Extent();
  return bytes_extent(g.ptr, (size_t)((int64_t)(c.num_pages - 1) * g.page_stride + (int64_t)(c.page_size - 1) * g.token_stride +
                                      (int64_t)(c.num_heads - 1) * g.head_stride + c.head_dim) * 2);
}

bool overlaps(const Extent& a, const Extent& b) {
  return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

kda_status check_words(const char* name, const void* p, bool needed) {
  if (needed && p == nullptr) return fail(KDA_EINVAL, "%s is NULL", name);
  if (!aligned(p, 4)) return fail(KDA_EINVAL, "%s is not 4-byte aligned", name);
  return KDA_OK;
}

// Rows of heads, in bytes: row i, head j at lo + i b + j h, dim bytes long. A stride that no second entry uses is 0.
struct Rows {
  uint64_t lo, b, h, head_span, dim;  // head_span: from a row's first byte to behind its last
  Extent e;
};

Rows rows_of(const void* p, int64_t n, int64_t b_stride, int64_t heads, int64_t h_stride, int64_t dim) {
  Rows r;
  r.lo = reinterpret_cast<uintptr_t>(p);
  r.b = n > 1 ? (uint64_t)b_stride * 2 : 0;
  r.h = heads > 1 ? (uint64_t)h_stride * 2 : 0;
  r.dim = (uint64_t)dim * 2;
  r.head_span = (uint64_t)(heads - 1) * r.h + r.dim;
  r.e = rows_extent(p, n, b_stride, heads, h_stride, dim);
  return r;
}

// Whether two tensors may share a byte. They do not where their ranges are apart, and not where they lie beside one another
// in a common period: modulo a divisor of the strides, every row (every head of every row) of a tensor falls on one
// interval, and the two intervals are apart (columns of the rows of one buffer, or of its heads).
bool overlaps(const Rows& x, const Rows& y) {
  if (!overlaps(x.e, y.e)) return false;
  const uint64_t rows = std::gcd(x.b, y.b), heads = std::gcd(rows, std::gcd(x.h, y.h));
  auto apart = [&](uint64_t period, uint64_t x_span, uint64_t y_span) {
    if (period == 0) return false;
    const uint64_t to_y = (y.lo % period + period - x.lo % period) % period;
    return to_y >= x_span && period - to_y >= y_span;
  };
  return !apart(rows, x.head_span, y.head_span) && !apart(heads, x.dim, y.dim);
}

// A bf16 tensor of n rows (below 2^31, of at most 2^17 heads). Strides in [0, 2^40) and a span of rows of at most 2^60
// elements, so that no extent overflows.
kda_status check_rows(const char* name, const void* p, int64_t n, int64_t b_stride, int64_t h_stride) {
  if (p == nullptr) return fail(KDA_EINVAL, "%s is NULL", name);
  if (!aligned(p, 2)) return fail(KDA_EINVAL, "%s is not 2-byte aligned", name);
  if (b_stride < 0 || h_stride < 0) return fail(KDA_EINVAL, "%s has a negative stride", name);
  if (b_stride >> 40 || h_stride >> 40) return fail(KDA_EUNSUPPORTED, "%s has a stride of 2^40 or more", name);
  if (n > 1 && b_stride > (int64_t{1} << 60) / (n - 1))
    return fail(KDA_EUNSUPPORTED, "%s has rows that span more than 2^60 elements", name);
  return KDA_OK;
}

kda_status check_pages(const char* name, const kda_pages& g, const kda_paged_cache& c) {
  if (c.num_pages == 0) return KDA_OK;
  if (g.ptr == nullptr) return fail(KDA_EINVAL, "%s.ptr is NULL with num_pages = %d", name, c.num_pages);
  if (!aligned(g.ptr, 2)) return fail(KDA_EINVAL, "%s.ptr is not 2-byte aligned", name);
  if (g.page_stride < 0 || g.token_stride < 0 || g.head_stride < 0)
    return fail(KDA_EINVAL, "%s has a negative stride", name);
  if (g.page_stride >> 31 || g.token_stride >> 31 || g.head_stride >> 31)
    return fail(KDA_EUNSUPPORTED, "%s has a stride of 2^31 elements or more", name);
  return KDA_OK;
}

kda_status check_cache(const kda_paged_cache& c) {
  if (c.num_pages < 0) return fail(KDA_EINVAL, "cache.num_pages = %d is negative", c.num_pages);
  if (c.page_size < 1) return fail(KDA_EINVAL, "cache.page_size = %d is below 1", c.page_size);
  if (c.num_heads < 1) return fail(KDA_EINVAL, "cache.num_heads = %d is below 1", c.num_heads);
  if (c.num_heads > 1024) return fail(KDA_EUNSUPPORTED, "cache.num_heads = %d is above 1024", c.num_heads);
  if (c.head_dim < 1 || c.head_dim > 256) return fail(KDA_EUNSUPPORTED, "cache.head_dim = %d outside 1..256", c.head_dim);
  if ((long long)c.num_pages * c.page_size > 0x7fffffffLL)
    return fail(KDA_EUNSUPPORTED, "num_pages * page_size = %lld tokens, 2^31 or more",
                (long long)c.num_pages * c.page_size);
  kda_status s = check_pages("cache.k", c.k, c);
  return s != KDA_OK ? s : check_pages("cache.v", c.v, c);
}

kda_status check_table(const int32_t* table, int64_t stride, int32_t width, int32_t page_size, int32_t requests) {
  if (width < 1) return fail(KDA_EINVAL, "table_width = %d is below 1", width);
  if ((long long)width * page_size > 0x7fffff00LL)  // positions rounded up to whole units of keys stay in 32 bits
    return fail(KDA_EUNSUPPORTED, "table_width * page_size = %lld tokens, above 2^31 - 256", (long long)width * page_size);
  if (requests > 1 && stride < width)
    return fail(KDA_EINVAL, "table_stride = %lld is below table_width = %d", (long long)stride, width);
  if (requests > 1 && stride >> 40) return fail(KDA_EUNSUPPORTED, "table_stride = %lld, 2^40 or more", (long long)stride);
  return check_words("table", table, true);
}

kda_status check_requests(int32_t n) {
  if (n < 0) return fail(KDA_EINVAL, "num_requests = %d is negative", n);
  if (n > KDA_MAX_REQUESTS) return fail(KDA_EUNSUPPORTED, "num_requests = %d is above %d", n, KDA_MAX_REQUESTS);
  return KDA_OK;
}

// 16-byte accesses to rows of heads: the pointer and both strides.
bool wide_rows(const void* p, int64_t b_stride, int64_t h_stride) {
  return aligned(p, 16) && b_stride % 8 == 0 && h_stride % 8 == 0;
}

// CTAs of the tensor-core attention: one an SM, each with a counter in the workspace's zeroed part. 0 without a device.
int attention_ctas() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  const int most = KDA_ATTENTION_WORKSPACE_ZEROED / (int)sizeof(unsigned);
  return sms < most ? sms : most;
}

bool wide_pages(const kda_pages& g) {
  return aligned(g.ptr, 16) && g.page_stride % 8 == 0 && g.token_stride % 8 == 0 && g.head_stride % 8 == 0;
}

}  // namespace

extern "C" {

kda_status kda_paged_plan(const kda_plan_params* p, void* stream) {
  if (p == nullptr) return fail(KDA_EINVAL, "params is NULL");
  kda_status s = check_requests(p->num_requests);
  if (s != KDA_OK) return s;
  if (p->num_tokens < 0) return fail(KDA_EINVAL, "num_tokens = %d is negative", p->num_tokens);
  if (p->page_size < 1) return fail(KDA_EINVAL, "page_size = %d is below 1", p->page_size);
  if (p->num_pages < 0) return fail(KDA_EINVAL, "num_pages = %d is negative", p->num_pages);
  if ((long long)p->num_pages * p->page_size > 0x7fffffffLL)
    return fail(KDA_EUNSUPPORTED, "num_pages * page_size = %lld tokens, 2^31 or more",
                (long long)p->num_pages * p->page_size);
  if (p->free_capacity < 0) return fail(KDA_EINVAL, "free_capacity = %d is negative", p->free_capacity);
  const bool any = p->num_requests > 0;
  if (any && (s = check_table(p->table, p->table_stride, p->table_width, p->page_size, p->num_requests)) != KDA_OK)
    return s;
  const struct {
    const char* name;
    const void* ptr;
    bool needed;
  } words[] = {{"cached", p->cached, any},
               {"new_len", p->new_len, any},
               {"free_pages", p->free_pages, p->free_capacity > 0},
               {"free_count", p->free_count, true},
               {"free_count_out", p->free_count_out, true},
               {"cu_new", p->cu_new, true},
               {"kv_len", p->kv_len, any},
               {"positions", p->positions, p->num_tokens > 0},
               {"slots", p->slots, p->num_tokens > 0},
               {"error_word", p->error_word, false}};
  for (const auto& w : words)
    if ((s = check_words(w.name, w.ptr, w.needed)) != KDA_OK) return s;
  // what the call writes overlaps nothing else: other CTAs still read the inputs
  const size_t R = (size_t)p->num_requests, T = (size_t)p->num_tokens;
  const struct {
    const char* name;
    Extent e;
  } parts[] = {{"free_count_out", bytes_extent(p->free_count_out, 4)},
               {"cu_new", bytes_extent(p->cu_new, (R + 1) * 4)},
               {"kv_len", bytes_extent(p->kv_len, R * 4)},
               {"positions", bytes_extent(p->positions, T * 4)},
               {"slots", bytes_extent(p->slots, T * 4)},
               {"table", any ? bytes_extent(p->table, (size_t)((R - 1) * p->table_stride + p->table_width) * 4) : Extent()},
               {"free_count", bytes_extent(p->free_count, 4)},
               {"free_pages", bytes_extent(p->free_pages, (size_t)p->free_capacity * 4)},
               {"cached", bytes_extent(p->cached, R * 4)},
               {"new_len", bytes_extent(p->new_len, R * 4)}};
  for (int i = 0; i < 6; ++i)
    for (int j = i + 1; j < 10; ++j)
      if (overlaps(parts[i].e, parts[j].e)) return fail(KDA_EINVAL, "%s overlaps %s", parts[i].name, parts[j].name);
  const cudaError_t e = kda::launch_paged_plan(*p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(KDA_ELAUNCH, "kda_paged_plan launch: %s", cudaGetErrorString(e));
  return ok();
}

kda_status kda_rope_append(const kda_rope_params* p, void* stream) {
  if (p == nullptr) return fail(KDA_EINVAL, "params is NULL");
  kda_status s = check_cache(p->cache);
  if (s != KDA_OK) return s;
  const int D = p->cache.head_dim, Hkv = p->cache.num_heads;
  if (p->num_tokens < 0) return fail(KDA_EINVAL, "num_tokens = %d is negative", p->num_tokens);
  if (p->num_q_heads < 1) return fail(KDA_EINVAL, "num_q_heads = %d is below 1", p->num_q_heads);
  if (p->num_q_heads > 16384) return fail(KDA_EUNSUPPORTED, "num_q_heads = %d is above 16384", p->num_q_heads);
  if (p->rotary_dim < 0 || p->rotary_dim > D || p->rotary_dim % 2)
    return fail(KDA_EINVAL, "rotary_dim = %d is not an even number in 0..%d", p->rotary_dim, D);
  if (!isfinite(p->mscale)) return fail(KDA_EINVAL, "mscale is not finite");
  if (p->num_tokens == 0) return ok();
  if ((s = check_rows("q", p->q.ptr, p->num_tokens, p->q.b_stride, p->q.h_stride)) != KDA_OK) return s;
  if ((s = check_rows("k", p->k.ptr, p->num_tokens, p->k.b_stride, p->k.h_stride)) != KDA_OK) return s;
  if ((s = check_rows("v", p->v.ptr, p->num_tokens, p->v.b_stride, p->v.h_stride)) != KDA_OK) return s;
  if ((s = check_rows("q_out", p->q_out, p->num_tokens, p->q_out_b_stride, p->q_out_h_stride)) != KDA_OK) return s;
  if ((s = check_words("positions", p->positions, true)) != KDA_OK) return s;
  if ((s = check_words("slots", p->slots, true)) != KDA_OK) return s;
  if ((s = check_words("error_word", p->error_word, false)) != KDA_OK) return s;
  if (p->rotary_dim > 0 && (p->freqs == nullptr || !aligned(p->freqs, 8)))
    return fail(KDA_EINVAL, "freqs is NULL or not 8-byte aligned");
  const int64_t T = p->num_tokens;
  const Rows q = rows_of(p->q.ptr, T, p->q.b_stride, p->num_q_heads, p->q.h_stride, D);
  const Rows k = rows_of(p->k.ptr, T, p->k.b_stride, Hkv, p->k.h_stride, D);
  const Rows v = rows_of(p->v.ptr, T, p->v.b_stride, Hkv, p->v.h_stride, D);
  const Rows o = rows_of(p->q_out, T, p->q_out_b_stride, p->num_q_heads, p->q_out_h_stride, D);
  const Extent ck = pages_extent(p->cache.k, p->cache), cv = pages_extent(p->cache.v, p->cache);
  const bool in_place = p->q_out == p->q.ptr;
  if (in_place && ((p->q_out_b_stride != p->q.b_stride && T > 1) ||
                   (p->q_out_h_stride != p->q.h_stride && p->num_q_heads > 1)))
    return fail(KDA_EINVAL, "q_out is q with other strides");
  if (!in_place && (overlaps(o, q) || overlaps(o, k) || overlaps(o, v)))
    return fail(KDA_EINVAL, "q_out overlaps q, k or v");
  for (const Extent& c : {ck, cv})
    if (overlaps(c, q.e) || overlaps(c, k.e) || overlaps(c, v.e) || overlaps(c, o.e))
      return fail(KDA_EINVAL, "the cache overlaps q, k, v or q_out");
  const bool wide = D % 16 == 0 && p->rotary_dim % 16 == 0 && wide_rows(p->q.ptr, p->q.b_stride, p->q.h_stride) &&
                    wide_rows(p->k.ptr, p->k.b_stride, p->k.h_stride) &&
                    wide_rows(p->v.ptr, p->v.b_stride, p->v.h_stride) &&
                    wide_rows(p->q_out, p->q_out_b_stride, p->q_out_h_stride) &&
                    (p->cache.num_pages == 0 || (wide_pages(p->cache.k) && wide_pages(p->cache.v)));
  const cudaError_t e = kda::launch_rope_append(*p, wide, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(KDA_ELAUNCH, "kda_rope_append launch: %s", cudaGetErrorString(e));
  return ok();
}

kda_status kda_rope_freqs(uint64_t* freqs, int32_t rotary_dim, double base, int32_t scaling, double factor,
                          double original_len, double low, double high) {
  if (freqs == nullptr) return fail(KDA_EINVAL, "freqs is NULL");
  if (rotary_dim < 2 || rotary_dim > 256 || rotary_dim % 2)
    return fail(KDA_EINVAL, "rotary_dim = %d is not an even number in 2..256", rotary_dim);
  if (!(base > 1.0) || !isfinite(base)) return fail(KDA_EINVAL, "base is not a finite number above 1");
  if (scaling < KDA_ROPE_PLAIN || scaling > KDA_ROPE_PARTS) return fail(KDA_EINVAL, "scaling = %d outside 0..3", scaling);
  if (!(factor >= 1.0) || !isfinite(factor)) return fail(KDA_EINVAL, "factor is not a finite number of 1 or more");
  if (scaling == KDA_ROPE_BASE && rotary_dim < 4)
    return fail(KDA_EINVAL, "KDA_ROPE_BASE needs rotary_dim > 2 (got %d)", rotary_dim);
  if (scaling == KDA_ROPE_PARTS &&
      (!(original_len > 0.0) || !isfinite(original_len) || !(low >= 0.0) || !(high > low) || !isfinite(high)))
    return fail(KDA_EINVAL, "KDA_ROPE_PARTS needs original_len > 0 and 0 <= low < high, all finite");
  const double turn = 6.283185307179586476925286766559;
  const double b = scaling == KDA_ROPE_BASE ? base * pow(factor, rotary_dim / (rotary_dim - 2.0)) : base;
  if (!isfinite(b)) return fail(KDA_EINVAL, "base * factor^(rotary_dim / (rotary_dim - 2)) is not finite");
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double f = pow(b, -2.0 * i / rotary_dim);
    if (scaling == KDA_ROPE_LINEAR) f /= factor;
    if (scaling == KDA_ROPE_PARTS) {
      double w = (f * original_len / turn - low) / (high - low);
      w = w < 0.0 ? 0.0 : w > 1.0 ? 1.0 : w;
      f = w * f + (1.0 - w) * f / factor;
    }
    freqs[i] = (uint64_t)rint(ldexp(f / turn, 64));  // f <= 1 radian: below 2^62
  }
  return ok();
}

size_t kda_paged_attention_workspace_bytes(int32_t head_dim) {
  if (head_dim < 1 || head_dim > 256) return 0;
  const int ctas = attention_ctas();
  if (ctas == 0) return 0;
  // only the tensor-core kernel, which takes these head sizes, leaves parts
  const size_t parts = head_dim == 64 || head_dim == 128 ? kda::paged_attention_parts_bytes(head_dim, ctas) : 0;
  return KDA_ATTENTION_WORKSPACE_ZEROED + parts;
}

kda_status kda_paged_attention(const kda_attention_params* p, void* workspace, size_t workspace_bytes, void* stream) {
  if (p == nullptr) return fail(KDA_EINVAL, "params is NULL");
  kda_status s = check_requests(p->num_requests);
  if (s != KDA_OK) return s;
  if ((s = check_cache(p->cache)) != KDA_OK) return s;
  const int D = p->cache.head_dim, Hkv = p->cache.num_heads;
  if (p->num_tokens < 0) return fail(KDA_EINVAL, "num_tokens = %d is negative", p->num_tokens);
  if (p->num_q_heads < 1 || p->num_q_heads % Hkv)
    return fail(KDA_EINVAL, "num_q_heads = %d is not a multiple of cache.num_heads = %d", p->num_q_heads, Hkv);
  if (p->num_q_heads / Hkv > 128)
    return fail(KDA_EUNSUPPORTED, "%d query heads share a key-value head, more than 128", p->num_q_heads / Hkv);
  if ((long long)p->num_tokens * p->num_q_heads > 0x7fffffffLL)
    return fail(KDA_EUNSUPPORTED, "num_tokens * num_q_heads = %lld, 2^31 or more",
                (long long)p->num_tokens * p->num_q_heads);
  if (p->window < 0) return fail(KDA_EINVAL, "window = %d is negative", p->window);
  if (!isfinite(p->scale) || !(p->scale > 0.f)) return fail(KDA_EINVAL, "scale is not a finite number above 0");
  if (p->num_requests == 0 || p->num_tokens == 0) return ok();
  if ((s = check_table(p->table, p->table_stride, p->table_width, p->cache.page_size, p->num_requests)) != KDA_OK) return s;
  if ((s = check_rows("q", p->q.ptr, p->num_tokens, p->q.b_stride, p->q.h_stride)) != KDA_OK) return s;
  if ((s = check_rows("out", p->out, p->num_tokens, p->out_b_stride, p->out_h_stride)) != KDA_OK) return s;
  if ((s = check_words("cu_new", p->cu_new, true)) != KDA_OK) return s;
  if ((s = check_words("kv_len", p->kv_len, true)) != KDA_OK) return s;
  if ((s = check_words("lse", p->lse, false)) != KDA_OK) return s;
  if ((s = check_words("error_word", p->error_word, false)) != KDA_OK) return s;
  const size_t rows = (size_t)p->num_tokens * p->num_q_heads, R = (size_t)p->num_requests;
  const Rows q = rows_of(p->q.ptr, p->num_tokens, p->q.b_stride, p->num_q_heads, p->q.h_stride, D);
  const Rows out = rows_of(p->out, p->num_tokens, p->out_b_stride, p->num_q_heads, p->out_h_stride, D);
  const Extent& o = out.e;
  const Extent l = bytes_extent(p->lse, p->lse ? rows * 4 : 0);
  const struct {
    const char* name;
    Extent e;
  } inputs[] = {{"q", q.e},
                {"cache.k", pages_extent(p->cache.k, p->cache)},
                {"cache.v", pages_extent(p->cache.v, p->cache)},
                {"table", bytes_extent(p->table, (size_t)((R - 1) * p->table_stride + p->table_width) * 4)},
                {"cu_new", bytes_extent(p->cu_new, (R + 1) * 4)},
                {"kv_len", bytes_extent(p->kv_len, R * 4)}};
  if (overlaps(out, q)) return fail(KDA_EINVAL, "out overlaps q");
  for (const auto& in : inputs) {
    if (&in != inputs && overlaps(o, in.e)) return fail(KDA_EINVAL, "out overlaps %s", in.name);
    if (overlaps(l, in.e)) return fail(KDA_EINVAL, "lse overlaps %s", in.name);
  }
  if (overlaps(o, l)) return fail(KDA_EINVAL, "out overlaps lse");
  const size_t need = kda_paged_attention_workspace_bytes(D);
  if (need == 0) return fail(KDA_ELAUNCH, "kda_paged_attention: no current device");
  if (workspace == nullptr || !aligned(workspace, 16)) return fail(KDA_EINVAL, "workspace is NULL or not 16-byte aligned");
  if (workspace_bytes < need)
    return fail(KDA_EINVAL, "workspace_bytes = %zu is below the %zu this call needs (kda_paged_attention_workspace_bytes)",
                workspace_bytes, need);
  const Extent w = bytes_extent(workspace, need);
  for (const auto& in : inputs)
    if (overlaps(w, in.e)) return fail(KDA_EINVAL, "workspace overlaps %s", in.name);
  if (overlaps(w, o) || overlaps(w, l)) return fail(KDA_EINVAL, "workspace overlaps out or lse");
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorNotSupported;
  if (kda::paged_attention_on_tensor_cores(p->cache)) e = kda::launch_paged_attention_tc(*p, workspace, attention_ctas(), st);
  if (e == cudaErrorNotSupported) e = kda::launch_paged_attention_simt(*p, st);
  if (e != cudaSuccess) return fail(KDA_ELAUNCH, "kda_paged_attention launch: %s", cudaGetErrorString(e));
  return ok();
}

}  // extern "C"
