// kda_paged.cu - the page plan of a step, rotary positions with the append to
// the paged cache, and paged attention on the CUDA cores (include/kda_paged.h).
#include "kda_device.cuh"
#include "kda_paged.cuh"
#include "kda_paged_launch.h"

namespace kda {

// ---------------------------------------------------------------- page plan
//
// cu = exclusive sum of new_len, pages handed out = exclusive sum of need: two
// prefix sums over the requests, then one independent search per row and per
// page. The bytes are few (a 16k-token step writes 130 KB), so a call is bound
// by the latency of one launch and a chain of dependent loads: lengths, table
// entry, store. Every CTA therefore sums all the requests itself (at most
// 4096, two values each) instead of waiting for another CTA's sums, and the
// rows are split over the CTAs.

constexpr int PLAN_THREADS = 256;

struct PlanSmem {
  int32_t* cu;    // [R + 1] row offsets, saturated at INT32_MAX
  int32_t* pages; // [R + 1] needs summed up to a request
  int32_t* kept;  // [R] cached tokens of an admitted request, -1 of one turned down
};

struct PlanRequest {
  long long rows, need;  // rows in the packing, pages asked for
  bool fits;             // lengths in order
};

__device__ __forceinline__ PlanRequest plan_request(const kda_plan_params& p, int r, int& cached) {
  PlanRequest q{0, 0, true};
  if (r >= p.num_requests) return q;
  const int n = p.new_len[r];
  cached = p.cached[r];
  q.rows = n > 0 ? n : 0;
  q.fits = n >= 0 && cached >= 0 && (long long)cached + n <= (long long)p.table_width * p.page_size;
  if (q.fits) {
    const long long P = p.page_size;
    q.need = ((long long)cached + n + P - 1) / P - ((long long)cached + P - 1) / P;
  }
  return q;
}

// Largest i in [0, n) with a[i] <= x (a[0] <= x, a non-decreasing).
__device__ __forceinline__ int last_at_most(const int32_t* a, int n, int x) {
  int lo = 0;
  while (n > 1) {
    const int half = n >> 1;
    if (a[lo + half] <= x) lo += half;
    n -= half;
  }
  return lo;
}

__device__ __forceinline__ int saturate(long long x) { return x > 0x7fffffffLL ? 0x7fffffff : (int)x; }

__global__ void __launch_bounds__(PLAN_THREADS) kda_paged_plan_kernel(kda_plan_params p) {
  extern __shared__ int32_t plan_smem[];
  const int R = p.num_requests, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  PlanSmem s{plan_smem, plan_smem + R + 1, plan_smem + 2 * (R + 1)};
  __shared__ long long warp_rows[PLAN_THREADS / 32], warp_need[PLAN_THREADS / 32];
  __shared__ int taken_all, bad_all;
  if (tid == 0) taken_all = bad_all = 0;
  earlier_work();
  const int free_now = min(max(*p.free_count, 0), p.free_capacity);
  __syncthreads();

  long long rows0 = 0, need0 = 0;  // sums over the requests before this chunk of PLAN_THREADS
  for (int base = 0; base < R; base += PLAN_THREADS) {
    const int r = base + tid;
    int cached = 0;
    PlanRequest q = plan_request(p, r, cached);
    long long rows = q.rows;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, rows, o);
      if (lane >= o) rows += a;
    }
    if (lane == 31) warp_rows[warp] = rows;
    __syncthreads();
    long long all_rows = 0;
    for (int w = 0; w < PLAN_THREADS / 32; ++w) {
      if (w < warp) rows += warp_rows[w];
      all_rows += warp_rows[w];
    }
    const long long row_end = rows0 + rows;
    // a request whose rows end past num_tokens takes no pages
    const bool in_rows = row_end <= p.num_tokens;
    if (!in_rows) q.need = 0;
    long long need = q.need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, need, o);
      if (lane >= o) need += a;
    }
    if (lane == 31) warp_need[warp] = need;
    __syncthreads();
    long long all_need = 0;
    for (int w = 0; w < PLAN_THREADS / 32; ++w) {
      if (w < warp) need += warp_need[w];
      all_need += warp_need[w];
    }
    const long long need_end = need0 + need;
    if (r < R) {
      const bool served = q.need == 0 || need_end <= free_now;
      const bool ok = q.fits && in_rows && served;
      s.cu[r] = saturate(row_end - q.rows);
      s.pages[r] = saturate(need_end - q.need);
      s.kept[r] = ok ? cached : -1;
      if (ok && q.need > 0) atomicMax(&taken_all, (int)need_end);
      const int bad = (!q.fits || !in_rows ? (int)KDA_ERR_LENGTHS : 0) | (!served ? (int)KDA_ERR_PAGES : 0);
      if (bad) atomicOr(&bad_all, bad);
      if (blockIdx.x == 0) {
        p.cu_new[r] = s.cu[r];
        p.kv_len[r] = ok ? cached + (int)q.rows : 0;
      }
    }
    rows0 += all_rows;
    need0 += all_need;
    __syncthreads();
  }
  if (tid == 0) {
    s.cu[R] = saturate(rows0);
    s.pages[R] = saturate(need0);
  }
  __syncthreads();
  const int taken = taken_all;
  if (blockIdx.x == 0 && tid == 0) {
    p.cu_new[R] = s.cu[R];
    *p.free_count_out = free_now - taken;
    if (bad_all && p.error_word) atomicOr(p.error_word, (unsigned)bad_all);
  }
  // rows and pages are counted without a sign: below 2^31, and a step of the whole grid beyond that must not wrap
  const unsigned first = blockIdx.x * PLAN_THREADS + tid, stride = gridDim.x * PLAN_THREADS;
  const unsigned num_tokens = (unsigned)p.num_tokens;
  if (R == 0) {
    for (unsigned t = first; t < num_tokens; t += stride) p.positions[t] = p.slots[t] = -1;
    return;
  }

  const int P = p.page_size;
  // new pages into the table: every page index below `taken` belongs to an admitted request
  for (unsigned u = first; u < (unsigned)taken; u += stride) {
    const int i = (int)u, r = last_at_most(s.pages, R, i);
    const int have = (int)(((long long)s.kept[r] + P - 1) / P);
    p.table[(int64_t)r * p.table_stride + have + (i - s.pages[r])] = p.free_pages[free_now - 1 - i];
  }
  bool bad_page = false;
  for (unsigned u = first; u < num_tokens; u += stride) {
    const int t = (int)u;
    int pos = -1, slot = -1;
    if (t < s.cu[R]) {
      const int r = last_at_most(s.cu, R, t);
      const int cached = s.kept[r];
      if (cached >= 0) {
        pos = cached + (t - s.cu[r]);
        const int have = (int)(((long long)cached + P - 1) / P);
        const int e = pos / P;
        // an entry written in this call is taken from the free list again, so no thread waits for another's store
        const int page = e < have ? p.table[(int64_t)r * p.table_stride + e]
                                  : p.free_pages[free_now - 1 - (s.pages[r] + e - have)];
        if (page >= 0 && page < p.num_pages)
          slot = page * P + (pos - e * P);
        else
          bad_page = true;
      }
    }
    p.positions[t] = pos;
    p.slots[t] = slot;
  }
  if (bad_page && p.error_word) atomicOr(p.error_word, KDA_ERR_PAGES);
}

cudaError_t launch_paged_plan(const kda_plan_params& p, cudaStream_t s) {
  const int rows = p.num_tokens > p.num_requests ? p.num_tokens : p.num_requests;
  int grid = rows / PLAN_THREADS + (rows % PLAN_THREADS != 0);
  grid = grid < 1 ? 1 : grid > 152 ? 152 : grid;
  const size_t smem = (size_t)(3 * p.num_requests + 2) * sizeof(int32_t);
  static DeviceFlags done;
  const cudaError_t e =
      set_smem_limit_once(kda_paged_plan_kernel, (3 * KDA_MAX_REQUESTS + 2) * sizeof(int32_t), done);
  if (e != cudaSuccess) return e;
  return launch_early(kda_paged_plan_kernel, dim3((unsigned)grid), PLAN_THREADS, smem, s, p);
}

// ---------------------------------------------------------------- rotary positions and append
//
// One CTA per row: its rotary_dim / 2 sines and cosines are formed once, in
// shared memory, for all query and key heads of the row (a sincos costs more
// than the traffic of the pair it turns). The rest is a copy, bound by memory:
// a thread moves two runs of VEC values, the two halves of VEC pairs when the
// halves are paired, 2 VEC consecutive values else; VEC = 8 (16-byte accesses)
// when every row allows it, 1 otherwise. What a row waits for (its position,
// its values) is covered by the other rows of the SM: with one task a thread in
// flight and 16 CTAs an SM, 8192 rows of 32 + 8 + 8 heads of 128 take 32.3 us
// (6.2 TB/s of reads and writes, 92 % of a plain copy); three tasks in flight
// need 56 registers, 9 CTAs an SM and 8 us more; 256 threads a row 4 us more.

constexpr int ROPE_THREADS = 128, ROPE_CTAS = 16;  // a full SM: 32 registers a thread

template <int VEC>
struct alignas(2 * VEC) Run {
  uint16_t x[VEC];
};

template <int VEC>
__device__ __forceinline__ Run<VEC> load_run(const uint16_t* p) {
  Run<VEC> r;
  if constexpr (VEC == 8)
    *reinterpret_cast<uint4*>(r.x) = *reinterpret_cast<const uint4*>(p);
  else
    r.x[0] = *p;
  return r;
}

template <int VEC>
__device__ __forceinline__ void store_run(uint16_t* p, const Run<VEC>& r) {
  if constexpr (VEC == 8)
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(r.x);
  else
    *p = r.x[0];
}

// One task: a run of VEC values at `a` and one at `b` of a head, turned or not.
template <int VEC>
struct RopeTask {
  const uint16_t* src;
  uint16_t* dst;
  int a, b, c;    // c: the first pair's run, -1 when nothing turns
  bool two;       // an odd head_dim ends in a single value (VEC == 1)
  Run<VEC> ra, rb;
};

template <int VEC>
__global__ void __launch_bounds__(ROPE_THREADS, ROPE_CTAS) kda_rope_append_kernel(kda_rope_params p) {
  __shared__ float2 turn[128];  // mscale (cos, sin) of pair i
  const int t = blockIdx.x, tid = threadIdx.x;
  const int half = p.rotary_dim >> 1, D = p.cache.head_dim;
  const int Hq = p.num_q_heads, Hkv = p.cache.num_heads;
  const int per_head = (D + 2 * VEC - 1) / (2 * VEC), tasks = (Hq + 2 * Hkv) * per_head;
  earlier_work();
  const int pos = p.positions[t], slot = p.slots[t];
  const uint64_t freq = tid < half ? p.freqs[tid] : 0u;
  const uint16_t* const qi = static_cast<const uint16_t*>(p.q.ptr) + (int64_t)t * p.q.b_stride;
  const uint16_t* const ki = static_cast<const uint16_t*>(p.k.ptr) + (int64_t)t * p.k.b_stride;
  const uint16_t* const vi = static_cast<const uint16_t*>(p.v.ptr) + (int64_t)t * p.v.b_stride;
  // Per head D / (2 VEC) tasks (rounded up): first the pairs, then what passes unchanged.
  RopeTask<VEC> j;
  auto load = [&](int i) {
    const int h = i / per_head, c = i - h * per_head;
    j.src = h < Hq ? qi + (int64_t)h * p.q.h_stride
                   : h < Hq + Hkv ? ki + (int64_t)(h - Hq) * p.k.h_stride : vi + (int64_t)(h - Hq - Hkv) * p.v.h_stride;
    j.c = h < Hq + Hkv && c * VEC < half ? c * VEC : -1;
    j.a = 2 * c * VEC;
    j.b = j.a + VEC;
    if (j.c >= 0 && !p.interleaved) {
      j.a = j.c;
      j.b = j.a + half;
    }
    j.two = j.b < D;
    j.ra = load_run<VEC>(j.src + j.a);
    j.rb = j.ra;
    if (j.two) j.rb = load_run<VEC>(j.src + j.b);
  };
  // The first task's values are asked for before the position is known.
  if (tid < tasks) load(tid);

  if (pos < 0) return;
  if (tid < half) {  // half <= 128 = ROPE_THREADS
    // the exact phase in 2^-64 turns; its upper 32 bits as a signed number of half turns
    const uint64_t phase = (uint64_t)(uint32_t)pos * freq;
    float sn, cs;
    sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &sn, &cs);
    turn[tid] = make_float2(p.mscale * cs, p.mscale * sn);
  }
  const long long slots = (long long)p.cache.num_pages * p.cache.page_size;
  const bool append = slot >= 0 && slot < slots;
  if (!append && slot != -1 && tid == 0 && p.error_word) atomicOr(p.error_word, KDA_ERR_PAGES);
  const int64_t page = append ? slot / p.cache.page_size : 0, off = append ? slot % p.cache.page_size : 0;
  uint16_t* const ck = static_cast<uint16_t*>(p.cache.k.ptr) + page * p.cache.k.page_stride + off * p.cache.k.token_stride;
  uint16_t* const cv = static_cast<uint16_t*>(p.cache.v.ptr) + page * p.cache.v.page_stride + off * p.cache.v.token_stride;
  uint16_t* const qo = static_cast<uint16_t*>(p.q_out) + (int64_t)t * p.q_out_b_stride;
  __syncthreads();

  auto finish = [&](int i) {
    const int h = i / per_head;
    if (h >= Hq && !append) return;
    j.dst = h < Hq ? qo + (int64_t)h * p.q_out_h_stride
                   : h < Hq + Hkv ? ck + (int64_t)(h - Hq) * p.cache.k.head_stride
                                  : cv + (int64_t)(h - Hq - Hkv) * p.cache.v.head_stride;
    if (j.c >= 0) {
      if (VEC == 8 && p.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const int e0 = VEC == 8 ? e : 0, e1 = VEC == 8 ? e + 1 : 0;
          const float2 u = turn[(j.a + e) >> 1], w = turn[(j.b + e) >> 1];
          const float xa = bf16_bits_to_float(j.ra.x[e0]), ya = bf16_bits_to_float(j.ra.x[e1]);
          j.ra.x[e0] = float_to_bf16_bits(xa * u.x - ya * u.y);
          j.ra.x[e1] = float_to_bf16_bits(ya * u.x + xa * u.y);
          const float xb = bf16_bits_to_float(j.rb.x[e0]), yb = bf16_bits_to_float(j.rb.x[e1]);
          j.rb.x[e0] = float_to_bf16_bits(xb * w.x - yb * w.y);
          j.rb.x[e1] = float_to_bf16_bits(yb * w.x + xb * w.y);
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float2 u = turn[j.c + e];
          const float x = bf16_bits_to_float(j.ra.x[e]), y = bf16_bits_to_float(j.rb.x[e]);
          j.ra.x[e] = float_to_bf16_bits(x * u.x - y * u.y);
          j.rb.x[e] = float_to_bf16_bits(y * u.x + x * u.y);
        }
      }
    }
    store_run<VEC>(j.dst + j.a, j.ra);
    if (j.two) store_run<VEC>(j.dst + j.b, j.rb);
  };
  for (int i = tid; i < tasks;) {
    finish(i);
    i += ROPE_THREADS;
    if (i < tasks) load(i);
  }
}

cudaError_t launch_rope_append(const kda_rope_params& p, bool wide, cudaStream_t s) {
  const dim3 grid((unsigned)p.num_tokens);
  return wide ? launch_early(kda_rope_append_kernel<8>, grid, ROPE_THREADS, 0, s, p)
              : launch_early(kda_rope_append_kernel<1>, grid, ROPE_THREADS, 0, s, p);
}

// ---------------------------------------------------------------- attention on the CUDA cores
//
// A block per (row, query head), any head_dim, page size, stride and alignment.
// The row's keys go by in blocks of 32, in turn over the block's warps: lane j
// forms the whole score of key j (q in shared memory, its own key row), the warp
// joins the block's maximum and sum with its running ones, then the lanes hold
// the head's dimensions and add the 32 value rows, each weight broadcast from
// its lane. The warps' sums are joined in their order at the end. WIDE: rows on
// 16 bytes (and head_dim a multiple of 8), so that a lane reads 8 values of a
// key, and 2 of a value row, at a time.
//
// Bound by the issue of its loads and products: every query head of a group
// reads the keys again (from L2 or L1). 32 requests of 4000 tokens, 32 query
// heads over 8 of 96: 399 us, 0.98 TB/s of the cache's bytes (a warp a row with
// loads of single values: 2440); one such request of 1000 tokens 26 us (422);
// 512 new tokens over 2000: 2.6 ms (10.5).

constexpr int ATTN_WARPS = 8;
constexpr int ATTN_MAX_D = 256;

template <bool WIDE>
__global__ void __launch_bounds__(ATTN_WARPS * 32) kda_paged_attention_simt_kernel(kda_attention_params p) {
  __shared__ __align__(16) float qs[ATTN_MAX_D];
  __shared__ float part_o[ATTN_WARPS][ATTN_MAX_D], part_m[ATTN_WARPS], part_l[ATTN_WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int D = p.cache.head_dim, P = p.cache.page_size, g = p.num_q_heads / p.cache.num_heads;
  const uint16_t* const kc = static_cast<const uint16_t*>(p.cache.k.ptr);
  const uint16_t* const vc = static_cast<const uint16_t*>(p.cache.v.ptr);
  const int r = blockIdx.y;
  earlier_work();
  const AttnRequest q = attn_request(p, r);
  if (blockIdx.x == 0 && tid == 0 && q.bad && p.error_word) atomicOr(p.error_word, q.bad);
  const int32_t* const table = p.table + (int64_t)r * p.table_stride;
  const long long items = (long long)q.n * p.num_q_heads;
  bool bad_page = false;
  // the dimension that acc[i] of this lane holds
  auto dim = [&](int i) { return WIDE ? 64 * (i >> 1) + 2 * lane + (i & 1) : 32 * i + lane; };
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int j = (int)(it / p.num_q_heads), h = (int)(it % p.num_q_heads), hk = h / g;
    const int64_t row = (int64_t)q.row0 + j;
    const int pos = q.kv - q.n + j;
    const uint16_t* const qr = static_cast<const uint16_t*>(p.q.ptr) + row * p.q.b_stride + (int64_t)h * p.q.h_stride;
    if (tid < D) qs[tid] = bf16_bits_to_float(qr[tid]);
    __syncthreads();  // also: the row before has been put out
    const int lo = first_key(pos, p.window), hi = pos + 1;  // keys [lo, hi)
    float m = -INFINITY, l = 0.f, acc[ATTN_MAX_D / 32];
#pragma unroll
    for (int i = 0; i < ATTN_MAX_D / 32; ++i) acc[i] = 0.f;
    for (long long k0 = (long long)lo + warp * 32; k0 < hi; k0 += ATTN_WARPS * 32) {
      const int key = (int)k0 + lane;
      float s = -INFINITY;
      int page = -1, place = 0;
      if (key < hi) {
        page = table[key / P];
        place = key % P;
        if (page < 0 || page >= p.cache.num_pages) {
          page = -1;
          bad_page = true;
        }
        s = 0.f;
        if (page >= 0) {
          const uint16_t* const kr = kc + page * p.cache.k.page_stride + (int64_t)place * p.cache.k.token_stride +
                                     (int64_t)hk * p.cache.k.head_stride;
          if (WIDE) {
#pragma unroll 4
            for (int c = 0; c < D; c += 8) {
              const uint4 x = *reinterpret_cast<const uint4*>(kr + c);
              const float4 q0 = *reinterpret_cast<const float4*>(qs + c), q1 = *reinterpret_cast<const float4*>(qs + c + 4);
              s = fmaf(q0.x, __uint_as_float(x.x << 16), s);
              s = fmaf(q0.y, __uint_as_float(x.x & 0xffff0000u), s);
              s = fmaf(q0.z, __uint_as_float(x.y << 16), s);
              s = fmaf(q0.w, __uint_as_float(x.y & 0xffff0000u), s);
              s = fmaf(q1.x, __uint_as_float(x.z << 16), s);
              s = fmaf(q1.y, __uint_as_float(x.z & 0xffff0000u), s);
              s = fmaf(q1.z, __uint_as_float(x.w << 16), s);
              s = fmaf(q1.w, __uint_as_float(x.w & 0xffff0000u), s);
            }
          } else {
            for (int c = 0; c < D; ++c) s = fmaf(qs[c], bf16_bits_to_float(kr[c]), s);
          }
        }
        s *= p.scale;
      }
      float mb = s;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, o));
      const float mn = fmaxf(m, mb), base = mn == -INFINITY ? 0.f : mn;
      const float w = expf(s - base), fade = expf(m - base);
      l = l * fade + warp_sum(w);
      m = mn;
#pragma unroll
      for (int i = 0; i < ATTN_MAX_D / 32; ++i) acc[i] *= fade;
      const int count = (int)min(32LL, hi - k0);
#pragma unroll 4
      for (int u = 0; u < count; ++u) {
        const float wu = __shfl_sync(0xffffffffu, w, u);
        const int pu = __shfl_sync(0xffffffffu, page, u), at = __shfl_sync(0xffffffffu, place, u);
        if (pu < 0) continue;  // the same for the whole warp
        const uint16_t* const vr = vc + pu * p.cache.v.page_stride + (int64_t)at * p.cache.v.token_stride +
                                   (int64_t)hk * p.cache.v.head_stride;
        if (WIDE) {
#pragma unroll
          for (int i = 0; i < ATTN_MAX_D / 32; i += 2)
            if (dim(i) < D) {
              const uint32_t x = *reinterpret_cast<const uint32_t*>(vr + dim(i));
              acc[i] = fmaf(wu, __uint_as_float(x << 16), acc[i]);
              acc[i + 1] = fmaf(wu, __uint_as_float(x & 0xffff0000u), acc[i + 1]);
            }
        } else {
#pragma unroll
          for (int i = 0; i < ATTN_MAX_D / 32; ++i)
            if (dim(i) < D) acc[i] = fmaf(wu, bf16_bits_to_float(vr[dim(i)]), acc[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < ATTN_MAX_D / 32; ++i)
      if (dim(i) < D) part_o[warp][dim(i)] = acc[i];
    if (lane == 0) {
      part_m[warp] = m;
      part_l[warp] = l;
    }
    __syncthreads();
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < ATTN_WARPS; ++i) top = fmaxf(top, part_m[i]);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f, o = 0.f;
#pragma unroll
    for (int i = 0; i < ATTN_WARPS; ++i) {
      const float w = expf(part_m[i] - base);
      sum = fmaf(part_l[i], w, sum);
      if (tid < D) o = fmaf(part_o[i][tid], w, o);
    }
    const bool empty = hi <= lo;
    uint16_t* const out = static_cast<uint16_t*>(p.out) + row * p.out_b_stride + (int64_t)h * p.out_h_stride;
    if (tid < D) out[tid] = float_to_bf16_bits(empty ? 0.f : o / sum);
    if (p.lse != nullptr && tid == 0) p.lse[row * p.num_q_heads + h] = empty ? -INFINITY : top + logf(sum);
  }
  if (bad_page && p.error_word) atomicOr(p.error_word, KDA_ERR_PAGES);
}

cudaError_t launch_paged_attention_simt(const kda_attention_params& p, cudaStream_t s) {
  const long long rows = (long long)p.num_tokens * p.num_q_heads;
  const long long per = rows / p.num_requests + 1;
  const dim3 grid((unsigned)(per > 4096 ? 4096 : per), (unsigned)p.num_requests);
  auto rows16 = [](const kda_pages& g) {
    return (reinterpret_cast<uintptr_t>(g.ptr) & 15) == 0 && g.page_stride % 8 == 0 && g.token_stride % 8 == 0 &&
           g.head_stride % 8 == 0;
  };
  const bool wide = p.cache.head_dim % 8 == 0 && rows16(p.cache.k) && rows16(p.cache.v);
  return launch_early(wide ? kda_paged_attention_simt_kernel<true> : kda_paged_attention_simt_kernel<false>, grid,
                      ATTN_WARPS * 32, 0, s, p);
}

}  // namespace kda
