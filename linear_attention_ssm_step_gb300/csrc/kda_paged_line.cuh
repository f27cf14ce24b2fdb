// kda_paged_line.cuh - the line of units that the paged-attention kernels on the
// tensor cores share out, and what else they have in common.
//
// An item is one key-value head and w consecutive new tokens of one request (of
// the rows of all its query heads); its units are runs of 128 keys that any of
// its rows sees. The items of all requests form one line of units, which the
// persistent CTAs share out evenly, at any unit: lengths may be as ragged as
// they like and few rows over a long cache still fill the GPU. Every CTA finds
// its share itself from the requests' lengths, and one of its warps walks it.
#pragma once

#include "kda_fp8_codec.cuh"
#include "kda_paged.cuh"
#include "kda_tc.cuh"

namespace kda {

constexpr int UNIT = 128;   // keys a unit

// A run of units of one item, for one CTA.
struct Segment {
  int row0, ntok;        // first row of q, new tokens of the item
  int head;              // key-value head
  int pos0;              // position of the first token
  int request;
  int lo, hi;            // keys any of its rows sees: [lo, hi)
  int u0, u1;            // units of this run
  int dual;              // more tokens than a tile of rows holds: two tiles (kda_paged_tc.cu)
  int part, parts, cta0; // this run's place among the item's parts, held by the CTAs from cta0 on
};

// The keys [lo, hi) that item i (tokens i w .. of n, the first at position pos) sees, and its units.
struct Span {
  int lo, hi, u0, u1;
};

__device__ __forceinline__ Span item_span(int pos, int n, int i, int w, int window) {
  Span s;
  s.hi = max(0, pos + min(n, (i + 1) * w));
  s.lo = first_key(pos + i * w, window);
  if (s.hi == 0) s.lo = 0;
  s.u0 = s.lo / UNIT;
  s.u1 = max(s.u0 + 1, (s.hi + UNIT - 1) / UNIT);  // rows that see no key still need their zeros
  return s;
}

// Length on the line of one key-value head of a request: n tokens, w an item, which takes LEAD beside its units. Called by
// whole warps, one request a lane; a request of many items (a long chunk) is summed by the warp together.
template <int LEAD>
__device__ __forceinline__ int head_units(int pos, int n, int w, int window) {
  const int items = (n + w - 1) / w;
  int units = 0;
  if (items <= 4)
    for (int i = 0; i < items; ++i) {
      const Span s = item_span(pos, n, i, w, window);
      units += LEAD + s.u1 - s.u0;
    }
  unsigned many = __ballot_sync(0xffffffffu, items > 4);
  const int lane = threadIdx.x & 31;
  while (many) {
    const int src = __ffs(many) - 1;
    many &= many - 1;
    const int pn = __shfl_sync(0xffffffffu, pos, src), nn = __shfl_sync(0xffffffffu, n, src);
    const int ni = (nn + w - 1) / w;
    int part = 0;
    for (int i = lane; i < ni; i += 32) {
      const Span s = item_span(pn, nn, i, w, window);
      part += LEAD + s.u1 - s.u0;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    if (lane == src) units = part;
  }
  return units;
}

// ---------------------------------------------------------------- waits and votes

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// mbar_wait_bounded with the clock read only every 64th try: reading it takes longer than most of the waits here last.
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity) {
  unsigned long long t0 = 0;
#pragma unroll 1
  for (unsigned it = 1; it < WAIT_LIMIT_ITERS; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      const unsigned long long now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > WAIT_LIMIT_NS) return false;
    }
  }
  return false;
}

// A wait of a whole warp; false for every lane if it gave up for any. The first try, which mostly finds the phase done,
// is on its own, away from the bounded loop's counting: the warp that issues the products waits four times a pair of
// units (two chunks of 2048 tokens: 567 us against 584).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_bounded(bar, parity));
}

// A value that all lanes hold, for the compiler to keep in a uniform register.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }

__device__ __forceinline__ void mbar_init_only(uint64_t* bar, uint32_t count) {  // the fence follows
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}

// A barrier of `count` threads that tells all of them whether `x` held for any.
__device__ __forceinline__ bool bar_any(uint32_t id, uint32_t count, bool x) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)x), "r"(id), "r"(count)
      : "memory");
  return any != 0;
}

// 16 bytes from global to shared memory, asynchronously (both 16-byte aligned); the wait for all of this thread's.
__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// ---------------------------------------------------------------- numbers

// The largest of three (a NaN among them is passed over).
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / x and ln x to 2^-22 of themselves or better, for sums of weights: bf16 outputs and a log of fp32 terms need no more, and
// the exact forms are long code for once a run. Sums are from 2^-8 on, those of a cache in 8 bits, where weights hold value
// scales and sums do not, from 2^-34 to 2^70 and more: there a reference and the logarithm of its sum may be far larger than
// their sum, lse, which is then off by 2^-21 of the larger (1e-5 where the value scales are 2^-40).
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float ln(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y * 0.6931471805599453f;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t codes_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)two));
  return r;
}

__device__ __forceinline__ uint32_t f16x2_to_codes(uint32_t x) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// A query x as hi + lo, two E4M3 numbers of x 2^-e with the head's largest in (224, 448]. bf16's eight bits are four in
// each, exact down to 2^-2 (2^-9 of the largest or more); below, lo is off by half the subnormals' step, 2^-10, less than
// 2^-17 of the largest.
//
// The exponents e of N heads, each of which lies in LANES lanes, 8 numbers a lane. A head that is not finite has 128 (and
// NaN for codes).
template <int N, int LANES>
__device__ __forceinline__ void query_exponents(const uint4 (&z)[N], int (&e)[N]) {
  uint32_t top[N];  // largest magnitude as bf16 bits (a NaN is above infinity)
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t words[4] = {z[i].x, z[i].y, z[i].z, z[i].w};
    uint32_t t = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) t = __vmaxu2(t, words[j] & 0x7fff7fffu);
    top[i] = max(t >> 16, t & 0xffffu);
  }
#pragma unroll
  for (int o = LANES / 2; o >= 1; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) top[i] = max(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
#pragma unroll
  for (int i = 0; i < N; ++i)
    e[i] = top[i] >= 0x7f80u ? 128 : top[i] > 0 ? max(row_exponent(__uint_as_float(top[i] << 16)), -100) : 0;
}

// The codes of 8 numbers: the upper parts, and the lower ones.
__device__ __forceinline__ void query_codes(const uint4& z, int e, uint2& hi, uint2& lo) {
  const uint32_t words[4] = {z.x, z.y, z.z, z.w};
  const float down = e < 128 ? pow2f(-e) : __uint_as_float(0x7fc00000u);
  uint32_t h[4], r[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float u, w;
    unpack_bf16x2(words[j], u, w);
    const uint32_t x = pack_f16x2(u * down, w * down);  // exact: a step of fp16's subnormals is 2^-24
    h[j] = f16x2_to_codes(x);
    r[j] = f16x2_to_codes(sub_f16x2(x, codes_to_f16x2(h[j])));
  }
  hi = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  lo = make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
}

// 2^e for the scores, -100 <= e <= 128.
__device__ __forceinline__ float query_up(int e) { return pow2f(min(e, 127)); }

// ---------------------------------------------------------------- codes in shared memory

// K-major rows of D codes: 128 bytes with the 128-byte swizzle, or 64 bytes with the 64-byte swizzle (mode 4, 8-row groups
// 512 bytes apart; chunk c of row r sits at chunk c ^ (r / 2 % 4)).
template <int D>
__device__ __forceinline__ uint64_t code_desc(uint32_t saddr) {
  if constexpr (D == 128) return sw128_desc(saddr);
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1u << 16) | ((uint64_t)(512u >> 4) << 32) |
         ((uint64_t)1u << 46) | ((uint64_t)4u << 61);
}
template <int D>
__device__ __forceinline__ uint32_t code_chunk(uint32_t row, uint32_t c) {  // byte offset
  return D == 128 ? row * 128 + ((c ^ (row & 7)) << 4) : row * 64 + ((c ^ (row >> 1 & 3)) << 4);
}

// ---------------------------------------------------------------- the line

// Where a CTA's share begins: the request, and the first unit of the line that is the request's.
struct LineStart {
  AttnRequest request;
  int number, prefix;
};

// Its share: units [begin, end). The line is shared evenly over `ctas` CTAs, the first `rest` of which have share + 1.
struct LineShare {
  int ctas, share, rest, begin, end;
  unsigned bad;  // of the requests that this thread has looked at
};

// Called by all THREADS of a CTA; leaves `start` to be read after the next barrier. warp_sum: THREADS / 32 ints.
template <int THREADS, int LEAD>
__device__ __forceinline__ LineShare line_share(const kda_attention_params& p, int w, int* warp_sum, LineStart& start) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  LineShare line{0, 0, 0, 0, 0, 0u};
  int total = 0;
  AttnRequest mine_r{0, 0, 0, 0u};
  int mine = 0, before = 0;  // the units of this thread's request in the latest block, and those before it
  const int R = p.num_requests;
  const bool one_block = R <= THREADS;
  bool summed = false;  // warp_sum holds an earlier block's sums (of this pass or of the one before)
  auto block_units = [&](int base) {
    const int r = base + tid;
    mine_r = AttnRequest{0, 0, 0, 0u};
    if (r < R) mine_r = attn_request(p, r);
    line.bad |= mine_r.bad;
    mine = head_units<LEAD>(mine_r.kv - mine_r.n, mine_r.n, w, p.window) * p.cache.num_heads;
    int scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += x;
    }
    if (summed) __syncthreads();  // every warp has read the sums of the block before
    summed = true;
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    before = scan - mine;
    int all = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i < warp) before += warp_sum[i];
      all += warp_sum[i];
    }
    return all;
  };
  // Requests in one block are looked at once; else once for the sum and once to find where this CTA's share begins.
  const int cta = blockIdx.x;
  for (int pass = one_block ? 1 : 0; pass < 2; ++pass) {
    int prefix = 0;
    for (int base = 0; base < R; base += THREADS) {
      const int all = block_units(base);
      if (pass == 0 || one_block) total += all;
      if (pass == 0 && base + THREADS < R) continue;
      if (pass == 0 || one_block) {
        line.ctas = min(total, (int)gridDim.x);
        if (cta >= line.ctas) break;
        line.share = total / line.ctas;
        line.rest = total - line.share * line.ctas;
        line.begin = cta * line.share + min(cta, line.rest);
        line.end = line.begin + line.share + (cta < line.rest ? 1 : 0);
      }
      if (pass == 1 && line.begin >= prefix + before && line.begin < prefix + before + mine) {
        start.request = mine_r;
        start.number = base + tid;
        start.prefix = prefix + before;
      }
      prefix += all;
    }
    if (cta >= line.ctas) break;
  }
  return line;
}

// A barrier of the whole CTA, and the share's end: its begin where the requests' rows cannot be told apart.
__device__ __forceinline__ int line_end(const kda_attention_params& p, const LineShare& line) {
  if (!__syncthreads_or(line.bad & KDA_ERR_SEQLENS)) return line.end;
  // Ranges can share rows only where some bounds are out of order. Together they may then hold more rows than there are,
  // for which the sums above are not made (32 bits): nothing is done.
  long long rows = 0;
  for (int r = threadIdx.x & 31; r < p.num_requests; r += 32) rows += attn_request(p, r).n;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) rows += __shfl_xor_sync(0xffffffffu, rows, o);
  return rows > p.num_tokens ? line.begin : line.end;
}

// Cuts the share's units [line.begin, end) into segments, one after another to put(Segment), which returns whether to go on.
// Called by a whole warp. False if put gave up.
template <int LEAD, typename Put>
__device__ __forceinline__ bool line_walk(const kda_attention_params& p, int w, const LineShare& line, int end,
                                          const LineStart& start, Put&& put) {
  const int lane = threadIdx.x & 31, cta = blockIdx.x, window = p.window, Hkv = p.cache.num_heads;
  const int begin = line.begin, share = line.share, rest = line.rest;
  int r = start.number;
  int at = begin;
  int prefix = start.prefix;  // first unit of the current head's first item
  int head = 0, item = 0;
  bool fresh = true;  // the place inside request r is still to be found
  while (at < end && r < p.num_requests) {
    const AttnRequest q = fresh ? start.request : attn_request(p, r);
    const int pos = q.kv - q.n, items = (q.n + w - 1) / w;
    if (fresh) {
      // whole heads first, then 32 items at a time
      int uh;
      if (items == 1) {
        const Span s = item_span(pos, q.n, 0, w, window);
        uh = LEAD + s.u1 - s.u0;
      } else {
        uh = __shfl_sync(0xffffffffu, head_units<LEAD>(pos, lane == 0 ? q.n : 0, w, window), 0);
      }
      head = (at - prefix) / uh;
      prefix += uh * head;
      item = 0;
      for (int base = 0; items > 1 && base < items; base += 32) {
        const int i = base + lane;
        int u = 0;
        if (i < items) {
          const Span s = item_span(pos, q.n, i, w, window);
          u = LEAD + s.u1 - s.u0;
        }
        int scan = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, scan, o);
          if (lane >= o) scan += x;
        }
        const bool here = i < items && prefix + scan > at;
        const unsigned found = __ballot_sync(0xffffffffu, here);
        if (found) {
          const int src = __ffs(found) - 1;
          item = base + src;
          prefix += __shfl_sync(0xffffffffu, scan - u, src);
          break;
        }
        prefix += __shfl_sync(0xffffffffu, scan, 31);
      }
      fresh = false;
    }
    // `prefix` is the first unit of item `item` of head `head`
    while (at < end && head < Hkv && items > 0) {
      const Span s = item_span(pos, q.n, item, w, window);
      const int units0 = prefix + LEAD, item_end = units0 + (s.u1 - s.u0);
      const int from = max(at, units0), stop = min(end, item_end);
      at = stop;
      prefix = item_end;
      const int i = item;
      if (++item == items) {
        item = 0;
        ++head;
      }
      if (from >= stop) continue;  // the share ends before the item's first unit
      Segment g;
      g.row0 = q.row0 + i * w;
      g.ntok = min(q.n - i * w, w);
      g.head = item == 0 ? head - 1 : head;
      g.pos0 = pos + i * w;
      g.request = r;
      g.lo = s.lo;
      g.hi = s.hi;
      g.u0 = s.u0 + (from - units0);
      g.u1 = s.u0 + (stop - units0);
      g.dual = 0;
      // the CTA that holds unit x of the line
      auto holder = [&](int x) {
        if (x >= begin && x < end) return cta;
        const int longer = rest * (share + 1);
        return x < longer ? x / (share + 1) : rest + (x - longer) / share;
      };
      g.cta0 = holder(units0);
      g.parts = holder(item_end - 1) - g.cta0 + 1;
      g.part = cta - g.cta0;
      if (!put(g)) return false;
    }
    ++r;
    head = item = 0;
  }
  Segment last{};
  last.ntok = -1;
  return put(last);
}

}  // namespace kda
