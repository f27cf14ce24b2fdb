// kda_paged_fp8.cu - the append to a paged cache held in 8 bits, and reading it
// back (include/kda_paged_fp8.h).
#include <type_traits>

#include "kda_device.cuh"
#include "kda_fp8_codec.cuh"
#include "kda_paged.cuh"
#include "kda_paged_launch.h"
#include "kda_rope.cuh"

namespace kda {

constexpr int SCALE_TOKENS = KDA_FP8_SCALE_TOKENS;
constexpr int SCALE_LOW = -40, SCALE_HIGH = 40;  // exponents of the scales

// ---------------------------------------------------------------- append
//
// One CTA per row turns the row's queries as kda_rope_append_kernel does. Keys
// and values go by the block: a scale needs the largest magnitude of all the
// rows that fall into one block (a run: at most 16 rows that follow one
// another), so a warp takes one side and head of a whole run. The run's CTAs
// share its 2 x heads such tasks evenly, CTA i of n taking every n-th: a chunk
// has as much to do in each CTA as a decode step, whose runs are single rows.
// Every CTA finds its run itself, from the slots of the 15 rows on either side.
//
// A task reads its rows once, into registers as bf16 (two a lane and row for
// head_dim 128), goes over them for the largest magnitude, and again to encode.
// Keys are turned in both passes, by sines and cosines of all the run's rows
// that the CTA's threads leave in shared memory; these are the fast ones (off
// by 2^-20, where a code rounds by 2^-4), since each of up to 16 CTAs forms
// them. Other head sizes, and rows off their alignment, read the rows twice.

constexpr int APPEND_THREADS = 128, APPEND_WARPS = APPEND_THREADS / 32;

// A run: rows t0 .. t0 + n - 1, at tokens first .. of a block; i: this CTA's row of it.
struct BlockRun {
  int t0, n, i;
  int page, block, first;
};

// The run of row t, whose slot is in the cache. Called by whole warps.
__device__ __forceinline__ BlockRun block_run(const kda_rope_params& p, int t, int slot) {
  const int lane = threadIdx.x & 31, P = p.cache.page_size;
  BlockRun r;
  r.page = slot / P;
  const int place = slot - r.page * P;
  r.block = place / SCALE_TOKENS;
  const int off = place - r.block * SCALE_TOKENS, size = min(SCALE_TOKENS, P - r.block * SCALE_TOKENS);
  const int d = lane - 15;  // -15 .. 16; 16 is never in the block
  bool in = false;
  if (off + d >= 0 && off + d < size && (long long)t + d >= 0 && (long long)t + d < p.num_tokens)
    in = p.positions[t + d] >= 0 && p.slots[t + d] == slot + d;
  const uint32_t rows = __ballot_sync(0xffffffffu, in);  // bit 15 (row t) is set
  r.i = __clz(~(rows << 17));                            // rows right before t
  r.n = r.i + __ffs(~(rows >> 15)) - 1;
  r.t0 = t - r.i;
  r.first = off - r.i;
  return r;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// The scale of a block: the exponent that its new rows need, and what its earlier tokens (if any) have. `old` is read where
// there are some.
struct BlockScale {
  float scale, inverse;
  float again;  // what the earlier tokens' codes are multiplied by, 0: they stay
};

__device__ __forceinline__ BlockScale new_scale(float top, bool earlier, float old) {
  const int e = top > 0.f ? min(max(row_exponent(top), SCALE_LOW), SCALE_HIGH) : SCALE_LOW;
  const float need = pow2f(e);
  BlockScale b;
  b.scale = earlier ? fmaxf(old, need) : need;
  b.inverse = 1.f / b.scale;  // exact for a power of two
  b.again = earlier && need > old ? old / need : 0.f;
  return b;
}

__device__ __forceinline__ uint32_t encode4(const float* x, float inverse) {
  return f32x2_to_e4m3x2(pk2(x[0] * inverse, x[1] * inverse)) |
         (f32x2_to_e4m3x2(pk2(x[2] * inverse, x[3] * inverse)) << 16);
}

// One side and head of a run, E consecutive elements a lane and row (32 E = head_dim).
template <int E>
__device__ __forceinline__ void append_wide(const kda_rope_params& p, const BlockRun& run, const uint16_t* src,
                                            int64_t row_stride, uint8_t* block, int64_t token_stride, float* scale,
                                            const float2 (*turn)[128], bool turned) {
  const int lane = threadIdx.x & 31, half = p.rotary_dim >> 1;
  constexpr int W = E / 2;  // words a row
  using Codes = std::conditional_t<E == 4, uint32_t, uint16_t>;
  const float old = run.first > 0 ? *scale : 0.f;
  uint32_t raw[SCALE_TOKENS][W];
#pragma unroll
  for (int i = 0; i < SCALE_TOKENS; ++i) {
    const uint16_t* const row = src + i * row_stride + lane * E;
#pragma unroll
    for (int w = 0; w < W; ++w) raw[i][w] = 0;
    if (i < run.n) {
      if constexpr (E == 4)
        *reinterpret_cast<uint2*>(raw[i]) = *reinterpret_cast<const uint2*>(row);
      else
        raw[i][0] = *reinterpret_cast<const uint32_t*>(row);
    }
  }
  const bool mine = turned && lane * E < p.rotary_dim, lower = lane * E < half;
  const int partner = !mine || p.interleaved ? lane : lower ? lane + half / E : lane - half / E;
  const int pair = p.interleaved ? lane * W : lower ? lane * E : lane * E - half;
  auto row_values = [&](int i, float (&x)[E]) {
#pragma unroll
    for (int w = 0; w < W; ++w) unpack_bf16x2(raw[i][w], x[2 * w], x[2 * w + 1]);
    if (!turned) return;
    const float2* const u = turn[i] + pair;
    if (p.interleaved) {
      if (!mine) return;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float a = x[2 * w], b = x[2 * w + 1];
        x[2 * w] = a * u[w].x - b * u[w].y;
        x[2 * w + 1] = b * u[w].x + a * u[w].y;
      }
    } else {
      float y[E];
#pragma unroll
      for (int w = 0; w < W; ++w) unpack_bf16x2(__shfl_sync(0xffffffffu, raw[i][w], partner), y[2 * w], y[2 * w + 1]);
      if (!mine) return;
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = lower ? x[e] * u[e].x - y[e] * u[e].y : x[e] * u[e].x + y[e] * u[e].y;
    }
  };
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < SCALE_TOKENS; ++i) {
    if (i >= run.n) break;  // the same for the whole warp
    float x[E];
    row_values(i, x);
#pragma unroll
    for (int e = 0; e < E; ++e) top = fmaxf(top, fabsf(x[e]));
  }
  const BlockScale b = new_scale(warp_max(top), run.first > 0, old);
  uint8_t* const at = block + lane * E;
  if (b.again > 0.f) {
#pragma unroll 1
    for (int j = 0; j < run.first; ++j) {
      Codes* const c = reinterpret_cast<Codes*>(at + j * token_stride);
      float x[4] = {};
      e4m3x4_to_floats(*c, x);
      *c = (Codes)encode4(x, b.again);
    }
  }
#pragma unroll
  for (int i = 0; i < SCALE_TOKENS; ++i) {
    if (i >= run.n) break;
    float x[E], z[4] = {};
    row_values(i, x);
#pragma unroll
    for (int e = 0; e < E; ++e) z[e] = x[e];
    *reinterpret_cast<Codes*>(at + (run.first + i) * token_stride) = (Codes)encode4(z, b.inverse);
  }
  if (lane == 0) *scale = b.scale;
}

// The same for any head_dim and alignment, an element at a time.
__device__ __forceinline__ void append_any(const kda_rope_params& p, const BlockRun& run, const uint16_t* src,
                                           int64_t row_stride, uint8_t* block, int64_t token_stride, float* scale,
                                           const float2 (*turn)[128], bool turned) {
  const int lane = threadIdx.x & 31, half = p.rotary_dim >> 1, D = p.cache.head_dim;
  const float old = run.first > 0 ? *scale : 0.f;
  auto value = [&](int i, int c) {
    const uint16_t* const row = src + i * row_stride;
    const float x = bf16_bits_to_float(row[c]);
    if (!turned || c >= p.rotary_dim) return x;
    const bool lower = p.interleaved ? c % 2 == 0 : c < half;
    const int step = p.interleaved ? 1 : half;
    const float y = bf16_bits_to_float(row[lower ? c + step : c - step]);
    const float2 u = turn[i][p.interleaved ? c >> 1 : lower ? c : c - half];
    return lower ? x * u.x - y * u.y : x * u.x + y * u.y;
  };
  float top = 0.f;
  for (int i = 0; i < run.n; ++i)
    for (int c = lane; c < D; c += 32) top = fmaxf(top, fabsf(value(i, c)));
  const BlockScale b = new_scale(warp_max(top), run.first > 0, old);
  if (b.again > 0.f)
    for (int j = 0; j < run.first; ++j)
      for (int c = lane; c < D; c += 32) {
        uint8_t* const code = block + j * token_stride + c;
        *code = (uint8_t)f32x2_to_e4m3x2(pk2(e4m3_to_float(*code) * b.again, 0.f));
      }
  for (int i = 0; i < run.n; ++i)
    for (int c = lane; c < D; c += 32)
      block[(run.first + i) * token_stride + c] = (uint8_t)f32x2_to_e4m3x2(pk2(value(i, c) * b.inverse, 0.f));
  if (lane == 0) *scale = b.scale;
}

// Sine and cosine of a phase in 2^-64 turns, off by 2^-20 at most.
__device__ __forceinline__ float2 fast_turn(uint64_t phase, float mscale) {
  const float angle = (float)(int32_t)(phase >> 32) * 1.4629180792671596e-09f;  // pi 2^-31: within [-pi, pi]
  return make_float2(mscale * __cosf(angle), mscale * __sinf(angle));
}

template <int VEC, int E>
__global__ void __launch_bounds__(APPEND_THREADS) kda_rope_append_fp8_kernel(kda_rope_params p, kda_paged_scales sc) {
  __shared__ float2 turn[128];                                     // mscale (cos, sin) of this row's pairs
  __shared__ __align__(16) float2 run_turn[SCALE_TOKENS][128];     // and of the run's rows
  const int t = blockIdx.x, tid = threadIdx.x, warp = tid >> 5;
  const int half = p.rotary_dim >> 1, D = p.cache.head_dim;
  const int Hq = p.num_q_heads, Hkv = p.cache.num_heads;
  const int per_head = (D + 2 * VEC - 1) / (2 * VEC), tasks = Hq * per_head;
  earlier_work();
  const int pos = p.positions[t], slot = p.slots[t];
  const uint64_t freq = tid < half ? p.freqs[tid] : 0u;
  const uint16_t* const qi = static_cast<const uint16_t*>(p.q.ptr) + (int64_t)t * p.q.b_stride;
  RopeTask<VEC> j;
  auto load = [&](int i) {
    const int h = i / per_head, c = i - h * per_head;
    j.src = qi + (int64_t)h * p.q.h_stride;
    j.c = c * VEC < half ? c * VEC : -1;
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
  if (tid < tasks) load(tid);  // asked for before the position is known

  if (pos < 0) return;
  if (tid < half) {  // half <= 128 = APPEND_THREADS
    const uint64_t phase = (uint64_t)(uint32_t)pos * freq;
    float sn, cs;
    sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &sn, &cs);
    turn[tid] = make_float2(p.mscale * cs, p.mscale * sn);
  }
  const long long slots = (long long)p.cache.num_pages * p.cache.page_size;
  const bool append = slot >= 0 && slot < slots;
  if (!append && slot != -1 && tid == 0 && p.error_word) atomicOr(p.error_word, KDA_ERR_PAGES);
  BlockRun run{};
  if (append) {
    run = block_run(p, t, slot);
    if (run.i < Hkv)  // its first task is one of keys
      for (int x = tid; x < run.n * half; x += APPEND_THREADS) {
        const int i = x / half, c = x - i * half;
        run_turn[i][c] = fast_turn((uint64_t)(uint32_t)p.positions[run.t0 + i] * p.freqs[c], p.mscale);
      }
  }
  __syncthreads();

  uint16_t* const qo = static_cast<uint16_t*>(p.q_out) + (int64_t)t * p.q_out_b_stride;
  for (int i = tid; i < tasks;) {
    if (j.c >= 0) turn_task<VEC>(j, turn, p.interleaved);
    j.dst = qo + (int64_t)(i / per_head) * p.q_out_h_stride;
    store_run<VEC>(j.dst + j.a, j.ra);
    if (j.two) store_run<VEC>(j.dst + j.b, j.rb);
    i += APPEND_THREADS;
    if (i < tasks) load(i);
  }
  if (!append) return;
  for (int x = run.i + run.n * warp; x < 2 * Hkv; x += run.n * APPEND_WARPS) {
    const bool keys = x < Hkv;
    const int h = keys ? x : x - Hkv;
    const kda_view& v = keys ? p.k : p.v;
    const kda_pages& g = keys ? p.cache.k : p.cache.v;
    const kda_page_scales& f = keys ? sc.k : sc.v;
    const uint16_t* const src =
        static_cast<const uint16_t*>(v.ptr) + (int64_t)run.t0 * v.b_stride + (int64_t)h * v.h_stride;
    uint8_t* const block = static_cast<uint8_t*>(g.ptr) + (int64_t)run.page * g.page_stride +
                           (int64_t)run.block * SCALE_TOKENS * g.token_stride + (int64_t)h * g.head_stride;
    float* const scale = f.ptr + (int64_t)run.page * f.page_stride + (int64_t)run.block * f.block_stride +
                         (int64_t)h * f.head_stride;
    if constexpr (E > 0)
      append_wide<E>(p, run, src, v.b_stride, block, g.token_stride, scale, run_turn, keys && half > 0);
    else
      append_any(p, run, src, v.b_stride, block, g.token_stride, scale, run_turn, keys && half > 0);
  }
}

cudaError_t launch_rope_append_fp8(const kda_rope_params& p, const kda_paged_scales& sc, bool q_wide, int lane_elems,
                                   cudaStream_t s) {
  const dim3 grid((unsigned)p.num_tokens);
  auto go = [&](auto kernel) { return launch_early(kernel, grid, APPEND_THREADS, 0, s, p, sc); };
  if (lane_elems == 4) return q_wide ? go(kda_rope_append_fp8_kernel<8, 4>) : go(kda_rope_append_fp8_kernel<1, 4>);
  if (lane_elems == 2) return q_wide ? go(kda_rope_append_fp8_kernel<8, 2>) : go(kda_rope_append_fp8_kernel<1, 2>);
  return q_wide ? go(kda_rope_append_fp8_kernel<8, 0>) : go(kda_rope_append_fp8_kernel<1, 0>);
}

// ---------------------------------------------------------------- read
//
// A CTA per 16 packed rows: its threads go through the requests, and each
// request marks the rows of the tile that it covers; 16 threads then find their
// rows' pages; then all copy, 16 codes and 32 bytes of output a thread at a time
// where the rows allow it. Bound by memory: a byte in and two out an element.

constexpr int READ_THREADS = 256, READ_ROWS = 16;

struct ReadRow {
  int page, place;  // page -1: zeros, -2: not written
};

template <bool WIDE>
__global__ void __launch_bounds__(READ_THREADS) kda_paged_read_fp8_kernel(kda_read_params p, kda_paged_scales sc) {
  __shared__ int owner[READ_ROWS];
  __shared__ ReadRow rows[READ_ROWS];
  const int tid = threadIdx.x, R = p.num_requests;
  const int row0 = (int)blockIdx.x * READ_ROWS;
  const int Hkv = p.cache.num_heads, D = p.cache.head_dim, P = p.cache.page_size;
  if (tid < READ_ROWS) owner[tid] = -1;
  earlier_work();
  __syncthreads();
  for (int r = tid; r < R; r += READ_THREADS) {
    const AttnRequest q = paged_request(p, p.cu_rows, r);
    if (blockIdx.x == 0 && q.bad && p.error_word) atomicOr(p.error_word, q.bad);
    for (int i = max(q.row0 - row0, 0); i < min(q.row0 - row0 + q.n, READ_ROWS); ++i) owner[i] = r;
  }
  __syncthreads();
  if (tid < READ_ROWS) {
    ReadRow x{-2, 0};
    const int r = owner[tid];
    if (r >= 0) {
      const AttnRequest q = paged_request(p, p.cu_rows, r);
      const int token = q.kv - q.n + (row0 + tid - q.row0);
      x.page = -1;
      if (token >= 0) {
        x.page = p.table[(int64_t)r * p.table_stride + token / P];
        x.place = token % P;
        if (x.page < 0 || x.page >= p.cache.num_pages) {
          x.page = -1;
          if (p.error_word) atomicOr(p.error_word, KDA_ERR_PAGES);
        }
      }
    }
    rows[tid] = x;
  }
  __syncthreads();
  constexpr int V = WIDE ? 16 : 1;  // elements at a time
  const int per_head = D / V, per_row = 2 * Hkv * per_head;
  for (int x = tid; x < READ_ROWS * per_row; x += READ_THREADS) {
    const int i = x / per_row, y = x - i * per_row, side_head = y / per_head, c = (y - side_head * per_head) * V;
    const bool keys = side_head < Hkv;
    const int h = keys ? side_head : side_head - Hkv;
    const ReadRow row = rows[i];
    if (row.page == -2) continue;
    uint16_t* const out = keys ? static_cast<uint16_t*>(p.k_out) + (int64_t)(row0 + i) * p.k_out_b_stride + (int64_t)h * p.k_out_h_stride + c
                               : static_cast<uint16_t*>(p.v_out) + (int64_t)(row0 + i) * p.v_out_b_stride + (int64_t)h * p.v_out_h_stride + c;
    const kda_pages& g = keys ? p.cache.k : p.cache.v;
    const uint8_t* const codes = static_cast<const uint8_t*>(g.ptr) + (int64_t)row.page * g.page_stride +
                                 (int64_t)row.place * g.token_stride + (int64_t)h * g.head_stride + c;
    const float scale = row.page >= 0 ? block_scale(keys ? sc.k : sc.v, row.page, row.place, h) : 0.f;
    if constexpr (WIDE) {
      uint4 in = make_uint4(0, 0, 0, 0);
      if (row.page >= 0) in = *reinterpret_cast<const uint4*>(codes);
      const uint32_t words[4] = {in.x, in.y, in.z, in.w};
      uint32_t b[8];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        float f[4];
        e4m3x4_to_floats(words[w], f);
        b[2 * w] = pack_bf16x2(f[0] * scale, f[1] * scale);
        b[2 * w + 1] = pack_bf16x2(f[2] * scale, f[3] * scale);
      }
      reinterpret_cast<uint4*>(out)[0] = make_uint4(b[0], b[1], b[2], b[3]);
      reinterpret_cast<uint4*>(out)[1] = make_uint4(b[4], b[5], b[6], b[7]);
    } else {
      *out = row.page >= 0 ? float_to_bf16_bits(e4m3_to_float(*codes) * scale) : (uint16_t)0;
    }
  }
}

cudaError_t launch_paged_read_fp8(const kda_read_params& p, const kda_paged_scales& sc, bool wide, cudaStream_t s) {
  const dim3 grid((unsigned)(p.num_tokens / READ_ROWS + (p.num_tokens % READ_ROWS != 0)));
  return launch_early(wide ? kda_paged_read_fp8_kernel<true> : kda_paged_read_fp8_kernel<false>, grid, READ_THREADS, 0, s,
                      p, sc);
}

}  // namespace kda
