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
// A CTA per row turns its queries, as kda_rope_append_kernel does. Keys and
// values, in CTAs beside those, go by the block: a scale needs the largest
// magnitude of all the rows that fall into one block (a run: at most 16 rows,
// consecutive but for some that are not stored). A CTA has the runs that begin
// among its `span` rows, found from the positions and slots of these and of the 15
// before and behind; a task is one side and head of a run, and a warp takes it
// whole, reads its rows once, into registers as bf16 (two a lane and row for
// head_dim 128), goes over them for the largest magnitude, and again to encode.
// Keys are turned in both passes, by sines and cosines that the CTA forms once for
// all heads, in shared memory, by the fast functions (off by 2^-20, where a code
// rounds by 2^-4). Other head sizes, rows off their alignment and runs with rows
// left out read the rows twice (asking for every row of a run whether it is stored
// cost the chunk below 1.3 us more).
//
// Measured: 8192 rows of 32 + 8 + 8 heads of 128, 44 us, of which the queries 20
// and keys and values 23 to 30, bound by latency: 1400 instructions a task, issued
// in a third of the cycles. A CTA per row with its share of the run's tasks (each
// forming the run's sines and cosines again): 58 us; one with four warps a task
// and the turn in registers, 52 to 69. 256 decode rows 6.4 to 8.9 us: a launch, the
// slots, the rows and scales, the codes.

// A run: rows t0 .. t0 + n - 1, at tokens first .. of a block; those that are stored as bits, of which the first and the last
// are set.
struct BlockRun {
  int t0, n;
  uint32_t rows;
  int page, block, first;
};

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
  // 2^-e of a power of two 2^e, |e| < 127, by its exponent field (a division is a long subroutine)
  auto inverse = [](float x) { return __uint_as_float((254u << 23) - (__float_as_uint(x) & 0x7f800000u)); };
  b.inverse = inverse(b.scale);
  b.again = earlier && need > old ? old * inverse(need) : 0.f;
  return b;
}

__device__ __forceinline__ uint32_t encode4(const float* x, float inverse) {
  return f32x2_to_e4m3x2(pk2(x[0] * inverse, x[1] * inverse)) |
         (f32x2_to_e4m3x2(pk2(x[2] * inverse, x[3] * inverse)) << 16);
}

// One side and head of a run: where it lies.
struct BlockTask {
  const uint16_t* src;  // its first row
  int64_t row_stride, token_stride;
  uint8_t* block;       // codes of the block's first token
  float* scale;
  bool turned;
};

// The rows of a task, E consecutive elements a lane and row (32 E = head_dim), two a word.
template <int E>
struct RunRows {
  uint32_t raw[SCALE_TOKENS][E / 2];
  float old;  // the block's scale, where it has earlier tokens
};

template <int E>
__device__ __forceinline__ void load_rows(const BlockRun& run, const BlockTask& k, RunRows<E>& z) {
  const int lane = threadIdx.x & 31;
  z.old = run.first > 0 ? *k.scale : 0.f;
#pragma unroll
  for (int i = 0; i < SCALE_TOKENS; ++i) {
    const uint16_t* const row = k.src + i * k.row_stride + lane * E;
    if (i >= run.n) break;  // the same for the whole warp
    if constexpr (E == 4) {
      const uint2 x = *reinterpret_cast<const uint2*>(row);
      z.raw[i][0] = x.x;
      z.raw[i][1] = x.y;
    } else {
      z.raw[i][0] = *reinterpret_cast<const uint32_t*>(row);
    }
  }
}

// table: sines and cosines of the run's rows, rotary_dim / 2 a row.
template <int E>
__device__ __forceinline__ void append_rows(const kda_rope_params& p, const BlockRun& run, const BlockTask& k,
                                            const RunRows<E>& z, const float2* table) {
  const int lane = threadIdx.x & 31, half = p.rotary_dim >> 1;
  constexpr int W = E / 2;
  using Codes = std::conditional_t<E == 4, uint32_t, uint16_t>;
  const bool mine = k.turned && lane * E < p.rotary_dim, lower = lane * E < half;
  const int partner = !mine || p.interleaved ? lane : lower ? lane + half / E : lane - half / E;
  const int pair = p.interleaved ? lane * W : lower ? lane * E : lane * E - half;
  auto row_values = [&](int i, float (&x)[E]) {
#pragma unroll
    for (int w = 0; w < W; ++w) unpack_bf16x2(z.raw[i][w], x[2 * w], x[2 * w + 1]);
    if (!k.turned) return;
    const float2* const u = table + i * half + pair;
    if (p.interleaved) {
      if (!mine) return;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float a = x[2 * w], b = x[2 * w + 1];
        x[2 * w] = fmaf(a, u[w].x, -b * u[w].y);
        x[2 * w + 1] = fmaf(b, u[w].x, a * u[w].y);
      }
    } else {
      float y[E];
#pragma unroll
      for (int w = 0; w < W; ++w) unpack_bf16x2(__shfl_sync(0xffffffffu, z.raw[i][w], partner), y[2 * w], y[2 * w + 1]);
      if (!mine) return;
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = fmaf(x[e], u[e].x, lower ? -y[e] * u[e].y : y[e] * u[e].y);
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
  const BlockScale b = new_scale(warp_max(top), run.first > 0, z.old);
  uint8_t* const at = k.block + lane * E;
  if (b.again > 0.f) {
    constexpr int AT_ONCE = 5;  // tokens a trip to memory: all 15 in three
    for (int j0 = 0; j0 < run.first; j0 += AT_ONCE) {
      Codes c[AT_ONCE];
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j)
        if (j0 + j < run.first) c[j] = *reinterpret_cast<const Codes*>(at + (j0 + j) * k.token_stride);
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j) {
        if (j0 + j >= run.first) break;
        float four[4] = {};
        e4m3x4_to_floats(c[j], four);
        *reinterpret_cast<Codes*>(at + (j0 + j) * k.token_stride) = (Codes)encode4(four, b.again);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < SCALE_TOKENS; ++i) {
    if (i >= run.n) break;
    float x[E], four[4] = {};
    row_values(i, x);
#pragma unroll
    for (int e = 0; e < E; ++e) four[e] = x[e];
    *reinterpret_cast<Codes*>(at + (run.first + i) * k.token_stride) = (Codes)encode4(four, b.inverse);
  }
  if (lane == 0) *k.scale = b.scale;
}

// A task for any head_dim and alignment, an element at a time.
__device__ __forceinline__ void append_any(const kda_rope_params& p, const BlockRun& run, const BlockTask& k, const float2* table) {
  const int lane = threadIdx.x & 31, half = p.rotary_dim >> 1, D = p.cache.head_dim;
  const float old = run.first > 0 ? *k.scale : 0.f;
  auto value = [&](int i, int c) {
    const uint16_t* const row = k.src + i * k.row_stride;
    const float x = bf16_bits_to_float(row[c]);
    if (!k.turned || c >= p.rotary_dim) return x;
    const bool lower = p.interleaved ? c % 2 == 0 : c < half;
    const int step = p.interleaved ? 1 : half;
    const float y = bf16_bits_to_float(row[lower ? c + step : c - step]);
    const float2 u = table[i * half + (p.interleaved ? c >> 1 : lower ? c : c - half)];
    return fmaf(x, u.x, lower ? -y * u.y : y * u.y);
  };
  float top = 0.f;
  for (int i = 0; i < run.n; ++i)
    for (int c = lane; run.rows >> i & 1u && c < D; c += 32) top = fmaxf(top, fabsf(value(i, c)));
  const BlockScale b = new_scale(warp_max(top), run.first > 0, old);
  if (b.again > 0.f)
    for (int j = 0; j < run.first; ++j)
      for (int c = lane; c < D; c += 32) {
        uint8_t* const code = k.block + j * k.token_stride + c;
        *code = (uint8_t)f32x2_to_e4m3x2(pk2(e4m3_to_float(*code) * b.again, 0.f));
      }
  for (int i = 0; i < run.n; ++i)
    for (int c = lane; run.rows >> i & 1u && c < D; c += 32)
      k.block[(run.first + i) * k.token_stride + c] = (uint8_t)f32x2_to_e4m3x2(pk2(value(i, c) * b.inverse, 0.f));
  if (lane == 0) *k.scale = b.scale;
}

// Sine and cosine of a phase in 2^-64 turns, off by 2^-20 at most.
__device__ __forceinline__ float2 fast_turn(uint64_t phase, float mscale) {
  const float angle = (float)(int32_t)(phase >> 32) * 1.4629180792671596e-09f;  // pi 2^-31: within [-pi, pi]
  return make_float2(mscale * __cosf(angle), mscale * __sinf(angle));
}

constexpr int APPEND_WARPS = 8;  // a CTA

// The queries of row t.
template <int VEC>
__device__ __forceinline__ void turn_queries(const kda_rope_params& p, int t) {
  __shared__ float2 turn[128];  // mscale (cos, sin) of pair i
  const int tid = threadIdx.x, half = p.rotary_dim >> 1, D = p.cache.head_dim;
  const int per_head = (D + 2 * VEC - 1) / (2 * VEC), tasks = p.num_q_heads * per_head;
  const int pos = p.positions[t];
  const uint64_t freq = tid < half ? p.freqs[tid] : 0u;  // half <= 128, the fewest threads
  const uint16_t* const qi = static_cast<const uint16_t*>(p.q.ptr) + (int64_t)t * p.q.b_stride;
  uint16_t* const qo = static_cast<uint16_t*>(p.q_out) + (int64_t)t * p.q_out_b_stride;
  RopeTask<VEC> j;
  auto load = [&](int i) {
    const int h = i / per_head, c = i - h * per_head;
    j.src = qi + (int64_t)h * p.q.h_stride;
    j.dst = qo + (int64_t)h * p.q_out_h_stride;
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
  if (tid < half) {
    const uint64_t phase = (uint64_t)(uint32_t)pos * freq;
    float sn, cs;
    sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &sn, &cs);
    turn[tid] = make_float2(p.mscale * cs, p.mscale * sn);
  }
  __syncthreads();
  for (int i = tid; i < tasks;) {
    if (j.c >= 0) turn_task<VEC>(j, turn, p.interleaved);
    store_run<VEC>(j.dst + j.a, j.ra);
    if (j.two) store_run<VEC>(j.dst + j.b, j.rb);
    i += blockDim.x;
    if (i < tasks) load(i);
  }
}

// E: elements of a key or value row a lane takes at a time, 0 for any row; VEC: of a query's. The first `blocks` x `splits`
// CTAs have keys and values, `splits` of them the tasks of the same runs in turn; those behind (if any) a row of queries each.
template <int VEC, int E>
__global__ void __launch_bounds__(APPEND_WARPS * 32, 2)
    kda_rope_append_fp8_kernel(kda_rope_params p, kda_paged_scales sc, int span, int blocks, int splits) {
  extern __shared__ __align__(16) float2 table[];  // [16][rotary_dim / 2]
  __shared__ int positions[32];
  earlier_work();
  if ((int)blockIdx.x >= blocks * splits) {
    turn_queries<VEC>(p, (int)blockIdx.x - blocks * splits);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = (int)blockIdx.x % splits;
  const int half = p.rotary_dim >> 1, Hkv = p.cache.num_heads, P = p.cache.page_size;
  // Lane l has row t0 + l: this CTA's, and those behind that their runs may reach to; and, of the rows before, in which those
  // runs may have begun, row t0 - 15 + l.
  const int t0 = (int)blockIdx.x / splits * span;
  const long long near = (long long)t0 + lane, slots = (long long)p.cache.num_pages * P;
  const int back = lane - (SCALE_TOKENS - 1);
  int pos = -1, slot = -1, pos_back = -1, slot_back = -1;
  if (near < p.num_tokens) {
    pos = p.positions[near];
    slot = p.slots[near];
  }
  if (back < 0 && t0 + back >= 0) {
    pos_back = p.positions[t0 + back];
    slot_back = p.slots[t0 + back];
  }
  const bool bad = pos >= 0 && slot != -1 && (slot < 0 || slot >= slots);
  if (bad && lane < span && warp == 0 && split == 0 && p.error_word) atomicOr(p.error_word, KDA_ERR_PAGES);
  if (pos < 0 || bad) slot = -1;
  if (pos_back < 0) slot_back = -1;
  const int page = slot >= 0 ? slot / P : 0, off = slot >= 0 ? (slot - page * P) % SCALE_TOKENS : 0;
  const int base = slot - off;  // slot of the block's first token
  const uint32_t shift = (uint32_t)slot - (uint32_t)lane, shift_back = (uint32_t)slot_back - (uint32_t)back;
  uint32_t left = __ballot_sync(0xffffffffu, lane < span && slot >= 0);
  if (warp == 0) positions[lane] = pos;
  while (left) {  // the same for the whole CTA
    const int at = __ffs(left) - 1;
    const int base_at = __shfl_sync(0xffffffffu, base, at);
    const uint32_t shift_at = __shfl_sync(0xffffffffu, shift, at);
    // the stored rows of the block: those as far apart as their slots
    const uint32_t same = __ballot_sync(0xffffffffu, slot >= 0 && base == base_at && shift == shift_at);
    const uint32_t begun = __ballot_sync(0xffffffffu, slot_back >= base_at && shift_back == shift_at);  // with a smaller slot
    left &= ~same;
    if (begun) continue;  // by an earlier CTA
    BlockRun run;
    run.t0 = t0 + at;
    run.rows = same >> at;
    run.n = 32 - __clz(run.rows);  // at most 16, up to lane 30: `at` is below 16
    run.page = __shfl_sync(0xffffffffu, page, at);
    run.first = __shfl_sync(0xffffffffu, off, at);
    run.block = (base_at - run.page * P) / SCALE_TOKENS;
    auto task = [&](int x) {
      const bool keys = x < Hkv;
      const int h = keys ? x : x - Hkv;
      const kda_view& v = keys ? p.k : p.v;
      const kda_pages& g = keys ? p.cache.k : p.cache.v;
      const kda_page_scales& f = keys ? sc.k : sc.v;
      BlockTask k;
      k.src = static_cast<const uint16_t*>(v.ptr) + (int64_t)run.t0 * v.b_stride + (int64_t)h * v.h_stride;
      k.row_stride = v.b_stride;
      k.block = static_cast<uint8_t*>(g.ptr) + (int64_t)run.page * g.page_stride +
                (int64_t)run.block * SCALE_TOKENS * g.token_stride + (int64_t)h * g.head_stride;
      k.token_stride = g.token_stride;
      k.scale = f.ptr + (int64_t)run.page * f.page_stride + (int64_t)run.block * f.block_stride + (int64_t)h * f.head_stride;
      k.turned = keys && half > 0;
      return k;
    };
    int x = split * APPEND_WARPS + warp;
    RunRows<E == 0 ? 2 : E> rows;
    BlockTask k{};
    if (x < 2 * Hkv) {
      k = task(x);
      if constexpr (E > 0) load_rows<E>(run, k, rows);  // on their way while the table is formed
    }
    __syncthreads();  // positions are there; the table of the run before is read
    for (int y = tid; y < run.n * half; y += blockDim.x) {
      const int i = y / half, c = y - i * half;
      table[y] = fast_turn((uint64_t)(uint32_t)positions[at + i] * p.freqs[c], p.mscale);
    }
    __syncthreads();
    if (E == 0 || (run.rows & (run.rows + 1u))) {  // some are left out
      for (; x < 2 * Hkv; x += APPEND_WARPS * splits) append_any(p, run, task(x), table);
    } else if constexpr (E > 0) {
      while (x < 2 * Hkv) {
        append_rows<E>(p, run, k, rows, table);
        x += APPEND_WARPS * splits;
        if (x < 2 * Hkv) {
          k = task(x);
          load_rows<E>(run, k, rows);
        }
      }
    }
  }
}

cudaError_t launch_rope_append_fp8(const kda_rope_params& p, const kda_paged_scales& sc, bool q_wide, int lane_elems,
                                   cudaStream_t s) {
  // Up to 512 rows are mostly decode steps, whose rows may each be a run: a CTA per row. More are chunks, mostly: a CTA looks
  // for runs in up to 16 rows, 512 CTAs. What the rows are stands in device memory, so one rule has to do for both. This one,
  // and the best of spans of 1 to 16 rows with and without `splits`, us, 32 + 8 + 8 heads of 128, on decode rows in blocks of
  // their own and on one chunk: 300 rows 7.0 (5.8 without splits) and 9.9 (7.7); 600: 11.2 (9.5) and 12.0 (10.5); 1000: 17.9
  // (14.9) and 13.7 (12.2); 2000: 38.0 (34.3) and 25.3 (22.1); 4000: 62.6 (58.3) and 36.5 (31.7); 8000: 112 (106) and 57.9
  // (57.7).
  // Up to 2048 rows the queries are in the same launch (1000 rows of the chunk 13.7, 18.3 in two launches). With more they go
  // ahead in a launch of kda_rope_append_kernel without keys and values, which needs half the registers and runs at twice the
  // occupancy, and this kernel is brought in while it ends (4000 rows of the chunk 36.5, 45.2 in one launch; 2000 rows take 25.3
  // in one and 24.2 in two).
  const bool fused = p.num_tokens <= 2048;
  const int span = p.num_tokens <= 512 ? 1 : p.num_tokens < 16 * 512 ? (p.num_tokens + 511) / 512 : SCALE_TOKENS;
  const int blocks = p.num_tokens / span + (p.num_tokens % span != 0), tasks = 2 * p.cache.num_heads;
  // few runs: a task a warp
  const int splits = p.num_tokens < 4096 && tasks > APPEND_WARPS ? (tasks + APPEND_WARPS - 1) / APPEND_WARPS : 1;
  if (!fused) {
    kda_rope_params q = p;
    q.cache.num_heads = q.cache.num_pages = 0;
    q.error_word = nullptr;
    const cudaError_t e = launch_rope_append(q, q_wide, s);
    if (e != cudaSuccess) return e;
  }
  const size_t smem = (size_t)SCALE_TOKENS * (p.rotary_dim / 2) * sizeof(float2);  // at most 16 KB
  const dim3 grid((unsigned)(blocks * splits + (fused ? p.num_tokens : 0)));
  auto go = [&](auto kernel) { return launch_early(kernel, grid, 32 * APPEND_WARPS, smem, s, p, sc, span, blocks, splits); };
  if (lane_elems == 4) return q_wide ? go(kda_rope_append_fp8_kernel<8, 4>) : go(kda_rope_append_fp8_kernel<1, 4>);
  if (lane_elems == 2) return q_wide ? go(kda_rope_append_fp8_kernel<8, 2>) : go(kda_rope_append_fp8_kernel<1, 2>);
  return q_wide ? go(kda_rope_append_fp8_kernel<8, 0>) : go(kda_rope_append_fp8_kernel<1, 0>);
}

// ---------------------------------------------------------------- read
//
// A CTA per 16 packed rows: its threads go through the requests, and each
// request marks the rows of the tile that it covers; 16 threads then find their
// rows' pages; then all copy, 16 codes and 32 bytes of output a thread at a time
// where the rows allow it. Bound by memory: a byte in and two out an element (32
// requests of 1500..6000 tokens, 8 heads of 128: 120 us, 6.3 TB/s, 94 % of a copy).

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
