// kda_paged_fp8_rows.cu - paged attention over a cache in 8 bits for few rows
// (include/kda_paged_fp8.h): decode and verify steps, head_dim 64 or 128.
//
// Mathematics. As kda_paged_tc.cu, turned round: a unit's 128 keys are the rows
// of the products, the R rows of an item (query heads of a key-value head, times
// new tokens) their columns, so that nothing is padded to 128 rows and the codes
// of the cache enter both products as they lie in the pages:
//   S^T = K Q^T       Q as two E4M3 numbers each (query_codes), 2 R columns
//   P^T = exp2(y - m), y = scale log2e ks S + log2 vs: weights times value scales
//   O^T += V^T P^T    P as three E5M2 numbers each, 3 R columns
// A weight p <= 2^14, as fp16, is p1 + 2^-4 p2 + 2^-8 p3, exactly, subnormals
// included: in the binade of 2^E a part takes three bits and leaves at most
// 2^(E - 3), the next 2^(E - 7), the third nothing of fp16's eleven bits. So a
// weight is rounded by 2^-11 of itself, and below 2^-24 of the row's largest
// (which is kept at 2^10 or more) by 2^-35 of that: many small weights beside a
// large one still add up. (E4M3 parts hold as many bits, but of a weight at 2^-23
// of the largest one bit.) The parts have columns of their own in O^T and are
// added up at the end, in fp32. l sums the fp32 weights. The reference m of a row
// follows its maximum when that has grown by more than 4 (log2), for all keys
// together: m is the same in all threads, which agree on it by a vote a unit.
//
// A CTA is eight warps: four of softmax (a thread per key), and one warp each
// that issues the products, that loads (a tensor-map copy a page and side), that
// walks the line, and that prepares the queries and the scales of the runs to
// come. Nothing of a run's start is waited for: its keys, queries and scores are
// there when the run before ends. A run's O^T has a thread a dimension: outputs
// and parts are written as whole rows.
//
// What bounds it: memory, and what is not hidden behind it. 64 decode requests of
// 2048..8192 tokens, 8 key-value heads: 107 to 113 us by the machine, 5.6 to 5.9
// TB/s; a unit takes 1360 cycles at the copy's rate. In a build with clocks read on
// the way (126 us) a call began with 7800 cycles until the first scores and ended
// with an item's parts, 2300 to 2700 a trip to memory under load, hence eight parts
// a trip (four: 47 us against 43 for 4 requests of 16384..65536 tokens). With rows as the rows of the products (the
// kernel for chunks) the same 64 requests took 220 us, bound by the padding to 128
// rows and by the conversion of the values. 32 verify requests of 24 rows: 48 to
// 49 us, 17 of memory (48.0 with E4M3 parts of the weights).
// Scales: with one pair of units on its way a step waited for them under load
// (600 cycles a unit in the slowest CTAs); with two it does not.
#include <math.h>

#include "kda_paged_launch.h"
#include "kda_paged_line.cuh"

namespace kda {

namespace {

constexpr int THREADS = 256, SOFTMAX_THREADS = 128;
constexpr int PRODUCT_WARP = 4, LOAD_WARP = 5, WALK_WARP = 6, AHEAD_WARP = 7;
constexpr int RING = 4;    // segments the walking warp may be ahead
constexpr int LEAD = 3;    // what an item costs beside its units, in units
constexpr int SCALES = 4;  // pairs of units whose scales are held
constexpr int BLOCK = KDA_FP8_SCALE_TOKENS, BLOCKS = UNIT / BLOCK;
constexpr float LIFT = 10.f, SLACK = 4.f;  // log2 of the largest weight when the reference is set; its growth until the next
static_assert(LIFT + SLACK <= 14.f, "16 times what the first part of a weight leaves is a number of E5M2");
constexpr float LOG2E = 1.4426950408889634f;
constexpr float NOTHING = -3.402823466e38f;  // the reference of a row that has seen no key: no finite score is below it, and no
                                             // infinity, so that differences to it are numbers

template <int D, int R>
struct Shape {
  static constexpr int NS = 2 * R < 16 ? 16 : 2 * R;            // columns of S^T
  static constexpr int NP = (3 * R + 15) / 16 * 16;             // of O^T, with the parts of P
  static constexpr int STAGES = R == 32 && D == 128 ? 5 : 6;    // units of keys, and of values
  static constexpr uint32_t UNIT_BYTES = UNIT * D;
  static constexpr uint32_t Q_BYTES = NS * D, P_BYTES = NP * UNIT;
  static constexpr uint32_t K0 = 0, V0 = K0 + STAGES * UNIT_BYTES;
  static constexpr uint32_t Q0 = V0 + STAGES * UNIT_BYTES, P0 = Q0 + 2 * Q_BYTES;
  static constexpr uint32_t RAW0 = P0 + 2 * P_BYTES;            // queries as they come (head_dim 64)
  static constexpr uint32_t END = RAW0 + (D == 64 ? R * 128 : 0);
  static constexpr uint32_t S_COLS = NS, COLS = 2 * NS + NP;
  static constexpr uint32_t TMEM = COLS <= 64 ? 64 : COLS <= 128 ? 128 : 256;
};

struct alignas(16) UnitScales {
  float key[BLOCKS], log_value[BLOCKS], inv_value[BLOCKS];
};

template <int D, int R>
struct Shared {
  using S = Shape<D, R>;
  uint64_t k_full[S::STAGES], k_empty[S::STAGES], v_full[S::STAGES], v_empty[S::STAGES];
  uint64_t v_tail, q_full[2], q_empty[2], s_full[2], s_empty[2], p_full[2], p_done[2], seg_full[RING], seg_empty[RING], drain;
  uint64_t scale_full[SCALES], scale_empty[SCALES];
  UnitScales scales[SCALES][2];
  Segment seg[RING];
  alignas(16) float q_scale[2][R];  // scale log2e times the power of two by which a row's query was brought down
  alignas(16) float top[4][R];      // a warp's maxima, or sums
  alignas(16) float down[R], fade[R];  // -m, the same for all keys, and by how much it last moved
  int warp_sum[THREADS / 32];
  LineStart start;
  uint32_t tmem;
  int last_part;
};

struct RowsArgs {
  kda_attention_params p;
  kda_paged_scales sc;
  float* parts;        // workspace: 2 slots a CTA, each [R][D] of unnormalised O, then [R] of (m, l)
  unsigned* counters;  // one a CTA, zero between calls
  int q_wide;
  int box;             // keys a copy brings: min(page_size, UNIT)
  int group, item_tokens;
  unsigned inv_group;  // row / group = row * inv_group >> 16
  size_t slot_floats;
};

// D = A B^T over STEPS steps of K (32 codes each), issued by one elected lane of a converged warp, then an arrival on `done`
// and one on `free`. A_STEP, B_STEP: what a step adds to the descriptors.
template <int STEPS, int A_STEP, int B_STEP>
__device__ __forceinline__ void issue(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t fresh, uint32_t done,
                                      uint32_t free, uint32_t also) {
#pragma unroll
  for (int k = 0; k < STEPS; ++k)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 r;\n\telect.sync r|p, 0xffffffff;\n\tsetp.eq.b32 q, %4, 0;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, q;\n\t}" ::"r"(d),
        "l"(a + k * A_STEP), "l"(b + k * B_STEP), "r"(idesc), "r"(k == 0 ? fresh : 0u)
        : "memory");
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b32 r;\n\telect.sync r|p, 0xffffffff;\n\t"
      "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t"
      "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t"
      "setp.ne.and.b32 q, %2, 0, p;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%2];\n\t}" ::"r"(done),
      "r"(free), "r"(also)
      : "memory");
}

// The weights' operand: 16 columns of O^T (bytes) of a key side by side, key after key, the next 16 columns 128 keys on. N is
// contiguous, without a swizzle: leading byte offset, the next 8 keys; stride byte offset, the next 16 columns. A K step of
// 32 keys adds 512 bytes. So a thread stores what it has of its key in whole 16 bytes (a byte a column and key, in rows of
// keys, took 3 R stores: 32 verify requests of 24 rows 87.6 us).
__device__ __forceinline__ uint64_t weight_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128u >> 4) << 16) | ((uint64_t)(UNIT * 16u >> 4) << 32) |
         ((uint64_t)1u << 46);
}

__device__ __forceinline__ f32x2 add2(f32x2 x, f32x2 y) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// Two fp16 numbers to E5M2, and back: an E5M2 number is the upper byte of an fp16 one.
__device__ __forceinline__ uint32_t f16x2_to_e5m2x2(uint32_t x) {
  unsigned short r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t e5m2x2_to_f16x2(uint32_t two) { return __byte_perm(two, 0u, 0x1404); }

// N consecutive columns of this thread's lane, with the wait (N: 4, 8, 16, 32 or 64).
template <int N>
__device__ __forceinline__ void load_columns(uint32_t taddr, float (&out)[N]) {
  if constexpr (N == 4) {
    uint32_t z[4];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(z[0]), "=r"(z[1]), "=r"(z[2]), "=r"(z[3])
                 : "r"(taddr)
                 : "memory");
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = __uint_as_float(z[j]);
  } else if constexpr (N == 8) {
    tmem_ld8(taddr, out);
  } else if constexpr (N == 16) {
    tmem_ld16(taddr, out);
  } else {
    static_assert(N == 32 || N == 64, "");
    float lo[32], hi[32];
    if constexpr (N == 64)
      tmem_ld32x2(taddr, lo, hi);
    else
      tmem_ld32(taddr, lo);
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      out[j] = lo[j];
      if constexpr (N == 64) out[32 + j] = hi[j];
    }
  }
}

template <int N>
__device__ __forceinline__ void store_columns(uint32_t taddr, const float (&v)[N]) {
  if constexpr (N == 32) {
    tmem_st32(taddr, v);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      uint32_t z[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) z[j] = __float_as_uint(v[i + j]);
      tmem_st4(taddr + i, z);
    }
  }
}

// N (4 or 8) columns at taddr, taddr + step and taddr + 2 step, with one wait.
template <int N>
__device__ __forceinline__ void load_parts(uint32_t taddr, int step, float (&out)[3][N]) {
  uint32_t z[3][N];
#pragma unroll
  for (int i = 0; i < 3; ++i)
#pragma unroll
    for (int j = 0; j < N; j += 4)
      asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(z[i][j]), "=r"(z[i][j + 1]), "=r"(z[i][j + 2]), "=r"(z[i][j + 3])
                   : "r"(taddr + i * step + j)
                   : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 3; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      asm volatile("" : "+r"(z[i][j]));  // no use of it above the wait
      out[i][j] = __uint_as_float(z[i][j]);
    }
}

// The sums (or maxima) over a warp's lanes of R values a lane: lane l is left with that of value l % R. Each step sends half
// of what is left.
template <int R, bool MAX>
__device__ __forceinline__ float fold(float (&v)[R]) {
  const int lane = threadIdx.x & 31;
  auto join = [](float x, float y) { return MAX ? fmaxf(x, y) : x + y; };
#pragma unroll
  for (int s = R / 2; s >= 1; s >>= 1)
#pragma unroll
    for (int i = 0; i < s; ++i) {
      const float send = lane & s ? v[i] : v[i + s], keep = lane & s ? v[i + s] : v[i];
      v[i] = join(keep, __shfl_xor_sync(0xffffffffu, send, s));
    }
#pragma unroll
  for (int o = R; o < 32; o <<= 1) v[0] = join(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
  return v[0];
}

}  // namespace

template <int D, int R>
__global__ void __launch_bounds__(THREADS, 1)
    kda_paged_attention_fp8_rows_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                                        const __grid_constant__ RowsArgs a) {
  using S = Shape<D, R>;
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle's atoms are 1024-byte aligned
  Shared<D, R>& sh = *reinterpret_cast<Shared<D, R>*>(smem + S::END);
  const kda_attention_params& p = a.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = a.group, w = a.item_tokens;
  const int window = p.window;

  if (warp == 0) {  // a lane a stage
    if (lane < S::STAGES) {
      mbar_init_only(&sh.k_full[lane], 1);
      mbar_init_only(&sh.k_empty[lane], 1);
      mbar_init_only(&sh.v_full[lane], 1);
      mbar_init_only(&sh.v_empty[lane], 1);
    }
    if (lane < RING) {
      mbar_init_only(&sh.seg_full[lane], 1);
      mbar_init_only(&sh.seg_empty[lane], 4);  // the loading, product and ahead warps, the softmax group
    }
    if (lane < SCALES) {
      mbar_init_only(&sh.scale_full[lane], 1);
      mbar_init_only(&sh.scale_empty[lane], SOFTMAX_THREADS / 32);
    }
    if (lane < 2) {
      mbar_init_only(&sh.q_full[lane], 1);
      mbar_init_only(&sh.q_empty[lane], 1 + SOFTMAX_THREADS / 32);  // the run's scores are formed, its scales read
      mbar_init_only(&sh.s_full[lane], 1);
      mbar_init_only(&sh.s_empty[lane], SOFTMAX_THREADS / 32);
      mbar_init_only(&sh.p_full[lane], SOFTMAX_THREADS / 32);
      mbar_init_only(&sh.p_done[lane], 1);
    }
    if (lane == 2) mbar_init_only(&sh.v_tail, 1);
    if (lane == 3) mbar_init_only(&sh.drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  } else if (warp == LOAD_WARP && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
  }

  earlier_work();

  const int cta = blockIdx.x;
  const LineShare line = line_share<THREADS, LEAD>(p, w, sh.warp_sum, sh.start);
  if (blockIdx.x == 0 && line.bad && p.error_word) atomicOr(p.error_word, line.bad);
  if (cta >= line.ctas) return;  // the whole CTA: nothing allocated yet
  if (warp == PRODUCT_WARP) tmem_alloc(&sh.tmem, S::TMEM);
  tc_fence_before();
  const int end = line_end(p, line);
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  bool alive = true;

  if (warp == WALK_WARP) {
    uint32_t out = 0;
    auto put = [&](const Segment& g2) {
      const uint32_t slot = out % RING;
      if (!warp_wait(&sh.seg_empty[slot], (out / RING + 1) & 1)) return false;
      if (lane == 0) {
        sh.seg[slot] = g2;
        mbar_arrive(&sh.seg_full[slot]);
      }
      __syncwarp();
      ++out;
      return true;
    };
    alive = line_walk<LEAD>(p, w, line, end, sh.start, put);
  } else if (warp == LOAD_WARP) {
    // ---- keys and values of the CTA's units, a lane per copy
    const int P = p.cache.page_size, box = a.box;
    uint32_t n = 0, tails = 0;
    bool bad_page = false, pending = false;  // pending: a ragged unit of values is on its way
    int first = 0, last = UNIT;              // the keys of it that are in use
    // Weights of unseen keys are zero, but zero times what lies there need not be: clear those rows. Done when the next
    // values are to be loaded, so that the keys of the next run do not wait for it.
    auto clear_tail = [&]() {
      pending = false;
      if (!warp_wait(&sh.v_tail, tails & 1)) return false;
      ++tails;
      const uint32_t st = (n - 1) % S::STAGES;
      uint8_t* const dst = smem + S::V0 + st * S::UNIT_BYTES;
      for (int x = lane; x < UNIT * (D / 16); x += 32) {
        const int row = x / (D / 16);
        if (row < first || row >= last) *reinterpret_cast<uint4*>(dst + x * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.v_full[st]);
      return true;
    };
    for (uint32_t in = 0; alive; ++in) {
      const uint32_t slot = in % RING;
      alive = warp_wait(&sh.seg_full[slot], (in / RING) & 1);
      if (!alive) break;
      const Segment sg = sh.seg[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.seg_empty[slot]);
      if (sg.ntok < 0) break;
      const int32_t* const table = p.table + (int64_t)sg.request * p.table_stride;
      const int pieces = UNIT / box;  // at most 8
      for (int u = sg.u0; u < sg.u1; ++u) {
        const int key = u * UNIT + lane * box;
        const bool wanted = lane < pieces && key < sg.hi && key + box > sg.lo;
        int page = 0;
        if (wanted) {
          page = table[key / P];
          if (page < 0 || page >= p.cache.num_pages) {
            page = p.cache.num_pages;  // past the end: the copy brings zeros
            bad_page = true;
          }
        }
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, wanted)) * (uint32_t)box * D;
        const uint32_t st = n % S::STAGES, parity = (n / S::STAGES + 1) & 1;
        alive = warp_wait(&sh.k_empty[st], parity);
        if (!alive) break;
        if (lane == 0) mbar_expect_tx(&sh.k_full[st], bytes);
        __syncwarp();
        if (wanted) tma_load_4d(smem + S::K0 + st * S::UNIT_BYTES + lane * box * D, &kmap, 0, key % P, sg.head, page, &sh.k_full[st]);
        if (pending) alive = clear_tail();
        alive = alive && warp_wait(&sh.v_empty[st], parity);
        if (!alive) {
          ++n;  // keys are on their way
          break;
        }
        first = max(sg.lo - u * UNIT, 0);
        last = min(sg.hi - u * UNIT, UNIT);
        pending = first > 0 || last < UNIT;
        uint64_t* const bar = pending ? &sh.v_tail : &sh.v_full[st];
        if (lane == 0) mbar_expect_tx(bar, bytes);
        __syncwarp();
        if (wanted) tma_load_4d(smem + S::V0 + st * S::UNIT_BYTES + lane * box * D, &vmap, 0, key % P, sg.head, page, bar);
        ++n;
      }
    }
    if (alive && pending) alive = clear_tail();
    if (bad_page && p.error_word) atomicOr(p.error_word, KDA_ERR_PAGES);
    if (!alive) {  // copies in flight land before the CTA leaves
      mbar_drain_bounded(&sh.v_tail, tails & 1);
      for (uint32_t i = n > (uint32_t)S::STAGES ? n - S::STAGES : 0; i < n; ++i) {
        mbar_drain_bounded(&sh.k_full[i % S::STAGES], (i / S::STAGES) & 1);
        mbar_drain_bounded(&sh.v_full[i % S::STAGES], (i / S::STAGES) & 1);
      }
    }
  } else if (warp == AHEAD_WARP) {
    // ---- queries of the runs to come, as codes, and their units' scales, a pair of units at a time (16 lanes each: keys'
    // blocks, then values'). Two pairs are on their way meanwhile, and the page numbers of a third: under a full load of
    // memory the two trips of a scale take longer than a pair of units
    uint32_t pairs = 0;
    for (uint32_t in = 0; alive; ++in) {
      const uint32_t slot = in % RING;
      alive = warp_wait(&sh.seg_full[slot], (in / RING) & 1);
      if (!alive) break;
      const Segment sg = sh.seg[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.seg_empty[slot]);
      if (sg.ntok < 0) break;
      const int P = p.cache.page_size, b = lane & (BLOCKS - 1);
      const bool of_values = (lane & BLOCKS) != 0;
      const int32_t* const table = p.table + (int64_t)sg.request * p.table_stride;
      const kda_page_scales& of = of_values ? a.sc.v : a.sc.k;
      auto page_of = [&](int u0) {  // -1: no key of this lane's block is seen, or the page is none
        const int u = u0 + (lane >> 4);
        if (u >= sg.u1) return -1;
        const int key = u * UNIT + b * BLOCK;
        return key >= sg.hi || key + BLOCK <= sg.lo ? -1 : table[key / P];
      };
      auto scale_of = [&](int u0, int page) {
        return page < 0 || page >= p.cache.num_pages ? 1.f : block_scale(of, page, ((u0 + (lane >> 4)) * UNIT + b * BLOCK) % P, sg.head);
      };
      const int p0 = page_of(sg.u0), p1 = page_of(sg.u0 + 2);
      int page = page_of(sg.u0 + 4);
      float x0 = 1.f, x1 = 1.f;

      const uint32_t qb = in & 1;
      alive = warp_wait(&sh.q_empty[qb], (in / 2 + 1) & 1);
      if (!alive) break;
      {
        // brought asynchronously, then turned into codes row by row in a loop that is not unrolled: once-a-run code is
        // fetched anew each run. For head_dim 128 a row's codes go where its numbers lie.
        constexpr int LANES = D / 8, ROWS = 32 / LANES;  // lanes a row, rows a round
        const int rows = sg.ntok * g, ch = lane % LANES;
        const uint16_t* const qg =
            static_cast<const uint16_t*>(p.q.ptr) + (int64_t)sg.row0 * p.q.b_stride + (int64_t)(sg.head * g) * p.q.h_stride + ch * 8;
        uint8_t* const tile = smem + S::Q0 + qb * S::Q_BYTES;
        auto raw = [&](int r) {
          return D == 128 ? tile + (ch >> 3) * (R * 128) + r * 128 + (ch & 7) * 16 : smem + S::RAW0 + r * 128 + ch * 16;
        };
        for (int r = lane / LANES; r < rows; r += ROWS) {
          const int tk = (int)((uint32_t)r * a.inv_group >> 16);
          const uint16_t* const src = qg + (int64_t)tk * p.q.b_stride + (int64_t)(r - tk * g) * p.q.h_stride;
          if (a.q_wide) {
            copy_async16(raw(r), src);
          } else {
            uint32_t x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = (uint32_t)src[2 * k] | ((uint32_t)src[2 * k + 1] << 16);
            *reinterpret_cast<uint4*>(raw(r)) = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
        x0 = scale_of(sg.u0, p0);
        x1 = scale_of(sg.u0 + 2, p1);
        copy_async_wait();
        constexpr int N = R / ROWS < 4 ? R / ROWS : 4;  // rounds at a time
#pragma unroll 1
        for (int r0 = lane / LANES; r0 < R; r0 += N * ROWS) {
          uint4 z[N];
          int e[N];
#pragma unroll
          for (int i = 0; i < N; ++i)
            z[i] = r0 + i * ROWS < rows ? *reinterpret_cast<const uint4*>(raw(r0 + i * ROWS)) : make_uint4(0, 0, 0, 0);
          query_exponents<N, LANES>(z, e);
          __syncwarp();  // the rows' numbers are read
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int r = r0 + i * ROWS;
            uint2 hi, lo;
            query_codes(z[i], e[i], hi, lo);
            *reinterpret_cast<uint2*>(tile + code_chunk<D>(r, ch >> 1) + (ch & 1) * 8) = hi;
            *reinterpret_cast<uint2*>(tile + code_chunk<D>(R + r, ch >> 1) + (ch & 1) * 8) = lo;
            if (ch == 0) sh.q_scale[qb][r] = p.scale * LOG2E * query_up(e[i]);
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full[qb]);

      for (int u = sg.u0; u < sg.u1; u += 2, ++pairs) {
        const float x = x0;
        x0 = x1;
        x1 = scale_of(u + 4, page);
        page = page_of(u + 6);
        const uint32_t st = pairs % SCALES;
        alive = warp_wait(&sh.scale_empty[st], (pairs / SCALES + 1) & 1);
        if (!alive) break;
        UnitScales& us = sh.scales[st][lane >> 4];
        if (of_values) {
          us.log_value[b] = log2f(x);
          us.inv_value[b] = 1.f / x;
        } else {
          us.key[b] = x;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.scale_full[st]);
      }
    }
  } else if (warp == PRODUCT_WARP) {
    // ---- the products: a unit's scores one unit ahead of its values, over the ends of runs
    const uint32_t base = smem_addr(smem), tm = uniform(tmem);
    constexpr uint32_t M128 = 128u >> 4, F32 = 1u << 4, MN_MAJOR = 3u << 15;  // of A and B
    constexpr uint32_t B_E5M2 = 1u << 10;                                     // the weights; all others are E4M3 (0)
    constexpr uint32_t IDESC_S = F32 | ((uint32_t)S::NS >> 3 << 17) | (M128 << 24);
    constexpr uint32_t IDESC_O = F32 | B_E5M2 | MN_MAJOR | ((uint32_t)S::NP >> 3 << 17) | ((uint32_t)D >> 4 << 24);
    uint32_t n = 0;          // units whose scores have been issued
    uint32_t fresh = 0;      // the last of them begins a run
    auto values = [&](uint32_t m) {
      const uint32_t st = m % S::STAGES, buf = m & 1;
      if (!warp_wait(&sh.v_full[st], (m / S::STAGES) & 1) || !warp_wait(&sh.p_full[buf], (m / 2) & 1)) return false;
      tc_fence_after();
      issue<UNIT / 32, 32 * D / 16, 32>(tm + 2 * S::S_COLS, code_desc<D>(base + S::V0 + st * S::UNIT_BYTES),
                                        weight_desc(base + S::P0 + buf * S::P_BYTES), IDESC_O, fresh, smem_addr(&sh.p_done[buf]),
                                        smem_addr(&sh.v_empty[st]), 0u);
      return true;
    };
    for (uint32_t in = 0; alive; ++in) {
      const uint32_t slot = in % RING;
      alive = warp_wait(&sh.seg_full[slot], (in / RING) & 1);
      if (!alive) break;
      const int ntok = uniform(sh.seg[slot].ntok), units = uniform(sh.seg[slot].u1 - sh.seg[slot].u0);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.seg_empty[slot]);
      if (ntok < 0) break;
      const uint32_t qb = in & 1;
      alive = warp_wait(&sh.q_full[qb], (in / 2) & 1);
      const uint64_t dq = code_desc<D>(base + S::Q0 + qb * S::Q_BYTES);
      for (int i = 0; alive && i < units; ++i, ++n) {
        const uint32_t st = n % S::STAGES, buf = n & 1;
        alive = warp_wait(&sh.k_full[st], (n / S::STAGES) & 1) && warp_wait(&sh.s_empty[buf], (n / 2 + 1) & 1);
        if (!alive) break;
        tc_fence_after();
        issue<D / 32, 2, 2>(tm + buf * S::S_COLS, code_desc<D>(base + S::K0 + st * S::UNIT_BYTES), dq, IDESC_S, 1u,
                            smem_addr(&sh.s_full[buf]), smem_addr(&sh.k_empty[st]),
                            i + 1 == units ? smem_addr(&sh.q_empty[qb]) : 0u);
        if (n > 0) alive = values(n - 1);
        fresh = i == 0;
      }
    }
    if (alive && n > 0) alive = values(n - 1);
    if (!alive) {  // products in flight end before the tensor memory goes
      tc_commit_w(&sh.drain);
      mbar_drain_bounded(&sh.drain, 0);
    }
  } else {
    // ---- softmax: thread x has key x of a unit, and dimension x of the outputs (head_dim 64: lanes 0..15 of each warp)
    const int x = tid;
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    const uint32_t o_addr = tmem + 2 * S::S_COLS + lane_base;
    const int d = D == 128 ? x : warp * 16 + lane;
    const bool has_d = D == 128 || lane < 16;
    uint32_t n = 0, pairs_before = 0;
    for (uint32_t in = 0;; ++in) {
      const uint32_t slot = in % RING, qb = in & 1;
      alive = alive && warp_wait(&sh.seg_full[slot], (in / RING) & 1);
      if (bar_any(1, SOFTMAX_THREADS, !alive)) {  // the group leaves together
        alive = false;
        break;
      }
      const Segment& sg = sh.seg[slot];
      if (sg.ntok < 0) break;
      alive = warp_wait(&sh.q_full[qb], (in / 2) & 1);
      const int u0 = sg.u0, u1 = sg.u1, ntok = sg.ntok, pos0 = sg.pos0, rows = ntok * g;
      // every row sees the keys [all_lo, all_hi)
      const int all_lo = first_key(pos0 + ntok - 1, window), all_hi = pos0 + 1;
      if (x < R) sh.down[x] = -NOTHING;  // first read behind the votes of the first unit
      f32x2 down[R / 2], l[R / 2];       // -m and l of two rows each
#pragma unroll
      for (int r = 0; r < R; r += 2) {
        down[r / 2] = pk2(-NOTHING, -NOTHING);
        l[r / 2] = pk2(0.f, 0.f);
      }
      for (int u = u0; u < u1; ++u, ++n) {
        const uint32_t buf = n & 1, of_run = (uint32_t)(u - u0), pair_of = pairs_before + of_run / 2;
        if (of_run % 2 == 0) alive = alive && warp_wait(&sh.scale_full[pair_of % SCALES], (pair_of / SCALES) & 1);
        alive = alive && warp_wait(&sh.s_full[buf], (n / 2) & 1);
        f32x2 y[R / 2];  // two rows each
        if (alive) {  // a warp whose wait gave up stays with the group to its next vote
          tc_fence_after();
          const UnitScales& us = sh.scales[pair_of % SCALES][of_run % 2];
          const float f = us.key[x / BLOCK], lv = us.log_value[x / BLOCK];
          float s[2 * R];
          load_columns(tmem + buf * S::S_COLS + lane_base, s);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.s_empty[buf]);
          const f32x2 f2 = pk2(f, f), lv2 = pk2(lv, lv);
#pragma unroll
          for (int r = 0; r < R; r += 4) {
            const float4 q = *reinterpret_cast<const float4*>(&sh.q_scale[qb][r]);
            y[r / 2] = fma2(add2(pk2(s[r], s[r + 1]), pk2(s[R + r], s[R + r + 1])), mul2(pk2(q.x, q.y), f2), lv2);
            y[r / 2 + 1] = fma2(add2(pk2(s[r + 2], s[r + 3]), pk2(s[R + r + 2], s[R + r + 3])), mul2(pk2(q.z, q.w), f2), lv2);
          }
        }
        bool grown = !alive;
        const int key = u * UNIT + x;
        if (__builtin_expect((u + 1) * UNIT > all_hi || u * UNIT < all_lo, 0)) {
#pragma unroll
          for (int r = 0; r < R; r += 2) {
            float two[2];
            upk2(y[r / 2], two[0], two[1]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int pos = pos0 + (int)((uint32_t)(r + i) * a.inv_group >> 16);
              if (r + i < rows && (key > pos || key < first_key(pos, window))) two[i] = -INFINITY;
            }
            y[r / 2] = pk2(two[0], two[1]);
          }
        }
        float over = -INFINITY;  // the largest log2 of a weight
#pragma unroll
        for (int r = 0; r < R; r += 2) {
          float d0, d1;
          upk2(add2(y[r / 2], down[r / 2]), d0, d1);
          over = max3(over, d0, d1);
        }
        grown |= over > LIFT + SLACK;
        if (bar_any(1, SOFTMAX_THREADS, grown)) {
          float v[R];
#pragma unroll
          for (int r = 0; r < R; r += 2) upk2(y[r / 2], v[r], v[r + 1]);
          const float mine = fold<R, true>(v);
          if (lane < R) sh.top[warp][lane] = mine;
          if (bar_any(2, SOFTMAX_THREADS, !alive)) {
            alive = false;
            break;
          }
          // a thread a row finds its new reference, and all read them
          if (x < R) {
            const float top = fmaxf(fmaxf(sh.top[0][x], sh.top[1][x]), fmaxf(sh.top[2][x], sh.top[3][x])), was = sh.down[x];
            const bool moves = top + was > LIFT + SLACK;
            const float to = moves ? LIFT - top : was;
            sh.down[x] = to;
            sh.fade[x] = moves ? ex2(to - was) : 1.f;
          }
          bar_sync(2, SOFTMAX_THREADS);
          f32x2 fade[R / 2];
#pragma unroll
          for (int r = 0; r < R; r += 4) {
            const float4 d = *reinterpret_cast<const float4*>(&sh.down[r]), f = *reinterpret_cast<const float4*>(&sh.fade[r]);
            down[r / 2] = pk2(d.x, d.y);
            down[r / 2 + 1] = pk2(d.z, d.w);
            fade[r / 2] = pk2(f.x, f.y);
            fade[r / 2 + 1] = pk2(f.z, f.w);
            l[r / 2] = mul2(l[r / 2], fade[r / 2]);
            l[r / 2 + 1] = mul2(l[r / 2 + 1], fade[r / 2 + 1]);
          }
          if (of_run > 0) {  // O^T, once the product before is done
            alive = warp_wait(&sh.p_done[1 - buf], ((n - 1) / 2) & 1);
            if (alive) {
              tc_fence_after();
#pragma unroll 1
              for (int part = 0; part < 3; ++part) {
                float o[R];
                load_columns(o_addr + part * R, o);
#pragma unroll
                for (int r = 0; r < R; r += 2) upk2(mul2(pk2(o[r], o[r + 1]), fade[r / 2]), o[r], o[r + 1]);
                store_columns(o_addr + part * R, o);
              }
              tmem_st_wait();
            }
          }
        }
        // the place of the unit before the last is free when its product is done
        alive = alive && warp_wait(&sh.p_done[buf], (n / 2 + 1) & 1);
        if (!alive) continue;
        const float iv = sh.scales[pair_of % SCALES][of_run % 2].inv_value[x / BLOCK];
        uint32_t words[S::NP / 4] = {};  // the columns of this key, four a word
#pragma unroll
        for (int r = 0; r < R; r += 2) {
          float p0, p1;
          upk2(add2(y[r / 2], down[r / 2]), p0, p1);
          p0 = ex2(p0);
          p1 = ex2(p1);
          l[r / 2] = fma2(pk2(p0, p1), pk2(iv, iv), l[r / 2]);
          uint32_t rest = pack_f16x2(p0, p1);
#pragma unroll
          for (int part = 0; part < 3; ++part) {
            const uint32_t c = f16x2_to_e5m2x2(rest);
            words[(part * R + r) / 4] |= r % 4 ? c << 16 : c;
            if (part < 2) rest = mul_f16x2(sub_f16x2(rest, e5m2x2_to_f16x2(c)), 0x4c004c00u);  // 16
          }
        }
        uint8_t* const pt = smem + S::P0 + buf * S::P_BYTES + x * 16;
#pragma unroll
        for (int i = 0; i < S::NP / 16; ++i)
          *reinterpret_cast<uint4*>(pt + i * UNIT * 16) = make_uint4(words[4 * i], words[4 * i + 1], words[4 * i + 2], words[4 * i + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh.p_full[buf]);
          if (of_run % 2 == 1 || u + 1 == u1) mbar_arrive(&sh.scale_empty[pair_of % SCALES]);
        }
      }
      pairs_before += (uint32_t)(u1 - u0 + 1) / 2;

      // ---- the end of the run
      alive = alive && warp_wait(&sh.p_done[(n - 1) & 1], ((n - 1) / 2) & 1);
      if (lane == 0) mbar_arrive(&sh.q_empty[qb]);
      {
        float v[R];
#pragma unroll
        for (int r = 0; r < R; r += 2) upk2(l[r / 2], v[r], v[r + 1]);
        const float mine = fold<R, false>(v);
        if (lane < R) sh.top[warp][lane] = mine;
      }
      if (bar_any(2, SOFTMAX_THREADS, !alive)) {
        alive = false;
        break;
      }
      tc_fence_after();
      const bool direct = sg.parts == 1;
      const int head = sg.head, row0 = sg.row0;
      uint16_t* const out = static_cast<uint16_t*>(p.out) + (int64_t)row0 * p.out_b_stride + (int64_t)(head * g) * p.out_h_stride + d;
      auto out_at = [&](int r) {
        const int tk = (int)((uint32_t)r * a.inv_group >> 16);
        return out + (int64_t)tk * p.out_b_stride + (int64_t)(r - tk * g) * p.out_h_stride;
      };
      auto sees_none = [&](int r) { return pos0 + (int)((uint32_t)r * a.inv_group >> 16) < 0; };
      auto put_lse = [&](int r, float mm, float ll) {
        const int tk = (int)((uint32_t)r * a.inv_group >> 16);
        p.lse[((int64_t)row0 + tk) * p.num_q_heads + head * g + (r - tk * g)] = fmaf(mm, 0.6931471805599453f, ln(ll));
      };
      auto slot_of = [&](int q) { return q == 0 ? 2 * sg.cta0 + 1 : 2 * (sg.cta0 + q); };
      auto part_o = [&](int id) { return a.parts + (size_t)id * a.slot_floats; };
      auto part_ml = [&](int id) { return reinterpret_cast<float2*>(part_o(id) + R * D); };
      const int my_slot = sg.part == 0 ? 2 * cta + 1 : 2 * cta;
      constexpr int STEP = R < 8 ? 4 : 8;
#pragma unroll 1
      for (int r0 = 0; r0 < rows; r0 += STEP) {
        float o[3][STEP];
        load_parts(o_addr + r0, R, o);
#pragma unroll
        for (int i = 0; i < STEP; ++i) {
          const int r = r0 + i;
          if (r >= rows) break;
          const float sum = (sh.top[0][r] + sh.top[1][r]) + (sh.top[2][r] + sh.top[3][r]);
          const float value = fmaf(fmaf(o[2][i], 0.0625f, o[1][i]), 0.0625f, o[0][i]);
          if (direct) {
            if (has_d) *out_at(r) = float_to_bf16_bits(sees_none(r) ? 0.f : value * rcp(sum));
            if (x == r && p.lse != nullptr) put_lse(r, -sh.down[r], sum);
          } else {
            if (has_d) part_o(my_slot)[r * D + d] = value;
            if (x == r) part_ml(my_slot)[r] = make_float2(-sh.down[r], sum);
          }
        }
      }
      tc_fence_before();
      if (!direct) {
        bar_sync(1, SOFTMAX_THREADS);
        if (tid == 0) {
          __threadfence();  // of what the barrier has gathered
          const unsigned done = atomicAdd(&a.counters[sg.cta0], 1u);
          sh.last_part = done + 1 == (unsigned)sg.parts;
          if (sh.last_part) a.counters[sg.cta0] = 0;
          __threadfence();
        }
        bar_sync(2, SOFTMAX_THREADS);
        if (sh.last_part) {  // the last to arrive joins the parts, in their order: four dimensions of a row a thread
          constexpr int LANES = D / 4, AT_ONCE = 8;  // parts: a trip to memory takes 2000 cycles and more
          const int d4 = x % LANES * 4;
#pragma unroll 1
          for (int r = x / LANES; r < rows; r += SOFTMAX_THREADS / LANES) {
            float mm = -INFINITY, ll = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int q = 0; q < sg.parts; q += AT_ONCE) {
              float2 z[AT_ONCE];
              float4 v[AT_ONCE];
              float top = mm;
#pragma unroll
              for (int k = 0; k < AT_ONCE; ++k) {
                z[k] = make_float2(-INFINITY, 0.f);
                v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (q + k < sg.parts) {
                  const int id = slot_of(q + k);
                  z[k] = __ldcg(part_ml(id) + r);
                  v[k] = __ldcg(reinterpret_cast<const float4*>(part_o(id) + r * D + d4));
                }
              }
#pragma unroll
              for (int k = 0; k < AT_ONCE; ++k) top = fmaxf(top, z[k].x);
              const float f = ex2(mm - top);  // a reference is a number: NOTHING, or of scores that are no infinity
              ll *= f;
              acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
              for (int k = 0; k < AT_ONCE; ++k) {
                const float weight = ex2(z[k].x - top);
                ll = fmaf(z[k].y, weight, ll);
                acc = make_float4(fmaf(v[k].x, weight, acc.x), fmaf(v[k].y, weight, acc.y), fmaf(v[k].z, weight, acc.z),
                                  fmaf(v[k].w, weight, acc.w));
              }
              mm = top;
            }
            const float iv = sees_none(r) ? 0.f : rcp(ll);
            uint16_t* const dst = out_at(r) - d + d4;
            const float f4[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[i] = float_to_bf16_bits(sees_none(r) ? 0.f : f4[i] * iv);
            if (d4 == 0 && p.lse != nullptr) put_lse(r, mm, ll);
          }
        }
      }
      bar_sync(1, SOFTMAX_THREADS);  // sums and segment are read
      if (x == 0) mbar_arrive(&sh.seg_empty[slot]);
    }
  }
  if (!alive && lane == 0 && p.error_word) atomicOr(p.error_word, KDA_ERR_TIMEOUT);
  __syncwarp();

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == PRODUCT_WARP) tmem_dealloc(tmem, S::TMEM);
}

template <int D, int R>
static cudaError_t launch_rows(const RowsArgs& a, int ctas, cudaStream_t s) {
  constexpr size_t bytes = Shape<D, R>::END + sizeof(Shared<D, R>);
  static_assert(bytes <= 232448, "shared memory of one CTA");
  static DeviceFlags done;
  cudaError_t e = set_smem_limit_once(kda_paged_attention_fp8_rows_kernel<D, R>, bytes, done);
  if (e != cudaSuccess) return e;
  CUtensorMap km, vm;
  e = code_pages_tensor_map(a.p.cache.k, a.p.cache, a.box, &km);
  if (e == cudaSuccess) e = code_pages_tensor_map(a.p.cache.v, a.p.cache, a.box, &vm);
  if (e != cudaSuccess) return e;
  return launch_early(kda_paged_attention_fp8_rows_kernel<D, R>, dim3((unsigned)ctas), THREADS, bytes, s, km, vm, a);
}

// By the mean rows a request, which is all that the host knows. On 64 requests of 2048..8192 tokens, 32 heads over 8, single
// calls from a cold cache, this kernel and the one for chunks: 1 new token each 138 and 224 us, 4 each 142 and 226, 1..8 each
// 162 and 228. Decode tokens and a chunk in one call, 200 and 1000: 794 and 939 where the decodes have such contexts and the
// chunk 8192 tokens; but 1873 and 541 where they have 64..256 and the chunk 32768, whose keys are read once every 8 tokens.
// As two calls these take 522 and 451.
int paged_attention_few_rows(const kda_attention_params& p) {
  const long long group = p.num_q_heads / p.cache.num_heads;
  const long long tokens = ((long long)p.num_tokens + p.num_requests - 1) / p.num_requests;
  for (int rows = 4; rows <= 32; rows *= 2)
    if (tokens * group <= rows) return rows;
  return 0;
}

cudaError_t launch_paged_attention_fp8_rows(const kda_attention_params& p, const kda_paged_scales& sc, int rows,
                                            void* workspace, int ctas, cudaStream_t s) {
  const int group = p.num_q_heads / p.cache.num_heads;
  const long long tokens = rows / group;
  long long keys = (long long)p.table_width * p.cache.page_size;  // the line of units is counted in 32 bits
  if (p.window > 0 && p.window + tokens < keys) keys = p.window + tokens;
  const long long items = p.num_tokens / tokens + p.num_requests;
  if (items * (keys / UNIT + 2 + LEAD) > 0x7fffffffLL / p.cache.num_heads) return cudaErrorNotSupported;
  RowsArgs a;
  a.p = p;
  a.sc = sc;
  a.counters = static_cast<unsigned*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + KDA_ATTENTION_WORKSPACE_ZEROED);
  a.q_wide = (reinterpret_cast<uintptr_t>(p.q.ptr) & 15) == 0 && p.q.b_stride % 8 == 0 && p.q.h_stride % 8 == 0;
  a.box = p.cache.page_size < UNIT ? p.cache.page_size : UNIT;
  a.group = group;
  a.item_tokens = (int)tokens;
  a.inv_group = 65536u / (unsigned)group + 1u;  // for row < 32 and group <= 32 the excess is below 32 / 2^16 < 1 / group
  const int D = p.cache.head_dim;
  a.slot_floats = (size_t)rows * (D + 2);  // less than the room of kda_paged_attention's parts
  if (D == 128)
    return rows == 4 ? launch_rows<128, 4>(a, ctas, s) : rows == 8 ? launch_rows<128, 8>(a, ctas, s)
           : rows == 16 ? launch_rows<128, 16>(a, ctas, s) : launch_rows<128, 32>(a, ctas, s);
  return rows == 4 ? launch_rows<64, 4>(a, ctas, s) : rows == 8 ? launch_rows<64, 8>(a, ctas, s)
         : rows == 16 ? launch_rows<64, 16>(a, ctas, s) : launch_rows<64, 32>(a, ctas, s);
}

}  // namespace kda
