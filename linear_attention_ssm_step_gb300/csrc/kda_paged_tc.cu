// kda_paged_tc.cu - paged attention on the fifth-generation tensor cores
// (include/kda_paged.h), head_dim 64 or 128; FP8, over a cache in 8 bits
// (include/kda_paged_fp8.h), requests of more than 32 rows a key-value head (for
// fewer: kda_paged_fp8_rows.cu).
//
// Mathematics. For one key-value head and the rows that read it, over units of
// 128 keys: S = Q K^T, P = exp2(c (S - m)) with c = scale log2 e and m a running
// reference of the row's maximum, l += sum P, O += P V; out = O / l, lse = m
// scale + ln l. m follows the maximum only when that has grown by more than 8
// in log2 units (then O and l are scaled down once): P stays below 2^8, which
// changes no relative precision, and most units need no pass over O. P is rounded to bf16 for the product with V, since
// both operands of a product have one 16-bit type (fp32 weights would take two or three products); l sums it before that.
// Outputs are off by 2.0..2.4e-3 of their size against 64 bits, by 1.6..1.7e-3 where the weights are fp32: rounding the
// output to bf16 is most of both. S, m, l, O and the parts are fp32.
//
// Rows. The query heads of one key-value head and consecutive new tokens of one
// request are the rows of a tile of 128 (token-major), so that a key is read
// once for all of them: floor(128 / g) tokens of g heads. An item is one key-
// value head and two such tiles; its units run over the keys any of its rows
// sees.
//
// Split. The items of all requests form one line of units, which the persistent
// CTAs (one an SM) share out evenly, at any unit: lengths may be as ragged as
// they like and few rows over a long cache still fill the GPU. Every CTA finds
// its share itself from the requests' lengths. An item cut between CTAs leaves
// unnormalised O, m and l of each part in the workspace, and the CTA that
// finishes last joins them in the order of the parts: the same bits whichever
// comes last.
//
// A CTA is twelve warps: two softmax groups of four (a thread per row), and one
// warp each that loads keys and values (one tensor-map copy per page and 64
// columns), that issues the products, that walks the line, and that asks the
// next runs' queries into L2. With two row tiles, group t owns tile t; a single
// tile (decode, verify) takes the units in turn with the groups, each with its
// own O, joined at the end, so that in either case one group's exponentials run
// while the other's products do. S and P share tensor-memory columns: P (bf16)
// overwrites the S it came from and enters the second product from there. The
// next S into the same columns is issued right behind that product: the products
// of a CTA are issued by one warp and executed in the order of their issue.
//
// What bounds it. Few rows: memory (64 decode requests of 2048..8192 cached
// tokens, 8 key-value heads of 128: 192..197 us, 6.4 TB/s, 94 % of a plain copy).
// Chunks: the chain score product - registers - maximum - exponentials - weights
// - value product of a tile, 2600 cycles a pair of units where the tensor core
// needs 2048 (two chunks of 2048 tokens over 4096..16384 cached, 32 query heads:
// 530 us alone, 1.66 PFLOP/s, and 560..585 us in a loop, under the power cap).
// Small calls: latency (one decode request of 1000 tokens 10.1 us). Once-a-run code
// is kept short and in loops that are not unrolled: it is fetched anew each run.
//
// FP8. The codes of the keys go into the first product as they are, with the
// queries as two E4M3 numbers each (query_codes in kda_paged_line.cuh): two
// products at twice the rate of one of bf16, without a conversion of the keys,
// which read half the shared memory. Values become fp16, which holds them exactly,
// on the way from one buffer in shared memory to another, by four more warps: a
// product takes operands of one width, and weights in 8 bits would be too coarse.
// A block's scale of 16 keys is a factor of its scores, in the multiply-add that
// forms the exponent (y = f s + log2 vs), and the value scale an addend there: the
// weights that meet the values are exp2(y - m), their reference m of fp32 y, so
// that the sum l takes them times 1 / vs. fp16 weights of up to 2^14 (a reference
// set at 2^6, and 8 of growth) hold 11 bits down to 2^-14, so that keys of 2^-20
// of the largest weight still count.
// Two chunks of 2048 tokens over 4096..16384 cached, 32 query heads: 735 to 741 us,
// 1.37 PFLOP/s. What that costs beside the 16-bit cache's chain was measured on an
// earlier build of 767 to 772 us: 733 with the conversion of the values left out,
// 758 with one factor for all keys in place of the block scales, 698 with neither.
// Another build spent 13700 cycles a run until its queries were codes (the 16-bit
// kernel has them after 6600). How the loop over the units is compiled depends on
// code that runs once a run: builds that differ in that alone took 756 to 853.
// Scores taken twice from tensor memory to save registers: 1054.
#include <math.h>

#include <type_traits>

#include "kda_paged_launch.h"
#include "kda_paged_line.cuh"

namespace kda {

namespace {

constexpr int TILE = 128;   // rows a tile
constexpr int SOFTMAX_THREADS = 256;
// Which of the SM's four schedulers (warp mod 4) has which of them: with the loads on 1, beside softmax warps 1 and 5,
// verify and decode steps take 54.6 and 193.6 us, on 0 57.2 and 195.0; chunks 561 against 560.
constexpr int PRODUCT_WARP = 8, LOAD_WARP = 9, WALK_WARP = 10, AHEAD_WARP = 11;
constexpr int CONVERT_WARP = 12, CONVERT_WARPS = 4, CONVERT_REGS = 32;  // of a cache in 8 bits
constexpr int FIRST = 96;   // keys of a unit whose weights are handed over first, while the others' are formed
constexpr int RING = 4;  // segments the walking warp may be ahead
// What an item costs beside its units (its queries, its end), in units: each item takes LEAD + its units of the line. A
// first chunk of 4096 tokens, whose items have 1 to 32 units: 122 us at 3, 118 at 4, 119.5 at 5 (two tiles); 32 verify
// requests: 56.7 us at 1, 55.7 at 2, 54.6 at 4, 56.4 at 6 (one tile).
constexpr int LEAD = 4;
// A cache in 8 bits, whose queries become codes: a first chunk of 4096 tokens 179 us at 4, 171 at 7, 174 at 10.
constexpr int LEAD8 = 7;
constexpr int SCALES = 2;                                  // pairs of units whose scales are held
constexpr int BLOCK = KDA_FP8_SCALE_TOKENS, BLOCKS = UNIT / BLOCK;  // keys a scale, scales a unit

// FP8: a cache in 8 bits. A tile of queries is then two of E4M3 numbers, of half the size each.
template <int D, bool FP8>
struct Shape {
  // Registers a thread after the split: 256 x 208 + 128 x 88 = 384 x 168, what the block launches with; with the warps of
  // a cache in 8 bits 256 x 216 + 128 x 48 + 128 x 32 = 512 x 128.
  static constexpr int THREADS = FP8 ? 512 : 384;
  static constexpr int SOFTMAX_REGS = FP8 ? 216 : 208, OTHER_REGS = FP8 ? 48 : 88;
  static constexpr int K_STAGES = D == 128 ? 3 : 4;
  static constexpr int V_STAGES = D == 128 ? 2 : 4;
  static constexpr int R_STAGES = !FP8 ? 0 : D == 128 ? 3 : 4;  // units of values as they are in the cache
  static constexpr uint32_t TILE_BYTES = TILE * D * 2;         // also a unit of 16-bit keys or values
  static constexpr uint32_t CODE_BYTES = UNIT * D;             // a unit of codes
  static constexpr uint32_t KEY_BYTES = FP8 ? CODE_BYTES : TILE_BYTES;
  static constexpr uint32_t Q0 = 0, Q1 = TILE_BYTES;
  static constexpr uint32_t K0 = 2 * TILE_BYTES;
  static constexpr uint32_t R0 = K0 + K_STAGES * KEY_BYTES;
  static constexpr uint32_t V0 = R0 + R_STAGES * CODE_BYTES;
  // Where queries are brought in 16 bits: into their own place, but for codes of head_dim 64, whose rows lie otherwise.
  static constexpr bool OWN_RAW = FP8 && D == 64;
  static constexpr uint32_t RAW0 = OWN_RAW ? V0 + V_STAGES * TILE_BYTES : Q0, RAW1 = RAW0 + TILE_BYTES;
  static constexpr uint32_t END = V0 + V_STAGES * TILE_BYTES + (OWN_RAW ? 2 * TILE_BYTES : 0);
};

// A unit's scales by blocks: of the keys, and log2 and reciprocal of the values'.
struct alignas(16) UnitScales {
  float key[BLOCKS], log_value[BLOCKS], inv_value[BLOCKS];
};

template <int D, bool FP8>
struct Shared8 {};
template <int D>
struct Shared8<D, true> {
  static constexpr int R_STAGES = Shape<D, true>::R_STAGES;
  uint64_t r_full[R_STAGES], r_empty[R_STAGES], scale_full[SCALES], scale_empty[SCALES];
  UnitScales scales[SCALES][2];
};

template <int D, bool FP8>
struct Shared : Shared8<D, FP8> {
  using S = Shape<D, FP8>;
  uint64_t k_full[S::K_STAGES], k_empty[S::K_STAGES], v_full[S::V_STAGES], v_empty[S::V_STAGES];
  uint64_t v_tail, q_full[2], s_full[2], p_full[2][2], o_done[2], seg_full[RING], seg_empty[RING], drain;
  Segment seg[RING];
  // The groups' m and l when both share a tile. At the start of a run on a cache in 8 bits, m1[t][x] is the power of two by
  // which the query of thread x of group t was brought down: that thread alone reads it then, and writes m there later.
  union {
    float m1[2][TILE];
    int warp_sum[S::THREADS / 32];  // before the first run
  };
  float l1[2][TILE];
  LineStart start;
  uint32_t tmem;
  int last_part;
};

// ---------------------------------------------------------------- tensor memory in 32-column blocks

// 32 columns, without the wait.
__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// Names 32 registers a load fills, so that no use of them moves above the wait before it.
__device__ __forceinline__ void hold32(uint32_t* r) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29])
               :);
  asm volatile("" : "+r"(r[30]), "+r"(r[31]));
}

__device__ __forceinline__ void ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// Two fp32 at once: x y + z, x + y.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
// -m c twice; 0 for a row that has seen no key.
__device__ __forceinline__ uint64_t reference(float m, float c) {
  const float base = m == -INFINITY ? 0.f : -m * c;
  return pair(base, base);
}

// Weights exp2(c s + base) of N scores, in bf16 pairs; their fp32 sums are added to `sum`.
template <int N>
__device__ __forceinline__ void weights(const uint32_t* s, uint64_t c2, uint64_t base2, uint64_t (&sum)[4], uint32_t* w) {
#pragma unroll
  for (int j = 0; j < N / 2; ++j) {
    float e0, e1;
    unpair(fma2(pair(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), c2, base2), e0, e1);
    e0 = ex2(e0);
    e1 = ex2(e1);
    sum[j & 3] = add2(sum[j & 3], pair(e0, e1));
    w[j] = pack_bf16x2(e0, e1);
  }
}

// D = A B^T over N / 16 K steps, issued by one elected lane of a converged warp, and then an arrival on `done` (and on
// `free` if it is not 0) once they are complete. One statement, so that the descriptors of all steps are formed by adding
// constants: the warp that issues runs on its own, and every instruction of it costs the tensor core five cycles or more.
// A in shared memory, both operands K-major: a K step is 32 bytes, the fifth step on in the next 64-column region.
template <int N>
__device__ __forceinline__ void issue_scores(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t done, uint32_t free) {
  static_assert(N == 64 || N == 128, "");
  if constexpr (N == 128)
    asm volatile(
        "{\n\t.reg .pred p, q, t;\n\t.reg .b32 r;\n\t.reg .b64 x, y;\n\t"
        "elect.sync r|p, 0xffffffff;\n\tsetp.ne.b32 t, 0, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, t;\n\t"
        "add.s64 x, %1, 2;\n\tadd.s64 y, %2, 2;\n\t@p tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, q;\n\t"
        "add.s64 x, %1, 4;\n\tadd.s64 y, %2, 4;\n\t@p tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, q;\n\t"
        "add.s64 x, %1, 6;\n\tadd.s64 y, %2, 6;\n\t@p tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, q;\n\t"
        "add.s64 x, %1, 1024;\n\tadd.s64 y, %2, 1024;\n\t@p tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, q;\n\t"
        "add.s64 x, %1, 1026;\n\tadd.s64 y, %2, 1026;\n\t@p tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, q;\n\t"
        "add.s64 x, %1, 1028;\n\tadd.s64 y, %2, 1028;\n\t@p tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, q;\n\t"
        "add.s64 x, %1, 1030;\n\tadd.s64 y, %2, 1030;\n\t@p tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, q;\n\t"
        "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t"
        "setp.ne.and.b32 p, %5, 0, p;\n\t"
        "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(done), "r"(free)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q, t;\n\t.reg .b32 r;\n\t.reg .b64 x, y;\n\t"
        "elect.sync r|p, 0xffffffff;\n\tsetp.ne.b32 t, 0, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, t;\n\t"
        "add.s64 x, %1, 2;\n\tadd.s64 y, %2, 2;\n\t@p tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, q;\n\t"
        "add.s64 x, %1, 4;\n\tadd.s64 y, %2, 4;\n\t@p tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, q;\n\t"
        "add.s64 x, %1, 6;\n\tadd.s64 y, %2, 6;\n\t@p tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, q;\n\t"
        "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t"
        "setp.ne.and.b32 p, %5, 0, p;\n\t"
        "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(done), "r"(free)
        : "memory");
}

// The same for E4M3 operands, 32 a K step: the upper parts of the queries, then the lower ones (`tile` bytes on, in the
// descriptor's units of 16), with the same keys.
template <int N>
__device__ __forceinline__ void issue_scores8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t done, uint32_t free) {
  static_assert(N == 64 || N == 128, "");
#define KDA_MMA8(A, B, ACC) "@p tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], " A ", " B ", %3, " ACC ";\n\t"
#define KDA_MMA8_AT(X, Y) "add.s64 x, %1, " X ";\n\tadd.s64 y, %2, " Y ";\n\t" KDA_MMA8("x", "y", "q")
#define KDA_SCORES8(REST)                                                                                        \
  asm volatile(                                                                                                  \
      "{\n\t.reg .pred p, q, t;\n\t.reg .b32 r;\n\t.reg .b64 x, y;\n\t"                                        \
      "elect.sync r|p, 0xffffffff;\n\tsetp.ne.b32 t, 0, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t" KDA_MMA8("%1", "%2", "t") REST \
      "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t"                      \
      "setp.ne.and.b32 p, %5, 0, p;\n\t"                                                                        \
      "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t}" ::"r"(d),           \
      "l"(a), "l"(b), "r"(idesc), "r"(done), "r"(free)                                                           \
      : "memory")
  if constexpr (N == 128)
    KDA_SCORES8(KDA_MMA8_AT("2", "2") KDA_MMA8_AT("4", "4") KDA_MMA8_AT("6", "6") KDA_MMA8_AT("1024", "0")
                KDA_MMA8_AT("1026", "2") KDA_MMA8_AT("1028", "4") KDA_MMA8_AT("1030", "6"));
  else
    KDA_SCORES8(KDA_MMA8_AT("2", "2") KDA_MMA8_AT("512", "0") KDA_MMA8_AT("514", "2"));
#undef KDA_SCORES8
#undef KDA_MMA8_AT
#undef KDA_MMA8
}

// D += A B over keys [0, 96) or [96, 128) of a unit (D = on the first if `fresh`), A (bf16 pairs) in tensor memory, 8
// columns a K step; B with N contiguous, 2048 bytes a K step. The second part is followed by the arrivals.
__device__ __forceinline__ void issue_values_first(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t fresh) {
  asm volatile(
      "{\n\t.reg .pred p, q, t;\n\t.reg .b32 r, x;\n\t.reg .b64 y;\n\t"
      "elect.sync r|p, 0xffffffff;\n\tsetp.eq.b32 t, %4, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
"@p tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, t;\n\t"
"add.u32 x, %1, 8;\n\tadd.s64 y, %2, 128;\n\t@p tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, q;\n\t"
"add.u32 x, %1, 16;\n\tadd.s64 y, %2, 256;\n\t@p tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, q;\n\t"
"add.u32 x, %1, 24;\n\tadd.s64 y, %2, 384;\n\t@p tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, q;\n\t"
"add.u32 x, %1, 32;\n\tadd.s64 y, %2, 512;\n\t@p tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, q;\n\t"
"add.u32 x, %1, 40;\n\tadd.s64 y, %2, 640;\n\t@p tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, q;\n\t"
"}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(fresh)
      : "memory");
}
__device__ __forceinline__ void issue_values_last(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t done,
                                                  uint32_t free) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b32 r, x;\n\t.reg .b64 y;\n\t"
      "elect.sync r|p, 0xffffffff;\n\tsetp.eq.b32 q, 0, 0;\n\t"
"add.u32 x, %1, 48;\n\tadd.s64 y, %2, 768;\n\t@p tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, q;\n\t"
"add.u32 x, %1, 56;\n\tadd.s64 y, %2, 896;\n\t@p tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, q;\n\t"

      "setp.ne.and.b32 q, %4, 0, p;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t"
      "setp.ne.and.b32 p, %5, 0, p;\n\t"
      "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(done), "r"(free)
      : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* src) { asm volatile("prefetch.global.L2 [%0];" ::"l"(src)); }

// The thread's number, read again.
__device__ __forceinline__ uint32_t fresh_tid() {
  uint32_t x;
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(x));
  return x;
}

__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// The value operand: 64-column regions of TILE rows (keys) x 128 bytes, N (the columns) contiguous. Leading byte
// offset: the next 64 columns, TILE * 128 bytes on; stride byte offset: the next 8 keys, 1024 bytes on. A K step of
// 16 keys adds 2048 bytes to the start address.
__device__ __forceinline__ uint64_t value_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)((TILE * 128u) >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
         ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}
constexpr uint32_t B_MN_MAJOR = 1u << 16;  // instruction descriptor: B with N contiguous
// Formats of A and B in it (bits 7-9, 10-12): 0 is fp16 for products of 16-bit numbers, E4M3 for those of 8-bit ones.
constexpr uint32_t FORMATS = 63u << 7;

// Weights exp2(f s + base) of a block of 16 scores as fp16 pairs; their fp32 sum, times inv, is added to `sum`.
__device__ __forceinline__ void block_weights(const uint32_t* s, float f, float base, float inv, uint64_t& sum, uint32_t* w) {
  const uint64_t f2 = pair(f, f), base2 = pair(base, base);
  uint64_t part[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < BLOCK / 2; ++j) {
    float e0, e1;
    unpair(fma2(pair(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), f2, base2), e0, e1);
    e0 = ex2(e0);
    e1 = ex2(e1);
    part[j & 1] = add2(part[j & 1], pair(e0, e1));
    w[j] = pack_f16x2(e0, e1);
  }
  sum = fma2(add2(part[0], part[1]), pair(inv, inv), sum);
}

__device__ __forceinline__ float4 ld_shared4(const float* p) {
  float4 r;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "r"(smem_addr(p)) : "memory");
  return r;
}

__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(n) : "memory");
}

constexpr float LOG2E = 1.4426950408889634f;
constexpr float SLACK = 8.f;  // growth of the maximum (log2) that the reference may lag behind
constexpr float LIFT = 6.f;   // log2 of the largest fp16 weight when the reference is set: SLACK above it is below 2^15

struct AttnArgs {
  kda_attention_params p;
  kda_paged_scales sc;  // of a cache in 8 bits
  float* parts;        // workspace: 2 slots a CTA, each [D / 4][2 TILE] float4 of unnormalised O, then [2 TILE] of (m, l)
  unsigned* counters;  // one a CTA, zero between calls
  int q_wide, out_wide;
  int box;             // keys a copy brings: min(page_size, UNIT)
  int group, tile_tokens;  // query heads a key-value head, tokens a tile
  unsigned inv_group;      // row / group = row * inv_group >> 16
};

// A part's O by groups of four columns, the rows of a group side by side: a warp's threads (a row each) write and read
// whole lines.
template <int D>
__device__ __forceinline__ float4* part_o(const AttnArgs& a, int slot) {
  return reinterpret_cast<float4*>(a.parts + (size_t)slot * (2 * TILE) * (D + 2));
}
template <int D>
__device__ __forceinline__ float2* part_ml(const AttnArgs& a, int slot) {
  return reinterpret_cast<float2*>(a.parts + (size_t)slot * (2 * TILE) * (D + 2) + (size_t)(2 * TILE) * D);
}

}  // namespace

// Rows [from, to) of a tile of queries in 16 bits to codes, by the 128 threads of a group, each the chunks (8 numbers, D / 8 a
// row) that it has brought, from `raw` on. up, also: where the powers of two go by which rows were brought down. A function of
// its own, not inlined: inside the kernel it changed how the loop over the units was compiled (two chunks of 2048 tokens over
// 4096..16384 cached 788 us, against 756; with two rows a thread at a time 852).
template <int D>
__device__ __noinline__ void queries_to_codes(const uint8_t* raw, uint8_t* codes, float* up, float* also, int from, int to) {
  constexpr int CHUNKS = D / 8, ROUND = TILE / CHUNKS, N = 2;
  const int x = (int)(fresh_tid() & (TILE - 1)), ch = x % CHUNKS;
#pragma unroll 1
  for (int r0 = from; r0 < to; r0 += N * ROUND) {  // the same for the whole warp
    uint4 z[N];
    int e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      z[i] = make_uint4(0, 0, 0, 0);
      if (r0 + i * ROUND + x / CHUNKS < to) z[i] = *reinterpret_cast<const uint4*>(raw + (r0 - from + i * ROUND) * 128);
    }
    query_exponents<N, CHUNKS>(z, e);
    __syncwarp();  // the rows' chunks are read: for head_dim 128 their codes go where they lie
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = r0 + i * ROUND + x / CHUNKS;
      uint2 hi, lo;
      query_codes(z[i], e[i], hi, lo);
      if (r >= to) continue;
      uint8_t* const at = codes + code_chunk<D>(r, ch >> 1) + (ch & 1) * 8;
      *reinterpret_cast<uint2*>(at) = hi;
      *reinterpret_cast<uint2*>(at + UNIT * D) = lo;
      if (ch == 0) up[r] = also[r] = query_up(e[i]);
    }
  }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(Shape<D, FP8>::THREADS, 1)
    kda_paged_attention_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                                  const __grid_constant__ AttnArgs a) {
  using S = Shape<D, FP8>;
  constexpr int THREADS = S::THREADS;
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle's atoms are 1024-byte aligned
  Shared<D, FP8>& sh = *reinterpret_cast<Shared<D, FP8>*>(smem + S::END);
  const kda_attention_params& p = a.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = a.group;
  const int tpt = a.tile_tokens, w = 2 * tpt;  // tokens a tile, an item
  const int window = p.window;

  if (warp == 0) {  // a lane a stage: one thread would take a microsecond
    if (lane < S::K_STAGES) {
      mbar_init_only(&sh.k_full[lane], 1);
      mbar_init_only(&sh.k_empty[lane], 1);
    }
    if (lane < S::V_STAGES) {
      mbar_init_only(&sh.v_full[lane], FP8 ? CONVERT_WARPS : 1);
      mbar_init_only(&sh.v_empty[lane], 1);
    }
    if constexpr (FP8) {
      if (lane < S::R_STAGES) {
        mbar_init_only(&sh.r_full[lane], 1);
        mbar_init_only(&sh.r_empty[lane], CONVERT_WARPS);
      }
      if (lane < SCALES) {
        mbar_init_only(&sh.scale_full[lane], 1);
        mbar_init_only(&sh.scale_empty[lane], SOFTMAX_THREADS / 32);  // an arrival a warp
      }
    }
    if (lane < RING) {
      mbar_init_only(&sh.seg_full[lane], 1);
      // the loading, product and prefetching warps, both softmax groups; the converting warps
      mbar_init_only(&sh.seg_empty[lane], FP8 ? 5 + CONVERT_WARPS : 5);
    }
    if (lane < 2) {
      mbar_init_only(&sh.q_full[lane], TILE);
      mbar_init_only(&sh.s_full[lane], 1);
      mbar_init_only(&sh.p_full[lane][0], TILE / 32);  // an arrival a warp
      mbar_init_only(&sh.p_full[lane][1], TILE / 32);
      mbar_init_only(&sh.o_done[lane], 1);
    }
    if (lane == 2) mbar_init_only(&sh.v_tail, 1);
    if (lane == 3) mbar_init_only(&sh.drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  } else if (warp == LOAD_WARP && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
  }

  earlier_work();

  // ---- this CTA's share of the line of units
  const int cta = blockIdx.x;
  const LineShare line = line_share<THREADS, FP8 ? LEAD8 : LEAD>(p, w, sh.warp_sum, sh.start);
  if (blockIdx.x == 0 && line.bad && p.error_word) atomicOr(p.error_word, line.bad);
  if (cta >= line.ctas) return;  // the whole CTA: nothing allocated yet
  if (warp == PRODUCT_WARP) tmem_alloc(&sh.tmem, 512);
  tc_fence_before();
  const int end = line_end(p, line);
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t S_COL = tmem, O_COL = tmem + 2 * TILE;

  if (FP8 && warp >= CONVERT_WARP) {
    if constexpr (FP8) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CONVERT_REGS));
      bool alive = true;
      // ---- values from codes to fp16, which holds them exactly, in the layout of the product: a lane takes 16 codes of a
      // key, a warp groups of 8 keys. Both layouts are swizzled; the lanes of a quarter warp, which access shared memory
      // together, take four chunks of a row r and of a row r ^ 5 (head_dim 64: of rows r and r + 1, which lie in 128 bytes),
      // whose places differ in both. What a lane adds to the group's address never changes.
      // Keys that are not in use become zeros: their weights are zero, but zero times what lies there need not be.
      constexpr int HALVES = D / 64;  // of a group's rows
      const uint32_t c = lane & 3, q = lane >> 3;
      const uint32_t row = D == 128 ? (lane & 4 ? q ^ 5 : q) : lane >> 2;
      const uint32_t from = code_chunk<D>(row, c), to = row * 128 + ((2 * c ^ row) & 7) * 16;
      uint32_t n = 0;
      for (uint32_t in = 0; alive; ++in) {
        const uint32_t slot = in % RING;
        alive = warp_wait(&sh.seg_full[slot], (in / RING) & 1);
        if (!alive) break;
        const int ntok = sh.seg[slot].ntok, u0 = sh.seg[slot].u0, u1 = sh.seg[slot].u1, lo = sh.seg[slot].lo, hi = sh.seg[slot].hi;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.seg_empty[slot]);
        if (ntok < 0) break;
        for (int u = u0; u < u1; ++u, ++n) {
          const uint32_t rs = n % S::R_STAGES, vs = n % S::V_STAGES;
          alive = warp_wait(&sh.r_full[rs], (n / S::R_STAGES) & 1) && warp_wait(&sh.v_empty[vs], (n / S::V_STAGES + 1) & 1);
          if (!alive) break;
          constexpr int GROUPS = UNIT / 8 / CONVERT_WARPS;  // of a warp
          const int key0 = u * UNIT + (warp - CONVERT_WARP) * GROUPS * 8;
          const uint8_t* const src = smem + S::R0 + rs * S::CODE_BYTES + (warp - CONVERT_WARP) * (GROUPS * 8 * D);
          uint8_t* const dst = smem + S::V0 + vs * S::TILE_BYTES + (warp - CONVERT_WARP) * (GROUPS * 1024) + to;
          const bool ragged = lo > u * UNIT || hi < (u + 1) * UNIT;
          static_assert(GROUPS == 4, "");
#pragma unroll
          for (int part = 0; part < 2 * HALVES; ++part) {
            const int half = part / 2, i0 = part % 2 * 2;
            uint4 z[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) z[i] = *reinterpret_cast<const uint4*>(src + (i0 + i) * 8 * D + (from ^ (half * 64)));
            if (__builtin_expect(ragged, 0)) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int key = key0 + (i0 + i) * 8 + (int)row;
                if (key < lo || key >= hi) z[i] = make_uint4(0, 0, 0, 0);
              }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint8_t* const at = dst + half * (TILE * 128) + (i0 + i) * 1024;
              *reinterpret_cast<uint4*>(at) = make_uint4(codes_to_f16x2(z[i].x), codes_to_f16x2(z[i].x >> 16),
                                                         codes_to_f16x2(z[i].y), codes_to_f16x2(z[i].y >> 16));
              uint8_t* const beside = at + (((2 * c ^ row) & 1) ? -16 : 16);  // the place ^ 16
              *reinterpret_cast<uint4*>(beside) = make_uint4(codes_to_f16x2(z[i].z), codes_to_f16x2(z[i].z >> 16),
                                                             codes_to_f16x2(z[i].w), codes_to_f16x2(z[i].w >> 16));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sh.v_full[vs]);
            mbar_arrive(&sh.r_empty[rs]);
          }
        }
      }
      if (!alive && lane == 0 && p.error_word) atomicOr(p.error_word, KDA_ERR_TIMEOUT);
      __syncwarp();
    }
  } else if (warp >= SOFTMAX_THREADS / 32) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::OTHER_REGS));
    bool alive = true;

    if (warp == WALK_WARP) {
      // ---- the line of units, cut into segments
      uint32_t out = 0;
      auto put = [&](Segment g2) {
        g2.dual = g2.ntok > tpt;
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
      alive = line_walk<FP8 ? LEAD8 : LEAD>(p, w, line, end, sh.start, put);
    } else if (warp == LOAD_WARP) {
      // ---- keys and values of the CTA's units, a lane per copy; keys one unit ahead
      const int P = p.cache.page_size, box = a.box;
      constexpr int HALVES = FP8 ? 1 : D / 64;  // copies of a piece, by columns
      const int copies = (UNIT / box) * HALVES;
      const int piece = lane / HALVES, half = lane % HALVES;  // which keys of the unit, which columns
      uint32_t kn = 0, vn = 0, tails = 0;
      bool bad_page = false, pending = false;  // pending: a ragged unit of values is on its way
      int first = 0, last = UNIT;              // the keys of it that are in use
      // Weights of unseen keys are zero, but zero times what lies there need not be: clear those rows. Done when the next
      // values are to be loaded, so that the keys of the next run do not wait for it.
      auto clear_tail = [&]() {
        pending = false;
        if (!warp_wait(&sh.v_tail, tails & 1)) return false;
        ++tails;
        const uint32_t st = (vn - 1) % S::V_STAGES;
        uint8_t* const dst = smem + S::V0 + st * S::TILE_BYTES;
        for (int x = lane; x < TILE * (D / 8); x += 32) {
          const int row = (x >> 3) & (TILE - 1);
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
        // up to 32 copies: a unit of 128 keys of 128 columns in pages of 16 is 8 pieces, 16 copies
        auto load = [&](int u, bool values) {
          const int key = u * UNIT + piece * box;
          const bool wanted = lane < copies && key < sg.hi && key + box > sg.lo;
          int page = 0;
          if (wanted) {
            page = table[key / P];
            if (page < 0 || page >= p.cache.num_pages) {
              page = p.cache.num_pages;  // past the end: the copy brings zeros
              bad_page = true;
            }
          }
          const uint32_t n = values ? vn : kn, stages = values ? (FP8 ? S::R_STAGES : S::V_STAGES) : S::K_STAGES, st = n % stages;
          uint64_t *bar = values ? &sh.v_full[st] : &sh.k_full[st], *empty = values ? &sh.v_empty[st] : &sh.k_empty[st];
          uint8_t* dst = smem + (values ? S::V0 : S::K0) + st * (values ? S::TILE_BYTES : S::KEY_BYTES);
          if constexpr (FP8)
            if (values) {
              bar = &sh.r_full[st];
              empty = &sh.r_empty[st];
              dst = smem + S::R0 + st * S::CODE_BYTES;
            }
          if (!warp_wait(empty, (n / stages + 1) & 1)) return false;
          constexpr uint32_t ROW = FP8 ? D : 128;  // bytes a copy brings of a key
          const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, wanted)) * (uint32_t)box * ROW;
          if (values && !FP8) {
            first = max(sg.lo - u * UNIT, 0);
            last = min(sg.hi - u * UNIT, UNIT);
            pending = first > 0 || last < UNIT;
            if (pending) bar = &sh.v_tail;
          }
          if (values) {
            ++vn;
          } else {
            ++kn;
          }
          if (lane == 0) mbar_expect_tx(bar, bytes);
          __syncwarp();
          if (wanted)
            tma_load_4d(dst + half * (TILE * 128) + piece * box * ROW, values ? &vmap : &kmap, half * 64, key % P, sg.head,
                        page, bar);
          return true;
        };
        alive = load(sg.u0, false);
        for (int u = sg.u0; alive && u < sg.u1; ++u) {
          if (u + 1 < sg.u1) alive = load(u + 1, false);
          if (alive && pending) alive = clear_tail();
          if (alive) alive = load(u, true);
        }
      }
      if (alive && pending) alive = clear_tail();
      if (bad_page && p.error_word) atomicOr(p.error_word, KDA_ERR_PAGES);
      if (!alive) {  // copies in flight land before the CTA leaves
        if (!FP8) mbar_drain_bounded(&sh.v_tail, tails & 1);
        for (uint32_t i = kn > (uint32_t)S::K_STAGES ? kn - S::K_STAGES : 0; i < kn; ++i)
          mbar_drain_bounded(&sh.k_full[i % S::K_STAGES], (i / S::K_STAGES) & 1);
        if constexpr (FP8) {
          for (uint32_t i = vn > (uint32_t)S::R_STAGES ? vn - S::R_STAGES : 0; i < vn; ++i)
            mbar_drain_bounded(&sh.r_full[i % S::R_STAGES], (i / S::R_STAGES) & 1);
        } else {
          for (uint32_t i = vn > (uint32_t)S::V_STAGES ? vn - S::V_STAGES : 0; i < vn; ++i)
            mbar_drain_bounded(&sh.v_full[i % S::V_STAGES], (i / S::V_STAGES) & 1);
        }
      }
    } else if (warp == AHEAD_WARP) {
      // ---- the queries of the runs to come into L2: from memory they take 2400 cycles, in which a run could not start.
      // FP8: and the scales of the runs' units, a pair of units at a time (16 lanes each: keys' blocks, then values'), the
      // next pair on its way meanwhile. The queries then come ahead by the units whose scales are held.
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
        auto fetch = [&](int u0) {
          const int u = u0 + (lane >> 4);
          if (u >= sg.u1) return 1.f;
          const int key = u * UNIT + b * BLOCK;
          if (key >= sg.hi || key + BLOCK <= sg.lo) return 1.f;  // no key of it is seen
          const int page = table[key / P];
          return page < 0 || page >= p.cache.num_pages ? 1.f : block_scale(of_values ? a.sc.v : a.sc.k, page, key % P, sg.head);
        };
        float next = 1.f;
        if constexpr (FP8) next = fetch(sg.u0);
        if (in > 0) {  // the first are being fetched
          const uint16_t* const q =
              static_cast<const uint16_t*>(p.q.ptr) + (int64_t)sg.row0 * p.q.b_stride + (int64_t)(sg.head * g) * p.q.h_stride;
          for (int r = lane; r < sg.ntok * g; r += 32) {
            const uint16_t* const src = q + (int64_t)(r / g) * p.q.b_stride + (int64_t)(r % g) * p.q.h_stride;
            for (int ch = 0; ch < D; ch += 64) prefetch_l2(src + ch);
          }
        }
        if constexpr (FP8) {
          for (int u = sg.u0; u < sg.u1; u += 2, ++pairs) {
            const float x = next;
            next = fetch(u + 2);
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
      }
    } else if (warp == PRODUCT_WARP) {
      // ---- the products: the values of a tile, then its next scores, tile after tile. A product takes 64 cycles of the
      // tensor core (head_dim 128) and its issue waits for room in a short queue, so little may stand between two of them:
      // the warp stays together and its operands in uniform registers, and a run of products is one statement (formed one by
      // one, with an election each, they took 85 cycles).
      const uint32_t base = smem_addr(smem), tm = uniform(tmem);
      constexpr uint32_t IDESC_S = idesc_bf16_f32(TILE, UNIT) & ~(FP8 ? FORMATS : 0u);
      constexpr uint32_t IDESC_O = (idesc_bf16_f32(TILE, D) & ~(FP8 ? FORMATS : 0u)) | B_MN_MAJOR;
      auto key_desc = [](uint32_t saddr) { return FP8 ? code_desc<D>(saddr) : sw128_desc(saddr); };
      uint32_t ks = 0, kp = 0, vs = 0, vp = 0, wp[2] = {0, 0}, qp = 0;
      for (uint32_t in = 0; alive; ++in) {
        const uint32_t slot = in % RING;
        alive = warp_wait(&sh.seg_full[slot], (in / RING) & 1);
        if (!alive) break;
        const int ntok = uniform(sh.seg[slot].ntok), n = uniform(sh.seg[slot].u1 - sh.seg[slot].u0);
        const int dual = uniform(sh.seg[slot].dual);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.seg_empty[slot]);
        if (ntok < 0) break;
        alive = warp_wait(&sh.q_full[0], qp) && warp_wait(&sh.q_full[1], qp);
        qp ^= 1;
        const uint64_t dq0 = key_desc(base + S::Q0), dq1 = dual ? key_desc(base + S::Q1) : dq0;
        auto scores = [&](int t, bool early = false) {
          const bool first = !dual || t == 0, last = !dual || t == 1;
          if (first && !early) {
            if (!warp_wait(&sh.k_full[ks], kp)) return false;
            tc_fence_after();
          }
          const uint64_t dk = key_desc(base + S::K0 + ks * S::KEY_BYTES);
          if constexpr (FP8)
            issue_scores8<D>(tm + t * TILE, t ? dq1 : dq0, dk, IDESC_S, smem_addr(&sh.s_full[t]),
                             last ? smem_addr(&sh.k_empty[ks]) : 0u);
          else
            issue_scores<D>(tm + t * TILE, t ? dq1 : dq0, dk, IDESC_S, smem_addr(&sh.s_full[t]),
                            last ? smem_addr(&sh.k_empty[ks]) : 0u);
          if (last && ++ks == S::K_STAGES) {
            ks = 0;
            kp ^= 1;
          }
          return true;
        };
        auto values = [&](int t, bool fresh, bool end) {
          const bool first = !dual || t == 0, last = !dual || t == 1;
          if (first && !warp_wait(&sh.v_full[vs], vp)) return false;
          if (dual && t == 0 && !end && !warp_wait(&sh.k_full[ks], kp)) return false;
          if (!warp_wait(&sh.p_full[t][0], wp[t])) return false;
          tc_fence_after();
          const uint64_t v = value_desc(base + S::V0 + vs * S::TILE_BYTES);
          issue_values_first(tm + 2 * TILE + t * D, tm + t * TILE, v, IDESC_O, fresh);
          if (!warp_wait(&sh.p_full[t][1], wp[t])) return false;
          tc_fence_after();
          issue_values_last(tm + 2 * TILE + t * D, tm + t * TILE, v, IDESC_O, end ? smem_addr(&sh.o_done[t]) : 0u,
                            last ? smem_addr(&sh.v_empty[vs]) : 0u);
          wp[t] ^= 1;
          if (last && ++vs == S::V_STAGES) {
            vs = 0;
            vp ^= 1;
          }
          return true;
        };
        if (dual) {
          alive = alive && scores(0) && scores(1);
          for (int i = 0; alive && i < n; ++i) {
            alive = values(0, i == 0, i + 1 == n) && (i + 1 == n || scores(0, true)) && values(1, i == 0, i + 1 == n) &&
                    (i + 1 == n || scores(1));
          }
        } else {
          alive = alive && scores(0) && (n < 2 || scores(1));
          for (int i = 0; alive && i < n; i += 2) {
            alive = values(0, i == 0, i + 2 >= n) && (i + 2 >= n || scores(0)) &&
                    (i + 1 >= n || (values(1, i == 0, i + 3 >= n) && (i + 3 >= n || scores(1))));
          }
        }
      }
      if (!alive) {  // products in flight end before the tensor memory goes
        tc_commit_w(&sh.drain);
        mbar_drain_bounded(&sh.drain, 0);
      }
    }
    if (!alive && lane == 0 && p.error_word) atomicOr(p.error_word, KDA_ERR_TIMEOUT);
    __syncwarp();
  } else {
    // ---- softmax: group t, thread (row) x
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::SOFTMAX_REGS));
    const int t = warp >> 2;
    const float c = p.scale * LOG2E;
    // A reference m is in units of the scores, or (FP8) their log2: times to_log2 it is log2, times to_ln ln.
    const float to_log2 = FP8 ? 1.f : c, to_ln = FP8 ? 0.6931471805599453f : p.scale;
    uint32_t seen_s = 0, runs = 0;  // scores waited for; ends of runs
    uint32_t pairs_before = 0;      // FP8: pairs of units before this run
    bool alive = true;
    auto div_g = [&](int row) { return (int)((uint32_t)row * a.inv_group >> 16); };
    // Where a thread stands is worked out anew for each part of a run: kept over the units, it would cost them registers.
    // Row (tensor-memory lane) of the tile; when copying a tile, with D / 8 threads a row, row and 16-byte chunk.
    constexpr int ROWS_A_ROUND = TILE / (D / 8), ROUNDS = TILE / ROWS_A_ROUND;  // a multiple of 8 rows a round
    struct Place {
      int x, row, ch;
      uint32_t at;  // of the chunk in a tile in shared memory, as the products read it
    };
    auto place = [] {
      Place q;
      q.x = (int)(fresh_tid() & (TILE - 1));
      q.row = q.x / (D / 8);
      q.ch = q.x % (D / 8);
      q.at = (uint32_t)((q.ch >> 3) * (TILE * 128) + q.row * 128 + (((q.ch ^ q.row) & 7) << 4));
      return q;
    };
    // Offset of row r of a tile (token r / g, head r % g) in a tensor of those strides (below 2^31, so one multiplication each).
    auto row_offset = [&](int r, int64_t b_stride, int64_t h_stride) {
      const int tk = div_g(r);
      return (int64_t)tk * (int)b_stride + (int64_t)(r - tk * g) * (int)h_stride;
    };
    // The queries of a run: a group's tile, or its half of the tile that both share.
    auto fetch_q = [&](const Segment& n) {
      const Place me = place();
      const int tile0 = n.dual ? t * tpt : 0;  // first token of the tile
      const int from = n.dual ? 0 : t * (TILE / 2);
      const int to = min(min(n.ntok - tile0, tpt) * g, n.dual ? TILE : from + TILE / 2);
      const uint16_t* const qg = static_cast<const uint16_t*>(p.q.ptr) + (int64_t)(n.row0 + tile0) * p.q.b_stride +
                                 (int64_t)(n.head * g) * p.q.h_stride + me.ch * 8;
      uint8_t* const qs = smem + (n.dual && t ? S::RAW1 : S::RAW0) + me.at + from * 128;
      if (a.q_wide) {  // asynchronously, all rounds in flight
#pragma unroll 4
        for (int k = 0; k < ROUNDS; ++k) {
          const int r = from + me.row + k * ROWS_A_ROUND;
          if (r < to) copy_async16(qs + k * (ROWS_A_ROUND * 128), qg + row_offset(r, p.q.b_stride, p.q.h_stride));
        }
        copy_async_wait();
      } else {
#pragma unroll 1
        for (int k = 0; k < ROUNDS; ++k) {
          const int r = from + me.row + k * ROWS_A_ROUND;
          if (r >= to) break;
          const uint16_t* const src = qg + row_offset(r, p.q.b_stride, p.q.h_stride);
          uint32_t e[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) e[j] = (uint32_t)src[2 * j] | ((uint32_t)src[2 * j + 1] << 16);
          *reinterpret_cast<uint4*>(qs + k * (ROWS_A_ROUND * 128)) = make_uint4(e[0], e[1], e[2], e[3]);
        }
      }
      if constexpr (FP8) {  // to codes, each thread the chunks that it has brought
        const bool both = !n.dual;
        queries_to_codes<D>(qs, smem + (n.dual && t ? S::Q1 : S::Q0), &sh.m1[t][0], both ? &sh.m1[1 - t][0] : &sh.m1[t][0], from, to);
      }
      fence_proxy_async_smem();
      mbar_arrive(&sh.q_full[t]);
    };
    for (uint32_t in = 0;; ++in) {
      const uint32_t slot = in % RING;
      alive = warp_wait(&sh.seg_full[slot], (in / RING) & 1);
      if (bar_any(1, SOFTMAX_THREADS, !alive)) {  // both groups leave together
        alive = false;
        break;
      }
      const Segment& sg = sh.seg[slot];  // read again where needed: registers are short
      if (sg.ntok < 0) break;
      const int dual = sg.dual;
      fetch_q(sg);
      float query_scale = 0.f;
      if constexpr (FP8) {
        bar_sync(2, SOFTMAX_THREADS);
        // Above 2^-100, so that the factor of no block (2^-40 at the least) is 0, which makes NaN of a masked score's -inf;
        // scores of codes stay below 2^-35 then, and are nothing in an exponent.
        query_scale = fmaxf(c * sh.m1[t][fresh_tid() & (TILE - 1)], 0x1p-100f);
      }

      // Keys [lo, hi) that this thread's row sees; a row of no token is carried along unmasked and goes nowhere.
      struct Row {
        int tok;  // of the item
        bool valid;
        int lo, hi;
      };
      auto my_row = [&] {
        Row r;
        const int tk = div_g((int)(fresh_tid() & (TILE - 1)));
        r.tok = (sg.dual ? t * tpt : 0) + tk;
        r.valid = tk < tpt && r.tok < sg.ntok;
        r.hi = r.valid ? sg.pos0 + r.tok + 1 : 0x7fffffff;
        r.lo = r.valid ? first_key(r.hi - 1, window) : 0;
        return r;
      };
      bool valid;
      int all_lo, all_hi;
      {
        const Row r = my_row();
        valid = r.valid;
        all_lo = __reduce_max_sync(0xffffffffu, r.lo);
        all_hi = __reduce_min_sync(0xffffffffu, r.hi);
      }
      const bool warp_valid = __any_sync(0xffffffffu, valid);
      const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t s_addr = S_COL + t * TILE + lane_base, o_addr = O_COL + t * D + lane_base;
      float m = -INFINITY, l = 0.f;  // m: the reference, in units of the scores
      const int step = dual ? 1 : 2;
      int units = 0;
      for (int u = sg.u0 + (dual ? 0 : t); u < sg.u1; u += step) {
        // FP8: what the unit's scales give is made ready while its scores are still being formed
        const uint32_t of_run = (uint32_t)(u - sg.u0), pair_of = pairs_before + of_run / 2;
        float f[FP8 ? BLOCKS : 1], log_value[FP8 ? BLOCKS : 1];
        if constexpr (FP8) {
          if (!dual || of_run % 2 == 0) alive = alive && warp_wait(&sh.scale_full[pair_of % SCALES], (pair_of / SCALES) & 1);
          if (!alive) break;
          const UnitScales& us = sh.scales[pair_of % SCALES][of_run % 2];
#pragma unroll
          for (int b = 0; b < BLOCKS; b += 4) {
            const float4 key = ld_shared4(us.key + b), lv = ld_shared4(us.log_value + b);
            f[b] = query_scale * key.x;
            f[b + 1] = query_scale * key.y;
            f[b + 2] = query_scale * key.z;
            f[b + 3] = query_scale * key.w;
            log_value[b] = lv.x;
            log_value[b + 1] = lv.y;
            log_value[b + 2] = lv.z;
            log_value[b + 3] = lv.w;
          }
        }
        alive = alive && warp_wait(&sh.s_full[t], seen_s & 1);
        if (!alive) break;
        if (warp_valid) {
          tc_fence_after();
          uint32_t s[UNIT];
#pragma unroll
          for (int i = 0; i < UNIT; i += 32) ld32(s_addr + i, s + i);
          ld_wait();
#pragma unroll
          for (int i = 0; i < UNIT; i += 32) hold32(s + i);
          const int k0 = u * UNIT;
          if (__builtin_expect(k0 + UNIT > all_hi || k0 < all_lo, 0)) {
            const Row r = my_row();
            const int from = r.lo - k0, to = r.hi - k0;
#pragma unroll
            for (int b = 0; b < UNIT; b += 32) {
              // bits [from, to) of this block
              const uint32_t bits = low_bits(min(max(to - b, 0), 32)) & ~low_bits(min(max(from - b, 0), 32));
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!(bits >> i & 1u)) s[b + i] = 0xff800000u;  // -inf
            }
          }
          auto give = [&](int h) {  // these weights are there: the products that take them may start
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[t][h]);
          };
          auto fade_o = [&](float fade) {
#pragma unroll 1
            for (int i = 0; i < D; i += 16) {  // 16 columns at a time: the 128 scores stay in registers
              float o[16];
              tmem_ld16(o_addr + i, o);
              uint32_t o2[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) o2[j] = __float_as_uint(o[j] * fade);
              tmem_st16(o_addr + i, o2);
            }
          };
          uint32_t wa[16];
          if constexpr (FP8) {
            // y = f s is a score in log2 units, f its block's factor; weights times value scales are exp2(y + log2 vs - m)
            float top = -INFINITY;
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) {
              const uint32_t* const x = s + b * BLOCK;
              float t0 = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1])), t1 = fmaxf(__uint_as_float(x[2]), __uint_as_float(x[3]));
#pragma unroll
              for (int j = 4; j < BLOCK; j += 4) {
                t0 = max3(t0, __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
                t1 = max3(t1, __uint_as_float(x[j + 2]), __uint_as_float(x[j + 3]));
              }
              top = fmaxf(top, fmaf(fmaxf(t0, t1), f[b], log_value[b]));
            }
            const bool grown = valid && top - m > LIFT + SLACK;  // m = -inf: any key (-inf less itself is no number)
            if (__builtin_expect(__any_sync(0xffffffffu, grown), 0)) {
              const float fade = grown ? ex2(m - (top - LIFT)) : 1.f;
              if (grown) m = top - LIFT;
              l *= fade;
              if (units > 0) fade_o(fade);  // the product of the unit before is done: these scores waited for it
            }
            const float base = m == -INFINITY ? 0.f : -m;
            uint64_t sum = 0;
            const UnitScales& us = sh.scales[pair_of % SCALES][of_run % 2];
#pragma unroll
            for (int b0 = 0; b0 < BLOCKS; b0 += 4) {
              const float4 lv = ld_shared4(us.log_value + b0), iv = ld_shared4(us.inv_value + b0);  // again: registers are short
              const float logs[4] = {lv.x, lv.y, lv.z, lv.w}, invs[4] = {iv.x, iv.y, iv.z, iv.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int b = b0 + i;
                block_weights(s + b * BLOCK, f[b], base + logs[i], invs[i], sum, wa + 8 * (b & 1));
                if (b & 1) st16(s_addr + (b - 1) * (BLOCK / 2), wa);
                if ((b + 1) * BLOCK == FIRST) give(0);
              }
            }
            give(1);
            float l0, l1;
            unpair(sum, l0, l1);
            l += l0 + l1;
          } else {
            const uint64_t c2 = pair(c, c);
            uint64_t sum[4] = {0, 0, 0, 0}, base2 = reference(m, c);
            float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < UNIT; i += 8)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                tops[j] = max3(tops[j], __uint_as_float(s[i + 2 * j]), __uint_as_float(s[i + 2 * j + 1]));
            const float top = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]);
            const bool grown = valid && top > m && (top - m) * c > SLACK;  // m = -inf: any key
            if (__builtin_expect(__any_sync(0xffffffffu, grown), 0)) {
              const float fade = grown ? ex2((m - top) * c) : 1.f;
              if (grown) m = top;
              l *= fade;
              if (units > 0) fade_o(fade);  // the product of the unit before is done: these scores waited for it
              base2 = reference(m, c);
            }
            weights<32>(s, c2, base2, sum, wa);
            st16(s_addr, wa);
            weights<32>(s + 32, c2, base2, sum, wa);
            st16(s_addr + 16, wa);
            weights<32>(s + 64, c2, base2, sum, wa);
            st16(s_addr + 32, wa);
            give(0);
            weights<32>(s + FIRST, c2, base2, sum, wa);
            st16(s_addr + FIRST / 2, wa);
            give(1);
            float l0, l1;
            unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), l0, l1);
            l += l0 + l1;
          }
        } else if (lane == 0) {
          mbar_arrive(&sh.p_full[t][0]);
          mbar_arrive(&sh.p_full[t][1]);
        }
        if constexpr (FP8) {
          __syncwarp();
          const bool last = u + 1 == sg.u1;
          // the pair's second unit, or its only one: where one group takes that, it arrives for both
          if (lane == 0 && (!dual || last || of_run % 2 == 1))
            mbar_arrive_n(&sh.scale_empty[pair_of % SCALES], !dual && last && of_run % 2 == 0 ? 2 : 1);
        }
        ++seen_s;
        ++units;
      }

      pairs_before += (uint32_t)(sg.u1 - sg.u0 + 1) / 2;

      // ---- the end of the run
      const Place me = place();
      const int x = me.x;
      if (alive && units > 0) alive = warp_wait(&sh.o_done[t], runs++ & 1);
      if (units > 0) tc_fence_after();
      float fade = 1.f, fade_other = 0.f;  // what this thread's O is scaled by where the groups share a tile, and the other's
      if (!dual) {
        sh.m1[t][x] = m;
        sh.l1[t][x] = l;
      }
      if (bar_any(1, SOFTMAX_THREADS, !alive)) {
        alive = false;
        break;
      }
      if (!dual) {  // the same bits of m and l in both groups
        const float m0 = sh.m1[0][x], m1 = sh.m1[1][x];
        m = fmaxf(m0, m1);
        const float mb = m == -INFINITY ? 0.f : m, fade0 = ex2((m0 - mb) * to_log2), fade1 = ex2((m1 - mb) * to_log2);
        l = sh.l1[0][x] * fade0 + sh.l1[1][x] * fade1;
        fade = t ? fade1 : fade0;
        fade_other = t ? fade0 : fade1;
      }
      const bool direct = sg.parts == 1;
      const bool writes = (dual || t == 0) && valid;
      const int slot_id = sg.part == 0 ? 2 * cta + 1 : 2 * cta;
      const int part_row = (dual ? t * TILE : 0) + x;
      uint8_t* const tile = smem + (dual && t ? S::Q1 : S::Q0);
      const bool none = my_row().hi <= 0;  // sees no key: zeros (l is 0 too where every key's score is -inf, which gives 0 / 0)
      const float inv = rcp(l);
      // Where both groups have an O of one tile, each hands the other half of its columns (in the queries' place, which the
      // products are done with) and adds up the other half: columns [from, to) are this thread's.
      const bool two = !dual && sg.u1 - sg.u0 > 1;
      const int from = two ? t * (D / 2) : 0, to = two ? from + D / 2 : dual || t == 0 ? D : 0;
      // 32 columns of this thread's row, scaled, into the tile's own queries' place, which the products are done with.
      auto stage = [&](const float (&f)[32], int col, float scale, bool zero) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t b[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            b[e] = zero ? 0u : pack_bf16x2(f[8 * j + 2 * e] * scale, f[8 * j + 2 * e + 1] * scale);
          const uint32_t ch = col / 8 + j;
          *reinterpret_cast<uint4*>(tile + (ch >> 3) * (TILE * 128) + x * 128 + (((ch ^ x) & 7) << 4)) =
              make_uint4(b[0], b[1], b[2], b[3]);
        }
      };
      // 32 columns at a time, in loops that are not unrolled: this runs once a run, and its instructions come from afar
      if (two) {
        float* const give = reinterpret_cast<float*>(smem + (t ? S::Q1 : S::Q0)) + x;
        const float* const taken = reinterpret_cast<const float*>(smem + (t ? S::Q0 : S::Q1)) + x;
#pragma unroll 1
        for (int col = 0; warp_valid && col < D / 2; col += 32) {
          float f[32];
          tmem_ld32(o_addr + (D / 2 - from) + col, f);
#pragma unroll
          for (int j = 0; j < 32; ++j) give[(col + j) * TILE] = f[j];
        }
        bar_sync(2, SOFTMAX_THREADS);
#pragma unroll 1
        for (int col = 0; warp_valid && col < D / 2; col += 32) {
          float f[32];
          uint32_t b[32];
          tmem_ld32(o_addr + from + col, f);
#pragma unroll
          for (int j = 0; j < 32; ++j) b[j] = __float_as_uint(f[j] * fade + taken[(col + j) * TILE] * fade_other);
          st16(o_addr + from + col, b);
          st16(o_addr + from + col + 16, b + 16);
          tmem_st_wait();
        }
        if (direct) bar_sync(2, SOFTMAX_THREADS);  // the outputs go where the other group read
      }
#pragma unroll 1
      for (int col = from; col < to; col += 32) {
        float f[32];
        if (warp_valid) tmem_ld32(o_addr + col, f);
        if (!valid) continue;
        if (direct) {
          stage(f, col, inv, none);
        } else {
          float4* const o = part_o<D>(a, slot_id) + (col / 4) * (2 * TILE) + part_row;
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j * (2 * TILE)] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
        }
      }
      tc_fence_before();
      bool whole = direct;  // the rows' outputs are in shared memory
      if (!direct) {
        if (writes) part_ml<D>(a, slot_id)[part_row] = make_float2(m, l);
        __threadfence();
        bar_sync(1, SOFTMAX_THREADS);
        if (tid == 0) {
          const unsigned done = atomicAdd(&a.counters[sg.cta0], 1u);
          sh.last_part = done + 1 == (unsigned)sg.parts;
          if (sh.last_part) a.counters[sg.cta0] = 0;
          __threadfence();
        }
        bar_sync(2, SOFTMAX_THREADS);
        // The last to arrive joins the parts, in their order: many rows a thread each, few rows over all threads.
        auto slot_of = [&](int q) { return q == 0 ? 2 * sg.cta0 + 1 : 2 * (sg.cta0 + q); };
        auto joined_ml = [&](int r) {  // a row's maximum and sum
          float mm = -INFINITY, ll = 0.f;
#pragma unroll 1
          for (int q = 0; q < sg.parts; q += 8) {
            float2 z[8];
            float top = mm;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              z[i] = q + i < sg.parts ? __ldcg(part_ml<D>(a, slot_of(q + i)) + r) : make_float2(-INFINITY, 0.f);
              top = fmaxf(top, z[i].x);
            }
            const float mb = top == -INFINITY ? 0.f : top;
            ll *= ex2((mm - mb) * to_log2);
#pragma unroll
            for (int i = 0; i < 8; ++i) ll = fmaf(z[i].y, ex2((z[i].x - mb) * to_log2), ll);
            mm = top;
          }
          return make_float2(mm, ll);
        };
        if (sh.last_part) __threadfence();
        if (sh.last_part && (dual || sg.ntok * g > TILE / 2)) {  // half the columns a group where they share a tile
          whole = true;
          if (valid) {
            const float2 z = joined_ml(part_row);
            m = z.x;
            l = z.y;
            const float mb = m == -INFINITY ? 0.f : m, scale = rcp(l);
            const int join_to = dual ? D : (t + 1) * (D / 2);
#pragma unroll 1
            for (int col = dual ? 0 : t * (D / 2); col < join_to; col += 32) {
              float f[32];
#pragma unroll
              for (int j = 0; j < 32; ++j) f[j] = 0.f;
#pragma unroll 1
              for (int q = 0; q < sg.parts; q += 2) {  // two parts at a time: mostly there are no more
                float4 v[2][8];
                float w[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const bool on = q + i < sg.parts;
                  const int sid = slot_of(on ? q + i : q);
                  const float4* const o = part_o<D>(a, sid) + (col / 4) * (2 * TILE) + part_row;
#pragma unroll
                  for (int j = 0; j < 8; ++j) v[i][j] = on ? __ldcg(o + j * (2 * TILE)) : make_float4(0.f, 0.f, 0.f, 0.f);
                  w[i] = ex2((__ldcg(&part_ml<D>(a, sid)[part_row].x) - mb) * to_log2);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                  for (int j = 0; j < 8; ++j) {
                    f[4 * j] = fmaf(v[i][j].x, w[i], f[4 * j]);
                    f[4 * j + 1] = fmaf(v[i][j].y, w[i], f[4 * j + 1]);
                    f[4 * j + 2] = fmaf(v[i][j].z, w[i], f[4 * j + 2]);
                    f[4 * j + 3] = fmaf(v[i][j].w, w[i], f[4 * j + 3]);
                  }
              }
              stage(f, col, scale, none);
            }
          }
        } else if (sh.last_part) {
          // Four columns of a row a thread, `pad` rows a group of columns, so that neighbours read neighbours; a thread finds
          // its row's maximum and sum itself, from the same trip to memory as the columns.
          const int rows = sg.ntok * g, pad = (rows + 7) & ~7;  // of one tile
#pragma unroll 1
          for (int i0 = tid; i0 < pad * (D / 4); i0 += SOFTMAX_THREADS) {
            const int group = i0 / pad, row2 = i0 - group * pad;
            if (row2 >= rows) continue;
            const int at = group * (2 * TILE) + row2;
            float mm = -INFINITY, ll = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int q = 0; q < sg.parts; q += 8) {
              float2 z[8];
              float4 v[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const bool on = q + i < sg.parts;
                const int sid = slot_of(on ? q + i : q);
                z[i] = on ? __ldcg(part_ml<D>(a, sid) + row2) : make_float2(-INFINITY, 0.f);
                v[i] = on ? __ldcg(part_o<D>(a, sid) + at) : make_float4(0.f, 0.f, 0.f, 0.f);
              }
              float top = mm;
#pragma unroll
              for (int i = 0; i < 8; ++i) top = fmaxf(top, z[i].x);
              const float mb = top == -INFINITY ? 0.f : top, f = ex2((mm - mb) * to_log2);
              ll *= f;
              acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float w = ex2((z[i].x - mb) * to_log2);
                ll = fmaf(z[i].y, w, ll);
                acc.x = fmaf(v[i].x, w, acc.x);
                acc.y = fmaf(v[i].y, w, acc.y);
                acc.z = fmaf(v[i].z, w, acc.z);
                acc.w = fmaf(v[i].w, w, acc.w);
              }
              mm = top;
            }
            const float iv = rcp(ll);
            const int64_t row0 = (int64_t)sg.row0 + div_g(row2);
            const int h = sg.head * g + (row2 - div_g(row2) * g);
            uint16_t* const dst = static_cast<uint16_t*>(p.out) + row0 * p.out_b_stride + (int64_t)h * p.out_h_stride + group * 4;
            const bool none2 = sg.pos0 + div_g(row2) < 0;
            const uint32_t b0 = none2 ? 0u : pack_bf16x2(acc.x * iv, acc.y * iv);
            const uint32_t b1 = none2 ? 0u : pack_bf16x2(acc.z * iv, acc.w * iv);
            if (a.out_wide) {
              *reinterpret_cast<uint2*>(dst) = make_uint2(b0, b1);
            } else {
              dst[0] = (uint16_t)b0;
              dst[1] = (uint16_t)(b0 >> 16);
              dst[2] = (uint16_t)b1;
              dst[3] = (uint16_t)(b1 >> 16);
            }
            if (group == 0 && p.lse != nullptr) p.lse[row0 * p.num_q_heads + h] = mm * to_ln + ln(ll);
          }
        }
      }
      if (whole && !dual) bar_sync(1, SOFTMAX_THREADS);
      if (whole && (dual || t == 0)) {
        if (t == 0)
          bar_sync(3, TILE);
        else
          bar_sync(4, TILE);
        const int tile0 = dual ? t * tpt : 0, rows = min(sg.ntok - tile0, tpt) * g;
        uint16_t* const og = static_cast<uint16_t*>(p.out) + (int64_t)(sg.row0 + tile0) * p.out_b_stride +
                             (int64_t)(sg.head * g) * p.out_h_stride + me.ch * 8;
#pragma unroll 1
        for (int k0 = 0; k0 < ROUNDS; k0 += 4) {
          if (me.row + k0 * ROWS_A_ROUND >= rows) break;
          uint4 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = *reinterpret_cast<const uint4*>(tile + me.at + (k0 + k) * (ROWS_A_ROUND * 128));
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = me.row + (k0 + k) * ROWS_A_ROUND;
            if (r >= rows) continue;
            uint16_t* const dst = og + row_offset(r, p.out_b_stride, p.out_h_stride);
            if (a.out_wide) {
              *reinterpret_cast<uint4*>(dst) = v[k];
            } else {
              const uint32_t e[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                dst[2 * j] = (uint16_t)e[j];
                dst[2 * j + 1] = (uint16_t)(e[j] >> 16);
              }
            }
          }
        }
      }
      if (whole && writes && p.lse != nullptr)
        p.lse[((int64_t)sg.row0 + (dual ? t * tpt : 0) + div_g(x)) * p.num_q_heads + sg.head * g + (x - div_g(x) * g)] =
            m * to_ln + ln(l);  // no key, or scores of -inf alone: -inf; a score of +inf or NaN: NaN
      if (t == 0)
        bar_sync(3, TILE);
      else
        bar_sync(4, TILE);
      if (x == 0) mbar_arrive(&sh.seg_empty[slot]);
    }
    if (!alive && lane == 0 && p.error_word) atomicOr(p.error_word, KDA_ERR_TIMEOUT);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == PRODUCT_WARP) tmem_dealloc(tmem, 512);
}

size_t paged_attention_parts_bytes(int head_dim, int ctas) {
  return (size_t)ctas * 2 * (2 * TILE) * (head_dim + 2) * sizeof(float);
}

bool paged_attention_on_tensor_cores(const kda_paged_cache& c, bool fp8) {
  const int elems = fp8 ? 16 : 8;  // of 16 bytes
  auto rows16 = [&](const kda_pages& g) {
    return (reinterpret_cast<uintptr_t>(g.ptr) & 15) == 0 && g.page_stride % elems == 0 && g.token_stride % elems == 0 &&
           g.head_stride % elems == 0;
  };
  return (c.head_dim == 64 || c.head_dim == 128) && c.num_pages > 0 && c.page_size >= 16 &&
         (c.page_size & (c.page_size - 1)) == 0 && rows16(c.k) && rows16(c.v);
}

template <int D, bool FP8>
static cudaError_t launch_tc(const CUtensorMap& km, const CUtensorMap& vm, const AttnArgs& a, int ctas, cudaStream_t s) {
  constexpr size_t bytes = Shape<D, FP8>::END + sizeof(Shared<D, FP8>);
  static_assert(bytes <= 232448, "shared memory of one CTA");
  static DeviceFlags done;
  const cudaError_t e = set_smem_limit_once(kda_paged_attention_tc_kernel<D, FP8>, bytes, done);
  if (e != cudaSuccess) return e;
  return launch_early(kda_paged_attention_tc_kernel<D, FP8>, dim3((unsigned)ctas), Shape<D, FP8>::THREADS, bytes, s, km, vm, a);
}

cudaError_t launch_paged_attention_tc(const kda_attention_params& p, const kda_paged_scales* scales, void* workspace,
                                      int ctas, cudaStream_t s) {
  if ((p.q.b_stride | p.q.h_stride | p.out_b_stride | p.out_h_stride) >> 31) return cudaErrorNotSupported;
  // the line of units is counted in 32 bits: at most so many items of so many units a key-value head (for ranges that
  // share no rows; the kernel turns away others that hold more than num_tokens)
  if (p.num_tokens > 0x7fffffff - 2 * TILE) return cudaErrorNotSupported;
  const long long tokens = 2 * (TILE / (p.num_q_heads / p.cache.num_heads));
  long long keys = (long long)p.table_width * p.cache.page_size;
  if (p.window > 0 && p.window + tokens < keys) keys = p.window + tokens;
  const long long items = p.num_tokens / tokens + p.num_requests;
  if (items * (keys / UNIT + 2 + (scales ? LEAD8 : LEAD)) > 0x7fffffffLL / p.cache.num_heads) return cudaErrorNotSupported;
  AttnArgs a;
  a.p = p;
  a.sc = scales ? *scales : kda_paged_scales{};
  a.counters = static_cast<unsigned*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + KDA_ATTENTION_WORKSPACE_ZEROED);
  auto rows16 = [](const void* x, int64_t b, int64_t h) {
    return (reinterpret_cast<uintptr_t>(x) & 15) == 0 && b % 8 == 0 && h % 8 == 0;
  };
  a.q_wide = rows16(p.q.ptr, p.q.b_stride, p.q.h_stride);
  a.out_wide = rows16(p.out, p.out_b_stride, p.out_h_stride);
  a.box = p.cache.page_size < UNIT ? p.cache.page_size : UNIT;
  a.group = p.num_q_heads / p.cache.num_heads;
  a.tile_tokens = TILE / a.group;
  a.inv_group = 65536u / (unsigned)a.group + 1u;  // for row < 128 and group <= 128 the excess is below 128 / 2^16 < 1 / group
  CUtensorMap km, vm;
  const bool wide = p.cache.head_dim == 128;
  if (scales != nullptr) {
    const int rows = paged_attention_few_rows(p);
    cudaError_t e = rows > 0 ? launch_paged_attention_fp8_rows(p, *scales, rows, workspace, ctas, s) : cudaErrorNotSupported;
    if (e != cudaErrorNotSupported) return e;  // else too many items of few rows for its line; of this kernel's there are fewer
    e = code_pages_tensor_map(p.cache.k, p.cache, a.box, &km);
    if (e == cudaSuccess) e = code_pages_tensor_map(p.cache.v, p.cache, a.box, &vm);
    if (e != cudaSuccess) return e;
    return wide ? launch_tc<128, true>(km, vm, a, ctas, s) : launch_tc<64, true>(km, vm, a, ctas, s);
  }
  cudaError_t e = pages_tensor_map(p.cache.k, p.cache, a.box, &km);
  if (e == cudaSuccess) e = pages_tensor_map(p.cache.v, p.cache, a.box, &vm);
  if (e != cudaSuccess) return e;
  return wide ? launch_tc<128, false>(km, vm, a, ctas, s) : launch_tc<64, false>(km, vm, a, ctas, s);
}

}  // namespace kda
