// kda_rope.cuh - rotary positions: what the kernels that turn rows share.
#pragma once

#include "kda_device.cuh"

namespace kda {

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

// Turns the pairs of a task that has some (c >= 0) by the row's scaled sines and cosines.
template <int VEC>
__device__ __forceinline__ void turn_task(RopeTask<VEC>& j, const float2* turn, bool interleaved) {
  if (VEC == 8 && interleaved) {
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

}  // namespace kda
