// topk.cuh — the router's top-k of one token, by one warp (shared by the row map of route.cu and
// the slot plan of w4a16.cu).
#pragma once

#include <limits.h>
#include <math.h>
#include <stdint.h>

namespace nvfp4 {
namespace {

constexpr int kMaxE = 256;
constexpr int kMaxK = 32;
constexpr int kPerLane = kMaxE / 32;

// Top-k of token t by one warp.  Lane l holds experts l, l+32, ..., and lane j < k ends up
// holding the j-th selected expert.
__device__ __forceinline__ void topk_token(const float* __restrict__ logits, int t, int E, int k,
                                           int renorm, int lane, int32_t* ids, float* w) {
  float v[kPerLane];
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = lane + 32 * i;
    v[i] = e < E ? __ldg(logits + (int64_t)t * E + e) : -INFINITY;
    if (e < E) m = fmaxf(m, v[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));

  // Ordered keys: a larger float has a larger key, -0 and +0 the same one, a NaN none (0: it is
  // never selected).  A round is two warp reductions: the largest key, then the lowest expert that
  // has it.
  uint32_t key[kPerLane];
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const uint32_t b = __float_as_uint(v[i] + 0.0f);
    key[i] = lane + 32 * i < E && v[i] == v[i] ? ((b >> 31) ? ~b : b | 0x80000000u) : 0u;
  }
  int my_id = -1;
  float my_v = -INFINITY;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) best = max(best, key[i]);
    best = __reduce_max_sync(0xffffffffu, best);
    int be = INT_MAX;
    if (best != 0) {
#pragma unroll
      for (int i = kPerLane - 1; i >= 0; --i)
        if (key[i] == best) be = lane + 32 * i;
      be = static_cast<int>(__reduce_min_sync(0xffffffffu, static_cast<uint32_t>(be)));
#pragma unroll
      for (int i = 0; i < kPerLane; ++i)
        if (lane + 32 * i == be) key[i] = 0;
    }
    if (lane == j) {
      my_id = be;
      my_v = best == 0 ? -INFINITY
                       : __uint_as_float((best >> 31) ? best ^ 0x80000000u : ~best);
    }
  }
  const bool live = lane < k && my_id != INT_MAX && my_v > -INFINITY && m > -INFINITY;
  const float ex = live ? expf(my_v - m) : 0.0f;
  float denom = 0.0f;
  if (renorm) {
    denom = ex;
  } else {
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (lane + 32 * i < E && v[i] > -INFINITY && m > -INFINITY) denom += expf(v[i] - m);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) denom += __shfl_xor_sync(0xffffffffu, denom, o);
  if (lane < k) {
    ids[(int64_t)t * k + lane] = live ? my_id : -1;
    w[(int64_t)t * k + lane] = live ? ex / denom : 0.0f;
  }
}

}  // namespace
}  // namespace nvfp4
