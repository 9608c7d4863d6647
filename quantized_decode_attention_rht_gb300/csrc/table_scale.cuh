// The scale under which a codebook's centroids are rounded to fp16, as the tensor-core kernels multiply them.
#pragma once
#include "kvq_internal.cuh"

namespace kvq {
namespace {

// The scale of a codebook's table, out of 512 steps of 2^(1 / 512) that bring its largest magnitude
// to 2^-3 .. 2^-1: the one whose fp16 roundings r of the scaled centroids x are nearest, up to a common
// factor: least sum w (a r - x)^2 / scale^2 with a = 1 - slope, slope = sum w r (r - x) / sum w r^2.  (In those
// terms nothing cancels: the sum is sum w (r - x)^2 - slope sum w r (r - x).)  What a rounding does to a key
// adds up where its coordinates have one magnitude, and those of a key with an outlier channel all are
// near their root mean square.  So the centroids there weigh most: w = exp(-3.125 (|c| / c1 - 1)^2), c1 = the
// largest over 1.51, 2.15 or 2.73, what 2, 3 or 4 bits of N(0, 1) reach to.  (4-bit keys with x30 outlier
// channels: 1.3e-4 of the output instead of 2.9e-4 with equal weights and 128 steps.)  c: centroid `lane` in every
// lane (0 beyond the codebook); the candidates of thread `tid` of 512 / kEach: the best one's error, slope and number.
constexpr int kTableSteps = 512;
// 2^-3 over the largest magnitude's power of two (its bits given)
__device__ __forceinline__ float table_unit(uint32_t most) {
  return __uint_as_float((251u - min(max(most >> 23, 2u), 249u)) << 23);
}
template <int kEach = 4>
__device__ __forceinline__ void table_candidates(float c, int bits, int tid, float& least, float& slope, int& at) {
  constexpr int kSteps = kTableSteps, kThreads = kSteps / kEach;
  const int lane = tid & 31;
  const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(c)));
  const float over = (bits == 4 ? 2.73f : (bits == 3 ? 2.15f : 1.51f)) / __uint_as_float(max(most, 0x00800000u));
  const float away = fabsf(c) * over - 1.0f;
  const float weight = lane < (1 << bits) ? exp2f(-4.508f * away * away) : 0.f;  // 3.125 log2 e
  const float unit = table_unit(most);
  float mine[kEach], dd[kEach], rd[kEach], rr[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    mine[k] = exp2f((float)(k * kThreads + tid) * (1.0f / kSteps));
    dd[k] = rd[k] = rr[k] = 0.f;
  }
#pragma unroll 2
  for (int i = 0; i < (1 << bits); ++i) {
    const float ci = __shfl_sync(0xFFFFFFFFu, c, i) * unit, w = __shfl_sync(0xFFFFFFFFu, weight, i);
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const float x = ci * mine[k], r = __half2float(__float2half_rn(x)), d = r - x, wd = w * d;
      dd[k] = fmaf(wd, d, dd[k]);
      rd[k] = fmaf(wd, r, rd[k]);
      rr[k] = fmaf(w * r, r, rr[k]);
    }
  }
  least = INFINITY;
  slope = 0.f;
  at = tid;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const float a = rr[k] > 0.f ? __fdividef(rd[k], rr[k]) : 0.f;
    const float e = __fdividef(fmaf(-a, rd[k], dd[k]), mine[k] * mine[k]);
    if (e < least) {
      least = e;
      slope = a;
      at = k * kThreads + tid;
    }
  }
}

}  // namespace
}  // namespace kvq
