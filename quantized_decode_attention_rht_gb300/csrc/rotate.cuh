// The rotation of one vector by a warp, D / 32 neighbouring coordinates a lane.
#pragma once
#include "kvq_internal.cuh"

namespace kvq {
namespace {

// y = H (s * x) (unnormalised) for the lane's coordinates [lane * E, lane * E + E).
template <int E>
__device__ __forceinline__ void load_rotate(const uint16_t* src, const int8_t* sg, int lane, float (&y)[E]) {
  uint32_t xw[E / 2], sw[(E + 3) / 4];
  if constexpr (E == 2) {
    xw[0] = __ldg(reinterpret_cast<const uint32_t*>(src) + lane);
    sw[0] = __ldg(reinterpret_cast<const uint16_t*>(sg) + lane);
  } else if constexpr (E == 4) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(src) + lane);
    xw[0] = u.x;
    xw[1] = u.y;
    sw[0] = __ldg(reinterpret_cast<const uint32_t*>(sg) + lane);
  } else {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(src) + lane);
    xw[0] = u.x;
    xw[1] = u.y;
    xw[2] = u.z;
    xw[3] = u.w;
    const uint2 s2 = __ldg(reinterpret_cast<const uint2*>(sg) + lane);
    sw[0] = s2.x;
    sw[1] = s2.y;
  }
#pragma unroll
  for (int k = 0; k < E / 2; ++k) {
    // sign bytes 2k, 2k+1 (int8 +-1: bit 7 set for -1) -> fp16 sign bits 15, 31
    const uint32_t m = __byte_perm(sw[k >> 1], 0, (k & 1) ? 0x3424 : 0x1404) & 0x80008000u;
    const uint32_t xv = xw[k] ^ m;
    const __half2 h2 = *reinterpret_cast<const __half2*>(&xv);
    y[2 * k] = __low2float(h2);
    y[2 * k + 1] = __high2float(h2);
  }
#pragma unroll
  for (int hs = 1; hs < E; hs <<= 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if ((e & hs) == 0) {
        const float a = y[e], c = y[e + hs];
        y[e] = a + c;
        y[e + hs] = a - c;
      }
    }
  }
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const float sgn = (lane & m) ? -1.0f : 1.0f;  // upper lane keeps partner - own
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = fmaf(sgn, y[e], __shfl_xor_sync(0xFFFFFFFFu, y[e], m));
  }
}

// y <- H y (unnormalised), as load_rotate does it.
template <int E>
__device__ __forceinline__ void sign_free_rotate(int lane, float (&y)[E]) {
#pragma unroll
  for (int hs = 1; hs < E; hs <<= 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if ((e & hs) == 0) {
        const float a = y[e], c = y[e + hs];
        y[e] = a + c;
        y[e + hs] = a - c;
      }
    }
  }
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const float sgn = (lane & m) ? -1.0f : 1.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = fmaf(sgn, y[e], __shfl_xor_sync(0xFFFFFFFFu, y[e], m));
  }
}

}  // namespace
}  // namespace kvq
