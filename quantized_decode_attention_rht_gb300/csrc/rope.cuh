// Rotary positions: the angle of a pair, and the parameters of the kernels that turn heads.
//
// Pair j of a head at position p is turned by theta = p w_j.  What the turn needs is theta
// modulo a full turn, and in float32 the product p w_j has lost it long before today's
// context lengths (half an ulp of 2^20 radians is 0.06).  So a pair's frequency is stored as
// the fraction of a turn per token in 64-bit fixed point, t_j = floor(2^64 w_j / 2 pi) mod
// 2^64, and the position multiplies it modulo 2^64: the reduction is exact, for negative
// positions too, and only the stored frequency's own rounding (2^-53 relative, it comes from
// a double, and 2^-64 of a turn) grows with p.  The 64 bits, as a signed number, are the angle in
// [-1/2, 1/2) turns.  (The top 32 alone would do for the cosine, but a slow pair's angle at a
// small position, 2^-22 turns, would keep ten bits of its sine.)
#pragma once
#include "kvq_internal.cuh"

namespace kvq {

struct RopeParams {
  const unsigned long long* turns;  // [rot / 2]
  const int32_t* positions;         // [num_tokens]
  float scale;
  int rot, layout, neg;  // neg: the transpose (angles change sign)
};

// Angle in half turns, in [-1, 1), of a pair at a position: rounded once, to 2^-24 of itself.
__device__ __forceinline__ float rope_half_turns(unsigned long long turns, int position) {
  const unsigned long long phase = turns * (unsigned long long)(long long)position;
  return (float)(long long)phase * 1.0842021724855044e-19f;  // 2^-63
}

// (cos, sin) times the scale.  sincospif: within 1 ulp, so the float32 coefficients carry
// about 2e-7, far below the fp16 the heads are stored in.
__device__ __forceinline__ float2 rope_cos_sin(const RopeParams& r, int pair, int position) {
  float s, c;
  sincospif(rope_half_turns(__ldg(r.turns + pair), position), &s, &c);
  return make_float2(c * r.scale, (r.neg ? -s : s) * r.scale);
}

// Host side, shared by kvq_rope_apply and kvq_rope_append (rope.cu).
cudaError_t launch_rope(const RopeParams& rope, const kvq_heads* a, const kvq_heads* b, int tokens, int dim, int sms,
                        cudaStream_t stream);
kvq_status check_rope(const kvq_rope* rope, int head_dim);
kvq_status check_heads(const kvq_heads* h, int tokens, int dim, bool need_out);
RopeParams rope_params(const kvq_rope* rope, const int32_t* positions, int neg);

}  // namespace kvq
