// Host table of rotary frequencies (kvq_rope_table): plain C++, no device code.
#include <cmath>
#include <cstdint>

#include "../../include/kvq.h"

extern "C" KVQ_API kvq_status kvq_rope_table(double base, int32_t rot_dim, const kvq_rope_scaling* scaling,
                                             uint64_t* turns) {
  const int kind = scaling ? scaling->kind : KVQ_ROPE_SCALE_NONE;
  const double factor = scaling ? scaling->factor : 1.0;
  if (!turns || !std::isfinite(base) || !(base > 0.0) || rot_dim < 2 || rot_dim > 256 || rot_dim % 2)
    return KVQ_ERR_INVALID_ARGUMENT;
  if (kind < KVQ_ROPE_SCALE_NONE || kind > KVQ_ROPE_SCALE_BY_PARTS) return KVQ_ERR_INVALID_ARGUMENT;
  if (kind != KVQ_ROPE_SCALE_NONE && (!std::isfinite(factor) || !(factor > 0.0))) return KVQ_ERR_INVALID_ARGUMENT;
  if (kind == KVQ_ROPE_SCALE_BY_PARTS &&
      (!std::isfinite(scaling->original_context) || !(scaling->original_context > 0.0) ||
       !(scaling->low_turns >= 0.0) || !(scaling->high_turns > scaling->low_turns) ||
       !std::isfinite(scaling->high_turns)))
    return KVQ_ERR_INVALID_ARGUMENT;
  const double two_pi = 6.283185307179586476925;
  const double r = rot_dim;
  double b = base;
  if (kind == KVQ_ROPE_SCALE_BASE && rot_dim > 2) b = base * std::pow(factor, r / (r - 2.0));
  for (int j = 0; j < rot_dim / 2; ++j) {
    double w = std::pow(b, -2.0 * j / r);
    if (kind == KVQ_ROPE_SCALE_LINEAR) w /= factor;
    if (kind == KVQ_ROPE_SCALE_BY_PARTS) {
      // turns over the original context decide how much of the frequency is kept
      const double t = scaling->original_context * w / two_pi;
      double keep = (t - scaling->low_turns) / (scaling->high_turns - scaling->low_turns);
      keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
      w *= keep + (1.0 - keep) / factor;
    }
    if (!std::isfinite(w)) return KVQ_ERR_INVALID_ARGUMENT;
    const double f = std::fmod(w / two_pi, 1.0);  // whole turns per token do not matter
    // f < 1 is a double, so 2^64 f is below 2^64 and exact above its last bits
    turns[j] = static_cast<uint64_t>(std::ldexp(f, 64));
  }
  return KVQ_OK;
}
