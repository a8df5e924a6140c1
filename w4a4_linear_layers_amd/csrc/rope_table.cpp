// serq_rope_table: the host-side table of the rotary position embedding.

#include <cmath>

#include "serq.h"

extern "C" int serq_rope_table(int rot_dim, int max_pos, double theta, serq_rope_scaling scaling, double factor,
                               int orig_len, double low, double high, double mscale, float* table) {
  if (!table || rot_dim < 2 || rot_dim > 65536 || (rot_dim % 2) != 0 || max_pos < 1) return SERQ_EINVAL;
  if (!(theta > 0.0) || !std::isfinite(theta) || !std::isfinite(mscale)) return SERQ_EINVAL;
  if (scaling < SERQ_ROPE_PLAIN || scaling > SERQ_ROPE_BANDS) return SERQ_EINVAL;
  if (scaling != SERQ_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return SERQ_EINVAL;
  if (scaling == SERQ_ROPE_BASE && rot_dim == 2) return SERQ_EINVAL;
  if (scaling == SERQ_ROPE_BANDS &&
      (orig_len < 1 || !std::isfinite(low) || !std::isfinite(high) || !(low < high)))
    return SERQ_EINVAL;
  const int half = rot_dim / 2;
  const double two_pi = 6.283185307179586;
  if (scaling == SERQ_ROPE_BASE) theta *= std::pow(factor, rot_dim / (rot_dim - 2.0));
  for (int i = 0; i < half; ++i) {
    double f = std::pow(theta, -2.0 * i / rot_dim);
    if (scaling == SERQ_ROPE_LINEAR) f /= factor;
    if (scaling == SERQ_ROPE_BANDS) {
      const double turns = orig_len * f / two_pi;
      const double g = std::fmin(std::fmax((turns - low) / (high - low), 0.0), 1.0);
      f = (1.0 - g) * f / factor + g * f;
    }
    for (int p = 0; p < max_pos; ++p) {
      float* row = table + static_cast<size_t>(p) * rot_dim;
      row[i] = static_cast<float>(mscale * std::cos(p * f));
      row[half + i] = static_cast<float>(mscale * std::sin(p * f));
    }
  }
  return SERQ_OK;
}
