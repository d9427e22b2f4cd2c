// The rotation's table, computed in double precision on the host: far positions lose their angle
// in 32 bits (at position 10^5 an fp32 angle is off by up to 4e-3).
#include <cmath>

#include "host_common.h"

extern "C" int rc_rope_table(const double* inv_freq, int32_t num_pairs, int64_t first_position,
                             int64_t num_positions, double scale, float* out) {
  RC_CHECK_ARG(num_pairs > 0 && num_pairs % 8 == 0 && num_pairs <= 128 && first_position >= 0 &&
                   num_positions >= 0,
               "rc_rope_table: bad sizes");
  RC_CHECK_ARG(inv_freq && (out || num_positions == 0), "rc_rope_table: NULL pointer");
  RC_CHECK_ARG(std::isfinite(scale), "rc_rope_table: scale is not finite");
  for (int32_t i = 0; i < num_pairs; ++i)
    RC_CHECK_ARG(std::isfinite(inv_freq[i]), "rc_rope_table: inv_freq[%d] is not finite", i);
  for (int64_t p = 0; p < num_positions; ++p) {
    float* row = out + p * 2 * num_pairs;
    const double pos = (double)(first_position + p);
    for (int32_t i = 0; i < num_pairs; ++i) {
      row[i] = (float)(scale * std::cos(pos * inv_freq[i]));
      row[num_pairs + i] = (float)(scale * std::sin(pos * inv_freq[i]));
    }
  }
  return RC_OK;
}
