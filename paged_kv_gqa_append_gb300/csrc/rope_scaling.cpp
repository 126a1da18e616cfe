// Rotary frequencies of any rotary dimension and the usual scalings for
// contexts longer than the trained one, and their tables (host set-up).
//
// Compiled with -ffp-contract=off, as host.cpp: the arithmetic rounds exactly
// as written on every host.
#include <math.h>
#include <stddef.h>

#include "pkv.h"

extern "C" int pkv_rope_inv_freq_scaled(double* inv_freq, int pairs, double theta, int scaling,
                                        double factor, int original_max_pos, double beta_fast,
                                        double beta_slow, double* attention_factor) {
  if (!inv_freq || !attention_factor || pairs < 1 || pairs > PKV_ROPE_PAIRS || !(theta > 1.0) ||
      !isfinite(theta))
    return PKV_ERR_INVALID_ARGUMENT;
  if (scaling != PKV_ROPE_SCALING_NONE && (!(factor >= 1.0) || !isfinite(factor)))
    return PKV_ERR_INVALID_ARGUMENT;
  const double dim = 2.0 * (double)pairs;
  double base = theta, low = 0.0, width = 0.0;
  *attention_factor = 1.0;
  switch (scaling) {
    case PKV_ROPE_SCALING_NONE:
    case PKV_ROPE_SCALING_LINEAR:
      break;
    case PKV_ROPE_SCALING_NTK:
      if (pairs < 2) return PKV_ERR_INVALID_ARGUMENT;  // the exponent dim / (dim - 2)
      base = theta * pow(factor, dim / (dim - 2.0));
      break;
    case PKV_ROPE_SCALING_YARN: {
      if (original_max_pos < 1 || !(beta_fast > beta_slow) || !(beta_slow > 0.0) || !isfinite(beta_fast))
        return PKV_ERR_INVALID_ARGUMENT;
      // the pair index whose wave turns `beta` times over the original context
      const double two_pi = 6.283185307179586;
      const double fast = (double)pairs * log((double)original_max_pos / (beta_fast * two_pi)) / log(theta);
      const double slow = (double)pairs * log((double)original_max_pos / (beta_slow * two_pi)) / log(theta);
      low = fmax(0.0, floor(fast));
      const double high = fmin(dim - 1.0, ceil(slow));
      width = fmax(high - low, 0.001);
      *attention_factor = 0.1 * log(factor) + 1.0;
      break;
    }
    default:
      return PKV_ERR_INVALID_ARGUMENT;
  }
  for (int i = 0; i < pairs; ++i) {
    const double f = pow(base, -(2.0 * (double)i) / dim);
    if (scaling == PKV_ROPE_SCALING_LINEAR) {
      inv_freq[i] = f / factor;
    } else if (scaling == PKV_ROPE_SCALING_YARN) {
      // fast pairs keep their frequency, slow ones are divided, a ramp between
      const double ramp = fmin(1.0, fmax(0.0, ((double)i - low) / width));
      inv_freq[i] = f / factor * ramp + f * (1.0 - ramp);
    } else {
      inv_freq[i] = f;
    }
  }
  return PKV_OK;
}

extern "C" int pkv_rope_table_fill_scaled(float* host_cos, float* host_sin, int max_pos, int pairs,
                                          const double* inv_freq, double attention_factor) {
  if (!host_cos || !host_sin || !inv_freq || max_pos < 1 || pairs < 1 || pairs > PKV_ROPE_PAIRS ||
      !isfinite(attention_factor))
    return PKV_ERR_INVALID_ARGUMENT;
  for (int p = 0; p < max_pos; ++p) {
    for (int i = 0; i < pairs; ++i) {
      const double ang = (double)p * inv_freq[i];
      host_cos[(size_t)p * pairs + i] = (float)(cos(ang) * attention_factor);
      host_sin[(size_t)p * pairs + i] = (float)(sin(ang) * attention_factor);
    }
  }
  return PKV_OK;
}
