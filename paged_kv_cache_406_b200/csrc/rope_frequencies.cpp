// Rotary frequencies and their scalings for contexts longer than the ones a
// model was made for.  Host only, in 64 bits.
#include <algorithm>
#include <cmath>

#include "pkv_internal.h"

using pkv::fail;

extern "C" int pkv_rope_frequencies(int32_t rot_dim, double base, const pkv_rope_scaling_t* scaling, double* inv_freq,
                                    float* factor) {
  const char* fn = "pkv_rope_frequencies";
  if (!inv_freq || !factor) return fail(PKV_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  if (rot_dim <= 0 || rot_dim % 2 != 0) return fail(PKV_ERR_INVALID_ARG, "%s: rot_dim %d must be even and positive", fn, rot_dim);
  if (!(base > 1.0) || !std::isfinite(base)) return fail(PKV_ERR_INVALID_ARG, "%s: base must be above 1 and finite", fn);
  pkv_rope_scaling_t sc{};
  if (scaling) sc = *scaling;
  if (sc.kind != PKV_ROPE_PLAIN && (!(sc.scale >= 1.0) || !std::isfinite(sc.scale)))
    return fail(PKV_ERR_INVALID_ARG, "%s: scale must be at least 1 and finite", fn);
  const bool bands = sc.kind == PKV_ROPE_BANDS || sc.kind == PKV_ROPE_YARN;
  if (bands && (!(sc.slow > 0.0) || !(sc.fast > sc.slow) || !std::isfinite(sc.fast) || sc.original_positions <= 0))
    return fail(PKV_ERR_INVALID_ARG, "%s: need 0 < slow < fast and original_positions > 0", fn);
  const double two_pi = 6.283185307179586476925;
  double b = base;
  switch (sc.kind) {
    case PKV_ROPE_PLAIN:
    case PKV_ROPE_LINEAR:
    case PKV_ROPE_BANDS:
    case PKV_ROPE_YARN: break;
    case PKV_ROPE_BASE:
      if (rot_dim == 2) return fail(PKV_ERR_INVALID_ARG, "%s: a scaled base needs rot_dim > 2", fn);
      b = base * std::pow(sc.scale, static_cast<double>(rot_dim) / (rot_dim - 2));
      break;
    default: return fail(PKV_ERR_UNSUPPORTED, "%s: scaling kind %d", fn, sc.kind);
  }
  // the channel pair that makes `turns` turns over the original positions
  auto pair_of = [&](double turns) {
    return rot_dim * std::log(sc.original_positions / (turns * two_pi)) / (2.0 * std::log(base));
  };
  double first = 0, last = 1;
  if (sc.kind == PKV_ROPE_YARN) {
    first = std::max(std::floor(pair_of(sc.fast)), 0.0);
    last = std::min(std::ceil(pair_of(sc.slow)), rot_dim - 1.0);
    if (last <= first) last = first + 0.001;
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double f = std::pow(b, -2.0 * i / rot_dim);
    double keep = 1.0;  // share of the frequency that stays as it is
    if (sc.kind == PKV_ROPE_LINEAR) keep = 0.0;
    else if (sc.kind == PKV_ROPE_BANDS)
      keep = std::clamp((sc.original_positions * f / two_pi - sc.slow) / (sc.fast - sc.slow), 0.0, 1.0);
    else if (sc.kind == PKV_ROPE_YARN)
      keep = 1.0 - std::clamp((i - first) / (last - first), 0.0, 1.0);
    inv_freq[i] = keep == 1.0 ? f : f * keep + f / sc.scale * (1.0 - keep);
  }
  *factor = sc.kind == PKV_ROPE_YARN ? static_cast<float>(0.1 * std::log(sc.scale) + 1.0) : 1.0f;
  return pkv::ok();
}
