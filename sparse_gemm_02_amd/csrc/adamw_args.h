// Host-side checks of AdamW's hyper-parameters, shared by its C entry points.
#pragma once
#include <cmath>

#include "../../include/slope.h"
#include "launch.h"

namespace slope {

constexpr int64_t kAdamwMaxElems = int64_t(1) << 40;
constexpr int64_t kMultiMaxElems = int64_t(1) << 34;   // of a tensor, eight values a thread: below 2^32 threads

// Checks AdamW hyper-parameters and derives the per-update fp32 constants.
inline slope_status adamw_step(const slope_adamw_params* hp, AdamWStep* c) {
  if (!hp) return SLOPE_ERR_INVALID_ARG;
  if (hp->step < 1 || !(hp->beta1 >= 0.0 && hp->beta1 < 1.0) || !(hp->beta2 >= 0.0 && hp->beta2 < 1.0) ||
      !(hp->eps >= 0.0) || !std::isfinite(hp->eps) || !std::isfinite(hp->lr) || !std::isfinite(hp->weight_decay))
    return SLOPE_ERR_INVALID_ARG;
  const double t = (double)hp->step;
  const double bc1 = 1.0 - std::pow(hp->beta1, t), bc2 = 1.0 - std::pow(hp->beta2, t);
  c->decay = (float)(1.0 - hp->lr * hp->weight_decay);
  c->beta1 = (float)hp->beta1;
  c->omb1 = (float)(1.0 - hp->beta1);
  c->beta2 = (float)hp->beta2;
  c->omb2 = (float)(1.0 - hp->beta2);
  c->step_size = (float)(hp->lr / bc1);
  c->inv_sqrt_bc2 = (float)(1.0 / std::sqrt(bc2));
  c->eps = (float)hp->eps;
  return SLOPE_OK;
}

}  // namespace slope
