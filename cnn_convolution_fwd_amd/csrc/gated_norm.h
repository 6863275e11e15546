// Norms before and after a block, fused with its gate and residual scale
// (k_gated_norm.hip), behind cfwd_gated_norm of cfwd.h.
#pragma once

#include "internal.h"

namespace cfwd {

struct GatedNormArgs {
    const void *b, *residual, *gate;
    const float *post_weight, *post_bias, *pre_weight, *pre_bias;
    void *s, *h, *h_scales;
};

// Arguments checked by the caller.
cfwd_status gated_norm(const cfwd_gated_norm_desc* d, const GatedNormArgs& a, hipStream_t st);

}  // namespace cfwd
