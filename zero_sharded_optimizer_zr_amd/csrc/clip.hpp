// What captured graphs know of the gradient norm's and the clipped step's kernels.
#pragma once

#include "zr_clip.h"
#include "zr_math.hpp"

namespace zr {

// The end of a norm: what makes norm and factor of the sum.
struct NormFinish {
    double max_norm, eps, grad_scale;
    int32_t accumulate;
    zr_loss_scale *ls;
    zr_clip *clip;
};

// The kernels that take AdamWScalars, and those that take NormFinish (clip.hip).
int clip_scalar_slots(ScalarSlot *out);
int norm_finish_slots(ScalarSlot *out);

}  // namespace zr
