// visible_dispatch.h -- the launchers of the calls with a visible set.
#pragma once

#include "visible.cuh"

namespace gqa {

cudaError_t launch_q4(int head_dim, const VisibleParams& vp, const gqa_plan& plan, cudaStream_t s);
cudaError_t launch_f16_window(int head_dim, const VisibleParams& vp, const gqa_plan& plan,
                              cudaStream_t s);

}  // namespace gqa
