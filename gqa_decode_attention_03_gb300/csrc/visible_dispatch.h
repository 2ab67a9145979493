// visible_dispatch.h -- the launchers of the calls with a visible set.
#pragma once

#include "visible.cuh"

namespace gqa {

cudaError_t launch_q4(int head_dim, const Q4Params& qp, dim3 grid, cudaStream_t s);
cudaError_t launch_f16_window(int head_dim, const CUtensorMap& tk, const CUtensorMap& tv,
                              const PartialParams& p, dim3 grid, cudaStream_t s);
// rows that share a sequence: head_dim 64 or 128, grid (chunks, KV heads, groups of 128 / G rows)
cudaError_t launch_window_rows(int head_dim, const CUtensorMap& tk, const CUtensorMap& tv,
                               const Q4Params& qp, dim3 grid, cudaStream_t s);
cudaError_t launch_q4_rows(int head_dim, const Q4Params& qp, dim3 grid, cudaStream_t s);

}  // namespace gqa
