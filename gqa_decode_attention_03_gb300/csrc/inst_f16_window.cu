// inst_f16_window.cu -- instantiations of the f16 kernels that see a window.
#include "dispatch.h"
#include "partial_mma.cuh"
#include "visible_dispatch.h"

namespace gqa {

template <int D>
static cudaError_t launch_rows(const CUtensorMap& tk, const CUtensorMap& tv,
                               const PartialParams& p, dim3 grid, cudaStream_t s) {
  return p.group <= 8 ? launch_mma_f16<D, 1, true>(tk, tv, p, grid, s)
                      : launch_mma_f16<D, 2, true>(tk, tv, p, grid, s);
}

cudaError_t launch_f16_window(int head_dim, const CUtensorMap& tk, const CUtensorMap& tv,
                              const PartialParams& p, dim3 grid, cudaStream_t s) {
  if (head_dim == 64) return launch_rows<64>(tk, tv, p, grid, s);
  if (head_dim == 128) return launch_rows<128>(tk, tv, p, grid, s);
  return launch_rows<256>(tk, tv, p, grid, s);
}

}  // namespace gqa
