// visible_simple.cu -- decode attention over a row's visible positions, one CTA per (row, head).
//
// The formula as it stands: four warps take every fourth visible position, a lane holds D/32 dims
// of q and of the accumulator, the running maximum and sum are kept per warp in fp32 and the four
// states meet in shared memory.
#include "dispatch.h"
#include "visible.cuh"
#include "visible_dispatch.h"

namespace gqa {

constexpr int kSimpleWarps = 4;

template <int D>
__device__ __forceinline__ void simple_row(const PartialParams& p, const void* cache, int s, int g,
                                           int pos, int lane, float (&f)[D / 32]) {
  const __half* c = static_cast<const __half*>(cache) +
                    (((size_t)s * p.cache_cap + pos) * p.n_kv_heads + g) * D;
#pragma unroll
  for (int k = 0; k < D / 32; ++k) f[k] = __half2float(c[lane * (D / 32) + k]);
}

template <int D>
__global__ void __launch_bounds__(32 * kSimpleWarps) visible_simple_kernel(const VisibleParams vp) {
  constexpr int DPL = D / 32;
  const PartialParams& p = vp.base;
  __shared__ float mg[kSimpleWarps][D + 2];
  const int h = blockIdx.x, t = blockIdx.y, g = h / p.group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int s = 0;
  const int L = visible_row(p, t, h == 0 && threadIdx.x == 0, s);
  const Visible vis(L, vp.window, vp.n_sink);
  float q[DPL], o[DPL], f[DPL];
#pragma unroll
  for (int k = 0; k < DPL; ++k) {
    q[k] = p.q[((size_t)t * p.n_heads + h) * D + lane * DPL + k] * p.scale_log2;
    o[k] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int i = warp; i < vis.ns + L - vis.w0; i += kSimpleWarps) {
    const int pos = i < vis.ns ? i : i - vis.ns + vis.w0;
    simple_row<D>(p, p.kc, s, g, pos, lane, f);
    float x = 0.f;
#pragma unroll
    for (int k = 0; k < DPL; ++k) x = fmaf(q[k], f[k], x);
    x = warp_sum(x);
    const float mn = fmaxf(m, x);
    const float corr = m == -INFINITY ? 0.f : fast_exp2(m - mn), w = fast_exp2(x - mn);
    m = mn;
    l = l * corr + w;
    simple_row<D>(p, p.vc, s, g, pos, lane, f);
#pragma unroll
    for (int k = 0; k < DPL; ++k) o[k] = fmaf(w, f[k], o[k] * corr);
  }
#pragma unroll
  for (int k = 0; k < DPL; ++k) mg[warp][lane * DPL + k] = o[k];
  if (lane == 0) {
    mg[warp][D] = m;
    mg[warp][D + 1] = l;
  }
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += 32 * kSimpleWarps) {
    float M = -INFINITY, A = 0.f, Ls = 0.f;
    for (int w = 0; w < kSimpleWarps; ++w) M = fmaxf(M, mg[w][D]);
    for (int w = 0; w < kSimpleWarps; ++w) {
      const float e = mg[w][D] == -INFINITY ? 0.f : fast_exp2(mg[w][D] - M);
      A = fmaf(mg[w][d], e, A);
      Ls = fmaf(mg[w][D + 1], e, Ls);
    }
    p.out[((size_t)t * p.n_heads + h) * D + d] = gated(p, t, h, d, Ls > 0.f ? A / Ls : 0.f);
  }
}

cudaError_t launch_f16_window(int head_dim, const VisibleParams& vp, const gqa_plan&,
                              cudaStream_t s) {
  const dim3 grid(vp.base.n_heads, vp.base.n_tok);
  if (head_dim == 64)
    visible_simple_kernel<64><<<grid, 32 * kSimpleWarps, 0, s>>>(vp);
  else if (head_dim == 128)
    visible_simple_kernel<128><<<grid, 32 * kSimpleWarps, 0, s>>>(vp);
  else
    visible_simple_kernel<256><<<grid, 32 * kSimpleWarps, 0, s>>>(vp);
  return cudaGetLastError();
}

}  // namespace gqa
