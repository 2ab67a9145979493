// visible.cuh -- the positions a row sees through a sliding window with sinks.
#pragma once

#include "partial_kernel.cuh"

namespace gqa {

// A row of length L sees [0, ns) and [w0, L), ns <= w0: the sinks that lie before the window, and
// the window.  Without a window w0 is 0.  Entry i of the list is position i < ns ? i : i - ns + w0.
struct Visible {
  int L, w0, ns, n;  // n = ns + L - w0 entries
  __host__ __device__ Visible(int len, int window, int n_sink) : L(len) {
    w0 = window > 0 && window < len ? len - window : 0;
    ns = n_sink < w0 ? n_sink : w0;
    n = ns + L - w0;
  }
  __host__ __device__ int pos(int i) const { return i < ns ? i : i - ns + w0; }
};

struct VisibleParams {
  PartialParams base;  // kc, vc, ksc, vsc hold the cache's pointers whatever its kind
  int window, n_sink;
  float k_scale, v_scale;  // 4-bit caches
};

}  // namespace gqa
