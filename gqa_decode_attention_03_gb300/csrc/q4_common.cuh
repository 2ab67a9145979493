// q4_common.cuh -- the 4-bit cache's number formats and its ragged batches of rows.
//
// A value is e2m1(code) * e4m3(scale) * a power of two.  e2m1 has two significant bits and e4m3
// four, so their product has six at most and lies between 2^-10 and 2688: it is exact in f16, and
// the whole value in fp32.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "partial_mma.cuh"

namespace gqa {

// e4m3 bits (sign bit clear) -> fp32, exact.  The f16 with the same fields has bias 15 in place
// of 7: it is the value times 2^-8, subnormals included.
__device__ __forceinline__ float e4m3_to_f32(uint32_t b) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>((b & 0x7fu) << 7))) * 256.f;
}

// Eight e2m1 codes (a word, low nibble first) -> their values as four f16x2.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// e4m3 bytes in bits 0-7 and 16-23 of x -> an f16x2 of their values.
__device__ __forceinline__ __half2 e4m3x2_to_f16x2(uint32_t x) {
  const uint32_t h = (x & 0x007f007fu) << 7;  // the values times 2^-8
  return __hmul2(*reinterpret_cast<const __half2*>(&h), __float2half2_rn(256.f));
}

__device__ __forceinline__ uint32_t mul_h2(uint32_t a, __half2 s) {
  return h2_bits(__hmul2(*reinterpret_cast<const __half2*>(&a), s));
}

// The sequence holding row r of a ragged batch: the last s with row_off[s] <= r, or -1.  All 32
// lanes of the warp take part with the same r; each round looks at 32 entries, so 1024 sequences
// take two dependent loads.
__device__ __forceinline__ int ragged_find(const int32_t* __restrict__ row_off, int n_seq, int r) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = n_seq;
  for (;;) {
    const int step = (n + 31) / 32;
    const long long i = static_cast<long long>(lane) * step;
    const bool le = i < n && __ldg(row_off + lo + i) <= r;
    const int k = __popc(__ballot_sync(0xffffffffu, le));
    if (k == 0) return -1;
    lo += (k - 1) * step;
    if (step == 1) return lo;
    n = min(step, n - (k - 1) * step);
  }
}

}  // namespace gqa
