// append_q4.cu -- rows into and out of the 4-bit cache (kv_append_q4, kv_read_q4).
//
// A thread holds 8 consecutive dims of a (row, KV head) of K and of V: 32 bytes of fp32 and 4 bytes
// of codes each, so a warp's loads and stores cover whole 128-byte lines; two threads share the
// scale of 16 dims.  Threads are numbered dim slice first, then the row within a block of 16 rows,
// then the KV head: a row block of one head is one run of the head-major cache, so that its scales
// (8 bytes a position at D = 128) meet in whole 32-byte sectors.
#include <cuda_runtime_api.h>

#include <cmath>
#include <cstdio>

#include "gqa_decode.h"
#include "q4_common.cuh"

namespace gqa {

void set_last_error(const char* msg);  // host.cu: the text gqa_last_error() returns

constexpr int kRowBlock = 16;
constexpr int kQ4Threads = 128;

struct Q4Rows {
  uint8_t *kq, *vq, *ksc, *vsc;
  const int32_t* row_off;
  const int32_t* t0;
  int32_t* err;
  int n_rows, hk, n_seq;
  long long cap;
  float k_scale, v_scale;  // append: their inverses
};

// Where the thread's 8 dims are: the batch's element and the cache's (row, slice); false when the
// thread has no row.  Every lane of the warp has to call it.
template <int D>
__device__ __forceinline__ bool q4_place(const Q4Rows& a, long long& elem, long long& crow,
                                         int& slice) {
  constexpr int TPR = D / 8;                       // threads per (row, head): 8, 16 or 32
  constexpr int RPW = 32 / TPR;                    // rows of a warp
  const long long i = (long long)blockIdx.x * kQ4Threads + threadIdx.x;
  slice = static_cast<int>(i % TPR);
  const long long u = i / TPR;                     // (row block, head, row)
  const long long per = (long long)kRowBlock * a.hk;
  const long long rb = u / per;
  const int head = static_cast<int>(u % per / kRowBlock);
  const long long r = rb * kRowBlock + u % kRowBlock;
  const long long end = __ldg(a.row_off + a.n_seq);
  const bool in = r < a.n_rows && r < end;
  // a warp's rows are RPW consecutive ones of one head (kRowBlock is a multiple of RPW)
  const int r_first = __shfl_sync(0xffffffffu, static_cast<int>(min(r, (long long)INT32_MAX)), 0);
  int s = -1;
#pragma unroll
  for (int k = 0; k < RPW; ++k) {
    if (r_first + k >= a.n_rows || r_first + k >= end) break;
    const int f = ragged_find(a.row_off, a.n_seq, r_first + k);
    if (r == r_first + k) s = f;
  }
  if (!in) return false;
  const int first = s < 0 ? 0 : __ldg(a.row_off + s);
  if (s < 0 || r < first || r >= __ldg(a.row_off + s + 1)) {
    flag_error(a.err, GQA_ERR_SEQ_RANGE);
    return false;
  }
  const long long pos = (long long)__ldg(a.t0 + s) + (r - first);
  if (pos < 0 || pos >= a.cap) {
    flag_error(a.err, GQA_ERR_KVLEN_RANGE);
    return false;
  }
  elem = (r * a.hk + head) * D + slice * 8;
  crow = ((long long)s * a.hk + head) * a.cap + pos;
  return true;
}

// The e4m3 bits nearest to amax / 6, ties to even, at most 448, from the unrounded quotient: the
// quotient truncated to fp32 takes a set last bit when it is not exact, so that the second
// rounding sees which side of a midpoint it is on.
__device__ __forceinline__ uint32_t q4_scale(float amax) {
  const float c = fminf(amax, 6.f * 448.f);
  float t = __fdiv_rz(c, 6.f);
  if (fmaf(-6.f, t, c) != 0.f) t = __uint_as_float(__float_as_uint(t) | 1u);
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(t));
  return r & 0x7fu;
}

// The e2m1 code nearest to |y| / s, ties to the even code: a binary search of the midpoints
// 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, each times s exact in fp32.
__device__ __forceinline__ uint32_t q4_code(float y, float s) {
  const float a = fabsf(y);
  const bool b2 = a >= 1.75f * s;
  const bool b1 = a >= (b2 ? 3.5f : 0.75f) * s;
  const bool b0 = a > (b2 ? (b1 ? 5.f : 2.5f) : (b1 ? 1.25f : 0.25f)) * s;
  uint32_t c = (b2 ? 4u : 0u) | (b1 ? 2u : 0u) | (b0 ? 1u : 0u);
  if (y < 0.f && c) c |= 8u;
  return c;
}

// Quantises this thread's 8 dims of one side; its partner (lane xor 1) holds the other 8 of the
// scale's 16.  All lanes of the warp take part in the exchange.
__device__ __forceinline__ void q4_quantise(const float4& x0, const float4& x1, float inv, bool on,
                                            uint32_t& codes, uint32_t& scale) {
  float y[8] = {x0.x * inv, x0.y * inv, x0.z * inv, x0.w * inv,
                x1.x * inv, x1.y * inv, x1.z * inv, x1.w * inv};
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(y[e]));  // fmaxf drops a NaN
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  scale = on ? q4_scale(amax) : 0u;
  codes = 0;
  if (!scale) return;
  const float s = e4m3_to_f32(scale);
#pragma unroll
  for (int e = 0; e < 8; ++e) codes |= q4_code(y[e], s) << (4 * e);
}

template <int D>
__global__ void __launch_bounds__(kQ4Threads)
    append_q4_kernel(const float* __restrict__ k_new, const float* __restrict__ v_new, Q4Rows a) {
  long long elem = 0, crow = 0;
  int slice = 0;
  const bool on = q4_place<D>(a, elem, crow, slice);
  float4 k0{}, k1{}, v0{}, v1{};
  if (on) {
    k0 = __ldg(reinterpret_cast<const float4*>(k_new + elem));
    k1 = __ldg(reinterpret_cast<const float4*>(k_new + elem) + 1);
    v0 = __ldg(reinterpret_cast<const float4*>(v_new + elem));
    v1 = __ldg(reinterpret_cast<const float4*>(v_new + elem) + 1);
  }
  uint32_t kc, ks, vc, vs;
  q4_quantise(k0, k1, a.k_scale, on, kc, ks);
  q4_quantise(v0, v1, a.v_scale, on, vc, vs);
  if (!on) return;
  *reinterpret_cast<uint32_t*>(a.kq + crow * (D / 2) + slice * 4) = kc;
  *reinterpret_cast<uint32_t*>(a.vq + crow * (D / 2) + slice * 4) = vc;
  if ((slice & 1) == 0) {
    a.ksc[crow * (D / 16) + slice / 2] = static_cast<uint8_t>(ks);
    a.vsc[crow * (D / 16) + slice / 2] = static_cast<uint8_t>(vs);
  }
}

// 8 codes times scale s -> 8 values.
__device__ __forceinline__ void q4_values(uint32_t codes, float s, float (&f)[8]) {
  uint32_t h[4];
  e2m1x8_to_f16x2(codes, h);
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h[b]));
    f[2 * b] = x.x * s;
    f[2 * b + 1] = x.y * s;
  }
}

template <typename T>
__device__ __forceinline__ void q4_store(T* dst, const float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(dst)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    union {
      __half2 h[4];
      uint4 u;
    } o;
#pragma unroll
    for (int b = 0; b < 4; ++b) o.h[b] = __floats2half2_rn(f[2 * b], f[2 * b + 1]);
    *reinterpret_cast<uint4*>(dst) = o.u;
  }
}

template <int D, typename T>
__global__ void __launch_bounds__(kQ4Threads)
    read_q4_kernel(T* __restrict__ k_out, T* __restrict__ v_out, Q4Rows a) {
  long long elem = 0, crow = 0;
  int slice = 0;
  if (!q4_place<D>(a, elem, crow, slice)) return;
  const uint32_t kc = __ldg(reinterpret_cast<const uint32_t*>(a.kq + crow * (D / 2)) + slice);
  const uint32_t vc = __ldg(reinterpret_cast<const uint32_t*>(a.vq + crow * (D / 2)) + slice);
  const uint32_t ks = __ldg(a.ksc + crow * (D / 16) + slice / 2);
  const uint32_t vs = __ldg(a.vsc + crow * (D / 16) + slice / 2);
  float f[8];
  q4_values(kc, e4m3_to_f32(ks) * a.k_scale, f);
  q4_store(k_out + elem, f);
  q4_values(vc, e4m3_to_f32(vs) * a.v_scale, f);
  q4_store(v_out + elem, f);
}

bool q4_scale_ok(float s) {
  int e = 0;
  return std::isfinite(s) && s > 0.f && std::frexp(s, &e) == 0.5f && e >= -63 && e <= 65;
}

// The checks and the launch that both calls share; `go(blocks)` launches for the head size.
template <class Go>
gqa_status q4_rows_call(const char* name, const Q4Rows& a, int head_dim, const void* x,
                        const void* y, Go go) {
  auto bad = [&](gqa_status st, const char* what) {
    char buf[256];
    snprintf(buf, sizeof buf, "%s: %s", name, what);
    set_last_error(buf);
    return st;
  };
  if (a.n_rows < 0 || a.hk <= 0 || a.n_seq <= 0 ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return bad(GQA_EINVAL, "n_rows >= 0, n_kv_heads and n_seq >= 1, head_dim in {64, 128, 256}");
  if (a.cap <= 0 || a.cap % 16)
    return bad(GQA_EINVAL, "cache_cap must be a positive multiple of 16");
  if (!q4_scale_ok(a.k_scale) || !q4_scale_ok(a.v_scale))
    return bad(GQA_EINVAL, "k_scale and v_scale must be powers of two in [2^-64, 2^64]");
  if (a.n_rows == 0) return GQA_OK;
  if (!x || !y || !a.kq || !a.vq || !a.ksc || !a.vsc || !a.row_off || !a.t0)
    return bad(GQA_EINVAL, "a required pointer is NULL");
  auto bits = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  if ((bits(x) | bits(y) | bits(a.kq) | bits(a.vq) | bits(a.ksc) | bits(a.vsc)) & 15)
    return bad(GQA_EINVAL, "the rows, codes and scales must be 16-byte aligned");
  if ((bits(a.row_off) | bits(a.t0) | bits(a.err)) & 3)
    return bad(GQA_EINVAL, "row_off, t0 and err_word must be 4-byte aligned");
  const long long blocks_of_rows = (a.n_rows + (long long)kRowBlock - 1) / kRowBlock;
  if (blocks_of_rows * a.hk > (1LL << 40))
    return bad(GQA_EUNSUPPORTED, "too many rows for one launch");
  const long long threads = blocks_of_rows * kRowBlock * a.hk * (head_dim / 8);
  const long long blocks = (threads + kQ4Threads - 1) / kQ4Threads;
  if (blocks > 0x7fffffffLL) return bad(GQA_EUNSUPPORTED, "too many rows for one launch");
  go(static_cast<unsigned>(blocks));
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? GQA_OK : bad(GQA_ECUDA, cudaGetErrorString(e));
}

}  // namespace gqa

extern "C" gqa_status kv_append_q4(const float* k_new, const float* v_new, int n_rows,
                                   int n_kv_heads, int head_dim, const int32_t* row_off,
                                   const int32_t* t0, float k_scale, float v_scale, uint8_t* kq,
                                   uint8_t* vq, uint8_t* ksc, uint8_t* vsc, int n_seq,
                                   int64_t cache_cap, int32_t* err_word, cudaStream_t stream) {
  gqa::Q4Rows a{kq,     vq,         ksc,   vsc,       row_off, t0,     err_word,
                n_rows, n_kv_heads, n_seq, cache_cap, k_scale, v_scale};
  return gqa::q4_rows_call("kv_append_q4", a, head_dim, k_new, v_new, [&](unsigned blocks) {
    gqa::Q4Rows b = a;
    b.k_scale = 1.f / k_scale;
    b.v_scale = 1.f / v_scale;
    if (head_dim == 64)
      gqa::append_q4_kernel<64><<<blocks, gqa::kQ4Threads, 0, stream>>>(k_new, v_new, b);
    else if (head_dim == 128)
      gqa::append_q4_kernel<128><<<blocks, gqa::kQ4Threads, 0, stream>>>(k_new, v_new, b);
    else
      gqa::append_q4_kernel<256><<<blocks, gqa::kQ4Threads, 0, stream>>>(k_new, v_new, b);
  });
}

extern "C" gqa_status kv_read_q4(const uint8_t* kq, const uint8_t* vq, const uint8_t* ksc,
                                 const uint8_t* vsc, int n_seq, int64_t cache_cap, int n_rows,
                                 int n_kv_heads, int head_dim, const int32_t* row_off,
                                 const int32_t* t0, float k_scale, float v_scale, void* k_out,
                                 void* v_out, int out_f16, int32_t* err_word,
                                 cudaStream_t stream) {
  gqa::Q4Rows a{const_cast<uint8_t*>(kq),  const_cast<uint8_t*>(vq),
                const_cast<uint8_t*>(ksc), const_cast<uint8_t*>(vsc),
                row_off, t0, err_word, n_rows, n_kv_heads, n_seq, cache_cap, k_scale, v_scale};
  return gqa::q4_rows_call("kv_read_q4", a, head_dim, k_out, v_out, [&](unsigned blocks) {
    auto launch = [&](auto kern32, auto kern16) {
      if (out_f16)
        kern16<<<blocks, gqa::kQ4Threads, 0, stream>>>(static_cast<__half*>(k_out),
                                                       static_cast<__half*>(v_out), a);
      else
        kern32<<<blocks, gqa::kQ4Threads, 0, stream>>>(static_cast<float*>(k_out),
                                                       static_cast<float*>(v_out), a);
    };
    if (head_dim == 64)
      launch(gqa::read_q4_kernel<64, float>, gqa::read_q4_kernel<64, __half>);
    else if (head_dim == 128)
      launch(gqa::read_q4_kernel<128, float>, gqa::read_q4_kernel<128, __half>);
    else
      launch(gqa::read_q4_kernel<256, float>, gqa::read_q4_kernel<256, __half>);
  });
}
