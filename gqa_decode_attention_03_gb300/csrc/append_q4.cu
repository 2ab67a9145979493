// append_q4.cu -- rows into and out of the 4-bit cache (kv_append_q4, kv_read_q4).
//
// A row of a KV head is a unit; a CTA takes 16 units, K and V, in the batch's own order, so that the
// fp32 side is one run of memory (reading six sequences of up to 8192 rows of 8 heads of 128, caches
// and outputs not in L2: 38.0 us against 40.7 where a CTA takes 16 rows of one head).  A thread holds 8
// consecutive dims of a unit, 4 where it writes fp32, so that every load and store of a warp covers
// whole 32-byte sectors of rows and codes; two threads share the scale of 16 dims in appending.  New
// rows are asked for before their place is known: their address does not depend on it.
//
// Bound by memory: 19937 rows of 8 heads of 128 dims appended and read back as fp32 in 59.8 us on
// GB300, 373 MB at 6.2 TB/s; the sequences above read at 6.0 TB/s, 228 MB.  With the codes found by
// comparisons alone appending was bound by instructions (95 us in all); with every row's sequence
// searched for anew the two took 63.4 and 39.0 from L2 as far as it reached.
#include <cuda_runtime_api.h>

#include <climits>
#include <cmath>
#include <cstdio>
#include <type_traits>

#include "gqa_decode.h"
#include "q4_common.cuh"

namespace gqa {

void set_last_error(const char* msg);  // host.cu: the text gqa_last_error() returns

constexpr int kUnits = 16;  // of a CTA

struct Q4Rows {
  uint8_t *kq, *vq, *ksc, *vsc;
  const int32_t* row_off;
  const int32_t* t0;
  int32_t* err;
  int n_rows, hk, n_seq;
  long long cap;
  float k_scale, v_scale;  // append: their inverses
};

// Threads of a CTA with DPT dims of UNITS units at a time.
template <int D, int DPT, int UNITS>
constexpr int kQ4Threads = UNITS * (D / DPT);

// A row of the batch, its KV head, the thread's first element there.
struct Q4Slot {
  int r, head;
  long long elem;
};
// The thread's unit of units j, j + 1, .. of the CTA's.
template <int D, int DPT>
__device__ __forceinline__ Q4Slot q4_slot(const Q4Rows& a, int j) {
  const unsigned u = blockIdx.x * kUnits + j + threadIdx.x / (D / DPT);
  Q4Slot s;
  s.r = static_cast<int>(u / a.hk);
  s.head = static_cast<int>(u - s.r * a.hk);
  s.elem = (long long)u * D + threadIdx.x % (D / DPT) * DPT;
  return s;
}

// The sequence found last: it holds rows [first, next) of the batch.
struct Q4Seq {
  int s = -1, first = 0, next = INT_MIN;
};

// The cache row of the thread's row; false when no sequence holds it or its position is none of the
// cache's (flagged).  Every lane of the warp has to call it; a warp's units are consecutive, and the
// search is made anew only where their rows leave the sequence that the ones before belong to.
template <int D, int DPT>
__device__ __forceinline__ bool q4_place(const Q4Rows& a, const Q4Slot& sl, Q4Seq& q, long long& crow) {
  constexpr int RPW = D / DPT >= 32 ? 1 : 32 / (D / DPT);  // units, and rows at most, of a warp
  const int end = min(__ldg(a.row_off + a.n_seq), a.n_rows);
  const int r_first = __shfl_sync(0xffffffffu, sl.r, 0);
  const int r_last = __shfl_sync(0xffffffffu, sl.r, 31);  // (no row ahead: q serves the next units too)
  Q4Seq mine;
#pragma unroll
  for (int k = 0; k < RPW; ++k) {
    if (r_first + k > r_last || r_first + k >= end) break;
    if (r_first + k >= q.next) {
      q.s = ragged_find(a.row_off, a.n_seq, r_first + k);
      q.first = __ldg(a.row_off + max(q.s, 0));
      q.next = q.s < 0 ? INT_MIN : __ldg(a.row_off + q.s + 1);
    }
    if (sl.r == r_first + k) mine = q;
  }
  if (sl.r >= end) return false;
  if (mine.s < 0 || sl.r < mine.first || sl.r >= mine.next) {
    flag_error(a.err, GQA_ERR_SEQ_RANGE);
    return false;
  }
  const long long pos = (long long)__ldg(a.t0 + mine.s) + sl.r - mine.first;
  if (pos < 0 || pos >= a.cap) {
    flag_error(a.err, GQA_ERR_KVLEN_RANGE);
    return false;
  }
  crow = ((long long)mine.s * a.hk + sl.head) * a.cap + pos;
  return true;
}

// Two values to the nearest e4m3 codes, at most 448: a in the low byte.
__device__ __forceinline__ uint32_t e4m3x2_from_f32(float a, float b) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// The e4m3 bits nearest to amax / 6, ties to even, at most 448, from the unrounded quotient.  That is
// bracketed: the product with 1 / 6, both rounded towards 0, is at most 2^-22 below it, so 4 units in
// the last place more are at least it.  Where a midpoint lies between the ends the quotient truncated
// to fp32 takes a set last bit if it is not exact, so that the second rounding sees its side.
__device__ __forceinline__ uint32_t q4_scale(float amax) {
  const float c = fminf(amax, 6.f * 448.f);
  const float lo = __fmul_rz(c, __uint_as_float(0x3e2aaaaau));
  uint32_t r = e4m3x2_from_f32(lo, __uint_as_float(__float_as_uint(lo) + 4u));
  if ((r & 0xffu) != r >> 8) {
    float t = __fdiv_rz(c, 6.f);
    if (fmaf(-6.f, t, c) != 0.f) t = __uint_as_float(__float_as_uint(t) | 1u);
    r = e4m3x2_from_f32(t, t);
  }
  return r & 0x7fu;
}

// The e2m1 code nearest to |y| / s, ties to the even code: a binary search of the midpoints
// 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, each times s exact in fp32.  NaN gives 0.
__device__ __forceinline__ uint32_t q4_code(float y, float s) {
  const float a = fabsf(y);
  const bool b2 = a >= 1.75f * s;
  const bool b1 = a >= (b2 ? 3.5f : 0.75f) * s;
  const bool b0 = a > (b2 ? (b1 ? 5.f : 2.5f) : (b1 ? 1.25f : 0.25f)) * s;
  uint32_t c = (b2 ? 4u : 0u) | (b1 ? 2u : 0u) | (b0 ? 1u : 0u);
  if (y < 0.f && c) c |= 8u;
  return c;
}

// Eight values to the nearest e2m1 codes, the first in the low nibble.
__device__ __forceinline__ uint32_t e2m1x8_from_f32(const float (&q)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return r;
}

// The codes of 8 values y under scale s > 0, the quotient bracketed again: 1 / s to one unit in the
// last place, less two, is at most 3 units below it, and the truncated product at most 2^-21 below the
// quotient, so 8 units more are at least it.  Where both ends have the same codes those are the
// quotient's; elsewhere (a midpoint between the ends: ~2e-6 of random values, exact ties) the
// comparisons decide.  So they do for a NaN, whose upper end wraps round to a tiny value and code 0,
// and for a negative infinity, whose upper end is a NaN and takes the largest positive code.
__device__ __forceinline__ uint32_t q4_codes(const float (&y)[8], float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  r = __uint_as_float(__float_as_uint(r) - 2u);
  float lo[8], hi[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    lo[e] = __fmul_rz(y[e], r);
    hi[e] = __uint_as_float(__float_as_uint(lo[e]) + 8u);
  }
  uint32_t c = e2m1x8_from_f32(lo);
  if (c != e2m1x8_from_f32(hi)) {
    c = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) c |= q4_code(y[e], s) << (4 * e);
    return c;
  }
  const uint32_t some = (c | c >> 1 | c >> 2) & 0x11111111u;  // a code of 0 has no sign
  return c & (0x77777777u | some << 3);
}

// Quantises this thread's 8 dims of one side; its partner (lane xor 1) holds the other 8 of the
// scale's 16.  All lanes of the warp take part in the exchange.
__device__ __forceinline__ void q4_quantise(const float4& x0, const float4& x1, float inv,
                                            uint32_t& codes, uint32_t& scale) {
  const float y[8] = {x0.x * inv, x0.y * inv, x0.z * inv, x0.w * inv,
                      x1.x * inv, x1.y * inv, x1.z * inv, x1.w * inv};
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(y[e]));  // fmaxf drops a NaN
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  scale = q4_scale(amax);
  codes = scale ? q4_codes(y, e4m3_to_f32(scale)) : 0u;
}

template <int D>
__global__ void __launch_bounds__(kQ4Threads<D, 8, kUnits>)
    append_q4_kernel(const float* __restrict__ k_new, const float* __restrict__ v_new, Q4Rows a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const Q4Slot sl = q4_slot<D, 8>(a, 0);
  float4 k0{}, k1{}, v0{}, v1{};
  if (sl.r < a.n_rows) {
    k0 = __ldcs(reinterpret_cast<const float4*>(k_new + sl.elem));
    k1 = __ldcs(reinterpret_cast<const float4*>(k_new + sl.elem) + 1);
    v0 = __ldcs(reinterpret_cast<const float4*>(v_new + sl.elem));
    v1 = __ldcs(reinterpret_cast<const float4*>(v_new + sl.elem) + 1);
  }
  long long crow = 0;
  Q4Seq seq;
  const bool on = q4_place<D, 8>(a, sl, seq, crow);
  uint32_t kc, ks, vc, vs;
  q4_quantise(k0, k1, a.k_scale, kc, ks);
  q4_quantise(v0, v1, a.v_scale, vc, vs);
  if (!on) return;
  const int slice = threadIdx.x % (D / 8);
  *reinterpret_cast<uint32_t*>(a.kq + crow * (D / 2) + slice * 4) = kc;
  *reinterpret_cast<uint32_t*>(a.vq + crow * (D / 2) + slice * 4) = vc;
  if ((slice & 1) == 0) {
    a.ksc[crow * (D / 16) + slice / 2] = static_cast<uint8_t>(ks);
    a.vsc[crow * (D / 16) + slice / 2] = static_cast<uint8_t>(vs);
  }
}

// A thread in reading: 8 dims (fp32: 4) of two units 8 apart (f16: 25.0 us against 27.8 for the
// sequences above with one; four of fp32 looked up 64 short sequences too slowly, 7.3 us against 5.6).
template <typename T>
constexpr int kReadDims = sizeof(T) == 4 ? 4 : 8;
constexpr int kReadUnits = 8;

// The codes of a thread's dims, and their values times s, stored.
template <typename T>
__device__ __forceinline__ uint32_t q4_load(const uint8_t* src) {
  if constexpr (sizeof(T) == 4)
    return __ldg(reinterpret_cast<const uint16_t*>(src));
  else
    return __ldg(reinterpret_cast<const uint32_t*>(src));
}
template <typename T>
__device__ __forceinline__ void q4_store(T* dst, uint32_t codes, float s) {
  uint32_t h[4];
  e2m1x8_to_f16x2(codes, h);
  float2 x[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    x[b] = __half22float2(*reinterpret_cast<const __half2*>(&h[b]));
    x[b].x *= s;
    x[b].y *= s;
  }
  if constexpr (sizeof(T) == 4) {
    __stcs(reinterpret_cast<float4*>(dst), make_float4(x[0].x, x[0].y, x[1].x, x[1].y));
  } else {
    union {
      __half2 h2[4];
      uint4 u;
    } o;
#pragma unroll
    for (int b = 0; b < 4; ++b) o.h2[b] = __floats2half2_rn(x[b].x, x[b].y);
    __stcs(reinterpret_cast<uint4*>(dst), o.u);
  }
}

template <int D, typename T>
__global__ void __launch_bounds__(kQ4Threads<D, kReadDims<T>, kReadUnits>)
    read_q4_kernel(T* __restrict__ k_out, T* __restrict__ v_out, Q4Rows a) {
  constexpr int DPT = kReadDims<T>, N = kUnits / kReadUnits;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int slice = threadIdx.x % (D / DPT);
  Q4Slot sl[N];
  Q4Seq seq;
  bool on[N];
  uint32_t kc[N], vc[N], ks[N], vs[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    sl[j] = q4_slot<D, DPT>(a, j * kReadUnits);
    long long crow = 0;
    on[j] = q4_place<D, DPT>(a, sl[j], seq, crow);
    kc[j] = vc[j] = ks[j] = vs[j] = 0;
    if (on[j]) {
      kc[j] = q4_load<T>(a.kq + crow * (D / 2) + slice * (DPT / 2));
      vc[j] = q4_load<T>(a.vq + crow * (D / 2) + slice * (DPT / 2));
      ks[j] = __ldg(a.ksc + crow * (D / 16) + slice * DPT / 16);
      vs[j] = __ldg(a.vsc + crow * (D / 16) + slice * DPT / 16);
    }
  }
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (on[j]) {
      q4_store(k_out + sl[j].elem, kc[j], e4m3_to_f32(ks[j]) * a.k_scale);
      q4_store(v_out + sl[j].elem, vc[j], e4m3_to_f32(vs[j]) * a.v_scale);
    }
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
  const long long units = (long long)a.n_rows * a.hk;
  if (units > INT32_MAX - kUnits)
    return bad(GQA_EUNSUPPORTED, "n_rows * n_kv_heads must stay below 2^31 - 16");
  const long long blocks = (units + kUnits - 1) / kUnits;
  const cudaError_t e = go(static_cast<unsigned>(blocks));
  if (e == cudaSuccess) return GQA_OK;
  (void)cudaGetLastError();
  return bad(GQA_ECUDA, cudaGetErrorString(e));
}

// A launch whose scheduling overlaps the end of the kernel before it on the stream.
template <class Kern, class... Args>
cudaError_t q4_launch(Kern kern, unsigned blocks, int threads, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  cfg.attrs = at;
  cfg.numAttrs = cluster_attrs(at, 0, 1);
  return cudaLaunchKernelEx(&cfg, kern, args...);
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
    using namespace gqa;
    if (head_dim == 64)
      return q4_launch(append_q4_kernel<64>, blocks, kQ4Threads<64, 8, kUnits>, stream, k_new, v_new, b);
    if (head_dim == 128)
      return q4_launch(append_q4_kernel<128>, blocks, kQ4Threads<128, 8, kUnits>, stream, k_new, v_new, b);
    return q4_launch(append_q4_kernel<256>, blocks, kQ4Threads<256, 8, kUnits>, stream, k_new, v_new, b);
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
    using namespace gqa;
    auto launch = [&](auto d) {
      constexpr int D = decltype(d)::value;
      return out_f16 ? q4_launch(read_q4_kernel<D, __half>, blocks,
                                 kQ4Threads<D, kReadDims<__half>, kReadUnits>, stream,
                                 static_cast<__half*>(k_out), static_cast<__half*>(v_out), a)
                     : q4_launch(read_q4_kernel<D, float>, blocks,
                                 kQ4Threads<D, kReadDims<float>, kReadUnits>, stream,
                                 static_cast<float*>(k_out), static_cast<float*>(v_out), a);
    };
    if (head_dim == 64) return launch(std::integral_constant<int, 64>());
    if (head_dim == 128) return launch(std::integral_constant<int, 128>());
    return launch(std::integral_constant<int, 256>());
  });
}
