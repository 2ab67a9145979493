// q4_mma.cu -- decode attention over the 4-bit cache on the tensor cores.
//
// One CTA per (chunk of a row's visible tiles, KV head x head split, query row); each of its four
// warps streams every fourth tile of the chunk through a ring of its own and keeps its own running
// maximum, sum and accumulator, so nothing but the end of the chunk synchronises the CTA.  A tile
// is TP positions of one KV head: four contiguous runs of the head-major cache (codes and scales of
// K and of V), which the warp's first lane copies with cp.async.bulk; the ring holds NST tiles.
//
// Both products run as mma.sync m16n8k16 with fp32 sums.  A = up to 8 query heads, their f16 hi
// part in rows 0-7 and the f16 remainder in rows 8-15 (22 bits of q and of the softmax weights);
// B = cache values, exact in f16 (q4_common.cuh): one conversion makes two codes f16x2 and one
// f16x2 product applies their scales.
//
// Fragments.  The dims and positions that a fragment's indices stand for are chosen so that a
// thread's codes are contiguous (lane = 4 g + t):
//   q.k  k index: thread t holds dims of its own 16-byte run of a position's codes, words w and
//        bytes in order; q's A fragments are laid out alike.  n index: column n of n-tile nt is
//        position 8 nt + 4 (n & 1) + ((n >> 1) ^ 3 (n & 1)).
//   p.v  k index: the same positions, so the weights go from C to A layout in place; thread t's
//        four are 4 j + (t ^ 3 (j & 1)), j = 0..3: for every j the four t read different banks as
//        far as rows of 32 or 64 bytes allow.  n index: column n of n-tile i is dim n D/8 + i, so
//        a thread's codes of a position are one run of D/16 bytes, and at D = 128 one scale.
//        Two positions' codes are interleaved nibble by nibble before the conversion.
#include "dispatch.h"
#include "q4_common.cuh"
#include "visible.cuh"
#include "visible_dispatch.h"

namespace gqa {

template <int D>
struct Q4Cfg {
  static constexpr int NW = 4;                      // warps
  static constexpr int RB = D / 2, SB = D / 16;     // bytes of a position's codes and scales
  static constexpr int TP = kQ4Tile;                // positions of a tile
  static constexpr int NB = TP / 16, NTK = TP / 8;  // 16-position blocks, n-tiles of q.k
  static constexpr int STAGE = 2 * TP * (RB + SB);  // [K codes][V codes][K scales][V scales]
  static constexpr int NST = D == 64 ? 6 : (D == 128 ? 4 : 3);
  static constexpr int MIN_CTAS = D == 256 ? 2 : 3;
  static constexpr int KS = D / 16;                 // k-steps of q.k
  static constexpr int KW = D / 32;                 // words of a thread's codes of a K position
  static constexpr int VW = D / 64;                 // ... of a V position
  static constexpr int NT = D / 8;                  // n-tiles of p.v
  static constexpr bool QSMEM = D == 256;           // q's fragments in shared memory
  static constexpr int RING = NW * NST * STAGE;
  static constexpr int MERGE = NW * 8 * (D + 2) * 4;
  static constexpr int QF_OFF = cmax(RING, align_up(MERGE, 16));
  static constexpr int QF_BYTES = QSMEM ? KS * 32 * 16 : 0;
  static constexpr int BAR_OFF = QF_OFF + QF_BYTES;
  static constexpr int SMEM = BAR_OFF + NW * NST * 8;
  static constexpr float RESCALE_LOG2 = 8.f;
};

// e4m3 bytes in bits 0-7 and 16-23 of x -> an f16x2 of their values.
__device__ __forceinline__ __half2 e4m3x2_to_f16x2(uint32_t x) {
  const uint32_t h = (x & 0x007f007fu) << 7;  // the values times 2^-8
  return __hmul2(*reinterpret_cast<const __half2*>(&h), __float2half2_rn(256.f));
}

__device__ __forceinline__ uint32_t mul_h2(uint32_t a, __half2 s) {
  return h2_bits(__hmul2(*reinterpret_cast<const __half2*>(&a), s));
}

template <int D>
__global__ void __launch_bounds__(32 * Q4Cfg<D>::NW, Q4Cfg<D>::MIN_CTAS)
    q4_mma_kernel(const Q4Params qp) {
  using C = Q4Cfg<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  const PartialParams& p = qp.base;
  const int c = blockIdx.x, t = blockIdx.z;
  const int kvh = blockIdx.y / p.head_split;
  const int G = p.group / p.head_split;  // query heads of this CTA (<= 8)
  const int head0 = kvh * p.group + (blockIdx.y % p.head_split) * G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");

  int s = 0;
  const int L = visible_row(p, t, c == 0 && blockIdx.y == 0 && threadIdx.x == 0, s);
  const Visible vis(L, p.window, p.n_sink);
  const VisibleTiles<C::TP, 16> tiles(vis);
  const int nchunks = (tiles.n + p.chunk - 1) / p.chunk;  // p.chunk: tiles of a chunk
  if (c >= nchunks) {
    if (c == 0)  // nothing to see: zeros
      for (int i = threadIdx.x; i < G * D; i += blockDim.x)
        p.out[((size_t)t * p.n_heads + head0) * D + i] = 0.f;
    return;
  }
  const int i0 = c * p.chunk + warp, i1 = min((c + 1) * p.chunk, tiles.n);

  uint8_t* ring = smem + warp * C::NST * C::STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF) + warp * C::NST;
  const size_t slab = ((size_t)s * p.n_kv_heads + kvh) * p.cache_cap;
  auto issue = [&](int i, int st) {  // lane 0: tile i's four runs into stage st
    const int start = tiles.start(i);
    const int n = min(C::TP, (tiles.end(i) - start + 15) & ~15);  // cache_cap is a multiple of 16
    const size_t row = slab + start;
    uint8_t* dst = ring + st * C::STAGE;
    mbar_arrive_expect_tx(&full[st], 2 * n * (C::RB + C::SB));
    bulk_load(dst, static_cast<const uint8_t*>(p.kc) + row * C::RB, n * C::RB, &full[st]);
    bulk_load(dst + C::TP * C::RB, static_cast<const uint8_t*>(p.vc) + row * C::RB, n * C::RB,
              &full[st]);
    dst += 2 * C::TP * C::RB;
    bulk_load(dst, reinterpret_cast<const uint8_t*>(p.ksc) + row * C::SB, n * C::SB, &full[st]);
    bulk_load(dst + C::TP * C::SB, reinterpret_cast<const uint8_t*>(p.vsc) + row * C::SB,
              n * C::SB, &full[st]);
  };
  int issued = 0;  // the warp's tiles asked for so far (uniform)
  if (lane == 0) {
    for (int st = 0; st < C::NST; ++st) mbar_init(&full[st], 1);
    mbar_init_fence();
    for (int i = i0; issued < C::NST && i < i1; i += C::NW, ++issued) issue(i, issued);
  }
  __syncwarp();  // the barriers, before any lane waits on one
  issued = __shfl_sync(0xffffffffu, issued, 0);

  // q's A fragments: the head's row scaled by a power of two to [1, 2) as f16 hi + lo; sm takes
  // the power, the softmax scale and the cache's scale of K back in
  uint32_t qa[C::QSMEM ? 1 : C::KS][4];
  uint4* qf = reinterpret_cast<uint4*>(smem + C::QF_OFF) + lane;
  float sm;
  {
    const bool hv = gid < G;
    const float* qrow = p.q + ((size_t)t * p.n_heads + head0 + (hv ? gid : 0)) * D;
    float4 x[C::KS];
    float amax = 0.f;
#pragma unroll
    for (int ks = 0; ks < C::KS; ++ks) {
      const int w = ks / 2;  // word of the thread's run of codes, half of it
      const int d = (w / 4) * 128 + (D == 64 ? 16 : 32) * tig + 8 * (w % 4) + 4 * (ks & 1);
      x[ks] = hv ? __ldg(reinterpret_cast<const float4*>(qrow + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
      amax = fmaxf(amax, fmaxf(fmaxf(fabsf(x[ks].x), fabsf(x[ks].y)),
                               fmaxf(fabsf(x[ks].z), fabsf(x[ks].w))));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const uint32_t e = min(max(__float_as_uint(amax) >> 23, 1u), 253u);
    const float f = __uint_as_float((254u - e) << 23);  // 2^(127 - e)
    sm = p.scale_log2 * qp.k_scale * __uint_as_float(e << 23);
#pragma unroll
    for (int ks = 0; ks < C::KS; ++ks) {
      uint32_t a[4];
      split_hi_lo(x[ks].x * f, x[ks].y * f, a[0], a[1]);
      split_hi_lo(x[ks].z * f, x[ks].w * f, a[2], a[3]);
      if constexpr (C::QSMEM) {
        if (warp == 0) qf[ks * 32] = make_uint4(a[0], a[1], a[2], a[3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) qa[ks][k] = a[k];
      }
    }
  }
  if constexpr (C::QSMEM) __syncthreads();

  float o[C::NT][4];
#pragma unroll
  for (int n = 0; n < C::NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  float m_run = -INFINITY, l_run = 0.f;  // head gid; l_run over this thread's positions
  // this thread's rows of a 16-position block: K columns of both n-tiles, V positions
  const int krow = 4 * (gid & 1) + ((gid >> 1) ^ (3 * (gid & 1)));
  int done = 0;
  bool ok = true;
  for (int i = i0; i < i1; i += C::NW, ++done) {
    const int st = done % C::NST;
    ok = __all_sync(0xffffffffu, mbar_wait(&full[st], (done / C::NST) & 1));
    if (!ok) break;
    const uint8_t* sk = ring + st * C::STAGE;
    const uint8_t* sv = sk + C::TP * C::RB;
    const uint8_t* ssk = sv + C::TP * C::RB;
    const uint8_t* ssv = ssk + C::TP * C::SB;
    const int lo = tiles.lo(i) - tiles.start(i), hi = tiles.end(i) - tiles.start(i);
    // -- S = Q . K^T of the tile's 32 positions, four n-tiles
    float sc[C::NTK][4];
#pragma unroll
    for (int nt = 0; nt < C::NTK; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
    for (int k = 0; k < (C::KW + 3) / 4; ++k) {  // a thread's 16-byte runs of codes
      constexpr int W = cmin(C::KW, 4);
      uint32_t kw[C::NTK][W];
      __half2 ks2[C::NTK][W / 2];  // one scale per two words, broadcast
#pragma unroll
      for (int nt = 0; nt < C::NTK; ++nt) {
        const int r = 8 * nt + krow;
        if constexpr (D == 64) {
          const uint2 u = *reinterpret_cast<const uint2*>(sk + r * C::RB + 8 * tig);
          kw[nt][0] = u.x;
          kw[nt][1] = u.y;
          const uint32_t b0 = ssk[r * C::SB + tig];
          ks2[nt][0] = e4m3x2_to_f16x2(b0 | b0 << 16);
        } else {
          const uint4 u = *reinterpret_cast<const uint4*>(sk + r * C::RB + 64 * k + 16 * tig);
          kw[nt][0] = u.x;
          kw[nt][1] = u.y;
          kw[nt][2] = u.z;
          kw[nt][3] = u.w;
          const uint32_t b2 =
              *reinterpret_cast<const uint16_t*>(ssk + r * C::SB + 8 * k + 2 * tig);
          const __half2 h = e4m3x2_to_f16x2(__byte_perm(b2, 0, 0x4140));
          ks2[nt][0] = __low2half2(h);
          ks2[nt][1] = __high2half2(h);
        }
      }
#pragma unroll
      for (int w = 0; w < W; ++w) {
        uint32_t a[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int ks = 2 * (4 * k + w) + e;
          if constexpr (C::QSMEM) {
            const uint4 a4 = qf[ks * 32];
            a[e][0] = a4.x;
            a[e][1] = a4.y;
            a[e][2] = a4.z;
            a[e][3] = a4.w;
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) a[e][i] = qa[ks][i];
          }
        }
#pragma unroll
        for (int nt = 0; nt < C::NTK; ++nt) {
          uint32_t h[4];
          e2m1x8_to_f16x2(kw[nt][w], h);
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = mul_h2(h[e], ks2[nt][w / 2]);
          mma_f16(sc[nt], a[0], h[0], h[1]);
          mma_f16(sc[nt], a[1], h[2], h[3]);
        }
      }
    }
    // -- head gid's scores at positions 8 nt + 4 j + (tig ^ 3 j)
    float x[C::NTK][2];
    float mt = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < C::NTK; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) x[nt][j] = (sc[nt][j] + sc[nt][2 + j]) * sm;
    if (lo > 0 || hi < C::TP) {
#pragma unroll
      for (int nt = 0; nt < C::NTK; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = 8 * nt + 4 * j + (tig ^ (3 * j));
          if (r < lo || r >= hi) x[nt][j] = -INFINITY;
        }
    }
#pragma unroll
    for (int nt = 0; nt < C::NTK; ++nt) mt = fmaxf(mt, fmaxf(x[nt][0], x[nt][1]));
    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
    // -- the running maximum moves only when a tile exceeds it by 2^8 (weights <= 256)
    const bool grow = mt > m_run + C::RESCALE_LOG2;
    if (__any_sync(0xffffffffu, grow)) {
      const float m_new = grow ? mt : m_run;
      const float corr = m_run == -INFINITY ? 0.f : fast_exp2(m_run - m_new);
      m_run = m_new;
      l_run *= corr;
#pragma unroll
      for (int n = 0; n < C::NT; ++n) {
        o[n][0] *= corr;
        o[n][1] *= corr;
        o[n][2] *= corr;
        o[n][3] *= corr;
      }
    }
    const float mu = m_run == -INFINITY ? 0.f : m_run;
#pragma unroll
    for (int nt = 0; nt < C::NTK; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        x[nt][j] = fast_exp2(x[nt][j] - mu);  // 0 where masked
        l_run += x[nt][j];
      }
    // -- O += P . V, 16 positions at a time.  Codes of a masked position are finite whatever they
    //    hold, and weigh 0; behind the positions that were copied the stage holds older codes.
#pragma unroll
    for (int b = 0; b < C::NB; ++b) {
      uint32_t pa[4];
      split_hi_lo(x[2 * b][0], x[2 * b][1], pa[0], pa[1]);
      split_hi_lo(x[2 * b + 1][0], x[2 * b + 1][1], pa[2], pa[3]);
      uint32_t vw[4][C::VW];
      uint32_t vs[4];  // scales: one byte, or two at D = 256
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 16 * b + 4 * j + (tig ^ (3 * (j & 1)));
        const uint8_t* src = sv + r * C::RB + gid * (D / 16);
        if constexpr (D == 64) {
          vw[j][0] = *reinterpret_cast<const uint32_t*>(src);
          vs[j] = ssv[r * C::SB + gid / 2];
        } else if constexpr (D == 128) {
          const uint2 u = *reinterpret_cast<const uint2*>(src);
          vw[j][0] = u.x;
          vw[j][1] = u.y;
          vs[j] = ssv[r * C::SB + gid];
        } else {
          const uint4 u = *reinterpret_cast<const uint4*>(src);
          vw[j][0] = u.x;
          vw[j][1] = u.y;
          vw[j][2] = u.z;
          vw[j][3] = u.w;
          vs[j] = *reinterpret_cast<const uint16_t*>(ssv + r * C::SB + 2 * gid);
        }
      }
#pragma unroll
      for (int h = 0; h < (D == 256 ? 2 : 1); ++h) {  // scale groups of the thread's dims
        __half2 s01, s23;
        if constexpr (D == 256) {
          s01 = e4m3x2_to_f16x2(__byte_perm(vs[0], vs[1], h ? 0x5511 : 0x4400));
          s23 = e4m3x2_to_f16x2(__byte_perm(vs[2], vs[3], h ? 0x5511 : 0x4400));
        } else {
          s01 = e4m3x2_to_f16x2(vs[0] | vs[1] << 16);
          s23 = e4m3x2_to_f16x2(vs[2] | vs[3] << 16);
        }
        constexpr int WG = D == 256 ? 2 : C::VW;  // words of the group
#pragma unroll
        for (int w = 0; w < WG; ++w) {
          const int ww = WG * h + w;
          constexpr uint32_t M = 0x0f0f0f0fu;
          uint32_t e01[4], o01[4], e23[4], o23[4];  // even and odd dims of two positions
          e2m1x8_to_f16x2((vw[0][ww] & M) | ((vw[1][ww] << 4) & ~M), e01);
          e2m1x8_to_f16x2(((vw[0][ww] >> 4) & M) | (vw[1][ww] & ~M), o01);
          e2m1x8_to_f16x2((vw[2][ww] & M) | ((vw[3][ww] << 4) & ~M), e23);
          e2m1x8_to_f16x2(((vw[2][ww] >> 4) & M) | (vw[3][ww] & ~M), o23);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            mma_f16(o[8 * ww + 2 * k], pa, mul_h2(e01[k], s01), mul_h2(e23[k], s23));
            mma_f16(o[8 * ww + 2 * k + 1], pa, mul_h2(o01[k], s01), mul_h2(o23[k], s23));
          }
        }
      }
    }
    __syncwarp();  // every lane has read the stage
    const int nxt = i + C::NST * C::NW;
    if (nxt < i1) {
      if (lane == 0) issue(nxt, st);
      ++issued;
    }
  }
  if (!ok) {
    if (lane == 0) flag_error(p.err, GQA_ERR_TIMEOUT);
    for (int k = done; k < issued; ++k)  // no copy may outlive the CTA
      (void)mbar_wait(&full[k % C::NST], (k / C::NST) & 1);
  }
  l_run += __shfl_xor_sync(0xffffffffu, l_run, 1);
  l_run += __shfl_xor_sync(0xffffffffu, l_run, 2);
  keep_nan(m_run, l_run, o);

  // ---- the four warps' states meet in shared memory (over the rings, which are drained)
  __syncthreads();
  float* mg = reinterpret_cast<float*>(smem);  // [warp][8][D + 2]
  float* mrow = mg + (warp * 8 + gid) * (D + 2);
#pragma unroll
  for (int n = 0; n < C::NT; ++n) {
    mrow[2 * tig * (D / 8) + n] = o[n][0] + o[n][2];
    mrow[(2 * tig + 1) * (D / 8) + n] = o[n][1] + o[n][3];
  }
  if (tig == 0) {
    mrow[D] = m_run;
    mrow[D + 1] = l_run;
  }
  __syncthreads();
  const bool split = nchunks > 1;
  for (int idx = threadIdx.x; idx < G * D; idx += 32 * C::NW) {
    const int h = idx / D, d = idx % D;
    float M = -INFINITY, A = 0.f, Ls = 0.f;
#pragma unroll
    for (int w = 0; w < C::NW; ++w) M = fmaxf(M, mg[(w * 8 + h) * (D + 2) + D]);
#pragma unroll
    for (int w = 0; w < C::NW; ++w) {
      const float* r = mg + (w * 8 + h) * (D + 2);
      const float e = r[D] == -INFINITY ? 0.f : fast_exp2(r[D] - M);
      A = fmaf(r[d], e, A);
      Ls = fmaf(r[D + 1], e, Ls);
    }
    A *= qp.v_scale;
    const int head = head0 + h;
    if (split) {
      float* pr = p.part + (((size_t)t * p.n_split + c) * p.n_heads + head) * (D + 2);
      pr[d] = A;
      if (d == 0) {
        pr[D] = M == -INFINITY ? -INFINITY : M * kLn2;  // natural-log units
        pr[D + 1] = Ls;
      }
    } else {
      p.out[((size_t)t * p.n_heads + head) * D + d] = gated(p, t, head, d, Ls > 0.f ? A / Ls : 0.f);
    }
  }
  if (split)
    merge_if_last<D>(p, t, head0, G, (size_t)t * gridDim.y + blockIdx.y, nchunks, C::NW);
}

template <int D>
static cudaError_t launch_q4_d(const Q4Params& qp, dim3 grid, cudaStream_t s) {
  using C = Q4Cfg<D>;
  const void* fn = reinterpret_cast<const void*>(&q4_mma_kernel<D>);
  cudaError_t e = ensure_smem(fn, C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(32 * C::NW);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  cfg.attrs = at;
  cfg.numAttrs = cluster_attrs(at, 0, 1);
  return cudaLaunchKernelEx(&cfg, &q4_mma_kernel<D>, qp);
}

cudaError_t launch_q4(int head_dim, const Q4Params& qp, dim3 grid, cudaStream_t s) {
  if (head_dim == 64) return launch_q4_d<64>(qp, grid, s);
  if (head_dim == 128) return launch_q4_d<128>(qp, grid, s);
  return launch_q4_d<256>(qp, grid, s);
}

}  // namespace gqa
