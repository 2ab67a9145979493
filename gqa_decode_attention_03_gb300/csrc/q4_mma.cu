// q4_mma.cu -- decode attention over the 4-bit cache on the tensor cores.
//
// One CTA per (chunk of visible tiles, KV head x head split, group of rows); each of its four warps
// streams every fourth tile of the chunk through a ring of its own and keeps its own running
// maximum, sum and accumulator, so nothing but the end of the chunk synchronises the CTA.  A tile
// is TP positions of one KV head: four contiguous runs of the head-major cache (codes and scales of
// K and of V), which the warp's first lane copies with cp.async.bulk; the ring holds NST tiles.
//
// A group is one row, or, where rows share sequences, the consecutive rows whose (row, head) pairs
// fill the 8 rows of the products that a row's heads leave empty: their tiles are those of the
// union of what the rows see, sequence by sequence, and each pair masks its own.
//
// Both products run as mma.sync m16n8k16 with fp32 sums.  A = up to 8 pairs, their f16 hi
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
#include "umma.cuh"
#include "visible.cuh"
#include "visible_dispatch.h"

namespace gqa {

template <int D>
struct Q4Cfg {
  static constexpr int NW = 4;                      // warps
  static constexpr int RB = D / 2, SB = D / 16;     // bytes of a position's codes and scales
  static constexpr int TP = q4_tile(D);             // positions of a tile, worked on SP at a time
  static constexpr int SP = 32, NB = SP / 16, NTK = SP / 8;  // 16-position blocks, n-tiles of q.k
  static constexpr int STAGE = 2 * TP * (RB + SB);  // [K codes][V codes][K scales][V scales]
  static constexpr int NST = D == 64 ? 4 : 2;
  static constexpr int MIN_CTAS = D == 256 ? 2 : 3;
  static constexpr int KS = D / 16;                 // k-steps of q.k
  static constexpr int KW = D / 32;                 // words of a thread's codes of a K position
  static constexpr int VW = D / 64;                 // ... of a V position
  static constexpr int NT = D / 8;                  // n-tiles of p.v
  static constexpr bool QSMEM = D == 256;           // q's fragments stay in shared memory
  static constexpr int RING = NW * NST * STAGE;
  static constexpr int MERGE = NW * 8 * (D + 2) * 4;  // the warps' states, over the rings
  // q's fragments: in a place of their own, or (then read into registers) in warp 0's last stage
  // before it takes its first tile
  static constexpr int QF_BYTES = KS * 32 * 16;
  static constexpr int QF_OFF = QSMEM ? RING : (NST - 1) * STAGE;
  static constexpr int NST0 = QSMEM ? NST : NST - 1;  // tiles asked for before q is in
  static constexpr int BAR_OFF = RING + (QSMEM ? QF_BYTES : 0);
  static constexpr int SMEM = BAR_OFF + NW * NST * 8;
  static_assert(QSMEM || QF_BYTES <= STAGE, "q's fragments fit a stage");
  static_assert(MIN_CTAS * (SMEM + 2304 + 1024) <= 228 * 1024, "MIN_CTAS fit an SM");
  static_assert(MERGE <= RING && 8 * kQ4MaxSplit * 4 <= RING, "merge areas inside the rings");
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

// A run of a group's rows that share a sequence: the union of what they see, as tiles.
struct Q4Run {
  int seq, tiles0;  // sequence; index of its first tile in the group's list
  int na, base;     // tiles of the sinks; where the window tiles start
  int ns, end;      // [0, ns) (if na) and [base, end)
};

// The walk of a warp over its group's tiles; lists of several runs are in shared memory.
template <int TP>
struct Q4Walk {
  Q4Run r;
  int k, next;  // the run, and the index of the first tile behind it
  __device__ __forceinline__ void start(const Q4Run* runs) {
    r = runs[0];
    k = 0;
    next = runs[1].tiles0;
  }
  // moves on to tile i's run; start and end of the tile's positions
  __device__ __forceinline__ void tile(const Q4Run* runs, int i, int& start, int& end) {
    while (i >= next) {
      r = runs[++k];
      next = runs[k + 1].tiles0;
    }
    const int j = i - r.tiles0;
    start = j < r.na ? j * TP : r.base + (j - r.na) * TP;
    end = j < r.na ? r.ns : r.end;
  }
};

template <int D>
__global__ void __launch_bounds__(32 * Q4Cfg<D>::NW, Q4Cfg<D>::MIN_CTAS)
    q4_mma_kernel(const Q4Params qp) {
  using C = Q4Cfg<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  const PartialParams& p = qp.base;
  __shared__ Q4Run s_runs[C::NW][9];
  __shared__ float s_amax[C::NW][8];
  const int c = blockIdx.x;
  const int kvh = blockIdx.y / p.head_split;
  const int G = p.group / p.head_split;  // query heads of this CTA (<= 8)
  const int head0 = kvh * p.group + (blockIdx.y % p.head_split) * G;
  const int t0 = blockIdx.z * qp.rows, nr = min(qp.rows, p.n_tok - t0);
  const int np = nr * G;                 // pairs: row gid / G, head gid % G
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");

  // ---- the rows (lane k: row k), their runs (every warp its own table) and this pair's row
  Q4Run* runs = s_runs[warp];
  int seq = 0, len = 0;
  if (lane < nr)
    len = visible_row(p, t0 + lane, c == 0 && blockIdx.y == 0 && warp == 0, seq);
  const int prow = gid < np ? gid / G : 0;
  int prun = -1, nruns = 0, n = 0;
  {
    Q4Run r{};
    auto close = [&] {
      r.base &= ~15;
      if (r.base <= r.ns) r.base = r.ns = 0;  // the two parts meet: [0, end)
      r.tiles0 = n;
      r.na = (r.ns + C::TP - 1) / C::TP;
      n += r.na + (r.end - r.base + C::TP - 1) / C::TP;
      if (lane == 0) runs[nruns - 1] = r;
    };
    for (int k = 0; k < nr; ++k) {
      const Visible v(__shfl_sync(0xffffffffu, len, k), p.window, p.n_sink);
      const int sk = __shfl_sync(0xffffffffu, seq, k);
      if (v.L <= 0) continue;
      if (nruns == 0 || sk != r.seq) {
        if (nruns) close();
        ++nruns;
        r = Q4Run{sk, 0, 0, v.w0, v.ns, v.L};
      } else {
        r.base = min(r.base, v.w0);
        r.ns = max(r.ns, v.ns);
        r.end = max(r.end, v.L);
      }
      if (k == prow) prun = nruns - 1;
    }
    if (nruns) close();
    if (lane == 0) runs[nruns].tiles0 = n;
  }
  const Visible vis(__shfl_sync(0xffffffffu, len, prow), p.window, p.n_sink);
  // p.chunk tiles a chunk, more where the rows of a group see so different positions that the
  // grid's chunks would not reach
  const int per = max(p.chunk, (n + p.n_split - 1) / p.n_split);
  const int nchunks = (n + per - 1) / per;
  if (c >= nchunks) {
    if (c == 0)  // nothing to see: zeros
      for (int i = threadIdx.x; i < np * D; i += blockDim.x)
        p.out[((size_t)(t0 + i / (G * D)) * p.n_heads + head0) * D + i % (G * D)] = 0.f;
    return;
  }
  const int i0 = c * per + warp, i1 = min((c + 1) * per, n);

  uint8_t* ring = smem + warp * C::NST * C::STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF) + warp * C::NST;
  __syncwarp();  // the run table
  Q4Walk<C::TP> ahead, walk;
  ahead.start(runs);
  walk.start(runs);
  auto issue = [&](int i, int st) {  // tile i's four runs of bytes into stage st (lane 0 copies)
    int start, end;
    ahead.tile(runs, i, start, end);
    if (lane) return;
    const int m = min(C::TP, (end - start + 15) & ~15);  // cache_cap is a multiple of 16
    const size_t row = ((size_t)ahead.r.seq * p.n_kv_heads + kvh) * p.cache_cap + start;
    uint8_t* dst = ring + st * C::STAGE;
    mbar_arrive_expect_tx(&full[st], 2 * m * (C::RB + C::SB));
    bulk_load(dst, static_cast<const uint8_t*>(p.kc) + row * C::RB, m * C::RB, &full[st]);
    bulk_load(dst + C::TP * C::RB, static_cast<const uint8_t*>(p.vc) + row * C::RB, m * C::RB,
              &full[st]);
    dst += 2 * C::TP * C::RB;
    bulk_load(dst, reinterpret_cast<const uint8_t*>(p.ksc) + row * C::SB, m * C::SB, &full[st]);
    bulk_load(dst + C::TP * C::SB, reinterpret_cast<const uint8_t*>(p.vsc) + row * C::SB,
              m * C::SB, &full[st]);
  };
  if (lane == 0) {
    for (int st = 0; st < C::NST; ++st) mbar_init(&full[st], 1);
    mbar_init_fence();
  }
  __syncwarp();  // the barriers, before any lane waits on one
  int issued = 0;  // the warp's tiles asked for so far
  for (int i = i0; issued < C::NST0 && i < i1; i += C::NW, ++issued) issue(i, issued);

  // ---- q's A fragments: the pair's row scaled by a power of two to [1, 2) as f16 hi + lo; sm
  //      takes the power, the softmax scale and the cache's scale of K back in.  Each warp makes
  //      those of its quarter of the k-steps.
  uint4* qf = reinterpret_cast<uint4*>(smem + C::QF_OFF) + lane;
  float sm;
  {
    constexpr int KW = C::KS / C::NW;
    const bool hv = gid < np;
    const float* qrow = p.q + ((size_t)(t0 + prow) * p.n_heads + head0 + (hv ? gid % G : 0)) * D;
    float4 x[KW];
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < KW; ++e) {
      const int ks = warp * KW + e, w = ks / 2;  // word of the thread's run of codes, half of it
      const int d = (w / 4) * 128 + (D == 64 ? 16 : 32) * tig + 8 * (w % 4) + 4 * (ks & 1);
      x[e] = hv ? __ldg(reinterpret_cast<const float4*>(qrow + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
      amax = fmaxf(amax, fmaxf(fmaxf(fabsf(x[e].x), fabsf(x[e].y)),
                               fmaxf(fabsf(x[e].z), fabsf(x[e].w))));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    if (tig == 0) s_amax[warp][gid] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < C::NW; ++w) amax = fmaxf(amax, s_amax[w][gid]);
    const uint32_t e2 = min(max(__float_as_uint(amax) >> 23, 1u), 253u);
    const float f = __uint_as_float((254u - e2) << 23);  // 2^(127 - e2)
    sm = p.scale_log2 * qp.k_scale * __uint_as_float(e2 << 23);
#pragma unroll
    for (int e = 0; e < KW; ++e) {
      uint32_t a[4];
      split_hi_lo(x[e].x * f, x[e].y * f, a[0], a[1]);
      split_hi_lo(x[e].z * f, x[e].w * f, a[2], a[3]);
      qf[(warp * KW + e) * 32] = make_uint4(a[0], a[1], a[2], a[3]);
    }
  }
  __syncthreads();
  uint32_t qa[C::QSMEM ? 1 : C::KS][4];
  if constexpr (!C::QSMEM) {
#pragma unroll
    for (int ks = 0; ks < C::KS; ++ks) {
      const uint4 a4 = qf[ks * 32];
      qa[ks][0] = a4.x;
      qa[ks][1] = a4.y;
      qa[ks][2] = a4.z;
      qa[ks][3] = a4.w;
    }
    fence_async_smem();  // the copy below follows these accesses
    __syncthreads();
    const int i = i0 + C::NST0 * C::NW;
    if (i < i1) issue(i, issued++);
  }

  float o[C::NT][4];
#pragma unroll
  for (int n = 0; n < C::NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  float m_run = -INFINITY, l_run = 0.f;  // pair gid; l_run over this thread's positions
  // this thread's rows of a 16-position block: K columns of both n-tiles, V positions
  const int krow = 4 * (gid & 1) + ((gid >> 1) ^ (3 * (gid & 1)));
  int done = 0;
  bool ok = true;
  for (int i = i0; i < i1; i += C::NW, ++done) {
    const int st = done % C::NST;
    ok = __all_sync(0xffffffffu, mbar_wait(&full[st], (done / C::NST) & 1));
    if (!ok) break;
    const uint8_t* stage = ring + st * C::STAGE;
    // rows of the tile that the pair sees: [lo, hi) and [0, ns); a pad pair takes any
    int start, end;
    walk.tile(runs, i, start, end);
    int hi = gid >= np ? C::TP : walk.k == prun ? min(vis.L, end) - start : 0;
    int lo = gid >= np ? 0 : vis.w0 - start, ns = vis.ns - start;
    const bool whole = __all_sync(0xffffffffu, hi >= C::TP && (lo <= 0 || ns >= C::TP));
#pragma unroll 1
    for (int r0 = 0; r0 < C::TP && start + r0 < end; r0 += C::SP, hi -= C::SP, lo -= C::SP, ns -= C::SP) {
    const uint8_t* sk = stage + r0 * C::RB;
    const uint8_t* sv = sk + C::TP * C::RB;
    const uint8_t* ssk = stage + 2 * C::TP * C::RB + r0 * C::SB;
    const uint8_t* ssv = ssk + C::TP * C::SB;
    // -- S = Q . K^T of 32 positions, four n-tiles
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
    // -- pair gid's scores at positions 8 nt + 4 j + (tig ^ 3 j)
    float x[C::NTK][2];
    float mt = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < C::NTK; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) x[nt][j] = (sc[nt][j] + sc[nt][2 + j]) * sm;
    if (!whole) {
#pragma unroll
      for (int nt = 0; nt < C::NTK; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = 8 * nt + 4 * j + (tig ^ (3 * j));
          if (r >= hi || (r < lo && r >= ns)) x[nt][j] = -INFINITY;
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
    }
    __syncwarp();  // every lane has read the stage
    const int nxt = i + C::NST * C::NW;
    if (nxt < i1) {
      issue(nxt, st);
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
  for (int n2 = 0; n2 < C::NT; ++n2) {
    mrow[2 * tig * (D / 8) + n2] = o[n2][0] + o[n2][2];
    mrow[(2 * tig + 1) * (D / 8) + n2] = o[n2][1] + o[n2][3];
  }
  if (tig == 0) {
    mrow[D] = m_run;
    mrow[D + 1] = l_run;
  }
  __shared__ float s_w[C::NW][8], s_m[8], s_l[8];  // the warps' weights; the pair's maximum, sum
  __syncthreads();
  if (threadIdx.x < 8) {
    const int h = threadIdx.x;
    float M = -INFINITY, Ls = 0.f;
#pragma unroll
    for (int w = 0; w < C::NW; ++w) M = fmaxf(M, mg[(w * 8 + h) * (D + 2) + D]);
#pragma unroll
    for (int w = 0; w < C::NW; ++w) {
      const float* r = mg + (w * 8 + h) * (D + 2);
      const float e = r[D] == -INFINITY ? 0.f : fast_exp2(r[D] - M);
      s_w[w][h] = e * qp.v_scale;
      Ls = fmaf(r[D + 1], e, Ls);
    }
    s_m[h] = M == -INFINITY ? -INFINITY : M * kLn2;  // natural-log units
    s_l[h] = Ls;
  }
  __syncthreads();
  const bool split = nchunks > 1;
  const size_t rec = (size_t)p.n_heads * (D + 2);  // floats between a pair's chunks
  for (int h = warp; h < np; h += C::NW) {         // a warp a pair
    const int row = h / G, t = t0 + row, head = head0 + h - row * G;
    const float inv = s_l[h] > 0.f ? 1.f / s_l[h] : 0.f;
    float* dst = split ? p.part + ((size_t)t * p.n_split + c) * rec + (size_t)head * (D + 2)
                       : p.out + ((size_t)t * p.n_heads + head) * D;
    float e[C::NW];
#pragma unroll
    for (int w = 0; w < C::NW; ++w) e[w] = s_w[w][h] * (split ? 1.f : inv);
#pragma unroll
    for (int d = 2 * lane; d < D; d += 64) {
      float2 a = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < C::NW; ++w) {
        const float2 x = *reinterpret_cast<const float2*>(mg + (w * 8 + h) * (D + 2) + d);
        a.x = fmaf(x.x, e[w], a.x);
        a.y = fmaf(x.y, e[w], a.y);
      }
      if (!split) a = make_float2(gated(p, t, head, d, a.x), gated(p, t, head, d + 1, a.y));
      *reinterpret_cast<float2*>(dst + d) = a;
    }
    if (split && lane == 0) *reinterpret_cast<float2*>(dst + D) = make_float2(s_m[h], s_l[h]);
  }
  if (!split) return;

  // ---- the group's last CTA (a ticket; nobody waits) merges its chunks by log-sum-exp: a warp
  //      finds a pair's weights, then the threads fold the chunks' records, 16 loads in flight
  __shared__ int s_last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0)
    s_last = atomicInc(p.counters + (size_t)blockIdx.z * gridDim.y + blockIdx.y,
                       (unsigned)(nchunks - 1)) == (unsigned)(nchunks - 1);
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  float* wt = reinterpret_cast<float*>(smem);  // [8][nchunks]
  for (int h = warp; h < np; h += C::NW) {
    const int row = h / G;
    const float* src =
        p.part + (size_t)(t0 + row) * p.n_split * rec + (size_t)(head0 + h - row * G) * (D + 2);
    float M = -INFINITY, Ls = 0.f;
    for (int cc = lane; cc < nchunks; cc += 32) {
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(src + (size_t)cc * rec + D));
      const float mn = fmaxf(M, ml.x);
      if (mn != -INFINITY) Ls = Ls * __expf(M - mn) + ml.y * __expf(ml.x - mn);
      M = mn;
      wt[h * nchunks + cc] = ml.x;
    }
    const float Mw = warp_max(M);
    Ls = warp_sum(M == -INFINITY ? 0.f : Ls * __expf(M - Mw));
    const float inv = Ls > 0.f ? 1.f / Ls : 0.f;
    for (int cc = lane; cc < nchunks; cc += 32) {
      const float m = wt[h * nchunks + cc];
      wt[h * nchunks + cc] = m == -INFINITY ? 0.f : __expf(m - Mw) * inv;
    }
  }
  __syncthreads();
  constexpr int TPP = D / 2;  // threads of a pair, two dims each
  static_assert((32 * C::NW) % TPP == 0, "whole pairs a pass");
  const int d = 2 * (threadIdx.x % TPP);
  for (int h = threadIdx.x / TPP; h < np; h += 32 * C::NW / TPP) {
    const int row = h / G, t = t0 + row, head = head0 + h - row * G;
    const float* src = p.part + (size_t)t * p.n_split * rec + (size_t)head * (D + 2) + d;
    const float* e = wt + h * nchunks;
    float2 a = make_float2(0.f, 0.f);
    for (int cc = 0; cc < nchunks; cc += 16) {
      float2 v[16];
#pragma unroll
      for (int k = 0; k < 16; ++k)  // past the last chunk: the last one again, weight 0
        v[k] = __ldcg(reinterpret_cast<const float2*>(src + (size_t)min(cc + k, nchunks - 1) * rec));
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float w = cc + k < nchunks ? e[cc + k] : 0.f;
        a.x = fmaf(v[k].x, w, a.x);
        a.y = fmaf(v[k].y, w, a.y);
      }
    }
    *reinterpret_cast<float2*>(p.out + ((size_t)t * p.n_heads + head) * D + d) =
        make_float2(gated(p, t, head, d, a.x), gated(p, t, head, d + 1, a.y));
  }
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
