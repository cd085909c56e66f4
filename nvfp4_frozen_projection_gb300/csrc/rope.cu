// Norms of queries and keys for each head with the rotary position embedding in the same
// pass, and their backward.  For one head x [D] of a token at position pos:
//
//   n = x rstd, rstd = 1 / sqrt(mean(x^2) + eps);  z = n gamma  (z = x without norms);
//   y = R z: the pairs (z_i, z_{i + rot/2}), or (z_2i, z_{2i+1}), of the first `rot` columns
//   turn by the angle pos inv_freq_i, the columns behind them stay.
//   backward: g = R^T dy;  dgamma = sum g n;  dn = g gamma;
//             dx = rstd (dn - n mean(dn n))   (dx = g without norms).
//
// Angles are kept in turns as 64-bit fractions: turns_i = inv_freq_i / (2 pi) 2^64, and
// pos turns_i mod 2^64 is the exact fraction of a turn, however far the position.  Its upper
// 32 bits, as FP32, go to sincospif.
//
// Both directions are bound by HBM: 4 bytes a value forward, 6 backward (4 without norms).
// A block works for the queries or for the keys.  A group of 8, 16 or 32 of its lanes holds a
// head and takes heads of one token in turn, so that a lane computes the sines of its columns
// once for all of them.  A lane has both halves of four pairs, 8 columns: four angles, and
// nothing to exchange but the sums over a head.  With few tokens the heads of a token are
// shared out over more groups.  8192 x 40 x 128 with norms: 31 us, 5.4 TB/s; backward 26624 x
// 40 x 64 without norms: 45 us, 6.0 TB/s, with them 69, 5.9, with both dgammas 80, 5.1: a second
// launch, 6 us, and the sums.  The loads in flight are those that a thread's registers hold,
// since the values go straight to them.  (A tile of tokens with its angles in shared memory and
// neighbouring groups on neighbouring heads: 45 us forward, 107 backward.)
#include "common.cuh"
#include "kernels.h"

namespace pact {

constexpr int kRopeThreads = 256;
constexpr int kRopeBlocks = 4;     // an SM: 64 registers a thread
// The backward holds eight heads of two tensors a thread instead: 26624 x 40 x 64 80 us with
// two blocks, against 89 with four heads, 110 with two heads and four blocks.
constexpr int kRopeBwdBlocks = 2;
constexpr int kRopeBwdMost = 16;   // an SM, in all

// A lane's 8 columns as two vectors of four, u and v: the halves of four pairs, or (behind the
// turned columns) neighbours that stay.  Pairs of halves: u from column a on, v from column b
// on; neighbouring pairs (PAIRS): the even and the odd ones of 8 columns from a on.
struct Cols {
  int a, b;
  bool turned;
};
template <bool PAIRS>
__device__ __forceinline__ Cols lane_cols(int sl, int rot) {
  Cols c;
  c.turned = sl * 8 < rot;
  c.a = PAIRS || !c.turned ? sl * 8 : sl * 4;
  c.b = PAIRS || !c.turned ? c.a + 4 : (rot >> 1) + c.a;
  return c;
}

struct Vec {
  float2 u[2], v[2];
};
template <bool PAIRS>
__device__ __forceinline__ uint4 load_cols(const uint16_t* row, const Cols& c) {
  if constexpr (PAIRS) return *reinterpret_cast<const uint4*>(row + c.a);
  const uint2 lo = *reinterpret_cast<const uint2*>(row + c.a);
  const uint2 hi = *reinterpret_cast<const uint2*>(row + c.b);
  return make_uint4(lo.x, lo.y, hi.x, hi.y);
}
__device__ __forceinline__ float2 bf16x2_f2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <bool PAIRS>
__device__ __forceinline__ Vec unpack(const uint4& w) {
  const float2 a = bf16x2_f2(w.x), b = bf16x2_f2(w.y), c = bf16x2_f2(w.z), d = bf16x2_f2(w.w);
  Vec r;
  if constexpr (PAIRS) {
    r.u[0] = make_float2(a.x, b.x);
    r.u[1] = make_float2(c.x, d.x);
    r.v[0] = make_float2(a.y, b.y);
    r.v[1] = make_float2(c.y, d.y);
  } else {
    r.u[0] = a;
    r.u[1] = b;
    r.v[0] = c;
    r.v[1] = d;
  }
  return r;
}
template <bool PAIRS>
__device__ __forceinline__ void store_cols(uint16_t* row, const Cols& c, const Vec& r) {
  if constexpr (PAIRS) {
    *reinterpret_cast<uint4*>(row + c.a) =
        make_uint4(pack_bf16x2(r.u[0].x, r.v[0].x), pack_bf16x2(r.u[0].y, r.v[0].y),
                   pack_bf16x2(r.u[1].x, r.v[1].x), pack_bf16x2(r.u[1].y, r.v[1].y));
  } else {
    *reinterpret_cast<uint2*>(row + c.a) =
        make_uint2(pack_bf16x2(r.u[0].x, r.u[0].y), pack_bf16x2(r.u[1].x, r.u[1].y));
    *reinterpret_cast<uint2*>(row + c.b) =
        make_uint2(pack_bf16x2(r.v[0].x, r.v[0].y), pack_bf16x2(r.v[1].x, r.v[1].y));
  }
}

// Cosines and sines of the lane's four pairs.
struct Turn {
  float2 c[2], s[2];
};
template <bool PAIRS>
__device__ __forceinline__ Turn make_turn(const Cols& cols, bool live, int pos,
                                          const int64_t* turns) {
  float c[4] = {1.0f, 1.0f, 1.0f, 1.0f}, s[4] = {};
  if (live && cols.turned) {
    const int i0 = PAIRS ? cols.a >> 1 : cols.a;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint64_t phase = (uint64_t)(int64_t)pos * (uint64_t)turns[i0 + e];
      sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s[e], &c[e]);
    }
  }
  Turn t;
  t.c[0] = make_float2(c[0], c[1]);
  t.c[1] = make_float2(c[2], c[3]);
  t.s[0] = make_float2(s[0], s[1]);
  t.s[1] = make_float2(s[2], s[3]);
  return t;
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 neg(float2 v) { return make_float2(-v.x, -v.y); }

template <int SEG>
__device__ __forceinline__ float seg_sum(float v) {
#pragma unroll
  for (int o = SEG / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// 1 / sqrt(mean + eps); rsqrtf is within 2 units in the last place.
__device__ __forceinline__ float rstd_of(float ss, float inv_d, float eps) {
  return rsqrtf(__fmaf_rn(ss, inv_d, eps));
}

template <int SEG, bool NORM, bool PAIRS>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks) k_qk_norm_rope(const RopeParams p) {
  constexpr int U = 4;  // heads in flight
  const bool isk = (int)blockIdx.x >= p.side[0].blocks;
  const RopeSide& sd = p.side[isk];
  const int sl = threadIdx.x & (SEG - 1);
  const int64_t seg = (int64_t)(blockIdx.x - (isk ? p.side[0].blocks : 0)) * (kRopeThreads / SEG) +
                      threadIdx.x / SEG;
  // a dead group stays for the shuffles of its warp, with no heads
  const bool alive = seg < sd.segs;
  const int64_t t = alive ? seg / sd.chunks : 0;
  const int h0 = alive ? (int)(seg - t * sd.chunks) * sd.per : 0;
  const int heads = alive && sl * 8 < p.D && PACT_IN(t < p.T) ? min(sd.per, sd.heads - h0) : 0;
  const Cols cols = lane_cols<PAIRS>(sl, p.rot);
  const uint16_t* x = sd.x + t * sd.ld + (int64_t)h0 * p.D;
  uint16_t* out = sd.out + t * sd.ldo + (int64_t)h0 * p.D;
  uint4 w[U];
  auto load = [&](int hb) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      w[i] = make_uint4(0, 0, 0, 0);
      if (hb + i < heads) w[i] = load_cols<PAIRS>(x + (hb + i) * p.D, cols);
    }
  };
  load(0);  // on their way while the angles are computed
  const Turn tn = make_turn<PAIRS>(cols, heads > 0, p.positions[t], p.turns);
  const float inv_d = 1.0f / (float)p.D;
  // u' = u uc - v vs, v' = v vc + u us: the gammas go into the coefficients
  float2 uc[2], us[2], vc[2], vs[2];
  Vec g;
  g.u[0] = g.u[1] = g.v[0] = g.v[1] = both(1.0f);
  if (NORM && heads > 0) g = unpack<PAIRS>(load_cols<PAIRS>(sd.gamma, cols));
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    uc[e] = __fmul2_rn(tn.c[e], g.u[e]);
    us[e] = __fmul2_rn(tn.s[e], g.u[e]);
    vc[e] = __fmul2_rn(tn.c[e], g.v[e]);
    vs[e] = __fmul2_rn(neg(tn.s[e]), g.v[e]);
  }
  for (int hb = 0; hb < sd.per; hb += U) {
    if (hb > 0) load(hb);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (hb + i >= sd.per) break;  // for the whole block
      const Vec f = unpack<PAIRS>(w[i]);
      Vec o;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        o.u[e] = __ffma2_rn(f.u[e], uc[e], __fmul2_rn(f.v[e], vs[e]));
        o.v[e] = __ffma2_rn(f.v[e], vc[e], __fmul2_rn(f.u[e], us[e]));
      }
      if constexpr (NORM) {
        float2 q = __fmul2_rn(f.u[0], f.u[0]);
        q = __ffma2_rn(f.u[1], f.u[1], q);
        q = __ffma2_rn(f.v[0], f.v[0], q);
        q = __ffma2_rn(f.v[1], f.v[1], q);
        const float2 r = both(rstd_of(seg_sum<SEG>(q.x + q.y), inv_d, p.eps));
#pragma unroll
        for (int e = 0; e < 2; ++e) o.u[e] = __fmul2_rn(o.u[e], r), o.v[e] = __fmul2_rn(o.v[e], r);
      }
      if (hb + i < heads) store_cols<PAIRS>(out + (hb + i) * p.D, cols, o);
    }
  }
}

// Backward; a side's x is dy, xf the forward's input (NORM).  DG: the sum for dgamma of this
// block's groups goes to part[block][D], group by group in order.
template <int SEG, bool NORM, bool PAIRS, bool DG>
__global__ void __launch_bounds__(kRopeThreads, kRopeBwdBlocks)
    k_qk_norm_rope_bwd(const RopeParams p, float* part) {
  constexpr int U = 8;  // heads in flight
  constexpr int GROUPS = kRopeThreads / SEG;
  __shared__ float sums[DG ? GROUPS * 8 * SEG : 1];
  const bool isk = (int)blockIdx.x >= p.side[0].blocks;
  const RopeSide& sd = p.side[isk];
  const int block = (int)blockIdx.x - (isk ? p.side[0].blocks : 0);
  const int sl = threadIdx.x & (SEG - 1), group = threadIdx.x / SEG;
  const float inv_d = 1.0f / (float)p.D;
  const Cols cols = lane_cols<PAIRS>(sl, p.rot);
  Vec gm, acc;
#pragma unroll
  for (int e = 0; e < 2; ++e) gm.u[e] = gm.v[e] = acc.u[e] = acc.v[e] = both(0.0f);
  if (NORM && sl * 8 < p.D) gm = unpack<PAIRS>(load_cols<PAIRS>(sd.gamma, cols));
  for (int64_t first = (int64_t)block * GROUPS; first < sd.segs;
       first += (int64_t)sd.blocks * GROUPS) {
    const int64_t seg = first + group;
    const bool alive = seg < sd.segs;
    const int64_t t = alive ? seg / sd.chunks : 0;
    const int h0 = alive ? (int)(seg - t * sd.chunks) * sd.per : 0;
    const int heads = alive && sl * 8 < p.D && PACT_IN(t < p.T) ? min(sd.per, sd.heads - h0) : 0;
    const uint16_t* dy = sd.x + t * sd.ld + (int64_t)h0 * p.D;
    const uint16_t* x = NORM ? sd.xf + t * sd.ldxf + (int64_t)h0 * p.D : nullptr;
    uint16_t* out = sd.out + t * sd.ldo + (int64_t)h0 * p.D;
    uint4 wy[U], wx[U];
    auto load = [&](int hb) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        wy[i] = wx[i] = make_uint4(0, 0, 0, 0);
        if (hb + i < heads) {
          wy[i] = load_cols<PAIRS>(dy + (hb + i) * p.D, cols);
          if constexpr (NORM) wx[i] = load_cols<PAIRS>(x + (hb + i) * p.D, cols);
        }
      }
    };
    load(0);  // on their way while the angles are computed
    const Turn tn = make_turn<PAIRS>(cols, heads > 0, p.positions[t], p.turns);
    for (int hb = 0; hb < sd.per; hb += U) {
      if (hb > 0) load(hb);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (hb + i >= sd.per) break;  // for the whole block
        const Vec f = unpack<PAIRS>(wy[i]);
        Vec g;  // turned back
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          g.u[e] = __ffma2_rn(f.u[e], tn.c[e], __fmul2_rn(f.v[e], tn.s[e]));
          g.v[e] = __ffma2_rn(f.v[e], tn.c[e], __fmul2_rn(neg(f.u[e]), tn.s[e]));
        }
        if constexpr (NORM) {
          Vec n = unpack<PAIRS>(wx[i]), d;
          float2 ss = both(0.0f), dot = both(0.0f);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            ss = __ffma2_rn(n.u[e], n.u[e], ss);
            ss = __ffma2_rn(n.v[e], n.v[e], ss);
            d.u[e] = __fmul2_rn(g.u[e], gm.u[e]);
            d.v[e] = __fmul2_rn(g.v[e], gm.v[e]);
            dot = __ffma2_rn(d.u[e], n.u[e], dot);
            dot = __ffma2_rn(d.v[e], n.v[e], dot);
          }
          // a head that is not there has no norm: with eps 0 its rstd would be infinite
          const float there = rstd_of(seg_sum<SEG>(ss.x + ss.y), inv_d, p.eps);
          const float rstd = hb + i < heads ? there : 0.0f;
          const float c = seg_sum<SEG>(dot.x + dot.y) * rstd * inv_d;  // mean(dn n)
          const float2 r = both(rstd), mc = both(-c);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            n.u[e] = __fmul2_rn(n.u[e], r);
            n.v[e] = __fmul2_rn(n.v[e], r);
            if constexpr (DG) {  // zero in lanes and heads that hold nothing
              acc.u[e] = __ffma2_rn(g.u[e], n.u[e], acc.u[e]);
              acc.v[e] = __ffma2_rn(g.v[e], n.v[e], acc.v[e]);
            }
            g.u[e] = __fmul2_rn(r, __ffma2_rn(n.u[e], mc, d.u[e]));
            g.v[e] = __fmul2_rn(r, __ffma2_rn(n.v[e], mc, d.v[e]));
          }
        }
        if (hb + i < heads) store_cols<PAIRS>(out + (hb + i) * p.D, cols, g);
      }
    }
  }
  if constexpr (DG) {
    if (sl * 8 < p.D) {
      const float u[4] = {acc.u[0].x, acc.u[0].y, acc.u[1].x, acc.u[1].y};
      const float v[4] = {acc.v[0].x, acc.v[0].y, acc.v[1].x, acc.v[1].y};
      float* row = sums + group * (8 * SEG);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        row[PAIRS ? cols.a + 2 * e : cols.a + e] = u[e];
        row[PAIRS ? cols.a + 2 * e + 1 : cols.b + e] = v[e];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.D; c += kRopeThreads) {
      float s = 0.0f;
      for (int g = 0; g < GROUPS; ++g) s += sums[g * (8 * SEG) + c];
      if (PACT_IN(c < p.D)) part[(int64_t)blockIdx.x * p.D + c] = s;
    }
  }
}

// dgamma_q, dgamma_k [D] from the blocks' sums, those of the queries first.  Four columns a
// block (D is a multiple of 16), 256 threads each, so that a thread's few rows are all on
// their way at once; joined by butterflies and in order.  The joined sums have an
// array of their own: a warp that is ahead must not store over rows that another has yet to
// read.
__global__ void __launch_bounds__(1024)
    k_qk_dgamma(const float* part, int bq, int bk, int D, float* dgq, float* dgk) {
  __shared__ float sums[32][4], joined[4][4];
  const int x = threadIdx.x & 3, y = threadIdx.x >> 2;
  const bool isk = (int)blockIdx.x * 4 >= D;
  const int c = (int)blockIdx.x * 4 + x - (isk ? D : 0);
  const float* from = part + (isk ? (int64_t)bq * D : 0) + c;
  const int rows = isk ? bk : bq;
  float s = 0.0f;
#pragma unroll 8
  for (int b = y; b < rows; b += 256) s += from[(int64_t)b * D];
  auto eight = [](float v) {  // over the eight rows of a warp
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
  };
  s = eight(s);
  if ((threadIdx.x & 31) < 4) sums[threadIdx.x >> 5][x] = s;
  __syncthreads();
  if (threadIdx.x < 128) {
    s = eight(sums[y][x]);
    if ((threadIdx.x & 31) < 4) joined[threadIdx.x >> 5][x] = s;
  }
  __syncthreads();
  if (threadIdx.x < 4 && PACT_IN(c < D))
    (isk ? dgk : dgq)[c] = (joined[0][x] + joined[1][x]) + (joined[2][x] + joined[3][x]);
}

__global__ void k_rope_turns(const double* inv_freq, int n, int64_t* turns) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  double f = inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi): radians to turns
  f -= floor(f);
  // 2^64 f, the lower half separately: f may be just below one
  const double hi = floor(f * 4294967296.0);
  const double lo = (f * 4294967296.0 - hi) * 4294967296.0;
  if (PACT_IN(i < n)) turns[i] = (int64_t)(((uint64_t)hi << 32) + (uint64_t)lo);
}

static int seg_lanes(int D) { return D <= 64 ? 8 : (D <= 128 ? 16 : 32); }

// Heads a group takes: all of a token's, or fewer where that leaves threads idle.  Blocks:
// one for its groups, but (most > 0) no more than `most` for both sides, shared by heads.
static void rope_plan(RopeParams& p, int num_sms, int most) {
  const int seg = seg_lanes(p.D), gs = kRopeThreads / seg;
  const int heads = p.side[0].heads + p.side[1].heads;
  const int64_t groups = (int64_t)num_sms * kRopeBlocks * gs;
  const int64_t per = (p.T * heads + groups - 1) / groups;
  int64_t want[2];
  for (int w = 0; w < 2; ++w) {
    RopeSide& s = p.side[w];
    const int64_t at_most = per < s.heads ? per : s.heads;
    s.chunks = (int)((s.heads + at_most - 1) / at_most);
    s.per = (s.heads + s.chunks - 1) / s.chunks;
    s.chunks = (s.heads + s.per - 1) / s.per;
    s.segs = p.T * s.chunks;
    want[w] = (s.segs + gs - 1) / gs;
  }
  if (most > 0 && want[0] + want[1] > most) {
    const int64_t k = (int64_t)most * p.side[1].heads / heads;
    const int64_t bk = k < 1 ? 1 : k;
    want[1] = want[1] < bk ? want[1] : bk;
    want[0] = want[0] < most - want[1] ? want[0] : most - want[1];
  }
  p.side[0].blocks = (int)want[0];
  p.side[1].blocks = (int)want[1];
}

template <int SEG>
static void launch_fwd(const RopeParams& p, bool norm, bool pairs, cudaStream_t st) {
  const unsigned grid = (unsigned)(p.side[0].blocks + p.side[1].blocks);
  if (norm && pairs)
    k_qk_norm_rope<SEG, true, true><<<grid, kRopeThreads, 0, st>>>(p);
  else if (norm)
    k_qk_norm_rope<SEG, true, false><<<grid, kRopeThreads, 0, st>>>(p);
  else if (pairs)
    k_qk_norm_rope<SEG, false, true><<<grid, kRopeThreads, 0, st>>>(p);
  else
    k_qk_norm_rope<SEG, false, false><<<grid, kRopeThreads, 0, st>>>(p);
}

cudaError_t launch_qk_norm_rope(RopeParams& p, int pairs, int num_sms, cudaStream_t st) {
  const int seg = seg_lanes(p.D);
  rope_plan(p, num_sms, 0);
  const bool norm = p.side[0].gamma != nullptr;
  note_launch();
  if (seg == 8)
    launch_fwd<8>(p, norm, pairs, st);
  else if (seg == 16)
    launch_fwd<16>(p, norm, pairs, st);
  else
    launch_fwd<32>(p, norm, pairs, st);
  return cudaGetLastError();
}

// Blocks of the backward: a few waves, which leave less of the last one empty than one of
// blocks that go on would, and not so many that the sums for dgamma weigh.
int64_t rope_bwd_blocks(int64_t T, int hq, int hk, int D, int num_sms) {
  RopeParams p = {};
  p.T = T;
  p.D = D;
  p.side[0].heads = hq;
  p.side[1].heads = hk;
  rope_plan(p, num_sms, kRopeBwdMost * num_sms);
  return (int64_t)p.side[0].blocks + p.side[1].blocks;
}

template <int SEG>
static void launch_bwd(const RopeParams& p, bool norm, bool pairs, bool dg, float* part,
                       cudaStream_t st) {
  const unsigned grid = (unsigned)(p.side[0].blocks + p.side[1].blocks);
#define PACT_ROPE_BWD(N, P, G) k_qk_norm_rope_bwd<SEG, N, P, G><<<grid, kRopeThreads, 0, st>>>(p, part)
  if (!norm && pairs)
    PACT_ROPE_BWD(false, true, false);
  else if (!norm)
    PACT_ROPE_BWD(false, false, false);
  else if (pairs && dg)
    PACT_ROPE_BWD(true, true, true);
  else if (pairs)
    PACT_ROPE_BWD(true, true, false);
  else if (dg)
    PACT_ROPE_BWD(true, false, true);
  else
    PACT_ROPE_BWD(true, false, false);
#undef PACT_ROPE_BWD
}

cudaError_t launch_qk_norm_rope_bwd(RopeParams& p, int pairs, float* dgq, float* dgk, float* part,
                                    int num_sms, cudaStream_t st) {
  const int seg = seg_lanes(p.D);
  rope_plan(p, num_sms, kRopeBwdMost * num_sms);
  const bool norm = p.side[0].gamma != nullptr, dg = dgq != nullptr;
  note_launch();
  if (seg == 8)
    launch_bwd<8>(p, norm, pairs, dg, part, st);
  else if (seg == 16)
    launch_bwd<16>(p, norm, pairs, dg, part, st);
  else
    launch_bwd<32>(p, norm, pairs, dg, part, st);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !dg) return e;
  note_launch();
  k_qk_dgamma<<<2 * p.D / 4, 1024, 0, st>>>(part, p.side[0].blocks, p.side[1].blocks, p.D, dgq,
                                                 dgk);
  return cudaGetLastError();
}

cudaError_t launch_rope_turns(const double* inv_freq, int n, int64_t* turns, cudaStream_t st) {
  note_launch();
  k_rope_turns<<<(n + 127) / 128, 128, 0, st>>>(inv_freq, n, turns);
  return cudaGetLastError();
}

}  // namespace pact
