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
// head, 8 values (16 bytes) a lane, and takes heads of one token in turn, so that a lane
// computes the sines of its columns once for all of them; a pair's other half comes from the
// lane that holds it as packed BF16.  With few tokens the heads of a token are shared out
// over more groups.
#include "common.cuh"
#include "kernels.h"

namespace pact {

constexpr int kRopeThreads = 256;
constexpr int kRopeBlocks = 4;     // an SM: 64 registers a thread
constexpr int kRopeBwdBlocks = 3;  // 80
constexpr int kRopeBwdMost = 16;   // an SM, in all

// The rotation of one lane's 8 columns, two at a time: y = own c + other s.  The other half
// of a pair comes from the lane `other`, or (PAIRS) is the neighbouring column.
struct Turn {
  float2 c[4], s[4];
  int other;    // lane offset of the other half
  bool turned;  // the lane's columns lie in the first rot
};

template <bool PAIRS>
__device__ __forceinline__ Turn make_turn(int col, int rot, int pos, const int64_t* turns,
                                          bool back) {
  Turn t;
  t.turned = col < rot;
  t.other = 0;
  if (!t.turned) {
#pragma unroll
    for (int e = 0; e < 4; ++e) t.c[e] = make_float2(1.0f, 1.0f), t.s[e] = make_float2(0.0f, 0.0f);
    return t;
  }
  const int half = rot >> 1;
  const bool first = PAIRS || col < half;
  if (!PAIRS) t.other = first ? (half >> 3) : -(half >> 3);
  const int i0 = PAIRS ? col >> 1 : (first ? col : col - half);
  float c[8], s[8];
#pragma unroll
  for (int e = 0; e < (PAIRS ? 4 : 8); ++e) {
    const uint64_t phase = (uint64_t)(int64_t)pos * (uint64_t)turns[i0 + e];
    sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s[e], &c[e]);
    // of a pair (a, b): a' = a c - b s, b' = b c + a s; backward the other way round
    if (first != back) s[e] = -s[e];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    t.c[e] = PAIRS ? make_float2(c[e], c[e]) : make_float2(c[2 * e], c[2 * e + 1]);
    t.s[e] = PAIRS ? make_float2(s[e], -s[e]) : make_float2(s[2 * e], s[2 * e + 1]);
  }
  return t;
}

__device__ __forceinline__ void unpack8(const uint4& v, float2* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    f[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 pack8(const float2* f) {
  return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y),
                    pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y));
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 swapped(float2 v) { return make_float2(v.y, v.x); }

template <int SEG>
__device__ __forceinline__ float seg_sum(float v) {
#pragma unroll
  for (int o = SEG / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// The lanes' other halves of a pair, as packed BF16.
__device__ __forceinline__ uint4 shfl_v4(const uint4& v, int lane) {
  return make_uint4(__shfl_sync(0xFFFFFFFFu, v.x, lane), __shfl_sync(0xFFFFFFFFu, v.y, lane),
                    __shfl_sync(0xFFFFFFFFu, v.z, lane), __shfl_sync(0xFFFFFFFFu, v.w, lane));
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
  const int lane = threadIdx.x & 31, col = (lane & (SEG - 1)) * 8;
  const int64_t seg = (int64_t)(blockIdx.x - (isk ? p.side[0].blocks : 0)) * (kRopeThreads / SEG) +
                      threadIdx.x / SEG;
  // a dead group stays for the shuffles of its warp, with no heads
  const bool alive = seg < sd.segs;
  const int64_t t = alive ? seg / sd.chunks : 0;
  const int h0 = alive ? (int)(seg - t * sd.chunks) * sd.per : 0;
  const int heads = alive && col < p.D && PACT_IN(t < p.T) ? min(sd.per, sd.heads - h0) : 0;
  const Turn tn = make_turn<PAIRS>(heads ? col : p.rot, p.rot, p.positions[t], p.turns, false);
  const int other = lane + tn.other;
  const float inv_d = 1.0f / (float)p.D;
  // the gammas go into the coefficients: y = rstd (own (gamma c) + other (gamma' s))
  float2 c[4], s[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] = tn.c[e], s[e] = tn.s[e];
  if (NORM && heads) {
    float2 g[4], o[4];
    unpack8(*reinterpret_cast<const uint4*>(sd.gamma + col), g);
    if constexpr (PAIRS) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = swapped(g[e]);
    } else {
      unpack8(*reinterpret_cast<const uint4*>(sd.gamma + col + 8 * tn.other), o);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = __fmul2_rn(c[e], g[e]), s[e] = __fmul2_rn(s[e], o[e]);
  }
  const uint16_t* x = sd.x + t * sd.ld + (int64_t)h0 * p.D + col;
  uint16_t* out = sd.out + t * sd.ldo + (int64_t)h0 * p.D + col;
  for (int hb = 0; hb < sd.per; hb += U) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u] = make_uint4(0, 0, 0, 0);
      if (hb + u < heads) v[u] = *reinterpret_cast<const uint4*>(x + (hb + u) * p.D);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 f[4], o[4];
      unpack8(v[u], f);
      if constexpr (PAIRS) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = swapped(f[e]);
      } else {
        unpack8(shfl_v4(v[u], other), o);
      }
      float2 r = both(1.0f);
      if constexpr (NORM) {
        float2 q = both(0.0f);
#pragma unroll
        for (int e = 0; e < 4; ++e) q = __ffma2_rn(f[e], f[e], q);
        r = both(rstd_of(seg_sum<SEG>(q.x + q.y), inv_d, p.eps));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[e] = __ffma2_rn(f[e], c[e], __fmul2_rn(o[e], s[e]));
        if constexpr (NORM) f[e] = __fmul2_rn(f[e], r);
      }
      if (hb + u < heads) *reinterpret_cast<uint4*>(out + (hb + u) * p.D) = pack8(f);
    }
  }
}

// Backward; a side's x is dy, xf the forward's input (NORM).  DG: the sum for dgamma of this
// block's groups goes to part[block][D], group by group in order.
template <int SEG, bool NORM, bool PAIRS, bool DG>
__global__ void __launch_bounds__(kRopeThreads, kRopeBwdBlocks)
    k_qk_norm_rope_bwd(const RopeParams p, float* part) {
  constexpr int U = NORM ? 2 : 4;  // heads in flight
  constexpr int GROUPS = kRopeThreads / SEG;
  __shared__ float sums[DG ? GROUPS * 8 * SEG : 1];
  const bool isk = (int)blockIdx.x >= p.side[0].blocks;
  const RopeSide& sd = p.side[isk];
  const int block = (int)blockIdx.x - (isk ? p.side[0].blocks : 0);
  const int lane = threadIdx.x & 31, col = (lane & (SEG - 1)) * 8, group = threadIdx.x / SEG;
  const float inv_d = 1.0f / (float)p.D;
  float2 acc[DG ? 4 : 1] = {}, gm[4] = {};
  if (NORM && col < p.D) unpack8(*reinterpret_cast<const uint4*>(sd.gamma + col), gm);
  for (int64_t first = (int64_t)block * GROUPS; first < sd.segs;
       first += (int64_t)sd.blocks * GROUPS) {
    const int64_t seg = first + group;
    const bool alive = seg < sd.segs;
    const int64_t t = alive ? seg / sd.chunks : 0;
    const int h0 = alive ? (int)(seg - t * sd.chunks) * sd.per : 0;
    const int heads = alive && col < p.D && PACT_IN(t < p.T) ? min(sd.per, sd.heads - h0) : 0;
    const Turn tn = make_turn<PAIRS>(heads ? col : p.rot, p.rot, p.positions[t], p.turns, true);
    const int other = lane + tn.other;
    const uint16_t* dy = sd.x + t * sd.ld + (int64_t)h0 * p.D + col;
    const uint16_t* x = NORM ? sd.xf + t * sd.ldxf + (int64_t)h0 * p.D + col : nullptr;
    uint16_t* out = sd.out + t * sd.ldo + (int64_t)h0 * p.D + col;
    for (int hb = 0; hb < sd.per; hb += U) {
      uint4 v[U], w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v[u] = w[u] = make_uint4(0, 0, 0, 0);
        if (hb + u < heads) {
          v[u] = *reinterpret_cast<const uint4*>(dy + (hb + u) * p.D);
          if constexpr (NORM) w[u] = *reinterpret_cast<const uint4*>(x + (hb + u) * p.D);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float2 g[4], o[4];
        unpack8(v[u], g);
        if constexpr (PAIRS) {
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = swapped(g[e]);
        } else {
          unpack8(shfl_v4(v[u], other), o);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) g[e] = __ffma2_rn(g[e], tn.c[e], __fmul2_rn(o[e], tn.s[e]));
        if constexpr (NORM) {
          float2 n[4];
          unpack8(w[u], n);
          float2 ss = both(0.0f), dot = both(0.0f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ss = __ffma2_rn(n[e], n[e], ss);
            o[e] = __fmul2_rn(g[e], gm[e]);
            dot = __ffma2_rn(o[e], n[e], dot);
          }
          const float rstd = rstd_of(seg_sum<SEG>(ss.x + ss.y), inv_d, p.eps);
          const float c = seg_sum<SEG>(dot.x + dot.y) * rstd * inv_d;  // mean(dn n)
          const float2 r = both(rstd), mc = both(-c);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            n[e] = __fmul2_rn(n[e], r);
            // zero in lanes and heads that hold nothing
            if constexpr (DG) acc[e] = __ffma2_rn(g[e], n[e], acc[e]);
            g[e] = __fmul2_rn(r, __ffma2_rn(n[e], mc, o[e]));
          }
        }
        if (hb + u < heads) *reinterpret_cast<uint4*>(out + (hb + u) * p.D) = pack8(g);
      }
    }
  }
  if constexpr (DG) {
    if (col < p.D) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<float2*>(sums + group * (8 * SEG) + col + 2 * e) = acc[e];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.D; c += kRopeThreads) {
      float s = 0.0f;
      for (int g = 0; g < GROUPS; ++g) s += sums[g * (8 * SEG) + c];
      if (PACT_IN(c < p.D)) part[(int64_t)blockIdx.x * p.D + c] = s;
    }
  }
}

// dgamma_q, dgamma_k [D] from the blocks' sums, those of the queries first.  16 columns a
// block (D is a multiple of 16), 64 threads each, which take every 64th row and are joined in
// order.
__global__ void __launch_bounds__(1024)
    k_qk_dgamma(const float* part, int bq, int bk, int D, float* dgq, float* dgk) {
  __shared__ float sums[64][17];
  const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
  const bool isk = (int)blockIdx.x * 16 >= D;
  const int c = (int)blockIdx.x * 16 + x - (isk ? D : 0);
  const float* from = part + (isk ? (int64_t)bq * D : 0) + c;
  const int rows = isk ? bk : bq;
  float s = 0.0f;
#pragma unroll 8
  for (int b = y; b < rows; b += 64) s += from[(int64_t)b * D];
  sums[y][x] = s;
  __syncthreads();
  if (threadIdx.x < 16) {
    s = 0.0f;
#pragma unroll 16
    for (int b = 0; b < 64; ++b) s += sums[b][threadIdx.x];
    if (PACT_IN(c < D)) (isk ? dgk : dgq)[c] = s;
  }
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
  k_qk_dgamma<<<2 * p.D / 16, 1024, 0, st>>>(part, p.side[0].blocks, p.side[1].blocks, p.D, dgq,
                                                 dgk);
  return cudaGetLastError();
}

cudaError_t launch_rope_turns(const double* inv_freq, int n, int64_t* turns, cudaStream_t st) {
  note_launch();
  k_rope_turns<<<(n + 127) / 128, 128, 0, st>>>(inv_freq, n, turns);
  return cudaGetLastError();
}

}  // namespace pact
