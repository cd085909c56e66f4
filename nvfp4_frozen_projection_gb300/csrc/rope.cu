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
// A group of 8, 16 or 32 lanes holds a head, 8 values (16 bytes) a lane, and takes the heads
// of one token in turn, so that a lane computes the sines of its columns once for all of
// them; a pair's other half comes from the lane that holds it as packed BF16.  With few
// tokens the heads of a token are shared out over more groups.
#include "common.cuh"
#include "kernels.h"

namespace pact {

constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 4;  // heads in flight a group

// Groups that fill the GPU: 152 SMs of 2048 threads, at most.
static int rope_chunks(int64_t T, int heads, int seg, int num_sms) {
  const int64_t want = (int64_t)num_sms * 2048 / seg;
  if (T >= want) return 1;
  const int64_t c = (want + T - 1) / T;
  return (int)(c < heads ? c : heads);
}

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

// The first `heads` heads of a token from x on (x, out: at this lane's columns).  NORM: the gammas
// are in the coefficients, y = rstd (own (gamma c) + other (gamma' s)).
template <int SEG, bool NORM, bool PAIRS>
__device__ __forceinline__ void rope_heads(const uint16_t* x, uint16_t* out, int rounds, int heads,
                                           int D, float inv_d, float eps, bool live, const float2* c,
                                           const float2* s, int other) {
  for (int hb = 0; hb < rounds; hb += kRopeUnroll) {
    uint4 v[kRopeUnroll];
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      v[u] = make_uint4(0, 0, 0, 0);
      if (live && hb + u < heads)
        v[u] = *reinterpret_cast<const uint4*>(x + (int64_t)(hb + u) * D);
    }
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
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
        r = both(rstd_of(seg_sum<SEG>(q.x + q.y), inv_d, eps));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[e] = __ffma2_rn(f[e], c[e], __fmul2_rn(o[e], s[e]));
        if constexpr (NORM) f[e] = __fmul2_rn(f[e], r);
      }
      if (live && hb + u < heads)
        *reinterpret_cast<uint4*>(out + (int64_t)(hb + u) * D) = pack8(f);
    }
  }
}

template <int SEG, bool NORM, bool PAIRS>
__global__ void __launch_bounds__(kRopeThreads)
    k_qk_norm_rope(const RopeParams p, int64_t segs, int chunks, int per) {
  const int lane = threadIdx.x & 31, sl = lane & (SEG - 1);
  const int64_t seg = (int64_t)blockIdx.x * (kRopeThreads / SEG) + threadIdx.x / SEG;
  // a dead group stays for the shuffles of its warp, with no heads
  const int64_t t = seg < segs ? seg / chunks : 0;
  const int h0 = seg < segs ? (int)(seg - t * chunks) * per : 0, H = p.hq + p.hk;
  const int h1 = seg < segs ? min(h0 + per, H) : 0;
  const bool live = seg < segs && sl * 8 < p.D && PACT_IN(t < p.T);
  const int col = sl * 8;
  const Turn tn = make_turn<PAIRS>(live ? col : p.rot, p.rot, p.positions[t], p.turns, false);
  const int other = lane + tn.other;
  const float inv_d = 1.0f / (float)p.D;
  // every group of a warp runs as many rounds as the longest, or shuffles would miss lanes
  auto run = [&](const uint16_t* x, uint16_t* out, const uint16_t* gamma, int a, int b) {
    float2 c[4], s[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = tn.c[e], s[e] = tn.s[e];
    if (NORM && live) {
      float2 g[4], o[4];
      unpack8(*reinterpret_cast<const uint4*>(gamma + col), g);
      if constexpr (PAIRS) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = swapped(g[e]);
      } else {
        unpack8(*reinterpret_cast<const uint4*>(gamma + col + 8 * tn.other), o);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) c[e] = __fmul2_rn(c[e], g[e]), s[e] = __fmul2_rn(s[e], o[e]);
    }
    const int n = __reduce_max_sync(0xFFFFFFFFu, max(b - a, 0));
    rope_heads<SEG, NORM, PAIRS>(x + (int64_t)a * p.D, out + (int64_t)a * p.D, n, b - a, p.D,
                                 inv_d, p.eps, live, c, s, other);
  };
  run(p.q + t * p.ldq + col, p.q_out + t * p.ldqo + col, p.gamma_q, h0, min(h1, p.hq));
  run(p.k + t * p.ldk + col, p.k_out + t * p.ldko + col, p.gamma_k, max(h0 - p.hq, 0), h1 - p.hq);
}

// Backward; q, k are dy, xq and xk the forward's inputs (NORM).  DG: the sums for dgamma_q
// and dgamma_k of this block's groups go to part[block][2][D], group by group in order.
template <int SEG, bool NORM, bool PAIRS, bool DG>
__device__ __forceinline__ void rope_heads_bwd(const uint16_t* dy, const uint16_t* x,
                                               uint16_t* out, int rounds, int heads, int D,
                                               float inv_d, float eps, bool live, const Turn& tn,
                                               int other, const float2* gm, float2* acc) {
  constexpr int U = NORM ? 2 : kRopeUnroll;
  for (int hb = 0; hb < rounds; hb += U) {
    uint4 v[U], w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u] = w[u] = make_uint4(0, 0, 0, 0);
      if (live && hb + u < heads) {
        v[u] = *reinterpret_cast<const uint4*>(dy + (int64_t)(hb + u) * D);
        if constexpr (NORM) w[u] = *reinterpret_cast<const uint4*>(x + (int64_t)(hb + u) * D);
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
        const float rstd = rstd_of(seg_sum<SEG>(ss.x + ss.y), inv_d, eps);
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
      if (live && hb + u < heads)
        *reinterpret_cast<uint4*>(out + (int64_t)(hb + u) * D) = pack8(g);
    }
  }
}

template <int SEG, bool NORM, bool PAIRS, bool DG>
__global__ void __launch_bounds__(kRopeThreads)
    k_qk_norm_rope_bwd(const RopeParams p, int64_t segs, int chunks, int per, float* part) {
  extern __shared__ float sums[];  // DG: [groups][2][8 SEG]
  const int lane = threadIdx.x & 31, sl = lane & (SEG - 1);
  constexpr int GROUPS = kRopeThreads / SEG;
  const int group = threadIdx.x / SEG;
  const int col = sl * 8, H = p.hq + p.hk;
  const bool inside = col < p.D;
  const float inv_d = 1.0f / (float)p.D;
  float2 acc[2][DG ? 4 : 1] = {};
  for (int64_t first = (int64_t)blockIdx.x * GROUPS; first < segs;
       first += (int64_t)gridDim.x * GROUPS) {
    const int64_t seg = first + group;
    const int64_t t = seg < segs ? seg / chunks : 0;
    const bool live = seg < segs && inside && PACT_IN(t < p.T);
    const int h0 = seg < segs ? (int)(seg - t * chunks) * per : 0;
    const int h1 = seg < segs ? min(h0 + per, H) : 0;
    const Turn tn = make_turn<PAIRS>(live ? col : p.rot, p.rot, p.positions[t], p.turns, true);
    const int other = lane + tn.other;
#pragma unroll
    for (int w = 0; w < 2; ++w) {  // queries, keys
      const int a = w ? max(h0 - p.hq, 0) : h0, b = w ? h1 - p.hq : min(h1, p.hq);
      const int64_t at = (int64_t)a * p.D + col;
      float2 gm[4] = {};
      if (NORM && live) unpack8(*reinterpret_cast<const uint4*>((w ? p.gamma_k : p.gamma_q) + col), gm);
      const int rounds = __reduce_max_sync(0xFFFFFFFFu, max(b - a, 0));
      rope_heads_bwd<SEG, NORM, PAIRS, DG>(
          (w ? p.k + t * p.ldk : p.q + t * p.ldq) + at,
          NORM ? (w ? p.xk + t * p.ldxk : p.xq + t * p.ldxq) + at : nullptr,
          (w ? p.k_out + t * p.ldko : p.q_out + t * p.ldqo) + at, rounds, b - a, p.D, inv_d, p.eps,
          live, tn, other, gm, acc[w]);
    }
  }
  if constexpr (DG) {
    if (inside) {
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<float2*>(sums + (group * 2 + w) * (8 * SEG) + col + 2 * e) = acc[w][e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.D; i += kRopeThreads) {
      const int w = i / p.D, c = i - w * p.D;
      float s = 0.0f;
      for (int g = 0; g < GROUPS; ++g) s += sums[(g * 2 + w) * (8 * SEG) + c];
      if (PACT_IN(i < 2 * p.D)) part[(int64_t)blockIdx.x * 2 * p.D + i] = s;
    }
  }
}

// dgamma_q, dgamma_k [D] from the blocks' sums: a warp a column, its lanes' sums over every
// 32nd block joined by a butterfly.
__global__ void __launch_bounds__(256)
    k_qk_dgamma(const float* part, int blocks, int D, float* dgq, float* dgk) {
  const int c = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (c >= 2 * D) return;
  float s = 0.0f;
  for (int b = lane; b < blocks; b += 32) s += part[(int64_t)b * 2 * D + c];
  s = seg_sum<32>(s);
  if (lane == 0 && PACT_IN(c < 2 * D)) (c < D ? dgq[c] : dgk[c - D]) = s;
}

__global__ void k_rope_turns(const double* inv_freq, int n, int64_t* turns) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  double f = inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi): radians to turns
  f -= floor(f);
  // 2^64 f, the lower half separately: f may be just below one
  const double hi = floor(f * 4294967296.0);
  const double lo = (f * 4294967296.0 - hi) * 4294967296.0;
  turns[i] = (int64_t)(((uint64_t)hi << 32) + (uint64_t)lo);
}

static int seg_lanes(int D) { return D <= 64 ? 8 : (D <= 128 ? 16 : 32); }

template <int SEG>
static void launch_fwd(const RopeParams& p, bool norm, bool pairs, int64_t segs, int chunks,
                       int per, unsigned grid, cudaStream_t st) {
  if (norm && pairs)
    k_qk_norm_rope<SEG, true, true><<<grid, kRopeThreads, 0, st>>>(p, segs, chunks, per);
  else if (norm)
    k_qk_norm_rope<SEG, true, false><<<grid, kRopeThreads, 0, st>>>(p, segs, chunks, per);
  else if (pairs)
    k_qk_norm_rope<SEG, false, true><<<grid, kRopeThreads, 0, st>>>(p, segs, chunks, per);
  else
    k_qk_norm_rope<SEG, false, false><<<grid, kRopeThreads, 0, st>>>(p, segs, chunks, per);
}

cudaError_t launch_qk_norm_rope(const RopeParams& p, int pairs, int num_sms, cudaStream_t st) {
  const int seg = seg_lanes(p.D), H = p.hq + p.hk;
  int chunks = rope_chunks(p.T, H, seg, num_sms);
  const int per = (H + chunks - 1) / chunks;
  chunks = (H + per - 1) / per;
  const int64_t segs = p.T * chunks, gs = kRopeThreads / seg;
  const unsigned grid = (unsigned)((segs + gs - 1) / gs);
  const bool norm = p.gamma_q != nullptr;
  note_launch();
  if (seg == 8)
    launch_fwd<8>(p, norm, pairs, segs, chunks, per, grid, st);
  else if (seg == 16)
    launch_fwd<16>(p, norm, pairs, segs, chunks, per, grid, st);
  else
    launch_fwd<32>(p, norm, pairs, segs, chunks, per, grid, st);
  return cudaGetLastError();
}

// Blocks of the backward: no more than 4 an SM, so that the sums for dgamma are few.
int64_t rope_bwd_blocks(int64_t T, int heads, int D, int num_sms) {
  const int seg = seg_lanes(D);
  int chunks = rope_chunks(T, heads, seg, num_sms);
  const int per = (heads + chunks - 1) / chunks;
  chunks = (heads + per - 1) / per;
  const int64_t gs = kRopeThreads / seg, blocks = (T * chunks + gs - 1) / gs;
  return blocks < 4ll * num_sms ? blocks : 4ll * num_sms;
}

template <int SEG>
static void launch_bwd(const RopeParams& p, bool norm, bool pairs, bool dg, int64_t segs,
                       int chunks, int per, unsigned grid, float* part, cudaStream_t st) {
  const size_t sm = dg ? (size_t)(kRopeThreads / SEG) * 2 * 8 * SEG * 4 : 0;
#define PACT_ROPE_BWD(N, P, G) \
  k_qk_norm_rope_bwd<SEG, N, P, G><<<grid, kRopeThreads, sm, st>>>(p, segs, chunks, per, part)
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

cudaError_t launch_qk_norm_rope_bwd(const RopeParams& p, int pairs, float* dgq, float* dgk,
                                    float* part, int num_sms, cudaStream_t st) {
  const int seg = seg_lanes(p.D), H = p.hq + p.hk;
  int chunks = rope_chunks(p.T, H, seg, num_sms);
  const int per = (H + chunks - 1) / chunks;
  chunks = (H + per - 1) / per;
  const int64_t segs = p.T * chunks;
  const bool norm = p.gamma_q != nullptr, dg = dgq != nullptr;
  const unsigned grid = (unsigned)rope_bwd_blocks(p.T, H, p.D, num_sms);
  note_launch();
  if (seg == 8)
    launch_bwd<8>(p, norm, pairs, dg, segs, chunks, per, grid, part, st);
  else if (seg == 16)
    launch_bwd<16>(p, norm, pairs, dg, segs, chunks, per, grid, part, st);
  else
    launch_bwd<32>(p, norm, pairs, dg, segs, chunks, per, grid, part, st);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !dg) return e;
  note_launch();
  k_qk_dgamma<<<(2 * p.D + 7) / 8, 256, 0, st>>>(part, (int)grid, p.D, dgq, dgk);
  return cudaGetLastError();
}

cudaError_t launch_rope_turns(const double* inv_freq, int n, int64_t* turns, cudaStream_t st) {
  note_launch();
  k_rope_turns<<<(n + 127) / 128, 128, 0, st>>>(inv_freq, n, turns);
  return cudaGetLastError();
}

}  // namespace pact
