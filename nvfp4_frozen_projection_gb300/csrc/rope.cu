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

// The rotation of one lane's 8 columns: y = own c + other s.
template <bool PAIRS>
struct Turn {
  float c[PAIRS ? 4 : 8], s[PAIRS ? 4 : 8];
  int other;    // lane offset of the other half
  bool turned;  // the lane's columns lie in the first rot
};

template <bool PAIRS>
__device__ __forceinline__ Turn<PAIRS> make_turn(int col, int rot, int pos, const int64_t* turns,
                                                 bool back) {
  Turn<PAIRS> t;
  t.turned = col < rot;
  t.other = 0;
  if (!t.turned) {
#pragma unroll
    for (int e = 0; e < (PAIRS ? 4 : 8); ++e) t.c[e] = 1.0f, t.s[e] = 0.0f;
    return t;
  }
  const int half = rot >> 1;
  const bool first = PAIRS || col < half;
  if (!PAIRS) t.other = first ? (half >> 3) : -(half >> 3);
  const int i0 = PAIRS ? col >> 1 : (first ? col : col - half);
#pragma unroll
  for (int e = 0; e < (PAIRS ? 4 : 8); ++e) {
    const uint64_t phase = (uint64_t)(int64_t)pos * (uint64_t)turns[i0 + e];
    float s, c;
    sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
    t.c[e] = c;
    // of a pair (a, b): a' = a c - b s, b' = b c + a s; backward the other way round
    t.s[e] = (first != back) ? -s : s;
  }
  return t;
}

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

__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

template <int SEG, bool NORM, bool PAIRS>
__global__ void __launch_bounds__(kRopeThreads)
    k_qk_norm_rope(const RopeParams p, int64_t segs, int chunks, int per) {
  const int lane = threadIdx.x & 31, sl = lane & (SEG - 1);
  const int64_t seg = (int64_t)blockIdx.x * (kRopeThreads / SEG) + threadIdx.x / SEG;
  if (seg - (lane / SEG) >= segs) return;  // a whole warp
  const bool live = seg < segs && sl * 8 < p.D;
  const int64_t t = seg < segs ? seg / chunks : 0;
  const int h0 = seg < segs ? (int)(seg - t * chunks) * per : 0;
  const int col = sl * 8, H = p.hq + p.hk;
  const Turn<PAIRS> tn = make_turn<PAIRS>(live ? col : p.rot, p.rot, p.positions[t], p.turns, false);
  const int other = lane + tn.other;
  // gammas of the lane's columns and, for halves, of the pair's other half
  uint4 gq = make_uint4(0, 0, 0, 0), gk = gq, oq = gq, ok = gq;
  if (NORM && live) {
    gq = *reinterpret_cast<const uint4*>(p.gamma_q + col);
    gk = *reinterpret_cast<const uint4*>(p.gamma_k + col);
    if (!PAIRS) {
      oq = *reinterpret_cast<const uint4*>(p.gamma_q + col + 8 * tn.other);
      ok = *reinterpret_cast<const uint4*>(p.gamma_k + col + 8 * tn.other);
    }
  }
  for (int hb = 0; hb < per; hb += kRopeUnroll) {
    uint4 v[kRopeUnroll];
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const int h = h0 + hb + u;
      v[u] = make_uint4(0, 0, 0, 0);
      if (live && hb + u < per && h < H)
        v[u] = *reinterpret_cast<const uint4*>(
            h < p.hq ? p.q + t * p.ldq + (int64_t)h * p.D + col
                     : p.k + t * p.ldk + (int64_t)(h - p.hq) * p.D + col);
    }
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const int h = h0 + hb + u;
      float f[8], o[8];
      bf16x8_to_f32(v[u], f);
      float rstd = 1.0f;
      if constexpr (NORM) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = __fmaf_rn(f[e], f[e], ss);
        ss = seg_sum<SEG>(ss);
        rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)p.D), p.eps)));
        float g[8];
        bf16x8_to_f32(h < p.hq ? gq : gk, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = f[e] * rstd * g[e];
      }
      if constexpr (PAIRS) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[2 * e] = f[2 * e] * tn.c[e] + f[2 * e + 1] * tn.s[e];
          o[2 * e + 1] = f[2 * e + 1] * tn.c[e] - f[2 * e] * tn.s[e];
        }
      } else {
        const uint4 w = shfl_v4(v[u], other);
        bf16x8_to_f32(w, o);
        if constexpr (NORM) {
          float g[8];
          bf16x8_to_f32(h < p.hq ? oq : ok, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = o[e] * rstd * g[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = f[e] * tn.c[e] + o[e] * tn.s[e];
      }
      if (live && hb + u < per && h < H && PACT_IN(t < p.T && col + 8 <= p.D))
        *reinterpret_cast<uint4*>(h < p.hq ? p.q_out + t * p.ldqo + (int64_t)h * p.D + col
                                           : p.k_out + t * p.ldko + (int64_t)(h - p.hq) * p.D +
                                                 col) = pack8(o);
    }
  }
}

// Backward; q, k are dy, xq and xk the forward's inputs (NORM).  DG: the sums for dgamma_q
// and dgamma_k of this block's groups go to part[block][2][D], group by group in order.
template <int SEG, bool NORM, bool PAIRS, bool DG>
__global__ void __launch_bounds__(kRopeThreads)
    k_qk_norm_rope_bwd(const RopeParams p, int64_t segs, int chunks, int per, float* part) {
  extern __shared__ float sums[];  // DG: [groups][2][8 SEG]
  const int lane = threadIdx.x & 31, sl = lane & (SEG - 1);
  constexpr int GROUPS = kRopeThreads / SEG;
  const int group = threadIdx.x / SEG;
  const int col = sl * 8, H = p.hq + p.hk;
  const bool inside = col < p.D;
  uint4 gq = make_uint4(0, 0, 0, 0), gk = gq;
  if (NORM && inside) {
    gq = *reinterpret_cast<const uint4*>(p.gamma_q + col);
    gk = *reinterpret_cast<const uint4*>(p.gamma_k + col);
  }
  float aq[DG ? 8 : 1] = {}, ak[DG ? 8 : 1] = {};
  for (int64_t first = (int64_t)blockIdx.x * GROUPS; first < segs;
       first += (int64_t)gridDim.x * GROUPS) {
    const int64_t seg = first + group;
    const bool live = seg < segs && inside;
    const int64_t t = seg < segs ? seg / chunks : 0;
    const int h0 = seg < segs ? (int)(seg - t * chunks) * per : 0;
    const Turn<PAIRS> tn = make_turn<PAIRS>(live ? col : p.rot, p.rot, p.positions[t], p.turns, true);
    const int other = lane + tn.other;
    constexpr int U = NORM ? 2 : kRopeUnroll;
    for (int hb = 0; hb < per; hb += U) {
      uint4 v[U], x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + hb + u;
        v[u] = x[u] = make_uint4(0, 0, 0, 0);
        if (live && hb + u < per && h < H) {
          const bool isq = h < p.hq;
          const int hh = isq ? h : h - p.hq;
          v[u] = *reinterpret_cast<const uint4*>((isq ? p.q + t * p.ldq : p.k + t * p.ldk) +
                                                 (int64_t)hh * p.D + col);
          if constexpr (NORM)
            x[u] = *reinterpret_cast<const uint4*>((isq ? p.xq + t * p.ldxq : p.xk + t * p.ldxk) +
                                                   (int64_t)hh * p.D + col);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + hb + u;
        float f[8], g[8];
        bf16x8_to_f32(v[u], f);
        if constexpr (PAIRS) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            g[2 * e] = f[2 * e] * tn.c[e] + f[2 * e + 1] * tn.s[e];
            g[2 * e + 1] = f[2 * e + 1] * tn.c[e] - f[2 * e] * tn.s[e];
          }
        } else {
          bf16x8_to_f32(shfl_v4(v[u], other), g);
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] = f[e] * tn.c[e] + g[e] * tn.s[e];
        }
        if constexpr (NORM) {
          float n[8], gm[8];
          bf16x8_to_f32(x[u], n);
          bf16x8_to_f32(h < p.hq ? gq : gk, gm);
          float ss = 0.0f, dot = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            ss = __fmaf_rn(n[e], n[e], ss);
            dot = __fmaf_rn(g[e] * gm[e], n[e], dot);
          }
          ss = seg_sum<SEG>(ss);
          dot = seg_sum<SEG>(dot);
          const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)p.D), p.eps)));
          const float c = __fdiv_rn(dot * rstd, (float)p.D);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            n[e] *= rstd;
            if constexpr (DG) {
              const float w = g[e] * n[e];  // zero in lanes and heads that hold nothing
              if (h < p.hq)
                aq[e] += w;
              else
                ak[e] += w;
            }
            g[e] = rstd * (g[e] * gm[e] - n[e] * c);
          }
        }
        if (live && hb + u < per && h < H && PACT_IN(t < p.T && col + 8 <= p.D))
          *reinterpret_cast<uint4*>(h < p.hq ? p.q_out + t * p.ldqo + (int64_t)h * p.D + col
                                             : p.k_out + t * p.ldko + (int64_t)(h - p.hq) * p.D +
                                                   col) = pack8(g);
      }
    }
  }
  if constexpr (DG) {
    if (inside) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sums[(group * 2 + 0) * (8 * SEG) + col + e] = aq[e];
        sums[(group * 2 + 1) * (8 * SEG) + col + e] = ak[e];
      }
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
