// RMSNorm with the residual's addition: forward to FP8, and backward.
//
//   h = bf16(x + residual);  rstd = 1 / sqrt(mean(h^2) + eps);  y = (h rstd) gamma
//   in FP32, quantised with one scale per 128 values (fp8.cuh).
//   backward, with n = h rstd and dn = dy gamma:
//     c = sum(dn n) / H;  dh = bf16(rstd (dn - n c) + dres);  dgamma = sum over rows dy n.
//   x and the residual have the same gradient, dh.
//
// Both are bound by HBM: 4 bytes read and 3 written per value forward (2 and 1
// without a residual), 6 read and 2 written backward.  A row is held in registers by
// a group of 1 to 16 warps, so each input is read once: thread vectors of 8 values
// (16 bytes), NV per thread, strided so that 16 neighbouring lanes hold one block of
// 128 and a warp's access is 512 contiguous bytes.  The sums over a row run lane by
// lane, then over the warp by a butterfly, then over the group's warps in order: the
// same order on every call.
#include "fp8.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace pact {

struct RowPlan {
  int nv;      // vectors of 8 per thread, 1..4
  int wpr;     // warps per row, a power of two, 1..16
  int groups;  // rows in flight per CTA
  int threads;
};

// Fewest warps per row that keep a thread's share at four vectors: fewer warps means
// fewer barriers.  With too few rows to fill the SMs a row is spread over more warps.
static RowPlan row_plan(int64_t M, int64_t H) {
  RowPlan p;
  p.wpr = 1;
  while (H > (int64_t)p.wpr * 1024) p.wpr *= 2;
  while (p.wpr < 8 && H > (int64_t)p.wpr * 256 && M * p.wpr < 2048) p.wpr *= 2;
  p.nv = (int)((H + p.wpr * 256 - 1) / (p.wpr * 256));
  p.threads = p.wpr > 8 ? 32 * p.wpr : 256;
  p.groups = p.threads / (32 * p.wpr);
  return p;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Sum over the wpr warps of a row group; slot: 16 floats of this group (one of two
// used in turn, so that a group's next sum does not overwrite values still read).
__device__ __forceinline__ float group_sum(float v, int wpr, int wl, int group, float* slot) {
  v = warp_sum(v);
  if (wpr == 1) return v;
  if ((threadIdx.x & 31) == 0) slot[wl] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * wpr) : "memory");
  float t = slot[0];
  for (int i = 1; i < wpr; ++i) t += slot[i];
  return t;
}

// Four CTAs an SM (64 registers): 26624 x 2048 in 60.5 us, 0.93 of HBM; with three 65.5,
// with five 70.8 (it spills).
template <int NV, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 4 : 2)
    k_add_rmsnorm_fp8(const uint16_t* x, const uint16_t* res, const uint16_t* gamma, int64_t M,
                      int64_t H, float eps, int wpr, uint16_t* h_out, uint8_t* q, float* s,
                      float* rstd_out) {
  __shared__ float slots[16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / wpr, wl = warp - group * wpr;
  const int64_t row = (int64_t)blockIdx.x * ((THREADS / 32) / wpr) + group;
  if (row >= M) return;  // a whole group
  uint4 hv[NV];
  const int64_t base = row * H;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = (int64_t)((i * wpr + wl) * 32 + lane) * 8;
    hv[i] = make_uint4(0u, 0u, 0u, 0u);
    if (c < H) hv[i] = *reinterpret_cast<const uint4*>(x + base + c);
  }
  if (res) {
    uint4 rv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t)((i * wpr + wl) * 32 + lane) * 8;
      rv[i] = make_uint4(0u, 0u, 0u, 0u);
      if (c < H) rv[i] = *reinterpret_cast<const uint4*>(res + base + c);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float a[8], b[8];
      bf16x8_to_f32(hv[i], a);
      bf16x8_to_f32(rv[i], b);
      hv[i] = make_uint4(pack_bf16x2(__fadd_rn(a[0], b[0]), __fadd_rn(a[1], b[1])),
                         pack_bf16x2(__fadd_rn(a[2], b[2]), __fadd_rn(a[3], b[3])),
                         pack_bf16x2(__fadd_rn(a[4], b[4]), __fadd_rn(a[5], b[5])),
                         pack_bf16x2(__fadd_rn(a[6], b[6]), __fadd_rn(a[7], b[7])));
      const int64_t c = (int64_t)((i * wpr + wl) * 32 + lane) * 8;
      if (c < H && PACT_IN(base + c + 8 <= M * H))
        *reinterpret_cast<uint4*>(h_out + base + c) = hv[i];
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float f[8];
    bf16x8_to_f32(hv[i], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = __fmaf_rn(f[e], f[e], ss);
  }
  ss = group_sum(ss, wpr, wl, group, slots + group * wpr);
  const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)H), eps)));
  if (wl == 0 && lane == 0 && PACT_IN(row < M)) rstd_out[row] = rstd;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = (int64_t)((i * wpr + wl) * 32 + lane) * 8;
    uint4 gv = make_uint4(0u, 0u, 0u, 0u);
    if (c < H) gv = *reinterpret_cast<const uint4*>(gamma + c);
    float f[8], g[8], amax = 0.0f;
    bf16x8_to_f32(hv[i], f);
    bf16x8_to_f32(gv, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[e] = __fmul_rn(__fmul_rn(f[e], rstd), g[e]);
      amax = fmaxf(amax, fabsf(f[e]));
    }
    const Fp8Scale sc = fp8_scale(half_warp_max(amax));
    if (c < H && PACT_IN(base + c + 8 <= M * H)) {
      *reinterpret_cast<uint2*>(q + base + c) = e4m3x8(f, sc.r);
      if ((lane & 15) == 0) s[(c >> 7) * M + row] = sc.s;
    }
  }
}

cudaError_t launch_add_rmsnorm_fp8(const uint16_t* x, const uint16_t* res, const uint16_t* gamma,
                                   int64_t M, int64_t H, float eps, uint16_t* h, uint8_t* q,
                                   float* s, float* rstd, cudaStream_t stream) {
  const RowPlan p = row_plan(M, H);
  const unsigned grid = (unsigned)((M + p.groups - 1) / p.groups);
  note_launch();
#define PACT_NORM(NV, T) \
  k_add_rmsnorm_fp8<NV, T><<<grid, T, 0, stream>>>(x, res, gamma, M, H, eps, p.wpr, h, q, s, rstd)
  if (p.threads == 512) {
    if (p.nv == 3) PACT_NORM(3, 512); else PACT_NORM(4, 512);
  } else if (p.nv == 1) {
    PACT_NORM(1, 256);
  } else if (p.nv == 2) {
    PACT_NORM(2, 256);
  } else if (p.nv == 3) {
    PACT_NORM(3, 256);
  } else {
    PACT_NORM(4, 256);
  }
#undef PACT_NORM
  return cudaGetLastError();
}

// ---------------------------------------------------------------- backward
// A persistent grid: a thread owns the same columns in every row, so gamma and dgamma's
// partial sums stay in its registers; each group writes one row of partial sums at the
// end, and a second kernel adds them in a fixed order.  The next row's vectors are loaded
// before this row is worked on: without that a row's three latencies (the loads, the sum
// over the group, dres) add up (8192 x 4096: 110 us, 2.4 TB/s).
// As row_plan, with at most two vectors a thread, since two rows are held at a time.  Above
// 8192 columns three or four, and the next row waits in shared memory (12288 columns, 2048
// rows: 42.6 us, 49.9 without the next row; up to 8192 columns that is slower, 4096 x 8192
// 58.9 us against 50.1).
static RowPlan bwd_plan(int64_t M, int64_t H) {
  RowPlan p;
  p.wpr = 1;
  const int64_t per_warp = H > 8192 ? 1024 : 512;
  while (H > (int64_t)p.wpr * per_warp) p.wpr *= 2;
  while (p.wpr < 8 && H > (int64_t)p.wpr * 256 && M * p.wpr < 2048) p.wpr *= 2;
  p.nv = (int)((H + p.wpr * 256 - 1) / (p.wpr * 256));
  p.threads = p.wpr > 8 ? 32 * p.wpr : 256;
  p.groups = p.threads / (32 * p.wpr);
  return p;
}

// The grid is that of a GB300 on any device, so that the size of the workspace and the order
// of dgamma's sums follow from the sizes alone.
static int bwd_ctas(int64_t M, const RowPlan& p) {
  const int64_t n = (M + p.groups - 1) / p.groups;
  const int most = 152 * (p.threads > 256 ? 1 : (p.nv == 1 ? 3 : 2));  // resident at once
  return (int)(n < most ? n : most);
}

// Small tensors: dgamma comes from CTAs of their own in the same launch, which read h and
// dy again, out of L2, 16 columns each; no second kernel and no workspace.  1333 x 1040:
// 6.5 us against 8.1 with partial sums, and a call of 8.5 us instead of 17.2; at
// 4000 x 1024 the kernels take 15.2 against 12.3 us and the calls about the same.
static bool bwd_in_one(int64_t M, int64_t H) { return M <= 4096 && M * H <= (int64_t)1 << 22; }

int64_t rmsnorm_bwd_partials(int64_t M, int64_t H) {
  if (bwd_in_one(M, H)) return 0;
  const RowPlan p = bwd_plan(M, H);
  return (int64_t)bwd_ctas(M, p) * p.groups;
}

template <int NV>
struct BwdRow {
  uint4 h[NV], dy[NV], dres[NV];
  float rstd;
};

// dgamma of 16 columns: two vectors of 8 across, 128 rows down, four in flight a thread;
// the rows of a thread in order, then over the warp by a butterfly, then the warps in order.
__device__ __forceinline__ void dgamma_columns(const uint16_t* h, const uint16_t* dy,
                                               const float* rstd, int64_t M, int64_t H, int64_t c0,
                                               float* dgamma, float (*sums)[16]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c = c0 + 8 * (lane & 1);
  float acc[8] = {};
  for (int64_t m = threadIdx.x >> 1; m < M; m += 4 * 128) {
    uint4 hv[4], dv[4];
    float r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t row = m + 128 * j;
      hv[j] = dv[j] = make_uint4(0u, 0u, 0u, 0u);
      r[j] = 0.0f;
      if (row < M) {
        hv[j] = *reinterpret_cast<const uint4*>(h + row * H + c);
        dv[j] = *reinterpret_cast<const uint4*>(dy + row * H + c);
        r[j] = rstd[row];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[8], d[8];
      bf16x8_to_f32(hv[j], f);
      bf16x8_to_f32(dv[j], d);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = __fmaf_rn(d[e], __fmul_rn(f[e], r[j]), acc[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int o = 16; o > 1; o >>= 1) acc[e] += __shfl_xor_sync(0xFFFFFFFFu, acc[e], o);
    if (lane < 2) sums[warp][8 * lane + e] = acc[e];
  }
  __syncthreads();
  if (threadIdx.x < 16) {
    float t = sums[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < 8; ++w) t += sums[w][threadIdx.x];
    if (PACT_IN(c0 + threadIdx.x < H)) dgamma[c0 + threadIdx.x] = t;
  }
}

// dgamma, when not null, is made by the CTAs from row_ctas on (H / 16 of them, 256
// threads).
template <int NV, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS > 256 ? 1 : (NV == 1 ? 3 : 2))
    k_add_rmsnorm_bwd(const uint16_t* h, const uint16_t* gamma, const float* rstd_in,
                      const uint16_t* dy, const uint16_t* dres, int64_t M, int64_t H, int wpr,
                      int row_ctas, uint16_t* dh, float* part, float* dgamma) {
  __shared__ float slots[2][16];
  // more than two vectors a thread: dgamma's partial sums and the next row in shared
  // memory, gamma in L1
  constexpr bool WIDE = NV > 2;
  extern __shared__ float4 wide_smem[];
  float4(*dg_wide)[THREADS] = reinterpret_cast<float4(*)[THREADS]>(wide_smem);
  uint4(*ahead)[THREADS] = reinterpret_cast<uint4(*)[THREADS]>(wide_smem + 2 * NV * THREADS);
  if constexpr (THREADS == 256) {
    __shared__ float sums[8][16];
    if ((int)blockIdx.x >= row_ctas) {
      dgamma_columns(h, dy, rstd_in, M, H, 16 * (int64_t)((int)blockIdx.x - row_ctas), dgamma, sums);
      return;
    }
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / wpr, wl = warp - group * wpr;
  const int groups = (THREADS / 32) / wpr;
  const float inv_h = __fdiv_rn(1.0f, (float)H);
  const int c0 = (wl * 32 + lane) * 8, cstep = wpr * 256;  // vector i: column c0 + i cstep
  uint4 gv[WIDE ? 1 : NV];
  float dg[WIDE ? 1 : NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (WIDE) {
      dg_wide[2 * i][threadIdx.x] = dg_wide[2 * i + 1][threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
      gv[i] = make_uint4(0u, 0u, 0u, 0u);
      if (c0 + i * cstep < H) gv[i] = *reinterpret_cast<const uint4*>(gamma + c0 + i * cstep);
#pragma unroll
      for (int e = 0; e < 8; ++e) dg[i][e] = 0.0f;
    }
  }
  auto gamma_of = [&](int i) {
    if constexpr (!WIDE) return gv[i];
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    return c0 + i * cstep < H ? *reinterpret_cast<const uint4*>(gamma + c0 + i * cstep) : z;
  };
  auto load = [&](int64_t row, BwdRow<NV>& r) {
    r.rstd = rstd_in[row];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      r.h[i] = r.dy[i] = r.dres[i] = make_uint4(0u, 0u, 0u, 0u);
      const int c = c0 + i * cstep;
      if (c < H) {
        r.h[i] = *reinterpret_cast<const uint4*>(h + row * H + c);
        r.dy[i] = *reinterpret_cast<const uint4*>(dy + row * H + c);
        if (dres) r.dres[i] = *reinterpret_cast<const uint4*>(dres + row * H + c);
      }
    }
  };
  // WIDE: the next row on its way into shared memory, each thread's vectors in slots of
  // its own
  float rstd_next = 0.0f;
  auto fetch = [&](int64_t row) {
    rstd_next = rstd_in[row];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * cstep;
      const uint32_t n = c < H ? 16u : 0u;  // none: zeros
      const int64_t at = c < H ? row * H + c : 0;
      cp_async16(smem_addr(&ahead[3 * i][threadIdx.x]), h + at, n);
      cp_async16(smem_addr(&ahead[3 * i + 1][threadIdx.x]), dy + at, n);
      cp_async16(smem_addr(&ahead[3 * i + 2][threadIdx.x]), dres ? dres + at : dy, dres ? n : 0u);
    }
    cp_async_commit();
  };
  int turn = 0;
  const int64_t step = (int64_t)row_ctas * groups;
  int64_t row = (int64_t)blockIdx.x * groups + group;
  BwdRow<NV> cur, next;
  if (row < M) {
    if constexpr (WIDE)
      fetch(row);
    else
      load(row, cur);
  }
  for (; row < M; row += step) {
    if constexpr (WIDE) {
      cp_async_wait<0>();
      cur.rstd = rstd_next;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        cur.h[i] = ahead[3 * i][threadIdx.x];
        cur.dy[i] = ahead[3 * i + 1][threadIdx.x];
        cur.dres[i] = ahead[3 * i + 2][threadIdx.x];
      }
      __syncwarp();  // the slots have been read
      if (row + step < M) fetch(row + step);
    } else if (row + step < M) {
      load(row + step, next);
    }
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[8], d[8], g[8];
      bf16x8_to_f32(cur.h[i], f);
      bf16x8_to_f32(cur.dy[i], d);
      bf16x8_to_f32(gamma_of(i), g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = __fmul_rn(f[e], cur.rstd);
        t = __fmaf_rn(__fmul_rn(d[e], g[e]), n, t);
        if constexpr (WIDE)
          f[e] = n;
        else
          dg[i][e] = __fmaf_rn(d[e], n, dg[i][e]);
      }
      if constexpr (WIDE) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float4 a = dg_wide[2 * i + k][threadIdx.x];
          a.x = __fmaf_rn(d[4 * k], f[4 * k], a.x);
          a.y = __fmaf_rn(d[4 * k + 1], f[4 * k + 1], a.y);
          a.z = __fmaf_rn(d[4 * k + 2], f[4 * k + 2], a.z);
          a.w = __fmaf_rn(d[4 * k + 3], f[4 * k + 3], a.w);
          dg_wide[2 * i + k][threadIdx.x] = a;
        }
      }
    }
    t = group_sum(t, wpr, wl, group, slots[turn] + group * wpr);
    turn ^= 1;
    const float c = __fmul_rn(t, inv_h);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = c0 + i * cstep;
      if (col >= H) continue;
      float f[8], d[8], g[8], r[8];
      bf16x8_to_f32(cur.h[i], f);
      bf16x8_to_f32(cur.dy[i], d);
      bf16x8_to_f32(gamma_of(i), g);
      bf16x8_to_f32(cur.dres[i], r);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = __fmul_rn(f[e], cur.rstd);
        f[e] = __fmaf_rn(cur.rstd, __fmaf_rn(-n, c, __fmul_rn(d[e], g[e])), r[e]);
      }
      const uint4 o = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                 pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
      if (PACT_IN(row * H + col + 8 <= M * H)) *reinterpret_cast<uint4*>(dh + row * H + col) = o;
    }
    if constexpr (!WIDE) cur = next;
  }
  if (!part) return;
  float* p = part + ((int64_t)blockIdx.x * groups + group) * H;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = c0 + i * cstep;
    if (c >= H || !PACT_IN((int)blockIdx.x < row_ctas && c + 8 <= H)) continue;
    if constexpr (WIDE) {
      *reinterpret_cast<float4*>(p + c) = dg_wide[2 * i][threadIdx.x];
      *reinterpret_cast<float4*>(p + c + 4) = dg_wide[2 * i + 1][threadIdx.x];
    } else {
      *reinterpret_cast<float4*>(p + c) = make_float4(dg[i][0], dg[i][1], dg[i][2], dg[i][3]);
      *reinterpret_cast<float4*>(p + c + 4) = make_float4(dg[i][4], dg[i][5], dg[i][6], dg[i][7]);
    }
  }
}

// dgamma[j] = sum over the P rows of part: 8 columns (a sector) a CTA, 64 row lanes, each
// in row order with eight loads in flight, then the lanes in order.
__global__ void __launch_bounds__(512)
    k_dgamma_reduce(const float* part, int P, int64_t H, float* dgamma) {
  __shared__ float sum[64][9];
  const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;
  const int64_t j = (int64_t)blockIdx.x * 8 + tx;  // H % 16 == 0
  float t = 0.0f;
  for (int p = ty; p < P; p += 8 * 64) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p + 64 * i < P ? part[(int64_t)(p + 64 * i) * H + j] : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += v[i];
  }
  sum[ty][tx] = t;
  __syncthreads();
  if (ty < 8) {
    t = sum[8 * ty][tx];
#pragma unroll
    for (int i = 1; i < 8; ++i) t += sum[8 * ty + i][tx];
    sum[8 * ty][tx] = t;
  }
  __syncthreads();
  if (ty == 0) {
    t = sum[0][tx];
#pragma unroll
    for (int i = 1; i < 8; ++i) t += sum[8 * i][tx];
    if (PACT_IN(j < H)) dgamma[j] = t;
  }
}

cudaError_t launch_add_rmsnorm_bwd(const uint16_t* h, const uint16_t* gamma, const float* rstd,
                                   const uint16_t* dy, const uint16_t* dres, int64_t M, int64_t H,
                                   uint16_t* dh, float* dgamma, float* part, cudaStream_t stream) {
  const RowPlan p = bwd_plan(M, H);
  const int grid = bwd_ctas(M, p);
  const bool small = dgamma && bwd_in_one(M, H);
  // in the same launch unless dh overwrites what the columns read, or the rows take larger
  // CTAs
  const bool one = small && p.threads == 256 && dh != dy && dh != h;
  const int cols = (int)(H / 16);
  float* pp = dgamma && !small ? part : nullptr;
  if (small && !one) {
    note_launch();
    k_add_rmsnorm_bwd<1, 256><<<cols, 256, 0, stream>>>(h, gamma, rstd, dy, nullptr, M, H, 1,
                                                              0, nullptr, nullptr, dgamma);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  note_launch();
  // five vectors of 16 bytes for each of a thread's: two of sums, three of the next row
  const size_t smem = p.nv > 2 ? (size_t)p.nv * 5 * 16 * p.threads : 0;
  if (smem) {
    cudaError_t e = cudaFuncSetAttribute(
        p.nv == 4 ? k_add_rmsnorm_bwd<4, 512> : k_add_rmsnorm_bwd<3, 512>,
        cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
#define PACT_NORM(NV, T)                                                                     \
  k_add_rmsnorm_bwd<NV, T>                                                                   \
      <<<grid + (one ? cols : 0), T, smem, stream>>>(h, gamma, rstd, dy, dres, M, H, p.wpr, grid, \
                                                     dh, pp, one ? dgamma : nullptr)
  if (p.nv == 4)
    PACT_NORM(4, 512);
  else if (p.nv == 3)
    PACT_NORM(3, 512);
  else if (p.threads == 512)
    PACT_NORM(2, 512);
  else if (p.nv == 2)
    PACT_NORM(2, 256);
  else
    PACT_NORM(1, 256);
#undef PACT_NORM
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !dgamma || small) return e;
  note_launch();
  k_dgamma_reduce<<<(unsigned)(H / 8), 512, 0, stream>>>(part, grid * p.groups, H, dgamma);
  return cudaGetLastError();
}

}  // namespace pact
