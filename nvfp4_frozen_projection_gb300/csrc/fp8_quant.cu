// FP8 quantiser of BF16 activations and gradients (one scale per 128 values of a row)
// and the offline weight packs (one scale per 128 x 128 tile).
#include "fp8.cuh"
#include "kernels.h"

namespace pact {

// Rows per warp of the quantiser.  A warp takes one block column of kQRows rows, a
// half warp per row and step; its loads are all issued before the first is used.
constexpr int kQRows = 8;

// HBM bounds it: 2 bytes read and 1.03 written a value.  8192 x 16384 takes 60 us, the rate
// of a plain copy; 66.9 with the scale made by every lane (74 % of the issue slots) and
// 62.7 with five CTAs an SM instead of six.
__global__ void __launch_bounds__(256, 6)
    k_quant_fp8(const uint16_t* __restrict__ x, int64_t M, int64_t K, int64_t ldx, uint32_t units,
                FastDiv kb_div, uint8_t* __restrict__ q, float* __restrict__ s) {
  const uint32_t unit = blockIdx.x * 8u + (threadIdx.x >> 5);
  if (unit >= units) return;  // whole warps
  const int lane = threadIdx.x & 31, half = lane >> 4;
  const uint32_t rg = kb_div.div(unit), kb = unit - rg * kb_div.d;
  const int64_t m0 = (int64_t)rg * kQRows;
  const int64_t c = (int64_t)kb * 128 + 8 * (lane & 15);
  const bool col_ok = c < K;  // K % 16 == 0: a vector of 8 lies inside or outside whole
  uint4 v[kQRows / 2];
#pragma unroll
  for (int i = 0; i < kQRows / 2; ++i) {
    const int64_t m = m0 + 2 * i + half;
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (col_ok && m < M) v[i] = *reinterpret_cast<const uint4*>(x + m * ldx + c);
  }
  // The block maxima are BF16 values: two steps' travel through the half warp in one
  // word.  Lane j < 8 then makes the scale of row m0 + j, one division pair for the warp
  // instead of one for each row and lane, and hands its factor out.
  uint32_t pk[kQRows / 4];
#pragma unroll
  for (int i = 0; i < kQRows / 4; ++i) {
    pk[i] = (absmax_bf16x8_bits_any(v[2 * i]) >> 16) | absmax_bf16x8_bits_any(v[2 * i + 1]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
      pk[i] = __vmaxu2(pk[i], __shfl_xor_sync(0xFFFFFFFFu, pk[i], o));
  }
  // row j = 2 (2 p + e) + half: word p = j / 4, its low (e = 0) or high half, e = j / 2 % 2
  const uint32_t w0 = __shfl_sync(0xFFFFFFFFu, pk[0], (lane & 1) * 16);
  const uint32_t w1 = __shfl_sync(0xFFFFFFFFu, pk[1], (lane & 1) * 16);
  const uint32_t w = (lane & 4) ? w1 : w0;
  const Fp8Scale mine = fp8_scale(__uint_as_float((lane & 2) ? w & 0xFFFF0000u : w << 16));
#pragma unroll
  for (int i = 0; i < kQRows / 2; ++i) {
    const int64_t m = m0 + 2 * i + half;
    const float r = __shfl_sync(0xFFFFFFFFu, mine.r, 2 * i + half);
    float xf[8];
    bf16x8_to_f32(v[i], xf);
    if (col_ok && m < M && PACT_IN(m * K + c + 8 <= M * K))
      *reinterpret_cast<uint2*>(q + m * K + c) = e4m3x8(xf, r);
  }
  if (lane < kQRows && m0 + lane < M && PACT_IN((int64_t)kb * 128 < K))
    s[(int64_t)kb * M + m0 + lane] = mine.s;
}

cudaError_t launch_quant_fp8(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, uint8_t* q,
                             float* s, cudaStream_t stream) {
  const uint32_t kb = (uint32_t)((K + 127) / 128);
  const uint32_t units = (uint32_t)((M + kQRows - 1) / kQRows) * kb;
  note_launch();
  k_quant_fp8<<<(units + 7) / 8, 256, 0, stream>>>(x, M, K, ldx, units, FastDiv::make(kb), q, s);
  return cudaGetLastError();
}

// One CTA per 128 x 128 tile of W [N, K]: amax, then the codes of the forward layout
// [N, K] (scales [ceil(N/128), ceil(K/128)]) or of the backward layout [K, N] (codes
// and scales transposed).  Offline: the backward layout goes through shared memory so
// that its stores are coalesced, and that is all the tuning it gets.  W is read twice, the
// second time out of L1 or L2: 8192 x 16384 takes 145 us forward and 167 backward, against
// 99 for one read and one write out of HBM.
__global__ void __launch_bounds__(256)
    k_pack_fp8(const float* __restrict__ W, int64_t N, int64_t K, int backward,
               uint8_t* __restrict__ q, float* __restrict__ s) {
  __shared__ float red[8];
  __shared__ uint8_t tile[128][132];
  const int nkb = (int)((K + 127) / 128), nnb = (int)((N + 127) / 128);
  const int nb = (int)(blockIdx.x / nkb), kb = (int)(blockIdx.x % nkb);
  const int64_t n0 = (int64_t)nb * 128, k0 = (int64_t)kb * 128;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool col_ok = k0 + 4 * lane < K;
  float amax = 0.0f;
  for (int i = warp; i < 128; i += 8)
    if (n0 + i < N && col_ok) {
      const float4 w = *reinterpret_cast<const float4*>(W + (n0 + i) * K + k0 + 4 * lane);
      amax = fmaxf(amax, fmaxf(fmaxf(fabsf(w.x), fabsf(w.y)), fmaxf(fabsf(w.z), fabsf(w.w))));
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  if (lane == 0) red[warp] = amax;
  __syncthreads();
  amax = red[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) amax = fmaxf(amax, red[i]);
  const Fp8Scale f = fp8_scale(amax);
  if (threadIdx.x == 0 && PACT_IN(nb < nnb && kb < nkb))
    s[backward ? (int64_t)kb * nnb + nb : (int64_t)nb * nkb + kb] = f.s;
  for (int i = warp; i < 128; i += 8) {
    if (n0 + i >= N || !col_ok) continue;
    const float4 w = *reinterpret_cast<const float4*>(W + (n0 + i) * K + k0 + 4 * lane);
    const uint32_t c = e4m3x2(__fmul_rn(w.x, f.r), __fmul_rn(w.y, f.r)) |
                       (e4m3x2(__fmul_rn(w.z, f.r), __fmul_rn(w.w, f.r)) << 16);
    if (backward)
      *reinterpret_cast<uint32_t*>(&tile[i][4 * lane]) = c;
    else if (PACT_IN((n0 + i) * K + k0 + 4 * lane + 4 <= N * K))
      *reinterpret_cast<uint32_t*>(q + (n0 + i) * K + k0 + 4 * lane) = c;
  }
  if (!backward) return;
  __syncthreads();
  for (int j = warp; j < 128; j += 8) {  // row k0 + j of the backward layout
    if (k0 + j >= K || n0 + 4 * lane >= N) continue;
    const uint32_t c = tile[4 * lane][j] | (tile[4 * lane + 1][j] << 8) |
                       (tile[4 * lane + 2][j] << 16) | ((uint32_t)tile[4 * lane + 3][j] << 24);
    if (PACT_IN((k0 + j) * N + n0 + 4 * lane + 4 <= N * K))
      *reinterpret_cast<uint32_t*>(q + (k0 + j) * N + n0 + 4 * lane) = c;
  }
}

cudaError_t launch_pack_fp8(const float* W, int64_t N, int64_t K, int backward, uint8_t* q,
                            float* s, cudaStream_t stream) {
  const int64_t tiles = ((N + 127) / 128) * ((K + 127) / 128);
  note_launch();
  k_pack_fp8<<<(unsigned)tiles, 256, 0, stream>>>(W, N, K, backward, q, s);
  return cudaGetLastError();
}

}  // namespace pact
