// FP8 matrix product with a scale for each block of 128 along the reduction:
//
//   OUT[m, n] = bf16( sum_b sx[b, m] sw[n / 128, b] sum_{k in block b} X[m, k] W[n, k]
//                     [+ ADD[m, n]] )
//
// X [M, K] and W [N, K] are E4M3 (K contiguous), sx FP32 [ceil(K/128), M], sw FP32
// [ceil(N/128), ceil(K/128)].  A block's products are summed on the tensor cores in
// FP32; each block's sum is then multiplied by its two scales and added in FP32
// registers, so scales are any FP32 numbers, not powers of two only.  The input
// gradient is the same product on the weight's backward layout.
#include "fp8.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace pact {

// ---------------------------------------------------------------- few tokens
// A CTA computes 16 output columns (rows of W) for up to 8 NT tokens; its warps share
// the blocks of K among them and add their sums through shared memory in warp order.
// The product is turned: W is the row operand (16 rows) and the tokens the column
// operand (8 each), so that a single token wastes 7/8 of the tensor work but none of
// the reads.  Within a block, lane 4 g + t holds the 16-byte pieces t and t + 4 of row
// g: the order of k inside the contraction is free as long as both operands use the
// same one, so the fragments come straight from global memory, 64 contiguous bytes of
// a row per access.
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kFewWarps = 8;

template <int NT>
__global__ void __launch_bounds__(32 * kFewWarps)
    k_fp8_few(const uint8_t* __restrict__ x, const float* __restrict__ sx,
              const uint8_t* __restrict__ w, const float* __restrict__ sw, int64_t M, int64_t N,
              int64_t K, const uint16_t* add, uint16_t* out) {
  __shared__ float sums[kFewWarps][16][8 * NT + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * (8 * NT);
  const int nkb = (int)((K + 127) / 128);
  float acc[NT][4] = {};
  for (int kb = warp; kb < nkb; kb += kFewWarps) {
    const int64_t k0 = (int64_t)kb * 128 + 16 * t;
    uint4 a[2][2], b[NT][2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int64_t k = k0 + 64 * c;
      const bool ok = k < K;
      const uint4 z = make_uint4(0u, 0u, 0u, 0u);
      a[0][c] = ok ? *reinterpret_cast<const uint4*>(w + (n0 + g) * K + k) : z;
      a[1][c] = ok ? *reinterpret_cast<const uint4*>(w + (n0 + g + 8) * K + k) : z;
#pragma unroll
      for (int j = 0; j < NT; ++j)
        b[j][c] = ok && m0 + 8 * j + g < M
                      ? *reinterpret_cast<const uint4*>(x + (m0 + 8 * j + g) * K + k)
                      : z;
    }
    const float s = sw[(n0 >> 7) * nkb + kb];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float d[4] = {};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        mma_e4m3(d, a[0][c].x, a[1][c].x, a[0][c].y, a[1][c].y, b[j][c].x, b[j][c].y);
        mma_e4m3(d, a[0][c].z, a[1][c].z, a[0][c].w, a[1][c].w, b[j][c].z, b[j][c].w);
      }
      const int64_t m = m0 + 8 * j + 2 * t;  // the token of d[0] and d[2]; d[1], d[3]: m + 1
      const float s0 = m < M ? __fmul_rn(sx[(int64_t)kb * M + m], s) : 0.0f;
      const float s1 = m + 1 < M ? __fmul_rn(sx[(int64_t)kb * M + m + 1], s) : 0.0f;
      acc[j][0] = __fmaf_rn(d[0], s0, acc[j][0]);
      acc[j][1] = __fmaf_rn(d[1], s1, acc[j][1]);
      acc[j][2] = __fmaf_rn(d[2], s0, acc[j][2]);
      acc[j][3] = __fmaf_rn(d[3], s1, acc[j][3]);
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[warp][g + 8 * (i >> 1)][8 * j + 2 * t + (i & 1)] = acc[j][i];
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * 8 * NT; i += 32 * kFewWarps) {
    const int n = i & 15, m = i >> 4;
    if (m0 + m >= M) break;
    float v = sums[0][n][m];
#pragma unroll
    for (int k = 1; k < kFewWarps; ++k) v += sums[k][n][m];
    const int64_t at = (m0 + m) * N + n0 + n;
    if (add) v += __uint_as_float((uint32_t)add[at] << 16);
    if (PACT_IN(at < M * N)) out[at] = (uint16_t)(pack_bf16x2(v, v) & 0xFFFFu);
  }
}

template <int NT>
static cudaError_t launch_few(const uint8_t* x, const float* sx, const uint8_t* w,
                              const float* sw, int64_t M, int64_t N, int64_t K,
                              const uint16_t* add, uint16_t* out, cudaStream_t stream) {
  const dim3 grid((unsigned)(N / 16), (unsigned)((M + 8 * NT - 1) / (8 * NT)));
  note_launch();
  k_fp8_few<NT><<<grid, 32 * kFewWarps, 0, stream>>>(x, sx, w, sw, M, N, K, add, out);
  return cudaGetLastError();
}

cudaError_t launch_fp8_few(const uint8_t* x, const float* sx, const uint8_t* w, const float* sw,
                           int64_t M, int64_t N, int64_t K, const uint16_t* add, uint16_t* out,
                           cudaStream_t stream) {
  if (M <= 8) return launch_few<1>(x, sx, w, sw, M, N, K, add, out, stream);
  if (M <= 16) return launch_few<2>(x, sx, w, sw, M, N, K, add, out, stream);
  return launch_few<4>(x, sx, w, sw, M, N, K, add, out, stream);
}

}  // namespace pact
