// The norm of many gradients together, and clipping by it:
//   norm = sqrt(sum over all values g^2);  coef = min(1, max_norm / (norm + 1e-6));
//   out = g coef.
//
// Bound by HBM: every value is read for the norm, and read and written again where it is
// clipped.  The tensors of a list are cut into chunks of 4096 values; a grid of blocks takes
// the chunks in turn and writes one FP64 sum a block.  The second launch, which every block
// opens by adding those sums in the same order, takes the chunks from the last to the first:
// what the norm read last is still in L2, and what is read and written there need not stay.
// 83.9 M values into another buffer: 162 us, 1.0 GB of traffic at 6.2 TB/s.
//
// Squares are added in FP32 over 16 values of a thread, four such sums again in FP32, and
// those in FP64.  A thread whose largest value of the 16 lies outside [2^-50, 2^60], where an
// FP32 square could overflow or vanish, adds them in FP64 instead.
#include "common.cuh"
#include "kernels.h"

namespace pact {

constexpr int kGradThreads = 256;
// Chunks at the end of the list that the first pass leaves in L2 for the second: 64 MB.
constexpr int64_t kGradKept = 4096;
static_assert(kGradChunk == kGradThreads * 16, "a thread has four vectors of a chunk");

struct GradSpan {
  int64_t tensor, at;
  int len;
};

// The tensor and the values of chunk c: the last tensor whose first chunk is not behind it,
// looked for from tensor `lo` on, 32 places at a time.  Every lane of the warp calls this.
__device__ __forceinline__ GradSpan grad_span(const GradTable& t, int64_t c, int64_t lo) {
  const int lane = threadIdx.x & 31;
  for (int64_t n = t.count - lo; n > 1;) {
    const int64_t step = (n + 31) >> 5, at = lane * step;
    const unsigned not_behind = __ballot_sync(0xFFFFFFFFu, at < n && t.first[at < n ? lo + at : lo] <= c);
    const int64_t by = (31 - __clz(not_behind)) * step;  // lane 0 is always among them
    lo += by;
    n = n - by < step ? n - by : step;
  }
  GradSpan s;
  s.tensor = lo;
  s.at = (c - t.first[lo]) * kGradChunk;
  const int64_t left = t.numel[lo] - s.at;
  s.len = (int)(left < kGradChunk ? left : kGradChunk);
  return s;
}

// The block's sum, in thread 0.
__device__ __forceinline__ double block_sum(double v, double* slots) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < kGradThreads / 32; ++i) s += slots[i];
  }
  return s;
}

__global__ void __launch_bounds__(kGradThreads, kGradBlocks)
    k_grad_sums(const GradTable t, double* part) {
  __shared__ double slots[kGradThreads / 32];
  double sum = 0.0;
  float few = 0.0f;  // of up to four chunks
  int held = 0;
  int64_t c = blockIdx.x;
  GradSpan sp = {};
  if (c < t.chunks) sp = grad_span(t, c, 0);
  while (c < t.chunks) {
    const float* g = t.data[sp.tensor] + sp.at;
    float4 v[4];
    const bool vec = ((uintptr_t)g & 15u) == 0, keep = t.chunks - c <= kGradKept;
    if (vec && sp.len == kGradChunk) {
      const float4* at = reinterpret_cast<const float4*>(g) + threadIdx.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = keep ? at[i * kGradThreads] : __ldcs(at + i * kGradThreads);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = (i * kGradThreads + (int)threadIdx.x) * 4;
        v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (e < sp.len) v[i].x = g[e];
        if (e + 1 < sp.len) v[i].y = g[e + 1];
        if (e + 2 < sp.len) v[i].z = g[e + 2];
        if (e + 3 < sp.len) v[i].w = g[e + 3];
      }
    }
    // the next chunk is looked up while these values are on their way
    c += gridDim.x;
    if (c < t.chunks) sp = grad_span(t, c, sp.tensor);
    float s = 0.0f, top = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s += v[i].x * v[i].x + v[i].y * v[i].y + (v[i].z * v[i].z + v[i].w * v[i].w);
      top = fmaxf(fmaxf(fmaxf(top, fabsf(v[i].x)), fabsf(v[i].y)),
                  fmaxf(fabsf(v[i].z), fabsf(v[i].w)));
    }
    if (top <= 0x1p60f && !(top < 0x1p-50f && top > 0.0f)) {
      few += s;
      if (++held == 4) {
        sum += (double)few;
        few = 0.0f;
        held = 0;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sum += (double)v[i].x * v[i].x;
        sum += (double)v[i].y * v[i].y;
        sum += (double)v[i].z * v[i].z;
        sum += (double)v[i].w * v[i].w;
      }
    }
  }
  sum = block_sum(sum + (double)few, slots);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// APPLY: clip into out (which may be the list itself); else the norm alone, by one block.
template <bool APPLY>
__global__ void __launch_bounds__(kGradThreads, kGradBlocks)
    k_grad_clip(const GradTable t, float* const* out, const double* part, int parts,
                double max_norm, float* norm_out) {
  __shared__ double slots[kGradThreads / 32];
  double sum = 0.0;
  for (int i = threadIdx.x; i < parts; i += kGradThreads) sum += part[i];
  sum = block_sum(sum, slots);
  __shared__ float shared_coef;
  if (threadIdx.x == 0) {  // alone: FP64 is slow, and a warp takes as long as a thread
    // In FP32 where the sum, the norm and the limit are far from its ends: an FP64 root and
    // quotient are 2 us of latency, and either is rounded to FP32 in the end.
    const bool usual = sum > 1e-30 && sum < 1e30 && max_norm < 1e30;
    const double norm = usual ? (double)__fsqrt_rn((float)sum) : sqrt(sum);
    if (blockIdx.x == 0) *norm_out = (float)norm;
    if constexpr (APPLY) {
      const double q = usual ? (double)__fdiv_rn((float)max_norm, (float)norm + 1e-6f)
                             : max_norm / (norm + 1e-6);
      shared_coef = q > 1.0 ? 1.0f : (float)q;  // a NaN stays one
    }
  }
  if constexpr (APPLY) {
    __syncthreads();
    const float coef = shared_coef;
    for (int64_t i = blockIdx.x; i < t.chunks; i += gridDim.x) {
      const GradSpan sp = grad_span(t, t.chunks - 1 - i, 0);
      const float* g = t.data[sp.tensor] + sp.at;
      float* o = out[sp.tensor] + sp.at;
      if (o == g && coef == 1.0f) continue;  // nothing to clip
      if ((((uintptr_t)g | (uintptr_t)o) & 15u) == 0) {
        float4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = (j * kGradThreads + (int)threadIdx.x) * 4;
          if (e + 4 <= sp.len) v[j] = __ldcs(reinterpret_cast<const float4*>(g + e));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = (j * kGradThreads + (int)threadIdx.x) * 4;
          if (e + 4 <= sp.len) {
            __stcs(reinterpret_cast<float4*>(o + e),
                   make_float4(v[j].x * coef, v[j].y * coef, v[j].z * coef, v[j].w * coef));
          } else {
            for (int k = e; k < sp.len; ++k) o[k] = g[k] * coef;
          }
        }
      } else {
        for (int e = threadIdx.x; e < sp.len; e += kGradThreads) o[e] = g[e] * coef;
      }
    }
  }
}

int64_t grad_norm_blocks(int64_t chunks, int num_sms) {
  const int64_t most = (int64_t)kGradBlocks * num_sms;
  return chunks < 1 ? 1 : (chunks < most ? chunks : most);
}

cudaError_t launch_grad_norm(const GradTable& t, float* const* out, double max_norm, float* norm,
                             double* part, int num_sms, cudaStream_t st) {
  const int blocks = (int)grad_norm_blocks(t.chunks, num_sms);
  note_launch();
  k_grad_sums<<<blocks, kGradThreads, 0, st>>>(t, part);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  note_launch();
  if (out)
    k_grad_clip<true><<<blocks, kGradThreads, 0, st>>>(t, out, part, blocks, max_norm, norm);
  else
    k_grad_clip<false><<<1, kGradThreads, 0, st>>>(t, out, part, blocks, max_norm, norm);
  return cudaGetLastError();
}

}  // namespace pact
