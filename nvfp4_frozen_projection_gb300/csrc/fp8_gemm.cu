// FP8 matrix product with a scale for each block of 128 along the reduction:
//
//   OUT[m, n] = bf16( sum_b sx[b, m] sw[n / 128, b] sum_{k in block b} X[m, k] W[n, k]
//                     [+ ADD[m, n]] )
//
// X [M, K] and W [N, K] are E4M3 (K contiguous), sx FP32 [ceil(K/128), M], sw FP32
// [ceil(N/128), ceil(K/128)].  A block's products are summed on the tensor cores in
// FP32; each block's sum is then multiplied by its two scales and added in FP32
// registers, so scales need not be powers of two.  The two scales are multiplied first, in
// FP32: a product below 2^-126 (block maxima near 2^-117 against ordinary weights) has
// fewer than 24 bits.  The input gradient is the same product on the weight's backward
// layout.
#include "fp8.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

#include <atomic>
#include <cmath>
#include <type_traits>

namespace pact {

// ---------------------------------------------------------------- few tokens
// A CTA computes 16 output columns (rows of W) for 8 or 16 tokens; its warps share the
// blocks of K among them and add their sums through shared memory in warp order.  Further
// tokens are other CTAs' (blockIdx.y), which read the weight out of L2: 32 x 2048 x 2048
// 4.0 us, against 6.0 with 32 tokens a CTA and 7.8 on tcgen05.
// The product is turned: W is the row operand (16 rows) and the tokens the column
// operand (8 each), so that a single token wastes 7/8 of the tensor work but none of
// the reads.  Within a block, lane 4 g + t holds the 16-byte pieces t and t + 4 of row
// g: the order of k inside the contraction is free as long as both operands use the
// same one, so a fragment is a 16-byte read.
// The weight's way out of HBM bounds it: 1 x 8192 x 8192 takes 13.9 us (4.8 TB/s) with up
// to 128 KB of the weight an SM on their way into shared memory; with the next block's
// fragments on their way into registers it took 17.6.  A weight that stays in L2 from one
// call to the next is faster (1 x 8192 x 8192 11.3, 1 x 4096 x 8192 6.5 against 8.8).
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A block's scales, of a lane's tokens and of the weight.
template <int NT>
struct FewScales {
  float s0[NT], s1[NT], sw;
};

// WARPS share the blocks of K.  Each has a ring in shared memory, filled by asynchronous
// copies, whose stages hold a block's 16 rows of W and 8 NT rows of X, 128 bytes each; row
// r's 16-byte piece p lies at p ^ 4 (r % 2), so that a quarter warp's reads, four pieces of
// two rows, meet no bank twice.  The next block's scales are loaded while this one is
// multiplied.
template <int NT>
struct FewCfg {
  static constexpr int DEPTH = NT == 1 ? 4 : 3;
  static constexpr int STAGE = 2048 + NT * 1024;
};

template <int NT, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 16 / WARPS)
    k_fp8_few(const uint8_t* __restrict__ x, const float* __restrict__ sx,
              const uint8_t* __restrict__ w, const float* __restrict__ sw, int64_t M, int64_t N,
              int64_t K, const uint16_t* add, uint16_t* out) {
  __shared__ float sums[WARPS][16][8 * NT + 1];
  extern __shared__ uint4 few_ring[];
  constexpr int DEPTH = FewCfg<NT>::DEPTH, STAGE = FewCfg<NT>::STAGE;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int nkb = (int)((K + 127) / 128);
  const int64_t m0 = (int64_t)blockIdx.y * 8 * NT;
  const float* swr = sw + (n0 >> 7) * nkb;
  const uint32_t ring = smem_addr(few_ring) + (uint32_t)warp * (DEPTH * STAGE);
  // lane l copies piece l % 8 of the rows l / 8 + 4 i
  const int cr = lane >> 3, cp = lane & 7;
  const uint8_t* wc = w + (n0 + cr) * K + 16 * cp;
  const uint8_t* xc = x + (m0 + cr) * K + 16 * cp;
  const uint32_t cdst = ring + (uint32_t)(cr * 128 + ((cp ^ ((cr & 1) << 2)) << 4));
  auto fetch = [&](int kb, int stage) {
    if (kb < nkb) {
      const bool ok = (int64_t)kb * 128 + 16 * cp < K;  // K % 16 == 0: a piece is in or out
      const int64_t k0 = (int64_t)kb * 128;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        cp_async16(cdst + (uint32_t)(stage * STAGE + i * 512), ok ? wc + k0 + i * 4 * K : w,
                   ok ? 16u : 0u);
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i) {  // zeros past K and past the last token
        const bool in = ok && m0 + cr + 4 * i < M;
        cp_async16(cdst + (uint32_t)(stage * STAGE + 2048 + i * 512),
                   in ? xc + k0 + i * 4 * K : x, in ? 16u : 0u);
      }
    }
    cp_async_commit();
  };
  // rows g and g + 8, pieces t and t + 4
  const uint32_t rsrc = ring + (uint32_t)(g * 128), sw0 = (uint32_t)((t ^ ((g & 1) << 2)) << 4);
  auto load = [&](int kb, FewScales<NT>& f) {
    f.sw = swr[kb];
#pragma unroll
    for (int j = 0; j < NT; ++j) {  // the tokens of d[0] and d[2], d[1] and d[3]
      const int64_t m = m0 + 8 * j + 2 * t;
      f.s0[j] = m < M ? sx[(int64_t)kb * M + m] : 0.0f;
      f.s1[j] = m + 1 < M ? sx[(int64_t)kb * M + m + 1] : 0.0f;
    }
  };
  float acc[NT][4] = {};
  FewScales<NT> cur, next;
#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i) fetch(warp + i * WARPS, i);
  if (warp < nkb) load(warp, cur);
  int stage = 0;
  for (int kb = warp; kb < nkb; kb += WARPS) {
    __syncwarp();  // the block before has been read out of the stage that is filled now
    fetch(kb + (DEPTH - 1) * WARPS, stage == 0 ? DEPTH - 1 : stage - 1);
    if (kb + WARPS < nkb) load(kb + WARPS, next);
    cp_async_wait<DEPTH - 1>();
    __syncwarp();  // every lane's copies of this block have landed
    uint4 a[2 + NT][2];  // two groups of eight rows of W, then the tokens
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < 2 + NT; ++i)
        a[i][c] = ld_shared_v4(rsrc + (uint32_t)(stage * STAGE + i * 1024) + (sw0 ^ (64u * c)));
    if (++stage == DEPTH) stage = 0;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float d[4] = {};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        mma_e4m3(d, a[0][c].x, a[1][c].x, a[0][c].y, a[1][c].y, a[2 + j][c].x, a[2 + j][c].y);
        mma_e4m3(d, a[0][c].z, a[1][c].z, a[0][c].w, a[1][c].w, a[2 + j][c].z, a[2 + j][c].w);
      }
      const float s0 = __fmul_rn(cur.s0[j], cur.sw), s1 = __fmul_rn(cur.s1[j], cur.sw);
      acc[j][0] = __fmaf_rn(d[0], s0, acc[j][0]);
      acc[j][1] = __fmaf_rn(d[1], s1, acc[j][1]);
      acc[j][2] = __fmaf_rn(d[2], s0, acc[j][2]);
      acc[j][3] = __fmaf_rn(d[3], s1, acc[j][3]);
    }
    cur = next;
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[warp][g + 8 * (i >> 1)][8 * j + 2 * t + (i & 1)] = acc[j][i];
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * 8 * NT; i += 32 * WARPS) {
    const int n = i & 15, m = i >> 4;
    if (m0 + m >= M) break;
    float v = sums[0][n][m];
#pragma unroll
    for (int k = 1; k < WARPS; ++k) v += sums[k][n][m];
    const int64_t at = (m0 + m) * N + n0 + n;
    if (add) v += __uint_as_float((uint32_t)add[at] << 16);
    if (PACT_IN(at < M * N)) out[at] = (uint16_t)(pack_bf16x2(v, v) & 0xFFFFu);
  }
}

template <int NT, int WARPS>
static cudaError_t launch_few(const uint8_t* x, const float* sx, const uint8_t* w,
                              const float* sw, int64_t M, int64_t N, int64_t K,
                              const uint16_t* add, uint16_t* out, cudaStream_t stream) {
  constexpr int ring = WARPS * FewCfg<NT>::DEPTH * FewCfg<NT>::STAGE;
  static std::atomic<uint64_t> attribute_set;  // a bit per device
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64) return cudaErrorInvalidDevice;
  if (!(attribute_set.load(std::memory_order_acquire) >> dev & 1)) {
    cudaError_t e = cudaFuncSetAttribute(k_fp8_few<NT, WARPS>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, ring);
    if (e != cudaSuccess) return e;
    attribute_set.fetch_or((uint64_t)1 << dev, std::memory_order_release);
  }
  note_launch();
  k_fp8_few<NT, WARPS><<<dim3((unsigned)(N / 16), (unsigned)((M + 8 * NT - 1) / (8 * NT))),
                         32 * WARPS, ring, stream>>>(x, sx, w, sw, M, N, K, add, out);
  return cudaGetLastError();
}

// Warps a CTA: 16 where each CTA has an SM to itself, 8 where two of those share one, else
// 4 (us with 16, 8, 4): 1 x 2048 x 8192 4.5, 4.9, 6.0; 1 x 4096 x 4096 5.2, 4.4, 4.6;
// 1 x 8192 x 8192 18.9, 15.7, 14.1; 64 x 2048 x 2048 8.8, 6.2, 5.7.
static int few_warps(int64_t M, int64_t N, int sms) {
  const int64_t ctas = (N / 16) * ((M + 15) / 16);
  return ctas <= sms ? 16 : (ctas <= 2 * sms ? 8 : 4);
}

cudaError_t launch_fp8_few(const uint8_t* x, const float* sx, const uint8_t* w, const float* sw,
                           int64_t M, int64_t N, int64_t K, const uint16_t* add, uint16_t* out,
                           int sms, cudaStream_t stream) {
  const int warps = few_warps(M, N, sms);
#define PACT_FEW(NT)                                                                       \
  (warps == 16  ? launch_few<NT, 16>(x, sx, w, sw, M, N, K, add, out, stream)              \
   : warps == 8 ? launch_few<NT, 8>(x, sx, w, sw, M, N, K, add, out, stream)               \
                : launch_few<NT, 4>(x, sx, w, sw, M, N, K, add, out, stream))
  return M <= 8 ? PACT_FEW(1) : PACT_FEW(2);
#undef PACT_FEW
}

// ---------------------------------------------------------------- which kernel
// The estimated time (us) of each way to run a product decides.  The constants are fitted
// to GB300 measurements of M 1 .. 8192, N 512 .. 131072, K 512 .. 28672 (launch included;
// b = blocks of 128 along K); smaller products follow the same formulas.
//   few     up to 8 tokens 2.2 + the whole waves of resident CTAs + the last one.  A wave
//           that fills `full` of the places takes the longer of its bytes of W at 6.2e6 a us
//           and 0.5 + (0.3 + 0.4 full + 0.012 (M - 1)) blocks of a warp.
//           More tokens: 2.2 + the longer of N K / 4.3e6 and waves (0.5 + 0.9 blocks of a
//           warp)                        16 x 4096 x 4096 5.8 us; 24 x 2048 x 2048 4.0;
//                                        256 x 512 x 512 3.1
//   tiles   2.7 + waves (1.2 + 0.27 b)   512 x 2048 x 512 5.0; 128 x 4096 x 8192 21.4;
//                                        8192 x 4096 x 8192 263
//   shared  6.3 + 0.29 b / CTAs          128 x 4096 x 8192 12.5; 512 x 1024 x 16384 15.8
//   pairs   5.0 + waves (1.5 + 0.41 b)   256 x 4096 x 8192 31.4; 2048 x 2048 x 2048 12.9;
//                                        8192 x 4096 x 8192 196
// and none but `few` under the weight's way out of HBM: 4.5 + N K / 6.2e6 up to 8 tokens,
// 3 + N K / 5.6e6 beyond.  Sharing a tile's blocks among a cluster's CTAs helps where there
// are few tiles; clusters of three or four with this much shared memory fill 128 of 152 SMs,
// pairs all of them.
// Up to 8 tokens, with weights that come out of HBM (us; few, the best other way; the one
// taken first):
//   1 x  8192 x  8192  few 13.9, shared 17.3     1 x 28672 x  8192  few 37.9, tiles 45.0
//   1 x  8192 x 16384  few 24.8, shared 27.6     1 x 16384 x 16384  few 46.4, tiles 48.8
//   1 x 14336 x 14336  tiles 37.6, few 39.3      8 x 12288 x 12288  tiles 30.9, few 37.1
//   1 x  5120 x 13824  few 17.2, shared 18.7     8 x 10240 x  8192  tiles 20.6, few 22.8
// Of 32 weights at 1, 2, 5 and 8 tokens the estimate takes the slower way for six products,
// which then take 2 to 6 % longer (2 x 5120 x 13824: shared 18.7, few 17.7).
enum Fp8Way { kFew, kTiles, kShared, kPairs };
struct Fp8Plan {
  Fp8Way way;
  int split;
  int64_t whole;  // pairs: the tiles before a last wave of halves, 0 without one
};
static Fp8Plan fp8_plan(int64_t M, int64_t N, int64_t K, int sms) {
  Fp8Plan p = {kFew, 1, 0};
  const double b = (double)((K + 127) / 128);
  const double tiles = (double)((M + 127) / 128) * (double)((N + 127) / 128);
  double best = 2.7 + std::ceil(tiles / sms) * (1.2 + 0.27 * b);
  p.way = kTiles;
  for (int s = 2; s <= 4; ++s) {
    const double t = 6.3 + 0.29 * std::ceil(b / s);
    if (tiles * s <= (s == 2 ? sms : sms * 128 / 152) && b >= 2 * s && t < best) {
      best = t;
      p.way = kShared;
      p.split = s;
    }
  }
  if (M > 128 && N > 128) {
    const double pairs = (double)((M + 255) / 256) * (double)((N + 255) / 256);
    // tiles left over for at most half the pairs go as halves, in a launch of their own
    // (5 us), where that beats a wave of whole ones: 8192 x 2048 x 16384 took 225 us with
    // a wave of 28 tiles and takes 209 with 56 halves
    const double wave = 1.5 + 0.41 * b, full = std::floor(pairs / (sms / 2));
    const double left = pairs - full * (sms / 2);
    const bool halves = full > 0 && left > 0 && 2 * left <= sms / 2 && 5.0 + 0.65 * wave < wave;
    const double t = 5.0 + full * wave + (left == 0 ? 0.0 : (halves ? 5.0 + 0.65 * wave : wave));
    if (t < best) {
      best = t;
      p.way = kPairs;
      p.split = 1;
      p.whole = halves ? (int64_t)(full * (sms / 2)) : 0;
    }
  }
  const double weight = (double)N * (double)K;
  const int warps = few_warps(M, N, sms);
  const double ctas = (double)(N / 16) * (double)((M + 15) / 16);
  const double slots = 16.0 * sms / warps;  // resident CTAs
  const double rounds = std::ceil(b / warps);
  double few, floor;
  if (M <= 8) {
    auto wave = [&](double full) {
      return std::fmax(full * slots * 16.0 * (double)K / 6.2e6,
                       0.5 + (0.3 + 0.4 * full + 0.012 * (double)(M - 1)) * rounds);
    };
    const double whole = std::ceil(ctas / slots) - 1.0;
    few = 2.2 + whole * wave(1.0) + wave(ctas / slots - whole);
    floor = 4.5 + weight / 6.2e6;
  } else {
    few = 2.2 + std::fmax(weight / 4.3e6, std::fmax(1.0, ctas / slots) * (0.5 + 0.9 * rounds));
    floor = 3.0 + weight / 5.6e6;
  }
  // up to 1024 tokens, beyond which nothing was measured (and the grid would grow too high)
  if (M <= 1024 && few < std::fmax(best, floor)) p.way = kFew;
  return p;
}

void fp8_plan_of(int64_t M, int64_t N, int64_t K, int sms, int64_t plan[3]) {
  const Fp8Plan p = fp8_plan(M, N, K, sms);
  plan[0] = p.way;
  plan[1] = p.way == kFew ? few_warps(M, N, sms) : (p.way == kShared ? p.split : 1);
  plan[2] = p.way == kPairs ? p.whole : 0;
}

bool fp8_is_few(int64_t M, int64_t N, int64_t K, int sms) {
  return fp8_plan(M, N, K, sms).way == kFew;
}

// ---------------------------------------------------------------- many tokens
// A persistent CTA per SM (128 x 128 tiles), or CTA pair (cluster of two along M,
// .cta_group::2, 256 x 256 tiles).  Per block of K (128 bytes of a row, one ring stage)
// the tensor cores write fresh accumulators; the epilogue warps multiply them by the
// block's scales and add them to sums in registers while the next MMAs run into other
// accumulator buffers.  A thread owns one row, and a warp's columns lie in one block of
// 128 outputs, so a block's two scales are a single factor per thread.
//
// All 512 TMEM columns pass once per round of MMA, commit, the epilogue's wait, its
// loads, its arrival and the issuer's wait, so a pair's 256 columns of a block are two
// sub-blocks of 128 (64 rows of W from each CTA), freed one by one.
//   warp 0      TMA producer: X and W tiles (128-byte rows, 128B swizzle) into the ring
//               (in a pair, each CTA's copies signal the leader's barriers)
//   warps 1-2   MMA issuers (in a pair, the leader's), warp 1 the TMEM allocator
//   warp 3      the blocks' scales, up to 16 blocks ahead, into a ring of their own
//   warps 4-11  epilogue: two warps per TMEM lane quarter, each half of the columns
// The first warpgroup gives its registers to the epilogue, whose threads hold 128 sums
// and the columns that land.
//
// 8192 x 4096 x 8192 takes 196 to 200 us (2.8 PFLOP/s, 0.75 of twice the measured BF16 rate).
// When it took 203, it took 193 without the additions and 153 with one barrier round for
// 16 blocks instead of one: what is left is that round.  Measured and not kept, all at
// this size: 16 epilogue warps of 64 columns (232 us), loads carried over from one block to
// the next (238, it spills), an issuer and a barrier for each sub-block with epilogue
// warps that take both sub-blocks (238) or one each (230), the same with two issuers
// (205), slices of 32 columns (200, no difference).  Runs differ by 5 % with where the
// tensors lie in memory.
template <bool PAIR>
struct Fp8Cfg {
  static constexpr int STAGES = 6;
  static constexpr int CM = PAIR ? 2 : 1;
  static constexpr int BN = PAIR ? 256 : 128;
  static constexpr int NSUB = PAIR ? 2 : 1;  // sub-blocks of a block
  static constexpr int CYC = PAIR ? 2 : 4;   // blocks with accumulators in TMEM
  static constexpr int NBUF = CYC * NSUB;    // buffers of 128 columns
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = 128 * 128;  // 128 rows of W in this CTA's shared memory
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  // ring of the scales, one slot per block: sx of 128 rows, sw of the warps' two halves;
  // one barrier for each half of the ring
  static constexpr int SCL_OFF = STAGES * STAGE_BYTES;
  static constexpr int SCL_SLOT = 128 * 4 + 16;
  static constexpr int SCL_DEPTH = 16, SCL_HALF = SCL_DEPTH / 2;
  // output staging: per epilogue warp 32 rows x 32 BF16 columns, 64-byte swizzled rows
  static constexpr int STG_OFF = (SCL_OFF + SCL_DEPTH * SCL_SLOT + 1023) / 1024 * 1024;
  static constexpr int STG_BUF = 2048;
  static constexpr int BAR_OFF = STG_OFF + 8 * STG_BUF;
  static constexpr int SMEM_BYTES = BAR_OFF + 512 + 1024;  // + barriers + alignment slack
  static constexpr int THREADS = 384;
  // registers a thread: at launch (65536 / 384 threads, a multiple of 8), and the
  // shares of the first and of the two epilogue warpgroups
  static constexpr int LAUNCH_REGS = 168, LOW_REGS = 56, EPI_REGS = 224;
  static_assert(LOW_REGS + 2 * EPI_REGS <= 3 * LAUNCH_REGS, "register shares");
  static constexpr int EPI_WARPS = 8;
  static constexpr int EPI_COLS = BN / 2;  // columns of an epilogue warp, 64 of a sub-block
  // Two issuers take the blocks in turn.  An accumulator's blocks all come from one of
  // them, and before it asks for a buffer it has been given the one two blocks earlier:
  // no thread is ever two rounds ahead, where a barrier's parity looks the same.
  static constexpr int ISSUERS = 2;
  static constexpr int ROUND = PAIR ? 6 : 12;  // blocks until ring and buffers repeat together
  // barriers: full[S], empty[S], acc_full[CYC], acc_empty[NBUF], scl_full[2],
  // scl_empty[2], final
  static constexpr int NBARS = 2 * STAGES + CYC + NBUF + 5;
  static_assert(BAR_OFF % 8 == 0 && NBARS * 8 <= 504 && SMEM_BYTES <= 232448, "shared memory");
  static_assert(ROUND % STAGES == 0 && ROUND % CYC == 0 && CYC % ISSUERS == 0, "turns");
  static_assert(NBUF * 128 <= 512, "TMEM columns");
};

__host__ __device__ constexpr uint32_t idesc_e4m3(int n, int m) {
  // D = F32 (bits 4-5 = 1), A = B = E4M3 (0)
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

constexpr int kMaxSplit = 4;  // CTAs that share the blocks of one tile
constexpr uint64_t kFp8WaitNs = 2000000000ull;  // 2 s per pipeline wait

// PART: the units are halves (128 columns) of a pair's tiles, for the tiles that do not
// fill a last wave.  Every block still goes round both sub-blocks' buffers, the second
// unused.
template <bool PAIR, bool SPLIT, bool ADD, bool PART>
__global__ void __launch_bounds__(384, 1)
    k_fp8_gemm(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
               const __grid_constant__ CUtensorMap tmOut, const Fp8GemmParams p) {
  using C = Fp8Cfg<PAIR>;
  constexpr int STAGES = C::STAGES, CM = C::CM, BN = C::BN, NSUB = C::NSUB, NBUF = C::NBUF;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t full0 = base + C::BAR_OFF, empty0 = full0 + 8 * STAGES;
  const uint32_t accf0 = empty0 + 8 * STAGES, acce0 = accf0 + 8 * C::CYC;
  const uint32_t sclf0 = acce0 + 8 * NBUF, scle0 = sclf0 + 16;
  const uint32_t final_bar = scle0 + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::BAR_OFF + 504);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::BAR_OFF + 508);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  static_assert(!(PAIR && SPLIT), "a cluster is a pair or shares the blocks of one tile");
  static_assert(PAIR || !PART, "halves of a pair's tile");
  const uint32_t crank = PAIR ? cluster_ctarank() : 0u;
  const int num_mc = (p.num_m + CM - 1) / CM;
  const int nunits = p.units;
  const int csize = SPLIT ? p.split : CM;  // CTAs of a cluster
  const int unit0 = (int)blockIdx.x / csize, nclusters = (int)gridDim.x / csize;
  // the blocks of K that this CTA adds up
  const uint32_t krank = SPLIT ? cluster_ctarank() : 0u;
  const int kb0 = SPLIT ? (int)((int64_t)p.nkb * krank / p.split) : 0;
  const int nk = (SPLIT ? (int)((int64_t)p.nkb * (krank + 1) / p.split) : p.nkb) - kb0;
  const int band = p.band_mc;
  // Waits on barriers that are signalled from outside this CTA in a pair.  wait_x: the
  // copies, and the stages that MMAs have read.  wait_tmem: accumulators that are full, and
  // buffers that are free.  What these order are MMAs and TMEM reads alone, which
  // tcgen05.wait::ld and the tcgen05 fences on both sides keep in place, so releases and
  // waits are relaxed (8192 x 4096 x 8192 208.5 us, 211.5 with waits that acquire).
  auto wait_x_for = [&](uint32_t bar, uint32_t par, uint64_t ns, const volatile uint32_t* flag) {
    return PAIR ? mbar_wait_cluster(bar, par, ns, flag) : mbar_wait(bar, par, ns, flag);
  };
  auto wait_x = [&](uint32_t bar, uint32_t par) {
    return wait_x_for(bar, par, kFp8WaitNs, abort_flag);
  };
  auto wait_tmem = [&](uint32_t bar, uint32_t par) {
    return PAIR ? mbar_wait_cluster<true>(bar, par, kFp8WaitNs, abort_flag)
                : mbar_wait(bar, par, kFp8WaitNs, abort_flag);
  };
  // the first row and column of unit u
  auto unit_mn = [&](int u, int& m0, int& n0) {
    const int t = p.first + (PART ? u >> 1 : u);
    const int bi = t / (band * p.num_n), r = t - bi * band * p.num_n;
    const int mc0 = bi * band, bm = min(band, num_mc - mc0);
    const int n = r / bm;
    m0 = ((mc0 + (r - n * bm)) * CM + (int)crank) * 128;
    n0 = n * BN + (PART ? 128 * (u & 1) : 0);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < C::CYC; ++b) mbar_init(accf0 + 8 * b, 1);
    // one arrival per epilogue warp of each CTA
    for (int b = 0; b < NBUF; ++b) mbar_init(acce0 + 8 * b, C::EPI_WARPS * CM);
    for (int i = 0; i < 2; ++i) {
      mbar_init(sclf0 + 8 * i, 32);  // the lanes of the scale warp
      mbar_init(scle0 + 8 * i, C::EPI_WARPS);
    }
    mbar_init(final_bar, C::ISSUERS);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmX);
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmOut);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_addr(tmem_slot), 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_addr(tmem_slot), 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // the peer's barriers are initialised
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (warp < 4) {
    setmaxnreg_dec<C::LOW_REGS>();  // the same instruction for the whole warpgroup
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- TMA producer
      const uint32_t lead_full0 = PAIR ? cluster_addr(full0, 0) : full0;
      uint32_t pend = 0, pend_par = 0, phase = 0;
      int stage = 0;
      bool ok = true;
      for (int u = unit0; u < nunits && ok; u += nclusters) {
        int m0, n0;
        unit_mn(u, m0, n0);
        // of half a tile each CTA uses 64 rows of W, the first of the box (a box of those
        // alone gained nothing)
        const int nb = n0 + (int)crank * (PART ? 64 : 128);
        for (int kb = kb0; kb < kb0 + nk; ++kb) {
          if (!wait_x(empty0 + 8 * stage, phase ^ 1u)) {
            ok = false;
            break;
          }
          // whole boxes arrive: zeros past K and past the last row.  (With fewer than 128
          // rows in all, X's boxes are no higher than those: boxes mostly past M are slow,
          // 24 x 16384 x 2048 11.6 us against 9.0.  The rows above hold whatever the
          // memory held, and reach only sums that are not stored.)  The leader's barrier
          // counts the bytes of both CTAs; the peer's may come before the leader expects
          // them, and the phase still waits for the leader's own arrival.
          const uint32_t sb = base + stage * C::STAGE_BYTES;
          if (!PAIR || crank == 0)
            mbar_expect_tx(full0 + 8 * stage, CM * (p.box_m * 128 + C::B_BYTES));
          if constexpr (PAIR) {
            const uint32_t fb = lead_full0 + 8 * stage;
            tma_load_2d_pair(sb, &tmX, kb * 128, m0, fb);
            tma_load_2d_pair(sb + C::A_BYTES, &tmW, kb * 128, nb, fb);
          } else {
            tma_load_2d(sb, &tmX, kb * 128, m0, full0 + 8 * stage);
            tma_load_2d(sb + C::A_BYTES, &tmW, kb * 128, nb, full0 + 8 * stage);
          }
          pend |= 1u << stage;
          pend_par = (pend_par & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        raise_error(abort_flag, p.status, PACT_DEV_TIMEOUT | PACT_DEV_ROLE_TMA);
        // let copies already in flight land before the CTA can exit; the peer of a pair
        // has no barrier of its own to see that by and waits a millisecond, a thousand
        // times a copy's latency
        if (PAIR && crank != 0) {
          const uint64_t t0 = global_timer_ns();
          while (global_timer_ns() - t0 < 1000000ull) {
          }
        } else {
          for (int s = 0; s < STAGES; ++s)
            if (pend & (1u << s))
              wait_x_for(full0 + 8 * s, (pend_par >> s) & 1u, 10000000ull, nullptr);
        }
      } else if constexpr (PAIR) {
        // the leader's commits arrive on this CTA's empty barriers: wait for the last
        // STAGES of them before the CTA may exit
        for (int i = 0; i < STAGES; ++i) {
          wait_x(empty0 + 8 * stage, phase ^ 1u);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
    if (warp >= 1 && warp <= C::ISSUERS && lane == 0 && crank == 0) {
      // ---------------------------------------------------------- MMA issuers
      // Issuing is slow for one thread: about 60 cycles an MMA, 50 to 100 a commit and 135
      // a wait, even on a barrier that is long complete; a block of a pair's tile has
      // eight MMAs of 64 cycles.  Several threads take the blocks in turn.  A pass over
      // the ring is unrolled, so that a stage's and a buffer's addresses are the base and
      // a constant.
      const int my_units = unit0 < nunits ? (nunits - unit0 + nclusters - 1) / nclusters : 0;
      constexpr uint32_t idesc = idesc_e4m3(128, 128 * CM);
      const uint64_t d0 = smem_desc(base, 16, 1024, 2);
      bool ok = true;
      const int64_t blocks = (int64_t)my_units * nk;
      auto issue = [&](auto turn_c) {
        constexpr int turn = decltype(turn_c)::value;
        uint32_t pass = 0;
        for (int64_t first = 0; first < blocks && ok; first += C::ROUND, ++pass) {
#pragma unroll
          for (int i = turn; i < C::ROUND; i += C::ISSUERS) {
            if (first + i >= blocks) break;
            const int s = i % STAGES, cyc = i % C::CYC;
            const uint32_t fills = pass * (C::ROUND / STAGES) + i / STAGES;
            const uint32_t uses = pass * (C::ROUND / C::CYC) + i / C::CYC;
            const uint32_t seen = mbar_test_two<PAIR>(full0 + 8 * s, fills & 1u,
                                                      acce0 + 8 * (cyc * NSUB), (uses & 1u) ^ 1u);
            if (!(seen & 1u) && !wait_x(full0 + 8 * s, fills & 1u)) {
              ok = false;
              break;
            }
            uint32_t lo = (uint32_t)d0;
            asm volatile("" : "+r"(lo));  // not kept in registers for every stage
            const uint64_t da = ((d0 >> 32) << 32) | (lo + s * (C::STAGE_BYTES >> 4));
#pragma unroll
            for (int h = 0; h < NSUB; ++h) {
              const int buf = cyc * NSUB + h;
              if (!(h == 0 && (seen & 2u)) && !wait_tmem(acce0 + 8 * buf, (uses & 1u) ^ 1u)) {
                ok = false;
                break;
              }
              if (PART && h == 1) continue;
              tc_fence_after();
              // sub-block h of a pair takes rows 64 h .. 64 h + 63 of each CTA's tile of W
              const uint64_t db = da + ((C::A_BYTES + h * 64 * 128) >> 4);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                mma_f8<PAIR>(tmem + buf * 128, da + 2u * j, db + 2u * j, idesc, j > 0);
            }
            if (!ok) break;
            if constexpr (PAIR) {
              mma_commit_pair(accf0 + 8 * cyc, (uint16_t)3u);
              mma_commit_pair(empty0 + 8 * s, (uint16_t)3u);
            } else {
              mma_commit(accf0 + 8 * cyc);
              mma_commit(empty0 + 8 * s);
            }
          }
        }
      };
      if (warp == 1)
        issue(std::integral_constant<int, 0>());
      else
        issue(std::integral_constant<int, 1>());
      if (!ok) raise_error(abort_flag, p.status, PACT_DEV_TIMEOUT | PACT_DEV_ROLE_MMA);
      // every MMA issued by these threads has completed once final_bar flips
      if constexpr (PAIR)
        mma_commit_pair(final_bar, (uint16_t)1u);
      else
        mma_commit(final_bar);
      mbar_wait(final_bar, 0, kFp8WaitNs, nullptr);
    }
    if (warp == 3) {
      // ---------------------------------------------------------- scales
      // Loads by the epilogue threads themselves, three blocks ahead, held them up for
      // 30 % of the kernel's time (220 us against 155, 8192 x 4096 x 8192): they queue
      // behind the tiles' copies.  A barrier for each block cost the epilogue's wait
      // another 7 % (221 against 206 us), so there is one for eight blocks.
      uint32_t slot = 0, phase = 0;
      bool ok = true;
      for (int u = unit0; u < nunits && ok; u += nclusters) {
        int m0, n0;
        unit_mn(u, m0, n0);
        // columns past N have no scale of their own: their sums are not stored
        const float* psw = p.sw + kb0 +
                           (int64_t)(min(n0 + (PART ? 0 : (lane & 1) * C::EPI_COLS), p.N - 1) >> 7) *
                               p.nkb;
        const float* psx = p.sx + (int64_t)kb0 * p.M + m0 + lane;
        for (int kb = 0; kb < nk; ++kb, psx += p.M, ++psw) {
          const uint32_t half = slot / C::SCL_HALF;
          if (slot % C::SCL_HALF == 0 &&
              !mbar_wait(scle0 + 8 * half, phase ^ 1u, kFp8WaitNs, abort_flag)) {
            raise_error(abort_flag, p.status, PACT_DEV_TIMEOUT | PACT_DEV_ROLE_SF);
            ok = false;
            break;
          }
          const uint32_t at = base + C::SCL_OFF + slot * C::SCL_SLOT;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool in = m0 + lane + 32 * i < p.M;  // rows past M: zero
            cp_async4(at + 4 * (lane + 32 * i), in ? psx + 32 * i : p.sx, in ? 4u : 0u);
          }
          if (lane < 2) cp_async4(at + 512 + 4 * lane, psw, 4u);
          if (slot % C::SCL_HALF == C::SCL_HALF - 1) cp_async_mbar_arrive(sclf0 + 8 * half);
          if (++slot == C::SCL_DEPTH) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      if (slot % C::SCL_HALF) cp_async_mbar_arrive(sclf0 + 8 * (slot / C::SCL_HALF));
      cp_async_commit();
      cp_async_wait<0>();
    }
    if constexpr (SPLIT) {
      __syncwarp();
      cluster_sync();  // the epilogue's partial sums
    }
  } else {
    // ------------------------------------------------------------ epilogue
    setmaxnreg_inc<C::EPI_REGS>();
    const int q = warp & 3;            // TMEM lane quarter this warp may access
    const int half = (warp - 4) >> 2;  // which half of the columns
    constexpr int COLS = PART ? 64 : C::EPI_COLS;  // of this warp
    const int c0 = half * COLS;
    const uint32_t tq = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(half * 64);
    // blocks so far, from which the buffer, the ring slot and their parities follow (one
    // register: the sums and slices leave few)
    uint32_t blk = 0;
    bool ok = true;
    const uint32_t acce = PAIR ? cluster_addr(acce0, 0) : acce0;  // at the leader
    static_assert((C::CYC & (C::CYC - 1)) == 0 && C::SCL_DEPTH == 16 && C::SCL_HALF == 8, "bits");
    auto buf = [&]() { return blk & (uint32_t)(C::CYC - 1); };
    // the next block's accumulators and, for every eighth, scales
    auto wait_block = [&]() {
      if ((blk & 7u) == 0 && !mbar_wait(sclf0 + (blk & 8u), (blk >> 4) & 1u, kFp8WaitNs, abort_flag))
        return false;
      return wait_tmem(accf0 + 8 * buf(), (blk / C::CYC) & 1u);
    };
    auto scale = [&]() {
      const uint32_t at = base + C::SCL_OFF + (blk & 15u) * C::SCL_SLOT;
      const float s = __fmul_rn(ld_shared_f32(at + 4u * (uint32_t)(q * 32 + lane)),
                                ld_shared_f32(at + 512u + 4u * (uint32_t)half));
      if ((blk & 7u) == 7u) {  // that half of the ring has been read
        __syncwarp();
        if (lane == 0) mbar_arrive(scle0 + (blk & 8u));
      }
      return s;
    };
    for (int u = unit0; u < nunits && ok; u += nclusters) {
      int m0, n0;
      unit_mn(u, m0, n0);
      if constexpr (ADD) {  // the addend's rows are in L2 when the sums are done
        const int64_t m = m0 + q * 32 + lane;
        if (m < p.M) {
#pragma unroll
          for (int c = 0; c < COLS; c += 64)
            if (n0 + c0 + c < p.N)
              asm volatile("prefetch.global.L2 [%0];" ::"l"(p.add + m * p.N + n0 + c0 + c));
        }
      }
      float2 acc[COLS / 2];
#pragma unroll
      for (int i = 0; i < COLS / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
      auto release = [&](int h) {  // buffer h of the block: its columns have landed
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR)
            mbar_arrive_remote_relaxed(acce + 8 * (buf() * NSUB + h));
          else
            mbar_arrive(acce + 8 * (buf() * NSUB + h));
        }
      };
      for (int kb = 0; kb < nk; ++kb, ++blk) {
        if (!(ok = wait_block())) break;
        tc_fence_after();
        const uint32_t tb = tq + buf() * (NSUB * 128);
        uint32_t v[2][16];
        tmem_ld16(tb, v[0]);
        const float s = scale();
#pragma unroll
        for (int c = 0; c < COLS / 16; ++c) {
          tmem_ld_wait16(v[c & 1]);
          if (c + 1 < COLS / 16)  // the next slice lands while this one is added
            tmem_ld16(tb + (c + 1) / 4 * 128 + (c + 1) % 4 * 16, v[(c + 1) & 1]);
          if (c % 4 == 3) release(c / 4);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            acc[8 * c + i] =
                __ffma2_rn(make_float2(__uint_as_float(v[c & 1][2 * i]),
                                       __uint_as_float(v[c & 1][2 * i + 1])),
                           make_float2(s, s), acc[8 * c + i]);
        }
        if constexpr (PART) release(1);  // not written
      }
      if (!ok) raise_error(abort_flag, p.status, PACT_DEV_TIMEOUT | PACT_DEV_ROLE_EPI);
      if (!ok) break;
      if constexpr (SPLIT) {
        // the one tile of this CTA: its partial sums go into the ring, which every copy and
        // MMA is done with, as [128][128] FP32 with the 16-byte pieces of row r in the
        // order piece ^ (r % 32), so that neither writing a row per lane nor reading along
        // a row meets a bank twice
        const int r = q * 32 + lane;
#pragma unroll
        for (int i = 0; i < C::EPI_COLS / 4; ++i) {
          const int piece = (c0 / 4 + i) ^ (r & 31);
          *reinterpret_cast<float4*>(smem + r * 512 + piece * 16) =
              make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x, acc[2 * i + 1].y);
        }
        break;
      }
      // 32 columns at a time through shared memory and out by TMA, which clips rows past M
      // and columns past N.  (Stored by the lanes, a row each, an instruction touches 32
      // rows: 2 us a tile on the load/store unit.)
      if (m0 + q * 32 >= p.M) continue;
      const int live = min(p.N - n0 - c0, COLS);  // columns inside the output
      // 64 columns of the addend, 32 bytes a load where its alignment allows; the next 64
      // land while those before are stored
      uint32_t a[32];
      const int64_t m = m0 + q * 32 + lane;
      auto load_add = [&](int b) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // N % 16 == 0: 16 columns lie inside or outside whole
          uint32_t* t = a + 8 * k;
#pragma unroll
          for (int i = 0; i < 8; ++i) t[i] = 0u;
          if (m >= p.M || 64 * b + 16 * k >= live) continue;
          const uint16_t* at = p.add + m * p.N + n0 + c0 + 64 * b + 16 * k;
          if (p.add32) {
            asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                         : "=r"(t[0]), "=r"(t[1]), "=r"(t[2]), "=r"(t[3]), "=r"(t[4]), "=r"(t[5]),
                           "=r"(t[6]), "=r"(t[7])
                         : "l"(at)
                         : "memory");
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint4 x = *reinterpret_cast<const uint4*>(at + 8 * i);
              t[4 * i] = x.x;
              t[4 * i + 1] = x.y;
              t[4 * i + 2] = x.z;
              t[4 * i + 3] = x.w;
            }
          }
        }
      };
      if constexpr (ADD) load_add(0);
      const uint32_t stg = base + C::STG_OFF + (uint32_t)((warp - 4) * C::STG_BUF);
      uint8_t* row = smem + (stg - base) + 64 * lane;
      const uint32_t sw = (uint32_t)(lane >> 1) & 3u;  // 64-byte swizzle of the store's map
#pragma unroll
      for (int b = 0; b < COLS / 64; ++b) {
        if constexpr (ADD) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            acc[32 * b + i] = __fadd2_rn(acc[32 * b + i],
                                         make_float2(__uint_as_float(a[i] << 16),
                                                     __uint_as_float(a[i] & 0xFFFF0000u)));
          if (b + 1 < COLS / 64) load_add(b + 1);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (64 * b + 32 * j >= live) continue;  // uniform across the warp
          const float2* f = acc + 32 * b + 16 * j;
          if (lane == 0) bulk_wait_read<0>();  // the previous store has read the buffer
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(row + 16 * (k ^ sw)) = make_uint4(
                pack_bf16x2(f[4 * k].x, f[4 * k].y), pack_bf16x2(f[4 * k + 1].x, f[4 * k + 1].y),
                pack_bf16x2(f[4 * k + 2].x, f[4 * k + 2].y),
                pack_bf16x2(f[4 * k + 3].x, f[4 * k + 3].y));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tmOut, stg, n0 + c0 + 64 * b + 32 * j, m0 + q * 32);
            bulk_commit();
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();
    if constexpr (SPLIT) {
      __syncwarp();
      cluster_sync();  // every CTA's partial sums are in its shared memory
      // this CTA's rows of the tile: a warp takes a row of 128 columns, four a lane, and
      // adds the CTAs' sums in their order
      int m0, n0;
      unit_mn(unit0, m0, n0);
      const int r0 = 128 * (int)krank / p.split, r1 = 128 * (int)(krank + 1) / p.split;
      const int n = n0 + 4 * lane;
      for (int r = r0 + warp - 4; r < r1; r += 32) {  // four rows at a time
        float4 v[4][kMaxSplit];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int rj = min(r + 8 * j, r1 - 1);
          const uint32_t at = base + (uint32_t)(rj * 512 + ((lane ^ (rj & 31)) * 16));
#pragma unroll
          for (int c = 0; c < kMaxSplit; ++c)
            v[j][c] = c < p.split ? ld_shared_cluster_v4f32(cluster_addr(at, (uint32_t)c))
                                  : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t m = m0 + r + 8 * j;
          if (r + 8 * j >= r1 || m >= p.M || n >= p.N) continue;
          float4 t = v[j][0];
#pragma unroll
          for (int c = 1; c < kMaxSplit; ++c) {
            t.x += v[j][c].x;
            t.y += v[j][c].y;
            t.z += v[j][c].z;
            t.w += v[j][c].w;
          }
          if (p.add) {
            const uint2 a = *reinterpret_cast<const uint2*>(p.add + m * p.N + n);
            t.x += __uint_as_float(a.x << 16);
            t.y += __uint_as_float(a.x & 0xFFFF0000u);
            t.z += __uint_as_float(a.y << 16);
            t.w += __uint_as_float(a.y & 0xFFFF0000u);
          }
          if (PACT_IN(m * p.N + n + 4 <= (int64_t)p.M * p.N))
            *reinterpret_cast<uint2*>(p.out + m * p.N + n) =
                make_uint2(pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w));
        }
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  // no CTA leaves while another may still signal it or read its sums
  if constexpr (PAIR || SPLIT) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem, 512);
    else
      tmem_dealloc(tmem, 512);
  }
}

// The tiles from `first` on, `count` of them (0: to the last).
template <bool PAIR, bool SPLIT, bool ADD, bool PART = false>
static cudaError_t launch_tiles(const Fp8GemmLaunch& L, int split, cudaStream_t stream,
                                int64_t first = 0, int64_t count = 0) {
  using C = Fp8Cfg<PAIR>;
  auto kern = k_fp8_gemm<PAIR, SPLIT, ADD, PART>;
  static std::atomic<int> max_clusters[64];  // per device, once its attribute is set
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = SPLIT ? split : C::CM;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int resident = max_clusters[dev].load(std::memory_order_acquire);
  if (resident == 0) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    // the register shares add up only with this many at launch: a build that came out
    // with fewer would wait for registers that nobody gives back
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
    if (fa.numRegs != C::LAUNCH_REGS) return cudaErrorInvalidKernelImage;
    int n = L.num_sms / C::CM;
    if (PAIR) {
      cfg.gridDim = dim3(L.num_sms / C::CM * C::CM);
      e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
      if (e != cudaSuccess) return e;
      if (n < 1) return cudaErrorInvalidConfiguration;
    }
    resident = n;
    max_clusters[dev].store(n, std::memory_order_release);
  }
  Fp8GemmParams p = L.p;
  p.num_m = (p.M + 127) / 128;
  p.num_n = (p.N + C::BN - 1) / C::BN;
  const int num_mc = (p.num_m + C::CM - 1) / C::CM;
  const int64_t tiles = (int64_t)num_mc * p.num_n;  // < 2^30, checked by the caller
  p.first = (int)first;
  p.units = (int)((count ? count : tiles - first) * (PART ? 2 : 1));
  const int clusters = SPLIT || p.units < resident ? p.units : resident;
  cfg.gridDim = dim3(clusters * (SPLIT ? split : C::CM));
  p.split = split;
  // tile order as in the NVFP4 GEMM: one band while X fits in L2 beside the tiles of W
  // in flight, else bands just wide enough to keep every cluster busy
  p.band_mc = num_mc;
  if ((double)p.num_m * 128.0 * (double)L.K > 32.0 * 1024 * 1024) {
    // from the device's size, so that every launch over these tiles has the same order
    const int b = (L.num_sms / C::CM + p.num_n - 1) / p.num_n;
    p.band_mc = b < 1 ? 1 : (b > num_mc ? num_mc : b);
  }
  note_launch();
  return cudaLaunchKernelEx(&cfg, kern, L.tmX, L.tmW, L.tmOut, p);
}

cudaError_t launch_fp8_gemm(const Fp8GemmLaunch& L, cudaStream_t stream) {
  const Fp8Plan plan = fp8_plan(L.p.M, L.p.N, L.K, L.num_sms);
  if (plan.way == kShared) return launch_tiles<false, true, false>(L, plan.split, stream);
  if (plan.way == kPairs) {
    const cudaError_t e = L.p.add ? launch_tiles<true, false, true>(L, 1, stream, 0, plan.whole)
                                  : launch_tiles<true, false, false>(L, 1, stream, 0, plan.whole);
    if (e != cudaSuccess || !plan.whole) return e;
    return L.p.add ? launch_tiles<true, false, true, true>(L, 1, stream, plan.whole)
                   : launch_tiles<true, false, false, true>(L, 1, stream, plan.whole);
  }
  return L.p.add ? launch_tiles<false, false, true>(L, 1, stream)
                 : launch_tiles<false, false, false>(L, 1, stream);
}

}  // namespace pact
