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


bool fp8_is_few(int64_t M, int64_t N, int64_t K) { return M <= 32; }

// ---------------------------------------------------------------- many tokens
// A persistent CTA per SM, or CTA pair (cluster of two along M, .cta_group::2, 256 x BN
// tiles).  Per block of K (128 bytes of a row, one ring stage, four MMAs) the tensor
// cores write a fresh accumulator; the epilogue warps multiply it by the block's scales
// and add it to sums in registers while the next blocks' MMAs run into the other
// accumulator buffers.  A thread owns one row, and a warp's columns lie in one block of
// 128 outputs, so a block's two scales are a single factor per thread.
//   warp 0     TMA producer
//   warp 1     TMEM allocator and MMA issuer (in a pair, the peer's relays to the
//              leader that the peer's tiles have landed)
//   warps 2-9  epilogue: two warps per TMEM lane quarter, each half of the columns
template <int BN, int STAGES, bool PAIR>
struct Fp8Cfg {
  static constexpr int CM = PAIR ? 2 : 1;
  static constexpr int B_ROWS = PAIR ? BN / 2 : BN;  // rows of W in this CTA's shared memory
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = B_ROWS * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STG_OFF = STAGES * STAGE_BYTES;
  static constexpr int STG_BUF = 2048;  // 32 rows x 32 BF16, 64-byte swizzled rows
  static constexpr int NSTG = 2;
  static constexpr int BAR_OFF = STG_OFF + 8 * NSTG * STG_BUF;
  static constexpr int SMEM_BYTES = BAR_OFF + 512 + 1024;  // + barriers + alignment slack
  static constexpr int NBUF = 512 / BN;                    // accumulator buffers in TMEM
  static constexpr int THREADS = 320;
  static constexpr int EPI_COLS = BN / 2;
  static constexpr int NCH = EPI_COLS / 32;
  // barriers: full[S], empty[S], peer[S], acc_full[NBUF], acc_empty[NBUF], final
  static constexpr int NBARS = 3 * STAGES + 2 * NBUF + 1;
  static_assert(BN == 128 || BN == 256, "a warp's columns lie in one block of 128");
  static_assert(NBARS * 8 <= 504 && SMEM_BYTES <= 232448, "shared memory budget");
};

__host__ __device__ constexpr uint32_t idesc_e4m3(int n, int m) {
  // D = F32 (bits 4-5 = 1), A = B = E4M3 (0)
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

constexpr uint64_t kFp8WaitNs = 2000000000ull;  // 2 s per pipeline wait

template <int BN, int STAGES, bool PAIR>
__global__ void __launch_bounds__(320, 1)
    k_fp8_gemm(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
               const __grid_constant__ CUtensorMap tmOut, const Fp8GemmParams p) {
  using C = Fp8Cfg<BN, STAGES, PAIR>;
  constexpr int CM = C::CM, NBUF = C::NBUF;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t full0 = base + C::BAR_OFF, empty0 = full0 + 8 * STAGES;
  const uint32_t peer0 = empty0 + 8 * STAGES;
  const uint32_t accf0 = peer0 + 8 * STAGES, acce0 = accf0 + 8 * NBUF;
  const uint32_t final_bar = acce0 + 8 * NBUF;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::BAR_OFF + 504);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::BAR_OFF + 508);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = PAIR ? cluster_ctarank() : 0u;
  const int num_mc = (p.num_m + CM - 1) / CM;
  const int nunits = num_mc * p.num_n;
  const int unit0 = (int)blockIdx.x / CM, nclusters = (int)gridDim.x / CM;
  const int band = p.band_mc;
  auto unit_mn = [&](int u, int& m0, int& n0) {
    const int bi = u / (band * p.num_n), r = u - bi * band * p.num_n;
    const int mc0 = bi * band, bm = min(band, num_mc - mc0);
    const int n = r / bm;
    m0 = ((mc0 + (r - n * bm)) * CM + (int)crank) * 128;
    n0 = n * BN;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
      mbar_init(peer0 + 8 * s, 1);
    }
    for (int b = 0; b < NBUF; ++b) {
      mbar_init(accf0 + 8 * b, 1);
      mbar_init(acce0 + 8 * b, 8 * CM);  // one arrival per epilogue warp of each CTA
    }
    mbar_init(final_bar, 1);
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

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t pend = 0, pend_par = 0, phase = 0;
      int stage = 0;
      bool ok = true;
      for (int u = unit0; u < nunits && ok; u += nclusters) {
        int m0, n0;
        unit_mn(u, m0, n0);
        const int nb = n0 + (int)crank * C::B_ROWS;
        for (int kb = 0; kb < p.nkb; ++kb) {
          if (!mbar_wait(empty0 + 8 * stage, phase ^ 1u, kFp8WaitNs, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t fb = full0 + 8 * stage, sb = base + stage * C::STAGE_BYTES;
          // whole boxes arrive: zeros past K and past the last row
          mbar_expect_tx(fb, C::STAGE_BYTES);
          tma_load_2d(sb, &tmX, kb * 128, m0, fb);
#pragma unroll
          for (int r = 0; r < C::B_ROWS; r += 128)
            tma_load_2d(sb + C::A_BYTES + r * 128, &tmW, kb * 128, nb + r, fb);
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
        // let copies already in flight land before the CTA can exit
        for (int s = 0; s < STAGES; ++s)
          if (pend & (1u << s)) mbar_wait(full0 + 8 * s, (pend_par >> s) & 1u, 10000000ull, nullptr);
      } else if constexpr (PAIR) {
        // the leader's commits arrive on this CTA's empty barriers: wait for the last
        // STAGES of them before the CTA may exit
        for (int i = 0; i < STAGES; ++i) {
          mbar_wait(empty0 + 8 * stage, phase ^ 1u, kFp8WaitNs, abort_flag);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const int my_units = unit0 < nunits ? (nunits - unit0 + nclusters - 1) / nclusters : 0;
    uint32_t phase = 0;
    int stage = 0;
    if (PAIR && crank != 0) {
      if (lane == 0) {
        for (int64_t i = (int64_t)my_units * p.nkb; i > 0; --i) {
          if (!mbar_wait(full0 + 8 * stage, phase, kFp8WaitNs, abort_flag)) {
            raise_error(abort_flag, p.status, PACT_DEV_TIMEOUT | PACT_DEV_ROLE_MMA);
            break;
          }
          mbar_arrive_cta(peer0 + 8 * stage, 0);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    } else if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3(BN, 128 * CM);
      const uint64_t da0 = smem_desc(base, 16, 1024, 2);
      const uint64_t db0 = smem_desc(base + C::A_BYTES, 16, 1024, 2);
      bool ok = true;
      int buf = 0;
      uint32_t aphase = 0;
      for (int64_t i = (int64_t)my_units * p.nkb; i > 0; --i) {
        const bool got = PAIR ? mbar_wait_cluster(acce0 + 8 * buf, aphase ^ 1u, kFp8WaitNs, abort_flag)
                              : mbar_wait(acce0 + 8 * buf, aphase ^ 1u, kFp8WaitNs, abort_flag);
        if (!got || !mbar_wait(full0 + 8 * stage, phase, kFp8WaitNs, abort_flag) ||
            (PAIR && !mbar_wait_cluster(peer0 + 8 * stage, phase, kFp8WaitNs, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t soff = (uint64_t)(stage * (C::STAGE_BYTES >> 4));
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma_f8<PAIR>(tmem + buf * BN, da0 + soff + 2u * j, db0 + soff + 2u * j, idesc, j > 0);
        if constexpr (PAIR) {
          mma_commit_pair(empty0 + 8 * stage, (uint16_t)3u);
          mma_commit_pair(accf0 + 8 * buf, (uint16_t)3u);
        } else {
          mma_commit(empty0 + 8 * stage);
          mma_commit(accf0 + 8 * buf);
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
        if (++buf == NBUF) {
          buf = 0;
          aphase ^= 1u;
        }
      }
      if (!ok) raise_error(abort_flag, p.status, PACT_DEV_TIMEOUT | PACT_DEV_ROLE_MMA);
      // every MMA issued by this thread has completed once final_bar flips
      if constexpr (PAIR)
        mma_commit_pair(final_bar, (uint16_t)1u);
      else
        mma_commit(final_bar);
      mbar_wait(final_bar, 0, kFp8WaitNs, nullptr);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;  // TMEM lane quarter this warp may access
    const int ew = warp - 2;
    const int c0 = (ew >> 2) * C::EPI_COLS;
    const uint32_t stg = base + C::STG_OFF + (uint32_t)(ew * C::NSTG * C::STG_BUF);
    const uint32_t tq = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)c0;
    int buf = 0;
    uint32_t aphase = 0, nstore = 0;
    bool ok = true;
    for (int u = unit0; u < nunits && ok; u += nclusters) {
      int m0, n0;
      unit_mn(u, m0, n0);
      const int m = m0 + q * 32 + lane;
      const bool row_ok = m < p.M;
      const bool blk_live = m0 + q * 32 < p.M;
      // columns past N have no scale of their own: their sums are not stored
      const int nblk = min(n0 + c0, p.N - 1) >> 7;
      const float* sxp = p.sx + (row_ok ? m : 0);
      const float* swp = p.sw + (int64_t)nblk * p.nkb;
      float2 acc[C::EPI_COLS / 2];
#pragma unroll
      for (int i = 0; i < C::EPI_COLS / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
      float s_next = row_ok ? __fmul_rn(*sxp, *swp) : 0.0f;
      for (int kb = 0; kb < p.nkb; ++kb) {
        const float s = s_next;
        if (kb + 1 < p.nkb) {
          sxp += p.M;
          ++swp;
          s_next = row_ok ? __fmul_rn(*sxp, *swp) : 0.0f;
        }
        if (!(PAIR ? mbar_wait_cluster(accf0 + 8 * buf, aphase, kFp8WaitNs, abort_flag)
                   : mbar_wait(accf0 + 8 * buf, aphase, kFp8WaitNs, abort_flag))) {
          raise_error(abort_flag, p.status, PACT_DEV_TIMEOUT | PACT_DEV_ROLE_EPI);
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int ch = 0; ch < C::NCH; ++ch) {
          uint32_t v[32];
          tmem_ld32(tq + (uint32_t)(buf * BN + 32 * ch), v);
          tmem_ld_wait();
          if (ch == C::NCH - 1) {  // the buffer is free once the last slice has landed
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if constexpr (PAIR)
                mbar_arrive_cta_relaxed(acce0 + 8 * buf, 0u);  // at the leader
              else
                mbar_arrive(acce0 + 8 * buf);
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i)
            acc[16 * ch + i] = __ffma2_rn(
                make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])),
                make_float2(s, s), acc[16 * ch + i]);
        }
        if (++buf == NBUF) {
          buf = 0;
          aphase ^= 1u;
        }
      }
      if (!ok) break;
#pragma unroll
      for (int ch = 0; ch < C::NCH; ++ch) {
        const int n = n0 + c0 + 32 * ch;
        if (n >= p.N || !blk_live) continue;  // uniform across the warp
        uint32_t o[16];
        if (p.add && row_ok) {
          const uint16_t* ap = p.add + (int64_t)m * p.N + n;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // N % 16 == 0: a vector of 8 columns lies inside or outside whole
            uint4 a = make_uint4(0u, 0u, 0u, 0u);
            if (n + 8 * k < p.N) a = *reinterpret_cast<const uint4*>(ap + 8 * k);
            o[4 * k] = a.x;
            o[4 * k + 1] = a.y;
            o[4 * k + 2] = a.z;
            o[4 * k + 3] = a.w;
          }
#pragma unroll
          for (int i = 0; i < 16; ++i)
            acc[16 * ch + i] = __fadd2_rn(
                acc[16 * ch + i], make_float2(__uint_as_float(o[i] << 16),
                                              __uint_as_float(o[i] & 0xFFFF0000u)));
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = pack_bf16x2(acc[16 * ch + i].x, acc[16 * ch + i].y);
        const uint32_t sb = stg + (nstore % C::NSTG) * C::STG_BUF;
        if (nstore >= (uint32_t)C::NSTG && lane == 0) bulk_wait_read<C::NSTG - 1>();
        __syncwarp();
        uint8_t* row = smem + (sb - base) + 64 * lane;
        const uint32_t sw = (uint32_t)(lane >> 1) & 3u;  // 64-byte swizzle of the store's map
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4*>(row + 16 * (k ^ sw)) =
              make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&tmOut, sb, n, m0 + q * 32);  // clips rows past M and columns past N
          bulk_commit();
        }
        ++nstore;
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // no CTA leaves while its peer may still signal it
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem, 512);
    else
      tmem_dealloc(tmem, 512);
  }
}

template <int BN, int STAGES, bool PAIR>
static cudaError_t launch_tiles(const Fp8GemmLaunch& L, cudaStream_t stream) {
  using C = Fp8Cfg<BN, STAGES, PAIR>;
  auto kern = k_fp8_gemm<BN, STAGES, PAIR>;
  static int max_clusters[64] = {};  // per device, once its attribute is set
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C::CM;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (max_clusters[dev] == 0) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    int n = L.num_sms / C::CM;
    if (PAIR) {
      cfg.gridDim = dim3(L.num_sms / C::CM * C::CM);
      e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
      if (e != cudaSuccess) return e;
      if (n < 1) return cudaErrorInvalidConfiguration;
    }
    max_clusters[dev] = n;
  }
  Fp8GemmParams p = L.p;
  p.num_m = (p.M + 127) / 128;
  p.num_n = (p.N + BN - 1) / BN;
  const int num_mc = (p.num_m + C::CM - 1) / C::CM;
  const int64_t units = (int64_t)num_mc * p.num_n;
  if (units >= (int64_t)1 << 30) return cudaErrorInvalidValue;
  const int clusters = (int)(units < max_clusters[dev] ? units : max_clusters[dev]);
  cfg.gridDim = dim3(clusters * C::CM);
  // tile order as in the NVFP4 GEMM: one band while X fits in L2 beside the tiles of W
  // in flight, else bands just wide enough to keep every cluster busy
  p.band_mc = num_mc;
  if ((double)p.num_m * 128.0 * (double)L.K > 32.0 * 1024 * 1024) {
    const int b = (clusters + p.num_n - 1) / p.num_n;
    p.band_mc = b < 1 ? 1 : (b > num_mc ? num_mc : b);
  }
  note_launch();
  return cudaLaunchKernelEx(&cfg, kern, L.tmX, L.tmW, L.tmOut, p);
}

cudaError_t launch_fp8_gemm(const Fp8GemmLaunch& L, cudaStream_t stream) {
  if (L.p.M > 128 && L.p.N > 128) return launch_tiles<256, 6, true>(L, stream);
  return launch_tiles<128, 6, false>(L, stream);
}

}  // namespace pact
