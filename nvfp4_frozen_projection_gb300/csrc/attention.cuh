// What the attention kernels share: the search of a unit's sequence, the tile of packed
// (token, head) rows, and the tensor-core instructions with an operand in tensor memory.
//
// Rows of a query tile.  The query heads of one key head share its keys, so a tile holds
// tpt tokens times gp of those heads, row = token * gp + head: keys and values are loaded
// once for all of them, and a single token of a grouped model fills several rows.  gp is
// the largest divisor of the group that is at most 128, tpt = 128 / gp.
#pragma once

#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace pact {

constexpr uint64_t kAttnWaitNs = 2000000000ull;  // 2 s per pipeline wait
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// D = F32, A = B = BF16, M = 128.  TB: B lies N-major (its rows run along the reduction).
__host__ __device__ constexpr uint32_t attn_idesc(int n, bool tb) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (tb ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
         (8u << 24);
}

// D (FP32, TMEM) (+)= A * B^T with A (BF16, two values a column) in TMEM.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int32_t c0,
                                            int32_t c1, int32_t c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// The warp's number, known to be the same in all of its lanes.
__device__ __forceinline__ int warp_index() {
  return __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0);
}

// Whether this lane is the one of its warp that issues copies and MMAs.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}

// A place in a ring of shared-memory tiles and the parity of its turn.
struct RingPos {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void advance(int stages, int by = 1) {
    stage += by;
    if (stage >= stages) {
      stage -= stages;
      phase ^= 1u;
    }
  }
};

// Wait for a tcgen05.ld of 32 columns, whose registers are operands so that nothing
// computed from them moves ahead of the wait.
__device__ __forceinline__ void tmem_ld_wait32(uint32_t* v) {
  tmem_ld_wait16(v);
#pragma unroll
  for (int i = 16; i < 32; ++i) asm volatile("" : "+r"(v[i]));
}

// A tile in shared memory: DP / 64 boxes of `rows` rows of 128 bytes, 128-byte swizzle.
// K-major descriptors step 32 bytes within a box and by a box every four steps; N-major
// ones step two groups of 8 rows (2048 bytes) each 16 rows, boxes BOX bytes apart along N.
constexpr uint32_t kBox = 128 * 128;
__device__ __forceinline__ uint64_t desc_k(uint32_t tile) { return smem_desc(tile, 16, 1024, 2); }
__device__ __forceinline__ uint64_t desc_n(uint32_t tile) { return smem_desc(tile, kBox, 1024, 2); }
__device__ __forceinline__ uint64_t step_k(uint64_t d, int k) {
  return d + (uint64_t)((k >> 2) * (kBox >> 4) + (k & 3) * 2);
}
__device__ __forceinline__ uint64_t step_n(uint64_t d, int k) { return d + (uint64_t)(k * 128); }

// Zero rows [from, 128) of a tile of `boxes` boxes, by a warp; what a product over the rows
// must not take from a neighbouring sequence: 0 * NaN is NaN.
__device__ __forceinline__ void zero_rows(uint8_t* tile, int boxes, int from, int lane) {
  for (int b = 0; b < boxes; ++b)
    for (int o = from * 128 + lane * 16; o < (int)kBox; o += 512)
      *reinterpret_cast<uint4*>(tile + b * kBox + o) = make_uint4(0u, 0u, 0u, 0u);
}

// Sequence b of the packed rows: offsets are clamped to the tensors, so that no value of
// them leads outside.
struct Seq {
  int q0, lq, k0, lk;
  int tile;   // of this sequence
  int tiles;  // of this sequence
};

// Units are numbered by sequence, then by tile.  A role's units ascend, so its search goes
// on where the last one ended; 32 sequences a step, one a lane.
struct SeqFinder {
  const int* cu_q;
  const int* cu_k;
  int nseq, tq, tk;
  int per;        // tokens a unit
  bool over_k;    // units are tiles of keys
  int b0 = 0;
  int64_t base = 0;

  __device__ __forceinline__ static int clampi(int v, int lo, int hi) {
    return v < lo ? lo : (v > hi ? hi : v);
  }

  // Every lane of the warp calls this; false behind the last unit.
  __device__ __forceinline__ bool find(int64_t t, Seq& s) {
    const int lane = threadIdx.x & 31;
    while (b0 < nseq) {
      const int b = b0 + lane;
      int q0 = 0, lq = 0, k0 = 0, lk = 0, n = 0;
      if (b < nseq) {
        q0 = clampi(__ldg(cu_q + b), 0, tq);
        lq = clampi(__ldg(cu_q + b + 1), q0, tq) - q0;
        k0 = clampi(__ldg(cu_k + b), 0, tk);
        lk = clampi(__ldg(cu_k + b + 1), k0, tk) - k0;
        n = ((over_k ? lk : lq) + per - 1) / per;
      }
      int64_t incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += up;
      }
      const unsigned hit = __ballot_sync(0xFFFFFFFFu, t < base + incl);
      if (hit) {
        const int l = __ffs(hit) - 1;
        s.q0 = __shfl_sync(0xFFFFFFFFu, q0, l);
        s.lq = __shfl_sync(0xFFFFFFFFu, lq, l);
        s.k0 = __shfl_sync(0xFFFFFFFFu, k0, l);
        s.lk = __shfl_sync(0xFFFFFFFFu, lk, l);
        s.tiles = __shfl_sync(0xFFFFFFFFu, n, l);
        s.tile = (int)(t - base - (__shfl_sync(0xFFFFFFFFu, incl, l) - s.tiles));
        return true;
      }
      base += __shfl_sync(0xFFFFFFFFu, incl, 31);
      b0 += 32;
    }
    return false;
  }
};

__device__ __forceinline__ SeqFinder seq_finder(const AttnParams& p, int per, bool over_k) {
  SeqFinder f;
  f.cu_q = p.cu_q;
  f.cu_k = p.cu_k;
  f.nseq = p.nseq;
  f.tq = p.tq;
  f.tk = p.tk;
  f.per = per;
  f.over_k = over_k;
  return f;
}

// Token of a row of a tile; rows < 128 and gp <= 128, where the product is exact.
__device__ __forceinline__ int row_token(const AttnParams& p, int row) {
  return (int)(((uint32_t)row * p.gp_mul) >> 16);
}

// Rows of 64 BF16 columns held one a lane (w: 8 pieces of 16 bytes) go out as whole rows of
// 128 bytes, four an instruction: the lanes of each group of 8 exchange pieces, so that lane
// l of a group ends up with piece l of each of the group's rows.  Stored as they are held, a
// piece a lane, an instruction would touch 32 rows.  addr(r): where row r's columns begin,
// null for a row that is not stored; cols: how many of the 64 columns there are.
template <typename Addr>
__device__ __forceinline__ void store_rows64(uint32_t (&w)[32], int lane, int cols, Addr addr) {
#pragma unroll
  for (int s = 1; s < 8; s <<= 1) {
    const bool up = (lane & s) != 0;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (c & s) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t lo = w[4 * c + k], hi = w[4 * (c | s) + k];
        const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? lo : hi, s);
        w[4 * c + k] = up ? got : lo;
        w[4 * (c | s) + k] = up ? hi : got;
      }
    }
  }
  const int piece = lane & 7;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint16_t* a = addr((lane & ~7) + i);
    if (a != nullptr && piece * 8 < cols)
      *reinterpret_cast<uint4*>(a + piece * 8) =
          make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
}

}  // namespace pact
