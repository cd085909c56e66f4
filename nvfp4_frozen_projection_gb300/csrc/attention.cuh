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
// A wait of a role that has nothing to do while others go through all the keys of a unit, at
// most those of the tensor: 20 us a tile of keys more, of which none takes 3.
__device__ __forceinline__ uint64_t unit_wait_ns(const AttnParams& p) {
  return kAttnWaitNs + (uint64_t)((uint32_t)p.tk >> 7) * 20000ull;
}
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
  int tile;  // of this sequence
};

// The order of units.  Up to 32 sequences: by the tiles that a unit goes over, in at most 32
// levels from the most to the fewest, so that no heavy unit comes last; a CTA takes unit k of
// the first row of gridDim.x units, the last but k of the second, and so on in turn (unit_of).
// More sequences: by sequence, then by tile, which costs something where lengths differ: 32 of
// 64 to 1700 tokens, 16/4 heads of 128, 79 us by levels and 95 in the sequences' order, backward
// 251 and 327.  Units of a role ascend, so its search goes on where the last one ended; 32
// sequences a step, one a lane.
//
// OVER_K: units are tiles of keys that go over tiles of tpt tokens; else units are `per`
// tokens that go over tiles of 128 keys.  With causal the first key tiles, or the last
// tokens, go over the most: rank 0 is the heaviest tile of a sequence.
template <bool OVER_K>
struct SeqFinder {
  const int* cu_q;
  const int* cu_k;
  int nseq, tq, tk;
  int per, tpt;
  bool causal;
  int b0 = -32, level = 0, step = 0;
  uint32_t base = 0;
  int q0 = 0, lq = 0, k0 = 0, lk = 0, n = 0;  // of this lane's sequence; n: its tiles
  int above = 0, here = 0;  // its tiles above this level, and with those in it
  uint32_t incl = 0;        // the level's tiles of the lanes up to this one

  __device__ __forceinline__ static int clampi(int v, int lo, int hi) {
    return v < lo ? lo : (v > hi ? hi : v);
  }

  __device__ __forceinline__ void load() {
    const int b = b0 + (int)(threadIdx.x & 31);
    q0 = lq = k0 = lk = n = 0;
    if (b < nseq) {
      q0 = clampi(__ldg(cu_q + b), 0, tq);
      lq = clampi(__ldg(cu_q + b + 1), q0, tq) - q0;
      k0 = clampi(__ldg(cu_k + b), 0, tk);
      lk = clampi(__ldg(cu_k + b + 1), k0, tk) - k0;
      n = ((OVER_K ? lk : lq) + per - 1) / per;
    }
  }

  // How many of the sequence's tiles go over `work` tiles or more (work > 0).
  __device__ __forceinline__ int count(int work) const {
    const int64_t off = (int64_t)lk - lq;
    if (OVER_K) {
      const int m = (lq + tpt - 1) / tpt - work;  // the last tile of tokens to begin with
      if (m < 0) return 0;
      const int64_t end = (int64_t)(m + 1) * tpt;
      if (!causal || end > lq) return n;
      const int64_t c = (end + off + 127) >> 7;
      return c < 0 ? 0 : (c > n ? n : (int)c);
    }
    const int64_t x = (int64_t)(work - 1) * 128 + 1;  // keys seen at least
    if (x > lk) return 0;
    if (!causal) return n;
    const int64_t y = x - off;  // tokens up to the tile's end at least
    if (y > lq) return 0;
    return y <= per ? n : n - (int)((y + per - 1) / per) + 1;
  }

  __device__ __forceinline__ void at_level() {
    above = here;
    here = level > 0 ? count(level) : n;
    incl = (uint32_t)(here - above);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if ((int)(threadIdx.x & 31) >= o) incl += up;
    }
  }

  __device__ __forceinline__ void take(Seq& s, int lane, int tile) {
    s.q0 = __shfl_sync(0xFFFFFFFFu, q0, lane);
    s.lq = __shfl_sync(0xFFFFFFFFu, lq, lane);
    s.k0 = __shfl_sync(0xFFFFFFFFu, k0, lane);
    s.lk = __shfl_sync(0xFFFFFFFFu, lk, lane);
    const int tiles = __shfl_sync(0xFFFFFFFFu, n, lane);
    s.tile = causal && !OVER_K ? tiles - 1 - tile : tile;
  }

  // Every lane of the warp calls this; false behind the last unit.
  __device__ __forceinline__ bool find(uint32_t t, Seq& s) {
    const bool levels = nseq <= 32;
    if (b0 < 0) {
      b0 = 0;
      load();
      level = 0;
      if (levels) {
        const int most = __reduce_max_sync(0xFFFFFFFFu, OVER_K ? (lq + tpt - 1) / tpt : (lk + 127) / 128);
        step = (most + 31) / 32;
        if (step < 1) step = 1;
        level = most;
      }
      at_level();
    }
    for (;;) {
      const unsigned hit = __ballot_sync(0xFFFFFFFFu, t < base + incl);
      if (hit) {
        const int l = __ffs(hit) - 1;
        // the rank within the sequence: those of higher levels, and of this one before it
        take(s, l, __shfl_sync(0xFFFFFFFFu, above, l) +
                       (int)(t - base - __shfl_sync(0xFFFFFFFFu, incl - (uint32_t)(here - above), l)));
        return true;
      }
      base += __shfl_sync(0xFFFFFFFFu, incl, 31);
      if (levels) {
        if (level <= 0) return false;
        level -= step;
      } else {
        b0 += 32;
        if (b0 >= nseq) return false;
        load();
        here = 0;
      }
      at_level();
    }
  }
};

__device__ __forceinline__ int clampi(int v, int lo, int hi) {
  return v < lo ? lo : (v > hi ? hi : v);
}

// Units end here whatever the offsets say; the host refuses sizes that need more (FastDiv).
constexpr uint32_t kMaxUnit = 0x7FFFFFFFu;

// Unit i of this CTA's.
__device__ __forceinline__ uint32_t unit_of(uint32_t i) {
  return i * gridDim.x + ((i & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// Whether token t is of a sequence.  Every lane of the warp calls this.
__device__ __forceinline__ bool in_sequence(const int* cu, int nseq, int rows, int64_t t) {
  bool in = false;
  if (t < rows)
    for (int b = threadIdx.x & 31; b < nseq; b += 32) {
      const int from = clampi(__ldg(cu + b), 0, rows);
      in = in || (t >= from && t < clampi(__ldg(cu + b + 1), from, rows));
    }
  return __any_sync(0xFFFFFFFFu, in);
}

template <bool OVER_K>
__device__ __forceinline__ SeqFinder<OVER_K> seq_finder(const AttnParams& p, int per) {
  SeqFinder<OVER_K> f;
  f.cu_q = p.cu_q;
  f.cu_k = p.cu_k;
  f.nseq = p.nseq;
  f.tq = p.tq;
  f.tk = p.tk;
  f.per = per;
  f.tpt = p.tpt;
  f.causal = p.causal != 0;
  return f;
}

// Token of a row of a tile; rows < 128 and gp <= 128, where the product is exact.
__device__ __forceinline__ int row_token(const AttnParams& p, int row) {
  return (int)(((uint32_t)row * p.gp_mul) >> 16);
}

// Rows of 64 BF16 columns held one a lane (w: 8 pieces of 16 bytes) go out as whole rows of
// 128 bytes, four an instruction: the lanes of each group of 8 exchange pieces, so that lane
// l of a group ends up with piece l of each of the group's rows.  Stored as they are held, a
// piece a lane, an instruction would touch 32 rows.  Row r of a tile is at
// out + (r / gp) ld + (r % gp) D; from: the warp's first row; rows: the tile's rows that are
// stored; cols: how many of the 64 columns there are.
__device__ __forceinline__ void store_rows64(uint32_t (&w)[32], int lane, int from, int rows,
                                             int cols, uint16_t* out, int64_t ld, int D, int gp,
                                             uint32_t gp_mul) {
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
  const int piece = lane & 7, r0 = from + (lane & ~7);
  const int t = (int)(((uint32_t)r0 * gp_mul) >> 16);
  int g = r0 - t * gp;
  uint16_t* a = out + (int64_t)t * ld + (int64_t)g * D + piece * 8;
  const int64_t wrap = ld - (int64_t)(gp - 1) * D;
  const int live = piece * 8 < cols ? rows - r0 : 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i < live)
      *reinterpret_cast<uint4*>(a) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    const bool last = ++g == gp;
    a += last ? wrap : (int64_t)D;
    g = last ? 0 : g;
  }
}

// Minus infinity in the columns from x on of 128 scores, by the bits of a word: eight of them
// become predicates in one instruction, where comparisons take one each.
__device__ __forceinline__ void mask_from(uint32_t* v, int x) {
#pragma unroll
  for (int c = 0; c < 128; c += 32) {
    // bits of the columns seen
    const int n = x - c;
    const uint32_t bits = n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u);
#pragma unroll
    for (int e = 0; e < 32; ++e) v[c + e] = (bits >> e & 1u) ? v[c + e] : 0xFF800000u;
  }
}

}  // namespace pact
