// Attention over packed sequences, backward.  The probabilities are computed again from the
// forward's lse, P = exp(scale S - lse):
//   delta = sum_d do o;  dP = do v^T;  dS = P (dP - delta);
//   dq = scale dS k;  dk = scale dS^T q;  dv = P^T do, the last two summed over the query
//   heads that share a key head.
//
// Three launches.  delta is a pass over do and o (HBM).  dq and dk|dv are kernels of their
// own, each with its sums in TMEM from the first tile to the last: seven products a tile in
// place of the five of one kernel, whose dq would have to be added up in memory over all key
// tiles, in an order that changes from run to run.  A CTA has one tile of 128 rows; two
// threads issue the products, two warpgroups hold a row a thread and half its columns each.
// Where there are few units, those of one of the two are cut up and a fourth launch adds what
// their parts make, in FP32.
//
//   dq:     rows are queries.  TMEM: S (0), dP (128), dS (256, BF16), dq (320).  One thread
//           issues S of the next keys as soon as this one has been read, the other dP of the
//           next keys and, once dS is there, dq += dS k.
//   dk|dv:  rows are keys, columns the (token, head) rows of a query tile; one thread issues
//           S^T and dv += P^T do, the other dP^T and dk += dS^T q.
//           D <= 64: S^T (0), dP^T (128), P^T (256), dS^T (320), dv (384), dk (448); the next
//           S^T or dP^T comes as soon as this one has been read.
//           D > 64: there is no room for that.  P^T lies over S^T, dS^T over dP^T, dv at 256,
//           dk at 384, and the next S^T comes behind dv += P^T do, the next dP^T behind
//           dk += dS^T q: MMAs of one thread run in order.
// So the tensor cores have work while exponentials are taken.  P and dS are rounded to BF16
// for their products, the type of the operands beside them; everything else is FP32.  Error of
// the gradients against 64 bits, relative: 0.0024, of which their own rounding is 0.0017.
//
// What bounds it (8 x 1024 causal, 32/8 heads of 128: 250 us, of which delta takes 24, dq 109
// and dk|dv 124 when each runs by itself).  dq: 1740 to 2000 cycles a tile, of which the
// products need 1536.  dk|dv: 2500, of which 2048; after P is there, dv += P^T do and the next
// S^T, 1024 cycles, and the signals lie between one exponential phase and the next.  At D = 64
// it is the latencies of the computing warps, two a scheduler: 1600 and 2350 cycles a tile, with
// the tensor pipe 30 % busy and issue slots 40 %.  The ends of units cost 4000 to 6000 cycles,
// against 4 to 30 tiles of such sequences (dq: 1 to 8 tiles a unit there, so a third of its time);
// the next launch starts on the SMs that dq leaves.  Seven products in place of five put the
// floor at 126 us in place of 90.
#include "attention.cuh"
#include "dependent.cuh"

namespace pact {

// TMEM column of step k (16 of 128 columns) of a BF16 operand.  OWN: it has 64 columns of its
// own.  Else it lies over the FP32 tile that it was made from: each warpgroup's half of that,
// 64 columns, becomes 32 at its own first column, so that neither half lies over what the
// other still reads.
template <bool OWN>
__device__ __forceinline__ uint32_t half_step(int k) {
  return OWN ? k * 8 : (k >> 2) * 64 + (k & 3) * 8;
}

// ------------------------------------------------------------------ delta
template <int SEG>
__global__ void __launch_bounds__(256) k_attn_delta(const AttnParams p) {
  const int lane = threadIdx.x & 31, sl = lane & (SEG - 1);
  const int64_t row = (int64_t)blockIdx.x * (256 / SEG) + threadIdx.x / SEG;
  const int64_t rows = (int64_t)p.tq * p.hq;
  const bool live = row < rows && sl * 8 < p.D;
  const int64_t t = live ? row / p.hq : 0;
  const int h = live ? (int)(row - t * p.hq) : 0;
  float sum = 0.0f;
  if (live) {
    float a[8], b[8];
    bf16x8_to_f32(*reinterpret_cast<const uint4*>(p.dout + t * p.lddo + (int64_t)h * p.D + sl * 8), a);
    bf16x8_to_f32(*reinterpret_cast<const uint4*>(p.o_in + t * p.ldoi + (int64_t)h * p.D + sl * 8), b);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = __fmaf_rn(a[e], b[e], sum);
  }
#pragma unroll
  for (int o = SEG / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (live && sl == 0 && PACT_IN(t < p.tq && h < p.hq)) p.delta[(int64_t)h * p.tq + t] = sum;
}

// A row of sums times f, FP32: `cols` columns out of TMEM (zeros, when there is none).
__device__ __forceinline__ void store_part(float* out, uint32_t ta, int cols, bool store, bool have,
                                           float f) {
  for (int b = 0; b < cols; b += 16) {
    uint32_t o[16];
    if (have) {
      tmem_ld16(ta + b, o);
      tmem_ld_wait16(o);
    }
    if (store) {
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (have && f != 0.0f)
          x = make_float4(__uint_as_float(o[e]) * f, __uint_as_float(o[e + 1]) * f,
                          __uint_as_float(o[e + 2]) * f, __uint_as_float(o[e + 3]) * f);
        *reinterpret_cast<float4*>(out + b + e) = x;
      }
    }
  }
}

// ------------------------------------------------------------------ a ring of tiles
// The copying warp's side of a ring of shared-memory tiles.  `valid` rows of a tile belong to
// the sequence; a tile with fewer than `rows` has the others zeroed before the MMAs see it.
template <int BOXES, int STAGES>
struct TileRing {
  static constexpr uint32_t TILE = BOXES * kBox;
  uint32_t tiles;  // shared address of the ring
  uint8_t* mem;
  uint32_t full, empty, tail;
  volatile uint32_t* abort_flag;
  int stage = 0;
  uint32_t phase = 0, tails = 0, pend = 0, pend_par = 0;

  __device__ __forceinline__ bool load(const CUtensorMap* tm, int head, int row, int rows,
                                       int valid, int lane) {
    if (!mbar_wait(empty + 8 * stage, phase ^ 1u, kAttnWaitNs, abort_flag)) return false;
    const bool whole = valid >= rows;
    const uint32_t dst = tiles + stage * TILE, bar = whole ? full + 8 * stage : tail;
    if (lane == 0) {
      mbar_expect_tx(bar, (uint32_t)rows * 128 * BOXES);
#pragma unroll
      for (int b = 0; b < BOXES; ++b) tma_load_3d(dst + b * kBox, tm, b * 64, head, row, bar);
    }
    __syncwarp();
    if (whole) {
      pend |= 1u << stage;
      pend_par = (pend_par & ~(1u << stage)) | (phase << stage);
    } else {
      if (!mbar_wait(tail, tails & 1u, kAttnWaitNs, nullptr)) return false;
      ++tails;
      zero_rows(mem + stage * TILE, BOXES, valid, lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full + 8 * stage);
    }
    if (++stage == STAGES) {
      stage = 0;
      phase ^= 1u;
    }
    return true;
  }
  // copies in flight land before the CTA can exit
  __device__ __forceinline__ void drain() {
    for (int s = 0; s < STAGES; ++s)
      if (pend & (1u << s)) mbar_wait(full + 8 * s, (pend_par >> s) & 1u, 10000000ull, nullptr);
  }
};

// -lse log2 e and delta of a query tile's rows, four a lane; `none` for the -lse of rows that
// hold no query.  And their way through shared memory.
__device__ __forceinline__ void load_stats(const AttnParams& p, const Seq& s, int h0, int tok0,
                                           float none, int lane, float (&nl)[4], float (&de)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int x = k * 32 + lane, rt = row_token(p, x), tok = tok0 + rt;
    nl[k] = none;
    de[k] = 0.0f;
    if (x < p.tpt * p.gp && tok < s.lq) {
      const int64_t at = (int64_t)(h0 + x - rt * p.gp) * p.tq + s.q0 + tok;
      nl[k] = -p.lse_in[at] * kLog2e;
      de[k] = p.delta[at];
    }
  }
}
__device__ __forceinline__ void store_stats(float* st, int lane, const float (&nl)[4],
                                            const float (&de)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    st[k * 32 + lane] = nl[k];
    st[128 + k * 32 + lane] = de[k];
  }
  __syncwarp();
}

template <int DP>
struct BwdCfg {
  static constexpr int BOXES = DP / 64;
  static constexpr uint32_t TILE = BOXES * kBox;
  static constexpr int STAGES = DP == 64 ? 8 : 5;
  // dq: rings of K, which a tile holds from S to dq, and of V
  static constexpr int NK = DP == 64 ? 4 : 3, NV = STAGES - NK;
  static constexpr bool OWN_P = DP == 64;  // dk|dv: P and dS have TMEM columns of their own
  static constexpr int SUM_COL = OWN_P ? 384 : 256, SUM_STEP = OWN_P ? 64 : 128;
  // two tiles that stay for a unit, the ring, and two buffers of 128 -lse and delta
  static constexpr uint32_t RING_OFF = 2 * TILE, STAT_OFF = RING_OFF + STAGES * TILE;
  static constexpr uint32_t BAR_OFF = STAT_OFF + 2048;
  // 23 barriers and the ring's; behind them the TMEM slot and the abort flag
  static constexpr uint32_t SLOT_OFF = BAR_OFF + 184 + 16 * STAGES, SMEM = SLOT_OFF + 16;
  static_assert(SMEM <= 232448, "shared memory");
};

// Shared addresses of the barriers; those with a number in brackets lie 8 bytes apart.
struct BwdBars {
  uint32_t fix_full, fix_empty;  // [2] the two tiles of a unit
  uint32_t s_full, dp_full;      // S and dP are there
  uint32_t s_read, dp_read;      // and have been read
  uint32_t p_full;               // [2] P is there: the first and the second half of each half
  uint32_t ds_full;              // dS is there
  uint32_t p_empty, ds_empty;    // and their products are done
  uint32_t acc_full;
  uint32_t tail;                   // [2]
  uint32_t final_bar;              // [2]
  uint32_t stat_full, stat_empty;  // [2] -lse and delta
  uint32_t full, empty;            // the ring
};
__device__ __forceinline__ BwdBars bwd_bars(uint32_t b, int stages) {
  BwdBars r;
  r.fix_full = b;
  r.fix_empty = b + 16;
  r.s_full = b + 32;
  r.dp_full = b + 40;
  r.s_read = b + 48;
  r.dp_read = b + 56;
  r.p_full = b + 64;
  r.ds_full = b + 80;
  r.p_empty = b + 88;
  r.ds_empty = b + 96;
  r.acc_full = b + 104;
  r.tail = b + 112;
  r.final_bar = b + 128;
  r.stat_full = b + 144;
  r.stat_empty = b + 160;
  r.full = b + 184;
  r.empty = r.full + 8 * stages;
  return r;
}

// ------------------------------------------------------------------ dq
// PARTS: the key tiles of a unit are cut into p.parts runs, each a unit of its own.
template <int DP, bool PARTS>
__global__ void __launch_bounds__(384, 1)
    k_attn_dq(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmdO,
              const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
              const AttnParams p) {
  using C = BwdCfg<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_addr(smem);
  if (base & 1023u) {  // the swizzle needs it, and the budget leaves no room to round up
    if (threadIdx.x == 0) atomicOr(p.status, (unsigned)PACT_DEV_BOUNDS);
    return;
  }
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::SLOT_OFF);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::SLOT_OFF + 4);
  let_dependents_start();  // dk|dv needs nothing of dq: it takes the SMs that this one leaves
  const BwdBars B = bwd_bars(base + C::BAR_OFF, C::STAGES);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(B.fix_full + 8 * i, 1);
      mbar_init(B.fix_empty + 8 * i, 1);
    }
    mbar_init(B.s_full, 1);
    mbar_init(B.dp_full, 1);
    mbar_init(B.s_read, 8);  // the computing warps
    mbar_init(B.dp_read, 8);
    mbar_init(B.ds_full, 8);
    mbar_init(B.ds_empty, 1);
    mbar_init(B.acc_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(B.tail + 8 * i, 1);
      mbar_init(B.final_bar + 8 * i, 1);
      mbar_init(B.stat_full + 8 * i, 1);
      mbar_init(B.stat_empty + 8 * i, 8);
    }
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(B.full + 8 * s, 1);
      mbar_init(B.empty + 8 * s, 2);  // the issuers
    }
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  SeqFinder<false> finder = seq_finder<false>(p, p.tpt);
  Seq s;
  int tok0, nk, kvh, h0, part = 0;
  auto next_unit = [&](uint32_t u) {
    if (u >= kMaxUnit) return false;
    if (PARTS) {
      const uint32_t whole = u / (uint32_t)p.parts;
      part = (int)(u - whole * (uint32_t)p.parts);
      u = whole;
    }
    const uint32_t t = p.units_div.div(u);
    const int hu = (int)(u - t * p.units_h);
    if (!finder.find(t, s)) return false;
    kvh = p.subs == 1 ? hu : hu / p.subs;
    h0 = kvh * p.group + (hu - kvh * p.subs) * p.gp;
    tok0 = s.tile * p.tpt;
    int kend = s.lk;
    if (p.causal) kend = clampi(min(tok0 + p.tpt, s.lq) + s.lk - s.lq, 0, s.lk);
    nk = (kend + 127) / 128;
    if (PARTS) {  // keys are counted from the first one of this part on
      const int first = (int)((int64_t)nk * part / p.parts);
      nk = (int)((int64_t)nk * (part + 1) / p.parts) - first;
      s.k0 += first * 128;
      s.lk -= first * 128;
    }
    return true;
  };

  if (warp >= 8) {
    setmaxnreg_dec<72>();
    if (warp == 8) {
      // ------------------------------------------------------------ copies
      TileRing<C::BOXES, C::NK> kring;
      TileRing<C::BOXES, C::NV> vring;
      kring.tiles = base + C::RING_OFF;
      kring.mem = smem + C::RING_OFF;
      kring.full = B.full;
      kring.empty = B.empty;
      kring.tail = B.tail;
      vring.tiles = kring.tiles + C::NK * C::TILE;
      vring.mem = kring.mem + C::NK * C::TILE;
      vring.full = B.full + 8 * C::NK;
      vring.empty = B.empty + 8 * C::NK;
      vring.tail = B.tail + 8;
      kring.abort_flag = vring.abort_flag = abort_flag;
      uint32_t uses = 0;
      bool ok = true;
      auto load_fix = [&](int i, const CUtensorMap* tm) {
        if (!mbar_wait(B.fix_empty + 8 * i, (uses & 1u) ^ 1u, kAttnWaitNs, abort_flag)) return false;
        if (lane == 0) {
          mbar_expect_tx(B.fix_full + 8 * i, (uint32_t)(p.tpt * p.gp) * 128 * C::BOXES);
#pragma unroll
          for (int b = 0; b < C::BOXES; ++b)
            tma_load_3d(base + i * C::TILE + b * kBox, tm, b * 64, h0, s.q0 + tok0, B.fix_full + 8 * i);
        }
        __syncwarp();
        return true;
      };
      uint32_t fixed = 0;
      for (uint32_t turn = 0; ok && next_unit(unit_of(turn)); ++turn) {
        if (nk == 0) continue;
        for (int j = 0; j < nk && ok; ++j) {
          const int row = s.k0 + j * 128, valid = s.lk - j * 128;
          if (j == 0) {
            ok = load_fix(0, &tmQ);
            if (ok) fixed = 1;
          }
          ok = ok && kring.load(&tmK, kvh, row, 128, valid, lane);
          if (j == 0) {
            ok = ok && load_fix(1, &tmdO);
            if (ok) fixed = 2;
          }
          ok = ok && vring.load(&tmV, kvh, row, 128, valid, lane);
        }
        if (ok) {
          ++uses;
          fixed = 0;
        }
      }
      if (!ok) {
        if (lane == 0) raise_error(abort_flag, p.status, PACT_DEV_TIMEOUT | PACT_DEV_ROLE_TMA);
        kring.drain();
        vring.drain();
        for (uint32_t i = 0; i < fixed; ++i) mbar_wait(B.fix_full + 8 * i, uses & 1u, 10000000ull, nullptr);
      }
    } else if (warp < 11) {
      // ------------------------------------------------------------ MMAs
      const int issuer = warp - 9;
      RingPos k, v;
      uint32_t uses = 0, tiles = 0;
      bool ok = true;
      const uint32_t idesc_s = attn_idesc(128, false), idesc_d = attn_idesc(p.D, true);
      const int ksteps = p.D / 16;
      const bool lead = elected();
      const uint64_t dfix = desc_k(base + issuer * C::TILE);
      const uint64_t dk0 = desc_k(base + C::RING_OFF), dn0 = desc_n(base + C::RING_OFF);
      auto wait = [&](uint32_t bar, uint32_t par) {
        return mbar_wait(bar, par, kAttnWaitNs, abort_flag);
      };
      // 128 x 128 product of this issuer's fixed tile and a ring tile over the head's columns
      auto mma_rows = [&](uint32_t d, int st) {
        const uint64_t db = dk0 + (uint64_t)(st * (C::TILE >> 4));
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
          if (k < ksteps) mma_bf16(tmem + d, step_k(dfix, k), step_k(db, k), idesc_s, k > 0);
      };
      for (uint32_t turn = 0; ok && next_unit(unit_of(turn)); ++turn) {
        if (nk == 0) continue;
        if (!(ok = wait(B.fix_full + 8 * issuer, uses & 1u))) break;
        ++uses;
        if (issuer == 0) {
          for (int j = 0; j < nk; ++j, ++tiles) {
            if (!(ok = wait(B.full + 8 * k.stage, k.phase) && wait(B.s_read, (tiles & 1u) ^ 1u)))
              break;
            tc_fence_after();
            if (lead) {
              mma_rows(0, k.stage);
              mma_commit(B.s_full);
              mma_commit(B.empty + 8 * k.stage);
              if (j + 1 == nk) mma_commit(B.fix_empty);
            }
            __syncwarp();
            k.advance(C::NK);
          }
        } else {
          for (int j = 0; j <= nk; ++j) {
            // dP of tile j, dq of tile j - 1
            if (j < nk) {
              const int st = C::NK + v.stage;
              if (!(ok = wait(B.full + 8 * st, v.phase) &&
                         wait(B.dp_read, ((tiles + j) & 1u) ^ 1u)))
                break;
              tc_fence_after();
              if (lead) {
                mma_rows(128, st);
                mma_commit(B.dp_full);
                mma_commit(B.empty + 8 * st);  // for both issuers: the other has no use of V
                mma_commit(B.empty + 8 * st);
                if (j + 1 == nk) mma_commit(B.fix_empty + 8);
              }
              __syncwarp();
              v.advance(C::NV);
            }
            if (j > 0) {
              if (!(ok = wait(B.full + 8 * k.stage, k.phase) &&
                         wait(B.ds_full, (tiles + j - 1) & 1u)))
                break;
              tc_fence_after();
              if (lead) {
                const uint64_t d = dn0 + (uint64_t)(k.stage * (C::TILE >> 4));
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  mma_bf16_ta(tmem + 320, tmem + 256 + half_step<true>(i), step_n(d, i), idesc_d,
                              (j > 1 || i > 0) ? 1u : 0u);
                mma_commit(B.ds_empty);
                mma_commit(B.empty + 8 * k.stage);
                if (j == nk) mma_commit(B.acc_full);
              }
              __syncwarp();
              k.advance(C::NK);
            }
          }
          tiles += nk;
        }
      }
      if (lead) {
        if (!ok) raise_error(abort_flag, p.status, PACT_DEV_TIMEOUT | PACT_DEV_ROLE_MMA);
        mma_commit(B.final_bar + 8 * issuer);
        mbar_wait(B.final_bar + 8 * issuer, 0, kAttnWaitNs, nullptr);
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------ -lse and delta of the rows
      uint32_t units = 0;
      bool ok = true;
      for (uint32_t turn = 0; ok && next_unit(unit_of(turn)); ++turn) {
        if (nk == 0) continue;
        const uint32_t buf = units & 1u;
        float nl[4], de[4];
        load_stats(p, s, h0, tok0, 0.0f, lane, nl, de);
        // at most two units ahead: it waits while the computing warps go through one
        if (!(ok = mbar_wait(B.stat_empty + 8 * buf, ((units >> 1) & 1u) ^ 1u, unit_wait_ns(p), abort_flag)))
          break;
        store_stats(reinterpret_cast<float*>(smem + C::STAT_OFF + buf * 1024), lane, nl, de);
        if (lane == 0) mbar_arrive(B.stat_full + 8 * buf);
        ++units;
      }
      if (!ok && lane == 0) raise_error(abort_flag, p.status, PACT_DEV_TIMEOUT | PACT_DEV_ROLE_SF);
    }
  } else {
    // -------------------------------------------------------------- a row and 64 columns a thread
    setmaxnreg_inc<216>();
    const int half = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
    const float c = p.c;
    uint32_t tiles = 0, uses = 0, turn = 0;
    bool ok = true;
    for (bool more = next_unit(unit_of(0)); more;) {
      const int tok = tok0 + row_token(p, row), n = nk;
      const int lim = p.causal ? min(s.lk, tok + 1 + s.lk - s.lq) : s.lk;
      const int lim_all = p.causal ? min(s.lk, tok0 + 1 + s.lk - s.lq) : s.lk;
      float nlse = 0.0f, delta = 0.0f;
      if (n > 0) {
        const uint32_t buf = uses & 1u;
        if (!(ok = mbar_wait(B.stat_full + 8 * buf, (uses >> 1) & 1u, kAttnWaitNs, abort_flag))) break;
        const float* st = reinterpret_cast<const float*>(smem + C::STAT_OFF + buf * 1024);
        nlse = st[row];
        delta = st[128 + row];
        __syncwarp();
        if (lane == 0) mbar_arrive(B.stat_empty + 8 * buf);
      }
      // S of the next tile is loaded while dS is stored
      uint32_t v[64];
      const uint32_t ts = tl + half * 64, td = tl + 128 + half * 64;
      auto load_s = [&](uint32_t tile) {
        if (!mbar_wait(B.s_full, tile & 1u, kAttnWaitNs, abort_flag)) return false;
        tc_fence_after();
        tmem_ld32(ts, v);
        tmem_ld32(ts + 32, v + 32);
        return true;
      };
      auto s_loaded = [&]() {
        tmem_ld_wait32(v);
        tmem_ld_wait32(v + 32);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(B.s_read);
      };
      if (n > 0) {
        if (!(ok = load_s(tiles))) break;
        s_loaded();
      }
      for (int j = 0; j < n; ++j, ++tiles) {
        float pr[64];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float2 x = __ffma2_rn(
              make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])),
              make_float2(c, c), make_float2(nlse, nlse));
          pr[2 * e] = ex2_ftz(x.x);
          pr[2 * e + 1] = ex2_ftz(x.y);
        }
        if ((j + 1) * 128 > lim_all) {
#pragma unroll
          for (int q = 0; q < 64; q += 32) {
            const int x = lim - j * 128 - half * 64 - q;  // columns that are seen
            const uint32_t bits = x >= 32 ? 0xFFFFFFFFu : (x <= 0 ? 0u : (1u << x) - 1u);
#pragma unroll
            for (int e = 0; e < 32; ++e) pr[q + e] = (bits >> e & 1u) ? pr[q + e] : 0.0f;
          }
        }
        if (!(ok = mbar_wait(B.dp_full, tiles & 1u, kAttnWaitNs, abort_flag))) break;
        tc_fence_after();
        tmem_ld32(td, v);
        tmem_ld32(td + 32, v + 32);
        tmem_ld_wait32(v);
        tmem_ld_wait32(v + 32);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(B.dp_read);
        uint32_t w[32];
#pragma unroll
        for (int e = 0; e < 32; ++e)
          w[e] = pack_bf16x2(pr[2 * e] * (__uint_as_float(v[2 * e]) - delta),
                             pr[2 * e + 1] * (__uint_as_float(v[2 * e + 1]) - delta));
        if (!(ok = mbar_wait(B.ds_empty, (tiles & 1u) ^ 1u, kAttnWaitNs, abort_flag))) break;
        tc_fence_after();
        tmem_st32(tl + 256 + half * 32, w);
        if (j + 1 < n && !(ok = load_s(tiles + 1))) break;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(B.ds_full);
        if (j + 1 < n) s_loaded();
      }
      if (!ok) break;
      // the search for the next unit runs while the last product does
      const int rows = min(p.tpt, s.lq - tok0) * p.gp, t0 = s.q0 + tok0, head = h0;
      float* const own = PARTS ? p.part_o + (int64_t)part * p.tq * p.hq * p.D : nullptr;
      more = next_unit(unit_of(++turn));
      if (n > 0) {
        if (!(ok = mbar_wait(B.acc_full, uses & 1u, kAttnWaitNs, abort_flag))) break;
        ++uses;
        tc_fence_after();
      }
      const int b = half * 64, cols = p.D - b;
      if (cols <= 0) continue;
      if (PARTS) {
        const int t = row_token(p, row);
        const bool store = row < rows && PACT_IN(t0 + t < p.tq);
        store_part(own + ((int64_t)(t0 + t) * p.hq + head + row - t * p.gp) * p.D + b, tl + 320 + b,
                   min(cols, 64), store, n > 0, lim > 0 ? p.scale : 0.0f);
        continue;
      }
      uint32_t w[32];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint32_t o[16];
        const bool have = n > 0 && h * 16 < cols;
        if (have) {
          tmem_ld16(tl + 320 + b + 16 * h, o);
          tmem_ld_wait16(o);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[8 * h + e] = have && lim > 0 ? pack_bf16x2(__uint_as_float(o[2 * e]) * p.scale,
                                                       __uint_as_float(o[2 * e + 1]) * p.scale)
                                         : 0u;
      }
      if (PACT_IN(t0 < p.tq))
        store_rows64(w, lane, quarter * 32, rows, min(cols, 64),
                     p.dq + (int64_t)t0 * p.lddq + (int64_t)head * p.D + b, p.lddq, p.D, p.gp,
                     p.gp_mul);
    }
    if (!ok && lane == 0) raise_error(abort_flag, p.status, PACT_DEV_TIMEOUT | PACT_DEV_ROLE_EPI);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ dk and dv
// PARTS: the query tiles of a unit are cut into p.parts_q runs, each a unit of its own.
template <int DP, bool PARTS>
__global__ void __launch_bounds__(384, 1)
    k_attn_dkdv(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmdO,
                const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const AttnParams p) {
  using C = BwdCfg<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_addr(smem);
  if (base & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.status, (unsigned)PACT_DEV_BOUNDS);
    return;
  }
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::SLOT_OFF);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::SLOT_OFF + 4);
  const BwdBars B = bwd_bars(base + C::BAR_OFF, C::STAGES);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(B.fix_full, 1);
    mbar_init(B.fix_empty, 2);  // the issuers
    mbar_init(B.s_full, 1);
    mbar_init(B.dp_full, 1);
    mbar_init(B.s_read, 8);  // the computing warps
    mbar_init(B.dp_read, 8);
    mbar_init(B.p_full, 8);
    mbar_init(B.p_full + 8, 8);
    mbar_init(B.ds_full, 8);
    mbar_init(B.p_empty, 1);
    mbar_init(B.ds_empty, 1);
    mbar_init(B.acc_full, 2);
    mbar_init(B.tail, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(B.final_bar + 8 * i, 1);
      mbar_init(B.stat_full + 8 * i, 1);
      mbar_init(B.stat_empty + 8 * i, 8);
    }
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(B.full + 8 * s, 1);
      mbar_init(B.empty + 8 * s, 2);
    }
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == 9) {
    // rows that no copy writes (gp that does not divide 128) are zeros for good
    for (int st = 0; st < C::STAGES; ++st)
      zero_rows(smem + C::RING_OFF + st * C::TILE, C::BOXES, p.tpt * p.gp, lane);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (PARTS) let_dependents_start();

  SeqFinder<true> finder = seq_finder<true>(p, 128);
  Seq s;
  // first key; first query tile and how many; iterations, from i0 on, over them and the subgroups
  int key0, kvh, qt0, nqt, n, i0 = 0, part = 0;
  auto next_unit = [&](uint32_t u) {
    if (u >= kMaxUnit) return false;
    if (PARTS) {
      const uint32_t whole = u / (uint32_t)p.parts_q;
      part = (int)(u - whole * (uint32_t)p.parts_q);
      u = whole;
    }
    const uint32_t t = p.hk_div.div(u);
    kvh = (int)(u - t * p.hk);
    if (!finder.find(t, s)) return false;
    key0 = s.tile * 128;
    qt0 = 0;
    if (p.causal) qt0 = clampi(key0 - (s.lk - s.lq), 0, s.lq) / p.tpt;
    nqt = (s.lq + p.tpt - 1) / p.tpt - qt0;
    n = nqt * p.subs;
    if (PARTS) {
      i0 = (int)((int64_t)n * part / p.parts_q);
      n = (int)((int64_t)n * (part + 1) / p.parts_q) - i0;
    }
    return true;
  };
  // iteration i of a unit: its first query head, and its tile's first token
  auto tile_of = [&](int i, int& h0, int& tok0) {
    if (PARTS) i += i0;
    const int sub = p.subs == 1 ? 0 : i / nqt;
    h0 = kvh * p.group + sub * p.gp;
    tok0 = (qt0 + i - sub * nqt) * p.tpt;
  };

  if (warp >= 8) {
    setmaxnreg_dec<72>();
    if (warp == 8) {
      // ------------------------------------------------------------ copies
      TileRing<C::BOXES, C::STAGES> ring;
      ring.tiles = base + C::RING_OFF;
      ring.mem = smem + C::RING_OFF;
      ring.full = B.full;
      ring.empty = B.empty;
      ring.tail = B.tail;
      ring.abort_flag = abort_flag;
      uint32_t uses = 0;
      bool ok = true, fixed = false;
      for (uint32_t turn = 0; ok && next_unit(unit_of(turn)); ++turn) {
        if (n == 0) continue;
        if (!(ok = mbar_wait(B.fix_empty, (uses & 1u) ^ 1u, kAttnWaitNs, abort_flag))) break;
        if (lane == 0) {
          mbar_expect_tx(B.fix_full, 2 * C::TILE);
#pragma unroll
          for (int b = 0; b < C::BOXES; ++b) {
            tma_load_3d(base + b * kBox, &tmK, b * 64, kvh, s.k0 + key0, B.fix_full);
            tma_load_3d(base + C::TILE + b * kBox, &tmV, b * 64, kvh, s.k0 + key0, B.fix_full);
          }
        }
        __syncwarp();
        fixed = true;
        for (int i = 0; i < n && ok; ++i) {
          int h0, tok0;
          tile_of(i, h0, tok0);
          const int rows = p.tpt * p.gp, valid = min(p.tpt, s.lq - tok0) * p.gp;
          ok = ring.load(&tmQ, h0, s.q0 + tok0, rows, valid, lane);
          ok = ok && ring.load(&tmdO, h0, s.q0 + tok0, rows, valid, lane);
        }
        if (ok) {
          ++uses;
          fixed = false;
        }
      }
      if (!ok) {
        if (lane == 0) raise_error(abort_flag, p.status, PACT_DEV_TIMEOUT | PACT_DEV_ROLE_TMA);
        ring.drain();
        if (fixed) mbar_wait(B.fix_full, uses & 1u, 10000000ull, nullptr);
      }
    } else if (warp < 11) {
      // ------------------------------------------------------------ MMAs
      // issuer 0: S^T = k q^T and dv += P^T do;  issuer 1: dP^T = v do^T and dk += dS^T q
      const int issuer = warp - 9;
      RingPos at;  // of Q of the current tile; dO follows it
      uint32_t uses = 0, tiles = 0;
      bool ok = true;
      const uint32_t idesc_s = attn_idesc(128, false), idesc_d = attn_idesc(p.D, true);
      const int ksteps = p.D / 16;
      const bool lead = elected();
      const uint64_t dfix = desc_k(base + issuer * C::TILE);
      const uint64_t dk0 = desc_k(base + C::RING_OFF), dn0 = desc_n(base + C::RING_OFF);
      constexpr bool OWN = C::OWN_P;
      const uint32_t sum = tmem + C::SUM_COL + issuer * C::SUM_STEP, prod = tmem + issuer * 128;
      const uint32_t in_col = OWN ? tmem + 256 + issuer * 64 : prod;
      const uint32_t read = issuer ? B.dp_read : B.s_read;
      const uint32_t in_empty = issuer ? B.ds_empty : B.p_empty;
      const uint32_t out_full = issuer ? B.dp_full : B.s_full;
      auto wait = [&](uint32_t bar, uint32_t par) {
        return mbar_wait(bar, par, kAttnWaitNs, abort_flag);
      };
      for (uint32_t turn = 0; ok && next_unit(unit_of(turn)); ++turn) {
        if (n == 0) continue;
        if (!(ok = wait(B.fix_full, uses & 1u))) break;
        ++uses;
        for (int i = 0; i <= n; ++i) {
          // the sum of tile i - 1, over dO (issuer 0) or Q (1), and the product of tile i, over
          // Q (issuer 0) or dO (1)
          RingPos r = at, x = at;
          x.advance(C::STAGES, issuer);
          // one or two places back, which is a turn of the parity further on
          r.advance(C::STAGES, C::STAGES - 2 + (issuer ? 0 : 1));
          // P comes in two parts, steps 0 1 4 5 and 2 3 6 7: the first one's product runs
          // while the second is computed.  dS, which has time, comes whole.
          auto issue_sum = [&]() {
            if (!(ok = wait(B.full + 8 * r.stage, r.phase ^ 1u))) return;
            // with P it is the next S that the computing warps wait for: what it needs first
            if (!OWN && !issuer && i < n && !(ok = wait(B.full + 8 * x.stage, x.phase))) return;
            const uint64_t d = dn0 + (uint64_t)(r.stage * (C::TILE >> 4));
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              if (part == 0 || !issuer) {
                if (!(ok = wait(issuer ? B.ds_full : B.p_full + 8 * part, (tiles + i - 1) & 1u))) return;
                tc_fence_after();
              }
              if (lead) {
#pragma unroll
                for (int k = 2 * part; k < 2 * part + 6; k += (k & 1) ? 3 : 1)
                  mma_bf16_ta(sum, in_col + half_step<OWN>(k), step_n(d, k), idesc_d,
                              (i > 1 || k > 0) ? 1u : 0u);
              }
              __syncwarp();
            }
          };
          auto sum_issued = [&]() {
            if (lead) {
              if (OWN) mma_commit(in_empty);
              mma_commit(B.empty + 8 * r.stage);
              if (i == n) mma_commit(B.acc_full);
            }
            __syncwarp();
          };
          if (!OWN && i > 0) {
            issue_sum();
            if (!ok) break;
            if (issuer || i == n) sum_issued();
          }
          if (i < n) {
            if ((OWN || issuer || i == 0) && !(ok = wait(B.full + 8 * x.stage, x.phase))) break;
            if (OWN && !(ok = wait(read, ((tiles + i) & 1u) ^ 1u))) break;
            tc_fence_after();
            if (lead) {
              const uint64_t d = dk0 + (uint64_t)(x.stage * (C::TILE >> 4));
#pragma unroll
              for (int k = 0; k < DP / 16; ++k)
                if (k < ksteps) mma_bf16(prod, step_k(dfix, k), step_k(d, k), idesc_s, k > 0);
              mma_commit(out_full);
              mma_commit(B.empty + 8 * x.stage);
              if (i + 1 == n) mma_commit(B.fix_empty);
            }
            __syncwarp();
            if (!OWN && !issuer && i > 0) sum_issued();
          }
          if (OWN && i > 0) {
            issue_sum();
            if (!ok) break;
            sum_issued();
          }
          if (i < n) at.advance(C::STAGES, 2);
        }
        tiles += n;
      }
      if (lead) {
        if (!ok) raise_error(abort_flag, p.status, PACT_DEV_TIMEOUT | PACT_DEV_ROLE_MMA);
        mma_commit(B.final_bar + 8 * issuer);
        mbar_wait(B.final_bar + 8 * issuer, 0, kAttnWaitNs, nullptr);
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------ -lse and delta of the columns
      uint32_t tiles = 0;
      bool ok = true;
      for (uint32_t turn = 0; ok && next_unit(unit_of(turn)); ++turn) {
        for (int i = 0; i < n; ++i, ++tiles) {
          int h0, tok0;
          tile_of(i, h0, tok0);
          const uint32_t buf = tiles & 1u;
          float nl[4], de[4];
          load_stats(p, s, h0, tok0, -INFINITY, lane, nl, de);  // rows of no query: P = 0
          if (!(ok = mbar_wait(B.stat_empty + 8 * buf, ((tiles >> 1) & 1u) ^ 1u, kAttnWaitNs,
                               abort_flag)))
            break;
          store_stats(reinterpret_cast<float*>(smem + C::STAT_OFF + buf * 1024), lane, nl, de);
          if (lane == 0) mbar_arrive(B.stat_full + 8 * buf);
        }
      }
      if (!ok && lane == 0) raise_error(abort_flag, p.status, PACT_DEV_TIMEOUT | PACT_DEV_ROLE_SF);
    }
  } else {
    // -------------------------------------------------------------- a key and 64 columns a thread
    setmaxnreg_inc<216>();
    const int half = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t tl = tmem + lanes + half * 64, tp = tmem + lanes + 256 + half * 32;
    const float c = p.c;
    uint32_t tiles = 0, uses = 0;
    bool ok = true;
    for (uint32_t turn = 0; ok && next_unit(unit_of(turn)); ++turn) {
      const int key = key0 + row;
      // OWN_P: S of the next tile is there early, and is loaded while dS is stored
      uint32_t v[64];
      auto load_s = [&](uint32_t tile) {
        if (!mbar_wait(B.stat_full + 8 * (tile & 1u), (tile >> 1) & 1u, kAttnWaitNs, abort_flag) ||
            !mbar_wait(B.s_full, tile & 1u, kAttnWaitNs, abort_flag))
          return false;
        tc_fence_after();
        tmem_ld32(tl, v);
        tmem_ld32(tl + 32, v + 32);
        return true;
      };
      auto s_loaded = [&]() {
        tmem_ld_wait32(v);
        tmem_ld_wait32(v + 32);
        if (C::OWN_P) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(B.s_read);
        }
      };
      if (C::OWN_P && n > 0) {
        if (!(ok = load_s(tiles))) break;
        s_loaded();
      }
      for (int i = 0; i < n; ++i, ++tiles) {
        int h0, tok0;
        tile_of(i, h0, tok0);
        const uint32_t buf = tiles & 1u;
        const float* st = reinterpret_cast<const float*>(smem + C::STAT_OFF + buf * 1024) + half * 64;
        if (!C::OWN_P) {
          if (!(ok = load_s(tiles))) break;
          s_loaded();
        }
        // the first column whose token sees this key
        int x = 0;
        if (p.causal && key0 + 127 - (s.lk - s.lq) > tok0) {
          const int64_t x0 = (int64_t)(key - (s.lk - s.lq) - tok0) * p.gp - half * 64;
          x = (int)(x0 > 64 ? 64 : (x0 < 0 ? 0 : x0));
        }
        const bool masked = __any_sync(0xFFFFFFFFu, x > 0);
        if (C::OWN_P) {
          if (!(ok = mbar_wait(B.p_empty, (tiles & 1u) ^ 1u, kAttnWaitNs, abort_flag))) break;
          tc_fence_after();
        }
        float pr[64];
        uint32_t w[32];
#pragma unroll
        for (int part = 0; part < 2; ++part) {
#pragma unroll
          for (int e = 8 * part; e < 8 * part + 8; ++e) {
            const float4 nl = *reinterpret_cast<const float4*>(st + 4 * e);
            const float2 a = __ffma2_rn(
                make_float2(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1])),
                make_float2(c, c), make_float2(nl.x, nl.y));
            const float2 b = __ffma2_rn(
                make_float2(__uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3])),
                make_float2(c, c), make_float2(nl.z, nl.w));
            pr[4 * e] = ex2_ftz(a.x);
            pr[4 * e + 1] = ex2_ftz(a.y);
            pr[4 * e + 2] = ex2_ftz(b.x);
            pr[4 * e + 3] = ex2_ftz(b.y);
          }
          if (masked) {
            const int n0 = x - 32 * part;  // columns that do not see this key
            const uint32_t bits = n0 >= 32 ? 0u : (n0 <= 0 ? 0xFFFFFFFFu : 0xFFFFFFFFu << n0);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              pr[32 * part + e] = (bits >> e & 1u) ? pr[32 * part + e] : 0.0f;
          }
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = pack_bf16x2(pr[32 * part + 2 * e], pr[32 * part + 2 * e + 1]);
          tmem_st16((C::OWN_P ? tp : tl) + 16 * part, w);
          if (C::OWN_P && part == 0) continue;  // nobody waits for the first part alone
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (C::OWN_P) mbar_arrive(B.p_full);
            mbar_arrive(B.p_full + 8 * part);
          }
        }

        if (!(ok = mbar_wait(B.dp_full, tiles & 1u, kAttnWaitNs, abort_flag))) break;
        tc_fence_after();
        tmem_ld32(tl + 128, v);
        tmem_ld32(tl + 160, v + 32);
        tmem_ld_wait32(v);
        tmem_ld_wait32(v + 32);
        if (C::OWN_P) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(B.dp_read);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float4 de = *reinterpret_cast<const float4*>(st + 128 + 4 * e);
          w[2 * e] = pack_bf16x2(pr[4 * e] * (__uint_as_float(v[4 * e]) - de.x),
                                 pr[4 * e + 1] * (__uint_as_float(v[4 * e + 1]) - de.y));
          w[2 * e + 1] = pack_bf16x2(pr[4 * e + 2] * (__uint_as_float(v[4 * e + 2]) - de.z),
                                     pr[4 * e + 3] * (__uint_as_float(v[4 * e + 3]) - de.w));
        }
        if (C::OWN_P) {
          if (!(ok = mbar_wait(B.ds_empty, (tiles & 1u) ^ 1u, kAttnWaitNs, abort_flag))) break;
          tc_fence_after();
        }
        tmem_st32(C::OWN_P ? tp + 64 : tl + 128, w);
        if (C::OWN_P && i + 1 < n && !(ok = load_s(tiles + 1))) break;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(B.ds_full);
          mbar_arrive(B.stat_empty + 8 * buf);
        }
        if (C::OWN_P && i + 1 < n) s_loaded();
      }
      if (!ok) break;
      if (n > 0) {
        if (!(ok = mbar_wait(B.acc_full, uses & 1u, kAttnWaitNs, abort_flag))) break;
        ++uses;
        tc_fence_after();
      }
      // one warpgroup stores dv, the other dk
      const uint32_t ta = tmem + lanes + C::SUM_COL + half * C::SUM_STEP;
      uint16_t* out = half ? p.dk : p.dv;
      const int64_t ld = half ? p.lddk : p.lddv;
      const float f = half ? p.scale : 1.0f;
      if (PARTS) {
        const int64_t at = (int64_t)s.k0 + key;
        const bool store = key < s.lk && PACT_IN(at < p.tk);
        store_part(p.part_kv +
                       (((half ? p.parts_q : 0) + part) * (int64_t)p.tk + at) * p.hk * p.D + kvh * p.D,
                   ta, p.D, store, n > 0, f);
        continue;
      }
      for (int b = 0; b < p.D; b += 64) {
        const int cols = min(64, p.D - b);
        uint32_t w[32];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t o[16];
          const bool have = n > 0 && h * 16 < cols;
          if (have) {
            tmem_ld16(ta + b + 16 * h, o);
            tmem_ld_wait16(o);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            w[8 * h + e] = have ? pack_bf16x2(__uint_as_float(o[2 * e]) * f,
                                              __uint_as_float(o[2 * e + 1]) * f)
                                : 0u;
        }
        if (PACT_IN(s.k0 + key0 < p.tk))
          store_rows64(w, lane, quarter * 32, s.lk - key0, cols,
                       out + (int64_t)(s.k0 + key0) * ld + (int64_t)kvh * p.D + b, ld, p.D, 1, 65536u);
      }
    }
    if (!ok && lane == 0) raise_error(abort_flag, p.status, PACT_DEV_TIMEOUT | PACT_DEV_ROLE_EPI);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  wait_for_prerequisites();  // done means done with dq, too
}

// ------------------------------------------------------------------ the parts together
struct AttnSum {
  const float* parts;  // [count, rows, heads, D]
  uint16_t* out;
  int64_t ld, first;  // warps before these
  const int* cu;
  int count, rows, heads, groups;
};
struct AttnSums {
  AttnSum of[3];
  int n;
};
// The sums of the parts in their order.  2^seg lanes have a row; a warp's rows are heads of
// one token.
__global__ void __launch_bounds__(256) k_attn_sum(const AttnSums sums, int nseq, int D, int seg) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  AttnSum a = sums.of[0];
  for (int i = 1; i < sums.n; ++i)
    if (w >= sums.of[i].first) a = sums.of[i];
  const int64_t t = (w - a.first) / a.groups;
  const int h = (int)(w - a.first - t * a.groups) * (32 >> seg) + (lane >> seg);
  const int c = (lane & ((1 << seg) - 1)) * 8;
  const bool in = in_sequence(a.cu, nseq, a.rows, t);  // others stay as they were
  wait_for_prerequisites();
  if (!in || h >= a.heads || c >= D) return;
  const int64_t step = (int64_t)a.rows * a.heads * D;
  const float* at = a.parts + (t * a.heads + h) * D + c;
  float acc[8] = {};
  for (int s = 0; s < a.count; ++s) {
    const float4 x = *reinterpret_cast<const float4*>(at + s * step);
    const float4 y = *reinterpret_cast<const float4*>(at + s * step + 4);
    acc[0] += x.x, acc[1] += x.y, acc[2] += x.z, acc[3] += x.w;
    acc[4] += y.x, acc[5] += y.y, acc[6] += y.z, acc[7] += y.w;
  }
  uint32_t out[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) out[e] = pack_bf16x2(acc[2 * e], acc[2 * e + 1]);
  if (PACT_IN(t < a.rows && h < a.heads))
    *reinterpret_cast<uint4*>(a.out + t * a.ld + (int64_t)h * D + c) =
        make_uint4(out[0], out[1], out[2], out[3]);
}

// Few units leave SMs without work.  dq and dk|dv run beside each other then (the latter takes
// what SMs the former has left), so that it pays to cut up the one that is by far the longer:
// dk|dv where query heads share key heads, dq where a few queries see many keys.  There are no
// more parts than SMs for them, none of fewer than four tiles, and none at all below 16 tiles a
// unit (on average: the lengths are on the device).  One part and with this rule, us: 8192
// causal, 8/1 heads of 128, 752 and 464; 2048, 8/2 heads of 128, 96 and 57; 1024, 16/2 heads of
// 64, 93 and 43; 512, 8/1 heads of 64, 56 and 29; 256 over 2304 keys, 4 heads of 128, 32 and 25.
// Where both are as long it does not: 4096 both ways, 2 heads of 64, 55 as it is, 80 with dk|dv
// in two parts, 73 with both.
static int bwd_parts(int64_t units, int64_t tiles, int64_t others) {
  constexpr int64_t kSms = 152, kMost = 16;  // whatever the device has
  if (tiles < 16 || tiles < 2 * others || units * 2 > kSms) return 1;
  int64_t parts = kSms / units;
  if (parts > tiles / 4) parts = tiles / 4;
  return (int)(parts < kMost ? parts : kMost);
}
static int64_t query_tiles(int64_t tq, int64_t nseq, int hq, int hk) {
  return tq * (hq / hk) / (128 * nseq);
}
int attn_parts_dq(int64_t tq, int64_t tk, int64_t nseq, int hq, int hk) {
  const int gp = attn_tile_heads(hq / hk);
  return bwd_parts(attn_units(tq, 128 / gp, nseq, hq / gp), tk / nseq / 128,
                   query_tiles(tq, nseq, hq, hk));
}
int attn_parts_dkdv(int64_t tq, int64_t tk, int64_t nseq, int hq, int hk) {
  return bwd_parts(attn_units(tk, 128, nseq, hk), query_tiles(tq, nseq, hq, hk), tk / nseq / 128);
}

template <int DP>
static cudaError_t launch_bwd(const AttnBwdLaunch& L, unsigned gq, unsigned gk, cudaStream_t st) {
  constexpr uint32_t sm = BwdCfg<DP>::SMEM;
  const AttnParams& p = L.p;
  const auto dq = p.parts > 1 ? k_attn_dq<DP, true> : k_attn_dq<DP, false>;
  const auto dkdv = p.parts_q > 1 ? k_attn_dkdv<DP, true> : k_attn_dkdv<DP, false>;
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(dq, cudaFuncAttributeMaxDynamicSharedMemorySize, sm)) ||
      (e = cudaFuncSetAttribute(dkdv, cudaFuncAttributeMaxDynamicSharedMemorySize, sm)))
    return e;
  note_launch();
  dq<<<gq, 384, sm, st>>>(L.tmQ, L.tmdO, L.tmK, L.tmV, p);
  if ((e = cudaGetLastError())) return e;
  note_launch();
  if ((e = launch_dependent(dkdv, gk, 384, sm, st, L.tmQ, L.tmdO, L.tmK, L.tmV, p))) return e;
  if (p.parts == 1 && p.parts_q == 1) return cudaSuccess;
  int seg = 1;
  while (8 << seg < p.D) ++seg;
  AttnSums sums = {};
  int64_t warps = 0;
  auto add = [&](const float* parts, int count, uint16_t* out, int64_t ld, const int* cu, int rows,
                 int heads) {
    const int groups = (heads + (32 >> seg) - 1) / (32 >> seg);
    sums.of[sums.n++] = AttnSum{parts, out, ld, warps, cu, count, rows, heads, groups};
    warps += (int64_t)rows * groups;
  };
  if (p.parts > 1) add(p.part_o, p.parts, p.dq, p.lddq, p.cu_q, p.tq, p.hq);
  if (p.parts_q > 1) {
    add(p.part_kv, p.parts_q, p.dv, p.lddv, p.cu_k, p.tk, p.hk);
    add(p.part_kv + (int64_t)p.parts_q * p.tk * p.hk * p.D, p.parts_q, p.dk, p.lddk, p.cu_k, p.tk, p.hk);
  }
  note_launch();
  return launch_dependent(k_attn_sum, (unsigned)((warps + 7) / 8), 256, 0, st, sums, p.nseq, p.D, seg);
}

cudaError_t launch_attn_bwd(const AttnBwdLaunch& L, cudaStream_t st) {
  const AttnParams& p = L.p;
  const int64_t rows = (int64_t)p.tq * p.hq;
  note_launch();
  if (p.D <= 64)
    k_attn_delta<8><<<(unsigned)((rows + 31) / 32), 256, 0, st>>>(p);
  else
    k_attn_delta<16><<<(unsigned)((rows + 15) / 16), 256, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t uq = attn_units(p.tq, p.tpt, p.nseq, p.units_h) * p.parts;
  const int64_t uk = attn_units(p.tk, 128, p.nseq, p.hk) * p.parts_q;
  const unsigned gq = (unsigned)(uq < L.num_sms ? uq : L.num_sms);
  const unsigned gk = (unsigned)(uk < L.num_sms ? uk : L.num_sms);
  return p.D <= 64 ? launch_bwd<64>(L, gq, gk, st) : launch_bwd<128>(L, gq, gk, st);
}

}  // namespace pact
