// Attention over packed sequences, forward:
//   S = q k^T;  P = softmax(scale S) over the visible keys;  o = P v;
//   lse = log(sum of exp(scale S)).
// With causal, query i of a sequence's lq sees key j of its lk when j <= i + lk - lq.
//
// One pass over the keys with the running maximum and sum of the softmax.  A CTA has two
// tiles of 128 query rows (attention.cuh) against tiles of 128 keys, and a warpgroup for each,
// a row a thread; while one softmax runs, the tensor cores work for the other tile.  TMEM
// columns of tile i: S_i at 128 i;
//   D > 64:   P_i (BF16) over the first half of S_i, O_i at 256 + 128 i.  The next S_i has to
//             wait for P_i V.
//   D <= 64:  O_i at 256 + 64 i, P_i at 384 + 64 i: the next S_i is computed as soon as the
//             softmax has read this one.
// A thread for each tile issues its products; MMAs of one thread run in order, so (D > 64)
// S_i may be issued behind the P_i V that reads P_i out of the same columns.  Keys and values
// pass through one ring of shared memory.
//
// What bounds it.  Heads of 128: a pair of tiles against 128 keys has 2048 cycles of products
// (16 MMAs of 64 cycles for each tile) and takes about 3000 to 3700: the softmax of a tile,
// 1370 cycles, the signals to and from the issuers, 300, and P V and the next S, 768, follow
// one another, and the other tile fills the gaps in part.  16384 causal, 16/4 heads of 128: 767
// to 810 us, 1.36 to 1.43 PFLOP/s, by the power cap.  Heads of 64: the latencies of the softmax,
// 2250 cycles a pair of tiles (its 32768 exponentials are 1024), with two warps a scheduler to
// cover them: exponentials' pipe and tensor pipe 30 % busy, issue slots 48 %; 26 x 1024 causal,
// 32/8 heads of 64: 164 us.  CTA pairs, which halve what shared memory has to deliver, were
// slower (16384: 816 us): a tile then waits for the softmax of two CTAs.  A third warpgroup for
// the end of a unit was slower, too (8 x 1024, 32/8 heads of 128: 107 us, 78 without): four
// warps store two tiles one after the other.
//
// Where there are few units, they have one tile, and their keys are cut into parts, units of
// their own, and a second kernel joins what these say of a row (attn_fwd_plan).  A token over
// many keys is then bound by HBM: 131072 keys, 32/8 heads of 128, 100 us, 5.4 TB/s; 16 of them
// over 16384 each, 165 us, 6.5.  The kernels for parts spill 36 bytes a thread (heads of 128) and
// 16 (64), those without parts none.
//
// The running maximum m of a row moves only when a new one is above it by more than 2^8 in
// the exponentials' scale: the sums stay far from FP32's range, and the rescaling of O in
// TMEM that a moved m needs is rare.  P is rounded to BF16 for its product, since the tensor
// cores take it as they take V (TF32 would halve their rate, two BF16 parts double the work);
// its sum is of the FP32 values, and sums, maxima and O are FP32.  Error of o against 64 bits,
// relative: 0.0020, of which its own rounding to BF16 is 0.0016.
#include "attention.cuh"
#include "dependent.cuh"

namespace pact {

template <int DP>
struct FwdCfg {
  static constexpr bool OWN_P = DP == 64;  // P has TMEM columns of its own
  static constexpr int O_COL = 256, O_STEP = OWN_P ? 64 : 128;
  static constexpr int P_COL = OWN_P ? 384 : 0, P_STEP = OWN_P ? 64 : 128;
  static constexpr int BOXES = DP / 64;
  static constexpr uint32_t TILE = BOXES * kBox;
  static constexpr int STAGES = DP == 64 ? 8 : 5;
  static constexpr uint32_t Q_OFF = 0, KV_OFF = 2 * TILE;
  static constexpr uint32_t BAR_OFF = KV_OFF + STAGES * TILE;
  static constexpr uint32_t SMEM = BAR_OFF + 512;
  // q_full[2] q_empty[2] s_full[2] p_full[2][2] o_done[2] final[2] tail - kv_full[ST] kv_empty[ST]
  // s_read[2] lag unit_full[3] unit_empty[3] before the ring's
  static constexpr int NBARS = 25 + 2 * STAGES;
  static constexpr uint32_t UNIT_OFF = BAR_OFF + 384;  // three descriptions of a unit
  static_assert(SMEM <= 232448 && NBARS * 8 <= 384, "shared memory");
};

// PARTS: the key tiles of a unit are cut into p.parts runs, each a unit of its own.
template <int DP, bool PARTS>
__global__ void __launch_bounds__(384, 1)
    k_attn_fwd(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
               const __grid_constant__ CUtensorMap tmV, const AttnParams p) {
  using C = FwdCfg<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_addr(smem);
  if (base & 1023u) {  // the swizzle needs it, and the budget leaves no room to round up
    if (threadIdx.x == 0) atomicOr(p.status, (unsigned)PACT_DEV_BOUNDS);
    return;
  }
  const uint32_t bars = base + C::BAR_OFF;
  const uint32_t q_full = bars, q_empty = bars + 16, s_full = bars + 32, p_full = bars + 48,
                 o_done = bars + 80, final_bar = bars + 96, tail_bar = bars + 112,
                 s_read = bars + 128, lag_bar = bars + 144, unit_full = bars + 152, unit_empty = bars + 176,
                 kv_full = bars + 200,
                 kv_empty = kv_full + 8 * C::STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::BAR_OFF + 504);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::BAR_OFF + 508);
  const int warp = warp_index(), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + 8 * i, 1);
      mbar_init(q_empty + 8 * i, 1);
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 16 * i, 4);  // the warps of a tile, for each half of its keys
      mbar_init(p_full + 16 * i + 8, 4);
      mbar_init(o_done + 8 * i, 1);
      mbar_init(s_read + 8 * i, 4);
      mbar_init(final_bar + 8 * i, 1);
    }
    mbar_init(tail_bar, 1);
    mbar_init(lag_bar, 1);
    for (int u = 0; u < 3; ++u) {
      mbar_init(unit_full + 8 * u, 1);
      mbar_init(unit_empty + 8 * u, 10);  // the warps of the softmax and the issuers
    }
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(kv_full + 8 * s, 1);
      mbar_init(kv_empty + 8 * s, 2);  // the issuers
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
  if (PARTS) let_dependents_start();

  // A unit: tok0[i], the first tokens of its tiles; kend[i], the keys that they see, and nk[i]
  // tiles of them; h0, its first query head.  The copying warp looks the units up and hands
  // them to the other warps.  With PARTS keys are counted from tile `first` on, and there are
  // `run` tiles of them.
  int q0, lq, lk, tok0[2], kend[2], nk[2], h0, part = 0;
  auto set_unit = [&](int4 d, int head, int first, int run) {
    q0 = d.x;
    lq = d.y;
    lk = d.z;
    h0 = head;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      tok0[i] = i < p.unit_tiles ? d.w + i * p.tpt : lq;
      kend[i] = 0;
      if (tok0[i] < lq) {
        kend[i] = lk;
        if (p.causal) kend[i] = clampi(min(tok0[i] + p.tpt, lq) + lk - lq, 0, lk);
        if (PARTS) kend[i] = clampi(kend[i] - first * 128, 0, run * 128);
      }
      nk[i] = (kend[i] + 127) / 128;
    }
    if (PARTS) lk -= first * 128;
  };
  RingPos slot;
  bool ok = true;
  auto next_unit = [&]() {  // false behind the last one, and (ok false) when it took too long
    // a tile without keys waits here while the other tile goes through its own
    if (!(ok = mbar_wait(unit_full + 8 * slot.stage, slot.phase, unit_wait_ns(p), abort_flag))) return false;
    const int4* d = reinterpret_cast<const int4*>(smem + C::UNIT_OFF + 32 * slot.stage);
    const int4 a = d[0], b = d[1];
    __syncwarp();
    if (lane == 0) mbar_arrive(unit_empty + 8 * slot.stage);
    slot.advance(3);
    set_unit(a, b.x, b.z, b.w);
    part = b.y >> 1;
    return b.y != 0;
  };

  if (warp >= 8) {
    setmaxnreg_dec<56>();
    if (warp == 8) {
      // ------------------------------------------------------------ copies
      int stage = 0;
      uint32_t phase = 0, q_uses[2] = {0, 0}, tails = 0;
      uint32_t pend = 0, pend_par = 0;
      int kvh = 0;
      auto load_kv = [&](const CUtensorMap* tm, int row, int valid) {
        if (!mbar_wait(kv_empty + 8 * stage, phase ^ 1u, kAttnWaitNs, abort_flag)) return false;
        const uint32_t dst = base + C::KV_OFF + stage * C::TILE, full = kv_full + 8 * stage;
        if (valid >= 128) {
          if (lane == 0) {
            mbar_expect_tx(full, C::TILE);
#pragma unroll
            for (int b = 0; b < C::BOXES; ++b)
              tma_load_3d(dst + b * kBox, tm, b * 64, kvh, row, full);
          }
          pend |= 1u << stage;
          pend_par = (pend_par & ~(1u << stage)) | (phase << stage);
        } else {  // rows behind the sequence become zeros before the MMAs see the tile
          if (lane == 0) {
            mbar_expect_tx(tail_bar, C::TILE);
#pragma unroll
            for (int b = 0; b < C::BOXES; ++b)
              tma_load_3d(dst + b * kBox, tm, b * 64, kvh, row, tail_bar);
          }
          __syncwarp();
          if (!mbar_wait(tail_bar, tails & 1u, kAttnWaitNs, nullptr)) return false;
          ++tails;
          zero_rows(smem + C::KV_OFF + stage * C::TILE, C::BOXES, valid, lane);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(full);
        }
        __syncwarp();
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
        return true;
      };
      auto load_q = [&](int i) {
        if (!mbar_wait(q_empty + 8 * i, (q_uses[i] & 1u) ^ 1u, kAttnWaitNs, abort_flag)) return false;
        ++q_uses[i];
        if (lane == 0) {
          const uint32_t rows = (uint32_t)(p.tpt * p.gp), full = q_full + 8 * i;
          mbar_expect_tx(full, rows * 128 * C::BOXES);
#pragma unroll
          for (int b = 0; b < C::BOXES; ++b)
            tma_load_3d(base + C::Q_OFF + i * C::TILE + b * kBox, &tmQ, b * 64, h0, q0 + tok0[i],
                        full);
        }
        __syncwarp();
        return true;
      };
      SeqFinder<false> finder = seq_finder<false>(p, p.unit_tiles * p.tpt);
      Seq s;
      for (uint32_t turn = 0;; ++turn) {
        const uint32_t turned = unit_of(turn);
        const uint32_t u = PARTS ? turned / (uint32_t)p.parts : turned, t = p.units_div.div(u);
        const int hu = (int)(u - t * p.units_h);
        const bool there = u < kMaxUnit && finder.find(t, s);
        kvh = p.subs == 1 ? hu : hu / p.subs;
        const int4 where = make_int4(s.q0, s.lq, s.lk, s.tile * p.unit_tiles * p.tpt);
        const int head = kvh * p.group + (hu - kvh * p.subs) * p.gp;
        int first = 0, run = 0;
        if (PARTS) {
          set_unit(where, head, 0, (1 << 24) - 1);
          const int all = max(nk[0], nk[1]);
          part = (int)(turned - u * (uint32_t)p.parts);
          first = (int)((int64_t)all * part / p.parts);
          run = (int)((int64_t)all * (part + 1) / p.parts) - first;
        }
        set_unit(where, head, first, run);
        if (!(ok = mbar_wait(unit_empty + 8 * slot.stage, slot.phase ^ 1u, kAttnWaitNs, abort_flag)))
          break;
        if (lane == 0) {
          int4* d = reinterpret_cast<int4*>(smem + C::UNIT_OFF + 32 * slot.stage);
          d[0] = where;
          d[1] = make_int4(head, there ? 2 * part + 1 : 0, first, run);
          mbar_arrive(unit_full + 8 * slot.stage);
        }
        __syncwarp();
        slot.advance(3);
        if (!there) break;
        if (PARTS) s.k0 += first * 128;
        const int n = max(nk[0], nk[1]);
        // in the order of their use: K 0, then (OWN_P) K j + 1 and V j, or V j and K j + 1
        for (int j = -1; j < n && n > 0 && ok; ++j) {
          if (j < 0 && nk[0] > 0) ok = load_q(0);
          if (!C::OWN_P && j >= 0) ok = ok && load_kv(&tmV, s.k0 + j * 128, lk - j * 128);
          if (j + 1 < n) ok = ok && load_kv(&tmK, s.k0 + (j + 1) * 128, 128);
          if (C::OWN_P && j >= 0) ok = ok && load_kv(&tmV, s.k0 + j * 128, lk - j * 128);
          if (j < 0 && nk[1] > 0) ok = ok && load_q(1);
        }
        if (!ok) break;
      }
      if (!ok) {
        if (lane == 0) raise_error(abort_flag, p.status, PACT_DEV_TIMEOUT | PACT_DEV_ROLE_TMA);
        // copies in flight land before the CTA can exit
        for (int st = 0; st < C::STAGES; ++st)
          if (pend & (1u << st))
            mbar_wait(kv_full + 8 * st, (pend_par >> st) & 1u, 10000000ull, nullptr);
        for (int i = 0; i < 2; ++i)
          if (q_uses[i]) mbar_wait(q_full + 8 * i, (q_uses[i] & 1u) ^ 1u, 10000000ull, nullptr);
      }
    } else if (warp < 11) {
      // ------------------------------------------------------------ MMAs of tile i
      const int i = warp - 9;
      RingPos at;
      uint32_t q_uses = 0, p_uses = 0, s_uses = 0;
      bool lagged = false;
      const uint32_t idesc_s = attn_idesc(128, false), idesc_o = attn_idesc(p.D, true);
      const uint32_t ts = tmem + i * 128, to = tmem + C::O_COL + i * C::O_STEP;
      const uint32_t tp = tmem + C::P_COL + i * C::P_STEP;
      const int ksteps = p.D / 16;
      const uint64_t dq = desc_k(base + C::Q_OFF + i * C::TILE);
      const uint64_t dk0 = desc_k(base + C::KV_OFF), dv0 = desc_n(base + C::KV_OFF);
      const bool lead = elected();
      auto wait = [&](uint32_t bar, uint32_t par) {
        return mbar_wait(bar, par, kAttnWaitNs, abort_flag);
      };
      while (ok && next_unit()) {
        const int n = max(nk[0], nk[1]), my_nk = i ? nk[1] : nk[0], my_kend = i ? kend[1] : kend[0];
        if (i == 0 && !lagged && nk[0] == 0) {  // tile 1 has nobody to wait for
          if (lead) mbar_arrive(lag_bar);
          lagged = true;
        }
        // step j: the values of tile j - 1 and the keys of tile j, which come first in the
        // ring with OWN_P.  A wait or a commit costs the thread about 100 cycles: what lies
        // between P and the next S is as short as can be.
        for (int j = 0; j <= n && n > 0; ++j) {
          const bool pv = j > 0 && j - 1 < my_nk, qk = j < my_nk;
          RingPos v = at, k = at;
          if (C::OWN_P ? j > 0 && j < n : false) v.advance(C::STAGES);
          if (!C::OWN_P && j > 0) k.advance(C::STAGES);
          if (j < n && !(ok = wait(kv_full + 8 * k.stage, k.phase))) break;
          if (j > 0 && !(ok = wait(kv_full + 8 * v.stage, v.phase))) break;
          if (qk && j == 0) {
            if (!(ok = wait(q_full + 8 * i, q_uses & 1u))) break;
            ++q_uses;
            // Once, tile 1 starts half a step behind tile 0, and stays there: with both at
            // the same point, both softmax warpgroups wait for the tensor cores, and then
            // both work while those idle.
            if (i == 1 && !lagged) {
              if (!(ok = wait(lag_bar, 0))) break;
              lagged = true;
            }
          }
          auto issue_qk = [&]() {
            const uint64_t d = dk0 + (uint64_t)(k.stage * (C::TILE >> 4));
#pragma unroll
            for (int e = 0; e < DP / 16; ++e)
              if (e < ksteps) mma_bf16(ts, step_k(dq, e), step_k(d, e), idesc_s, e > 0);
            mma_commit(s_full + 8 * i);
            mma_commit(kv_empty + 8 * k.stage);
            if (j == my_nk - 1) mma_commit(q_empty + 8 * i);
          };
          if (C::OWN_P && qk) {  // once the softmax has read the S before it
            if (!(ok = wait(s_read + 8 * i, (s_uses & 1u) ^ 1u))) break;
            ++s_uses;
            tc_fence_after();
            if (lead) issue_qk();
            __syncwarp();
          }
          const uint64_t d = dv0 + (uint64_t)(v.stage * (C::TILE >> 4));
          if (pv) {
            if (!(ok = wait(p_full + 16 * i, p_uses & 1u))) break;
            tc_fence_after();
            if (lead) {
              if (i == 0 && !lagged) mbar_arrive(lag_bar);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                mma_bf16_ta(to, tp + e * 8, step_n(d, e), idesc_o, (j > 1 || e > 0) ? 1u : 0u);
            }
            lagged = lagged || i == 0;
            __syncwarp();
            if (!(ok = wait(p_full + 16 * i + 8, p_uses & 1u))) break;
            ++p_uses;
            tc_fence_after();
          }
          if (lead) {
            if (pv && my_kend - (j - 1) * 128 > 64) {
#pragma unroll
              for (int e = 4; e < 8; ++e) mma_bf16_ta(to, tp + e * 8, step_n(d, e), idesc_o, 1u);
            }
            // a stage that this tile has no use of is released all the same
            if (pv)
              mma_commit(kv_empty + 8 * v.stage);
            else if (j > 0)
              mbar_arrive(kv_empty + 8 * v.stage);
            if (!C::OWN_P && qk) issue_qk();
            if (pv) mma_commit(o_done + 8 * i);
            if (!qk && j < n) mbar_arrive(kv_empty + 8 * k.stage);
          }
          __syncwarp();
          at.advance(C::STAGES, j == 0 || j == n ? 1 : 2);
        }
      }
      if (lead) {
        if (!ok) raise_error(abort_flag, p.status, PACT_DEV_TIMEOUT | PACT_DEV_ROLE_MMA);
        mma_commit(final_bar + 8 * i);  // every MMA and commit of this thread has completed then
        mbar_wait(final_bar + 8 * i, 0, kAttnWaitNs, nullptr);
      }
      __syncwarp();
    }
  } else {
    // -------------------------------------------------------------- softmax, a row a thread
    setmaxnreg_inc<224>();
    const int i = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t ts = tmem + lanes + i * 128, to = tmem + lanes + C::O_COL + i * C::O_STEP;
    const uint32_t tp = tmem + lanes + C::P_COL + i * C::P_STEP;
    const float c = p.c;
    uint32_t uses = 0;  // S tiles so far
    while (ok && next_unit()) {
      const int n = i ? nk[1] : nk[0], my_kend = i ? kend[1] : kend[0], my_tok = i ? tok0[1] : tok0[0];
      const int tok = my_tok + row_token(p, row);
      // keys that this row sees, and that every row of the tile sees
      const int lim = p.causal ? min(lk, tok + 1 + lk - lq) : lk;
      const int lim_all = p.causal ? min(lk, my_tok + 1 + lk - lq) : lk;
      float m = -INFINITY, l = 0.0f;
      for (int j = 0; j < n; ++j, ++uses) {
        if (!(ok = mbar_wait(s_full + 8 * i, uses & 1u, kAttnWaitNs, abort_flag))) break;
        tc_fence_after();
        uint32_t v[128];
#pragma unroll
        for (int b = 0; b < 4; ++b) tmem_ld32(ts + 32 * b, v + 32 * b);
#pragma unroll
        for (int b = 0; b < 4; ++b) tmem_ld_wait32(v + 32 * b);
        if (C::OWN_P) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_read + 8 * i);
        }
        if ((j + 1) * 128 > lim_all) mask_from(v, lim - j * 128);
        // the exponentials of half b: their sums, and P's packed columns
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        uint32_t w[32];
        auto exps = [&](int b, float mc) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float2 x = __ffma2_rn(make_float2(__uint_as_float(v[64 * b + 2 * e]),
                                              __uint_as_float(v[64 * b + 2 * e + 1])),
                                  make_float2(c, c), make_float2(mc, mc));
            x.x = ex2_ftz(x.x);
            x.y = ex2_ftz(x.y);
            sum[e & 1] = __fadd2_rn(sum[e & 1], x);
            w[e] = pack_bf16x2(x.x, x.y);
          }
        };
        auto row_max = [&]() {
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 128; e += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mx[k] = fmaxf(mx[k], fmaxf(__uint_as_float(v[e + 2 * k]), __uint_as_float(v[e + 2 * k + 1])));
          return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        };
        // P of this tile takes the place of the last one's, whose product must be done
        auto wait_pv = [&]() {
          return j == 0 || mbar_wait(o_done + 8 * i, (uses - 1u) & 1u, kAttnWaitNs, abort_flag);
        };
        // From the second tile on the exponentials begin with the old maximum, beside the
        // search for the new one (the one needs the MUFU, the other the ALU), and are taken
        // again in the rare case that it moves.
        bool again = j == 0;
        float mc = m == -INFINITY ? 0.0f : -m * c;
        if (!again) {
          exps(0, mc);
          again = __any_sync(0xFFFFFFFFu, (row_max() - m) * c > 8.0f);
        }
        bool waited = false;
        if (again) {
          const float top = row_max();
          const bool move = (top - m) * c > 8.0f;
          if (j == 0) {
            m = top;
          } else if (__any_sync(0xFFFFFFFFu, move)) {
            const float m2 = move ? top : m;
            const float f = move ? ex2_ftz((m - m2) * c) : 1.0f;
            l *= f;
            m = m2;
            // O holds the products so far once the last P V has completed
            if (!(ok = wait_pv())) break;
            waited = true;
            tc_fence_after();
            for (int b = 0; b < p.D; b += 16) {
              uint32_t o[16];
              tmem_ld16(to + b, o);
              tmem_ld_wait16(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(to + b, o);
            }
            tmem_st_wait();
          }
          mc = m == -INFINITY ? 0.0f : -m * c;
          sum[0] = sum[1] = make_float2(0.0f, 0.0f);
          exps(0, mc);
        }
        if (C::OWN_P && !waited) {
          if (!(ok = wait_pv())) break;
          tc_fence_after();
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if (b == 0 || my_kend - j * 128 > 64) {  // else no key of the second half is seen
            if (b == 1) exps(1, mc);
            tmem_st32(tp + 32 * b, w);
            tmem_st_wait();
            tc_fence_before();
          }
          __syncwarp();
          // the first half's product runs while the second half is computed
          if (lane == 0) mbar_arrive(p_full + 16 * i + 8 * b);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      if (!ok) break;
      // ---------------------------------------------------------- o and lse
      const int rows = min(p.tpt, lq - my_tok) * p.gp;
      if (rows <= 0) continue;
      const bool empty = n == 0 || lim <= 0;
      if (row < rows && PACT_IN(q0 + tok < p.tq)) {
        const int h = h0 + row - row_token(p, row) * p.gp;
        (PARTS ? p.part_lse + (int64_t)part * p.hq * p.tq : p.lse)[(int64_t)h * p.tq + q0 + tok] =
            empty ? -INFINITY : (m * c + log2f(l)) * kLn2;
      }
      const float inv = l > 0.0f ? __fdiv_rn(1.0f, l) : l;  // a NaN stays one
      if (n > 0) {
        if (!(ok = mbar_wait(o_done + 8 * i, (uses - 1u) & 1u, kAttnWaitNs, abort_flag))) break;
        tc_fence_after();
      }
      if (PARTS) {
        if (n > 0) {
          const int h = h0 + row - row_token(p, row) * p.gp;
          float* at = p.part_o + (((int64_t)part * p.tq + q0 + tok) * p.hq + h) * p.D;
          for (int b = 0; b < p.D; b += 16) {
            uint32_t o[16];
            tmem_ld16(to + b, o);
            tmem_ld_wait16(o);
            if (row < rows && PACT_IN(q0 + tok < p.tq)) {
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<float4*>(at + b + e) =
                    make_float4(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv,
                                __uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
            }
          }
        }
        continue;
      }
      for (int b = 0; b < p.D; b += 64) {
        uint32_t w[32];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t o[16];
          if (n > 0) {  // columns past D hold nothing of use
            tmem_ld16(to + b + 16 * h, o);
            tmem_ld_wait16(o);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            w[8 * h + e] = empty ? 0u : pack_bf16x2(__uint_as_float(o[2 * e]) * inv,
                                                    __uint_as_float(o[2 * e + 1]) * inv);
        }
        if (PACT_IN(q0 + my_tok < p.tq))
          store_rows64(w, lane, quarter * 32, rows, min(64, p.D - b),
                       p.o + (int64_t)(q0 + my_tok) * p.ldo + (int64_t)h0 * p.D + b, p.ldo, p.D, p.gp,
                       p.gp_mul);
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
}

// ------------------------------------------------------------------ the parts together
//   lse = log sum exp lse_s;  o = sum exp(lse_s - lse) o_s.
// 2^seg lanes have a row; a warp's rows are heads of one token.  Starts while the forward
// still runs, and finds out meanwhile whether its token is of a sequence.
__global__ void __launch_bounds__(256) k_attn_join(const AttnParams p, int seg, int groups) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t t64 = w / groups;
  const int t = (int)t64, sl = lane & ((1 << seg) - 1);
  const int h = (int)(w - t64 * groups) * (32 >> seg) + (lane >> seg);
  const bool in = in_sequence(p.cu_q, p.nseq, p.tq, t64);  // others stay as they were
  wait_for_prerequisites();
  if (!in || h >= p.hq || sl * 8 >= p.D) return;
  const float* ls = p.part_lse + (int64_t)h * p.tq + t;
  const int64_t step = (int64_t)p.hq * p.tq;
  float top = -INFINITY;
  for (int s = 0; s < p.parts; ++s) top = fmaxf(top, ls[s * step]);
  const float base = top == -INFINITY ? 0.0f : top;
  const float* at = p.part_o + ((int64_t)t * p.hq + h) * p.D + sl * 8;
  float sum = 0.0f, acc[8] = {};
  for (int s = 0; s < p.parts; ++s) {
    const float l = ls[s * step];
    if (l == -INFINITY) continue;  // this part saw no key; its row may not be there
    const float f = ex2_ftz((l - base) * kLog2e);
    const float4 a = *reinterpret_cast<const float4*>(at + s * step * p.D);
    const float4 b = *reinterpret_cast<const float4*>(at + s * step * p.D + 4);
    sum += f;
    const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = __fmaf_rn(f, x[e], acc[e]);
  }
  const bool empty = sum == 0.0f;
  const float inv = empty ? 0.0f : __fdiv_rn(1.0f, sum);
  if (!PACT_IN(t < p.tq && h < p.hq)) return;
  if (sl == 0) p.lse[(int64_t)h * p.tq + t] = empty ? -INFINITY : base + log2f(sum) * kLn2;
  uint32_t out[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) out[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  *reinterpret_cast<uint4*>(p.o + (int64_t)t * p.ldo + (int64_t)h * p.D + sl * 8) =
      make_uint4(out[0], out[1], out[2], out[3]);
}

// ------------------------------------------------------------------ few units
// They leave SMs without work while each goes through all of its keys.
constexpr int64_t kSms = 152;  // whatever the device has

// Keys in parts pay for more ends of units and the join, 3 us and more, so there are no more
// parts than SMs for them, none of fewer than two tiles, and none at all below 16 tiles of keys
// a sequence (on average: the lengths are on the device, so a long sequence among many short
// ones stays whole: 8192 causal, 2/1 heads of 128, 91 alone and 122 with 31 of 128 tokens).  One
// part and with this rule, us: 8192
// causal, one head of 128, 118 and 52; 4096, 2 heads of 64, 49 and 29; a token over 2048 keys,
// 8/1 heads, 26 and 13, over 16384, 162 and 27, over 131072, 32/8 heads, 1203 and 100.  More
// parts than that: 8 x 1 over 2048, 32/8 heads, 26, with two 20, with three 27; 1024 keys (8
// tiles): 21, with four 20.
static int parts_of(int64_t units, int64_t tiles) {
  if (tiles < 16 || units * 2 > kSms) return 1;
  int64_t parts = kSms / units;
  if (parts > tiles / 2) parts = tiles / 2;
  return (int)(parts < 32 ? parts : 32);
}

// Units of one tile go through their keys faster than units of two, which share the tensor
// cores, and where there are few units it is the longest that counts: 1024, 8 heads of 128, 16.0
// us for 20.8; 2048, 16 heads, 29.3 for 36.2; 4000, 8/4 heads, 51 for 65; 512, 2 heads, 11.3 for
// 14.0.  Two tiles do more work in the same time, which tells where all SMs are at work: 8192,
// 8/1 heads, 119 us for 153; 6 x 900, 8/2 heads, 20.5 for 24.2; 4 x 500, 16/4 heads of 64, 11.9
// for 15.0; and where parts make up for fewer units: 8192, one head, 52 for 57.
AttnFwdPlan attn_fwd_plan(int64_t tq, int64_t tk, int64_t nseq, int hq, int hk) {
  const int gp = attn_tile_heads(hq / hk), tpt = 128 / gp;
  const int64_t tiles = tk / nseq / 128;
  const int64_t one = attn_units(tq, tpt, nseq, hq / gp);
  const int64_t two = attn_units(tq, 2 * tpt, nseq, hq / gp);
  const int p1 = parts_of(one, tiles), p2 = parts_of(two, tiles);
  if (two > (tiles < 5 ? kSms / 2 : kSms) || (p2 >= 4 && p1 < p2)) return AttnFwdPlan{2, p2};
  return AttnFwdPlan{1, p1};
}

template <int DP, bool PARTS>
static cudaError_t launch_fwd(const AttnFwdLaunch& L, unsigned grid, cudaStream_t st) {
  constexpr uint32_t sm = FwdCfg<DP>::SMEM;
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(k_attn_fwd<DP, PARTS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                sm)))
    return e;
  note_launch();
  k_attn_fwd<DP, PARTS><<<grid, 384, sm, st>>>(L.tmQ, L.tmK, L.tmV, L.p);
  return cudaGetLastError();
}

cudaError_t launch_attn_fwd(const AttnFwdLaunch& L, cudaStream_t st) {
  const AttnParams& p = L.p;
  const int64_t units = attn_units(p.tq, p.unit_tiles * p.tpt, p.nseq, p.units_h) * p.parts;
  const unsigned grid = (unsigned)(units < L.num_sms ? units : L.num_sms);
  if (p.parts == 1)
    return p.D <= 64 ? launch_fwd<64, false>(L, grid, st) : launch_fwd<128, false>(L, grid, st);
  const cudaError_t e =
      p.D <= 64 ? launch_fwd<64, true>(L, grid, st) : launch_fwd<128, true>(L, grid, st);
  if (e) return e;
  int seg = 1;
  while (8 << seg < p.D) ++seg;
  const int groups = (p.hq + (32 >> seg) - 1) / (32 >> seg);
  note_launch();
  return launch_dependent(k_attn_join, (unsigned)(((int64_t)p.tq * groups + 7) / 8), 256, 0, st, p,
                          seg, groups);
}

}  // namespace pact
