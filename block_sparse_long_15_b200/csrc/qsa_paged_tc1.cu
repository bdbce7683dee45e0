// Attention of chunks of new tokens over a paged K/V cache on 5th-generation tensor cores
// (tcgen05), one 128-row tile per CTA: head_dim 256 and 64, and head_dim 128 for sequences of no
// more than 128 (token, head) rows. See qsa_paged_tc.cu for head_dim 128 otherwise and
// qsa_paged_plan.cuh for how the work is divided.
//
// At head_dim 256 O of one tile takes 256 TMEM columns, so a CTA holds T = 128 / G tokens of one
// KV head against 64-key chunks, 1024 clocks of products and 512 of exponentials each. With few
// rows (drafted tokens) K and V are read for one tile anyway, and the call is bound by HBM.
// Q sits in TMEM too: the QK product then reads only K from shared memory, at half the rate that
// its 64 columns would need with both operands there, and shared memory is left to 192 KB of K and
// V stages. S is double-buffered, so the softmax of a chunk runs beside the products of its
// neighbours:
//   warp 0      TMA producer: K and V of a chunk into two rings, 3 deep (6 at head_dim 128, 8 at 64);
//               one lane per page box and 64 columns;
//   warp 1      MMA issuer (TMEM owner): O += P(n) V, S = Q K(n + 2)^T into the buffer that
//               P(n) has just left;
//   warp 2      builder;
//   warps 4-11  softmax, 16 rows per warp, two threads a row with 32 logits each, Q of the next
//               unit into TMEM, and the epilogue.
// TMEM: O, then Q, then two buffers of S (then P, in its first half).
// Every wait is bounded; on expiry the kernel records QSA_ERR_TIMEOUT and unwinds.
//
// Measured at head_dim 256, 16 / 2 heads: chunks of 1 .. 1500 tokens of 6 sequences (0.53 TFLOP)
// 500 us, 1.05 PFLOP/s, tensor pipe 52 % busy: the way from S to P (TMEM loads, exponentials, stores,
// two barriers) is longer than the products of one chunk that run beside it. Two groups of softmax
// warps taking chunks in turn, with the reference passed through shared memory, spilled (96 registers)
// and took 8 % more. 3 or 4 drafted tokens of 16 sequences of 2K .. 16K (336 MB) 72 us, 69 in a graph.
#include "qsa_paged_plan.cuh"

namespace qsa {
namespace {

constexpr int kChunk = 64;  // keys per chunk
template <int D_>
struct One {
  static constexpr int kD = D_, kTiles = 1, kChunk = qsa::kChunk;
};
constexpr int kThreads = 384;
constexpr int kBuilderWarp = 2;
constexpr int kSoftWarp0 = 4;
constexpr int kSoftWarps = 8;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kGroupBytes = kChunk * 128;  // 64 columns of a chunk's rows

template <int D_>
struct Layout {
  static constexpr int kNR = D_ == 256 ? 3 : D_ == 128 ? 6 : 8;  // depth of each ring
  static constexpr int kGroups = D_ / 64;
  static constexpr uint32_t kStageBytes = kChunk * D_ * 2;
  static constexpr uint32_t kColQ = D_, kColS = D_ + D_ / 2;
  static constexpr uint32_t kOffK = 0;
  static constexpr uint32_t kOffV = kOffK + kNR * kStageBytes;
  static constexpr uint32_t kOffBar = kOffV + kNR * kStageBytes;
  static constexpr uint32_t kOffMisc = kOffBar + 512;
  static constexpr uint32_t kOffInfo = kOffMisc + 64;
  static constexpr uint32_t kOffBits = kOffInfo + 2 * kInfoBytes;
  // barrier slots
  static constexpr int kBarKFull = 0;
  static constexpr int kBarKEmpty = kBarKFull + kNR;
  static constexpr int kBarVFull = kBarKEmpty + kNR;
  static constexpr int kBarVEmpty = kBarVFull + kNR;
  static constexpr int kBarSFull = kBarVEmpty + kNR;     // [S buffer]
  static constexpr int kBarPFull = kBarSFull + 2;        // [S buffer][step], 8 arrivals
  static constexpr int kBarPVDone = kBarPFull + 4;       // a phase per PV
  static constexpr int kBarODone = kBarPVDone + 1;       // a phase per unit: its last PV completed
  static constexpr int kBarQFull = kBarODone + 1;        // a phase per unit: Q is in TMEM, 8 arrivals
  static constexpr int kBarQEmpty = kBarQFull + 1;       // a phase per unit: its last QK completed
  static constexpr int kBarSlotFull = kBarQEmpty + 1;    // [slot], the builder's 32 lanes
  static constexpr int kBarSlotFree = kBarSlotFull + 2;  // [slot], producer + MMA warp + softmax warps
  static constexpr int kBarDrain = kBarSlotFree + 2;     // every MMA of the block completed
  static constexpr int kNumBars = kBarDrain + 1;
  static_assert(kNumBars * 8 <= 512, "barrier area");
};

template <int D_, bool kSel>
__global__ void __launch_bounds__(kThreads, 1)
k_paged_tc1(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
            const __grid_constant__ TcParams P) {
  typedef One<D_> X;
  typedef Layout<D_> Y;
  constexpr int kD = D_, kNR = Y::kNR;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t *bars = (uint64_t *)(base + Y::kOffBar);
  uint32_t *tmem_slot = (uint32_t *)(base + Y::kOffMisc);
  volatile int *abort_flag = (volatile int *)(base + Y::kOffMisc + 8);
  uint8_t *plan = base + Y::kOffBits + (kSel ? 2 * kBitSlotBytes : 0);
  const PlanArea L = {(long long *)plan, (SeqGeo *)(plan + (size_t)(P.nb + 1) * 8)};

  const Dims &D = P.D;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = P.T, G = D.G;
  auto info = [&](int s) { return (const UnitInfo *)(base + Y::kOffInfo + s * kInfoBytes); };
  auto token_bits = [&](int s) { return (const uint32_t *)(base + Y::kOffBits + s * kBitSlotBytes); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < Y::kNumBars; ++i) {
      uint32_t count = 1;
      if ((i >= Y::kBarPFull && i < Y::kBarPFull + 4) || i == Y::kBarQFull) count = kSoftWarps;
      if (i == Y::kBarSlotFull || i == Y::kBarSlotFull + 1) count = 32;
      if (i == Y::kBarSlotFree || i == Y::kBarSlotFree + 1) count = 2 + kSoftWarps;
      mbar_init(&bars[i], count);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  make_plan<X>(P, L, blockIdx.x == 0 ? P.status : nullptr);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  pdl_trigger();  // the merge may take its place; it waits for this kernel's end

  if (warp == kBuilderWarp) {
    const SlotArea area = {&bars[Y::kBarSlotFull], &bars[Y::kBarSlotFree], base + Y::kOffInfo, base + Y::kOffBits, abort_flag};
    build_segments<X, kSel>(P, area, L, lane);
  } else if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    // Lane i * groups + e holds the pool plane (page, KV head) of the i-th box of the next chunk (-1:
    // no token there, or a page outside the pool) and loads its columns 64 e ..
    const int n_lanes = Y::kGroups * (kChunk / P.box), box_i = lane / Y::kGroups, e = lane % Y::kGroups;
    const uint32_t box_bytes = (uint32_t)P.box * 128;
    int j = 0, jk = 0;  // chunks so far, and their K
    bool fail = false;
    for (int su = 0; !fail; ++su) {
      const int s = su & 1;
      if (!idle_wait_warp(&bars[Y::kBarSlotFull + s], (su >> 1) & 1)) {
        fail = true;
        break;
      }
      const UnitInfo I = *info(s);
      if (!I.live) break;
      const Chunks<X, kSel> ch(I, token_bits(s) + kBitWords, P.W);
      const int t_hi = I.len - I.n + min(I.n, I.r0 + T) - 1;  // the unit's last visible key
      auto plane = [&](int c) {
        int z = -1;
        const int key = c * kChunk + box_i * P.box;
        if (c >= 0 && lane < n_lanes && key <= t_hi) {
          const int page = P.P.table[(size_t)I.b * P.P.max_pages + (key >> P.P.ps_shift)];
          if (page >= 0 && page < P.P.n_pages) z = page * D.Hkv + I.g;
          else record_status(P.status, QSA_ERR_DEVICE_CHECK);
        }
        return z;
      };
      int c = ch.next(ch.ca);
      int z = plane(c);
      while (c >= 0) {
        const int cn = ch.next(c + 1), zn = plane(cn);  // read ahead
        const int st = j % kNR, y = (c * kChunk + box_i * P.box) & (P.P.ps - 1);
        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, z >= 0)) * box_bytes;
        const uint32_t at = st * Y::kStageBytes + e * kGroupBytes + box_i * box_bytes;
        if (j >= kNR && !warp_wait(&bars[Y::kBarKEmpty + st], ((j / kNR) & 1) ^ 1)) {
          fail = true;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&bars[Y::kBarKFull + st], bytes);
        __syncwarp();
        if (z >= 0) tma_load_3d(&tm_k, &bars[Y::kBarKFull + st], base + Y::kOffK + at, e * 64, y, z);
        ++jk;
        if (j >= kNR && !warp_wait(&bars[Y::kBarVEmpty + st], ((j / kNR) & 1) ^ 1)) {
          fail = true;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&bars[Y::kBarVFull + st], bytes);
        __syncwarp();
        if (z >= 0) tma_load_3d(&tm_v, &bars[Y::kBarVFull + st], base + Y::kOffV + at, e * 64, y, z);
        __syncwarp();
        c = cn;
        z = zn;
        ++j;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[Y::kBarSlotFree + s]);
    }
    if (fail) {
      if (lane == 0) record_status(P.status, QSA_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    // after a timeout, here or in another warp, copies may be in flight: they land before the block ends
    for (int i = max(0, jk - kNR); i < jk; ++i) warp_wait(&bars[Y::kBarKFull + i % kNR], (i / kNR) & 1);
    for (int i = max(0, j - kNR); i < j; ++i) warp_wait(&bars[Y::kBarVFull + i % kNR], (i / kNR) & 1);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc_qk = idesc_bf16_f32(kRows, kChunk, false, false);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(kRows, kD, false, true);
    const uint64_t k_desc0 = sdesc_sw128(smem_u32(base + Y::kOffK), 16, 1024);
    const uint64_t v_desc0 = sdesc_sw128(smem_u32(base + Y::kOffV), kGroupBytes, 1024);
    int nk = 0, nv = 0;  // QKs and PVs so far, over all units
    int units = 0;
    bool fail = false, first = true;  // the unit's next PV overwrites O
    auto issue_qk = [&]() -> bool {   // S(nk) = Q K(nk)^T into S buffer nk % 2
      const int st = nk % kNR;
      if (!warp_wait(&bars[Y::kBarKFull + st], (nk / kNR) & 1)) return false;
      tc_fence_after();
      const uint64_t kd = k_desc0 + (uint64_t)((st * Y::kStageBytes) >> 4);
      const uint32_t d = tbase + Y::kColS + (nk & 1) * kChunk;
#pragma unroll
      for (int kk = 0; kk < kD / 16; ++kk)
        mma_ts_w(d, tbase + Y::kColQ + kk * 8, kd + (uint64_t)(((kk >> 2) * kGroupBytes + (kk & 3) * 32) >> 4), idesc_qk,
                 kk > 0 ? 1u : 0u);
      mma_commit_w(&bars[Y::kBarSFull + (nk & 1)]);
      mma_commit_w(&bars[Y::kBarKEmpty + st]);
      ++nk;
      return true;
    };
    for (int su = 0; !fail; ++su) {
      const int s = su & 1;
      if (!idle_wait_warp(&bars[Y::kBarSlotFull + s], (su >> 1) & 1)) {
        fail = true;
        break;
      }
      const UnitInfo *I = info(s);
      const int live = I->live, part = I->part;
      if (!live) break;
      const Chunks<X, kSel> ch(*I, token_bits(s) + kBitWords, P.W);
      const int t_hi = I->len - I->n + min(I->n, I->r0 + T) - 1;
      if (part & 1) {
        first = true;
        if (!warp_wait(&bars[Y::kBarQFull], units & 1)) {
          fail = true;
          break;
        }
        ++units;
        tc_fence_after();
      }
      // c: the next PV's chunk, ca: the next QK's, which runs two ahead
      int c = ch.next(ch.ca), ca = c;
      bool q_done = false;
      auto advance_qk = [&]() {
        if (ca < 0 || !issue_qk()) return ca < 0;
        ca = ch.next(ca + 1);
        if (ca < 0 && (part & 2)) {
          mma_commit_w(&bars[Y::kBarQEmpty]);
          q_done = true;
        }
        return true;
      };
      if (!advance_qk() || !advance_qk()) fail = true;
      for (; c >= 0 && !fail; c = ch.next(c + 1)) {
        const int st = nv % kNR;
        if (!warp_wait(&bars[Y::kBarVFull + st], (nv / kNR) & 1)) {
          fail = true;
          break;
        }
        tc_fence_after();
        // V rows behind the unit's last visible key are zeroed: their P is zero, but the slots (or
        // what an unloaded box left) may hold NaN, and 0 * NaN is NaN.
        const int valid_rows = t_hi + 1 - c * kChunk;
        if (valid_rows < kChunk) {
          uint8_t *vs = base + Y::kOffV + st * Y::kStageBytes;
          for (int rr = max(valid_rows, 0) + lane; rr < kChunk; rr += 32)
            for (int q = 0; q < Y::kGroups; ++q) {
              uint4 *p4 = (uint4 *)(vs + q * kGroupBytes + rr * 128);
#pragma unroll
              for (int x = 0; x < 8; ++x) p4[x] = make_uint4(0, 0, 0, 0);
            }
          fence_proxy_async_smem();
          __syncwarp();
        }
        const uint64_t vd = v_desc0 + (uint64_t)((st * Y::kStageBytes) >> 4);
        const uint32_t pcol = tbase + Y::kColS + (nv & 1) * kChunk;
#pragma unroll
        for (int step = 0; step < 2 && !fail; ++step) {
          // a step brings 16 keys of each half of the chunk
          if (!warp_wait(&bars[Y::kBarPFull + 2 * (nv & 1) + step], (nv >> 1) & 1)) fail = true;
          tc_fence_after();
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int kk = 2 * e + step;
            mma_ts_w(tbase, pcol + kk * 8, vd + (uint64_t)((kk * 2048) >> 4), idesc_pv, (!first || step > 0 || e > 0) ? 1u : 0u);
          }
        }
        if (fail) break;
        first = false;
        mma_commit_w(&bars[Y::kBarVEmpty + st]);
        mma_commit_w(&bars[Y::kBarPVDone]);
        ++nv;
        // S of two chunks on goes into the buffer that this PV reads; MMAs run in issue order
        if (!advance_qk()) fail = true;
      }
      if (!fail && (part & 2)) {
        if (!q_done) mma_commit_w(&bars[Y::kBarQEmpty]);
        mma_commit_w(&bars[Y::kBarODone]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[Y::kBarSlotFree + s]);
    }
    if (fail && lane == 0) {
      record_status(P.status, QSA_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    mma_commit_w(&bars[Y::kBarDrain]);  // and MMAs complete
    warp_wait(&bars[Y::kBarDrain], 0);
  } else if (warp >= kSoftWarp0) {
    // ---------------------------------------------------------------- softmax + epilogue
    // Warp (lane group, sub-group) owns 16 rows: thread t < 16 holds its row's first 32 keys of every
    // chunk, the first half of its Q and of its O, thread t + 16 the others.
    const int row0 = 32 * (warp & 3) + 16 * ((warp - kSoftWarp0) >> 2);
    const int hh = lane >> 4, row = row0 + (lane & 15);
    const int tok = row / G, h = row % G;
    const uint32_t lane_addr = tbase + ((uint32_t)row0 << 16);
    const uint64_t scale2 = f2_splat(P.sl2);
    int n_all = 0, units = 0;  // chunks and units so far
    bool some = false;         // a chunk of this unit
    float m_ref = -INFINITY, l = 0.f;
    bool fail = false;
    for (int su = 0; !fail; ++su) {
      const int s = su & 1;
      if (!idle_wait_warp(&bars[Y::kBarSlotFull + s], (su >> 1) & 1)) {
        fail = true;
        break;
      }
      const UnitInfo *I = info(s);
      if (!I->live) break;
      const int part_of = I->part;
      const int t0 = I->len - I->n + I->r0;  // the unit's first position
      const bool valid = tok < T && I->r0 + tok < I->n;
      const int t = valid ? t0 + tok : -1;
      const size_t at = (((size_t)I->q0 + (valid ? I->r0 + tok : 0)) * D.Hq + I->g * G + h) * kD + hh * (kD / 2);
      if (part_of & 1) {
        some = false;
        m_ref = -INFINITY;
        l = 0.f;
        // Q of the unit, once every QK of the unit before has completed
        constexpr int kQ = (kD + 127) / 128;  // 64 dims at a time (32 at head_dim 64)
        uint32_t q[kQ][32];
        const uint4 *src = (const uint4 *)(P.q + at);
#pragma unroll
        for (int i = 0; i < kD / 16; ++i) {
          const uint4 x = valid ? src[i] : make_uint4(0, 0, 0, 0);
          uint32_t *d = &q[i / 8][4 * (i % 8)];
          d[0] = x.x, d[1] = x.y, d[2] = x.z, d[3] = x.w;
        }
        if (units > 0 && !warp_wait(&bars[Y::kBarQEmpty], (units - 1) & 1)) {
          fail = true;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < kQ; ++i)
          if (kD == 64) tmem_st16_split_lo<16>(lane_addr + Y::kColQ, q[i]);
          else tmem_st32_split<kD / 4>(lane_addr + Y::kColQ + 32 * i, q[i]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[Y::kBarQFull]);
        ++units;
      }
      const Chunks<X, kSel> ch(*I, token_bits(s) + kBitWords, P.W);
      // A chunk whose last key is no further than t_free needs no mask per key: without a selection
      // the position of the warp's first row, with one the unit's last visible key.
      const int t_free = kSel ? t0 + min(I->n - I->r0, T) - 1 : t0 + row0 / G;
      const int h_tail = kSel ? (t + 1) / D.B * (D.B / kHalf) : 0;  // the trailing range starts at this chunk
      const uint32_t *my_bits = token_bits(s) + (valid ? tok : 0) * P.W;
      for (int c = ch.next(ch.ca); c >= 0; c = ch.next(c + 1)) {
        // this thread's first `lim` keys are visible: up to the position, or, in a selected block, all
        int lim = min(max(t + 1 - c * kChunk - hh * 32, 0), 32);
        bool part = c * kChunk + kChunk - 1 > t_free, any = true;
        if (kSel) {
          if (c < h_tail) lim = (my_bits[(c - ch.ca) >> 5] >> ((c - ch.ca) & 31)) & 1u ? 32 : 0;
          part = part || __any_sync(0xffffffffu, lim > 0 && lim < 32);
          any = __any_sync(0xffffffffu, lim > 0);
        }
        const uint32_t s_col = lane_addr + Y::kColS + (n_all & 1) * kChunk;
        if (!warp_wait(&bars[Y::kBarSFull + (n_all & 1)], (n_all >> 1) & 1)) {
          fail = true;
          break;
        }
        tc_fence_after();
        uint32_t sv[32];
        float mx = -INFINITY;
        if (any) {
          tmem_ld32_split<32>(s_col, sv);
          tmem_ld_wait();
          mx = part ? max_quarter<false>(sv, lim) : max_quarter<true>(sv, 32);
          if (kSel && lim == 0) mx = -INFINITY;
        }
        const float cmax = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16)) * P.sl2;
        bool rescale = false;
        float alpha = 1.f;
        if (cmax > -INFINITY) {
          if (m_ref == -INFINITY) {
            m_ref = cmax;
          } else if (cmax > m_ref + 8.f) {
            rescale = true;
            alpha = ex2_approx(m_ref - cmax);
            m_ref = cmax;
          }
        }
        if (__any_sync(0xffffffffu, rescale)) {
          // A row that had a reference had a chunk before. S of this chunk being there proves the PV
          // before the last complete, so one parity wait covers the last; the next one waits for
          // this warp's arrival below.
          if (!warp_wait(&bars[Y::kBarPVDone], (n_all - 1) & 1)) {
            fail = true;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int cb = 0; cb < kD / 64; ++cb) {
            uint32_t ov[32];
            tmem_ld32_split<kD / 2>(lane_addr + cb * 32, ov);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 32; ++q) ov[q] = __float_as_uint(__uint_as_float(ov[q]) * alpha);
            tmem_st32_split<kD / 2>(lane_addr + cb * 32, ov);
          }
          l *= alpha;
        }
        uint64_t acc[2] = {0, 0};
        auto step_done = [&](int step) {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[Y::kBarPFull + 2 * (n_all & 1) + step]);
        };
        // a thread that sees none of its keys takes +inf as its reference: p = 0
        const uint64_t negm2 = f2_splat(!kSel || part || lim ? -m_ref : -INFINITY);
        if (any && !part) {
          p_quarter<true, 0, 16>(sv, 32, scale2, negm2, acc);
          tmem_st8_split_of<16, 0>(s_col, sv);
          p_quarter<true, 16, 24>(sv, 32, scale2, negm2, acc);  // beside the store
          step_done(0);
          p_quarter<true, 24, 32>(sv, 32, scale2, negm2, acc);
        } else {
          if (any) p_quarter<false>(sv, lim, scale2, negm2, acc);
          else zero_quarter(sv);
          tmem_st8_split_of<16, 0>(s_col, sv);
          step_done(0);
        }
        tmem_st8_split_of<16, 8>(s_col + 8, sv);
        float sum0, sum1;
        f2_unpack(f2_add(acc[0], acc[1]), sum0, sum1);
        l += sum0 + sum1;
        step_done(1);
        some = true;
        ++n_all;
      }
      if ((part_of & 2) || fail) {
        const float lt = l + __shfl_xor_sync(0xffffffffu, l, 16);  // the row's sum over both key ranges
        // ------------------------------------------------------------ epilogue
        const bool have_o = !fail && warp_wait(&bars[Y::kBarODone], (units - 1) & 1) && some;
        if (!have_o && some && !fail) fail = true;
        if (fail) {
          if (lane == 0) record_status(P.status, QSA_ERR_TIMEOUT);
          *abort_flag = 1;
        }
        tc_fence_after();
        const bool keep = have_o && lt > 0.f;  // a row that sees nothing is written as zeros
        const int slot = I->slot;
        const float inv = keep ? 1.f / lt : 0.f;
        const size_t pr = (size_t)max(slot, 0) * kRows + row;
        if (slot >= 0 && valid && hh == 0)
          *(float2 *)(P.part_ml + pr * 2) = make_float2(keep ? m_ref : -INFINITY, keep ? lt : 0.f);
#pragma unroll 1
        for (int cb = 0; cb < kD / 32; ++cb) {
          uint32_t ov[16];
          __syncwarp();
          if (have_o) {  // the same for the whole warp
            tmem_ld16_split<kD / 2>(lane_addr + cb * 16, ov);
            tmem_ld_wait();
          }
          if (valid && slot < 0) {
            uint32_t pk[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
              pk[q] = keep ? pack_bf16x2(__uint_as_float(ov[2 * q]) * inv, __uint_as_float(ov[2 * q + 1]) * inv) : 0u;
            uint4 *o4 = (uint4 *)(P.out + at + cb * 16);
            o4[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            o4[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
          } else if (valid && have_o) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *(uint4 *)(P.part_o + part_at<X>(slot, row, hh * (kD / 2) + cb * 16 + 4 * q)) =
                  make_uint4(ov[4 * q], ov[4 * q + 1], ov[4 * q + 2], ov[4 * q + 3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[Y::kBarSlotFree + s]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, kTmemCols);
  }
}

template <int D_>
size_t smem_of(bool sel, int nb) {
  return 1024 + Layout<D_>::kOffBits + (sel ? 2 * kBitSlotBytes : 0) + plan_bytes(nb);
}
static_assert(1024 + Layout<256>::kOffBits + 2 * kBitSlotBytes + plan_bytes(kMaxSeqs) <= 227 * 1024, "shared memory");
static_assert(1024 + Layout<128>::kOffBits + 2 * kBitSlotBytes + plan_bytes(kMaxSeqs) <= 227 * 1024, "shared memory");

template <int D_>
cudaError_t launch_d(const Dims &D, const Paged &G, const void *q, const void *k_pages, const void *v_pages,
                     const int32_t *sel, void *out, int min_rows, void *scratch, int *status, cudaStream_t st) {
  auto kern = sel ? k_paged_tc1<D_, true> : k_paged_tc1<D_, false>;
  auto launch = [&](const TcParams &P, const CUtensorMap &tk, const CUtensorMap &tv, size_t smem) {
    const cudaError_t e = ensure_smem(kern, smem);
    return e == cudaSuccess ? launch_maybe_pdl(kern, dim3(P.C), dim3(kThreads), smem, st, false, tk, tv, P) : e;
  };
  return launch_chunks<One<D_>>(launch, smem_of<D_>, D, G, q, k_pages, v_pages, sel, out, min_rows, scratch, status, st);
}

}  // namespace

size_t paged_tc1_workspace(const Dims &D) {
  return D.d == 256 ? partials_bytes<One<256>>() : D.d == 128 ? partials_bytes<One<128>>() : partials_bytes<One<64>>();
}

cudaError_t launch_paged_tc1(const Dims &D, const Paged &G, const void *q, const void *k_pages, const void *v_pages,
                             const int32_t *sel, void *out, int min_rows, void *scratch, int *status, cudaStream_t st) {
  auto launch = D.d == 256 ? launch_d<256> : D.d == 128 ? launch_d<128> : launch_d<64>;
  return launch(D, G, q, k_pages, v_pages, sel, out, min_rows, scratch, status, st);
}

}  // namespace qsa
