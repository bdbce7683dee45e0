// Attention of chunks of new tokens over a paged K/V cache on 5th-generation tensor cores
// (tcgen05), head_dim 128: over every visible token, or over each token's selected blocks
// and its trailing range.
//   S = Q K^T, P = 2^(S scale log2 e - m), O += P V, out = O / sum P
//
// Work unit: one KV head of one sequence and 2 T consecutive tokens, T = 128 / G, held as two
// 128-row MMA tiles A and B of (token, query head) rows that share every K/V chunk in shared
// memory. A chunk is 128 keys, gathered from the pages by TMA (one box per page and 64
// columns). 4 * 128 * 128 * 128 products and 2 * 128 * 128 exponentials per chunk: at 4096
// products and 16 exponentials a clock an SM needs 2048 clocks for either, and the QK
// products read their operands at the full rate of shared memory, so tensor pipe, MUFU and
// shared memory bound it together.
//
// The work is divided among the CTAs as qsa_paged_plan.cuh describes. Inside a CTA the roles are
// pipelined across units:
//   warp 0      TMA producer: Q, then K of chunk j and V of chunk j - 1 into ring entry j;
//               its lanes hold the page numbers of the next chunk's boxes;
//   warp 1      MMA issuer (TMEM owner): per chunk O_A += P_A V, S_A = Q_A K'^T, then B;
//   warp 2      builder: the next unit's geometry, selection lists and chunk bitmaps;
//   warps 4-19  softmax, eight per tile, 16 rows per warp, two threads a row with 64 logits
//               each, 32 in registers at a time (16x32bx2 TMEM accesses): row max by one
//               shuffle, P in bf16 over the first half of each S half, in two steps that the
//               PV product takes as they come, O rescaled only when the max has moved by more
//               than 2^8, and the epilogue. Four warps a scheduler: with one thread a row the
//               exponentials and the arithmetic around them did not overlap (1560-1630 us at
//               8K of 32K tokens).
// Every wait is bounded; on expiry the kernel records QSA_ERR_TIMEOUT and unwinds.
//
// Measured, 16 / 2 heads, pages of 64: 8192 tokens of 32768 1515 us alone (1.27 PFLOP/s, 0.77 of
// cuBLAS), 1740 in long loops under the power cap; tensor pipe 60 % busy, MUFU 62 %. A part of the
// exponentials as polynomials on the FMA pipe: no gain, the issue slots are as scarce. 4096 tokens of
// 24000, 64 independently selected blocks each: 655 us, in which 16 tokens see nearly every
// block between them and the products of the whole context are made (0.74 TFLOP, 1.1 PFLOP/s). The
// row kernel, which reads every token's own blocks, is bound by L2 there (1535 us). Products per
// 64-key half that a tile sees: 675 to 775 us, the shorter MMAs save less than their issue costs.
#include "qsa_paged_plan.cuh"

namespace qsa {
namespace {

constexpr int kD = 128;      // head dim served
constexpr int kTiles = 2;    // tiles per unit
constexpr int kChunk = 128;  // keys per chunk
constexpr int kNE = 2;       // ring depth: entry j holds K of chunk j and V of chunk j - 1
struct Two128 {
  static constexpr int kD = qsa::kD, kTiles = qsa::kTiles, kChunk = qsa::kChunk;
};
constexpr int kThreads = 640;
constexpr int kBuilderWarp = 2;
constexpr int kSoftWarp0 = 4;  // first softmax warp
constexpr int kSoftWarps = 16;
constexpr uint32_t kTmemCols = 512;  // S of tile w at 128 w, O of tile w at 256 + 128 w

constexpr uint32_t kQBytes = kRows * kD * 2;    // per tile, two 64-column halves
constexpr uint32_t kKVBytes = kChunk * kD * 2;  // per K (or V) chunk, two halves
constexpr uint32_t kEntryBytes = 2 * kKVBytes;
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffE = kOffQ + kTiles * kQBytes;
constexpr uint32_t kOffBar = kOffE + kNE * kEntryBytes;
constexpr uint32_t kOffMisc = kOffBar + 256;
constexpr uint32_t kOffInfo = kOffMisc + 64;
constexpr uint32_t kOffBits = kOffInfo + 2 * kInfoBytes;  // with a selection: [slot] kBitSlotBytes

// barrier slots
constexpr int kBarQ = 0;                        // Q of the unit landed
constexpr int kBarQEmpty = 1;                   // every QK of the unit completed
constexpr int kBarFull = 2;                     // [ring entry]
constexpr int kBarEmpty = kBarFull + kNE;       // [ring entry]
constexpr int kBarSFull = kBarEmpty + kNE;      // [tile]
constexpr int kBarPFull = kBarSFull + 2;        // [tile][step], 8 arrivals
constexpr int kBarPVDone = kBarPFull + 4;       // [tile]
constexpr int kBarSlotFull = kBarPVDone + 2;    // [slot], the builder's 32 lanes
constexpr int kBarSlotFree = kBarSlotFull + 2;  // [slot], producer + MMA warp + softmax warps
constexpr int kBarDrain = kBarSlotFree + 2;     // every MMA of the block completed
constexpr int kNumBars = kBarDrain + 1;
static_assert(kNumBars * 8 <= 256, "barrier area");

// A softmax thread's place: warp (tile w, lane group, sub-group) owns 16 rows of its tile; lane
// t < 16 holds its row's first 64 keys of every chunk and the first 64 columns of its O, lane
// t + 16 the same row's others.
struct SoftPlace {
  int w, row0, hh, row, tok, h;  // tile, the warp's first row, half, row, token of the unit, head of the group
  bool in_tile;                  // G need not divide 128
};
__device__ __forceinline__ SoftPlace soft_place(int tid, int T, int G) {
  SoftPlace p;
  const int warp = tid >> 5, lane = tid & 31, sw = warp - kSoftWarp0;
  p.w = sw >> 3;
  p.row0 = 32 * (warp & 3) + 16 * ((sw >> 2) & 1);
  p.hh = lane >> 4;
  p.row = p.row0 + (lane & 15);
  p.tok = p.w * T + p.row / G;
  p.h = p.row % G;
  p.in_tile = p.row / G < T;
  return p;
}

template <bool kSel>
__global__ void __launch_bounds__(kThreads, 1)
k_paged_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
           const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TcParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t *bars = (uint64_t *)(base + kOffBar);
  uint32_t *tmem_slot = (uint32_t *)(base + kOffMisc);
  volatile int *abort_flag = (volatile int *)(base + kOffMisc + 8);
  uint8_t *plan = base + kOffBits + (kSel ? 2 * kBitSlotBytes : 0);
  const PlanArea L = {(long long *)plan, (SeqGeo *)(plan + (size_t)(P.nb + 1) * 8)};

  const Dims &D = P.D;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = P.T, G = D.G;
  auto info = [&](int s) { return (const UnitInfo *)(base + kOffInfo + s * kInfoBytes); };
  auto token_bits = [&](int s) { return (const uint32_t *)(base + kOffBits + s * kBitSlotBytes); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t count = 1;
      if (i >= kBarPFull && i < kBarPFull + 4) count = 8;
      if (i == kBarSlotFull || i == kBarSlotFull + 1) count = 32;
      if (i == kBarSlotFree || i == kBarSlotFree + 1) count = 2 + kSoftWarps;
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
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  make_plan<Two128>(P, L, blockIdx.x == 0 ? P.status : nullptr);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  pdl_trigger();  // the merge may take its place; it waits for this kernel's end

  if (warp == kBuilderWarp) {
    const SlotArea area = {&bars[kBarSlotFull], &bars[kBarSlotFree], base + kOffInfo, base + kOffBits, abort_flag};
    build_segments<Two128, kSel>(P, area, L, lane);
  } else if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    // Lane i < 128 / box holds the pool plane (page, KV head) of the i-th box of the next chunk
    // (-1: no token there, or a page outside the pool; nothing is loaded), and issues that box.
    const int n_box = kChunk / P.box;
    const uint32_t box_bytes = (uint32_t)P.box * 128;  // 64 columns of a box
    int j = 0, qn = 0;
    bool fail = false, have_q = false;
    for (int su = 0; !fail; ++su) {
      const int s = su & 1;
      if (!idle_wait_warp(&bars[kBarSlotFull + s], (su >> 1) & 1)) {
        fail = true;
        break;
      }
      const UnitInfo I = *info(s);
      if (!I.live) break;
      if (I.part & 1) have_q = false;
      const Chunks<Two128, kSel> ch(I, token_bits(s) + kBitWords, P.W);
      const int t_hi = I.len - I.n + min(I.n, I.r0 + kTiles * T) - 1;  // the unit's last visible key
      auto plane = [&](int c) {
        int z = -1;
        const int key = c * kChunk + lane * P.box;
        if (c >= 0 && lane < n_box && key <= t_hi) {
          const int page = P.P.table[(size_t)I.b * P.P.max_pages + (key >> P.P.ps_shift)];
          if (page >= 0 && page < P.P.n_pages) z = page * D.Hkv + I.g;
          else record_status(P.status, QSA_ERR_DEVICE_CHECK);
        }
        return z;
      };
      int c = ch.next(ch.ca);
      if (c >= 0) {
        int z = plane(c), zp = -1, cp = -1;  // boxes of K chunk c and of V chunk cp
        if (!have_q) {
          if (qn > 0 && !warp_wait(&bars[kBarQEmpty], (qn - 1) & 1)) {
            fail = true;
            break;
          }
          if (lane == 0) {
            mbar_arrive_expect_tx(&bars[kBarQ], (uint32_t)(kTiles * 2 * T * G * 128));
            for (int w = 0; w < kTiles; ++w) {
              uint8_t *dst = base + kOffQ + w * kQBytes;
              tma_load_3d(&tm_q, &bars[kBarQ], dst, 0, I.g * G, I.q0 + I.r0 + w * T);
              tma_load_3d(&tm_q, &bars[kBarQ], dst + kQBytes / 2, 64, I.g * G, I.q0 + I.r0 + w * T);
            }
          }
          have_q = true;
          ++qn;
        }
        while (c >= 0 || cp >= 0) {
          const int cn = c >= 0 ? ch.next(c + 1) : -1;
          const int zn = plane(cn);  // read ahead
          const int se = j % kNE;
          if (j >= kNE && !warp_wait(&bars[kBarEmpty + se], ((j / kNE) & 1) ^ 1)) {
            fail = true;
            break;
          }
          uint8_t *es = base + kOffE + se * kEntryBytes;
          const int boxes = __popc(__ballot_sync(0xffffffffu, z >= 0)) + __popc(__ballot_sync(0xffffffffu, zp >= 0));
          if (lane == 0) mbar_arrive_expect_tx(&bars[kBarFull + se], (uint32_t)boxes * 2 * box_bytes);
          __syncwarp();
          if (z >= 0) {
            const int y = (c * kChunk + lane * P.box) & (P.P.ps - 1);
            uint8_t *dst = es + lane * box_bytes;
            tma_load_3d(&tm_k, &bars[kBarFull + se], dst, 0, y, z);
            tma_load_3d(&tm_k, &bars[kBarFull + se], dst + kKVBytes / 2, 64, y, z);
          }
          if (zp >= 0) {
            const int y = (cp * kChunk + lane * P.box) & (P.P.ps - 1);
            uint8_t *dst = es + kKVBytes + lane * box_bytes;
            tma_load_3d(&tm_v, &bars[kBarFull + se], dst, 0, y, zp);
            tma_load_3d(&tm_v, &bars[kBarFull + se], dst + kKVBytes / 2, 64, y, zp);
          }
          __syncwarp();
          cp = c;
          zp = z;
          c = cn;
          z = zn;
          ++j;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kBarSlotFree + s]);
    }
    if (fail) {
      if (lane == 0) record_status(P.status, QSA_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    // after a timeout, here or in another warp, copies may be in flight: they land before the block ends
    for (int i = max(0, j - kNE); i < j; ++i) warp_wait(&bars[kBarFull + i % kNE], (i / kNE) & 1);
    if (qn > 0) warp_wait(&bars[kBarQ], (qn - 1) & 1);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc_qk = idesc_bf16_f32(kRows, kChunk, false, false);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(kRows, kD, false, true);
    int j = 0, qn = 0;
    int n_pv0 = 0, n_pv1 = 0;  // PVs issued per tile
    bool fail = false;
    // of the unit: its Q is there, its last QK is issued, the tile's next PV is its first
    bool have_q = false, q_done = false, first0 = true, first1 = true;
    const uint64_t q_desc0 = sdesc_sw128(smem_u32(base + kOffQ), 16, 1024);
    const uint64_t k_desc0 = sdesc_sw128(smem_u32(base + kOffE), 16, 1024);
    const uint64_t v_desc0 = sdesc_sw128(smem_u32(base + kOffE + kKVBytes), kKVBytes / 2, 1024);
    auto issue_qk = [&](int w, int se) {  // S_w = Q_w K^T from ring entry se
      const uint64_t qd = q_desc0 + (uint64_t)((w * kQBytes) >> 4);
      const uint64_t kd = k_desc0 + (uint64_t)((se * kEntryBytes) >> 4);
      const uint32_t d = tbase + (uint32_t)(w * 128);
#pragma unroll
      for (int kk = 0; kk < kD / 16; ++kk) {
        const uint64_t off_q = (uint64_t)(((kk >> 2) * (kQBytes / 2) + (kk & 3) * 32) >> 4);
        const uint64_t off_k = (uint64_t)(((kk >> 2) * (kKVBytes / 2) + (kk & 3) * 32) >> 4);
        mma_ss_w(d, qd + off_q, kd + off_k, idesc_qk, kk > 0 ? 1u : 0u);
      }
      mma_commit_w(&bars[kBarSFull + w]);
    };
    // O_w (+)= P_w V from ring entry se once P_w is written; a unit's first PV overwrites O
    auto issue_pv = [&](int w, int se, bool first) -> bool {
      const int cnt = w ? n_pv1++ : n_pv0++;
      const uint64_t vd = v_desc0 + (uint64_t)((se * kEntryBytes) >> 4);
      const uint32_t o = tbase + 256u + (uint32_t)(w * 128), pcol = tbase + (uint32_t)(w * 128);
#pragma unroll
      for (int step = 0; step < 2; ++step) {
        if (!warp_wait(&bars[kBarPFull + 2 * w + step], cnt & 1)) return false;
        tc_fence_after();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // keys 16 kk .. of half kk / 4 sit at columns 64 (kk / 4) + 8 (kk % 4); a step brings 32 keys of each
          const int kk = (e >> 1) * 4 + step * 2 + (e & 1);
          mma_ts_w(o, pcol + (kk >> 2) * 64 + (kk & 3) * 8, vd + (uint64_t)((kk * 2048) >> 4), idesc_pv,
                   (!first || step > 0 || e > 0) ? 1u : 0u);
        }
      }
      mma_commit_w(&bars[kBarPVDone + w]);
      return true;
    };
    for (int su = 0; !fail; ++su) {
      const int s = su & 1;
      if (!idle_wait_warp(&bars[kBarSlotFull + s], (su >> 1) & 1)) {
        fail = true;
        break;
      }
      const int live = info(s)->live, part = info(s)->part;
      const int t_hi = info(s)->len - info(s)->n + min(info(s)->n, info(s)->r0 + kTiles * T) - 1;
      if (!live) break;
      if (part & 1) have_q = q_done = false, first0 = first1 = true;
      const Chunks<Two128, kSel> ch(*info(s), token_bits(s) + kBitWords, P.W);
      int c = ch.next(ch.ca);
      if (c >= 0) {
        if (!have_q) {
          if (!warp_wait(&bars[kBarQ], qn & 1)) fail = true;
          ++qn;
          have_q = true;
          tc_fence_after();
        }
        if (!fail) {
          const int se = j % kNE;
          if (!warp_wait(&bars[kBarFull + se], (j / kNE) & 1)) fail = true;
          tc_fence_after();
          for (int w = 0; w < kTiles && !fail; ++w)
            if (ch.has(w, c)) issue_qk(w, se);
          if (!fail) mma_commit_w(&bars[kBarEmpty + se]);
          ++j;
        }
        int cn = fail ? -1 : ch.next(c + 1);
        if (!fail && cn < 0 && (part & 2)) {
          mma_commit_w(&bars[kBarQEmpty]);
          q_done = true;
        }
        while (!fail && c >= 0) {
          const int se = j % kNE;
          if (!warp_wait(&bars[kBarFull + se], (j / kNE) & 1)) {
            fail = true;
            break;
          }
          tc_fence_after();
          // V rows behind the unit's last visible key are zeroed: their P is zero, but the
          // slots (or what an unloaded box left) may hold NaN, and 0 * NaN is NaN.
          const int valid_rows = t_hi + 1 - c * kChunk;
          if (valid_rows < kChunk) {
            uint8_t *vs = base + kOffE + se * kEntryBytes + kKVBytes;
            for (int rr = max(valid_rows, 0) + lane; rr < kChunk; rr += 32) {
              uint4 *p0 = (uint4 *)(vs + rr * 128);
              uint4 *p1 = (uint4 *)(vs + kKVBytes / 2 + rr * 128);
#pragma unroll
              for (int q = 0; q < 8; ++q) p0[q] = p1[q] = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          for (int w = 0; w < kTiles; ++w) {
            if (ch.has(w, c)) {
              if (!issue_pv(w, se, w ? first1 : first0)) {
                fail = true;
                break;
              }
              (w ? first1 : first0) = false;
            }
            if (cn >= 0 && ch.has(w, cn)) issue_qk(w, se);
          }
          if (fail) break;
          mma_commit_w(&bars[kBarEmpty + se]);
          ++j;
          const int cnn = cn >= 0 ? ch.next(cn + 1) : -1;
          if (cn >= 0 && cnn < 0 && (part & 2)) {
            mma_commit_w(&bars[kBarQEmpty]);
            q_done = true;
          }
          c = cn;
          cn = cnn;
        }
      }
      if (!fail && (part & 2) && have_q && !q_done) mma_commit_w(&bars[kBarQEmpty]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kBarSlotFree + s]);
    }
    if (fail && lane == 0) {
      record_status(P.status, QSA_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    mma_commit_w(&bars[kBarDrain]);  // and MMAs complete
    warp_wait(&bars[kBarDrain], 0);
  } else if (warp >= kSoftWarp0) {
    // ---------------------------------------------------------------- softmax + epilogue
    const int w = (warp - kSoftWarp0) >> 3;  // tile
    const uint32_t s_col = tbase + ((uint32_t)(32 * (warp & 3) + 16 * (((warp - kSoftWarp0) >> 2) & 1)) << 16) + w * 128;
    const uint32_t o_col = s_col + 256;
    const uint64_t scale2 = f2_splat(P.sl2);
    int n_all = 0;      // chunks of this tile over all units so far: S, P and PV phases
    bool some = false;  // a chunk of this unit
    float m_ref = -INFINITY, l = 0.f;
    bool fail = false;
    for (int su = 0; !fail; ++su) {
      const int s = su & 1;
      if (!idle_wait_warp(&bars[kBarSlotFull + s], (su >> 1) & 1)) {
        fail = true;
        break;
      }
      const UnitInfo *I = info(s);
      if (!I->live) break;
      if (I->part & 1) {
        some = false;
        m_ref = -INFINITY;
        l = 0.f;
      }
      const Chunks<Two128, kSel> ch(*I, token_bits(s) + kBitWords, P.W);
      // A chunk whose last key is no further than t_free needs no mask per key: without a selection
      // the position of the warp's first row, with one the unit's last visible key.
      int t_free, t = 0, h_tail = 0;
      const uint32_t *my_bits = nullptr;
      {
        const SoftPlace p = soft_place(fresh_tid(), T, G);
        const int t0 = I->len - I->n + I->r0;
        t_free = kSel ? t0 + min(I->n - I->r0, kTiles * T) - 1 : t0 + p.w * T + p.row0 / G;
        if (kSel) {
          const bool valid = p.in_tile && I->r0 + p.tok < I->n;
          t = valid ? t0 + p.tok : -1;
          h_tail = (t + 1) / D.B * (D.B / kHalf);  // the row's trailing range starts at this 64-key half
          my_bits = token_bits(s) + (valid ? p.tok : 0) * P.W;
        }
      }
      for (int c = ch.next(ch.ca); c >= 0; c = ch.next(c + 1)) {
        if (!ch.has(w, c)) continue;
        // This thread's first `lim` keys are visible: without a selection, or in the trailing
        // range, up to the position; else its half is a part of one block, seen whole or not.
        // Keys are masked one by one where some row sees a part of its half, or behind the last
        // visible key (NaN may be there). Elsewhere a thread sees all its keys or none; one that
        // sees none takes +inf as its reference: p = 0.
        int lim = kHalf;
        bool part = c * kChunk + kChunk - 1 > t_free, any = true;
        if (kSel) {
          const int half = 2 * c + (lane >> 4);
          lim = min(max(t + 1 - half * kHalf, 0), kHalf);
          if (half < h_tail) lim = (my_bits[(c - ch.ca) >> 4] >> (half - 2 * ch.ca & 31)) & 1u ? kHalf : 0;
          part = part || __any_sync(0xffffffffu, lim > 0 && lim < kHalf);
          any = __any_sync(0xffffffffu, lim > 0);
        } else if (part) {
          const SoftPlace p = soft_place(fresh_tid(), T, G);
          const bool valid = p.in_tile && I->r0 + p.tok < I->n;
          lim = valid ? min(max(I->len - I->n + I->r0 + p.tok + 1 - (2 * c + p.hh) * kHalf, 0), kHalf) : 0;
        }
        if (!warp_wait(&bars[kBarSFull + w], n_all & 1)) {
          fail = true;
          break;
        }
        tc_fence_after();
        // Logits come in 32 at a time, the second 32 twice (for the max, then for P): 64 of them in
        // registers at once spill.
        uint32_t sv[32];
        float mx = -INFINITY;
        if (any) {
          tmem_ld32_split<64>(s_col + 32, sv);
          tmem_ld_wait();
          mx = part ? max_quarter<false>(sv, lim - 32) : max_quarter<true>(sv, 32);
          tmem_ld32_split<64>(s_col, sv);
          tmem_ld_wait();
          mx = fmaxf(mx, part ? max_quarter<false>(sv, lim) : max_quarter<true>(sv, 32));
          if (kSel && lim == 0) mx = -INFINITY;
        }
        const float cmax = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16)) * P.sl2;
        bool rescale = false;
        float alpha = 1.f;
        if (cmax > -INFINITY) {  // the row sees a key here
          if (m_ref == -INFINITY) {
            m_ref = cmax;
          } else if (cmax > m_ref + 8.f) {
            rescale = true;
            alpha = ex2_approx(m_ref - cmax);
            m_ref = cmax;
          }
        }
        if (__any_sync(0xffffffffu, rescale)) {
          // A row that had a reference had a chunk before. O is stable once that chunk's PV has
          // completed, and the next one waits for this warp's arrivals below.
          if (!warp_wait(&bars[kBarPVDone + w], (n_all - 1) & 1)) {
            fail = true;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int cb = 0; cb < 4; ++cb) {
            uint32_t ov[16];
            tmem_ld16_split<64>(o_col + cb * 16, ov);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 16; ++q) ov[q] = __float_as_uint(__uint_as_float(ov[q]) * alpha);
            tmem_st16_split<64>(o_col + cb * 16, ov);
          }
          l *= alpha;
        }
        uint64_t acc[2] = {0, 0};
        auto step_done = [&](int step) {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kBarPFull + 2 * w + step]);
        };
        const uint64_t negm2 = f2_splat(!kSel || part || lim ? -m_ref : -INFINITY);
        if (any) {
          if (part) p_quarter<false>(sv, lim, scale2, negm2, acc);
          else p_quarter<true>(sv, 32, scale2, negm2, acc);
        } else {
          zero_quarter(sv);
        }
        tmem_st16_split_lo<64>(s_col, sv);
        if (any) {
          tmem_ld32_split<64>(s_col + 32, sv);
          tmem_ld_wait();
        }
        step_done(0);
        if (any) {
          if (part) p_quarter<false>(sv, lim - 32, scale2, negm2, acc);
          else p_quarter<true>(sv, 32, scale2, negm2, acc);
        }
        tmem_st16_split_lo<64>(s_col + 16, sv);
        float sum0, sum1;
        f2_unpack(f2_add(acc[0], acc[1]), sum0, sum1);
        l += sum0 + sum1;
        step_done(1);
        some = true;
        ++n_all;
      }
      if ((I->part & 2) || fail) {
        const float lt = l + __shfl_xor_sync(0xffffffffu, l, 16);  // the row's sum over both halves
        // ------------------------------------------------------------ epilogue
        // The unit's last PV of the tile is phase n_all - 1: the one before it completed
        // before S of the last chunk did, and the next one needs this warp's next P.
        bool have_o = false;
        if (some && !fail) {
          have_o = warp_wait(&bars[kBarPVDone + w], (n_all - 1) & 1);
          if (!have_o) fail = true;
        }
        if (fail) {
          if (lane == 0) record_status(P.status, QSA_ERR_TIMEOUT);
          *abort_flag = 1;
        }
        tc_fence_after();
        const SoftPlace p = soft_place(fresh_tid(), T, G);
        const bool valid = p.in_tile && I->r0 + p.tok < I->n;
        const bool keep = have_o && lt > 0.f;  // a row that sees nothing is written as zeros
        const int slot = I->slot;
        const float inv = keep ? 1.f / lt : 0.f;
        __nv_bfloat16 *orow =
            P.out + (((size_t)I->q0 + (valid ? I->r0 + p.tok : 0)) * D.Hq + I->g * G + p.h) * kD + p.hh * 64;
        const size_t pr = (size_t)max(slot, 0) * (kTiles * kRows) + w * kRows + p.row;
        if (slot >= 0 && valid && p.hh == 0)
          *(float2 *)(P.part_ml + pr * 2) = make_float2(keep ? m_ref : -INFINITY, keep ? lt : 0.f);
#pragma unroll 1
        for (int cb = 0; cb < 4; ++cb) {
          uint32_t ov[16];
          __syncwarp();
          if (have_o) {  // the same for the whole warp
            tmem_ld16_split<64>(o_col + cb * 16, ov);
            tmem_ld_wait();
          }
          if (valid && slot < 0) {
            uint32_t pk[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
              pk[q] = keep ? pack_bf16x2(__uint_as_float(ov[2 * q]) * inv, __uint_as_float(ov[2 * q + 1]) * inv) : 0u;
            uint4 *o4 = (uint4 *)(orow + cb * 16);
            o4[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            o4[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
          } else if (valid && have_o) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *(uint4 *)(P.part_o + part_at<Two128>(slot, w * kRows + p.row, p.hh * 64 + cb * 16 + 4 * q)) =
                  make_uint4(ov[4 * q], ov[4 * q + 1], ov[4 * q + 2], ov[4 * q + 3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kBarSlotFree + s]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, kTmemCols);
  }
}

// ---------------------------------------------------------------- host side
size_t smem_of(bool sel, int nb) {
  return 1024 + kOffBits + (sel ? 2 * kBitSlotBytes : 0) + plan_bytes(nb);
}
static_assert(1024 + kOffBits + 2 * kBitSlotBytes + plan_bytes(kMaxSeqs) <= 227 * 1024, "shared memory");

}  // namespace

// bf16, head_dim 64, 128 or 256, blocks of whole 64-key halves.
bool paged_tc_supported(const Dims &D, const Paged &G, bool sel) {
  return D.bf16 && (D.d == 64 || D.d == 128 || D.d == 256) && D.G <= 32 && (!sel || D.B % kHalf == 0) &&
         (long long)G.n_pages * D.Hkv <= 0x7fffffffLL;
}

// The one-tile kernel takes less.
size_t paged_tc_workspace(const Dims &D) { return D.d != kD ? paged_tc1_workspace(D) : partials_bytes<Two128>(); }

cudaError_t launch_paged_tc(const Dims &D, const Paged &G, const void *q, const void *k_pages, const void *v_pages,
                            const int32_t *sel, void *out, int min_rows, void *scratch, int *status, cudaStream_t st) {
  // Sequences whose rows fill no more than one tile leave the second one idle.
  if (D.d != kD || (long long)G.max_chunk * D.G <= kRows)
    return launch_paged_tc1(D, G, q, k_pages, v_pages, sel, out, min_rows, scratch, status, st);
  CUtensorMap tq;
  if (!encode_fn() || !make_map(&tq, q, kD, D.Hq, G.n_tok, D.G, kRows / D.G)) {
    note_error("paged attention tensor maps", cudaErrorInvalidValue);
    return cudaErrorInvalidValue;
  }
  auto kern = sel ? k_paged_tc<true> : k_paged_tc<false>;
  auto launch = [&](const TcParams &P, const CUtensorMap &tk, const CUtensorMap &tv, size_t smem) {
    const cudaError_t e = ensure_smem(kern, smem);
    return e == cudaSuccess ? launch_maybe_pdl(kern, dim3(P.C), dim3(kThreads), smem, st, false, tq, tk, tv, P) : e;
  };
  return launch_chunks<Two128>(launch, smem_of, D, G, q, k_pages, v_pages, sel, out, min_rows, scratch, status, st);
}

}  // namespace qsa
