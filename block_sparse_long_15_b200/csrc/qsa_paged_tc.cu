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
// Schedule: units differ in length and there may be fewer of them than SMs, so the keys that
// the units see, laid end to end, are cut into C equal ranges, C = one per SM (fewer for
// little work), and CTA c takes range c: no CTA waits for another, and at most the first and
// the last unit of a range are shared with neighbours. A part of a unit leaves its
// unnormalised O with (m, l) per row in the workspace, two slots per CTA, and k_paged_merge,
// one row a warp, joins them in order. Inside a CTA the roles are pipelined across units:
//   warp 18     builder: the next unit's geometry, selection lists and chunk bitmaps;
//   warp 0      TMA producer: Q, then K of chunk j and V of chunk j - 1 into ring entry j;
//               its lanes hold the page numbers of the next chunk's boxes;
//   warp 1      MMA issuer (TMEM owner): per chunk O_A += P_A V, S_A = Q_A K'^T, then B;
//   warps 2-17  softmax, eight per tile, 16 rows per warp, two threads a row (16x32bx2 TMEM
//               accesses): row max, P in bf16 over the first half of each S half, O rescaled
//               only when the max has moved by more than 2^8, and the epilogue.
// Every wait is bounded; on expiry the kernel records QSA_ERR_TIMEOUT and unwinds.
#include <cuda.h>
#include <math.h>

#include <algorithm>

#include "qsa_internal.h"
#include "sm100_ptx.cuh"

namespace qsa {
namespace {

using namespace sm100;

constexpr int kD = 128;      // head dim served
constexpr int kRows = 128;   // MMA M: (token, head) rows per tile
constexpr int kTiles = 2;    // tiles per unit
constexpr int kChunk = 128;  // keys per chunk
constexpr int kHalf = 64;    // keys a softmax thread holds of a chunk; smallest block size served
constexpr int kNE = 2;       // ring depth: entry j holds K of chunk j and V of chunk j - 1
constexpr int kThreads = 608;
constexpr int kBuilderWarp = 18;
constexpr int kSoftWarps = 16;
constexpr uint32_t kTmemCols = 512;  // S of tile w at 128 w, O of tile w at 256 + 128 w
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kMaxSeqs = 1024;   // sequences per launch
constexpr int kMaxCtas = 152;
constexpr int kMinKeys = 512;    // keys of a unit that make a CTA's range worth having

constexpr uint32_t kQBytes = kRows * kD * 2;    // per tile, two 64-column halves
constexpr uint32_t kKVBytes = kChunk * kD * 2;  // per K (or V) chunk, two halves
constexpr uint32_t kEntryBytes = 2 * kKVBytes;
constexpr uint32_t kSelSlotBytes = 8192;        // a unit's selection lists, if they fit
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffE = kOffQ + kTiles * kQBytes;
constexpr uint32_t kOffBar = kOffE + kNE * kEntryBytes;
constexpr uint32_t kOffMisc = kOffBar + 256;
constexpr uint32_t kOffInfo = kOffMisc + 64;
constexpr uint32_t kInfoBytes = 64;
constexpr uint32_t kOffSel = kOffInfo + 2 * kInfoBytes;

// barrier slots
constexpr int kBarQ = 0;                        // Q of the unit landed
constexpr int kBarQEmpty = 1;                   // every QK of the unit completed
constexpr int kBarFull = 2;                     // [ring entry]
constexpr int kBarEmpty = kBarFull + kNE;       // [ring entry]
constexpr int kBarSFull = kBarEmpty + kNE;      // [tile]
constexpr int kBarPFull = kBarSFull + 2;        // [tile], 8 arrivals
constexpr int kBarPVDone = kBarPFull + 2;       // [tile]
constexpr int kBarSlotFull = kBarPVDone + 2;    // [slot], the builder's 32 lanes
constexpr int kBarSlotFree = kBarSlotFull + 2;  // [slot], producer + MMA warp + softmax warps
constexpr int kBarSel = kBarSlotFree + 2;       // the builder's bulk copy of a unit's lists
constexpr int kNumBars = kBarSel + 1;
static_assert(kNumBars * 8 <= 256, "barrier area");

struct TcParams {
  Dims D;
  Paged P;
  const int32_t *sel;  // null: every visible token
  __nv_bfloat16 *out;
  float *part_o;       // [2 C][kTiles * kRows][kD] unnormalised O
  float *part_ml;      // [2 C][kTiles * kRows][2]
  int *status;
  int T;               // tokens per tile
  int C;               // CTAs
  int b0, nb;          // sequences of this launch
  int min_rows;        // sequences with fewer (token, head) rows are left to the row kernel
  int box;             // keys per TMA box: min(page size, kChunk)
  int bitmap_words;    // capacity of a chunk bitmap
};

// ---------------------------------------------------------------- the key list
// The list of all units' visible keys: sequence by sequence, KV head by KV head, unit by unit.
// Unit u of a sequence with n new tokens of len sees w(u) = len - n + min(n, (u + 1) 2T) keys.
struct SeqPlan {
  PagedSeq s;
  int units;        // per KV head
  long long keys;   // per KV head
};
__device__ __forceinline__ SeqPlan seq_plan(const TcParams &P, int b, int *status) {
  SeqPlan q;
  q.s = paged_seq(P.P, P.b0 + b, status);
  if ((long long)q.s.n * P.D.G < P.min_rows) q.s.n = 0;
  const int step = kTiles * P.T;
  q.units = (q.s.n + step - 1) / step;
  q.keys = 0;
  if (q.units) {
    const long long u = q.units - 1;
    q.keys = u * (q.s.len - q.s.n) + (long long)P.T * u * (u + 1) + q.s.len;
  }
  return q;
}
// Keys of the units before u (u < units) of one KV head.
__device__ __forceinline__ long long keys_before(const TcParams &P, const SeqPlan &q, long long u) {
  return u * (q.s.len - q.s.n) + (long long)P.T * u * (u + 1);
}

// pre[b]: keys of the sequences before b, in shared memory. Every thread of the block calls it.
__device__ void make_plan(const TcParams &P, long long *pre, int *status) {
  __shared__ long long s_sum[32];
  const int nt = blockDim.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (P.nb + nt - 1) / nt;
  const int a = min(P.nb, (int)threadIdx.x * per), z = min(P.nb, a + per);
  long long run = 0;
  for (int b = a; b < z; ++b) {
    run += seq_plan(P, b, status).keys * P.D.Hkv;
    pre[b + 1] = run;
  }
  long long incl = run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_sum[warp] = incl;
  if (threadIdx.x == 0) pre[0] = 0;
  __syncthreads();
  long long before = incl - run;
  for (int w = 0; w < warp; ++w) before += s_sum[w];
  for (int b = a; b < z; ++b) pre[b + 1] += before;
  __syncthreads();
}
__device__ __forceinline__ int ctas_of(const TcParams &P, long long total) {
  return (int)min((long long)P.C, (total + kMinKeys - 1) / kMinKeys);
}

struct Unit {
  int b, g, u;
  long long first;  // its first key's place in the list
  int w;            // keys it sees
  SeqPlan q;
};
__device__ __forceinline__ Unit unit_at(const TcParams &P, const long long *pre, long long x) {
  Unit r;
  int lo = 0, hi = P.nb;  // pre[lo] <= x < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid;
    else hi = mid;
  }
  r.b = lo;
  r.q = seq_plan(P, lo, nullptr);
  const long long in = x - pre[lo];
  r.g = (int)(in / r.q.keys);
  const long long y = in - r.g * r.q.keys;
  int ul = 0, uh = r.q.units;
  while (uh - ul > 1) {
    const int mid = (ul + uh) >> 1;
    if (keys_before(P, r.q, mid) <= y) ul = mid;
    else uh = mid;
  }
  r.u = ul;
  r.first = pre[lo] + r.g * r.q.keys + keys_before(P, r.q, ul);
  r.w = r.q.s.len - r.q.s.n + min(r.q.s.n, (ul + 1) * kTiles * P.T);
  return r;
}
// Where CTA c's range begins: c / C of the list, moved up to the next chunk of its unit (or to
// the unit's end).
__device__ __forceinline__ long long range_start(const TcParams &P, const long long *pre, long long total, int C, int c) {
  if (c >= C) return total;
  const long long x = (long long)c * total / C;
  const Unit r = unit_at(P, pre, x);
  const long long y = (x - r.first + kChunk - 1) / kChunk * kChunk;
  return r.first + min(y, (long long)r.w);
}
// The CTA whose range holds place x (a chunk's beginning): floor(c T / C) <= x < floor((c + 1) T / C).
__device__ __forceinline__ int cta_of(long long x, int C, long long total) {
  return (int)(((x + 1) * C + total - 1) / total) - 1;
}

// A segment as the builder hands it to the other warps.
struct UnitInfo {
  int live;  // 0: no segment left
  int b, g, q0, r0, n, len;
  int slot;  // partial slot, -1: the whole unit
  int nwords;
};
static_assert(sizeof(UnitInfo) <= kInfoBytes, "unit info area");

// Smallest set bit >= c in (bm0 | bm1), or -1.
__device__ __forceinline__ int next_chunk(const uint32_t *bm0, const uint32_t *bm1, int nwords, int c) {
  int w = c >> 5;
  if (w >= nwords) return -1;
  uint32_t bits = (bm0[w] | bm1[w]) & (0xffffffffu << (c & 31));
  while (true) {
    if (bits) return (w << 5) + __ffs(bits) - 1;
    if (++w >= nwords) return -1;
    bits = bm0[w] | bm1[w];
  }
}
__device__ __forceinline__ bool bit_of(const uint32_t *bm, int c) { return (bm[c >> 5] >> (c & 31)) & 1u; }
// The bits of word w that lie in [lo, hi).
__device__ __forceinline__ uint32_t span_word(int w, int lo, int hi) {
  const int a = max(lo - 32 * w, 0), z = min(hi - 32 * w, 32);
  if (a >= z) return 0u;
  return (z == 32 ? 0xffffffffu : (1u << z) - 1u) & ~((1u << a) - 1u);
}

// A wait taken by a whole warp: the same answer on every lane.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, kWaitNs));
}
// A wait off the critical path that sleeps between polls.
__device__ __forceinline__ bool idle_wait_warp(uint64_t *bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  bool ok = true;
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > kWaitNs) {
      ok = false;
      break;
    }
    __nanosleep(128);
  }
  return __all_sync(0xffffffffu, ok);
}

// P for one 32-key quarter held in registers (fp32 bits), written back in place over
// sv[0 .. 15] as bf16 pairs: p = 2^(s * scale - m) for keys below `lim`, 0 from there on.
// Returns the quarter's sum (of the fp32 values: only the product with V sees them in bf16).
template <bool kAll>
__device__ __forceinline__ float p_quarter(uint32_t (&sv)[32], int lim, uint64_t scale2, uint64_t negm2) {
  uint64_t acc0 = 0, acc1 = 0;
#pragma unroll
  for (int u = 0; u < 32; u += 2) {
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(sv[u], sv[u + 1]), scale2, negm2), x0, x1);
    float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
    if (!kAll) {
      p0 = (u < lim) ? p0 : 0.f;
      p1 = (u + 1 < lim) ? p1 : 0.f;
    }
    sv[u >> 1] = pack_bf16x2(p0, p1);
    if ((u >> 1) & 1) acc1 = f2_add(acc1, f2_pack(__float_as_uint(p0), __float_as_uint(p1)));
    else acc0 = f2_add(acc0, f2_pack(__float_as_uint(p0), __float_as_uint(p1)));
  }
  float s0, s1;
  f2_unpack(f2_add(acc0, acc1), s0, s1);
  return s0 + s1;
}
// Max of the first `lim` of 32 fp32 values.
template <bool kAll>
__device__ __forceinline__ float max_quarter(const uint32_t *sv, int lim) {
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int u = 0; u < 32; u += 8)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int a = u + 2 * e;
      mx[e] = max3f(mx[e], (kAll || a < lim) ? __uint_as_float(sv[a]) : -INFINITY,
                    (kAll || a + 1 < lim) ? __uint_as_float(sv[a + 1]) : -INFINITY);
    }
  return max3f(mx[0], mx[1], fmaxf(mx[2], mx[3]));
}

// ---------------------------------------------------------------- builder
// Kept out of line: its registers do not add to the softmax loop's.
__device__ __noinline__ void build_segments(const TcParams &P, uint8_t *base, uint32_t *bitmaps, const long long *pre,
                                            int lane) {
  uint64_t *bars = (uint64_t *)(base + kOffBar);
  volatile int *abort_flag = (volatile int *)(base + kOffMisc + 8);
  const int T = P.T, k = P.D.k, B = P.D.B, bw = P.bitmap_words;
  const bool sel_cached = kTiles * T * k * 4 <= (int)kSelSlotBytes;
  const long long total = pre[P.nb];
  const int C = ctas_of(P, total), c = blockIdx.x;
  long long x = c < C ? range_start(P, pre, total, C, c) : total;
  const long long lo = x, hi = c < C ? range_start(P, pre, total, C, c + 1) : total;
  bool fail = false;
  int n_bulk = 0;
  for (int su = 0;; ++su) {
    const int s = su & 1;
    if (su >= 2 && !idle_wait_warp(&bars[kBarSlotFree + s], ((su >> 1) - 1) & 1)) {
      fail = true;
      break;
    }
    UnitInfo &I = *(UnitInfo *)(base + kOffInfo + s * kInfoBytes);
    if (x >= hi || *abort_flag) {
      if (lane == 0) I.live = 0;
      __syncwarp();
      mbar_arrive(&bars[kBarSlotFull + s]);
      break;
    }
    const Unit r = unit_at(P, pre, x);
    const long long end = min(hi, r.first + r.w);
    const int ca = (int)((x - r.first) / kChunk), cb = (int)((end - r.first + kChunk - 1) / kChunk);
    const int r0 = r.u * kTiles * T, n = r.q.s.n, t0 = r.q.s.len - n;
    uint32_t *bm0 = bitmaps + (s * kTiles) * bw, *bm1 = bm0 + bw;
    const int nwords = (cb + 31) >> 5;
    if (!P.sel) {
      // every chunk up to the tile's last token
      const int c0 = min(cb, (t0 + min(n, r0 + T) - 1) / kChunk + 1);
      const int c1 = r0 + T < n ? min(cb, (t0 + min(n, r0 + 2 * T) - 1) / kChunk + 1) : 0;
      for (int w = lane; w < nwords; w += 32) {
        bm0[w] = span_word(w, ca, c0);
        bm1[w] = span_word(w, ca, c1);
      }
    } else {
      int32_t *sel_s = (int32_t *)(base + kOffSel + s * kSelSlotBytes);
      for (int w = lane; w < nwords; w += 32) bm0[w] = bm1[w] = 0;
      __syncwarp();
      // The unit's lists are one contiguous range: one bulk copy when it is aligned and fits.
      const int rows = min(kTiles * T, n - r0);
      const int32_t *src = P.sel + ((size_t)r.q.s.q0 + r0) * k;
      const uint32_t bytes = (uint32_t)(rows * k * 4);
      const bool bulk = sel_cached && ((reinterpret_cast<uintptr_t>(src) | bytes) & 15) == 0;
      if (bulk) {
        if (lane == 0) {
          fence_proxy_async_smem();  // the slot's last readers were generic-proxy loads
          mbar_arrive_expect_tx(&bars[kBarSel], bytes);
          bulk_load(sel_s, src, bytes, &bars[kBarSel]);
        }
        const bool got = warp_wait(&bars[kBarSel], n_bulk & 1);
        ++n_bulk;
        if (!got) {
          fail = true;
          break;
        }
      } else if (sel_cached) {
        for (int e = lane; e < rows * k; e += 32) sel_s[e] = src[e];
        __syncwarp();
      }
      const int32_t *lists = sel_cached ? sel_s : src;
      for (int tok = lane; tok < rows; tok += 32) {
        const int t = t0 + r0 + tok, n_c = (t + 1) / B;
        uint32_t *bm = tok < T ? bm0 : bm1;
        uint32_t word = 0;  // the bits of one word are gathered and set at once
        int wi = -1;
        auto set = [&](int ch) {
          if (ch < ca || ch >= cb) return;
          if ((ch >> 5) != wi) {
            if (wi >= 0) atomicOr(&bm[wi], word);
            wi = ch >> 5;
            word = 0;
          }
          word |= 1u << (ch & 31);
        };
        for (int i = 0; i < k; ++i) {
          const int j = lists[tok * k + i];
          if (j < 0 || j >= n_c) continue;
          for (int ch = j * B / kChunk; ch <= (j * B + B - 1) / kChunk; ++ch) set(ch);
        }
        if (n_c * B <= t)
          for (int ch = n_c * B / kChunk; ch <= t / kChunk; ++ch) set(ch);
        if (wi >= 0) atomicOr(&bm[wi], word);
      }
    }
    __syncwarp();
    if (lane == 0) {
      I.b = P.b0 + r.b;
      I.g = r.g;
      I.q0 = r.q.s.q0;
      I.r0 = r0;
      I.n = n;
      I.len = r.q.s.len;
      I.slot = ca == 0 && end == r.first + r.w ? -1 : 2 * c + (x == lo ? 0 : 1);
      I.nwords = nwords;
      I.live = 1;
    }
    __syncwarp();
    mbar_arrive(&bars[kBarSlotFull + s]);
    x = end;
  }
  if (fail) {
    if (lane == 0) record_status(P.status, QSA_ERR_TIMEOUT);
    *abort_flag = 1;
  }
}

__global__ void __launch_bounds__(kThreads, 1)
k_paged_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
           const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TcParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t *bars = (uint64_t *)(base + kOffBar);
  uint32_t *tmem_slot = (uint32_t *)(base + kOffMisc);
  volatile int *abort_flag = (volatile int *)(base + kOffMisc + 8);
  long long *pre = (long long *)(base + kOffSel + (P.sel ? 2 * kSelSlotBytes : 0));
  uint32_t *bitmaps = (uint32_t *)(pre + P.nb + 1);  // [slot][tile][bitmap_words]

  const Dims &D = P.D;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = P.T, G = D.G, k = D.k, B = D.B, bw = P.bitmap_words;
  const bool sel_cached = kTiles * T * k * 4 <= (int)kSelSlotBytes;
  auto info = [&](int s) { return (const UnitInfo *)(base + kOffInfo + s * kInfoBytes); };
  auto bitmap = [&](int s, int w) { return bitmaps + (s * kTiles + w) * bw; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t count = 1;
      if (i == kBarPFull || i == kBarPFull + 1) count = 8;
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
  make_plan(P, pre, blockIdx.x == 0 ? P.status : nullptr);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  if (warp == kBuilderWarp) {
    build_segments(P, base, bitmaps, pre, lane);
  } else if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    // Lane i < 128 / box holds the pool plane (page, KV head) of the i-th box of the next chunk
    // (-1: no token there, or a page outside the pool; nothing is loaded), and issues that box.
    const int n_box = kChunk / P.box;
    const uint32_t box_bytes = (uint32_t)P.box * 128;  // 64 columns of a box
    int j = 0, qn = 0;
    bool fail = false;
    for (int su = 0; !fail; ++su) {
      const int s = su & 1;
      if (!idle_wait_warp(&bars[kBarSlotFull + s], (su >> 1) & 1)) {
        fail = true;
        break;
      }
      const UnitInfo I = *info(s);
      if (!I.live) break;
      const uint32_t *bm0 = bitmap(s, 0), *bm1 = bitmap(s, 1);
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
      int c = next_chunk(bm0, bm1, I.nwords, 0);
      if (c >= 0) {
        int z = plane(c), zp = -1, cp = -1;  // boxes of K chunk c and of V chunk cp
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
        ++qn;
        while (c >= 0 || cp >= 0) {
          const int cn = c >= 0 ? next_chunk(bm0, bm1, I.nwords, c + 1) : -1;
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
          if (__any_sync(0xffffffffu, *abort_flag != 0)) {
            fail = true;
            break;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kBarSlotFree + s]);
    }
    if (fail) {
      if (lane == 0) record_status(P.status, QSA_ERR_TIMEOUT);
      *abort_flag = 1;
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc_qk = idesc_bf16_f32(kRows, kChunk, false, false);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(kRows, kD, false, true);
    int j = 0, qn = 0;
    int n_pv0 = 0, n_pv1 = 0;  // PVs issued per tile
    bool fail = false;
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
      if (!warp_wait(&bars[kBarPFull + w], cnt & 1)) return false;
      tc_fence_after();
      const uint64_t vd = v_desc0 + (uint64_t)((se * kEntryBytes) >> 4);
      const uint32_t o = tbase + 256u + (uint32_t)(w * 128), pcol = tbase + (uint32_t)(w * 128);
#pragma unroll
      for (int kk = 0; kk < kChunk / 16; ++kk)
        mma_ts_w(o, pcol + (kk >> 2) * 64 + (kk & 3) * 8, vd + (uint64_t)((kk * 2048) >> 4), idesc_pv,
                 (!first || kk > 0) ? 1u : 0u);
      mma_commit_w(&bars[kBarPVDone + w]);
      return true;
    };
    for (int su = 0; !fail; ++su) {
      const int s = su & 1;
      if (!idle_wait_warp(&bars[kBarSlotFull + s], (su >> 1) & 1)) {
        fail = true;
        break;
      }
      const int live = info(s)->live, nwords = info(s)->nwords;
      const int t_hi = info(s)->len - info(s)->n + min(info(s)->n, info(s)->r0 + kTiles * T) - 1;
      if (!live) break;
      const uint32_t *bm0 = bitmap(s, 0), *bm1 = bitmap(s, 1);
      int c = next_chunk(bm0, bm1, nwords, 0);
      if (c >= 0) {
        bool first0 = true, first1 = true;
        if (!warp_wait(&bars[kBarQ], qn & 1)) fail = true;
        ++qn;
        tc_fence_after();
        if (!fail) {
          const int se = j % kNE;
          if (!warp_wait(&bars[kBarFull + se], (j / kNE) & 1)) fail = true;
          tc_fence_after();
          for (int w = 0; w < kTiles && !fail; ++w)
            if (bit_of(w ? bm1 : bm0, c)) issue_qk(w, se);
          if (!fail) mma_commit_w(&bars[kBarEmpty + se]);
          ++j;
        }
        int cn = fail ? -1 : next_chunk(bm0, bm1, nwords, c + 1);
        if (!fail && cn < 0) mma_commit_w(&bars[kBarQEmpty]);
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
            if (bit_of(w ? bm1 : bm0, c)) {
              if (!issue_pv(w, se, w ? first1 : first0)) {
                fail = true;
                break;
              }
              (w ? first1 : first0) = false;
            }
            if (cn >= 0 && bit_of(w ? bm1 : bm0, cn)) issue_qk(w, se);
          }
          if (fail) break;
          mma_commit_w(&bars[kBarEmpty + se]);
          ++j;
          const int cnn = cn >= 0 ? next_chunk(bm0, bm1, nwords, cn + 1) : -1;
          if (cn >= 0 && cnn < 0) mma_commit_w(&bars[kBarQEmpty]);
          c = cn;
          cn = cnn;
          if (__any_sync(0xffffffffu, *abort_flag != 0)) fail = true;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kBarSlotFree + s]);
    }
    if (fail && lane == 0) {
      record_status(P.status, QSA_ERR_TIMEOUT);
      *abort_flag = 1;
    }
  } else {
    // ---------------------------------------------------------------- softmax + epilogue
    const int sw = warp - 2;
    const int w = sw >> 3;          // tile
    const int sub = (sw >> 2) & 1;  // which 16 of the lane group's 32 rows
    const int lg = warp & 3;        // TMEM lane group
    const int hh = lane >> 4;       // this thread's 64-key half of every chunk, and 64 columns of O
    const int row = 32 * lg + 16 * sub + (lane & 15);
    const int tok = w * T + row / G, h = row % G;
    const bool in_tile = row / G < T;  // G need not divide 128
    const uint32_t lane_addr = tbase + ((uint32_t)(32 * lg + 16 * sub) << 16);
    const uint32_t s_col = lane_addr + (uint32_t)(w * 128);
    const uint32_t o_col = lane_addr + 256u + (uint32_t)(w * 128);
    const float sl2 = D.scale * 1.4426950408889634f;
    int n_all = 0;  // chunks of this tile over all segments so far: S, P and PV phases
    bool fail = false;
    for (int su = 0; !fail; ++su) {
      const int s = su & 1;
      if (!idle_wait_warp(&bars[kBarSlotFull + s], (su >> 1) & 1)) {
        fail = true;
        break;
      }
      const UnitInfo *I = info(s);
      if (!I->live) break;
      const uint32_t *bm0 = bitmap(s, 0), *bm1 = bitmap(s, 1);
      const uint32_t *bm = w ? bm1 : bm0;
      const int nwords = I->nwords;
      const int t_last = I->len - I->n + min(I->n, I->r0 + kTiles * T) - 1;  // the unit's last visible key
      const bool valid = in_tile && I->r0 + tok < I->n;
      const int t = I->len - I->n + I->r0 + tok;  // this row's position
      const int n_c = valid && P.sel ? (t + 1) / B : 0;
      const int32_t *srow = sel_cached ? (const int32_t *)(base + kOffSel + s * kSelSlotBytes) + tok * k
                                       : P.sel + ((size_t)I->q0 + (valid ? I->r0 + tok : 0)) * k;
      float m_ref = -INFINITY, l = 0.f;
      int ptr = 0, n = 0;
      for (int c = next_chunk(bm0, bm1, nwords, 0); c >= 0; c = next_chunk(bm0, bm1, nwords, c + 1)) {
        if (!bit_of(bm, c)) continue;
        int lim = 0;  // this thread's first `lim` keys are visible
        if (valid) {
          const int key0 = c * kChunk + hh * kHalf;
          const int jb = P.sel ? key0 / B : 0;
          if (jb < n_c) {
            while (ptr < k && (unsigned)srow[ptr] < (unsigned)jb) ++ptr;
            lim = (ptr < k && srow[ptr] == jb) ? kHalf : 0;
          } else {
            lim = min(max(t + 1 - key0, 0), kHalf);
          }
        }
        const bool z = __all_sync(0xffffffffu, lim == 0);
        // Keys are masked one by one only where a thread sees part of its half or the chunk
        // reaches past the last visible key (NaN may be there). Elsewhere a thread sees all
        // its keys or none; one that sees none takes +inf as its reference: p = 0.
        const bool part = __any_sync(0xffffffffu, lim > 0 && lim < kHalf) || c * kChunk + kChunk - 1 > t_last;
        if (!warp_wait(&bars[kBarSFull + w], n_all & 1)) {
          fail = true;
          break;
        }
        tc_fence_after();
        float hmax = -INFINITY;
        if (!z) {
          uint32_t sv0[32], sv1[32];
          tmem_ld32_split<64>(s_col, sv0);
          tmem_ld32_split<64>(s_col + 32, sv1);
          tmem_ld_wait();
          if (part) {
            hmax = fmaxf(max_quarter<false>(sv0, lim), max_quarter<false>(sv1, lim - 32));
          } else {
            const float mx = fmaxf(max_quarter<true>(sv0, 32), max_quarter<true>(sv1, 32));
            hmax = lim ? mx : -INFINITY;
          }
        }
        const float cmax = fmaxf(hmax, __shfl_xor_sync(0xffffffffu, hmax, 16)) * sl2;
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
        float psum = 0.f;
        if (z) {
          uint32_t zk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) zk[e] = 0u;
          tmem_st32_split<64>(s_col, zk);
        } else {
          const uint64_t scale2 = f2_splat(sl2);
          const uint64_t negm2 = f2_splat(part || lim ? -m_ref : -INFINITY);
          uint32_t sv0[32], sv1[32];
          tmem_ld32_split<64>(s_col, sv0);
          tmem_ld_wait();
          psum = part ? p_quarter<false>(sv0, lim, scale2, negm2) : p_quarter<true>(sv0, 32, scale2, negm2);
          tmem_ld32_split<64>(s_col + 32, sv1);
          tmem_ld_wait();
          psum += part ? p_quarter<false>(sv1, lim - 32, scale2, negm2) : p_quarter<true>(sv1, 32, scale2, negm2);
          tmem_st32_split_lo<64>(s_col, sv0, sv1);
        }
        if (__any_sync(0xffffffffu, rescale)) {
          // O is stable once this tile's previous PV has completed, and the next one waits for
          // this warp's arrival below
          if (n >= 1 && !warp_wait(&bars[kBarPVDone + w], (n_all - 1) & 1)) {
            fail = true;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int cb = 0; cb < 2; ++cb) {
            uint32_t ov[32];
            tmem_ld32_split<64>(o_col + cb * 32, ov);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 32; ++q) ov[q] = __float_as_uint(__uint_as_float(ov[q]) * alpha);
            tmem_st32_split<64>(o_col + cb * 32, ov);
          }
          l *= alpha;
        }
        l += psum;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kBarPFull + w]);
        ++n;
        ++n_all;
        if (__any_sync(0xffffffffu, *abort_flag != 0)) {
          fail = true;
          break;
        }
      }
      const float lt = l + __shfl_xor_sync(0xffffffffu, l, 16);  // the row's sum over both halves
      // -------------------------------------------------------------- epilogue
      // The segment's last PV of the tile is phase n_all - 1: the one before it completed
      // before S of the last chunk did, and the next one needs this warp's next P.
      bool have_o = false;
      if (n > 0 && !fail) {
        have_o = warp_wait(&bars[kBarPVDone + w], (n_all - 1) & 1);
        if (!have_o) fail = true;
      }
      if (fail) {
        if (lane == 0) record_status(P.status, QSA_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      tc_fence_after();
      const bool keep = lt > 0.f;  // a row that sees nothing is written as zeros
      const int slot = I->slot;
      if (slot < 0) {
        const float inv = keep ? 1.f / lt : 0.f;
        __nv_bfloat16 *orow =
            P.out + (((size_t)I->q0 + (valid ? I->r0 + tok : 0)) * D.Hq + I->g * G + h) * kD + hh * 64;
#pragma unroll 1
        for (int cb = 0; cb < 4; ++cb) {
          uint32_t ov[16];
          if (have_o) {
            tmem_ld16_split<64>(o_col + cb * 16, ov);
            tmem_ld_wait();
          }
          uint32_t pk[8];
#pragma unroll
          for (int q = 0; q < 8; ++q)
            pk[q] = keep && have_o
                        ? pack_bf16x2(__uint_as_float(ov[2 * q]) * inv, __uint_as_float(ov[2 * q + 1]) * inv)
                        : 0u;
          if (valid) {
            uint4 *o4 = (uint4 *)(orow + cb * 16);
            o4[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            o4[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
          }
        }
      } else {
        const size_t pr = (size_t)slot * (kTiles * kRows) + w * kRows + row;
        if (valid && hh == 0)
          *(float2 *)(P.part_ml + pr * 2) = make_float2(have_o && keep ? m_ref : -INFINITY, keep ? lt : 0.f);
        if (have_o) {
#pragma unroll 1
          for (int cb = 0; cb < 4; ++cb) {
            uint32_t ov[16];
            tmem_ld16_split<64>(o_col + cb * 16, ov);
            tmem_ld_wait();
            if (valid) {
              uint4 *o4 = (uint4 *)(P.part_o + pr * kD + hh * 64 + cb * 16);
#pragma unroll
              for (int q = 0; q < 4; ++q) o4[q] = make_uint4(ov[4 * q], ov[4 * q + 1], ov[4 * q + 2], ov[4 * q + 3]);
            }
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

// ---------------------------------------------------------------- parts of a unit
// Block (c, y): if the last unit of CTA c's range begins there and goes on in later ranges, its
// rows 16 y .. 16 y + 15, one a warp at a time: out = sum 2^(m_p - m) O_p / sum 2^(m_p - m) l_p.
constexpr int kMergeWarps = 8, kMergeRows = 16;
__global__ void __launch_bounds__(kMergeWarps * 32) k_paged_merge(const __grid_constant__ TcParams P) {
  extern __shared__ long long s_pre[];
  make_plan(P, s_pre, nullptr);
  pdl_wait();  // the parts come from the kernel before
  const long long total = s_pre[P.nb];
  const int C = ctas_of(P, total), c = blockIdx.x;
  if (c + 1 >= C) return;
  const long long cut = range_start(P, s_pre, total, C, c + 1);
  if (cut >= total) return;
  const Unit r = unit_at(P, s_pre, cut);
  if (cut == r.first || cta_of(r.first, C, total) != c) return;
  const int c_last = cta_of(r.first + (r.w - 1) / kChunk * kChunk, C, total);
  const int s0 = 2 * c + (range_start(P, s_pre, total, C, c) == r.first ? 0 : 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = warp; e < kMergeRows; e += kMergeWarps) {
    const int rr = blockIdx.y * kMergeRows + e;  // tile rr / 128
    const int row = rr % kRows;
    const int tok = r.u * kTiles * P.T + rr / kRows * P.T + row / P.D.G;
    if (row / P.D.G >= P.T || tok >= r.q.s.n) continue;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = c; p <= c_last; ++p) {
      const size_t at = (size_t)(p == c ? s0 : 2 * p) * (kTiles * kRows) + rr;
      const float2 ml = *(const float2 *)(P.part_ml + at * 2);
      if (ml.x == -INFINITY) continue;  // the part sees nothing of the row
      const float4 x = *(const float4 *)(P.part_o + at * kD + lane * 4);
      const float mn = fmaxf(m, ml.x);
      const float fa = ex2_approx(m - mn), fb = ex2_approx(ml.x - mn);
      o.x = fmaf(fb, x.x, o.x * fa);
      o.y = fmaf(fb, x.y, o.y * fa);
      o.z = fmaf(fb, x.z, o.z * fa);
      o.w = fmaf(fb, x.w, o.w * fa);
      l = fmaf(fb, ml.y, l * fa);
      m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    __nv_bfloat16 *dst = P.out + (((size_t)r.q.s.q0 + tok) * P.D.Hq + r.g * P.D.G + row % P.D.G) * kD + lane * 4;
    *(uint2 *)dst = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  }
}

// ---------------------------------------------------------------- host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = (EncodeTiledFn)p;
  }
  return fn;
}

int sm_count() {
  static int n[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (!n[dev] && cudaDeviceGetAttribute(&n[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) n[dev] = 148;
  return n[dev];
}

// 3-D bf16 tensor map of dense rows of kD elements, 128-byte swizzle, zero fill out of bounds.
bool make_map(CUtensorMap *m, const void *ptr, uint64_t d1, uint64_t d2, uint32_t b1, uint32_t b2) {
  cuuint64_t dims[3] = {(cuuint64_t)kD, d1, d2};
  cuuint64_t strides[2] = {(cuuint64_t)kD * 2, d1 * kD * 2};
  cuuint32_t box[3] = {64, b1, b2};
  cuuint32_t estr[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kSmemMax = 227 * 1024;
int bitmap_words_of(const Paged &G) {
  const long long chunks = (((long long)G.max_pages << G.ps_shift) + kChunk - 1) / kChunk;
  return (int)((chunks + 31) / 32);
}
size_t smem_of(const Paged &G, bool sel, int nb) {
  return 1024 + kOffSel + (sel ? 2 * kSelSlotBytes : 0) + (size_t)(nb + 1) * 8 + (size_t)2 * kTiles * bitmap_words_of(G) * 4;
}

}  // namespace

// bf16, head_dim 128, blocks of whole 64-key halves; a cache whose chunk bitmaps fit shared memory.
bool paged_tc_supported(const Dims &D, const Paged &G, bool sel) {
  return D.bf16 && D.d == kD && D.G <= 32 && (!sel || D.B % kHalf == 0) &&
         (long long)G.n_pages * D.Hkv <= 0x7fffffffLL &&
         smem_of(G, sel, std::min(G.batch, kMaxSeqs)) <= kSmemMax;
}

size_t paged_tc_workspace() { return (size_t)2 * kMaxCtas * kTiles * kRows * (kD + 2) * sizeof(float); }

cudaError_t launch_paged_tc(const Dims &D, const Paged &G, const void *q, const void *k_pages, const void *v_pages,
                            const int32_t *sel, void *out, int min_rows, void *scratch, int *status, cudaStream_t st) {
  if (!encode_fn()) {
    note_error("cuTensorMapEncodeTiled entry point", cudaErrorNotSupported);
    return cudaErrorNotSupported;
  }
  TcParams P;
  P.D = D;
  P.P = G;
  P.sel = sel;
  P.out = (__nv_bfloat16 *)out;
  P.part_o = (float *)scratch;
  P.part_ml = P.part_o + (size_t)2 * kMaxCtas * kTiles * kRows * kD;
  P.status = status;
  P.T = kRows / D.G;
  P.C = std::min(sm_count(), kMaxCtas);
  P.min_rows = min_rows;
  P.box = std::min(G.ps, kChunk);
  P.bitmap_words = bitmap_words_of(G);
  CUtensorMap tq, tk, tv;
  const uint64_t planes = (uint64_t)G.n_pages * D.Hkv;
  if (!make_map(&tq, q, D.Hq, G.n_tok, D.G, P.T) || !make_map(&tk, k_pages, G.ps, planes, P.box, 1) ||
      !make_map(&tv, v_pages, G.ps, planes, P.box, 1)) {
    note_error("paged attention tensor maps", cudaErrorInvalidValue);
    return cudaErrorInvalidValue;
  }
  for (P.b0 = 0; P.b0 < G.batch; P.b0 += kMaxSeqs) {
    P.nb = std::min(kMaxSeqs, G.batch - P.b0);
    const size_t smem = smem_of(G, sel != nullptr, P.nb);
    cudaError_t e = ensure_smem(k_paged_tc, smem);
    if (e == cudaSuccess) {
      note_launch();
      e = launch_maybe_pdl(k_paged_tc, dim3(P.C), dim3(kThreads), smem, st, false, tq, tk, tv, P);
    }
    if (e == cudaSuccess) {
      note_launch();
      e = launch_maybe_pdl(k_paged_merge, dim3(P.C, kTiles * kRows / kMergeRows), dim3(kMergeWarps * 32),
                           (size_t)(P.nb + 1) * 8, st, true, P);
    }
    if (e != cudaSuccess) {
      note_error("paged chunk attention launch", e);
      return e;
    }
  }
  return cudaSuccess;
}

}  // namespace qsa
