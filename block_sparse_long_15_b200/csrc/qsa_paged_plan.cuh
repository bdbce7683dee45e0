// What the chunk attention kernels over a paged cache share: the division of the work, the
// warp that prepares it, and the merge of a unit's parts. A kernel's shape X has kD (head dim),
// kTiles (128-row MMA tiles per unit) and kChunk (keys per chunk).
//
// Units differ in length and there may be fewer of them than SMs, so the keys that the units
// see, laid end to end, are cut into C equal ranges, C = one per SM (fewer for little work),
// and CTA c takes range c: no CTA waits for another, and at most the first and the last unit of
// a range are shared with neighbours. A part of a unit leaves its unnormalised O with (m, l) per
// row in the workspace, two slots per CTA, and k_paged_merge, a row a lane, joins them in order.
#pragma once

#include <cuda.h>
#include <math.h>

#include <algorithm>

#include "qsa_internal.h"
#include "sm100_ptx.cuh"

namespace qsa {
namespace {

using namespace sm100;

constexpr int kRows = 128;  // MMA M: (token, head) rows per tile
constexpr int kHalf = 64;   // mask granularity: the smallest block size served
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kMaxSeqs = 512;   // sequences per launch: their geometry sits in shared memory
constexpr int kMaxCtas = 152;
// Keys that make a CTA's range worth having: small calls (3 chunks of 60 .. 256 of 256 .. 700 tokens at 64, 128 and 256
// dims) take 23, 36 and 45 us with 512, 18, 30 and 36 with 256, 17, 28 and 36 with 128, which costs 100 tokens
// of 1000 with 8 KV heads 17 us instead of 15.
constexpr int kMinKeys = 256;
constexpr int kBitWords = 2048;     // words of a segment's token bits
constexpr int kBitTileWords = 128;  // and of its tiles' bits
constexpr uint32_t kBitSlotBytes = (kBitWords + kBitTileWords) * 4;
constexpr uint32_t kInfoBytes = 64;

// A unit to be joined from the parts that CTAs c .. c_last left: the first in slot s0, the others
// in slots 2 p.
struct MergeJob {
  int c_last, s0;  // c_last < 0: none
  int q0, r0, n, g;
};

struct TcParams {
  Dims D;
  Paged P;
  const int32_t *sel;  // null: every visible token
  const __nv_bfloat16 *q;
  __nv_bfloat16 *out;
  float *part_o;       // [2 C][d / 4][rows of a unit][4] unnormalised O
  float *part_ml;      // [2 C][rows of a unit][2]: m (log2 domain), l
  MergeJob *jobs;  // [C] of the unit that begins in CTA c and goes on in others
  int *status;
  int T;               // tokens per tile
  float sl2;           // scale * log2(e)
  int C;               // CTAs
  int b0, nb;          // sequences of this launch
  int min_rows;        // sequences with fewer (token, head) rows are left to the row kernel
  int box;             // keys per TMA box: min(page size, chunk)
  int W;               // words a token's bits have in a segment
};

// ---------------------------------------------------------------- the key list
// The list of all units' visible keys: sequence by sequence, KV head by KV head, unit by unit.
// Unit u of a sequence with n new tokens of len sees w(u) = len - n + min(n, (u + 1) step) keys,
// step = tiles * T tokens. In shared memory: keys before each sequence, and the geometry.
struct SeqGeo {
  int q0, n, len;  // n = 0: nothing to do here
};
struct PlanArea {
  long long *pre;  // [nb + 1]
  SeqGeo *seq;     // [nb]
};
__host__ __device__ constexpr size_t plan_bytes(int nb) { return (size_t)(nb + 1) * 8 + (size_t)nb * sizeof(SeqGeo); }

// Divisions here have 64-bit operands that nearly always fit 32 bits, where they are much cheaper.
__device__ __forceinline__ long long div_pos(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// Keys of the units before u of one KV head (u = units: all of them).
template <class X>
__device__ __forceinline__ long long keys_before(const TcParams &P, const SeqGeo &q, int u) {
  const int step = X::kTiles * P.T;
  const long long k = (long long)u * (q.len - q.n) + (long long)step * u * (u + 1) / 2;
  return (long long)u * step > q.n ? k - ((long long)u * step - q.n) : k;  // the last unit may be short
}
template <class X>
__device__ __forceinline__ int units_of(const TcParams &P, const SeqGeo &q) {
  const int step = X::kTiles * P.T;
  return (q.n + step - 1) / step;
}

// Fills the plan. Every thread of the block calls it.
template <class X>
__device__ void make_plan(const TcParams &P, const PlanArea &L, int *status) {
  __shared__ long long s_sum[32];
  const int nt = blockDim.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (P.nb + nt - 1) / nt;
  const int a = min(P.nb, (int)threadIdx.x * per), z = min(P.nb, a + per);
  long long run = 0;
  for (int b = a; b < z; ++b) {
    const PagedSeq q = paged_seq(P.P, P.b0 + b, status);
    SeqGeo g = {q.q0, (long long)q.n * P.D.G < P.min_rows ? 0 : q.n, q.len};
    L.seq[b] = g;
    run += keys_before<X>(P, g, units_of<X>(P, g)) * P.D.Hkv;
    L.pre[b + 1] = run;
  }
  long long incl = run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_sum[warp] = incl;
  if (threadIdx.x == 0) L.pre[0] = 0;
  __syncthreads();
  long long before = incl - run;
  for (int w = 0; w < warp; ++w) before += s_sum[w];
  for (int b = a; b < z; ++b) L.pre[b + 1] += before;
  __syncthreads();
}
__device__ __forceinline__ int ctas_of(const TcParams &P, long long total) {
  return (int)min((long long)P.C, (total + kMinKeys - 1) / kMinKeys);
}

struct Unit {
  int b, g, u;
  long long first;  // its first key's place in the list
  int w;            // keys it sees
  SeqGeo s;
};
template <class X>
__device__ __forceinline__ Unit unit_at(const TcParams &P, const PlanArea &L, long long x) {
  Unit r;
  int lo = 0, hi = P.nb;  // pre[lo] <= x < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (L.pre[mid] <= x) lo = mid;
    else hi = mid;
  }
  r.b = lo;
  r.s = L.seq[lo];
  const long long per_head = div_pos(L.pre[lo + 1] - L.pre[lo], P.D.Hkv), in = x - L.pre[lo];
  r.g = (int)div_pos(in, per_head);
  const long long y = in - r.g * per_head;
  int ul = 0, uh = units_of<X>(P, r.s);
  while (uh - ul > 1) {
    const int mid = (ul + uh) >> 1;
    if (keys_before<X>(P, r.s, mid) <= y) ul = mid;
    else uh = mid;
  }
  r.u = ul;
  r.first = L.pre[lo] + r.g * per_head + keys_before<X>(P, r.s, ul);
  r.w = r.s.len - r.s.n + min(r.s.n, (ul + 1) * X::kTiles * P.T);
  return r;
}
// Where CTA c's range begins: c / C of the list, moved up to the next chunk of its unit (or to
// the unit's end).
template <class X>
__device__ __forceinline__ long long range_start(const TcParams &P, const PlanArea &L, long long total, int C, int c) {
  if (c >= C) return total;
  const long long x = div_pos((long long)c * total, C);
  const Unit r = unit_at<X>(P, L, x);
  const int y = ((int)(x - r.first) + X::kChunk - 1) / X::kChunk * X::kChunk;
  return r.first + min(y, r.w);
}
// The CTA whose range holds place x (a chunk's beginning): floor(c T / C) <= x < floor((c + 1) T / C).
__device__ __forceinline__ int cta_of(long long x, int C, long long total) {
  return (int)div_pos((x + 1) * C + total - 1, total) - 1;
}

// A segment as the builder hands it to the other warps.
struct UnitInfo {
  int live;  // 0: no segment left
  int b, g, q0, r0, n, len;
  int slot;  // partial slot, -1: the whole unit
  int ca, cb;     // chunks [ca, cb)
  int cend[2];    // without a selection tile w sees the chunks below cend[w]
  int part;       // bit 0: the first of the unit's segments here, bit 1: the last
};
static_assert(sizeof(UnitInfo) <= kInfoBytes, "unit info area");

// Where the builder works in shared memory: two slots of everything.
struct SlotArea {
  uint64_t *full, *free;  // barriers [slot]
  uint8_t *info;          // [slot] kInfoBytes
  uint8_t *bits;          // [slot] kBitSlotBytes: token bits, then tile bits; with a selection
  volatile int *abort_flag;
};

// The chunks of a segment: of the unit (the union of its tiles') and of each tile. With a
// selection bit H i + h of a bit list stands for 64 keys: part h of the H in chunk ca + i.
template <class X, bool kSel>
struct Chunks {
  static constexpr int H = X::kChunk / kHalf, kPer = 32 / H;  // chunks per word
  const uint32_t *bits;  // a tile's nw words after the other's
  int nw, ca, cend[2];
  __device__ __forceinline__ Chunks(const UnitInfo &I, const uint32_t *tile_bits, int W)
      : bits(tile_bits), nw(W), ca(I.ca), cend{I.cend[0], I.cend[1]} {}
  __device__ __forceinline__ uint32_t word(int w) const { return X::kTiles == 2 ? bits[w] | bits[nw + w] : bits[w]; }
  // Smallest chunk >= c of the unit, or -1.
  __device__ __forceinline__ int next(int c) const {
    if (!kSel) return c < (X::kTiles == 2 ? max(cend[0], cend[1]) : cend[0]) ? c : -1;
    int w = (c - ca) / kPer;
    if (w >= nw) return -1;
    uint32_t x = word(w) & (0xffffffffu << (H * ((c - ca) % kPer)));
    while (true) {
      if (x) return ca + w * kPer + (__ffs(x) - 1) / H;
      if (++w >= nw) return -1;
      x = word(w);
    }
  }
  __device__ __forceinline__ bool has(int w, int c) const {
    return kSel ? (bits[w * nw + (c - ca) / kPer] >> (H * ((c - ca) % kPer))) & ((1u << H) - 1u) : c < cend[w];
  }
};

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

// P for keys kFrom .. kTo - 1 of 32 held in registers (fp32 bits), written back in place over
// sv[kFrom / 2 ..] as bf16 pairs: p = 2^(s * scale - m) for keys below `lim`, 0 from there on. Adds
// them to acc (the fp32 values: only the product with V sees them in bf16, since both operands of an
// MMA have one type and V is bf16). Outputs are 2.3e-3 from the 64-bit form (2-norm), 1.7e-3 of it
// their own rounding to bf16; a second product with P's low half would take the MMAs of a chunk from two to three
// parts, where the tensor pipe is busy 60 % of the time already.
template <bool kAll, int kFrom = 0, int kTo = 32>
__device__ __forceinline__ void p_quarter(uint32_t (&sv)[32], int lim, uint64_t scale2, uint64_t negm2, uint64_t (&acc)[2]) {
#pragma unroll
  for (int u = kFrom; u < kTo; u += 2) {
    float p0, p1;
    f2_unpack(f2_fma(f2_pack(sv[u], sv[u + 1]), scale2, negm2), p0, p1);
    p0 = ex2_approx(p0);
    p1 = ex2_approx(p1);
    if (!kAll) {
      p0 = (u < lim) ? p0 : 0.f;
      p1 = (u + 1 < lim) ? p1 : 0.f;
    }
    sv[u >> 1] = pack_bf16x2(p0, p1);
    acc[(u >> 1) & 1] = f2_add(acc[(u >> 1) & 1], f2_pack(__float_as_uint(p0), __float_as_uint(p1)));
  }
}
__device__ __forceinline__ void zero_quarter(uint32_t (&sv)[32]) {
#pragma unroll
  for (int u = 0; u < 16; ++u) sv[u] = 0u;
}
// Max of the first `lim` of 32 fp32 values.
template <bool kAll>
__device__ __forceinline__ float max_quarter(const uint32_t (&sv)[32], int lim) {
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

// This thread's index, opaque to the compiler: what is derived from it is computed where it is
// used instead of being kept in registers across the softmax loop. (Shared memory leaves almost
// no L1, so a register that spills there costs a trip to L2 per chunk.)
__device__ __forceinline__ int fresh_tid() {
  int t;
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(t));
  return t;
}

// ---------------------------------------------------------------- builder
template <class X, bool kSel>
__device__ __forceinline__ void build_segments(const TcParams &P, const SlotArea &A, const PlanArea &L, int lane) {
  constexpr int H = X::kChunk / kHalf, kPer = 32 / H;  // bits per chunk, chunks per word
  const int T = P.T, k = P.D.k, B = P.D.B, W = P.W;
  const long long total = L.pre[P.nb];
  const int C = ctas_of(P, total), c = blockIdx.x;
  // lane 0 and lane 1 look for the two ends of the range
  const long long ends = c < C ? range_start<X>(P, L, total, C, c + (lane & 1)) : total;
  long long x = __shfl_sync(0xffffffffu, ends, 0);
  const long long lo = x, hi = __shfl_sync(0xffffffffu, ends, 1);
  MergeJob job = {-1, 0, 0, 0, 0, 0};
  int sub = -1;  // with a selection: first chunk of the unit's next segment; the bits of one have room for kPer W
  for (int su = 0;; ++su) {
    const int s = su & 1;
    if (su >= 2 && !idle_wait_warp(&A.free[s], ((su >> 1) - 1) & 1)) {
      if (lane == 0) record_status(P.status, QSA_ERR_TIMEOUT);
      *A.abort_flag = 1;
      break;
    }
    UnitInfo &I = *(UnitInfo *)(A.info + s * kInfoBytes);
    if (x >= hi || *A.abort_flag) {
      if (lane == 0) I.live = 0;
      __syncwarp();
      mbar_arrive(&A.full[s]);
      break;
    }
    const Unit r = unit_at<X>(P, L, x);
    const long long end = min(hi, r.first + r.w);
    const int c_lo = (int)((x - r.first) / X::kChunk), c_hi = (int)((end - r.first + X::kChunk - 1) / X::kChunk);
    const int ca = sub >= 0 ? sub : c_lo, cb = kSel ? min(c_hi, ca + kPer * W) : c_hi;
    const int r0 = r.u * X::kTiles * T, n = r.s.n, t0 = r.s.len - n;
    if (kSel) {
      uint32_t *bits = (uint32_t *)(A.bits + s * kBitSlotBytes), *tile_bits = bits + kBitWords;
      const int rows = min(X::kTiles * T, n - r0), h0 = H * ca, h1 = H * cb, per = B / kHalf;
      for (int i = lane; i < kBitWords + X::kTiles * W; i += 32) bits[i] = 0;
      __syncwarp();
      // Bits [a, z) of a token and of its tile, 4 at most (a block is 256 keys at most)
      auto set = [&](int tok, int a, int z) {
        a = max(a, h0), z = min(z, h1);
        if (a >= z) return;
        const uint64_t m = (uint64_t)((1u << (z - a)) - 1u) << ((a - h0) & 31);
        const int w = (a - h0) >> 5, tile = tok < T ? 0 : W;
        atomicOr(&bits[tok * W + w], (uint32_t)m);
        atomicOr(&tile_bits[tile + w], (uint32_t)m);
        if (m >> 32) {
          atomicOr(&bits[tok * W + w + 1], (uint32_t)(m >> 32));
          atomicOr(&tile_bits[tile + w + 1], (uint32_t)(m >> 32));
        }
      };
      // the lists, 32 entries of kLists tokens at a time, and the trailing ranges
      constexpr int kLists = 8;
      const int32_t *lists = P.sel + ((size_t)r.s.q0 + r0) * k;
      for (int tok = 0; tok < rows; tok += kLists)
        for (int i = lane; i < k; i += 32) {
          int j[kLists];
#pragma unroll
          for (int e = 0; e < kLists; ++e) j[e] = tok + e < rows ? lists[(tok + e) * k + i] : -1;
#pragma unroll
          for (int e = 0; e < kLists; ++e)
            if (j[e] >= 0 && j[e] < (t0 + r0 + tok + e + 1) / B) set(tok + e, j[e] * per, j[e] * per + per);
        }
      for (int tok = lane; tok < rows; tok += 32) {
        const int t = t0 + r0 + tok;
        set(tok, (t + 1) / B * per, t / kHalf + 1);
      }
      __syncwarp();
    }
    if (lane == 0) {
      I.b = P.b0 + r.b;
      I.g = r.g;
      I.q0 = r.s.q0;
      I.r0 = r0;
      I.n = n;
      I.len = r.s.len;
      I.slot = c_lo == 0 && end == r.first + r.w ? -1 : 2 * c + (x == lo ? 0 : 1);
      I.ca = ca;
      I.cb = cb;
      // every chunk up to the tile's last token
      I.cend[0] = min(cb, (t0 + min(n, r0 + T) - 1) / X::kChunk + 1);
      I.cend[1] = X::kTiles == 2 && r0 + T < n ? min(cb, (t0 + min(n, r0 + 2 * T) - 1) / X::kChunk + 1) : ca;
      I.part = (ca == c_lo ? 1 : 0) | (cb == c_hi ? 2 : 0);
      I.live = 1;
    }
    __syncwarp();
    mbar_arrive(&A.full[s]);
    if (c_lo == 0 && end < r.first + r.w)
      job = {cta_of(r.first + (r.w - 1) / X::kChunk * X::kChunk, C, total), 2 * c + (x == lo ? 0 : 1), r.s.q0, r0, n, r.g};
    if (cb == c_hi) x = end, sub = -1;
    else sub = cb;
  }
  if (lane == 0) P.jobs[c] = job;
}

// ---------------------------------------------------------------- parts of a unit
// A part's O lies by groups of four columns, the rows of the unit one after the other in each: a warp whose
// lanes hold rows (as TMEM hands them out) stores and loads it in runs. With the rows dense each of
// a warp's stores touched 32 lines, 4.7 us for the 256 rows of a block of k_paged_tc.
template <class X>
__device__ __forceinline__ size_t part_at(int slot, int row, int col) {
  return (((size_t)slot * (X::kD / 4) + col / 4) * (X::kTiles * kRows) + row) * 4;
}

// Block (c, y, z): rows 32 y .. of the unit that begins in CTA c's range and goes on in later ones, 128
// elements of each from 128 z on. A lane is a row, a warp 8 elements of it:
//   out = sum 2^(m_p - m) O_p / sum 2^(m_p - m) l_p.
// With cold caches 9 us behind drafted tokens of 16 sequences, 22 behind 148 long ranges (39 MB of parts).
constexpr int kMergeWarps = 16, kMergeRows = 32, kMergeParts = 8;
template <class X>
__global__ void __launch_bounds__(kMergeWarps * 32) k_paged_merge(const __grid_constant__ TcParams P) {
  pdl_trigger();  // the row kernel behind it, where there is one, needs nothing of this one
  pdl_wait();     // the parts come from the kernel before
  const int c = blockIdx.x;
  const MergeJob J = P.jobs[c];
  if (J.c_last < 0) return;
  const int rr = blockIdx.y * kMergeRows + (threadIdx.x & 31), row = rr % kRows;  // row of tile rr / 128
  const int col = blockIdx.z * 128 + (threadIdx.x >> 5) * 8;
  const int tok = J.r0 + rr / kRows * P.T + row / P.D.G;
  if (col >= X::kD || row / P.D.G >= P.T || tok >= J.n) return;
  auto slot = [&](int p) { return p == c ? J.s0 : 2 * p; };
  float m = -INFINITY, l = 0.f;
  float4 o0 = make_float4(0.f, 0.f, 0.f, 0.f), o1 = o0;
  for (int p0 = c; p0 <= J.c_last; p0 += kMergeParts) {  // the loads of eight parts at once
    float2 ml[kMergeParts];
    float4 x0[kMergeParts], x1[kMergeParts];
#pragma unroll
    for (int e = 0; e < kMergeParts; ++e) {
      ml[e] = make_float2(-INFINITY, 0.f);
      x0[e] = x1[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p0 + e <= J.c_last) {
        const int s = slot(p0 + e);
        ml[e] = *(const float2 *)(P.part_ml + ((size_t)s * (X::kTiles * kRows) + rr) * 2);
        x0[e] = *(const float4 *)(P.part_o + part_at<X>(s, rr, col));
        x1[e] = *(const float4 *)(P.part_o + part_at<X>(s, rr, col + 4));
      }
    }
    float mn = m;
#pragma unroll
    for (int e = 0; e < kMergeParts; ++e) mn = fmaxf(mn, ml[e].x);
    if (mn == -INFINITY) continue;  // none of these parts sees a key of the row
    const float fa = ex2_approx(m - mn);
    m = mn;
    l *= fa;
    o0.x *= fa, o0.y *= fa, o0.z *= fa, o0.w *= fa;
    o1.x *= fa, o1.y *= fa, o1.z *= fa, o1.w *= fa;
#pragma unroll
    for (int e = 0; e < kMergeParts; ++e) {
      if (ml[e].x == -INFINITY) continue;  // a part that sees nothing of the row left nothing
      const float f = ex2_approx(ml[e].x - mn);
      l = fmaf(f, ml[e].y, l);
      o0.x = fmaf(f, x0[e].x, o0.x);
      o0.y = fmaf(f, x0[e].y, o0.y);
      o0.z = fmaf(f, x0[e].z, o0.z);
      o0.w = fmaf(f, x0[e].w, o0.w);
      o1.x = fmaf(f, x1[e].x, o1.x);
      o1.y = fmaf(f, x1[e].y, o1.y);
      o1.z = fmaf(f, x1[e].z, o1.z);
      o1.w = fmaf(f, x1[e].w, o1.w);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  __nv_bfloat16 *dst = P.out + (((size_t)J.q0 + tok) * P.D.Hq + J.g * P.D.G + row % P.D.G) * X::kD + col;
  *(uint4 *)dst = make_uint4(pack_bf16x2(o0.x * inv, o0.y * inv), pack_bf16x2(o0.z * inv, o0.w * inv),
                             pack_bf16x2(o1.x * inv, o1.y * inv), pack_bf16x2(o1.z * inv, o1.w * inv));
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

// 3-D bf16 tensor map of dense rows of d elements, 128-byte swizzle, zero fill out of bounds.
bool make_map(CUtensorMap *m, const void *ptr, int d, uint64_t d1, uint64_t d2, uint32_t b1, uint32_t b2) {
  cuuint64_t dims[3] = {(cuuint64_t)d, d1, d2};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, d1 * d * 2};
  cuuint32_t box[3] = {64, b1, b2};
  cuuint32_t estr[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Fills P and calls launch(P, tk, tv, smem), then the merge, once per kMaxSeqs sequences; tk and
// tv are the tensor maps of the pools.
template <class X, typename Launch>
cudaError_t launch_chunks(Launch launch, size_t (*smem_of)(bool, int), const Dims &D, const Paged &G, const void *q,
                          const void *k_pages, const void *v_pages, const int32_t *sel, void *out, int min_rows,
                          void *scratch, int *status, cudaStream_t st) {
  if (!encode_fn()) {
    note_error("cuTensorMapEncodeTiled entry point", cudaErrorNotSupported);
    return cudaErrorNotSupported;
  }
  TcParams P;
  P.D = D;
  P.P = G;
  P.sel = sel;
  P.q = (const __nv_bfloat16 *)q;
  P.out = (__nv_bfloat16 *)out;
  P.part_o = (float *)scratch;
  P.part_ml = P.part_o + (size_t)2 * kMaxCtas * X::kTiles * kRows * X::kD;
  P.jobs = (MergeJob *)(P.part_ml + (size_t)2 * kMaxCtas * X::kTiles * kRows * 2);
  P.status = status;
  P.T = kRows / D.G;
  P.sl2 = D.scale * 1.4426950408889634f;
  P.C = std::min(sm_count(), kMaxCtas);
  P.min_rows = min_rows;
  P.box = std::min(G.ps, X::kChunk);
  P.W = std::min(kBitTileWords / X::kTiles, kBitWords / (X::kTiles * P.T));
  P.W -= 1 - P.W % 2;  // odd: the builder's lanes, a token each, hit different banks
  const uint64_t planes = (uint64_t)G.n_pages * D.Hkv;
  CUtensorMap tk, tv;
  if (!make_map(&tk, k_pages, X::kD, G.ps, planes, P.box, 1) || !make_map(&tv, v_pages, X::kD, G.ps, planes, P.box, 1)) {
    note_error("paged attention tensor maps", cudaErrorInvalidValue);
    return cudaErrorInvalidValue;
  }
  for (P.b0 = 0; P.b0 < G.batch; P.b0 += kMaxSeqs) {
    P.nb = std::min(kMaxSeqs, G.batch - P.b0);
    note_launch();
    cudaError_t e = launch(P, tk, tv, smem_of(sel != nullptr, P.nb));
    if (e == cudaSuccess) {
      note_launch();
      e = launch_maybe_pdl(k_paged_merge<X>, dim3(P.C, X::kTiles * kRows / kMergeRows, (X::kD + 127) / 128),
                           dim3(kMergeWarps * 32), 0, st, true, P);
    }
    if (e != cudaSuccess) {
      note_error("paged chunk attention launch", e);
      return e;
    }
  }
  return cudaSuccess;
}

template <class X>
size_t partials_bytes() {
  return (size_t)2 * kMaxCtas * X::kTiles * kRows * (X::kD + 2) * sizeof(float) + kMaxCtas * sizeof(MergeJob);
}

}  // namespace
}  // namespace qsa
