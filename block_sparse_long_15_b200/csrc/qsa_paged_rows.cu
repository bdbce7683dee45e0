// Attention of few query rows per sequence over a paged K/V cache (decode steps, drafted
// tokens), over every visible token or over the selected blocks and the trailing range:
//   out = softmax(scale q K^T) V
// for the (token, query head) rows that share a KV head. Also the path of every shape that
// the tensor-core chunk kernels do not serve.
//
// Each K and V row is read once per unit of R rows and used for 4 R d operations, so a
// decode step is bound by HBM: the design keeps loads in flight and everything else off
// their way.
//
// Work: a unit is one KV head of one sequence and up to R = 8 or 16 rows (of consecutive
// tokens; with a selection, of one token, whose list they share). Its keys are cut into
// 16-key tiles, which never cross a page. The tiles of all units, in order, form one list
// of T items, and each of C CTAs (as many as the device holds at once) takes the
// contiguous range [c T / C, (c + 1) T / C): every CTA streams the same number of bytes
// whatever the lengths, and at most its first and its last unit are shared with other
// CTAs. Those leave fp32 partials (m, l, O) in the workspace, two slots per CTA, and the
// last CTA of a unit to finish merges them in order (a counter per unit, set back to zero),
// so the result does not depend on which CTA was last.
//
// Inside a CTA every warp streams its own share (tiles w, w + 4, ... of the range) through
// its own ring with cp.async, across unit boundaries, with no barrier but at the end of a
// unit. A tile is multiplied with warp-level MMAs m16n8k16 in the transposed form
// S^T = K Q^T (16 keys x 8 rows) and O^T += V^T P^T (16 dims x 8 rows): with keys and dims
// in the 16-row operand, the 8 heads of a group fill the 8 columns, where S = Q K^T would
// leave half of the rows empty. P^T turns from accumulator to operand layout with one
// movmatrix per 8 x 8.
//
// Measured, 16 / 2 heads of 128, pages of 64: 64 sequences of 4K .. 32K tokens (1.24 GB) 199 us, 6.2 TB/s;
// over 32 selected blocks each (137 MB) 32 us in a graph, of which the chain of length, list entry, page
// number and first tile takes 6 and the merge of units that CTAs share 2 to 6; one sequence of
// 1500 tokens 11 us, latency throughout.
#include <math.h>

#include <algorithm>

#include "qsa_internal.h"
#include "sm100_ptx.cuh"

namespace qsa {
namespace {

using namespace sm100;

constexpr int kTile = 16;    // keys per tile
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxSeqs = 512;   // sequences per launch (their geometry sits in shared memory)
constexpr int kMaxCtas = 1024;
constexpr int kMaxRows = 16;

struct RowsParams {
  int Hq, Hkv, G, d, B, k;
  float sl2;  // scale * log2(e)
  Paged P;
  const void *q, *kp, *vp;
  const int32_t *sel;
  void *out;
  int *done;      // [C] parts finished of the unit that starts in CTA c; zero between calls
  float *part_o;  // [2 C][R][d]
  float *part_ml; // [2 C][R][2]: m (log2 domain), l
  int *status;
  int R;          // rows per unit
  int C;          // CTAs
  int min_items;  // items that make a CTA worth having
  int tpb;        // tiles per selected block
  int rtk;        // units per token and KV head with a selection: ceil(G / R)
  int b0, nb;     // the sequences of this launch
  long long max_rows;  // sequences with as many (token, head) rows are left out
};

// ---------------------------------------------------------------- the list of items
struct SeqItems {
  int q0, n, len;  // n = 0: nothing to do here
  int rt, tiles;   // units per KV head, tiles per unit
};
struct Plan {
  long long *pre;   // [nb + 1] items before sequence b
  SeqItems *seq;    // [nb]
  long long T;
  int C;            // CTAs that take part
};
__host__ __device__ constexpr size_t plan_bytes(int nb) { return (size_t)(nb + 1) * 8 + (size_t)nb * sizeof(SeqItems); }

// Divisions here have 64-bit operands that nearly always fit 32 bits, where they are much cheaper.
__device__ __forceinline__ long long div_pos(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// Every CTA for itself: items per sequence and their prefix sums.
__device__ void make_plan(const RowsParams &P, uint8_t *smem, Plan &L) {
  __shared__ long long s_sum[kWarps];
  __shared__ int s_max[kWarps];
  L.pre = (long long *)smem;
  L.seq = (SeqItems *)(smem + (size_t)(P.nb + 1) * 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (P.nb + kThreads - 1) / kThreads;
  const int a = min(P.nb, (int)threadIdx.x * per), z = min(P.nb, a + per);
  long long run = 0;
  int most = 0;  // tiles of a unit
  for (int b = a; b < z; ++b) {
    PagedSeq s = paged_seq(P.P, P.b0 + b, P.status);
    if ((long long)s.n * P.G >= P.max_rows) s.n = 0;
    int rt, tiles;
    if (P.sel) {
      rt = s.n * P.rtk;
      // an upper bound for every row of the sequence: its blocks and a trailing range
      tiles = min(s.len / P.B, P.k) * P.tpb + (min(s.len, P.B - 1) + kTile - 1) / kTile;
      if (tiles == 0) tiles = 1;
    } else {
      rt = (int)div_pos((long long)s.n * P.G + P.R - 1, P.R);
      tiles = (s.len + kTile - 1) / kTile;
    }
    L.seq[b] = {s.q0, s.n, s.len, rt, tiles};
    if (rt > 0) most = max(most, tiles);
    run += (long long)rt * tiles * P.Hkv;
    L.pre[b + 1] = run;
  }
  long long incl = run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_sum[warp] = incl;
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) s_max[warp] = most;
  if (threadIdx.x == 0) L.pre[0] = 0;
  __syncthreads();
  long long before = incl - run;
  for (int w = 0; w < warp; ++w) before += s_sum[w];
  for (int w = 0; w < kWarps; ++w) most = max(most, s_max[w]);
  for (int b = a; b < z; ++b) L.pre[b + 1] += before;
  __syncthreads();
  L.T = L.pre[P.nb];
  // A CTA should have as many items as make it worth having, and where few units are long, more: with n tiles
  // in a unit and i of them a CTA, streaming takes about i / 8 us and the merge of its n / i parts, which its
  // last CTA makes alone, n / 10 i. The rule goes by the longest unit of the batch and not by how many there are.
  // One sequence of 16000, 16 / 2 heads of 128, in a graph: 18.5 us, 32 with 8 items a CTA; two tokens of it 27 and
  // 58; of 8 KV heads, which fill the device without it, 20 and 17.
  const int items = max(P.min_items, (int)sqrtf(0.8f * (float)most));
  L.C = (int)min((long long)P.C, div_pos(L.T + items - 1, items));
}

// CTA of item i: floor(c T / C) <= i < floor((c + 1) T / C)
__device__ __forceinline__ int cta_of(long long i, int C, long long T) { return (int)div_pos((i + 1) * C + T - 1, T) - 1; }

// A unit: its sequence, KV head and rows, and where its items are in the list.
struct Unit {
  int b, g, r;           // sequence of the launch, KV head, unit of the sequence and head
  long long first, end;  // items
  SeqItems s;
};

__device__ __forceinline__ Unit unit_of(const RowsParams &P, const Plan &L, long long i) {
  int lo = 0, hi = P.nb;  // pre[lo] <= i < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (L.pre[mid] <= i) lo = mid;
    else hi = mid;
  }
  Unit u;
  u.b = lo;
  u.s = L.seq[lo];
  const int n = (int)div_pos(i - L.pre[lo], u.s.tiles);
  u.g = n / u.s.rt;
  u.r = n % u.s.rt;
  u.first = L.pre[lo] + (long long)n * u.s.tiles;
  u.end = u.first + u.s.tiles;
  return u;
}

// Row r of the unit: its packed token row and query head in the group; false behind the last.
__device__ __forceinline__ bool unit_row(const RowsParams &P, const Unit &u, int r, int &tok, int &h) {
  if (P.sel) {
    tok = u.r / P.rtk;
    h = (u.r % P.rtk) * P.R + r;
    return r < P.R && h < P.G;
  }
  const long long rr = (long long)u.r * P.R + r;
  tok = (int)(rr / P.G);
  h = (int)(rr - (long long)tok * P.G);
  return r < P.R && tok < u.s.n;
}

// Keys of tile j of the unit: key0 .. key0 + nv - 1 (nv = 0: nothing to see).
__device__ __forceinline__ void tile_keys(const RowsParams &P, const Unit &u, int j, int &key0, int &nv) {
  if (P.sel) {
    const int tok = u.r / P.rtk, t = u.s.len - u.s.n + tok;
    const int n_c = (t + 1) / P.B, n_sel = min(n_c, P.k);
    const int i = j / P.tpb, off = (j - i * P.tpb) * kTile;
    if (i < n_sel) {
      const int blk = P.sel[(size_t)(u.s.q0 + tok) * P.k + i];
      const bool in = blk >= 0 && blk < n_c;
      key0 = in ? blk * P.B + off : 0;
      nv = in ? min(kTile, P.B - off) : 0;
    } else {
      key0 = n_c * P.B + (j - n_sel * P.tpb) * kTile;
      nv = max(0, min(kTile, t + 1 - key0));
    }
  } else {
    const int tok = min((long long)u.s.n - 1, ((long long)u.r * P.R + P.R - 1) / P.G);
    key0 = j * kTile;
    nv = max(0, min(kTile, u.s.len - u.s.n + tok + 1 - key0));
  }
  if (nv == 0) key0 = 0;
}

// Element row of a key in the pools ([page][Hkv][slot]), or -1 for a page outside the pool.
__device__ __forceinline__ long long key_row(const RowsParams &P, const Unit &u, int key) {
  const int page = P.P.table[(size_t)(P.b0 + u.b) * P.P.max_pages + (key >> P.P.ps_shift)];
  if (page < 0 || page >= P.P.n_pages) {
    record_status(P.status, QSA_ERR_DEVICE_CHECK);
    return -1;
  }
  return ((((long long)page * P.Hkv + u.g) << P.P.ps_shift) | (key & (P.P.ps - 1)));
}

// ---------------------------------------------------------------- the end of a segment
// Column of element c of row r in a buffer of R rows: 8-element groups move with the row,
// so that the lanes of an accumulator fragment (4 row pairs x 8 columns) hit 32 banks.
__device__ __forceinline__ int swz(int r, int c) { return c ^ (((r >> 1) & 3) << 3); }

template <typename T>
__device__ __forceinline__ void store4(T *p, float4 v);
template <>
__device__ __forceinline__ void store4<float>(float *p, float4 v) { *(float4 *)p = v; }
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16 *p, float4 v) {
  *(uint2 *)p = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

__device__ __forceinline__ float weight_of(float m, float m_max) { return m == -INFINITY ? 0.f : ex2_approx(m - m_max); }

// The CTA's items [i0, i1) of unit u are done: the warps' buffers buf[w] ([R][d] fp32, swizzled or not)
// with their wm / wl hold them. A whole unit is written out; a part goes to the CTA's slot. Ends
// with a barrier.
template <typename T, bool kSwz>
__device__ __forceinline__ void finish_segment(const RowsParams &P, const Plan &L, const Unit &u, long long i0, long long i1,
                                               long long lo, float *const (&buf)[kWarps], const float *wm, const float *wl) {
  const int d = P.d, R = P.R, d4 = d >> 2;
  const int c = blockIdx.x;
  const bool whole = i0 == u.first && i1 == u.end;
  const int slot = 2 * c + (i0 == lo ? 0 : 1);
  __syncthreads();  // the buffers are written
  for (int e = threadIdx.x; e < R * d4; e += kThreads) {
    const int r = e / d4, c4 = (e - r * d4) * 4;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, wm[w * kMaxRows + r]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = weight_of(wm[w * kMaxRows + r], m);
      const float4 x = *(const float4 *)(buf[w] + r * d + (kSwz ? swz(r, c4) : c4));
      o.x = fmaf(f, x.x, o.x);
      o.y = fmaf(f, x.y, o.y);
      o.z = fmaf(f, x.z, o.z);
      o.w = fmaf(f, x.w, o.w);
      l = fmaf(f, wl[w * kMaxRows + r], l);
    }
    if (whole) {
      int tok, h;
      if (unit_row(P, u, r, tok, h)) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const bool any = l > 0.f;  // a row that sees nothing is written as zeros
        store4((T *)P.out + ((size_t)(u.s.q0 + tok) * P.Hq + u.g * P.G + h) * d + c4,
               make_float4(any ? o.x * inv : 0.f, any ? o.y * inv : 0.f, any ? o.z * inv : 0.f, any ? o.w * inv : 0.f));
      }
    } else {
      *(float4 *)(P.part_o + ((size_t)slot * R + r) * d + c4) = o;
      if (c4 == 0) *(float2 *)(P.part_ml + ((size_t)slot * R + r) * 2) = make_float2(m, l);
    }
  }
  __syncthreads();  // the buffers are free; a part is written
}

// The CTA's part of unit u, if it is one, is counted, and where the count is complete the unit is
// merged. At once, not after the CTA's last segment, where it costs 1.5 us more (35.2 against 33.7 at
// the 64-sequence step over selected blocks): the other CTA of the SM covers it here.
template <typename T>
__device__ __forceinline__ void settle(const RowsParams &P, const Plan &L, const Unit &u, long long i0, long long i1) {
  constexpr int kAtOnce = 8;  // parts whose loads go out together: 12.4 -> 11.0 us for the sequence of 1500, of 4
  __shared__ int s_last;
  if (i0 == u.first && i1 == u.end) return;
  const int d = P.d, R = P.R, d4 = d >> 2;
  const int c_first = cta_of(u.first, L.C, L.T), n_parts = cta_of(u.end - 1, L.C, L.T) - c_first + 1;
  if (threadIdx.x == 0) {
    // the barrier before orders the CTA's partial before this release; the last part acquires them all
    int old;
    asm volatile("atom.add.acq_rel.gpu.s32 %0, [%1], 1;" : "=r"(old) : "l"(&P.done[c_first]) : "memory");
    s_last = old == n_parts - 1;
  }
  __syncthreads();
  if (s_last) {
    const int s0 = 2 * c_first + (div_pos((long long)c_first * L.T, L.C) == u.first ? 0 : 1);
    for (int e = threadIdx.x; e < R * d4; e += kThreads) {
      const int r = e / d4, c4 = (e - r * d4) * 4;
      int tok, h;
      if (!unit_row(P, u, r, tok, h)) continue;
      float m = -INFINITY, l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int p0 = 0; p0 < n_parts; p0 += kAtOnce) {
        float2 ml[kAtOnce];
        float4 x[kAtOnce];
        float mn = m;
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) {
          const int p = p0 + q;
          const size_t at = (size_t)(p == 0 ? s0 : 2 * (c_first + p)) * R + r;
          ml[q] = p < n_parts ? __ldcg((const float2 *)(P.part_ml + at * 2)) : make_float2(-INFINITY, 0.f);
          x[q] = p < n_parts ? __ldcg((const float4 *)(P.part_o + at * d + c4)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) mn = fmaxf(mn, ml[q].x);
        const float fa = weight_of(m, mn);
        o.x *= fa, o.y *= fa, o.z *= fa, o.w *= fa;
        l *= fa;
        m = mn;
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) {
          const float f = weight_of(ml[q].x, mn);
          o.x = fmaf(f, x[q].x, o.x);
          o.y = fmaf(f, x[q].y, o.y);
          o.z = fmaf(f, x[q].z, o.z);
          o.w = fmaf(f, x[q].w, o.w);
          l = fmaf(f, ml[q].y, l);
        }
      }
      const bool any = l > 0.f;
      const float inv = any ? 1.f / l : 0.f;
      store4((T *)P.out + ((size_t)(u.s.q0 + tok) * P.Hq + u.g * P.G + h) * d + c4,
             make_float4(any ? o.x * inv : 0.f, any ? o.y * inv : 0.f, any ? o.z * inv : 0.f, any ? o.w * inv : 0.f));
    }
    if (threadIdx.x == 0) P.done[c_first] = 0;
  }
  __syncthreads();
}

// ---------------------------------------------------------------- bf16, warp MMAs
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// D += A * B, m16n8k16, bf16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16 bytes global -> shared; `bytes` of them are read, the rest is zero.
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int D, int NT>
struct MmaLayout {
  static constexpr int kStages = D == 64 ? 4 : 3;
  static constexpr uint32_t kRowBytes = D * 2;
  static constexpr uint32_t kHalfBytes = kTile * kRowBytes;   // K (or V) of a tile
  static constexpr uint32_t kStageBytes = 2 * kHalfBytes;
  static constexpr uint32_t kWarpBytes = kStages * kStageBytes;
  static constexpr uint32_t kOffMeta = kWarps * kWarpBytes;                // [warp][stage] key0, nv
  static constexpr uint32_t kOffMl = kOffMeta + kWarps * kStages * 8;      // wm, wl [warp][kMaxRows]
  static constexpr uint32_t kOffPlan = kOffMl + 2 * kWarps * kMaxRows * 4;
  // a tile's stage holds a warp's fp32 output while its segment is merged
  static_assert(8 * NT * D * 4 <= kStageBytes, "merge buffer");
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads) k_paged_rows(const __grid_constant__ RowsParams P) {
  typedef MmaLayout<D, NT> Y;
  constexpr int S = Y::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t *ring = smem + warp * Y::kWarpBytes;
  int2 *meta = (int2 *)(smem + Y::kOffMeta) + warp * S;
  float *wm = (float *)(smem + Y::kOffMl), *wl = wm + kWarps * kMaxRows;

  Plan L;
  make_plan(P, smem + Y::kOffPlan, L);
  const int c = blockIdx.x;
  if (c >= L.C) {
    pdl_wait();
    return;
  }
  const long long lo = div_pos((long long)c * L.T, L.C), hi = div_pos((long long)(c + 1) * L.T, L.C);

  // ---- this warp's stream: iteration n is item lo + warp + kWarps n
  long long row_l = 0;  // lane l: pool row, first key and key count of iteration 32 (n / 32) + l
  int key_l = 0, nv_l = 0;
  auto prefetch = [&](int n) {
    if ((n & 31) == 0) {
      const long long i = lo + warp + (long long)kWarps * (n + lane);
      nv_l = 0;
      row_l = 0;
      key_l = 0;
      if (i < hi) {
        const Unit u = unit_of(P, L, i);
        tile_keys(P, u, (int)(i - u.first), key_l, nv_l);
        if (nv_l > 0) {
          row_l = key_row(P, u, key_l);
          if (row_l < 0) row_l = 0, nv_l = 0;
        }
      }
    }
    const long long row = __shfl_sync(0xffffffffu, row_l, n & 31);
    const int key0 = __shfl_sync(0xffffffffu, key_l, n & 31), nv = __shfl_sync(0xffffffffu, nv_l, n & 31);
    const int st = n % S;
    if (lane == 0) meta[st] = make_int2(key0, nv);
    if (lo + warp + (long long)kWarps * n < hi) {
      const uint32_t dst = smem_u32(ring + st * Y::kStageBytes);
      const char *ks = (const char *)P.kp + row * Y::kRowBytes, *vs = (const char *)P.vp + row * Y::kRowBytes;
      constexpr int kChunks = D / 8;  // 16-byte pieces of a row
#pragma unroll
      for (int e0 = 0; e0 < kTile * kChunks; e0 += 32) {
        const int e = e0 + lane, r = e / kChunks, q = e % kChunks;
        const uint32_t at = dst + r * Y::kRowBytes + ((q ^ (r & 7)) << 4);
        const int take = r < nv ? 16 : 0;  // keys that nobody sees are zero
        const uint32_t src = take ? r * Y::kRowBytes + q * 16 : 0u;
        cp16(at, ks + src, take);
        cp16(at + Y::kHalfBytes, vs + src, take);
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int n = 0; n < S - 1; ++n) prefetch(n);

  int n = 0;  // iterations done
  for (long long i0 = lo; i0 < hi;) {
    const Unit u = unit_of(P, L, i0);
    const long long i1 = min(hi, u.end);
    // queries as the B operand: lane holds row lane / 4 of each 8-row group, dims
    // 16 kk + 2 (lane % 4) + {0, 1, 8, 9}
    uint32_t qf[D / 16][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      int tok, h;
      const bool in = unit_row(P, u, nt * 8 + (lane >> 2), tok, h);
      const uint32_t *src =
          (const uint32_t *)((const __nv_bfloat16 *)P.q + ((size_t)(u.s.q0 + (in ? tok : 0)) * P.Hq + u.g * P.G + (in ? h : 0)) * D) +
          (lane & 3);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qf[kk][nt][0] = in ? src[kk * 8] : 0u;
        qf[kk][nt][1] = in ? src[kk * 8 + 4] : 0u;
      }
    }
    // positions of the two rows (columns of S^T) of each group that this lane accumulates
    int tcol[NT][2], t_first = 0x7fffffff;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        int tok, h;
        const bool in = unit_row(P, u, nt * 8 + 2 * (lane & 3) + e, tok, h);
        tcol[nt][e] = in ? u.s.len - u.s.n + tok : -1;
        if (in) t_first = min(t_first, tcol[nt][e]);
      }
    t_first = __reduce_min_sync(0xffffffffu, t_first);

    float m[NT][2], l[NT][2], o[D / 16][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt) o[dt][nt][0] = o[dt][nt][1] = o[dt][nt][2] = o[dt][nt][3] = 0.f;
    }

    for (; lo + warp + (long long)kWarps * n < i1; ++n) {
      __syncwarp();  // every lane is done with the stage that is filled next
      prefetch(n + S - 1);
      cp_wait<S - 1>();
      __syncwarp();
      const int st = n % S;
      const int2 kn = meta[st];
      if (kn.y == 0) continue;
      const uint32_t kb = smem_u32(ring + st * Y::kStageBytes), vb = kb + Y::kHalfBytes;
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
      {
        const int r = (lane & 7) + 8 * ((lane >> 3) & 1);
        const uint32_t at = kb + r * Y::kRowBytes;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t a[4];
          ldsm_x4(at + (((kk * 2 + (lane >> 4)) ^ (r & 7)) << 4), a);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(s[nt], a, qf[kk][nt][0], qf[kk][nt][1]);
        }
      }
      // s[nt]: keys lane / 4 (elements 0, 1) and lane / 4 + 8 (2, 3), rows 2 (lane % 4) + {0, 1}
      const bool part = kn.y < kTile || kn.x + kTile - 1 > t_first;
      const int k0 = lane >> 2;
      uint32_t pb[NT][2];
      bool moved = false;
      float fix[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = s[nt][e] * P.sl2;
          if (part) {
            const int key = k0 + 8 * (e >> 1);
            if (key >= kn.y || kn.x + key > tcol[nt][e & 1]) x[e] = -INFINITY;
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(x[e], x[e + 2]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float mn = fmaxf(m[nt][e], mx);
          fix[nt][e] = mn == -INFINITY ? 1.f : ex2_approx(m[nt][e] - mn);
          moved |= mn != m[nt][e];
          m[nt][e] = mn;
          const float ref = mn == -INFINITY ? 0.f : mn;
          const float p0 = ex2_approx(x[e] - ref), p1 = ex2_approx(x[e + 2] - ref);
          l[nt][e] = fmaf(l[nt][e], fix[nt][e], p0 + p1);
          x[e] = p0;
          x[e + 2] = p1;
        }
        // P in bf16 for the product, whose operands have one type (V is bf16); its sum stays in fp32 of the
        // unrounded values. Outputs are 2.3e-3 from the 64-bit form (2-norm), 1.7e-3 of it their own rounding to
        // bf16. A second product with P's low half leaves the 1.7e-3 and takes 203.2 us instead of 200.6 at 64
        // sequences of 4K .. 32K, 33.2 instead of 32.8 over selected blocks; the other attention kernels of this
        // library round P too.
        pb[nt][0] = transpose8x8(pack_bf16x2(x[0], x[1]));
        pb[nt][1] = transpose8x8(pack_bf16x2(x[2], x[3]));
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[dt][nt][e] *= fix[nt][e & 1];
      }
      {
        const int r = (lane & 7) + 8 * (lane >> 4);
        const uint32_t at = vb + r * Y::kRowBytes;
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) {
          uint32_t a[4];
          ldsm_x4_t(at + (((dt * 2 + ((lane >> 3) & 1)) ^ (r & 7)) << 4), a);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(o[dt][nt], a, pb[nt][0], pb[nt][1]);
        }
      }
    }
    // the stage consumed last is free until the next prefetch: it takes this warp's output
    __syncwarp();
    float *mine = (float *)(ring + ((n + S - 1) % S) * Y::kStageBytes);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 4);
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 8);
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 16);
        const int r = nt * 8 + 2 * (lane & 3) + e;
        if (lane < 4) {
          wm[warp * kMaxRows + r] = m[nt][e];
          wl[warp * kMaxRows + r] = l[nt][e];
        }
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) {
          mine[r * D + swz(r, dt * 16 + (lane >> 2))] = o[dt][nt][e];
          mine[r * D + swz(r, dt * 16 + 8 + (lane >> 2))] = o[dt][nt][e + 2];
        }
      }
    }
    // every warp's free stage, from the number of its iterations so far
    float *buf[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const long long left = i1 - lo - w;  // items of warp w below i1: ceil(left / kWarps)
      const int nw = left > 0 ? (int)((left + kWarps - 1) / kWarps) : 0;
      buf[w] = (float *)(smem + w * Y::kWarpBytes + ((nw + S - 1) % S) * Y::kStageBytes);
    }
    finish_segment<__nv_bfloat16, true>(P, L, u, i0, i1, lo, buf, wm, wl);
    settle<__nv_bfloat16>(P, L, u, i0, i1);
    i0 = i1;
  }
  cp_wait<0>();
  // As a programmatic dependent of the chunk kernels it needs nothing of theirs, but it must not
  // count as complete before they are.
  pdl_wait();
}

// ---------------------------------------------------------------- any type and shape, CUDA cores
// fp32, and bf16 head widths or block sizes without a tensor-core form: the same items and streams with
// units of R = 4 or 8 rows, everything in fp32. A warp holds all rows of the unit against the 16 keys
// of its tile, so that K and V are read from shared memory once for the R rows: lanes are
// (key, half of the dims) for the logits, whose weights then go through shared memory to lanes that are dims
// (and, up to 64 dims, halves of the keys). The ring holds K and V of a tile as entries of their own (of up
// to 512 bytes a row: two each at 256 dims in fp32).
// Measured in fp32: 3 chunks of 60 .. 256 tokens over 4 selected blocks of 32, 4 / 1 heads of 64, 23 us in a graph, latency; a
// step of 64 sequences of 2K .. 8K, 16 / 2 heads of 128, 162 us (4.1 TB/s); 4 chunks of 450 tokens of 2000, 1474 us
// (17.7 TFLOP/s: shared memory, and the softmax between the products). With 32 keys a step for the whole CTA and
// barriers around each they took 46, 371 and 1673.
template <typename T, int R, int kD_>
struct SimtLayout {
  static constexpr int kElems = 16 / sizeof(T);  // elements of 16 bytes
  static constexpr int kPart = kD_ * sizeof(T) <= 512 ? kD_ : 512 / sizeof(T), kParts = kD_ / kPart;  // dims of an entry
  static constexpr uint32_t kRowBytes = kPart * sizeof(T), kEntryBytes = kTile * kRowBytes;
  // Few entries and many warps: the logits and the softmax of a tile are one chain, which other warps cover. In
  // fp32, four chunks of 450 tokens of 2000, 16 / 2 heads: at 128 dims two entries and three CTAs an SM
  // 1474 us, three and two 1889; at 256 dims 3102 and 3583. At 64 dims three and four take 22.7 us for the small
  // case above and 978 for these chunks, four and three 24.6 and 899.
  static constexpr int kEntries = kRowBytes <= 256 ? 3 : 2;
  static constexpr int kCtas = kRowBytes <= 256 ? 4 : 3;  // per SM
  static constexpr uint32_t kWarpBytes = kEntries * kEntryBytes;
  static constexpr uint32_t kOffMeta = kWarps * kWarpBytes;            // [warp][4] key0, nv
  static constexpr uint32_t kOffMl = kOffMeta + kWarps * 4 * 8;        // wm, wl [warp][kMaxRows]
  static constexpr uint32_t kOffQ = kOffMl + 2 * kWarps * kMaxRows * 4;  // [R][kD_] fp32
  static constexpr uint32_t kOffP = kOffQ + R * kD_ * 4;               // [warp][key][R] fp32
  static constexpr uint32_t kOffPlan = kOffP + kWarps * kTile * R * 4;
  // a free entry holds a warp's fp32 output while its segment is merged
  static_assert(R * kD_ * 4 <= kEntryBytes, "merge buffer");
};

template <typename T>
__device__ __forceinline__ float4 load4(const T *p);
template <>
__device__ __forceinline__ float4 load4<float>(const float *p) { return *(const float4 *)p; }
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16 *p) {
  const uint2 w = *(const uint2 *)p;
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}

template <typename T, int R, int kD_>
__global__ void __launch_bounds__(kThreads, SimtLayout<T, R, kD_>::kCtas) k_paged_simt(const __grid_constant__ RowsParams P) {
  typedef SimtLayout<T, R, kD_> Y;
  constexpr int N = Y::kEntries, kElems = Y::kElems, kChunks = Y::kRowBytes / 16;
  constexpr int kPart = Y::kPart, kParts = Y::kParts, kPer = 2 * kParts;  // entries per tile
  constexpr int kGroups = kD_ == 256 ? 2 : 1, kIn = kGroups / kParts;     // groups of four dims of a lane in O, in an entry
  constexpr bool kSplit = kD_ == 64;           // 16 lanes hold O: the two halves of a warp take every other key
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d = P.d;
  auto chunks_of = [&](int part) { return min(kChunks, d / kElems - part * kChunks); };  // 16-byte pieces of a row
  uint8_t *ring = smem + warp * Y::kWarpBytes;
  int2 *meta = (int2 *)(smem + Y::kOffMeta) + warp * 4;
  float *wm = (float *)(smem + Y::kOffMl), *wl = wm + kWarps * kMaxRows;
  float *qs = (float *)(smem + Y::kOffQ), *ps = (float *)(smem + Y::kOffP) + warp * kTile * R;

  Plan L;
  make_plan(P, smem + Y::kOffPlan, L);
  const int c = blockIdx.x;
  if (c >= L.C) return;
  const long long lo = div_pos((long long)c * L.T, L.C), hi = div_pos((long long)(c + 1) * L.T, L.C);

  // ---- this warp's stream: iteration n is item lo + warp + kWarps n, entries kPer n .. (K) and kPer n + kParts .. (V)
  long long row_l = 0, next_l = 0;  // lane l: of iteration 32 (n / 32) + l the pool row of the first key, and of
  int key_l = 0, nv_l = 0, cut_l = kTile;  // key `cut`, the first one in another page; first key and key count
  auto prefetch = [&](int h) {
    const int n = h / kPer, j = h % kPer, part = j % kParts;
    if (j == 0 && (n & 31) == 0) {
      const long long i = lo + warp + (long long)kWarps * (n + lane);
      nv_l = 0;
      row_l = next_l = 0;
      key_l = 0;
      cut_l = kTile;
      if (i < hi) {
        const Unit u = unit_of(P, L, i);
        tile_keys(P, u, (int)(i - u.first), key_l, nv_l);
        if (nv_l > 0) {
          const int in_page = P.P.ps - (key_l & (P.P.ps - 1));
          row_l = key_row(P, u, key_l);
          if (row_l < 0) row_l = 0, nv_l = 0;
          if (in_page < nv_l) {
            cut_l = in_page;
            next_l = key_row(P, u, key_l + in_page);
            if (next_l < 0) next_l = 0, nv_l = in_page;
          }
        }
      }
    }
    const long long row = __shfl_sync(0xffffffffu, row_l, n & 31), next = __shfl_sync(0xffffffffu, next_l, n & 31);
    const int key0 = __shfl_sync(0xffffffffu, key_l, n & 31), nv = __shfl_sync(0xffffffffu, nv_l, n & 31);
    const int cut = __shfl_sync(0xffffffffu, cut_l, n & 31);
    if (lane == 0) meta[n & 3] = make_int2(key0, nv);
    if (lo + warp + (long long)kWarps * n < hi) {
      const uint32_t dst = smem_u32(ring + h % N * Y::kEntryBytes);
      const T *pool = (const T *)(j < kParts ? P.kp : P.vp);
      const int chunks = chunks_of(part);
#pragma unroll
      for (int e0 = 0; e0 < kTile * kChunks; e0 += 32) {
        const int e = e0 + lane, r = e / kChunks, q = e % kChunks;
        if (q >= chunks) continue;
        const int take = r < nv ? 16 : 0;  // keys that nobody sees are zero
        const T *src = take ? pool + (r < cut ? row + r : next + (r - cut)) * d + part * kPart + q * kElems : pool;
        cp16(dst + r * Y::kRowBytes + ((q ^ (r & 7)) << 4), src, take);
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int h = 0; h < N - 1; ++h) prefetch(h);

  int n = 0;  // iterations done
  for (long long i0 = lo; i0 < hi;) {
    const Unit u = unit_of(P, L, i0);
    const long long i1 = min(hi, u.end);
    for (int e = threadIdx.x; e < R * (d >> 2); e += kThreads) {
      const int r = e / (d >> 2), c4 = (e - r * (d >> 2)) * 4;
      int tok, h;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (unit_row(P, u, r, tok, h)) x = load4((const T *)P.q + ((size_t)(u.s.q0 + tok) * P.Hq + u.g * P.G + h) * d + c4);
      *(float4 *)(qs + r * kD_ + c4) = x;
    }
    int trow[R];  // positions of the rows
    {
      int tok, h;
      const int t = unit_row(P, u, lane, tok, h) ? u.s.len - u.s.n + tok : -1;
#pragma unroll
      for (int r = 0; r < R; ++r) trow[r] = __shfl_sync(0xffffffffu, t, r);
    }
    float m[R], l[R];
    float4 o[R][kGroups];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) o[r][g] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();  // the queries are there

    for (; lo + warp + (long long)kWarps * n < i1; ++n) {
      const int key = lane & 15;
      int2 kn;
      float acc[R];
#pragma unroll
      for (int r = 0; r < R; ++r) acc[r] = 0.f;
#pragma unroll
      for (int part = 0; part < kParts; ++part) {
        const int h = kPer * n + part;
        __syncwarp();  // every lane is done with the entry that is filled next
        prefetch(h + N - 1);
        cp_wait<N - 1>();
        __syncwarp();
        kn = meta[n & 3];
        if (kn.y == 0) continue;
        const uint8_t *kr = ring + h % N * Y::kEntryBytes + key * Y::kRowBytes;
        const int chunks = chunks_of(part);
#pragma unroll 2
        for (int q = lane >> 4; q < chunks; q += 2) {
          const T *at = (const T *)(kr + ((q ^ (key & 7)) << 4));
#pragma unroll
          for (int e = 0; e < kElems; e += 4) {
            const float4 x = load4(at + e);
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const float4 y = *(const float4 *)(qs + r * kD_ + part * kPart + q * kElems + e);
              acc[r] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, acc[r]))));
            }
          }
        }
      }
      if (kn.y > 0) {
        float p[R], fix[R];
        bool moved = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], 16);
          const float x = key < kn.y && kn.x + key <= trow[r] ? acc[r] * P.sl2 : -INFINITY;
          float mx = x;
#pragma unroll
          for (int s = 8; s; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
          const float mn = fmaxf(m[r], mx);
          fix[r] = mn == -INFINITY ? 1.f : ex2_approx(m[r] - mn);
          moved |= mn != m[r];
          p[r] = x == -INFINITY ? 0.f : ex2_approx(x - mn);
          l[r] = fmaf(l[r], fix[r], p[r]);
          m[r] = mn;
        }
        if (lane < kTile)
#pragma unroll
          for (int r = 0; r < R; r += 4) *(float4 *)(ps + lane * R + r) = make_float4(p[r], p[r + 1], p[r + 2], p[r + 3]);
        if (__any_sync(0xffffffffu, moved))
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int g = 0; g < kGroups; ++g) o[r][g].x *= fix[r], o[r][g].y *= fix[r], o[r][g].z *= fix[r], o[r][g].w *= fix[r];
      }
#pragma unroll
      for (int part = 0; part < kParts; ++part) {
        const int h = kPer * n + kParts + part;
        __syncwarp();  // the weights are there and the entry before has been read
        prefetch(h + N - 1);
        cp_wait<N - 1>();
        __syncwarp();
        if (kn.y == 0) continue;
        const uint8_t *vr = ring + h % N * Y::kEntryBytes;
        const int dim = kSplit ? 4 * (lane & 15) : 4 * lane;
#pragma unroll 4
        for (int i = 0; i < (kSplit ? kTile / 2 : kTile); ++i) {
          const int k = kSplit ? 2 * i + (lane >> 4) : i;
          float4 x[kIn];
#pragma unroll
          for (int g = 0; g < kIn; ++g) {  // behind d it is whatever was there, in lanes that write nothing
            const int e = dim + 128 * g;
            x[g] = load4((const T *)(vr + k * Y::kRowBytes + (((e / kElems) ^ (k & 7)) << 4)) + e % kElems);
          }
#pragma unroll
          for (int r = 0; r < R; r += 4) {
            const float4 w4 = *(const float4 *)(ps + k * R + r);
            const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
            for (int f = 0; f < 4; ++f)
#pragma unroll
              for (int g = 0; g < kIn; ++g) {
                float4 &y = o[r + f][part * kIn + g];
                y.x = fmaf(w[f], x[g].x, y.x);
                y.y = fmaf(w[f], x[g].y, y.y);
                y.z = fmaf(w[f], x[g].z, y.z);
                y.w = fmaf(w[f], x[g].w, y.w);
              }
          }
        }
      }
    }
    // the entry consumed last is free until the next prefetch: it takes this warp's output
    __syncwarp();
    float *mine = (float *)(ring + (kPer * n + N - 1) % N * Y::kEntryBytes);
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int s = 8; s; s >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], s);
      if (lane == 0) {
        wm[warp * kMaxRows + r] = m[r];
        wl[warp * kMaxRows + r] = l[r];
      }
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        float4 x = o[r][g];
        if (kSplit) {
          x.x += __shfl_xor_sync(0xffffffffu, x.x, 16);
          x.y += __shfl_xor_sync(0xffffffffu, x.y, 16);
          x.z += __shfl_xor_sync(0xffffffffu, x.z, 16);
          x.w += __shfl_xor_sync(0xffffffffu, x.w, 16);
        }
        const int e = (kSplit ? 4 * (lane & 15) : 4 * lane) + 128 * g;
        if (e < d && (!kSplit || lane < 16)) *(float4 *)(mine + r * d + e) = x;
      }
    }
    float *buf[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const long long left = i1 - lo - w;  // items of warp w below i1: ceil(left / kWarps)
      const int nw = left > 0 ? (int)((left + kWarps - 1) / kWarps) : 0;
      buf[w] = (float *)(smem + w * Y::kWarpBytes + (kPer * nw + N - 1) % N * Y::kEntryBytes);
    }
    finish_segment<T, false>(P, L, u, i0, i1, lo, buf, wm, wl);
    settle<T>(P, L, u, i0, i1);
    i0 = i1;
  }
  cp_wait<0>();
}

int sm_count() {
  static int n[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (!n[dev] && cudaDeviceGetAttribute(&n[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) n[dev] = 148;
  return n[dev];
}

// CTAs whose shared memory an SM holds at once (228 KB, 1 KB of it reserved per CTA), `most` at most
int ctas_per_sm(size_t smem, int most) { return std::max(1, std::min(most, (int)(228 * 1024 / (smem + 1024)))); }

template <int D, int NT>
cudaError_t launch_mma(RowsParams &P, cudaStream_t st, bool pdl) {
  typedef MmaLayout<D, NT> Y;
  const size_t smem = Y::kOffPlan + plan_bytes(P.nb);
  P.C = min(sm_count() * ctas_per_sm(smem, 3), kMaxCtas);
  cudaError_t e = ensure_smem(k_paged_rows<D, NT>, smem);
  if (e != cudaSuccess) return e;
  note_launch();
  return launch_maybe_pdl(k_paged_rows<D, NT>, dim3(P.C), dim3(kThreads), smem, st, pdl, P);
}

template <typename T, int R, int kD_>
cudaError_t launch_simt(RowsParams &P, cudaStream_t st) {
  typedef SimtLayout<T, R, kD_> Y;
  const size_t smem = Y::kOffPlan + plan_bytes(P.nb);
  P.C = min(sm_count() * ctas_per_sm(smem, Y::kCtas), kMaxCtas);
  cudaError_t e = ensure_smem(k_paged_simt<T, R, kD_>, smem);
  if (e != cudaSuccess) return e;
  note_launch();
  k_paged_simt<T, R, kD_><<<P.C, kThreads, smem, st>>>(P);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_simt(RowsParams &P, cudaStream_t st) {
  if (P.R == 4) return P.d <= 64 ? launch_simt<T, 4, 64>(P, st) : P.d <= 128 ? launch_simt<T, 4, 128>(P, st) : launch_simt<T, 4, 256>(P, st);
  return P.d <= 64 ? launch_simt<T, 8, 64>(P, st) : P.d <= 128 ? launch_simt<T, 8, 128>(P, st) : launch_simt<T, 8, 256>(P, st);
}

}  // namespace

// [kMaxCtas] counters, then two slots of fp32 partials per CTA.
size_t paged_rows_workspace(const Dims &D) {
  return (size_t)kMaxCtas * sizeof(int) + (size_t)2 * kMaxCtas * kMaxRows * (D.d + 2) * sizeof(float);
}

cudaError_t launch_paged_rows(const Dims &D, const Paged &G, const void *q, const void *k_pages, const void *v_pages,
                              const int32_t *sel, void *out, long long max_rows, void *scratch, int *status,
                              cudaStream_t st, bool pdl) {
  RowsParams P;
  P.Hq = D.Hq;
  P.Hkv = D.Hkv;
  P.G = D.G;
  P.d = D.d;
  P.B = D.B;
  P.k = D.k;
  P.sl2 = D.scale * 1.4426950408889634f;
  P.P = G;
  P.q = q;
  P.kp = k_pages;
  P.vp = v_pages;
  P.sel = sel;
  P.out = out;
  P.done = (int *)scratch;
  P.part_o = (float *)((char *)scratch + (size_t)kMaxCtas * sizeof(int));
  P.part_ml = P.part_o + (size_t)2 * kMaxCtas * kMaxRows * D.d;
  P.status = status;
  P.max_rows = max_rows;
  P.tpb = (D.B + kTile - 1) / kTile;
  const long long rows = sel ? D.G : std::min((long long)D.G * G.max_chunk, max_rows - 1);
  const bool mma = D.bf16 && (D.d == 64 || D.d == 128 || D.d == 256) && (!sel || D.B % kTile == 0);
  P.R = mma ? (rows <= 8 ? 8 : 16) : rows <= 4 ? 4 : 8;
  P.rtk = (D.G + P.R - 1) / P.R;
  P.min_items = 2 * kWarps;
  for (P.b0 = 0; P.b0 < G.batch; P.b0 += kMaxSeqs) {
    P.nb = min(kMaxSeqs, G.batch - P.b0);
    const bool dep = pdl && P.b0 == 0;  // the launches of this loop share the workspace
    cudaError_t e;
    if (!mma) e = D.bf16 ? launch_simt<__nv_bfloat16>(P, st) : launch_simt<float>(P, st);
    else if (D.d == 64) e = P.R == 8 ? launch_mma<64, 1>(P, st, dep) : launch_mma<64, 2>(P, st, dep);
    else if (D.d == 128) e = P.R == 8 ? launch_mma<128, 1>(P, st, dep) : launch_mma<128, 2>(P, st, dep);
    else e = P.R == 8 ? launch_mma<256, 1>(P, st, dep) : launch_mma<256, 2>(P, st, dep);
    if (e != cudaSuccess) {
      note_error("paged attention launch", e);
      return e;
    }
  }
  return cudaSuccess;
}

}  // namespace qsa
