// Norm and rotation of head rows, and the append of new tokens to a paged K/V cache.
//
// Every head x of d elements at position t becomes
//   y = x / sqrt(mean(x^2) + eps) * (w + w_off),  then for i < r/2, j = i + r/2:
//   (y_i, y_j) -> (y_i cos a - y_j sin a, y_j cos a + y_i sin a),  a = t theta^(-2i/r),
// in fp32, rounded once. Each element is read once and written once, with about 7 operations
// between: bound by HBM for a prompt (16K tokens, 32 + 4 heads of 128 in bf16, 302 MB: 56 us,
// 5.4 TB/s; appending as many, 330 MB with 256-byte pieces going to the pages: 72 us, 4.6 TB/s),
// by latency for a decode step (64 tokens: 3 us, 4 with the append).
//
// A warp takes the heads of one token (or, with few tokens, a part of them: each of them then
// computes the token's angles again). A head of d elements sits in d / 8 lanes, so a warp
// holds 256 / d heads at once; a lane holds 4 elements i .. i + 3 and their rotation partners
// i + r/2 .., as two 8-byte accesses, so the rotation needs no exchange, and the mean of
// squares is the only shuffle. Norm weight, cosine and sine are multiplied once per token
// and kind of head: out = rms (x_i (w_i c) - x_j (w_j s)), and so on.
//
// The angle is taken modulo a turn in integers: theta^(-2i/r) / 2 pi, as a 64-bit
// fraction of a turn, times t wraps round exactly, and its upper 32 bits are the phase
// to 2^-32 turn at any position. (An fp32 product t theta^(-2i/r) is off by 2^-8 rad at
// position 65536 already.)
#include <math.h>

#include <algorithm>
#include <limits>
#include <type_traits>

#include "qsa_internal.h"
#include "sm100_ptx.cuh"

namespace qsa {
namespace {

// Blocks of one warp: a warp that ends makes room for the next at once (blocks of four: 78 us instead
// of 72 to append 16K tokens, 58 instead of 56 for 16K rows of 32 + 4 heads of 128).
constexpr int kThreads = 32;
// Warp rows in flight per warp: those 16K rows take 61 us with 4, 57 with 6, 59 with 8; more warps with
// fewer registers each 61 to 68. Several tokens a warp, with the positions looked up for all of
// them at once: 65 to 73; a token's rows over two or three warps: 66 and 69.
constexpr int kBatch = 6;
constexpr int kMaxHalf = 128;   // rotary pairs of a head: head_dim <= 256
constexpr long long kFillWarps = 148 * 32;

struct NrParams {
  AppendArgs A;
  Paged P;
  const int32_t *pos;  // null: positions from P
  int n_tok, Hq, Hkv, d, di;
  int rot, rot_i;
  int parts;           // warps per token
  int sh_d, sh_i;      // log2 of the lanes of a head of d (di) elements
  int nq, nk, n_rows;  // a token's warp rows of q, of k, of everything
  float eps, w_off, inv_d;
  const void *qw, *kw;
  int *status;
  // theta^(-2i/rot) / 2 pi as fractions of a turn, times 2^64
  uint64_t freq[kMaxHalf], freq_i[kMaxHalf];
};

// Two groups of four elements as they are stored.
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> { uint2 a, b; };
template <> struct Raw<float> { uint4 a, b; };

__device__ __forceinline__ void load_raw(Raw<__nv_bfloat16> &r, const __nv_bfloat16 *p, const __nv_bfloat16 *q) {
  r.a = *(const uint2 *)p;
  r.b = *(const uint2 *)q;
}
__device__ __forceinline__ void load_raw(Raw<float> &r, const float *p, const float *q) {
  r.a = *(const uint4 *)p;
  r.b = *(const uint4 *)q;
}
__device__ __forceinline__ void store_raw(const Raw<__nv_bfloat16> &r, __nv_bfloat16 *p, __nv_bfloat16 *q) {
  *(uint2 *)p = r.a;
  *(uint2 *)q = r.b;
}
__device__ __forceinline__ void store_raw(const Raw<float> &r, float *p, float *q) {
  *(uint4 *)p = r.a;
  *(uint4 *)q = r.b;
}
// Four elements as two packed pairs of fp32, and back with one rounding.
__device__ __forceinline__ void unpack(const uint2 &r, uint64_t (&x)[2]) {
  x[0] = sm100::f2_pack(r.x << 16, r.x & 0xffff0000u);
  x[1] = sm100::f2_pack(r.y << 16, r.y & 0xffff0000u);
}
__device__ __forceinline__ void unpack(const uint4 &r, uint64_t (&x)[2]) {
  x[0] = sm100::f2_pack(r.x, r.y);
  x[1] = sm100::f2_pack(r.z, r.w);
}
__device__ __forceinline__ void pack(uint2 &r, const uint64_t (&x)[2]) {
  float a, b;
  sm100::f2_unpack(x[0], a, b);
  r.x = sm100::pack_bf16x2(a, b);
  sm100::f2_unpack(x[1], a, b);
  r.y = sm100::pack_bf16x2(a, b);
}
__device__ __forceinline__ void pack(uint4 &r, const uint64_t (&x)[2]) {
  float a, b;
  sm100::f2_unpack(x[0], a, b);
  r.x = __float_as_uint(a);
  r.y = __float_as_uint(b);
  sm100::f2_unpack(x[1], a, b);
  r.z = __float_as_uint(a);
  r.w = __float_as_uint(b);
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

enum { kSegQ = 0, kSegK = 1, kSegV = 2, kSegKi = 3 };

// Where a lane's elements are in a head: e0 .. e0 + 3 and e1 .. e1 + 3, rotation partners of each
// other in the lanes of the head's first `rot` elements.
struct Place {
  int lanes, j, e0, e1;
  bool live, turns;
};
__device__ __forceinline__ Place place_of(int dim, int shift, int rot, int lane) {
  Place p;
  p.lanes = 1 << shift;
  p.j = lane & (p.lanes - 1);
  p.live = p.j * 8 < dim;
  const int pairs = rot >> 3;  // lanes that rotate
  p.turns = p.j < pairs;
  p.e0 = p.turns ? 4 * p.j : 8 * p.j;
  p.e1 = p.turns ? p.e0 + (rot >> 1) : p.e0 + 4;
  return p;
}

// Cosine and sine of 2 pi turn / 2^32: the nearest quarter turn q and the rest x in
// [-pi/4, pi/4], whose Taylor sums to x^8 and x^9 are within 2^-25; a quarter turn swaps the
// two and moves a sign.
__device__ __forceinline__ void turn_cos_sin(uint32_t turn, float &c, float &s) {
  const uint32_t q = (turn + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(turn - (q << 30)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  const float y = x * x;
  float a = fmaf(y, 1.f / 362880.f, -1.f / 5040.f);
  a = fmaf(a, y, 1.f / 120.f);
  a = fmaf(a, y, -1.f / 6.f);
  a = fmaf(a * y, x, x);
  float b = fmaf(y, 1.f / 40320.f, -1.f / 720.f);
  b = fmaf(b, y, 1.f / 24.f);
  b = fmaf(b, y, -0.5f);
  b = fmaf(b, y, 1.f);
  const float u = q & 1 ? a : b, v = q & 1 ? b : a;
  c = (q + 1) & 2 ? -u : u;
  s = q & 2 ? -v : v;
}

// out0 = x0 a0 + x1 b0, out1 = x1 a1 + x0 b1 (times the norm)
struct Coef {
  uint64_t a0[2], b0[2], a1[2], b1[2];
};

// A lane's share of some of a token's warp rows of one kind of head: `rows` of them from src to dst,
// `step` elements apart.
template <typename T>
struct Rows {
  const T *src;
  T *dst;
  long long src_step, dst_step;
  int rows;
  int live;  // rows in which this lane holds elements
};
template <typename T>
__device__ __forceinline__ void load_rows(const Rows<T> &w, const Place &p, int r, Raw<T> (&raw)[kBatch]) {
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    raw[u] = Raw<T>{};
    if (r + u < w.live) load_raw(raw[u], w.src + (r + u) * w.src_step, w.src + (r + u) * w.src_step + (p.e1 - p.e0));
  }
}
// kCopy: as they are. The first batch is in raw already. kLanes: lanes of a head, 0 if only p knows.
template <typename T, int kLanes, bool kCopy>
__device__ __forceinline__ void run_rows(const Rows<T> &w, const Place &p, const Coef &c, bool normed, float inv_d, float eps,
                                         Raw<T> (&raw)[kBatch]) {
  using namespace sm100;
  const bool all_turn = __all_sync(0xffffffffu, p.turns);
  for (int r = 0; r < w.rows; r += kBatch) {
    if (r) load_rows(w, p, r, raw);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (r + u >= w.rows) break;  // the same for the whole warp
      if (!kCopy) {
        uint64_t x0[2], x1[2], y0[2], y1[2];
        unpack(raw[u].a, x0);
        unpack(raw[u].b, x1);
        if (normed) {
          const uint64_t q = f2_add(f2_fma(x0[0], x0[0], f2_mul(x0[1], x0[1])), f2_fma(x1[0], x1[0], f2_mul(x1[1], x1[1])));
          float sa, sb;
          f2_unpack(q, sa, sb);
          float ss = sa + sb;
          if (kLanes) {
#pragma unroll
            for (int o = kLanes >> 1; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          } else {
            for (int o = p.lanes >> 1; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          }
          const uint64_t rr = f2_splat(rsqrtf(fmaf(ss, inv_d, eps)));
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            x0[e] = f2_mul(x0[e], rr);
            x1[e] = f2_mul(x1[e], rr);
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // elements that do not rotate take nothing from their neighbours, infinities least of all
          y0[e] = f2_mul(x0[e], c.a0[e]);
          y1[e] = f2_mul(x1[e], c.a1[e]);
          if (all_turn || p.turns) {
            y0[e] = f2_fma(x1[e], c.b0[e], y0[e]);
            y1[e] = f2_fma(x0[e], c.b1[e], y1[e]);
          }
        }
        pack(raw[u].a, y0);
        pack(raw[u].b, y1);
      }
      if (r + u < w.live) store_raw(raw[u], w.dst + (r + u) * w.dst_step, w.dst + (r + u) * w.dst_step + (p.e1 - p.e0));
    }
  }
}

// kD: the head dim, 0 for one without an instantiation of its own
template <typename T, bool kPaged, int kD>
__global__ void __launch_bounds__(kThreads) k_norm_rope(const __grid_constant__ NrParams P) {
  using namespace sm100;
  const int lane = threadIdx.x;
  // warp `part` of token n
  const unsigned g = blockIdx.x;
  const int n = P.parts == 1 ? (int)g : (int)(g / (unsigned)P.parts), part = P.parts == 1 ? 0 : (int)(g % (unsigned)P.parts);
  const AppendArgs &A = P.A;

  // warp rows: those of q, then k, v and the indexer key
  constexpr int kLanes = kD / 8;
  const int d = kD ? kD : P.d, sh_d = kD == 64 ? 3 : kD == 128 ? 4 : kD == 256 ? 5 : P.sh_d;
  const Place pd = place_of(d, sh_d, P.rot, lane);
  const int sh = 5 - sh_d, per = 1 << sh, sub = lane >> sh_d;  // heads per warp row, the lane's among them
  const int f1 = P.nq, f2 = P.nq + P.nk, f3 = P.nq + (kPaged ? 2 : 1) * P.nk;  // first rows of k, v and ki
  const int i_begin = P.parts == 1 ? 0 : part * P.n_rows / P.parts;
  const int i_end = P.parts == 1 ? P.n_rows : (part + 1) * P.n_rows / P.parts;
  auto first_of = [&](int seg) { return seg == kSegQ ? 0 : seg == kSegK ? f1 : seg == kSegV ? f2 : f3; };

  // this warp's rows of one kind, without their destination
  auto rows_of = [&](int seg) {
    Rows<T> w;
    const int f = first_of(seg), lo = max(i_begin - f, 0), hi = min(i_end, seg == kSegKi ? P.n_rows : first_of(seg + 1)) - f;
    const T *base = seg == kSegQ ? (const T *)A.q + (long long)n * A.q_row
                    : seg == kSegK ? (const T *)A.k + (long long)n * A.k_row
                                   : (const T *)A.v + (long long)n * A.v_row;
    w.rows = max(hi - lo, 0);
    w.src_step = d << sh;
    w.src = base + ((lo << sh) + sub) * d + pd.e0;
    // the lane's head in row r is (lo + r) per + sub
    const int heads = (seg == kSegQ ? P.Hq : P.Hkv) - (lo << sh) - sub;
    w.live = pd.live ? min(w.rows, (heads + per - 1) >> sh) : 0;
    w.dst = nullptr;
    w.dst_step = 0;
    return w;
  };
  Place pi = pd;
  Rows<T> wi;  // the indexer key's row
  if (kPaged && A.ki) {
    pi = place_of(P.di, P.sh_i, P.rot_i, lane);
    wi.rows = max(i_end - max(i_begin, f3), 0);
    wi.src_step = 0;
    wi.src = (const T *)A.ki + (long long)n * A.ki_row + pi.e0;
    wi.live = pi.live && lane == pi.j ? wi.rows : 0;
  } else {
    wi.rows = 0;
  }

  // the first rows' loads go out before the position is known
  Raw<T> raw[kBatch];
  const int seg0 = i_begin < f1 ? kSegQ : i_begin < f2 ? kSegK : i_begin < f3 ? kSegV : kSegKi;
  if (!kPaged || seg0 != kSegKi) load_rows(rows_of(seg0), pd, 0, raw);
  else load_rows(wi, pi, 0, raw);

  int b = 0, t = 0, len = 0, page = 0;
  bool page_ok = true;
  if (!kPaged) {
    t = P.pos[n];
  } else {
    // the row's sequence: the last b with q_start[b] <= n, by a 32-way search
    int lo = 0, hi = P.P.batch;
    if (P.P.q_start[0] > n || P.P.q_start[hi] <= n) return;  // a row of no sequence
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int at = lo + step * (lane + 1);
      const int c = __popc(__ballot_sync(0xffffffffu, at < hi && P.P.q_start[at] <= n));
      hi = min(hi, lo + step * (c + 1));
      lo += step * c;
    }
    const PagedSeq s = paged_seq(P.P, lo, lane == 0 ? P.status : nullptr);
    if (!s.ok || n < s.q0 || n >= s.q0 + s.n) return;
    b = lo;
    t = s.len - s.n + (n - s.q0);
    len = s.len;
    page = P.P.table[(size_t)b * P.P.max_pages + (t >> P.P.ps_shift)];
    page_ok = page >= 0 && page < P.P.n_pages;
    if (lane == 0 && (!page_ok || (A.ki && len > A.ki_cap))) record_status(P.status, QSA_ERR_DEVICE_CHECK);
  }

  // cosine and sine of the lane's four pairs
  auto angles = [&](const uint64_t *freq, int j, uint64_t (&c)[2], uint64_t (&s)[2]) {
    float cs[4], sn[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // position times frequency, modulo a turn, in 2^-32 turns
      const uint32_t turn = (uint32_t)((freq[4 * j + e] * (uint64_t)(int64_t)t) >> 32);
      turn_cos_sin(turn, cs[e], sn[e]);
    }
    c[0] = f2_pack(__float_as_uint(cs[0]), __float_as_uint(cs[1]));
    c[1] = f2_pack(__float_as_uint(cs[2]), __float_as_uint(cs[3]));
    s[0] = f2_pack(__float_as_uint(sn[0]), __float_as_uint(sn[1]));
    s[1] = f2_pack(__float_as_uint(sn[2]), __float_as_uint(sn[3]));
  };
  const uint64_t one = f2_splat(1.f), minus = f2_splat(-1.f);
  uint64_t c[2] = {one, one}, s[2] = {0, 0};
  if (pd.turns && i_begin < f2) angles(P.freq, pd.j, c, s);
  auto coef_of = [&](const T *w) {
    uint64_t w0[2] = {one, one}, w1[2] = {one, one};
    if (w && pd.live) {
      Raw<T> rw;
      load_raw(rw, w + pd.e0, w + pd.e1);
      unpack(rw.a, w0);
      unpack(rw.b, w1);
      const uint64_t off = f2_splat(P.w_off);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        w0[e] = f2_add(w0[e], off);
        w1[e] = f2_add(w1[e], off);
      }
    }
    Coef k;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      k.a0[e] = f2_mul(w0[e], c[e]);
      k.b0[e] = f2_mul(f2_mul(w1[e], s[e]), minus);
      k.a1[e] = f2_mul(w1[e], c[e]);
      k.b1[e] = f2_mul(w0[e], s[e]);
    }
    return k;
  };

  const long long slot = kPaged ? (((long long)page * P.Hkv) << P.P.ps_shift) + (t & (P.P.ps - 1)) : 0;
#pragma unroll
  for (int seg = kSegQ; seg <= (kPaged ? kSegV : kSegK); ++seg) {
    Rows<T> w = rows_of(seg);
    if (w.rows == 0) continue;
    const int head = (max(i_begin - first_of(seg), 0) << sh) + sub;  // the lane's in the first row
    if (seg == kSegQ || !kPaged) {
      w.dst = seg == kSegQ ? (T *)A.q_out + (long long)n * A.q_out_row : (T *)A.k_out + (long long)n * A.k_out_row;
      w.dst += head * d + pd.e0;
      w.dst_step = d << sh;
    } else {
      w.dst = (T *)(seg == kSegK ? A.k_pages : A.v_pages) + (slot + ((long long)head << P.P.ps_shift)) * d + pd.e0;
      w.dst_step = ((long long)d << P.P.ps_shift) << sh;
      if (!page_ok) w.live = 0;
    }
    if (seg != seg0) load_rows(w, pd, 0, raw);
    const T *weight = (const T *)(seg == kSegQ ? P.qw : P.kw);
    if (seg == kSegV || (!weight && P.rot == 0)) {
      run_rows<T, kLanes, true>(w, pd, Coef{}, false, 0.f, 0.f, raw);
    } else {
      run_rows<T, kLanes, false>(w, pd, coef_of(weight), weight != nullptr, P.inv_d, P.eps, raw);
    }
  }
  if (kPaged && wi.rows) {
    if (len > A.ki_cap) wi.live = 0;
    wi.dst = (T *)A.ki_cache + ((size_t)b * A.ki_cap + t) * P.di + pi.e0;
    wi.dst_step = 0;
    if (seg0 != kSegKi) load_rows(wi, pi, 0, raw);
    Coef k;
    uint64_t ci[2] = {one, one}, si[2] = {0, 0};
    if (pi.turns) angles(P.freq_i, pi.j, ci, si);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      k.a0[e] = k.a1[e] = ci[e];
      k.b0[e] = f2_mul(si[e], minus);
      k.b1[e] = si[e];
    }
    if (P.rot_i == 0) run_rows<T, 0, true>(wi, pi, k, false, 0.f, 0.f, raw);
    else run_rows<T, 0, false>(wi, pi, k, false, 0.f, 0.f, raw);
  }
}

// theta^(-2i/rot) / 2 pi in 2^-64 turns, by repeated multiplication in the host's 80-bit floats: two
// roundings of 2^-64 a step for at most 128 steps, so that the turn at position t is off by less than |t| 2^-58.6,
// 2^-27 at the last int32. (64-bit floats were off by up to 1e-5 rad there, with a base of 1.25; they take
// 0.1 to 0.2 us less of the call.)
static_assert(std::numeric_limits<long double>::digits >= 64, "frequencies need 64 bits");
void frequencies(uint64_t *f, int rot, long double log2_theta) {
  if (rot <= 0) return;
  const long double ratio = exp2l(-2.0L * log2_theta / rot);
  long double x = 18446744073709551616.0L / 6.28318530717958647692528676655900577L;
  for (int i = 0; i < rot / 2; ++i, x *= ratio) f[i] = (uint64_t)x;
}

cudaError_t launch(const Dims &D, const NormRope &N, NrParams &P, cudaStream_t st) {
  P.Hq = D.Hq;
  P.Hkv = D.Hkv;
  P.d = D.d;
  P.di = D.di;
  P.rot = N.rot;
  P.rot_i = N.rot_i;
  P.eps = N.eps;
  P.w_off = N.w_off;
  P.inv_d = 1.f / (float)D.d;
  P.qw = N.qw;
  P.kw = N.kw;
  frequencies(P.freq, N.rot, N.log2_theta);
  frequencies(P.freq_i, N.rot_i, N.log2_theta);
  // With few tokens a token's rows are spread over more warps, down to one row a warp, until
  // there is a warp for each of about 32 per SM.
  P.sh_d = P.sh_i = 0;
  while ((8 << P.sh_d) < D.d) ++P.sh_d;
  while ((8 << P.sh_i) < D.di) ++P.sh_i;
  const int per = 32 >> P.sh_d;
  P.nq = P.A.q ? (D.Hq + per - 1) / per : 0;
  P.nk = P.A.k ? (D.Hkv + per - 1) / per : 0;
  P.n_rows = P.nq + P.nk * (P.pos ? 1 : 2) + (P.A.ki ? 1 : 0);
  P.parts = (int)std::max(1LL, std::min((long long)P.n_rows, kFillWarps / P.n_tok));
  const long long blocks = (long long)P.n_tok * P.parts;
  if (blocks > 0x7fffffffLL) return cudaErrorNotSupported;
  note_launch();
  auto pick = [&](auto d) {
    constexpr int kD = decltype(d)::value;
    return D.bf16 ? (P.pos ? k_norm_rope<__nv_bfloat16, false, kD> : k_norm_rope<__nv_bfloat16, true, kD>)
                  : (P.pos ? k_norm_rope<float, false, kD> : k_norm_rope<float, true, kD>);
  };
  auto kern = D.d == 64    ? pick(std::integral_constant<int, 64>{})
              : D.d == 128 ? pick(std::integral_constant<int, 128>{})
              : D.d == 256 ? pick(std::integral_constant<int, 256>{})
                           : pick(std::integral_constant<int, 0>{});
  kern<<<(unsigned)blocks, kThreads, 0, st>>>(P);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) note_error("k_norm_rope launch", e);
  return e;
}

}  // namespace

cudaError_t launch_norm_rope(const Dims &D, const NormRope &N, const int32_t *pos, int n_tok, const AppendArgs &A,
                             cudaStream_t st) {
  NrParams P;
  P.A = A;
  P.P = Paged{};
  P.pos = pos;
  P.n_tok = n_tok;
  P.status = nullptr;
  return launch(D, N, P, st);
}

cudaError_t launch_paged_append(const Dims &D, const NormRope &N, const Paged &G, const AppendArgs &A, int *status,
                                cudaStream_t st) {
  NrParams P;
  P.A = A;
  P.P = G;
  P.pos = nullptr;
  P.n_tok = G.n_tok;
  P.status = status;
  return launch(D, N, P, st);
}

}  // namespace qsa
