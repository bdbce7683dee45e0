// Norm and rotation of head rows, and the append of new tokens to a paged K/V cache.
//
// Every head x of d elements at position t becomes
//   y = x / sqrt(mean(x^2) + eps) * (w + w_off),  then for i < r/2, j = i + r/2:
//   (y_i, y_j) -> (y_i cos a - y_j sin a, y_j cos a + y_i sin a),  a = t theta^(-2i/r),
// in fp32, rounded once. Each element is read once and written once, with about 7
// operations between: bound by HBM for a prompt, by latency for a decode step.
//
// A token is one CTA's work: its heads (of q, k, v and the indexer key) are cut into
// rows of warp width, 8 elements (one or two 16-byte accesses) a lane, so a head of 128
// sits in 16 lanes and a warp takes two at once. The mean of squares is a shuffle
// reduction inside the head's lanes; the rotation partner of a lane's 8 elements is the
// lane r/16 further on, whose raw values arrive by shuffle, so nothing but the token's
// cosines and sines passes through shared memory.
//
// The angle is taken modulo a turn in integers: theta^(-2i/r) / 2 pi, as a 64-bit
// fraction of a turn, times t wraps round exactly, and its upper 32 bits are the phase
// to 2^-32 turn at any position. (An fp32 product t theta^(-2i/r) is off by 2^-8 rad at
// position 65536 already.)
#include <math.h>

#include "qsa_internal.h"
#include "sm100_ptx.cuh"

namespace qsa {
namespace {

constexpr int kWarps = 8;
constexpr int kBatch = 3;       // warp rows in flight per warp
constexpr int kMaxHalf = 128;   // rotary pairs of a head: head_dim <= 256

struct NrParams {
  AppendArgs A;
  Paged P;
  const int32_t *pos;  // null: positions from P
  int n_tok, Hq, Hkv, d, di;
  int rot, rot_i;
  float eps, w_off;
  const void *qw, *kw;
  int *status;
  // theta^(-2i/rot) / 2 pi as fractions of a turn, times 2^64
  uint64_t freq[kMaxHalf], freq_i[kMaxHalf];
};

template <typename T> struct Raw8 { uint4 w[sizeof(T) / 2]; };

template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T *p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.w[i] = ((const uint4 *)p)[i];
  return r;
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const Raw8<T> &r) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i) ((uint4 *)p)[i] = r.w[i];
}
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16> &r, float (&x)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack8(const Raw8<float> &r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[4 * i] = __uint_as_float(r.w[i].x);
    x[4 * i + 1] = __uint_as_float(r.w[i].y);
    x[4 * i + 2] = __uint_as_float(r.w[i].z);
    x[4 * i + 3] = __uint_as_float(r.w[i].w);
  }
}
__device__ __forceinline__ void pack8(Raw8<__nv_bfloat16> &r, const float (&x)[8]) {
  r.w[0] = make_uint4(sm100::pack_bf16x2(x[0], x[1]), sm100::pack_bf16x2(x[2], x[3]),
                      sm100::pack_bf16x2(x[4], x[5]), sm100::pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void pack8(Raw8<float> &r, const float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    r.w[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]),
                        __float_as_uint(x[4 * i + 3]));
}
template <typename T>
__device__ __forceinline__ Raw8<T> shfl8(const Raw8<T> &r, int src) {
  Raw8<T> o;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i) {
    o.w[i].x = __shfl_sync(0xffffffffu, r.w[i].x, src);
    o.w[i].y = __shfl_sync(0xffffffffu, r.w[i].y, src);
    o.w[i].z = __shfl_sync(0xffffffffu, r.w[i].z, src);
    o.w[i].w = __shfl_sync(0xffffffffu, r.w[i].w, src);
  }
  return o;
}

// lanes a head of dim elements takes: a power of two, 8 elements a lane
__device__ __forceinline__ int head_lanes(int dim) {
  int w = 1;
  while (w * 8 < dim) w <<= 1;
  return w;
}

enum { kSegQ = 0, kSegK = 1, kSegV = 2, kSegKi = 3 };

// A lane's share of one warp row of the token's heads.
struct Item {
  int seg, head, j, lanes;  // lane j of the head's `lanes`
  bool live;                // the lane holds elements of a head
};

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_norm_rope(const __grid_constant__ NrParams P) {
  __shared__ float s_cos[2 * kMaxHalf], s_sin[2 * kMaxHalf];  // q/k angles, then the indexer's
  __shared__ int s_seq[4];                                    // sequence (-1: none), position, length
  const int n = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const AppendArgs &A = P.A;

  const int wd = head_lanes(P.d), wi = head_lanes(P.di);
  const int per_d = 32 / wd;  // heads of d elements per warp row
  const int nq = A.q ? (P.Hq + per_d - 1) / per_d : 0;
  const int nk = A.k ? (P.Hkv + per_d - 1) / per_d : 0;
  const int nv = A.v ? nk : 0;
  const int n_items = nq + nk + nv + (A.ki ? 1 : 0);

  auto item = [&](int i) {
    Item it;
    it.live = i < n_items;
    int first = 0, heads = P.Hq, dim = P.d;
    it.seg = kSegQ;
    if (i >= nq + nk + nv) it.seg = kSegKi, first = nq + nk + nv, heads = 1, dim = P.di;
    else if (i >= nq + nk) it.seg = kSegV, first = nq + nk, heads = P.Hkv;
    else if (i >= nq) it.seg = kSegK, first = nq, heads = P.Hkv;
    it.lanes = it.seg == kSegKi ? wi : wd;
    it.j = lane & (it.lanes - 1);
    it.head = (i - first) * (32 / it.lanes) + lane / it.lanes;
    it.live = it.live && it.head < heads && it.j * 8 < dim;
    return it;
  };
  auto source = [&](const Item &it) {
    const long long row = it.seg == kSegQ ? A.q_row : it.seg == kSegK ? A.k_row : it.seg == kSegV ? A.v_row : A.ki_row;
    const void *base = it.seg == kSegQ ? A.q : it.seg == kSegK ? A.k : it.seg == kSegV ? A.v : A.ki;
    return (const T *)base + (long long)n * row + it.head * P.d + it.j * 8;
  };

  // the first rows' loads go out before the position is known
  Item items[kBatch];
  Raw8<T> raw[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    items[u] = item(warp + u * kWarps);
    raw[u] = Raw8<T>{};
    if (items[u].live) raw[u] = load8(source(items[u]));
  }

  int b = 0, t = 0, len = 0;
  if (P.pos) {
    t = P.pos[n];
  } else {
    // the row's sequence: the last b with q_start[b] <= n, by a 32-way search
    if (warp == 0) {
      int lo = 0, hi = P.P.batch;  // q_start[lo] <= n (if any), q_start[hi] > n
      if (P.P.q_start[0] > n || P.P.q_start[hi] <= n) {
        lo = -1;
      } else {
        while (hi - lo > 1) {
          const int step = (hi - lo + 31) / 32;
          const int at = lo + step * (lane + 1);
          const unsigned le = __ballot_sync(0xffffffffu, at < hi && P.P.q_start[at] <= n);
          const int c = __popc(le);
          hi = min(hi, lo + step * (c + 1));
          lo += step * c;
        }
      }
      int pos = -1, ln = 0;
      if (lo >= 0) {
        const PagedSeq s = paged_seq(P.P, lo, lane == 0 ? P.status : nullptr);
        if (s.ok && n >= s.q0 && n < s.q0 + s.n) {
          pos = s.len - s.n + (n - s.q0);
          ln = s.len;
        }
      }
      if (lane == 0) {
        s_seq[0] = pos >= 0 ? lo : -1;
        s_seq[1] = pos;
        s_seq[2] = ln;
      }
    }
    __syncthreads();
    b = s_seq[0];
    t = s_seq[1];
    len = s_seq[2];
    if (b < 0) return;  // a row of no sequence
  }
  for (int i = threadIdx.x; i < 2 * kMaxHalf; i += kWarps * 32) {
    const bool own = i < kMaxHalf;
    const int e = own ? i : i - kMaxHalf;
    if (2 * e < (own ? P.rot : A.ki ? P.rot_i : 0)) {
      // position times the frequency, modulo a turn; the signed upper half is the phase
      const uint64_t turn = (own ? P.freq[e] : P.freq_i[e]) * (uint64_t)(int64_t)t;
      const float half_turns = (float)(int32_t)(uint32_t)(turn >> 32) * 4.656612873077393e-10f;  // 2^-31
      sincospif(half_turns, &s_sin[i], &s_cos[i]);
    }
  }
  __syncthreads();

  // where the token's rows of the cache go
  int page = 0;
  bool page_ok = true;
  if (!P.pos) {
    page = P.P.table[(size_t)b * P.P.max_pages + (t >> P.P.ps_shift)];
    page_ok = page >= 0 && page < P.P.n_pages;
    if (!page_ok && threadIdx.x == 0) record_status(P.status, QSA_ERR_DEVICE_CHECK);
    if (A.ki && len > A.ki_cap && threadIdx.x == 0) record_status(P.status, QSA_ERR_DEVICE_CHECK);
  }

  for (int i0 = warp; i0 < n_items; i0 += kBatch * kWarps) {
    if (i0 != warp) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        items[u] = item(i0 + u * kWarps);
        raw[u] = Raw8<T>{};
        if (items[u].live) raw[u] = load8(source(items[u]));
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (i0 + u * kWarps >= n_items) continue;  // the same for the whole warp
      const Item it = items[u];
      const bool qk = it.seg == kSegQ || it.seg == kSegK;
      const T *w = qk ? (const T *)(it.seg == kSegQ ? P.qw : P.kw) : nullptr;
      const int rot = qk ? P.rot : it.seg == kSegKi ? P.rot_i : 0;
      Raw8<T> out = raw[u];
      if (w || rot) {
        float x[8], y[8];
        unpack8(raw[u], x);
        const int e0 = it.j * 8, half = rot >> 1;
        const bool turns = e0 < rot, lower = e0 < half;
        const int mate = turns ? (lower ? e0 + half : e0 - half) : e0;  // first element of the partner lane
        const Raw8<T> other = shfl8(raw[u], (lane & ~(it.lanes - 1)) + (mate >> 3));
        unpack8(other, y);
        if (w) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
          for (int o = it.lanes >> 1; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float r = rsqrtf(ss / (float)P.d + P.eps);
          if (it.live) {
            float wx[8], wy[8];
            unpack8(load8(w + e0), wx);
            unpack8(load8(w + mate), wy);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              x[e] = x[e] * r * (wx[e] + P.w_off);
              y[e] = y[e] * r * (wy[e] + P.w_off);
            }
          }
        }
        if (turns) {
          const int a = (it.seg == kSegKi ? kMaxHalf : 0) + (lower ? e0 : e0 - half);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = fmaf(y[e], lower ? -s_sin[a + e] : s_sin[a + e], x[e] * s_cos[a + e]);
        }
        pack8(out, x);
      }
      if (!it.live) continue;
      T *dst;
      if (it.seg == kSegQ) {
        dst = (T *)A.q_out + (long long)n * A.q_out_row + it.head * P.d;
      } else if (it.seg == kSegKi) {
        if (len > A.ki_cap) continue;
        dst = (T *)A.ki_cache + ((size_t)b * A.ki_cap + t) * P.di;
      } else if (P.pos) {
        dst = (T *)A.k_out + (long long)n * A.k_out_row + it.head * P.d;
      } else {
        if (!page_ok) continue;
        dst = (T *)(it.seg == kSegK ? A.k_pages : A.v_pages) +
              ((((size_t)page * P.Hkv + it.head) << P.P.ps_shift) + (t & (P.P.ps - 1))) * P.d;
      }
      store8(dst + it.j * 8, out);
    }
  }
}

// theta^(-2i/rot) / 2 pi in 2^-64 turns, by repeated multiplication: the i-th factor is off
// by i roundings of 2^-53, far below the 2^-32 turn that the kernel keeps.
void frequencies(uint64_t *f, int rot, double log2_theta) {
  if (rot <= 0) return;
  const double ratio = exp2(-2.0 * log2_theta / rot);
  double x = 18446744073709551616.0 / 6.283185307179586476925;
  for (int i = 0; i < rot / 2; ++i, x *= ratio) f[i] = x < 18446744073709549568.0 ? (uint64_t)x : ~0ull;
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
  P.qw = N.qw;
  P.kw = N.kw;
  frequencies(P.freq, N.rot, N.log2_theta);
  frequencies(P.freq_i, N.rot_i, N.log2_theta);
  note_launch();
  if (D.bf16) k_norm_rope<__nv_bfloat16><<<P.n_tok, kWarps * 32, 0, st>>>(P);
  else k_norm_rope<float><<<P.n_tok, kWarps * 32, 0, st>>>(P);
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
