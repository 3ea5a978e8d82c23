// Rotary positions of the queries and keys, alone or with the norm of every
// head in the same pass, and the backward of both (sm_100a).
//
// For pair i of a head at position t (i < r/2, r the rotated part of the
// head), with the angle f = t * freq_i and the plan's amplitude a:
//   y1 = a (x1 cos f - x2 sin f),   y2 = a (x2 cos f + x1 sin f);
// the transpose of that map is the same with -sin.  With the norm,
//   x -> x * rstd * w,  rstd = (mean(x^2) + eps)^(-1/2) over the whole head,
// comes first.  Its backward, g being the gradient rotated back:
//   dw += g * xhat,   dx = rstd (g w - xhat mean(g w xhat)),   xhat = x rstd.
//
// Everything here is bound by HBM: each operand is read once and each result
// written once, a few flops an element.  The sines and cosines are the only
// expensive part, and they depend on (token, pair) alone: a CTA takes a few
// tokens with all their heads (Q and K, every shard), puts their sines and
// cosines into shared memory once and uses them for every head.
//
// Angles: the plan holds freq_i / 2 pi as a 64-bit fraction of a turn, so
// t * turn_i mod 2^64 is the angle's fraction of a turn, exactly reduced by
// the integer product's wrap-around (error: t times the plan's, half a unit and
// 2^-62 of the frequency, at most 1.2 * 2^-64 turns): far positions lose
// nothing, where t * freq_i in fp32 would be off by 0.03 rad at 10^6.
//
// Two kernels of each: the vector one gives a thread 16 elements of a head
// (two 8-element chunks whose pairs belong together; dh/16 lanes a head) and
// needs dh and r to be multiples of 16 and 16-byte aligned buffers; the
// other one gives a warp a head, one pair or one element a lane at a time, and
// takes any even r <= dh <= 256 at element alignment.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "tp_device.cuh"
#include "tp_internal.h"
#include "tp_launch.cuh"

namespace tpk {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHead = 256;
constexpr int kMaxPairs = kMaxHead / 2;
constexpr int kMaxTok = 4;   // tokens a CTA takes at once

// n / d for 0 <= n < 2^31 by a multiplication (the round-up method: m =
// floor(2^32 (2^s - d) / d) + 1 with s the bits of d - 1).
struct FastDiv {
  uint32_t m;
  int32_t s, d;
  FastDiv() = default;
  explicit FastDiv(int32_t div) : d(div < 1 ? 1 : div) {
    s = 0;
    while ((int64_t(1) << s) < d) ++s;
    m = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1);
  }
  __device__ __forceinline__ int32_t div(int32_t n) const {
    return static_cast<int32_t>((__umulhi(m, static_cast<uint32_t>(n)) + static_cast<uint32_t>(n)) >> s);
  }
};

struct RopeParams {
  const void *Q, *K, *dYq, *dYk;   // K (and Q) may be null with 0 rows a token
  void *Qo, *Ko;
  const float *wq, *wk;
  float* partial;                  // backward: [grid][2][dh] sums of the weight gradients
  const int32_t* pos;              // null: token index
  int32_t T, p, hq, hk, dh, r2;    // heads per shard; r2 rotated pairs
  int32_t tok, row_split;          // tokens a CTA, rows of a token a CTA
  int32_t interleaved;
  FastDiv by_hq, by_hk;
  float eps, inv_dh, amp, sign;    // sign -1: rotate back
  uint64_t turn[kMaxPairs];        // fraction of a turn per position, 2^-64 units
};

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
// Eight elements as they came from memory: loads are issued together and
// converted where they are used.
template <typename E>
struct Raw8;
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <typename E>
__device__ __forceinline__ void store8(E* p, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
template <>
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    memcpy(&w[i], &b, 4);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Sines and cosines of tokens [t0, t0 + n) into shared memory, cs[tok][pair],
// sn[tok][pair] (amplitude and direction included).
__device__ __forceinline__ void fill_angles(const RopeParams& P, int32_t t0, int32_t n, float* cs,
                                            float* sn) {
  for (int32_t i = threadIdx.x; i < n * P.r2; i += kThreads) {
    const int32_t tl = i / P.r2, pair = i - tl * P.r2;
    const int64_t pos = P.pos != nullptr ? P.pos[t0 + tl] : t0 + tl;
    const uint64_t turns = static_cast<uint64_t>(pos) * P.turn[pair];   // mod one turn
    float s, c;
    sincospif(__ll2float_rn(static_cast<long long>(turns)) * 0x1p-63f, &s, &c);
    cs[tl * kMaxPairs + pair] = P.amp * c;
    sn[tl * kMaxPairs + pair] = P.amp * P.sign * s;
  }
}

// Offset of row w of token t in Q or K: rows go shard by shard, head by head.
__device__ __forceinline__ int64_t row_offset(const RopeParams& P, int32_t t, int32_t w, bool k) {
  const int32_t h = k ? P.hk : P.hq;
  const int32_t shard = k ? P.by_hk.div(w) : P.by_hq.div(w), head = w - shard * h;
  return ((static_cast<int64_t>(shard) * P.T + t) * h + head) * P.dh;
}

// The two 8-element chunks of lane u: rotated lanes hold the pairs 8u..8u+7,
// the lanes behind them 16 elements that pass through.
struct Chunk {
  int32_t lo, hi, pair0;
  bool turn, live;
};
__device__ __forceinline__ Chunk chunk_of(const RopeParams& P, int32_t u) {
  Chunk c;
  c.live = u * 16 < P.dh;
  c.turn = u * 8 < P.r2;
  c.pair0 = u * 8;
  c.lo = c.turn && !P.interleaved ? u * 8 : u * 16;
  c.hi = c.turn && !P.interleaved ? P.r2 + u * 8 : u * 16 + 8;
  return c;
}

__device__ __forceinline__ void rotate(const float (&c)[8], const float (&s)[8], bool interleaved,
                                       float (&a)[8], float (&b)[8]) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = a[2 * i], y = a[2 * i + 1];
      a[2 * i] = x * c[i] - y * s[i];
      a[2 * i + 1] = y * c[i] + x * s[i];
      const float z = b[2 * i], w = b[2 * i + 1];
      b[2 * i] = z * c[i + 4] - w * s[i + 4];
      b[2 * i + 1] = w * c[i + 4] + z * s[i + 4];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = a[i], y = b[i];
      a[i] = x * c[i] - y * s[i];
      b[i] = y * c[i] + x * s[i];
    }
  }
}

template <int L>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ------------------------------------------------------------------ forward
template <typename E, int L, bool NORM>
__global__ void __launch_bounds__(kThreads, 3) rope_vec_kernel(const __grid_constant__ RopeParams P) {
  __shared__ __align__(16) float cs[kMaxTok * kMaxPairs];
  __shared__ __align__(16) float sn[kMaxTok * kMaxPairs];
  constexpr int ROWS = kThreads / L;
  pdl_wait();
  pdl_launch_dependents();
  const int32_t t0 = blockIdx.x * P.tok;
  const int32_t ntok = min(P.tok, P.T - t0);
  const int32_t qrows = P.p * P.hq, rows = qrows + P.p * P.hk;
  const int32_t w0 = blockIdx.y * P.row_split, w1 = w0 + min(P.row_split, rows - w0);
  const Chunk c = chunk_of(P, threadIdx.x % L);
  // A thread keeps its token and its pairs, so its sines and cosines stay in
  // registers; it takes every (ROWS / tok)-th of the token's heads.  BATCH of
  // them are loaded together (bytes in flight against HBM's latency), the
  // first ones before the angles are computed.
  const int32_t per = ROWS / P.tok, slot = threadIdx.x / L;
  const int32_t tl = slot / per, t = t0 + tl;
  const bool live = tl < ntok && c.live;
  constexpr int BATCH = sizeof(E) == 2 && !NORM ? 3 : 2;
  float cv[8], sv[8];
  const int32_t steps = (w1 - w0 + per - 1) / per;
  for (int32_t step = 0; step < steps; step += BATCH) {
    Raw8<E> ra[BATCH], rb[BATCH];
    int64_t off[BATCH];
    bool isk[BATCH];
#pragma unroll
    for (int n = 0; n < BATCH; ++n) {
      int32_t w = w0 + slot - tl * per + (step + n) * per;
      const bool in = live && w < w1;
      isk[n] = w >= qrows;
      if (isk[n]) w -= qrows;
      off[n] = -1;
      ra[n].zero();
      rb[n].zero();
      if (in) {
        off[n] = row_offset(P, t, w, isk[n]);
        const E* src = static_cast<const E*>(isk[n] ? P.K : P.Q) + off[n];
        ra[n].load(src + c.lo);
        rb[n].load(src + c.hi);
      }
    }
    if (step == 0) {
      fill_angles(P, t0, ntok, cs, sn);
      __syncthreads();
      if (c.turn && live) {
        load8(cs + tl * kMaxPairs + c.pair0, cv);
        load8(sn + tl * kMaxPairs + c.pair0, sv);
      }
    }
#pragma unroll
    for (int n = 0; n < BATCH; ++n) {
      float va[8], vb[8];
      ra[n].get(va);
      rb[n].get(vb);
      if (NORM) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += va[e] * va[e] + vb[e] * vb[e];
        ss = sum_lanes<L>(ss);
        const float rstd = rsqrtf(ss * P.inv_dh + P.eps);
        const float* w = isk[n] ? P.wk : P.wq;
        if (w != nullptr && c.live) {
          float wl[8], wh[8];
          load8(w + c.lo, wl);
          load8(w + c.hi, wh);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            va[e] = va[e] * rstd * wl[e];
            vb[e] = vb[e] * rstd * wh[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            va[e] *= rstd;
            vb[e] *= rstd;
          }
        }
      }
      if (c.turn) rotate(cv, sv, P.interleaved, va, vb);
      if (off[n] >= 0) {
        E* dst = static_cast<E*>(isk[n] ? P.Ko : P.Qo) + off[n];
        store8<E>(dst + c.lo, va);
        store8<E>(dst + c.hi, vb);
      }
    }
  }
}

// Any even r <= dh <= 256: a warp a head, lane slot s < r/2 one pair, the
// slots behind it one element each.
constexpr int kSlots = kMaxHead / 32;
struct Slot {
  int32_t e0, e1;   // elements (e1 < 0: a single one)
};
__device__ __forceinline__ Slot slot_of(const RopeParams& P, int32_t s) {
  Slot x;
  if (s < P.r2) {
    x.e0 = P.interleaved ? 2 * s : s;
    x.e1 = P.interleaved ? 2 * s + 1 : s + P.r2;
  } else {
    x.e0 = P.r2 + s;
    x.e1 = -1;
  }
  return x;
}

template <typename E, bool NORM>
__global__ void __launch_bounds__(kThreads) rope_any_kernel(const __grid_constant__ RopeParams P) {
  __shared__ __align__(16) float cs[kMaxTok * kMaxPairs];
  __shared__ __align__(16) float sn[kMaxTok * kMaxPairs];
  pdl_wait();
  pdl_launch_dependents();
  const int32_t t0 = blockIdx.x * P.tok;
  const int32_t ntok = min(P.tok, P.T - t0);
  const int32_t qrows = P.p * P.hq, rows = qrows + P.p * P.hk;
  const int32_t w0 = blockIdx.y * P.row_split, nw = min(P.row_split, rows - w0);
  const int32_t lane = threadIdx.x % 32, nslots = P.dh - P.r2;
  fill_angles(P, t0, ntok, cs, sn);
  __syncthreads();
  for (int32_t i = threadIdx.x / 32; i < ntok * nw; i += kThreads / 32) {
    const int32_t tl = i / nw;
    int32_t w = w0 + i - tl * nw;
    const bool k = w >= qrows;
    if (k) w -= qrows;
    const int64_t off = row_offset(P, t0 + tl, w, k);
    const E* src = static_cast<const E*>(k ? P.K : P.Q) + off;
    E* dst = static_cast<E*>(k ? P.Ko : P.Qo) + off;
    const float* wt = k ? P.wk : P.wq;
    float a[kSlots], b[kSlots], ss = 0.0f;
#pragma unroll
    for (int n = 0; n < kSlots; ++n) {
      a[n] = b[n] = 0.0f;
      const int32_t s = lane + 32 * n;
      if (s < nslots) {
        const Slot x = slot_of(P, s);
        a[n] = ld1(src + x.e0);
        if (x.e1 >= 0) b[n] = ld1(src + x.e1);
        ss += a[n] * a[n] + b[n] * b[n];
      }
    }
    float rstd = 1.0f;
    if (NORM) rstd = rsqrtf(sum_lanes<32>(ss) * P.inv_dh + P.eps);
#pragma unroll
    for (int n = 0; n < kSlots; ++n) {
      const int32_t s = lane + 32 * n;
      if (s >= nslots) continue;
      const Slot x = slot_of(P, s);
      if (NORM) {
        a[n] *= rstd;
        b[n] *= rstd;
        if (wt != nullptr) {
          a[n] *= wt[x.e0];
          if (x.e1 >= 0) b[n] *= wt[x.e1];
        }
      }
      if (x.e1 >= 0) {
        const float cc = cs[tl * kMaxPairs + s], sc = sn[tl * kMaxPairs + s];
        st1(dst + x.e0, a[n] * cc - b[n] * sc);
        st1(dst + x.e1, b[n] * cc + a[n] * sc);
      } else {
        st1(dst + x.e0, a[n]);
      }
    }
  }
}

// ----------------------------------------------------------------- backward
// Persistent CTAs; the weight gradients stay in registers (each lane keeps
// its 16 elements for Q and for K) until the end, then go through shared
// memory into one row of `partial` per CTA, which fold_weight_grads adds in
// CTA order: the same bits on every run.
template <typename E, int L>
__global__ void __launch_bounds__(kThreads, 2)
    norm_rope_bwd_vec_kernel(const __grid_constant__ RopeParams P) {
  __shared__ __align__(16) float cs[kMaxTok * kMaxPairs];
  __shared__ __align__(16) float sn[kMaxTok * kMaxPairs];
  __shared__ float red[kThreads / 32][kMaxHead];
  constexpr int ROWS = kThreads / L;
  pdl_wait();
  pdl_launch_dependents();
  const int32_t u = threadIdx.x % L;
  const Chunk c = chunk_of(P, u);
  const int32_t per = ROWS / P.tok;   // a thread keeps its token of the CTA's and takes every per-th head
  const int32_t tl = static_cast<int32_t>(threadIdx.x) / L / per, lane_row = threadIdx.x / L - tl * per;
  float acc[2][16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[0][e] = acc[1][e] = 0.0f;
  for (uint32_t at = blockIdx.x * P.tok; at < static_cast<uint32_t>(P.T); at += gridDim.x * P.tok) {
    const int32_t t0 = static_cast<int32_t>(at);   // (at itself may pass 2^31)
    const int32_t ntok = min(P.tok, P.T - t0);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int32_t h = k ? P.hk : P.hq, nw = P.p * h;
      const E* X = static_cast<const E*>(k ? P.K : P.Q);
      const E* DY = static_cast<const E*>(k ? P.dYk : P.dYq);
      E* DX = static_cast<E*>(k ? P.Ko : P.Qo);
      const float* wt = k ? P.wk : P.wq;
      struct Row {
        Raw8<E> xa, xb, ga, gb;
        int64_t off;
      };
      auto fetch = [&](int32_t w, Row& r) {
        const bool in = tl < ntok && w < nw && c.live;
        r.off = -1;
        r.xa.zero();
        r.xb.zero();
        r.ga.zero();
        r.gb.zero();
        if (in) {
          r.off = row_offset(P, t0 + tl, w, k != 0);
          r.xa.load(X + r.off + c.lo);
          r.xb.load(X + r.off + c.hi);
          r.ga.load(DY + r.off + c.lo);
          r.gb.load(DY + r.off + c.hi);
        }
      };
      Row cur;
      fetch(lane_row, cur);
      if (k == 0) {   // (the first rows are on their way)
        __syncthreads();   // the angles of the previous tokens are no longer read
        fill_angles(P, t0, ntok, cs, sn);
        __syncthreads();
      }
      for (int32_t base = 0; base < nw; base += per) {
        Row nxt;
        // (fp32 rows take twice the registers: loaded where they are used)
        const bool more = base + per < nw;
        if (sizeof(E) == 2 && more) fetch(base + per + lane_row, nxt);
        const bool live = cur.off >= 0;
        const int64_t off = cur.off;
        float xa[8], xb[8], ga[8], gb[8];
        cur.xa.get(xa);
        cur.xb.get(xb);
        cur.ga.get(ga);
        cur.gb.get(gb);
        if (c.turn) {
          float cv[8], sv[8];
          load8(cs + tl * kMaxPairs + c.pair0, cv);
          load8(sn + tl * kMaxPairs + c.pair0, sv);
          rotate(cv, sv, P.interleaved, ga, gb);
        }
        float wa[8], wb[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) wa[e] = wb[e] = 1.0f;
        if (wt != nullptr && c.live) {
          load8(wt + c.lo, wa);
          load8(wt + c.hi, wb);
        }
        float ss = 0.0f, gx = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ss += xa[e] * xa[e] + xb[e] * xb[e];
          gx += ga[e] * wa[e] * xa[e] + gb[e] * wb[e] * xb[e];
        }
        ss = sum_lanes<L>(ss);
        gx = sum_lanes<L>(gx);
        const float inv_dh = P.inv_dh;
        const float rstd = rsqrtf(ss * inv_dh + P.eps);
        const float m = gx * rstd * inv_dh;   // mean(g w xhat)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float ha = xa[e] * rstd, hb = xb[e] * rstd;
          acc[k][e] += ga[e] * ha;
          acc[k][8 + e] += gb[e] * hb;
          xa[e] = rstd * (ga[e] * wa[e] - ha * m);
          xb[e] = rstd * (gb[e] * wb[e] - hb * m);
        }
        if (live) {
          store8<E>(DX + off + c.lo, xa);
          store8<E>(DX + off + c.hi, xb);
        }
        if (more) {
          if (sizeof(E) == 2)
            cur = nxt;
          else
            fetch(base + per + lane_row, cur);
        }
      }
    }
  }
  // over the warp's rows, then over the warps
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
#pragma unroll
      for (int o = 16; o >= L; o /= 2)
        acc[k][e] += __shfl_xor_sync(0xffffffffu, acc[k][e], o);
    }
    __syncthreads();
    if (threadIdx.x % 32 < L && c.live) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        red[threadIdx.x / 32][c.lo + e] = acc[k][e];
        red[threadIdx.x / 32][c.hi + e] = acc[k][8 + e];
      }
    }
    __syncthreads();
    for (int32_t e = threadIdx.x; e < P.dh; e += kThreads) {
      float s = 0.0f;
#pragma unroll
      for (int n = 0; n < kThreads / 32; ++n) s += red[n][e];
      P.partial[(static_cast<int64_t>(blockIdx.x) * 2 + k) * P.dh + e] = s;
    }
  }
}

template <typename E>
__global__ void __launch_bounds__(kThreads, 2)
    norm_rope_bwd_any_kernel(const __grid_constant__ RopeParams P) {
  __shared__ __align__(16) float cs[kMaxTok * kMaxPairs];
  __shared__ __align__(16) float sn[kMaxTok * kMaxPairs];
  __shared__ float red[kThreads / 32][kMaxHead];
  pdl_wait();
  pdl_launch_dependents();
  const int32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, nslots = P.dh - P.r2;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int32_t h = k ? P.hk : P.hq, nw = P.p * h;
    const E* X = static_cast<const E*>(k ? P.K : P.Q);
    const E* DY = static_cast<const E*>(k ? P.dYk : P.dYq);
    E* DX = static_cast<E*>(k ? P.Ko : P.Qo);
    const float* wt = k ? P.wk : P.wq;
    float acc[kSlots][2];
#pragma unroll
    for (int n = 0; n < kSlots; ++n) acc[n][0] = acc[n][1] = 0.0f;
    for (uint32_t at = blockIdx.x * P.tok; at < static_cast<uint32_t>(P.T); at += gridDim.x * P.tok) {
      const int32_t t0 = static_cast<int32_t>(at);   // (at itself may pass 2^31)
      const int32_t ntok = min(P.tok, P.T - t0);
      __syncthreads();
      fill_angles(P, t0, ntok, cs, sn);
      __syncthreads();
      for (int32_t i = warp; i < ntok * nw; i += kThreads / 32) {
        const int32_t tl = i / nw;
        const int64_t off = row_offset(P, t0 + tl, i - tl * nw, k != 0);
        float x[kSlots][2], g[kSlots][2], ss = 0.0f, gx = 0.0f;
#pragma unroll
        for (int n = 0; n < kSlots; ++n) {
          x[n][0] = x[n][1] = g[n][0] = g[n][1] = 0.0f;
          const int32_t s = lane + 32 * n;
          if (s >= nslots) continue;
          const Slot q = slot_of(P, s);
          x[n][0] = ld1(X + off + q.e0);
          const float d0 = ld1(DY + off + q.e0);
          if (q.e1 >= 0) {
            x[n][1] = ld1(X + off + q.e1);
            const float d1 = ld1(DY + off + q.e1);
            const float cc = cs[tl * kMaxPairs + s], sc = sn[tl * kMaxPairs + s];
            g[n][0] = d0 * cc - d1 * sc;
            g[n][1] = d1 * cc + d0 * sc;
          } else {
            g[n][0] = d0;
          }
          ss += x[n][0] * x[n][0] + x[n][1] * x[n][1];
          gx += g[n][0] * (wt ? wt[q.e0] : 1.0f) * x[n][0];
          if (q.e1 >= 0) gx += g[n][1] * (wt ? wt[q.e1] : 1.0f) * x[n][1];
        }
        ss = sum_lanes<32>(ss);
        gx = sum_lanes<32>(gx);
        const float inv_dh = P.inv_dh;
        const float rstd = rsqrtf(ss * inv_dh + P.eps);
        const float m = gx * rstd * inv_dh;
#pragma unroll
        for (int n = 0; n < kSlots; ++n) {
          const int32_t s = lane + 32 * n;
          if (s >= nslots) continue;
          const Slot q = slot_of(P, s);
          const float h0 = x[n][0] * rstd, h1 = x[n][1] * rstd;
          acc[n][0] += g[n][0] * h0;
          acc[n][1] += g[n][1] * h1;
          st1(DX + off + q.e0, rstd * (g[n][0] * (wt ? wt[q.e0] : 1.0f) - h0 * m));
          if (q.e1 >= 0) st1(DX + off + q.e1, rstd * (g[n][1] * (wt ? wt[q.e1] : 1.0f) - h1 * m));
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kSlots; ++n) {
      const int32_t s = lane + 32 * n;
      if (s >= nslots) continue;
      const Slot q = slot_of(P, s);
      red[warp][q.e0] = acc[n][0];
      if (q.e1 >= 0) red[warp][q.e1] = acc[n][1];
    }
    __syncthreads();
    for (int32_t e = threadIdx.x; e < P.dh; e += kThreads) {
      float s = 0.0f;
#pragma unroll
      for (int n = 0; n < kThreads / 32; ++n) s += red[n][e];
      P.partial[(static_cast<int64_t>(blockIdx.x) * 2 + k) * P.dh + e] = s;
    }
  }
}

// dw[k][e] = sum over CTAs of partial[cta][k][e]: 8 elements a CTA, 32 lanes of
// rows, each lane in CTA order, then the lanes in order.
constexpr int kFoldCols = 8, kFoldLanes = kThreads / kFoldCols;
__global__ void __launch_bounds__(kThreads)
    fold_weight_grads_kernel(const float* __restrict__ partial, float* dwq, float* dwk, int32_t n,
                             int32_t dh) {
  __shared__ float red[kFoldLanes][kFoldCols];
  pdl_wait();
  pdl_launch_dependents();
  const int32_t col = blockIdx.x * kFoldCols + threadIdx.x % kFoldCols, lane = threadIdx.x / kFoldCols;
  float s = 0.0f;
  if (col < 2 * dh) {
#pragma unroll 8
    for (int32_t i = lane; i < n; i += kFoldLanes) s += partial[static_cast<int64_t>(i) * 2 * dh + col];
  }
  red[lane][threadIdx.x % kFoldCols] = s;
  __syncthreads();
  if (lane == 0 && col < 2 * dh) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < kFoldLanes; ++i) s += red[i][threadIdx.x % kFoldCols];
    float* out = col < dh ? dwq : dwk;
    if (out != nullptr) out[col < dh ? col : col - dh] = s;
  }
}

bool vec_ok(const RopeCall& a) {
  if (a.dh % 16 != 0 || (a.plan != nullptr && a.plan->rotary_dim % 16 != 0)) return false;
  const void* ptrs[] = {a.Q, a.K, a.Qo, a.Ko, a.wq, a.wk, a.dYq, a.dYk};
  for (const void* p : ptrs)
    if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0) return false;
  return true;
}

RopeParams params_of(const RopeCall& a) {
  RopeParams P{};
  P.Q = a.Q;
  P.K = a.K;
  P.dYq = a.dYq;
  P.dYk = a.dYk;
  P.Qo = a.Qo;
  P.Ko = a.Ko;
  P.wq = a.wq;
  P.wk = a.wk;
  P.partial = a.partial;
  P.pos = a.pos;
  P.T = static_cast<int32_t>(a.T);
  P.p = a.p;
  P.hq = a.hq;
  P.hk = a.hk;
  P.dh = a.dh;
  P.by_hq = FastDiv(a.hq);
  P.by_hk = FastDiv(a.hk);
  P.inv_dh = 1.0f / static_cast<float>(a.dh);
  P.eps = a.eps;
  P.amp = 1.0f;
  P.sign = a.back ? -1.0f : 1.0f;
  if (a.plan != nullptr) {
    P.r2 = a.plan->rotary_dim / 2;
    P.interleaved = a.plan->layout == TP_ROPE_INTERLEAVED;
    P.amp = a.plan->amplitude;
    for (int i = 0; i < P.r2; ++i) P.turn[i] = a.plan->turn[i];
  }
  return P;
}

template <typename E, bool NORM>
cudaError_t launch_forward(const LaunchCtx& c, const RopeCall& a, const RopeParams& P, dim3 grid) {
  if (!vec_ok(a))
    return launch_pdl(rope_any_kernel<E, NORM>, grid, dim3(kThreads), 0, c.stream, P);
  const int units = a.dh / 16;
  if (units <= 4) return launch_pdl(rope_vec_kernel<E, 4, NORM>, grid, dim3(kThreads), 0, c.stream, P);
  if (units <= 8) return launch_pdl(rope_vec_kernel<E, 8, NORM>, grid, dim3(kThreads), 0, c.stream, P);
  return launch_pdl(rope_vec_kernel<E, 16, NORM>, grid, dim3(kThreads), 0, c.stream, P);
}

template <typename E>
cudaError_t launch_backward(const LaunchCtx& c, const RopeCall& a, const RopeParams& P, dim3 grid) {
  if (!vec_ok(a))
    return launch_pdl(norm_rope_bwd_any_kernel<E>, grid, dim3(kThreads), 0, c.stream, P);
  const int units = a.dh / 16;
  if (units <= 4)
    return launch_pdl(norm_rope_bwd_vec_kernel<E, 4>, grid, dim3(kThreads), 0, c.stream, P);
  if (units <= 8)
    return launch_pdl(norm_rope_bwd_vec_kernel<E, 8>, grid, dim3(kThreads), 0, c.stream, P);
  return launch_pdl(norm_rope_bwd_vec_kernel<E, 16>, grid, dim3(kThreads), 0, c.stream, P);
}

}  // namespace

// Forward: four tokens a CTA share their angles' shared-memory pass where
// that leaves every SM a few CTAs; with few tokens one token's heads are
// spread over CTAs, one pass of rows each, since only latency counts then.
cudaError_t launch_rope(const LaunchCtx& c, const RopeCall& a) {
  RopeParams P = params_of(a);
  const int32_t rows = a.p * (a.hq + a.hk);
  const int32_t pass = vec_ok(a) ? kThreads / (a.dh <= 64 ? 4 : a.dh <= 128 ? 8 : 16) : kThreads / 32;
  const bool wide = a.T * rows >= static_cast<int64_t>(c.num_sms) * 4 * kMaxTok * pass;
  P.tok = wide ? kMaxTok : 1;
  P.row_split = wide ? rows : pass;
  if (ceil_div(rows, P.row_split) > 65535) P.row_split = ceil_div(rows, 65535);
  const dim3 grid(ceil_div(a.T, P.tok), ceil_div(rows, P.row_split));
  const bool bf16 = a.dtype == TP_BF16;
  cudaError_t e;
  if (a.norm)
    e = bf16 ? launch_forward<__nv_bfloat16, true>(c, a, P, grid)
             : launch_forward<float, true>(c, a, P, grid);
  else
    e = bf16 ? launch_forward<__nv_bfloat16, false>(c, a, P, grid)
             : launch_forward<float, false>(c, a, P, grid);
  note_launch();
  return e;
}

constexpr int kBwdCtas = 296;   // two an SM, all at once
int64_t norm_rope_bwd_ctas(int64_t T) { return T < kBwdCtas ? (T > 0 ? T : 1) : kBwdCtas; }

cudaError_t launch_norm_rope_bwd(const LaunchCtx& c, const RopeCall& a) {
  RopeParams P = params_of(a);
  const int64_t ctas = norm_rope_bwd_ctas(a.T);
  // tokens a CTA takes at once: a power of two, since they share its row slots
  P.tok = a.T >= ctas * 4 ? 4 : a.T >= ctas * 2 ? 2 : 1;
  const dim3 grid(static_cast<unsigned>(ctas));
  cudaError_t e = a.dtype == TP_BF16 ? launch_backward<__nv_bfloat16>(c, a, P, grid)
                                     : launch_backward<float>(c, a, P, grid);
  note_launch();
  if (e != cudaSuccess || (a.dwq == nullptr && a.dwk == nullptr)) return e;
  e = launch_pdl(fold_weight_grads_kernel, dim3(ceil_div(2 * a.dh, kFoldCols)), dim3(kThreads), 0, c.stream,
                 static_cast<const float*>(a.partial), a.dwq, a.dwk, static_cast<int32_t>(ctas),
                 static_cast<int32_t>(a.dh));
  note_launch();
  return e;
}

}  // namespace tpk
