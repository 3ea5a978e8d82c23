// Device parts of scored attention: which keys a row and a tile see, the
// scores' cap and bias, and the look at operand rows that are not finite.
#pragma once

#include <cuda_bf16.h>

#include <climits>
#include <cstdint>

#include "tp_device.cuh"
#include "tp_score.h"
#include "tp_softmax.cuh"

namespace tpk {

// Key blocks [jb, je) that a tile of 128 query rows visits; block j is whole
// when every row of the tile sees all of it.
struct TileSpan {
  int32_t jb, je, in_lo, in_hi;
  __device__ __forceinline__ bool whole(int32_t j) const {
    return j * kAttnTile >= in_lo && (j + 1) * kAttnTile <= in_hi;
  }
};

__device__ __forceinline__ TileSpan tile_span(const MaskPlan& m, int32_t qb, int32_t q_blocks,
                                              int32_t T, int32_t causal) {
  TileSpan s{0, 0, 0, 0};
  if (qb >= q_blocks) return s;
  if (m.rows != nullptr) {
    const int4 t = m.q_tiles[qb];
    if (t.x >= t.y) return s;
    s.jb = t.x / kAttnTile;
    s.je = (t.y + kAttnTile - 1) / kAttnTile;
    s.in_lo = t.z;
    s.in_hi = t.w;
    return s;
  }
  const int32_t hi = causal ? min((qb + 1) * kAttnTile, T) : T;
  s.je = (hi + kAttnTile - 1) / kAttnTile;
  s.in_hi = causal ? qb * kAttnTile + 1 : T;
  return s;
}

// Query tiles by falling number of key blocks, for units dealt to the CTAs in
// turns from the two ends: documents of uneven length left one CTA with twice
// the others' blocks when the tiles came in their own order (4001 tokens in
// nine documents, 32 heads: forward 110 us, 98 sorted, when this was chosen).  Every thread of the CTA
// calls this behind the wait for the plan's kernel; null where the order does
// not matter: no mask, a unit a CTA at most, or more tiles than fit (their
// units are many, and even out).
constexpr int kOrderTiles = 512;
__device__ __forceinline__ const uint16_t* order_tiles(const MaskPlan& m, int32_t tiles, int32_t T,
                                                       int32_t causal, bool one_each, uint16_t* order,
                                                       uint16_t* blocks) {
  if (m.rows == nullptr || tiles > kOrderTiles || one_each) return nullptr;
  for (int32_t t = threadIdx.x; t < tiles; t += blockDim.x) {
    const TileSpan s = tile_span(m, t, tiles, T, causal);
    blocks[t] = static_cast<uint16_t>(s.je > s.jb ? s.je - s.jb : 0);
  }
  __syncthreads();
  for (int32_t t = threadIdx.x; t < tiles; t += blockDim.x) {
    const uint32_t mine = blocks[t];
    int32_t place = 0;
    for (int32_t o = 0; o < tiles; ++o) {
      const uint32_t b = blocks[o];
      place += b > mine || (b == mine && o < t);
    }
    order[place] = static_cast<uint16_t>(t);
  }
  __syncthreads();
  return order;
}

// Keys [x, y) that query row q sees; y < 0: the row lies in no document.
__device__ __forceinline__ int2 row_span(const MaskPlan& m, int32_t q, int32_t T, int32_t causal) {
  if (m.rows != nullptr) return q < T ? m.rows[q] : make_int2(0, -1);
  return make_int2(0, causal ? min(q + 1, T) : T);
}

// Queries [x, y) that see key k; y < 0: the key lies in no document.
__device__ __forceinline__ int2 key_span(const MaskPlan& m, int32_t k, int32_t T, int32_t causal) {
  if (m.rows != nullptr) return k < T ? m.keys[k] : make_int2(0, -1);
  return make_int2(causal ? k : 0, T);
}

// A raw product -> its capped score in log2 units, of any size.  The MUFU form
// is off by up to 2^-21 of the cap in every score: less than the products' own
// rounding at caps of tens, 0.2 at a cap of 10^6.  FINE: the polynomial where
// |scale s| <= cap/2, where that is what is lost (eight instructions more).
template <bool FINE>
__device__ __forceinline__ float cap_score(float s, const ScoreConsts& S) {
  const float far = copysignf(1.0f - 2.0f * rcp_approx(1.0f + ex2(fabsf(s) * S.two_x)), s);
  if (!FINE) return S.cap_log2 * far;
  constexpr float c0 = static_cast<float>(kTanh[0]), c1 = static_cast<float>(kTanh[1]);
  constexpr float c2 = static_cast<float>(kTanh[2]), c3 = static_cast<float>(kTanh[3]);
  const float x = s * S.x_of_s, u = x * x;
  const float near = x * fmaf(u, fmaf(u, fmaf(u, c3, c2), c1), c0);
  return S.cap_log2 * (fabsf(x) <= 0.5f ? near : far);
}

// Whether all of the warp's 32 products a row are small against the cap.
__device__ __forceinline__ bool all_small(const uint32_t* v, const ScoreConsts& S) {
  float mx[2] = {0.0f, 0.0f};
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    mx[0] = max3_nan(mx[0], fabsf(__uint_as_float(v[e])), fabsf(__uint_as_float(v[e + 1])));
    mx[1] = max3_nan(mx[1], fabsf(__uint_as_float(v[e + 2])), fabsf(__uint_as_float(v[e + 3])));
  }
  return __all_sync(0xffffffffu, max3_nan(mx[0], mx[1], mx[1]) <= S.small) != 0;
}

__device__ __forceinline__ void cap_small(uint32_t (&v)[32], const ScoreConsts& S) {
  const uint64_t c0 = f2_pack(S.poly[0], S.poly[0]), c1 = f2_pack(S.poly[1], S.poly[1]);
  const uint64_t c2 = f2_pack(S.poly[2], S.poly[2]), c3 = f2_pack(S.poly[3], S.poly[3]);
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const uint64_t s = f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
    const uint64_t u = f2_mul(s, s);
    const uint64_t z = f2_mul(s, f2_fma(u, f2_fma(u, f2_fma(u, c3, c2), c1), c0));
    float a, b;
    f2_unpack(z, a, b);
    v[e] = __float_as_uint(a);
    v[e + 1] = __float_as_uint(b);
  }
}

// 32 raw products -> capped scores in log2 units.  True where the warp took
// the form of cap_score (some row's |scale s| > cap/2, or a NaN).  Columns that a
// mask hides have a say in that too; the two forms agree to cap_score's accuracy.
// HIDE, for a caller in whose cut tiles another warp sets rows that are not
// finite to 0 meanwhile, so that their products are a matter of time: where one
// is large, columns that are not in `sure` are set to 0 and it is asked again.
// (In the forward, which has no such rows, that cost 355 -> 361 us.)
template <bool FINE, bool HIDE>
__device__ __forceinline__ bool cap_chunk(uint32_t (&v)[32], const ScoreConsts& S, bool cut, uint32_t sure) {
  bool slow = !all_small(v, S);
  if (HIDE && slow && cut) {
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!((sure >> e) & 1u)) v[e] = 0;
    slow = !all_small(v, S);
  }
  if (!slow) {
    cap_small(v, S);
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(cap_score<FINE>(__uint_as_float(v[e]), S));
  }
  return slow;
}

// Columns [lo, hi) of 32 as bits.
__device__ __forceinline__ uint32_t columns_in(int32_t lo, int32_t hi) {
  lo = min(max(lo, 0), 32);
  hi = min(max(hi, 0), 32);
  return hi > lo ? (0xffffffffu >> (32 - (hi - lo))) << lo : 0u;
}

// Scores -> scores - slope2 |dist0 + e|, all in log2 units; SCALE: v holds raw
// products and is scaled too.  side: -1 every key is at or before every row of
// the tile, 1 at or behind it (the distance is then linear in e), 0 mixed.
template <bool SCALE>
__device__ __forceinline__ void bias_chunk(uint32_t* v, float scale, float slope2, float dist0,
                                           int side) {
  if (side != 0) {
    // two running pairs of biases, eight steps of 4 g each (off by at most
    // 8 * 2^-24 of the bias): one packed add and one packed fma a pair
    const float g = side < 0 ? slope2 : -slope2;
    const uint64_t sc = f2_pack(scale, scale), step = f2_pack(4.0f * g, 4.0f * g);
    uint64_t bias[2];
    bias[0] = f2_pack(g * dist0, g * (dist0 + 1.0f));
    bias[1] = f2_pack(g * (dist0 + 2.0f), g * (dist0 + 3.0f));
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const uint64_t s = f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
      uint64_t& c = bias[(e / 2) & 1];
      const uint64_t z = SCALE ? f2_fma(s, sc, c) : f2_add(s, c);
      c = f2_add(c, step);
      float a, b;
      f2_unpack(z, a, b);
      v[e] = __float_as_uint(a);
      v[e + 1] = __float_as_uint(b);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const float s = SCALE ? __uint_as_float(v[e]) * scale : __uint_as_float(v[e]);
      v[e] = __float_as_uint(fmaf(-slope2, fabsf(dist0 + static_cast<float>(e)), s));
    }
  }
}

// Columns of a 32-column chunk that are not in `seen` become -inf.
__device__ __forceinline__ void mask_chunk(uint32_t (&v)[32], uint32_t seen) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (!((seen >> e) & 1u)) v[e] = 0xff800000u;
}

// Whether row `row` (0..127) of a 128 x 128 bf16 tile in shared memory (two
// 64-column halves, 128-byte swizzle) holds an infinity or a NaN; zeroing it.
__device__ __forceinline__ uint32_t row_chunk_addr(uint32_t tile, int row, int c) {
  return tile + (c >> 3) * 16384u + row * 128u + (((c & 7) ^ (row & 7)) * 16u);
}
__device__ __forceinline__ bool row_not_finite(uint32_t tile, int row) {
  // x * 0 + a is NaN from the first infinity or NaN on (four sums: the chain
  // of one would take longer than the loads)
  __nv_bfloat162 a[4];
  const __nv_bfloat162 zero = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = zero;
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    uint32_t w[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(row_chunk_addr(tile, row, c)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 x;
      memcpy(&x, &w[i], 4);
      a[i] = __hfma2(x, zero, a[i]);
    }
  }
  a[0] = __hadd2(__hadd2(a[0], a[1]), __hadd2(a[2], a[3]));
  return __hisnan(__low2bfloat16(a[0])) || __hisnan(__high2bfloat16(a[0]));
}
__device__ __forceinline__ void zero_row(uint32_t tile, int row) {
#pragma unroll
  for (int c = 0; c < 16; ++c)
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(row_chunk_addr(tile, row, c)),
                 "r"(0)
                 : "memory");
}

}  // namespace tpk
