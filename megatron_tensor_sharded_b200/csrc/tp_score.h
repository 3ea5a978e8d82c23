// Scored attention: what the kernels share with the launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "tp_internal.h"

namespace tpk {

constexpr int kAttnTile = 128;   // query rows and key rows of a tile

// The mask's plan (tp_attention_mask): per query row the keys it sees, [x, y)
// (y < 0: the row lies in no document); per tile of 128 query rows {least x,
// greatest y, greatest x, least y}, the first two over rows in a document; per
// key the queries [x, y) that see it, and per tile of 128 keys the query tiles
// [x, y) that may see one of them.
struct MaskPlan {
  int2* rows;
  int2* keys;
  int4* q_tiles;
  int2* k_tiles;
};
inline size_t mask_align(size_t n) { return (n + 255) & ~size_t(255); }
inline MaskPlan mask_plan(const void* buf, int64_t T) {
  if (buf == nullptr) return MaskPlan{};
  const size_t tiles = static_cast<size_t>(ceil_div(T, kAttnTile));
  uint8_t* b = static_cast<uint8_t*>(const_cast<void*>(buf));
  const size_t r = mask_align(static_cast<size_t>(T) * sizeof(int2));
  return MaskPlan{reinterpret_cast<int2*>(b), reinterpret_cast<int2*>(b + r),
                  reinterpret_cast<int4*>(b + 2 * r),
                  reinterpret_cast<int2*>(b + 2 * r + mask_align(tiles * sizeof(int4)))};
}
inline size_t mask_bytes(int64_t T) {
  const size_t tiles = static_cast<size_t>(ceil_div(T, kAttnTile));
  return 2 * mask_align(static_cast<size_t>(T) * sizeof(int2)) + mask_align(tiles * sizeof(int4)) +
         mask_align(tiles * sizeof(int2));
}

// tanh(x)/x in u = x^2 on [0, 1/4]: least-squares fit reweighted to the smallest
// relative error, 5.5e-7
constexpr double kTanh[4] = {0.999999463558197, -0.33326318860054016, 0.13190296292304993,
                             -0.04440222680568695};

// Caps up to 55: what the MUFU form loses (2^-21 of the cap, 2.6e-5) is less than
// the rounding of the products' fp32 sums, and the finer form costs up to a
// quarter of the forward's time where scores lie near the cap (4096 tokens, 64
// heads, queries of standard deviation 8, cap 50: 480 us, 597 with it).
constexpr float kCoarseCapLog2 = 80.0f;
enum { kNoCap = 0, kCoarseCap = 1, kFineCap = 2 };

// Scores z of a raw product s = q.k, in units of log2: z = log2(e) *
// (cap tanh(scale s / cap) - slope |i - j|).
struct ScoreConsts {
  float scale_log2;    // log2(e) scale
  float poly[4];       // z = s (p0 + u (p1 + u (p2 + u p3))), u = s^2, for |s| <= small
  float small;         // scale |s| / cap <= 1/2; -1: a poly is not a normal number
  float two_x;         // 2 log2(e) scale / cap: tanh by e^(2x) beyond it
  float cap_log2;      // log2(e) cap (0: scores are not capped)
  float scale;         // scale itself (gradients)
  float x_of_s;        // scale / cap
};
inline ScoreConsts score_consts(float scale, float cap) {
  const double l2e = 1.4426950408889634;
  ScoreConsts k{};
  k.scale = scale;
  k.scale_log2 = static_cast<float>(l2e * scale);
  if (cap > 0.0f) {
    const double x = static_cast<double>(scale) / cap;
    for (int i = 0; i < 4; ++i) k.poly[i] = static_cast<float>(l2e * cap * kTanh[i] * std::pow(x, 2 * i + 1));
    k.small = static_cast<float>(0.5 / x);
    // (scale/cap of 10^6 takes poly[3] past fp32 -- 0 times it is NaN --, a cap of
    // 10^6 below it; scores then go through x_of_s one by one)
    for (float c : k.poly)
      if (!std::isnormal(c)) k.small = -1.0f;
    k.two_x = static_cast<float>(2.0 * l2e * x);
    k.cap_log2 = static_cast<float>(l2e * cap);
    k.x_of_s = static_cast<float>(x);
  }
  return k;
}

inline int cap_form(const ScoreConsts& k) {
  return !(k.cap_log2 > 0.0f) ? kNoCap : k.cap_log2 <= kCoarseCapLog2 && k.small > 0.0f ? kCoarseCap : kFineCap;
}

struct ScoreCall {
  const void *Q, *K, *V;
  void* O;
  float* LSE;              // forward: may be null
  const void* dO;          // backward
  void *dQ, *dK, *dV;
  float* delta;            // backward: [p][hq][T] scratch
  uint8_t* k_bad;          // backward: [p][hkv][T] scratch
  float* part;             // backward: score_dkv_bytes() of scratch
  int64_t T;
  int p, hq, hkv;          // heads per shard
  bool causal;
  float scale, cap;
  const float* slopes;     // [p*hq] or null
  const void* mask;        // plan or null
};

struct DecodeCall {
  const void *Q, *Kn, *Vn;   // Kn, Vn: the tokens to append, or null
  void *Kc, *Vc, *O;
  float *LSE, *part;         // LSE may be null; part: decode_part_bytes()
  const int32_t* len;
  int64_t B, capacity;
  int p, hq, hkv;            // heads per shard
  float scale, cap;
  const float* slopes;
};
constexpr int kMaxDecodeCtas = 512;
constexpr int kDecodeTile = 64;   // keys
// Query heads of an item: 8 where one column tile holds the group, else 16; and
// the items of a sequence in a shard.
inline int decode_rows(int group) { return group <= 8 ? 8 : 16; }
inline int64_t decode_items(int hq, int hkv) {
  const int rows = decode_rows(hq / hkv);
  return static_cast<int64_t>(hkv) * ((hq / hkv + rows - 1) / rows);
}
// CTAs of a decode call, and the bytes of their partials.
int64_t decode_ctas(int num_sms, int64_t B, int64_t capacity, int p, int hq, int hkv);
size_t decode_part_bytes(int64_t ctas);
tp_status launch_attention_decode(const LaunchCtx& c, const DecodeCall& a);

cudaError_t launch_attention_mask(const LaunchCtx& c, const int32_t* off, int n_docs,
                                  const int32_t* prefix, bool causal, void* mask, int64_t T);
// Scratch of the backward's dK and dV for the call's sizes; kScoreDkvCtas: the
// SMs of a B200.
constexpr int kScoreDkvCtas = 148;
// A dkv unit's loads, start and stores, in steps (1999 tokens of five documents,
// 64/8 heads, whole backward, when this was chosen: 2 230 us, 4 226, 6 226, 8 228; a smaller one 49,
// 42, 41, 41).
constexpr int kUnitCost = 4;
int64_t score_dkv_ctas(const ScoreCall& a);
size_t score_dkv_bytes(const ScoreCall& a);
tp_status launch_attention_scored(const LaunchCtx& c, const ScoreCall& a);
tp_status launch_attention_scored_bwd(const LaunchCtx& c, const ScoreCall& a);

}  // namespace tpk
