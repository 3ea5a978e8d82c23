// Backward of scored attention (sm_100a): four launches.
//
// With P = exp(z - LSE), D_i = sum_d dO_id O_id and t the cap's tanh,
//   dV_j = sum_i P_ij dO_i,   dS_ij = P_ij (dO_i.v_j - D_i) (1 - t_ij^2),
//   dQ_i = scale sum_j dS_ij k_j,   dK_j = scale sum_i dS_ij q_i,
// dK and dV summed over the query heads that share a key/value head.
//
// 1. score_delta_kernel: D, and which rows of Q, dO and K hold infinities or
//    NaN, one pass over O, dO, Q and K (HBM-bound).
// 2. tc_scored_dkv_kernel: a unit is (shard, key/value head, 128 keys) and
//    walks every query tile that sees them, for every query head of the
//    group: dK and dV stay in TMEM from the first to the last, so the sum
//    over heads costs nothing and has a fixed order; dkv_join_kernel adds what
//    units on several CTAs left.
// 3. tc_scored_dq_kernel: a unit is (shard, query head, 128 queries) and walks
//    its key blocks with dQ in TMEM.
// Scores and probabilities are recomputed in both: seven products a tile
// instead of the five that one kernel with atomic adds to dQ would need, in
// exchange for the same bits on every run, no fp32 dQ in memory and no pass
// that converts it.  Both are bound by a step's chain of the tensor cores' work
// (4 and 3 products of 128 x 128 x 128 a tile, 57% and 50% of the time) and the
// softmax's arithmetic, which overlap as far as TMEM's 512 columns allow.
// 4096 causal tokens, 32 heads, cap: 271 and 230 us; with D, 582 in all.
//
// D comes from O as it was stored: dQ and dK are 0.0027 off in the 2-norm where
// an fp32 O would leave the 0.0024 of P's, dS's and their own rounding.
//
// dkv computes the transposed tiles S^T = K Q^T and dP^T = V dO^T: a thread
// then owns a key row, and P^T and dS^T, left in TMEM as bf16, are the A
// operands of dV += P^T dO and dK += dS^T Q, whose B operands are the tiles
// that S^T and dP^T read: no operand is transposed or written to shared
// memory.  dq likewise: dQ += dS K.  The sixteen arithmetic warps split a tile
// by column quarters; each quarter's bf16 result goes over the first half of
// its own scores, so the quarters never wait for one another.  S^T is free as
// soon as the warps hold it in registers, since P^T and dS^T both go over dP^T:
// the next S^T runs while they form P^T, and dV, dK and the next dP^T while
// they form the next P^T.  (With P^T over S^T, the next S^T waited for dV: 653
// us for the whole backward against 624 when that was changed.)
//
// A query that sees one key has P = 1 and dS = 0 exactly; dP - D leaves the
// rounding of two sums there, so w is set to 0 (times 0: a NaN stays).
//
// Masks, and rows that hold infinities or NaN outside what is seen, as in the
// forward kernel; here rows of Q and dO (dkv) and of K (dq) that the first kernel
// marked are set to 0 in tiles that a mask cuts, and what does see one is made
// NaN (through `hit`, through dS).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "tp_device.cuh"
#include "tp_internal.h"
#include "tp_launch.cuh"
#include "tp_score.cuh"
#include "tp_score.h"
#include "tp_softmax.cuh"

namespace tpk {
namespace {

constexpr int DH = 128;
constexpr int BT = kAttnTile;                // rows of a tile, keys or queries
constexpr int NA = 3;                        // ring slots of the tile that the next scores need early (Q; K)
constexpr int NB = 2;                        // and of its partner (dO; V)
constexpr int TILE_BYTES = 128 * 128 * 2;
constexpr int HALF_BYTES = TILE_BYTES / 2;
constexpr int VEC_BYTES = 2 * BT * 4;        // per slot: -LSE log2 e, -D
// 224 KB of tiles: no room to round the start up, it has to be aligned (checked)
constexpr int TILES_BYTES = (2 + NA + NB) * TILE_BYTES;
constexpr int SMEM_BYTES = TILES_BYTES + NB * VEC_BYTES + 512;
static_assert(2 * kOrderTiles * 2 <= NB * VEC_BYTES, "dq keeps its order of tiles in place of the vectors");
constexpr int NUM_THREADS = 640;
constexpr int ARITH = 512;                   // threads that form P and dS
constexpr uint32_t IDESC_KK = idesc_bf16_f32(BT, BT, 0, 0);   // both operands along head_dim
constexpr uint32_t IDESC_KN = idesc_bf16_f32(BT, DH, 0, 1);   // A in TMEM, B rows x head_dim
// Of every eight pairs of probabilities, those whose 2^x runs on the FMA pipe:
// none with the cap, whose own arithmetic there (11 clocks of a scheduler an
// element against the MUFU unit's 8) is the longer already.
template <int CAP>
constexpr int kPolyPairs = CAP ? 0 : 2;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWholeUnits = 6;                // units a CTA from which none is cut
constexpr int kCut = 1, kFirst = 2, kLast = 4, kEnd = 8;   // a step: cut by a mask; its unit's; the share's last
constexpr int PART_FLOATS = 2 * BT * DH;      // dV and dK of a key tile

struct BwdParams {
  int32_t T, p, hq, hkv, group, tiles, num_units, causal;
  int32_t whole;            // dkv: units are not cut
  MaskPlan mask;
  ScoreConsts s;
  float neg_inv_cap2;       // -(cap log2 e)^-2: 1 - tanh^2 = 1 + z^2 times it
  const float* slopes;
  const float* LSE;
  const float* delta;
  const uint8_t* k_bad;     // rows of K that hold an infinity or a NaN
  __nv_bfloat16 *dQ, *dK, *dV;
  float* part;              // dkv: [cta][slot][dV, dK][128][head_dim] of units that lie on several CTAs
  int4* cuts;               // dkv: where each CTA's share begins {key tile, head, step, steps of the unit}
  int64_t* total;           // dkv: steps of all units
  WaitCtl wait;
  int64_t debug_drop;
};

__device__ __forceinline__ int32_t unit_of(int32_t r) {
  const int32_t g = static_cast<int32_t>(gridDim.x), b = static_cast<int32_t>(blockIdx.x);
  return r * g + ((r & 1) ? g - 1 - b : b);
}

// A product of two shared-memory tiles along head_dim: D = A B^T.
__device__ __forceinline__ void mma_tiles(uint32_t d, uint32_t a, uint32_t b) {
  const uint32_t al = desc_lo(a, 16), bl = desc_lo(b, 16);
#pragma unroll
  for (int kk = 0; kk < DH / 16; ++kk) {
    const uint32_t off = desc_step((kk >> 2) * HALF_BYTES + (kk & 3) * 32);
    tc_mma_f16_lo(d, al + off, bl + off, IDESC_KK, kk > 0 ? 1u : 0u);
  }
}
// D (+)= A B with A (bf16, each column quarter at its 32 columns' start) in
// TMEM and B's 128 rows the contraction.
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint32_t b, bool add) {
  const uint32_t bl = desc_lo(b, HALF_BYTES);
#pragma unroll
  for (int kk = 0; kk < BT / 16; ++kk)
    tc_mma_f16_ts_lo(d, a + (kk >> 1) * 32 + (kk & 1) * 8, bl + desc_step(kk * 16 * 128), IDESC_KN,
                     (add || kk > 0) ? 1u : 0u);
}

__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                          int32_t head, int32_t row, int32_t shard) {
  for (int c = 0; c < 2; ++c)
    tma_load_3d(dst + c * HALF_BYTES, map, bar, head * DH + c * 64, row, shard);
}

// 32 raw products -> P as bf16 pairs in pk and w = P (1 - tanh^2).  nl(e):
// -LSE log2 e of columns e .. e + 3; seen: the columns that count where a mask
// cuts the tile, sure: those of them whose row of the other operand is finite
// (its rows that are not are set to 0 while the scores are formed, so whether
// they are NaN here is a matter of time: they must not choose the cap's form).
template <int CAP, bool BIAS, typename NegLse>
__device__ __forceinline__ void prob_chunk(uint32_t (&v)[32], float (&w)[32], uint32_t (&pk)[16],
                                           const BwdParams& P, float slope2, float dist0, int side,
                                           bool cut, uint32_t seen, uint32_t sure, NegLse nl) {
  if (CAP) {
    cap_chunk<CAP == kFineCap, true>(v, P.s, cut, sure);
    const uint64_t ic = f2_pack(P.neg_inv_cap2, P.neg_inv_cap2), one = f2_pack(1.0f, 1.0f);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const uint64_t z = f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
      f2_unpack(f2_fma(f2_mul(z, z), ic, one), w[e], w[e + 1]);
    }
  }
  if (BIAS) bias_chunk<!CAP>(v, P.s.scale_log2, slope2, dist0, side);
  const uint64_t sc2 = f2_pack(P.s.scale_log2, P.s.scale_log2);
  uint64_t n[2];
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    if (e % 4 == 0) nl(e, n[0], n[1]);
    uint64_t x = f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
    x = CAP || BIAS ? f2_add(x, n[(e / 2) & 1]) : f2_fma(x, sc2, n[(e / 2) & 1]);
    float a, b;
    if ((e / 2) % 8 < kPolyPairs<CAP>) {
      f2_unpack(exp2_poly5<true>(x), a, b);
    } else {
      float x0, x1;
      f2_unpack(x, x0, x1);
      a = ex2(x0);
      b = ex2(x1);
    }
    v[e] = __float_as_uint(a);
    v[e + 1] = __float_as_uint(b);
  }
  if (cut) {   // (the cap's derivative of what is not seen may be NaN)
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!((seen >> e) & 1u)) {
        v[e] = 0;
        if (CAP) w[e] = 0.0f;
      }
  }
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float a = __uint_as_float(v[e]), b = __uint_as_float(v[e + 1]);
    pk[e / 2] = pack2(a, b);
    if (CAP) {
      f2_unpack(f2_mul(f2_pack(a, b), f2_pack(w[e], w[e + 1])), w[e], w[e + 1]);
    } else {
      w[e] = a;
      w[e + 1] = b;
    }
  }
}

// 32 products dP -> dS = w (dP - D) as bf16 pairs; nd(e): -D of columns e .. e + 3.
template <typename NegDelta>
__device__ __forceinline__ void grad_chunk(uint32_t (&v)[32], const float (&w)[32], uint32_t (&pk)[16],
                                           bool cut, uint32_t seen, NegDelta nd) {
  uint64_t n[2];
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    if (e % 4 == 0) nd(e, n[0], n[1]);
    const uint64_t x = f2_add(f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), n[(e / 2) & 1]);
    float a, b;
    f2_unpack(f2_mul(x, f2_pack(w[e], w[e + 1])), a, b);
    v[e] = __float_as_uint(a);
    v[e + 1] = __float_as_uint(b);
  }
  if (cut) {   // 0 * NaN from what is not seen
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!((seen >> e) & 1u)) v[e] = 0;
  }
#pragma unroll
  for (int e = 0; e < 32; e += 2)
    pk[e / 2] = pack2(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
}

// 32 accumulator columns of the thread's row, times f, to bf16 at dst.
__device__ __forceinline__ void store_part_row(uint32_t taddr, float f, bool store,
                                               __nv_bfloat16* dst) {
  uint32_t v[32];
  tmem_ld_32x32b_x32(taddr, v);
  tmem_ld_wait();
  if (!store) return;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = pack2(__uint_as_float(v[g * 8 + 2 * i]) * f, __uint_as_float(v[g * 8 + 2 * i + 1]) * f);
    *reinterpret_cast<uint4*>(dst + g * 8) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

__device__ __forceinline__ void lds4(uint32_t addr, uint64_t& a, uint64_t& b) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr));
}
__device__ __forceinline__ void sts(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// The same columns in fp32.
__device__ __forceinline__ void keep_part_row(uint32_t taddr, float f, float* dst) {
  uint32_t v[32];
  tmem_ld_32x32b_x32(taddr, v);
  tmem_ld_wait();
#pragma unroll
  for (int g = 0; g < 8; ++g)
    *reinterpret_cast<float4*>(dst + g * 4) =
        make_float4(__uint_as_float(v[g * 4]) * f, __uint_as_float(v[g * 4 + 1]) * f,
                    __uint_as_float(v[g * 4 + 2]) * f, __uint_as_float(v[g * 4 + 3]) * f);
}

// ------------------------------------------------------------------ delta
// D[shard][head][t] = sum over the head of dO * O, NaN where the query's row of
// Q holds an infinity or a NaN (one of dO makes D one by itself); and for each
// row of K whether it does.  The kernels below look at a row in shared memory
// only where these say so.  (Looked at there in every tile that a mask cuts,
// they bound the backward of short documents: dK and dV of 1999 tokens in five
// took 149 us instead of 109.)
// 16 lanes a row, four rows of each lane loaded together.
constexpr int DELTA_ROWS = 64;   // rows of a CTA
// 0 if the eight values are finite, else NaN
__device__ __forceinline__ float zero_or_nan(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  __nv_bfloat162 a = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 x;
    memcpy(&x, &w[i], 4);
    a = __hfma2(x, __floats2bfloat162_rn(0.0f, 0.0f), a);
  }
  return __low2float(a) + __high2float(a);
}
// element of [shard][heads][T] that row [shard][t][head] is
__device__ __forceinline__ int64_t by_head(int64_t row, int64_t rows, int32_t T, int32_t heads) {
  int64_t st, shard;   // st = shard * T + t
  if (rows >> 31) {
    st = row / heads;
    shard = st / T;
  } else {
    st = static_cast<uint32_t>(row) / static_cast<uint32_t>(heads);
    shard = static_cast<uint32_t>(st) / static_cast<uint32_t>(T);
  }
  return (shard * heads + (row - st * heads)) * T + (st - shard * T);
}
__device__ __forceinline__ void load_rows(uint4 (&v)[4], const __nv_bfloat16* x, int64_t row0,
                                          int64_t rows, int lane) {
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const int64_t row = row0 + n * 16;
    v[n] = make_uint4(0, 0, 0, 0);
    if (row < rows) v[n] = *reinterpret_cast<const uint4*>(x + row * DH + lane * 8);
  }
}
// blocks [0, q_blocks): rows of Q; the others: of K
__global__ void __launch_bounds__(256)
    score_delta_kernel(const __nv_bfloat16* __restrict__ O, const __nv_bfloat16* __restrict__ dO,
                       const __nv_bfloat16* __restrict__ Q, const __nv_bfloat16* __restrict__ K,
                       float* __restrict__ delta, uint8_t* __restrict__ k_bad, uint32_t q_blocks,
                       int64_t shard_rows, int32_t T, int32_t hq, int32_t hkv) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x % 16;
  if (blockIdx.x >= q_blocks) {
    const int64_t rows = shard_rows * hkv;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x - q_blocks) * DELTA_ROWS + threadIdx.x / 16;
    uint4 k[4];
    load_rows(k, K, row0, rows, lane);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      float z = zero_or_nan(k[n]);
#pragma unroll
      for (int o = 8; o > 0; o /= 2) z += __shfl_xor_sync(0xffffffffu, z, o);
      const int64_t row = row0 + n * 16;
      if (lane == 0 && row < rows) k_bad[by_head(row, rows, T, hkv)] = z != z;
    }
    return;
  }
  const int64_t rows = shard_rows * hq;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * DELTA_ROWS + threadIdx.x / 16;
  uint4 a[4], b[4], q[4];
  load_rows(a, O, row0, rows, lane);
  load_rows(b, dO, row0, rows, lane);
  load_rows(q, Q, row0, rows, lane);
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const uint32_t x[4] = {a[n].x, a[n].y, a[n].z, a[n].w}, y[4] = {b[n].x, b[n].y, b[n].z, b[n].w};
    float s = zero_or_nan(q[n]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s += __uint_as_float(x[i] << 16) * __uint_as_float(y[i] << 16);
      s += __uint_as_float(x[i] & 0xffff0000u) * __uint_as_float(y[i] & 0xffff0000u);
    }
#pragma unroll
    for (int o = 8; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int64_t row = row0 + n * 16;
    if (lane == 0 && row < rows) delta[by_head(row, rows, T, hq)] = s;
  }
}

// ---------------------------------------------------------------- dK and dV
// Units, ordered by key tile (causal: the first keys are seen by most) and then
// (shard, key/value head), lie behind one another on a line of steps (a query
// head's query tile each, and kUnitCost for the loads and stores of the unit);
// every CTA gets an equal stretch of it.  A unit that the end of a stretch cuts
// leaves fp32 partials (slot 0: the part that a CTA finds begun, slot 1: the
// one that it begins), which dkv_join_kernel adds in the order of the CTAs.
// Handed out whole instead, units leave SMs idle where there are few of them or
// where documents make them differ: 369 us for the whole backward against 244
// (when this was chosen) for 1999 tokens of five documents, 64 query and 8
// key/value heads.  But a cut
// costs a store, a load and a sum of 128 KB, and where the CTAs take many units
// each, in turns from the two ends, their sums are even anyway: P.whole
// (kWholeUnits a CTA, no mask): 616 us against 648 cut, for 4096 tokens and 32
// heads.
__device__ __forceinline__ int2 key_tiles(const BwdParams& P, int32_t kb) {
  if (P.mask.rows != nullptr) return P.mask.k_tiles[kb];
  return make_int2(P.causal ? kb : 0, P.tiles);
}
__device__ __forceinline__ int64_t share_of(int64_t total, int64_t c, int64_t ctas) {
  return total * c / ctas;
}

__device__ __forceinline__ int4 lds_int4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts4(uint32_t addr, int a, int b, int c, int d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

struct Segment {
  int32_t kb, hh, shard, kvh, ia, ni;   // query tiles [ia, ia + ni)
  int32_t s0, s1, steps;                // steps [s0, s1) of the unit's
  uint32_t left;                        // of the CTA's share, from s0 on
  int32_t turn;
  __device__ __forceinline__ uint32_t cost() const { return static_cast<uint32_t>(steps + kUnitCost - s0); }
  __device__ __forceinline__ void set(const BwdParams& P) {
    const int2 t = key_tiles(P, kb);
    ia = t.x;
    ni = t.y - t.x;
    steps = P.group * ni;
    shard = hh / P.hkv;
    kvh = hh - shard * P.hkv;
    s1 = left < static_cast<uint32_t>(steps - s0) ? s0 + static_cast<int32_t>(left) : steps;
  }
  // start: {kb, hh, s0, left}
  __device__ __forceinline__ void begin(const BwdParams& P, int4 start) {
    kb = start.x;
    hh = start.y;
    s0 = start.z;
    left = static_cast<uint32_t>(start.w);
    turn = 0;
    if (P.whole) {
      take(P);
      return;
    }
    if (left > 0) set(P);
  }
  __device__ __forceinline__ bool last() const { return left <= cost(); }
  // P.whole: the CTA's turn-th unit
  __device__ __forceinline__ void take(const BwdParams& P) {
    const int32_t u = unit_of(turn), heads = P.p * P.hkv;
    left = 0;
    if (u >= P.num_units) return;
    kb = u / heads;
    hh = u - kb * heads;
    s0 = 0;
    left = 0x7fffffffu;
    set(P);
    if (unit_of(turn + 1) >= P.num_units) left = cost();
  }
  __device__ __forceinline__ void next(const BwdParams& P) {
    if (P.whole) {
      ++turn;
      take(P);
      return;
    }
    if (last()) {
      left = 0;
      return;
    }
    left -= cost();
    s0 = 0;
    if (++hh == P.p * P.hkv) {
      hh = 0;
      do {
        if (++kb >= P.tiles) {   // (a mask that is none)
          left = 0;
          return;
        }
        const int2 t = key_tiles(P, kb);
        ni = t.y - t.x;
      } while (ni <= 0);
    }
    set(P);
  }
  __device__ __forceinline__ bool whole() const { return s0 == 0 && s1 == steps; }
};

// This CTA's share of the line, by one warp; -> {kb, hh, s0, left} (lane 0).
__device__ __forceinline__ int4 find_share(const BwdParams& P, int lane) {
  const int64_t heads = static_cast<int64_t>(P.p) * P.hkv;
  int64_t total = 0;
  for (int32_t k0 = 0; k0 < P.tiles; k0 += 32) {
    const int2 t = k0 + lane < P.tiles ? key_tiles(P, k0 + lane) : make_int2(0, 0);
    int64_t x = t.y > t.x ? heads * (static_cast<int64_t>(P.group) * (t.y - t.x) + kUnitCost) : 0;
#pragma unroll
    for (int o = 16; o > 0; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
    total += x;
  }
  const int64_t w0 = share_of(total, blockIdx.x, gridDim.x);
  const int64_t w1 = share_of(total, blockIdx.x + 1, gridDim.x);
  int4 found = make_int4(0, 0, 0, 0);
  int64_t done = 0;
  for (int32_t k0 = 0; k0 < P.tiles && done <= w0 && w0 < w1; k0 += 32) {
    const int2 t = k0 + lane < P.tiles ? key_tiles(P, k0 + lane) : make_int2(0, 0);
    const int64_t steps = t.y > t.x ? static_cast<int64_t>(P.group) * (t.y - t.x) + kUnitCost : 0;
    int64_t x = heads * steps;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const int64_t before = done + x - heads * steps, at = w0 - before;
    const bool mine = steps > 0 && at >= 0 && at < heads * steps;
    const int32_t hh = mine ? static_cast<int32_t>(at / steps) : 0;
    const int32_t s0 = mine ? static_cast<int32_t>(at - hh * steps) : 0;
    const uint32_t who = __ballot_sync(0xffffffffu, mine);
    if (who != 0) {
      const int src = __ffs(who) - 1;
      found = make_int4(k0 + src, __shfl_sync(0xffffffffu, hh, src), __shfl_sync(0xffffffffu, s0, src),
                        static_cast<int32_t>(w1 - w0));
    }
    done += __shfl_sync(0xffffffffu, x, 31);
  }
  if (lane == 0) {
    Segment x;
    x.begin(P, found);
    if (x.left > 0 && x.s0 >= x.steps) x.next(P);   // begins behind a unit's steps
    found = make_int4(x.kb, x.hh, x.s0, static_cast<int32_t>(x.left));
    P.cuts[blockIdx.x] = x.left > 0 ? make_int4(x.kb, x.hh, x.s0, x.steps) : make_int4(0, 0, 0, 0);
    if (blockIdx.x == 0) *P.total = total;
  }
  return found;
}

template <int CAP, bool BIAS>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    tc_scored_dkv_kernel(const __grid_constant__ CUtensorMap mapQ,
                         const __grid_constant__ CUtensorMap mapK,
                         const __grid_constant__ CUtensorMap mapV,
                         const __grid_constant__ CUtensorMap mapdO,
                         const __grid_constant__ BwdParams P) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t base = smem_u32(smem_raw);
  if ((base & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(P.wait.err, kErrSmem);
    return;
  }
  const uint32_t sK = base, sV = base + TILE_BYTES;
  auto sQ = [&](uint32_t n) { return base + (2 + n % NA) * TILE_BYTES; };
  auto sdO = [&](uint32_t n) { return base + (2 + NA + n % NB) * TILE_BYTES; };
  auto vec = [&](uint32_t n, int which) {
    return base + TILES_BYTES + (n % NB) * VEC_BYTES + which * BT * 4;
  };
  uint8_t* const ctrl = smem_raw + TILES_BYTES + NB * VEC_BYTES;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(ctrl);
  const uint32_t kv_full = smem_u32(&bars[0]), kv_empty = smem_u32(&bars[1]);
  auto q_full = [&](uint32_t n) { return smem_u32(&bars[2 + n % NA]); };
  auto q_empty = [&](uint32_t n) { return smem_u32(&bars[5 + n % NA]); };
  auto do_full = [&](uint32_t n) { return smem_u32(&bars[8 + n % NB]); };
  auto do_empty = [&](uint32_t n) { return smem_u32(&bars[10 + n % NB]); };
  auto vec_full = [&](uint32_t n) { return smem_u32(&bars[12 + n % NB]); };
  const uint32_t s_full = smem_u32(&bars[14]), s_free = smem_u32(&bars[15]);
  const uint32_t dp_full = smem_u32(&bars[16]), ds_full = smem_u32(&bars[17]);
  const uint32_t acc_full = smem_u32(&bars[18]), acc_empty = smem_u32(&bars[19]);
  const uint32_t drain = smem_u32(&bars[20]);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 8 * 21);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* const bad = tmem_slot + 4;        // [NB][4]: its rows of dO or Q that are not finite
  // [3][4]: keys that see one, by unit number mod 3 (set by any column
  // quarter's thread of the key, read by all at the unit's end; cleared two
  // units ahead, when the last reader of the slot has moved on)
  uint32_t* const hit = tmem_slot + 4 + NB * 4;
  // what warps 2 and 3 tell the arithmetic warps, who then need not keep it:
  // [NB] of each step {query tile, kCut | ... | kEnd, slope log2 e, -}, and
  // [4] of each unit {key tile, head, where its sums go: -1 dK and dV, else the
  // slot of the partials, -}
  const uint32_t about = smem_u32(ctrl) + 320, about_unit = about + NB * 16;
  // [NB][4]: its queries that see one key only
  volatile uint32_t* const lone = reinterpret_cast<volatile uint32_t*>(ctrl + 464);
  const uint32_t share = smem_u32(ctrl) + 448;   // find_share's {kb, hh, s0, left}

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    mbar_init(kv_empty, 1);
    for (int s = 0; s < NA; ++s) {
      mbar_init(q_full(s), 1);
      mbar_init(q_empty(s), 1);
    }
    for (int s = 0; s < NB; ++s) {
      mbar_init(do_full(s), 1);
      mbar_init(do_empty(s), 1);
      mbar_init(vec_full(s), 64);
    }
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(s_free, ARITH);
    mbar_init(ds_full, ARITH);
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, ARITH);
    mbar_init(drain, 1);
    *abort_flag = 0;
    for (int i = 0; i < 12; ++i) hit[i] = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&mapQ);
    tma_prefetch_map(&mapK);
    tma_prefetch_map(&mapV);
    tma_prefetch_map(&mapdO);
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  const uint32_t tS = tm, tdP = tm + 128, tdV = tm + 256, tdK = tm + 384;
  pdl_wait();
  pdl_launch_dependents();
  if (warp == 0) {
    const int4 x = P.whole ? make_int4(0, 0, 0, unit_of(0) < P.num_units) : find_share(P, lane);
    if (lane == 0) sts4(share, x.x, x.y, x.z, x.w);
  }
  __syncthreads();
  const int4 start = lds_int4(share);

  // 96 registers a thread at launch: 128 x 64 + 512 x 104 <= 640 x 96
  if (warp < 4) {
    regs_shrink<64>();
    if (warp == 0) {
      if (lane == 0) {
        // ---------------------------------------------------------- producer
        uint32_t nu = 0, n = 0, nq = 0;   // nq: loads of Q
        bool ok = true;
        Segment x;
        for (x.begin(P, start); ok && x.left > 0; x.next(P)) {
          if (!wait_asleep(kv_empty, (nu & 1) ^ 1u, abort_flag, P.wait, kErrWaitAttn)) break;
          mbar_arrive_expect_tx(kv_full, 2 * TILE_BYTES);
          load_tile(sK, &mapK, kv_full, x.kvh, x.kb * BT, x.shard);
          load_tile(sV, &mapV, kv_full, x.kvh, x.kb * BT, x.shard);
          ++nu;
          {
            int32_t head = x.kvh * P.group + x.s0 / x.ni, i = x.ia + x.s0 % x.ni;
            for (int32_t st = x.s0; st < x.s1; ++st, ++n) {
              if (!wait_asleep(q_empty(n), ((n / NA) & 1) ^ 1u, abort_flag, P.wait, kErrWaitEmpty)) {
                ok = false;
                break;
              }
              mbar_arrive_expect_tx(q_full(n), TILE_BYTES);
              load_tile(sQ(n), &mapQ, q_full(n), head, i * BT, x.shard);
              if (!wait_asleep(do_empty(n), ((n / NB) & 1) ^ 1u, abort_flag, P.wait, kErrWaitEmpty)) {
                ok = false;
                ++nq;
                break;
              }
              if (n != P.debug_drop) {
                mbar_arrive_expect_tx(do_full(n), TILE_BYTES);
                load_tile(sdO(n), &mapdO, do_full(n), head, i * BT, x.shard);
              }
              ++nq;
              if (++i == x.ia + x.ni) {
                i = x.ia;
                ++head;
              }
            }
          }
        }
        // Teardown: let the last loads land before shared memory is released.
        if (nu > 0) wait_teardown(kv_full, (nu - 1) & 1, P.wait);
        for (uint32_t q = nq > NA ? nq - NA : 0; q < nq; ++q) wait_teardown(q_full(q), (q / NA) & 1, P.wait);
        for (uint32_t q = n > NB ? n - NB : 0; q < n; ++q)
          if (q != P.debug_drop) wait_teardown(do_full(q), (q / NB) & 1, P.wait);
      }
      __syncwarp();
    } else if (warp == 1) {
      {
        // -------------------------------------------------------- MMA issuer
        // The whole warp goes through the loop and one lane issues: what the
        // products' operands are made of is then the same for the warp, and
        // stays in uniform registers.
        const bool leader = elect_one();
        auto await = [&](uint32_t bar, uint32_t parity, unsigned code) {
          return __all_sync(0xffffffffu, wait_asleep(bar, parity, abort_flag, P.wait, code)) != 0;
        };
        uint32_t n = 0, nu = 0;
        bool ok = true;
        auto wait_q = [&](uint32_t m) {
          return await(q_full(m), (m / NA) & 1, kErrWaitFull);
        };
        auto wait_do = [&](uint32_t m) {
          return await(do_full(m), (m / NB) & 1, kErrWaitFull);
        };
        Segment x;
        for (x.begin(P, start); ok && x.left > 0; x.next(P)) {
          const int32_t steps = x.s1 - x.s0;
          if (!await(kv_full, nu & 1, kErrWaitFull) || !wait_q(n)) break;
          tc_fence_after();
          if (leader) mma_tiles(tS, sK, sQ(n));
          if (leader) tc_commit(s_full);
          if (!wait_do(n)) break;
          tc_fence_after();
          if (leader) mma_tiles(tdP, sV, sdO(n));
          if (leader) tc_commit(dp_full);
          if (leader && steps == 1) tc_commit(kv_empty);
          for (int32_t s = 0; s < steps; ++s, ++n) {
            const bool more = s + 1 < steps;
            if (more) {
              // the next scores as soon as the warps hold this step's
              if (!await(s_free, n & 1, kErrWaitAttn) || !wait_q(n + 1)) {
                ok = false;
                break;
              }
              tc_fence_after();
              if (leader) mma_tiles(tS, sK, sQ(n + 1));
              if (leader) tc_commit(s_full);
            }
            if (!await(ds_full, n & 1, kErrWaitAttn) ||
                (s == 0 && nu > 0 &&
                 !await(acc_empty, (nu - 1) & 1, kErrWaitAttn))) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (leader) mma_rows(tdV, tdP, sdO(n), s > 0);
            if (leader) tc_commit(do_empty(n));
            if (leader) mma_rows(tdK, tdP + 16, sQ(n), s > 0);
            if (leader) tc_commit(q_empty(n));
            if (more) {
              if (!wait_do(n + 1)) {
                ok = false;
                break;
              }
              tc_fence_after();
              if (leader) mma_tiles(tdP, sV, sdO(n + 1));
              if (leader) tc_commit(dp_full);
              if (leader && s + 2 == steps) tc_commit(kv_empty);   // K and V are read by S^T and dP^T alone
            }
          }
          if (!ok) break;
          if (leader) tc_commit(acc_full);
          ++nu;
        }
        if (leader) tc_commit(drain);
        wait_teardown(drain, 0, P.wait);
      }
      __syncwarp();
    } else {
      // --------------- per-query numbers of each step, and the look at its rows
      uint32_t n = 0, nu = 0;
      bool ok = true;
      const int me = (warp - 2) * 32 + lane;   // 0..63: rows me and me + 64 of the tile
      Segment x;
      for (x.begin(P, start); ok && x.left > 0; x.next(P), ++nu) {
        {
          int32_t g = x.s0 / x.ni, i = x.ia + x.s0 % x.ni;
          for (int32_t s = x.s0; s < x.s1; ++s, ++n) {
            const int64_t row0 =
                (static_cast<int64_t>(x.shard) * P.hq + x.kvh * P.group + g) * P.T;
            const bool cut = !tile_span(P.mask, i, P.tiles, P.T, P.causal).whole(x.kb);
            float lse[2], dl[2];
            bool only[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int32_t q = i * BT + h * 64 + me;
              const int2 keys = cut ? row_span(P.mask, q, P.T, P.causal) : make_int2(0, 0);
              only[h] = keys.y - keys.x == 1;
              const bool in = q < P.T;
              lse[h] = in ? -kLog2e * P.LSE[row0 + q] : -INFINITY;   // P = 0 behind the last row
              dl[h] = in ? -P.delta[row0 + q] : 0.0f;
            }
            ok = wait_asleep(do_empty(n), ((n / NB) & 1) ^ 1u, abort_flag, P.wait, kErrWaitEmpty);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              sts(vec(n, 0) + (h * 64 + me) * 4, lse[h]);
              sts(vec(n, 1) + (h * 64 + me) * 4, dl[h]);
            }
            // (vec_full comes before the products that read the tiles, and their
            // commits before the next loads)
            const uint32_t odd0 = __ballot_sync(0xffffffffu, cut && !(fabsf(dl[0]) < INFINITY));
            const uint32_t odd1 = __ballot_sync(0xffffffffu, cut && !(fabsf(dl[1]) < INFINITY));
            const bool look = (odd0 | odd1) != 0;
            if (me == 0) {
              float slope2 = 0.0f;
              if (BIAS) slope2 = kLog2e * P.slopes[x.shard * P.hq + x.kvh * P.group + g];
              sts4(about + (n % NB) * 16, i,
                   (cut ? kCut : 0) | (s == x.s0 ? kFirst : 0) | (s + 1 == x.s1 ? x.last() ? kLast | kEnd : kLast : 0),
                   __float_as_int(slope2), 0);
              if (s == x.s0)
                sts4(about_unit + (nu & 3) * 16, x.kb, x.hh, x.whole() ? -1 : x.s0 > 0 ? 0 : 1, 0);
            }
            uint32_t w[2] = {0u, 0u};
            if (look) {
              ok = wait_asleep(q_full(n), (n / NA) & 1, abort_flag, P.wait, kErrWaitFull) &&
                   wait_asleep(do_full(n), (n / NB) & 1, abort_flag, P.wait, kErrWaitFull);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
#pragma unroll 1
              for (int h = 0; h < 2; ++h) {
                const int row = h * 64 + me;
                const bool b0 = row_not_finite(sQ(n), row), b1 = row_not_finite(sdO(n), row);
                if (b0) zero_row(sQ(n), row);
                if (b1) zero_row(sdO(n), row);
                w[h] = __ballot_sync(0xffffffffu, b0 || b1);
              }
              fence_proxy_async_smem();
            }
            if (cut) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t one = __ballot_sync(0xffffffffu, only[h]);
                if (lane == 0) {
                  bad[(n % NB) * 4 + h * 2 + (warp - 2)] = w[h];
                  lone[(n % NB) * 4 + h * 2 + (warp - 2)] = one;
                }
              }
            }
            mbar_arrive(vec_full(n));
            if (++i == x.ia + x.ni) {
              i = x.ia;
              ++g;
            }
          }
        }
      }
    }
  } else {
    regs_grow<104>();
    // -------------------------------------------- P^T, dS^T and the outputs
    const int part = (warp - 4) / 4;         // columns [32 part, 32 part + 32)
    const int quad = warp & 3;
    const uint32_t off = (static_cast<uint32_t>(quad * 32) << 16) + part * 32;
    uint32_t n = 0, nu = 0;
    bool ok = true;
    int32_t key = 0;
    int2 by = make_int2(0, 0);   // queries that see the key
    for (bool end = start.w == 0; !end; ++n) {
      ok = wait_asleep(vec_full(n), (n / NB) & 1, abort_flag, P.wait, kErrWaitAttn);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int4 step = lds_int4(about + (n % NB) * 16);
      end = (step.y & kEnd) != 0;
      if (step.y & kFirst) {
        key = lds_int4(about_unit + (nu & 3) * 16).x * BT + quad * 32 + lane;
        by = key_span(P.mask, key, P.T, P.causal);
      }
      ok = wait_asleep(s_full, n & 1, abort_flag, P.wait, kErrWaitAttn);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      float w[32];
      uint32_t v[32], pk[16];
      tmem_ld_32x32b_x32(tS + off, v);
      const bool cut = (step.y & kCut) != 0;
      const uint32_t vl = vec(n, 0) + part * 128, vd = vec(n, 1) + part * 128;
      const int32_t q0 = step.x * BT + part * 32;
      const float dist0 = static_cast<float>(q0 - key);
      const int32_t kb = key / BT;
      const int side = step.x > kb ? 1 : step.x < kb ? -1 : 0;
      uint32_t seen = 0xffffffffu, odd = 0;   // columns that see this key; that are not finite
      if (cut) {
        seen = columns_in(by.x - q0, by.y - q0);
        odd = seen & bad[(n % NB) * 4 + part];
        if (odd != 0) atomicOr(&hit[(nu % 3) * 4 + quad], 1u << lane);
      }
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(s_free);
      prob_chunk<CAP, BIAS>(v, w, pk, P, __int_as_float(step.z), dist0, side, cut, seen, seen & ~odd,
                            [&](int e, uint64_t& a, uint64_t& b) { lds4(vl + e * 4, a, b); });
      const uint32_t one = cut ? lone[(n % NB) * 4 + part] : 0u;
      if (one != 0) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if ((one >> e) & 1u) w[e] *= 0.0f;
      }
      ok = wait_asleep(dp_full, n & 1, abort_flag, P.wait, kErrWaitAttn);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      tmem_ld_32x32b_x32(tdP + off, v);
      tmem_ld_wait();
      // P^T and dS^T over this quarter's own dP^T
      tmem_st_32x32b_x16(tdP + off, pk);
      grad_chunk(v, w, pk, cut, seen, [&](int e, uint64_t& a, uint64_t& b) { lds4(vd + e * 4, a, b); });
      tmem_st_32x32b_x16(tdP + off + 16, pk);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(ds_full);
      if (!(step.y & kLast)) continue;
      ok = wait_asleep(acc_full, nu & 1, abort_flag, P.wait, kErrWaitAttn);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      // keys of no document stay as they were
      const bool store = key < P.T && by.y >= 0;
      const int4 unit = lds_int4(about_unit + (nu & 3) * 16);
      const int32_t shard = unit.y / P.hkv, kvh = unit.y - shard * P.hkv;
      const int64_t row = ((static_cast<int64_t>(shard) * P.T + key) * P.hkv + kvh) * DH + part * 32;
      const uint32_t hits = *const_cast<volatile uint32_t*>(&hit[(nu % 3) * 4 + quad]);
      const float f = (hits >> lane) & 1u ? NAN : 1.0f;
      if (part == 0 && lane == 0) hit[((nu + 2) % 3) * 4 + quad] = 0;
      if (unit.z < 0) {
        store_part_row(tdV + off, f, store, P.dV + row);
        store_part_row(tdK + off, f * P.s.scale, store, P.dK + row);
      } else {
        float* const to = P.part + (static_cast<int64_t>(blockIdx.x) * 2 + unit.z) * PART_FLOATS +
                          (quad * 32 + lane) * DH + part * 32;
        keep_part_row(tdV + off, f, to);
        keep_part_row(tdK + off, f * P.s.scale, to + BT * DH);
      }
      tc_fence_before();
      mbar_arrive(acc_empty);
      ++nu;
    }
  }

  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tm, 512);
  }
}

// Adds the parts of the unit that the beginning of CTA c = blockIdx.x + 1's
// share cuts (the first such CTA's block does it), in the CTAs' order; 16 keys a
// block.
constexpr int JOIN_KEYS = 16;
__global__ void __launch_bounds__(256) dkv_join_kernel(const __grid_constant__ BwdParams P, int32_t ctas) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t c = blockIdx.x + 1;
  const int64_t total = *P.total;
  const int64_t w = share_of(total, c, ctas);
  if (w >= share_of(total, c + 1, ctas)) return;   // (fewer steps than CTAs)
  const int4 cut = P.cuts[c];
  const int64_t from = w - cut.z, to = from + cut.w;   // the unit's steps on the line
  int64_t first = c - 1;   // the CTA before with a share
  while (first > 0 && share_of(total, first, ctas) == w) --first;
  if (cut.z == 0 || share_of(total, first, ctas) > from) return;
  const int32_t row0 = blockIdx.y * JOIN_KEYS;
  constexpr int VECS = JOIN_KEYS * DH / 4 / 256;   // float4s of a thread in each of dV, dK
  float4 sum[2][VECS];
  auto add = [&](int64_t cta, int slot, bool first) {
    const float* part = P.part + (cta * 2 + slot) * PART_FLOATS + row0 * DH;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
#pragma unroll
      for (int i = 0; i < VECS; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(part + a * BT * DH + (threadIdx.x + i * 256) * 4);
        float4& t = sum[a][i];
        t = first ? x : make_float4(t.x + x.x, t.y + x.y, t.z + x.z, t.w + x.w);
      }
    }
  };
  add(first, 1, true);
  for (int64_t d = c; d < ctas && share_of(total, d, ctas) < to; ++d)
    if (share_of(total, d, ctas) < share_of(total, d + 1, ctas)) add(d, 0, false);
  const int32_t shard = cut.y / P.hkv, kvh = cut.y - shard * P.hkv;
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int32_t at = (threadIdx.x + i * 256) * 4, key = cut.x * BT + row0 + at / DH;
    if (key >= P.T || key_span(P.mask, key, P.T, P.causal).y < 0) continue;
    const int64_t out = ((static_cast<int64_t>(shard) * P.T + key) * P.hkv + kvh) * DH + at % DH;
    *reinterpret_cast<uint2*>(P.dV + out) =
        make_uint2(pack2(sum[0][i].x, sum[0][i].y), pack2(sum[0][i].z, sum[0][i].w));
    *reinterpret_cast<uint2*>(P.dK + out) =
        make_uint2(pack2(sum[1][i].x, sum[1][i].y), pack2(sum[1][i].z, sum[1][i].w));
  }
}

// --------------------------------------------------------------------- dQ
struct QueryUnit {
  int32_t shard, head, kvh, qb;
  TileSpan t;
};
__device__ __forceinline__ QueryUnit query_unit(const BwdParams& P, int32_t u, const uint16_t* order) {
  QueryUnit x;
  const int32_t heads = P.p * P.hq, hh = u % heads;
  x.qb = order != nullptr ? order[u / heads] : P.tiles - 1 - u / heads;   // causal: the longest first
  x.shard = hh / P.hq;
  x.head = hh % P.hq;
  x.kvh = x.head / P.group;
  x.t = tile_span(P.mask, x.qb, P.tiles, P.T, P.causal);
  return x;
}

template <int CAP, bool BIAS>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    tc_scored_dq_kernel(const __grid_constant__ CUtensorMap mapQ,
                        const __grid_constant__ CUtensorMap mapK,
                        const __grid_constant__ CUtensorMap mapV,
                        const __grid_constant__ CUtensorMap mapdO,
                        const __grid_constant__ BwdParams P) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t base = smem_u32(smem_raw);
  if ((base & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(P.wait.err, kErrSmem);
    return;
  }
  const uint32_t sQ = base, sdO = base + TILE_BYTES;
  auto sK = [&](uint32_t n) { return base + (2 + n % NA) * TILE_BYTES; };
  auto sV = [&](uint32_t n) { return base + (2 + NA + n % NB) * TILE_BYTES; };
  uint8_t* const ctrl = smem_raw + TILES_BYTES;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(ctrl);
  const uint32_t qd_full = smem_u32(&bars[0]), qd_empty = smem_u32(&bars[1]);
  auto k_full = [&](uint32_t n) { return smem_u32(&bars[2 + n % NA]); };
  auto k_empty = [&](uint32_t n) { return smem_u32(&bars[5 + n % NA]); };
  auto v_full = [&](uint32_t n) { return smem_u32(&bars[8 + n % NB]); };
  auto v_empty = [&](uint32_t n) { return smem_u32(&bars[10 + n % NB]); };
  auto s_full = [&](uint32_t b) { return smem_u32(&bars[12 + b]); };
  const uint32_t dp_full = smem_u32(&bars[14]), dp_free = smem_u32(&bars[15]);
  // (two: the warps may finish step n + 1 before the MMA thread has seen step n)
  auto ds_full = [&](uint32_t n) { return smem_u32(&bars[16 + (n & 1)]); };
  const uint32_t acc_full = smem_u32(&bars[18]), acc_empty = smem_u32(&bars[19]);
  // one a ring slot: warps 2 and 3 may be that many blocks ahead
  auto k_seen = [&](uint32_t i) { return smem_u32(&bars[20 + i % NA]); };
  const uint32_t drain = smem_u32(&bars[20 + NA]);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 8 * (21 + NA));
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* const bad = tmem_slot + 2;   // [NA][4]: keys of a cut block that are not finite

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    mbar_init(qd_full, 1);
    mbar_init(qd_empty, 1);
    for (int s = 0; s < NA; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 3);   // the issuing thread's commit, warps 2 and 3
      mbar_init(k_seen(s), 64);
    }
    for (int s = 0; s < NB; ++s) {
      mbar_init(v_full(s), 1);
      mbar_init(v_empty(s), 1);
    }
    for (int s = 0; s < 2; ++s) mbar_init(s_full(s), 1);
    mbar_init(dp_full, 1);
    mbar_init(dp_free, ARITH);
    mbar_init(ds_full(0), ARITH);
    mbar_init(ds_full(1), ARITH);
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, ARITH);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&mapQ);
    tma_prefetch_map(&mapK);
    tma_prefetch_map(&mapV);
    tma_prefetch_map(&mapdO);
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  const uint32_t tdP = tm + 256, tdQ = tm + 384;   // S buffers at 0 and 128
  pdl_wait();
  pdl_launch_dependents();
  uint16_t* const order_smem = reinterpret_cast<uint16_t*>(ctrl + 512);
  const uint16_t* const order =
      order_tiles(P.mask, P.tiles, P.T, P.causal, P.num_units <= static_cast<int32_t>(gridDim.x),
                  order_smem, order_smem + kOrderTiles);

  // 96 registers a thread at launch: 128 x 64 + 512 x 104 <= 640 x 96
  if (warp < 4) {
    regs_shrink<64>();
    if (warp == 0) {
      if (lane == 0) {
        // ---------------------------------------------------------- producer
        uint32_t nu = 0, n = 0, nk = 0;   // nk: loads of K
        bool ok = true;
        int32_t r = 0;
        for (int32_t u = unit_of(0); ok && u < P.num_units; u = unit_of(++r)) {
          const QueryUnit x = query_unit(P, u, order);
          if (x.t.jb >= x.t.je) continue;
          if (!wait_asleep(qd_empty, (nu & 1) ^ 1u, abort_flag, P.wait, kErrWaitAttn)) break;
          mbar_arrive_expect_tx(qd_full, 2 * TILE_BYTES);
          load_tile(sQ, &mapQ, qd_full, x.head, x.qb * BT, x.shard);
          load_tile(sdO, &mapdO, qd_full, x.head, x.qb * BT, x.shard);
          ++nu;
          for (int32_t j = x.t.jb; j < x.t.je; ++j, ++n) {
            if (!wait_asleep(k_empty(n), ((n / NA) & 1) ^ 1u, abort_flag, P.wait, kErrWaitEmpty)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(k_full(n), TILE_BYTES);
            load_tile(sK(n), &mapK, k_full(n), x.kvh, j * BT, x.shard);
            ++nk;
            if (!wait_asleep(v_empty(n), ((n / NB) & 1) ^ 1u, abort_flag, P.wait, kErrWaitEmpty)) {
              ok = false;
              break;
            }
            if (n != P.debug_drop) {
              mbar_arrive_expect_tx(v_full(n), TILE_BYTES);
              load_tile(sV(n), &mapV, v_full(n), x.kvh, j * BT, x.shard);
            }
          }
        }
        if (nu > 0) wait_teardown(qd_full, (nu - 1) & 1, P.wait);
        for (uint32_t q = nk > NA ? nk - NA : 0; q < nk; ++q) wait_teardown(k_full(q), (q / NA) & 1, P.wait);
        for (uint32_t q = n > NB ? n - NB : 0; q < n; ++q)
          if (q != P.debug_drop) wait_teardown(v_full(q), (q / NB) & 1, P.wait);
      }
      __syncwarp();
    } else if (warp == 1) {
      {
        // -------------------------------------------------------- MMA issuer
        // The whole warp goes through the loop and one lane issues: what the
        // products' operands are made of is then the same for the warp, and
        // stays in uniform registers.
        const bool leader = elect_one();
        auto await = [&](uint32_t bar, uint32_t parity, unsigned code) {
          return __all_sync(0xffffffffu, wait_asleep(bar, parity, abort_flag, P.wait, code)) != 0;
        };
        uint32_t n = 0, nu = 0;
        bool ok = true;
        auto issue_s = [&](uint32_t m) {
          if (!await(k_full(m), (m / NA) & 1, kErrWaitFull)) return false;
          tc_fence_after();
          if (leader) mma_tiles(tm + (m & 1) * 128, sQ, sK(m));
          if (leader) tc_commit(s_full(m & 1));
          return true;
        };
        auto issue_dp = [&](uint32_t m) {
          if (!await(v_full(m), (m / NB) & 1, kErrWaitFull)) return false;
          tc_fence_after();
          if (leader) mma_tiles(tdP, sdO, sV(m));
          if (leader) tc_commit(v_empty(m));
          if (leader) tc_commit(dp_full);
          return true;
        };
        int32_t r = 0;
        for (int32_t u = unit_of(0); ok && u < P.num_units; u = unit_of(++r)) {
          const QueryUnit x = query_unit(P, u, order);
          const int32_t steps = x.t.je - x.t.jb;
          if (steps <= 0) continue;
          if (!await(qd_full, nu & 1, kErrWaitFull) || !issue_s(n) ||
              !issue_dp(n))
            break;
          if (steps == 1) {
            if (leader) tc_commit(qd_empty);
          } else if (!issue_s(n + 1)) {
            break;
          }
          for (int32_t s = 0; s < steps; ++s, ++n) {
            if (s + 1 < steps) {
              // the warps have read dP of this step
              ok = await(dp_free, n & 1, kErrWaitAttn);
              if (ok) {
                tc_fence_after();
                ok = issue_dp(n + 1);
              }
              if (!ok) break;
              if (leader && s + 2 == steps) tc_commit(qd_empty);
            }
            if (!await(ds_full(n), (n >> 1) & 1, kErrWaitAttn) ||
                (s == 0 && nu > 0 &&
                 !await(acc_empty, (nu - 1) & 1, kErrWaitAttn))) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (leader) mma_rows(tdQ, tm + (n & 1) * 128, sK(n), s > 0);
            if (leader) tc_commit(k_empty(n));
            if (s + 2 < steps && !issue_s(n + 2)) {
              ok = false;
              break;
            }
          }
          if (!ok) break;
          if (leader) tc_commit(acc_full);
          ++nu;
        }
        if (leader) tc_commit(drain);
        wait_teardown(drain, 0, P.wait);
      }
      __syncwarp();
    } else {
      // ------------------------------------- keys in blocks that a mask cuts
      uint32_t n = 0, looked = 0;
      bool ok = true;
      int32_t r = 0;
      for (int32_t u = unit_of(0); ok && u < P.num_units; u = unit_of(++r)) {
        const QueryUnit x = query_unit(P, u, order);
        for (int32_t j = x.t.jb; j < x.t.je; ++j, ++n) {
          const bool cut = !x.t.whole(j);
          bool odd = false;
          if (cut) {
            const uint8_t* flags = P.k_bad + (static_cast<int64_t>(x.shard) * P.hkv + x.kvh) * P.T;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int32_t key = j * BT + h * 64 + (warp - 2) * 32 + lane;
              odd |= key < P.T && flags[key] != 0;
            }
          }
          ok = wait_asleep(k_full(n), (n / NA) & 1, abort_flag, P.wait, kErrWaitFull);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (cut) {
            uint32_t w[2] = {0u, 0u};
            if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
              for (int h = 0; h < 2; ++h) {
                const int row = h * 64 + (warp - 2) * 32 + lane;
                const bool is_bad = row_not_finite(sK(n), row);
                if (is_bad) zero_row(sK(n), row);
                w[h] = __ballot_sync(0xffffffffu, is_bad);
              }
              fence_proxy_async_smem();
            }
            if (lane == 0) {
              bad[(n % NA) * 4 + (warp - 2)] = w[0];
              bad[(n % NA) * 4 + 2 + (warp - 2)] = w[1];
            }
            __syncwarp();
            mbar_arrive(k_seen(looked));
            ++looked;
          }
          // (the slot is held for these warps in every block, as they wait for
          // every block's load: k_full two loads on has the parity of the phase
          // that they wait for, and would keep a late warp waiting)
          __syncwarp();
          if (lane == 0) mbar_arrive(k_empty(n));
        }
      }
    }
  } else {
    regs_grow<104>();
    // ------------------------------------------------ P, dS and the output
    const int part = (warp - 4) / 4;         // columns [32 part, 32 part + 32)
    const int quad = warp & 3;
    const uint32_t off = (static_cast<uint32_t>(quad * 32) << 16) + part * 32;
    uint32_t n = 0, nu = 0, looked = 0;
    bool ok = true;
    int32_t r = 0;
    for (int32_t u = unit_of(0); ok && u < P.num_units; u = unit_of(++r)) {
      const QueryUnit x = query_unit(P, u, order);
      if (x.t.jb >= x.t.je) continue;
      const int32_t q0 = x.qb * BT, q = q0 + quad * 32 + lane;
      const int2 span = row_span(P.mask, q, P.T, P.causal);
      const bool live = q < P.T && span.y >= 0;
      const int64_t vrow = (static_cast<int64_t>(x.shard) * P.hq + x.head) * P.T + q;
      const float lse2 = live ? -kLog2e * P.LSE[vrow] : 0.0f;
      const float dl = live ? -P.delta[vrow] : 0.0f;
      const uint64_t nlse = f2_pack(lse2, lse2), ndl = f2_pack(dl, dl);
      float slope2 = 0.0f;
      if (BIAS) slope2 = kLog2e * P.slopes[x.shard * P.hq + x.head];
      for (int32_t j = x.t.jb; j < x.t.je; ++j, ++n) {
        const uint32_t b = n & 1, tS = tm + b * 128 + off;
        const bool cut = !x.t.whole(j);
        ok = wait_asleep(s_full(b), (n >> 1) & 1, abort_flag, P.wait, kErrWaitAttn);
        if (cut) {
          ok = ok && wait_asleep(k_seen(looked), (looked / NA) & 1, abort_flag, P.wait, kErrWaitAttn);
          ++looked;
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const int32_t key0 = j * BT + part * 32, rl = span.x - key0, rh = span.y - key0;
        const float dist0 = static_cast<float>(key0 - q);
        const int side = j * BT + BT - 1 <= q0 ? -1 : j * BT >= q0 + BT - 1 ? 1 : 0;
        float w[32];
        uint32_t v[32], pk[16];
        const uint32_t seen = cut ? columns_in(rl, rh) : 0xffffffffu, odd = cut ? bad[(n % NA) * 4 + part] : 0u;
        tmem_ld_32x32b_x32(tS, v);
        tmem_ld_wait();
        // (P itself is not stored: dQ needs dS alone)
        prob_chunk<CAP, BIAS>(v, w, pk, P, slope2, dist0, side, cut, seen, seen & ~odd,
                              [&](int, uint64_t& a, uint64_t& b) { a = b = nlse; });
        if (odd & seen) {   // (its row of K is 0 now: the NaN goes through dS)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if ((odd & seen) >> e & 1u) w[e] = NAN;
        }
        if (cut && span.y - span.x == 1) {
#pragma unroll
          for (int e = 0; e < 32; ++e) w[e] *= 0.0f;
        }
        ok = wait_asleep(dp_full, n & 1, abort_flag, P.wait, kErrWaitAttn);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        tmem_ld_32x32b_x32(tdP + off, v);
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive(dp_free);
        grad_chunk(v, w, pk, cut, seen, [&](int, uint64_t& a, uint64_t& b) { a = b = ndl; });
        tmem_st_32x32b_x16(tS, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(ds_full(n));
      }
      if (!ok) break;
      ok = wait_asleep(acc_full, nu & 1, abort_flag, P.wait, kErrWaitAttn);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      store_part_row(tdQ + off, P.s.scale, live,
                     P.dQ + ((static_cast<int64_t>(x.shard) * P.T + q) * P.hq + x.head) * DH + part * 32);
      tc_fence_before();
      mbar_arrive(acc_empty);
      ++nu;
    }
  }

  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tm, 512);
  }
}

template <int CAP, bool BIAS>
tp_status launch_bwd(const LaunchCtx& c, BwdParams prm, const ScoreCall& a, const CUtensorMap& mQ,
                     const CUtensorMap& mK, const CUtensorMap& mV, const CUtensorMap& mdO) {
  static uint64_t attr_epoch[64] = {};
  static std::mutex mu;
  {
    std::lock_guard<std::mutex> lk(mu);
    const int dev = c.device & 63;
    if (attr_epoch[dev] != c.epoch) {
      if (cudaFuncSetAttribute(tc_scored_dkv_kernel<CAP, BIAS>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               SMEM_BYTES) != cudaSuccess ||
          cudaFuncSetAttribute(tc_scored_dq_kernel<CAP, BIAS>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               SMEM_BYTES) != cudaSuccess) {
        set_error_detail("cudaFuncSetAttribute failed: %s", cudaGetErrorString(cudaGetLastError()));
        return TP_ERR_CUDA;
      }
      attr_epoch[dev] = c.epoch;
    }
  }
  auto grid = [&](int32_t units) { return dim3(units < c.num_sms ? units : c.num_sms); };
  const int32_t ctas = static_cast<int32_t>(score_dkv_ctas(a));
  prm.num_units = prm.p * prm.hkv * prm.tiles;
  prm.whole = prm.mask.rows == nullptr && prm.num_units >= kWholeUnits * ctas;
  cudaError_t e = launch_pdl(tc_scored_dkv_kernel<CAP, BIAS>, dim3(ctas), dim3(NUM_THREADS),
                             SMEM_BYTES, c.stream, mQ, mK, mV, mdO, prm);
  note_launch();
  if (e == cudaSuccess && ctas > 1 && !prm.whole) {
    e = launch_pdl(dkv_join_kernel, dim3(ctas - 1, BT / JOIN_KEYS), dim3(256), 0, c.stream, prm, ctas);
    note_launch();
  }
  if (e == cudaSuccess) {
    prm.debug_drop = -1;   // an armed fault injection applies to the first launch only
    prm.num_units = prm.p * prm.hq * prm.tiles;
    e = launch_pdl(tc_scored_dq_kernel<CAP, BIAS>, grid(prm.num_units), dim3(NUM_THREADS),
                   SMEM_BYTES, c.stream, mQ, mK, mV, mdO, prm);
    note_launch();
  }
  if (e != cudaSuccess) {
    set_error_detail("scored attention backward launch failed: %s", cudaGetErrorString(e));
    return TP_ERR_CUDA;
  }
  return TP_OK;
}

template <int CAP>
tp_status launch_form(const LaunchCtx& c, const BwdParams& prm, const ScoreCall& a, const CUtensorMap& mQ,
                      const CUtensorMap& mK, const CUtensorMap& mV, const CUtensorMap& mdO) {
  if (prm.slopes != nullptr) return launch_bwd<CAP, true>(c, prm, a, mQ, mK, mV, mdO);
  return launch_bwd<CAP, false>(c, prm, a, mQ, mK, mV, mdO);
}

}  // namespace

// CTAs that share the steps of dK and dV: one an SM, fewer where they would get
// less than two steps each even without a mask (four instead of two: 28 us to 37
// for a call of such a size).
int64_t score_dkv_ctas(const ScoreCall& a) {
  const int64_t tiles = ceil_div(a.T, BT);
  const int64_t steps = static_cast<int64_t>(a.p) * a.hq * (a.causal ? tiles * (tiles + 1) / 2 : tiles * tiles);
  const int64_t most = (steps + 1) / 2;
  return most < kScoreDkvCtas ? (most < 1 ? 1 : most) : kScoreDkvCtas;
}
size_t score_dkv_bytes(const ScoreCall& a) {
  return static_cast<size_t>(score_dkv_ctas(a)) * (2 * PART_FLOATS * sizeof(float) + sizeof(int4)) + 256;
}

tp_status launch_attention_scored_bwd(const LaunchCtx& c, const ScoreCall& a) {
  CUtensorMap mQ, mK, mV, mdO;
  const int64_t wq = static_cast<int64_t>(a.hq) * DH, wk = static_cast<int64_t>(a.hkv) * DH;
  if (!make_map_a(&mQ, a.Q, wq, a.T, a.p) || !make_map_a(&mK, a.K, wk, a.T, a.p) ||
      !make_map_a(&mV, a.V, wk, a.T, a.p) || !make_map_a(&mdO, a.dO, wq, a.T, a.p))
    return TP_ERR_CUDA;
  const int64_t shard_rows = static_cast<int64_t>(a.p) * a.T;
  const int64_t q_blocks = (shard_rows * a.hq + DELTA_ROWS - 1) / DELTA_ROWS;
  const int64_t k_blocks = (shard_rows * a.hkv + DELTA_ROWS - 1) / DELTA_ROWS;
  cudaError_t e = launch_pdl(
      score_delta_kernel, dim3(static_cast<unsigned>(q_blocks + k_blocks)), dim3(256), 0, c.stream,
      static_cast<const __nv_bfloat16*>(a.O), static_cast<const __nv_bfloat16*>(a.dO),
      static_cast<const __nv_bfloat16*>(a.Q), static_cast<const __nv_bfloat16*>(a.K), a.delta, a.k_bad,
      static_cast<uint32_t>(q_blocks), shard_rows, static_cast<int32_t>(a.T),
      static_cast<int32_t>(a.hq), static_cast<int32_t>(a.hkv));
  note_launch();
  if (e != cudaSuccess) {
    set_error_detail("delta launch failed: %s", cudaGetErrorString(e));
    return TP_ERR_CUDA;
  }
  BwdParams prm{};
  prm.T = static_cast<int32_t>(a.T);
  prm.p = a.p;
  prm.hq = a.hq;
  prm.hkv = a.hkv;
  prm.group = a.hq / a.hkv;
  prm.tiles = ceil_div(a.T, BT);
  prm.causal = a.causal ? 1 : 0;
  prm.mask = mask_plan(a.mask, a.T);
  prm.s = score_consts(a.scale, a.cap);
  prm.neg_inv_cap2 = a.cap > 0.0f ? -1.0f / (prm.s.cap_log2 * prm.s.cap_log2) : 0.0f;
  prm.slopes = a.slopes;
  prm.LSE = a.LSE;
  prm.delta = a.delta;
  prm.k_bad = a.k_bad;
  prm.part = a.part;
  prm.cuts = reinterpret_cast<int4*>(a.part + score_dkv_ctas(a) * 2 * PART_FLOATS);
  prm.total = reinterpret_cast<int64_t*>(prm.cuts + score_dkv_ctas(a));
  prm.dQ = static_cast<__nv_bfloat16*>(a.dQ);
  prm.dK = static_cast<__nv_bfloat16*>(a.dK);
  prm.dV = static_cast<__nv_bfloat16*>(a.dV);
  prm.wait.err = c.err_word;
  prm.wait.timeout_ns = c.timeout_ns;
  prm.debug_drop = c.debug_drop;
  const int cap = cap_form(prm.s);
  if (cap == kFineCap) return launch_form<kFineCap>(c, prm, a, mQ, mK, mV, mdO);
  if (cap == kCoarseCap) return launch_form<kCoarseCap>(c, prm, a, mQ, mK, mV, mdO);
  return launch_form<kNoCap>(c, prm, a, mQ, mK, mV, mdO);
}

}  // namespace tpk
