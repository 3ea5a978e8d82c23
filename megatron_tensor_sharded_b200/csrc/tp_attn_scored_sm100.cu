// Attention with capped scores, a distance bias, and document, prefix or
// causal masks: the forward pass, one persistent tcgen05 launch (sm_100a),
// and the mask's plan.
//
//   z_ij = cap tanh(scale q_i.k_j / cap) - slope |i - j|   over the keys that
//   row i sees, an interval [lo_i, hi_i);  O_i = sum_j softmax(z_i)_j v_j,
//   LSE_i = log sum_j exp z_ij.
//
// Bound by the tensor cores (4 * 128 flops a visible pair) and, with the cap,
// by the softmax's arithmetic beside them.  The pipeline is that of
// tc_attn_kernel: a unit is a (shard, query head, pair of 128-row query
// tiles), K/V blocks of 128 keys go through a two-slot ring and feed both
// tiles, scores and probabilities stay in TMEM (P over the scores it came
// from), O accumulates in TMEM.  Roles (384 threads): warp 0 TMA, warp 1 MMA,
// warps 2..3 look at V where a mask cuts a block, warps 4..7 and 8..11 the
// softmax of one tile each, a thread a row.
//
// Blocks: each tile walks only the blocks between its rows' least and
// greatest visible key (from the mask's plan; arithmetic without one), and
// masks scores only in blocks that some row does not see whole.
//
// Cap: tanh by an odd polynomial in packed fp32 pairs where a chunk's scores
// are small against the cap (|scale s| <= cap/2 over 32 columns of a warp's
// rows: 2.5 FMA-pipe operations an element, error 5.5e-7 relative), else by
// 1 - 2/(1 + e^2x) on the MUFU unit (two MUFU operations an element more).
// tanh.approx's 2^-11 times a cap of 50 would be 0.02 in a score.  Capped
// scores lie in [-cap, cap], so without a bias no running maximum is needed
// as long as 2^(cap log2 e) and its sums stay far inside fp32: kBoundLog2.
// Then there is no maximum pass over the scores and O is never rescaled.
//
// A key that a row does not see adds nothing to it, whatever K and V hold
// there: its score is replaced by -inf before the softmax, and where a mask
// cuts a block warps 2..3 zero the rows of V that hold an infinity or NaN
// before P V reads them (0 * NaN would be NaN).  Rows that do see such a key
// are made NaN through its bit in `bad`.
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
constexpr int BQ = kAttnTile;
constexpr int BKV = kAttnTile;
constexpr int NQT = 2;                       // query tiles per unit
constexpr int NST = 2;                       // K/V ring slots
constexpr int TILE_BYTES = 128 * 128 * 2;
constexpr int HALF_BYTES = TILE_BYTES / 2;
constexpr int XCH_BYTES = NQT * 2 * 2 * BQ * 4;   // [tile][parity][column half][row]
constexpr int SMEM_BYTES = 1024 + NQT * TILE_BYTES + NST * 2 * TILE_BYTES + XCH_BYTES + 512;
constexpr int NUM_THREADS = 640;
constexpr uint32_t IDESC_S = idesc_bf16_f32(BQ, BKV, 0, 0);
constexpr uint32_t IDESC_O = idesc_bf16_f32(BQ, DH, 0, 1);
constexpr uint32_t O_COL0 = NQT * BKV, TMEM_COLS = 512;
constexpr float RESCALE_LOG2 = 8.0f;
constexpr float kBoundLog2 = 80.0f;          // |z| in log2 that needs no running maximum

enum { kPlain = 0, kBias = 1, kCap = 2, kCapAny = 3 };   // kCap: no bias, bounded

struct ScoredParams {
  int32_t T, p, hq, hkv, group, q_blocks, q_pairs, num_units, causal;
  MaskPlan mask;
  ScoreConsts s;
  const float* slopes;
  __nv_bfloat16* O;
  float* LSE;
  WaitCtl wait;
  int64_t debug_drop;
};

struct Unit {
  int32_t shard, head, kvh, qb0;
  TileSpan t[NQT];
  int32_t jmin, jmax;
  // (selected, not indexed: the softmax warps' tile is a run-time number)
  __device__ __forceinline__ TileSpan span(int i) const { return i == 0 ? t[0] : t[1]; }
  __device__ __forceinline__ bool active(int i, int32_t j) const {
    const TileSpan s = span(i);
    return j >= s.jb && j < s.je;
  }
  __device__ __forceinline__ bool any(int i) const {
    const TileSpan s = span(i);
    return s.je > s.jb;
  }
  // block j holds a key that some row of an active tile does not see
  __device__ __forceinline__ bool cut(int32_t j) const {
    return (active(0, j) && !t[0].whole(j)) || (active(1, j) && !t[1].whole(j));
  }
};

__device__ __forceinline__ Unit decode_unit(const ScoredParams& P, int32_t u) {
  Unit x;
  const int32_t heads = P.p * P.hq;
  const int32_t level = u / heads, hh = u % heads;
  const int32_t qp = P.q_pairs - 1 - level;   // causal: the longest first
  x.shard = hh / P.hq;
  x.head = hh % P.hq;
  x.kvh = x.head / P.group;
  x.qb0 = qp * NQT;
#pragma unroll
  for (int i = 0; i < NQT; ++i) x.t[i] = tile_span(P.mask, x.qb0 + i, P.q_blocks, P.T, P.causal);
  x.jmin = x.any(0) ? (x.any(1) ? min(x.t[0].jb, x.t[1].jb) : x.t[0].jb) : x.t[1].jb;
  x.jmax = x.any(0) ? (x.any(1) ? max(x.t[0].je, x.t[1].je) : x.t[0].je) : x.t[1].je;
  return x;
}

// Rounds of gridDim.x units, alternately forwards and backwards over the CTAs.
__device__ __forceinline__ int32_t unit_of(int32_t r) {
  const int32_t g = static_cast<int32_t>(gridDim.x), b = static_cast<int32_t>(blockIdx.x);
  return r * g + ((r & 1) ? g - 1 - b : b);
}

// Of every eight pairs of probabilities, those whose 2^x runs as a polynomial
// on the FMA pipe, so that it and the MUFU unit (16 a clock and SM) are busy
// for about as long: an element costs the FMA pipe 6 clocks of a scheduler
// with the cap and 2 to 3 without, 9 more where 2^x is there too, and the MUFU
// unit 8 where it is not.
template <int MODE>
constexpr int kPolyPairs = MODE == kCap || MODE == kCapAny ? 1 : 2;

// Probabilities of 32 scores: bf16 pairs into pk, fp32 sums into sum2.
// SCALE: x = v * sc + off, else v holds x itself.
template <int POLY, bool SCALE>
__device__ __forceinline__ void exp_chunk(const uint32_t (&v)[32], uint64_t sc2, uint64_t off2,
                                          uint64_t (&sum2)[2], uint32_t (&pk)[16]) {
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    uint64_t xa = f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
    if (SCALE) xa = f2_fma(xa, sc2, off2);
    float a0, a1;
    if ((e / 2) % 8 < POLY) {
      f2_unpack(exp2_poly5<false>(xa), a0, a1);
    } else {
      float x0, x1;
      f2_unpack(xa, x0, x1);
      a0 = ex2(x0);
      a1 = ex2(x1);
    }
    sum2[(e / 2) & 1] = f2_add(sum2[(e / 2) & 1], f2_pack(a0, a1));
    pk[e / 2] = pack2(a0, a1);
  }
}

// 32 raw products -> scores in log2 units (kPlain: still unscaled), -inf where
// the row does not see the key.  lost: a visible score is NaN (kCap has no
// maximum that would carry it).
template <int MODE>
__device__ __forceinline__ void score_chunk(uint32_t (&v)[32], const ScoreConsts& S, float slope2,
                                            float dist0, int side, bool whole, int32_t rl,
                                            int32_t rh, bool& lost) {
  bool slow = false;
  if (MODE == kCap || MODE == kCapAny) slow = cap_chunk(v, S);
  if (MODE == kBias || MODE == kCapAny)
    bias_chunk<MODE == kBias>(v, S.scale_log2, slope2, dist0, side);
  if (!whole) mask_chunk(v, rl, rh);
  if (MODE == kCap && slow) {
#pragma unroll
    for (int e = 0; e < 32; ++e) lost |= __uint_as_float(v[e]) != __uint_as_float(v[e]);
  }
}

template <int MODE>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    tc_attn_scored_kernel(const __grid_constant__ CUtensorMap mapQ,
                          const __grid_constant__ CUtensorMap mapK,
                          const __grid_constant__ CUtensorMap mapV,
                          const __grid_constant__ ScoredParams P) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  auto sQ = [&](uint32_t t) { return base + t * TILE_BYTES; };
  auto sK = [&](uint32_t st) { return base + NQT * TILE_BYTES + st * 2 * TILE_BYTES; };
  auto sV = [&](uint32_t st) { return sK(st) + TILE_BYTES; };
  constexpr int RING_END = NQT * TILE_BYTES + NST * 2 * TILE_BYTES;
  volatile float* const xch = reinterpret_cast<volatile float*>(smem_raw + (base - raw) + RING_END);
  uint8_t* const ctrl = smem_raw + (base - raw) + RING_END + XCH_BYTES;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(ctrl);
  const uint32_t q_full = smem_u32(&bars[0]), q_empty = smem_u32(&bars[1]);
  auto kv_full = [&](uint32_t s) { return smem_u32(&bars[2 + s]); };
  auto kv_empty = [&](uint32_t s) { return smem_u32(&bars[2 + NST + s]); };
  auto s_full = [&](uint32_t t) { return smem_u32(&bars[2 + 2 * NST + t]); };
  auto p_full = [&](uint32_t t) { return smem_u32(&bars[2 + 2 * NST + NQT + t]); };
  auto o_full = [&](uint32_t t) { return smem_u32(&bars[2 + 2 * NST + 2 * NQT + t]); };
  auto o_empty = [&](uint32_t t) { return smem_u32(&bars[2 + 2 * NST + 3 * NQT + t]); };
  auto v_seen = [&](uint32_t i) { return smem_u32(&bars[2 + 2 * NST + 4 * NQT + i]); };
  auto x_full = [&](uint32_t t) { return smem_u32(&bars[4 + 2 * NST + 4 * NQT + t]); };
  const uint32_t drain = smem_u32(&bars[6 + 2 * NST + 4 * NQT]);
  constexpr int NBARS = 7 + 2 * NST + 4 * NQT;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 8 * NBARS);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* const bad = tmem_slot + 2;   // [2][4]: keys of a looked-at block whose V is not finite

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < NST; ++s) {
      mbar_init(kv_full(s), 1);
      mbar_init(kv_empty(s), 3);   // the MMA thread's commit, warps 2 and 3
    }
    for (int t = 0; t < NQT; ++t) {
      mbar_init(s_full(t), 1);
      mbar_init(p_full(t), 256);
      mbar_init(o_full(t), 1);
      mbar_init(o_empty(t), 256);
      mbar_init(x_full(t), 256);
      mbar_init(v_seen(t), 64);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&mapQ);
    tma_prefetch_map(&mapK);
    tma_prefetch_map(&mapV);
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  pdl_wait();
  pdl_launch_dependents();
  // 96 registers a thread at launch: 128 x 64 + 512 x 104 <= 640 x 96
  if (warp < 4) {
    regs_shrink<64>();
    if (warp == 0) {
      if (lane == 0) {
        // ------------------------------------------------------------ producer
        uint32_t st = 0, ph = 0, nu = 0;
        int64_t issued = 0;
        bool ok = true;
        int32_t r = 0;
        for (int32_t u = unit_of(0); ok && u < P.num_units; u = unit_of(++r)) {
          const Unit x = decode_unit(P, u);
          if (x.jmin >= x.jmax) continue;
          if (!wait_bounded(q_empty, (nu & 1) ^ 1u, abort_flag, P.wait, kErrWaitAttn)) break;
          mbar_arrive_expect_tx(q_full, (x.any(0) + x.any(1)) * TILE_BYTES);
          for (int t = 0; t < NQT; ++t) {
            if (!x.any(t)) continue;
            for (int c = 0; c < 2; ++c)
              tma_load_3d(sQ(t) + c * HALF_BYTES, &mapQ, q_full, x.head * DH + c * 64,
                          (x.qb0 + t) * BQ, x.shard);
          }
          ++nu;
          for (int32_t j = x.jmin; j < x.jmax; ++j) {
            if (!wait_bounded(kv_empty(st), ph ^ 1u, abort_flag, P.wait, kErrWaitEmpty)) {
              ok = false;
              break;
            }
            if (issued != P.debug_drop) {
              mbar_arrive_expect_tx(kv_full(st), 2 * TILE_BYTES);
              for (int c = 0; c < 2; ++c) {
                tma_load_3d(sK(st) + c * HALF_BYTES, &mapK, kv_full(st), x.kvh * DH + c * 64, j * BKV,
                            x.shard);
                tma_load_3d(sV(st) + c * HALF_BYTES, &mapV, kv_full(st), x.kvh * DH + c * 64, j * BKV,
                            x.shard);
              }
            }
            ++issued;
            if (++st == NST) {
              st = 0;
              ph ^= 1u;
            }
          }
        }
        // Teardown: let the last loads land before shared memory is released.
        if (nu > 0) wait_teardown(q_full, (nu - 1) & 1, P.wait);
        const int64_t first = issued > NST ? issued - NST : 0;
        for (int64_t q = first; q < issued; ++q) {
          if (q == P.debug_drop) continue;
          wait_teardown(kv_full(static_cast<uint32_t>(q % NST)), static_cast<uint32_t>((q / NST) & 1),
                        P.wait);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      if (lane == 0) {
        // ---------------------------------------------------------- MMA issuer
        uint32_t kv_n = 0, nu = 0;     // K/V blocks and units so far
        uint32_t pv[NQT] = {0, 0};     // O += P V products per tile
        uint32_t ou[NQT] = {0, 0};     // units per tile with an output
        bool ok = true;
        auto wait_kv = [&](uint32_t n) {
          return wait_bounded(kv_full(n % NST), (n / NST) & 1, abort_flag, P.wait, kErrWaitFull);
        };
        auto issue_s = [&](uint32_t t, uint32_t n) {
          const uint32_t kst = n % NST;
  #pragma unroll
          for (int kk = 0; kk < DH / 16; ++kk) {
            const uint32_t off = (kk >> 2) * HALF_BYTES + (kk & 3) * 32;
            tc_mma_f16(tmem_base + t * BKV, smem_desc_sw128(sQ(t) + off, 16, 1024),
                       smem_desc_sw128(sK(kst) + off, 16, 1024), IDESC_S, kk > 0 ? 1u : 0u);
          }
          tc_commit(s_full(t));
        };
        int32_t r = 0;
        for (int32_t u = unit_of(0); ok && u < P.num_units; u = unit_of(++r)) {
          const Unit x = decode_unit(P, u);
          if (x.jmin >= x.jmax) continue;
          if (!wait_bounded(q_full, nu & 1, abort_flag, P.wait, kErrWaitAttn)) break;
          ++nu;
          // Only the Q K^T products read Q: it is handed back once the last one
          // of every tile is issued.
          int s_left = x.any(0) + x.any(1);
          auto start_s = [&](int t, int32_t j) {
            issue_s(t, kv_n + (j - x.jmin));
            if (j + 1 == x.t[t].je && --s_left == 0) tc_commit(q_empty);
          };
          if (!wait_kv(kv_n)) break;
          tc_fence_after();
  #pragma unroll
          for (int t = 0; t < NQT; ++t)
            if (x.active(t, x.jmin)) start_s(t, x.jmin);
          for (int32_t j = x.jmin; ok && j < x.jmax; ++j) {
            const uint32_t n = kv_n + (j - x.jmin), vst = n % NST;
            const bool a0 = x.active(0, j), a1 = x.active(1, j);
            if (!a0 && !a1) {   // no tile reads this block
              if (!wait_kv(n)) {
                ok = false;
                break;
              }
              mbar_arrive(kv_empty(vst));
            }
  #pragma unroll
            for (int t = 0; t < NQT; ++t) {
              const bool act = t == 0 ? a0 : a1;
              if (act) {
                if (j == x.t[t].jb && ou[t] > 0 &&
                    !wait_bounded(o_empty(t), (ou[t] - 1) & 1, abort_flag, P.wait, kErrWaitAttn)) {
                  ok = false;
                  break;
                }
                if (!wait_bounded(p_full(t), pv[t] & 1, abort_flag, P.wait, kErrWaitAttn)) {
                  ok = false;
                  break;
                }
                tc_fence_after();
  #pragma unroll
                for (int kk = 0; kk < BKV / 16; ++kk) {
                  const uint64_t bdesc = smem_desc_sw128(sV(vst) + kk * 16 * 128, HALF_BYTES, 1024);
                  tc_mma_f16_ts(tmem_base + O_COL0 + t * DH,
                                tmem_base + t * BKV + (kk >> 2) * 64 + (kk & 3) * 8, bdesc, IDESC_O,
                                (j > x.t[t].jb || kk > 0) ? 1u : 0u);
                }
                ++pv[t];
                if (t == NQT - 1 || !a1) tc_commit(kv_empty(vst));   // the block's last reader
              }
              if (x.active(t, j + 1)) {
                if (!wait_kv(n + 1)) {
                  ok = false;
                  break;
                }
                tc_fence_after();
                start_s(t, j + 1);
              } else if (act) {
                tc_commit(o_full(t));
              }
            }
          }
          if (!ok) break;
  #pragma unroll
          for (int t = 0; t < NQT; ++t)
            if (x.any(t)) ++ou[t];
          kv_n += x.jmax - x.jmin;
        }
        tc_commit(drain);
        wait_teardown(drain, 0, P.wait);
      }
      __syncwarp();
    } else {
      // ------------------------------------- values in blocks that a mask cuts
      uint32_t n = 0, looked = 0;
      bool ok = true;
      int32_t r = 0;
      for (int32_t u = unit_of(0); ok && u < P.num_units; u = unit_of(++r)) {
        const Unit x = decode_unit(P, u);
        for (int32_t j = x.jmin; j < x.jmax; ++j, ++n) {
          const uint32_t st = n % NST;
          ok = wait_bounded(kv_full(st), (n / NST) & 1, abort_flag, P.wait, kErrWaitFull);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (x.cut(j)) {
  #pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int row = h * 64 + (warp - 2) * 32 + lane;
              const bool is_bad = row_not_finite(sV(st), row);
              const uint32_t w = __ballot_sync(0xffffffffu, is_bad);
              if (is_bad) zero_row(sV(st), row);
              if (lane == 0) bad[(looked & 1) * 4 + h * 2 + (warp - 2)] = w;
            }
            fence_proxy_async_smem();
            mbar_arrive(v_seen(looked & 1));
            ++looked;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(kv_empty(st));
        }
      }
    }
  } else {
    regs_grow<104>();
    // ------------------------------------------------------- softmax / output
    // thread = row and column half: scores [64 half, 64 half + 64) of a block,
    // and those columns of O
    const int t = (warp - 4) / 8;
    const int half = ((warp - 4) / 4) & 1;
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tS = tmem_base + lane_off + t * BKV + half * 64;
    const uint32_t tO = tmem_base + lane_off + O_COL0 + t * DH + half * 64;
    constexpr bool HAS_MAX = MODE != kCap;
    const ScoreConsts& S = P.s;
    uint32_t sc = 0, uc = 0, looked = 0, xc = 0;
    bool ok = true;
    // hands v to the row's other half and takes its
    auto swap_halves = [&](float v, float* other) {
      xch[((t * 2 + (xc & 1)) * 2 + half) * BQ + row] = v;
      mbar_arrive(x_full(t));
      const bool got = wait_bounded(x_full(t), xc & 1, abort_flag, P.wait, kErrWaitAttn);
      *other = xch[((t * 2 + (xc & 1)) * 2 + (half ^ 1)) * BQ + row];
      ++xc;
      return __all_sync(0xffffffffu, got) != 0;
    };
    int32_t r = 0;
    for (int32_t u = unit_of(0); ok && u < P.num_units; u = unit_of(++r)) {
      const Unit x = decode_unit(P, u);
      const TileSpan mine = x.span(t);
      const int32_t q0 = (x.qb0 + t) * BQ;
      const int32_t q = q0 + row;
      const int2 seen = row_span(P.mask, q, P.T, P.causal);
      float slope2 = 0.0f;
      if (MODE == kBias || MODE == kCapAny)
        slope2 = P.slopes != nullptr ? 1.4426950408889634f * P.slopes[x.shard * P.hq + x.head] : 0.0f;
      float m = HAS_MAX ? -INFINITY : 0.0f, l = 0.0f;
      bool poison = false, lost = false;
      for (int32_t j = x.jmin; j < x.jmax; ++j) {
        const bool cut = x.cut(j);
        if (!x.active(t, j)) {
          looked += cut;
          continue;
        }
        ok = wait_bounded(s_full(t), sc & 1, abort_flag, P.wait, kErrWaitAttn);
        const int32_t key0 = j * BKV + half * 64, rl = seen.x - key0, rh = seen.y - key0;
        if (ok && cut) {
          ok = wait_bounded(v_seen(looked & 1), (looked >> 1) & 1, abort_flag, P.wait, kErrWaitAttn);
          if (ok) {
            const volatile uint32_t* b = bad + (looked & 1) * 4 + half * 2;
            if (b[0] | b[1]) {
              for (int e = 0; e < 64; ++e)
                poison |= e >= rl && e < rh && ((b[e >> 5] >> (e & 31)) & 1);
            }
          }
          ++looked;
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const bool whole = mine.whole(j);
        const float dist0 = static_cast<float>(key0 - q);
        const int side = j * BKV + BKV - 1 <= q0 ? -1 : j * BKV >= q0 + BQ - 1 ? 1 : 0;
        uint64_t sum2[2] = {f2_pack(0.0f, 0.0f), f2_pack(0.0f, 0.0f)};
        // (loops kept rolled: the instruction cache holds one chunk's code)
        if (HAS_MAX) {
          float acc[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(tS + c * 32, v);
            tmem_ld_wait();
            score_chunk<MODE>(v, S, slope2, dist0 + c * 32.0f, side, whole, rl - c * 32,
                              rh - c * 32, lost);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              acc[0] = max3_nan(acc[0], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
              acc[1] = max3_nan(acc[1], __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
            }
            if (MODE != kPlain) tmem_st_32x32b_x32(tS + c * 32, v);
          }
          if (MODE != kPlain) tmem_st_wait();
          float m_cand = max3_nan(acc[0], acc[1], acc[1]), other;
          ok = swap_halves(m_cand, &other);
          if (!ok) break;
          m_cand = max3_nan(m_cand, other, other);
          if (MODE == kPlain) m_cand *= S.scale_log2;
          const bool grow = !(m_cand <= m + RESCALE_LOG2);   // NaN too: it then stays in the sum
          const float alpha = grow ? ex2(m - m_cand) : 1.0f;
          if (grow) m = m_cand;
          l *= alpha;
          if (j > mine.jb && __any_sync(0xffffffffu, grow)) {
            // O += P V of the previous block has completed: it was issued
            // before this score block, whose commit we waited for
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              uint32_t v[32];
              tmem_ld_32x32b_x32(tO + c * 32, v);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
              tmem_st_32x32b_x32(tO + c * 32, v);
            }
          }
        }
        const float off = m == -INFINITY ? 0.0f : -m;   // nothing seen so far
        const float scale = MODE == kPlain ? S.scale_log2 : 1.0f;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          uint32_t v[32], pk[16];
          tmem_ld_32x32b_x32(tS + c * 32, v);
          tmem_ld_wait();
          if (MODE == kPlain && !whole) mask_chunk(v, rl - c * 32, rh - c * 32);
          if (MODE == kCap)
            score_chunk<MODE>(v, S, slope2, dist0, side, whole, rl - c * 32, rh - c * 32, lost);
          exp_chunk<kPolyPairs<MODE>, HAS_MAX>(v, f2_pack(scale, scale), f2_pack(off, off), sum2, pk);
          tmem_st_32x32b_x16(tS + c * 16, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(p_full(t));
        float s0, s1, s2, s3;
        f2_unpack(sum2[0], s0, s1);
        f2_unpack(sum2[1], s2, s3);
        l += (s0 + s1) + (s2 + s3);
        ++sc;
      }
      if (!ok) break;
      if (!x.any(t)) continue;
      // the row's sum over both halves; NaN where a half lost a NaN score, and
      // a mark where one saw a key whose value is not finite
      float other;
      ok = swap_halves(lost ? NAN : l, &other);
      if (!ok) break;
      l = lost ? NAN : half == 0 ? l + other : other + l;
      ok = swap_halves(poison ? 1.0f : 0.0f, &other);
      if (!ok) break;
      poison |= other != 0.0f;
      ok = wait_bounded(o_full(t), uc & 1, abort_flag, P.wait, kErrWaitAttn);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const float inv_l = poison ? NAN : l == 0.0f ? 0.0f : 1.0f / l;
      const bool store = q < P.T && seen.y >= 0;   // rows of no document stay as they were
      __nv_bfloat16* dst =
          P.O + ((static_cast<int64_t>(x.shard) * P.T + q) * P.hq + x.head) * DH + half * 64;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(tO + c * 32, v);
        tmem_ld_wait();
        if (store) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              o[i] = pack2(__uint_as_float(v[g * 8 + 2 * i]) * inv_l,
                           __uint_as_float(v[g * 8 + 2 * i + 1]) * inv_l);
            *reinterpret_cast<uint4*>(dst + c * 32 + g * 8) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      }
      if (store && half == 0 && P.LSE != nullptr)
        P.LSE[(static_cast<int64_t>(x.shard) * P.hq + x.head) * P.T + q] =
            l == 0.0f ? -INFINITY : 0.6931471805599453f * m + logf(l);
      tc_fence_before();
      mbar_arrive(o_empty(t));
      ++uc;
    }
  }

  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// ------------------------------------------------------------- mask's plan
// One CTA per tile of 128 rows: each row finds its document (binary search of
// the offsets) and writes its visible keys; the tile's summary follows.
__global__ void __launch_bounds__(kAttnTile)
    mask_rows_kernel(const int32_t* __restrict__ off, int32_t n_docs,
                     const int32_t* __restrict__ prefix, int32_t causal, MaskPlan plan, int32_t T) {
  __shared__ int32_t red[4][kAttnTile / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int32_t t = blockIdx.x * kAttnTile + threadIdx.x;
  int32_t lo = 0, hi = -1;
  int2 by = make_int2(0, -1);
  if (t < T) {
    int32_t a = 0, b = n_docs + 1;   // the last offset <= t is below b
    while (b - a > 1) {
      const int32_t mid = a + (b - a) / 2;
      if (off[mid] <= t)
        a = mid;
      else
        b = mid;
    }
    if (a < n_docs) {
      const int32_t ds = max(off[a], 0), de = min(off[a + 1], T);
      if (ds <= t && t < de) {
        lo = ds;
        hi = de;
        by = make_int2(ds, de);
        if (causal) {
          const int32_t free = prefix != nullptr ? min(max(prefix[a], 0), de - ds) : 0;
          hi = max(t + 1, ds + free);
          if (t >= ds + free) by.x = t;
        }
      }
    }
    plan.rows[t] = make_int2(lo, hi);
    plan.keys[t] = by;
  }
  const bool in = hi >= 0;
  int32_t v[4] = {in ? lo : INT_MAX, in ? hi : 0, t < T ? lo : 0, t < T ? hi : INT_MAX};
#pragma unroll
  for (int o = 16; o > 0; o /= 2) {
    v[0] = min(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    v[1] = max(v[1], __shfl_xor_sync(0xffffffffu, v[1], o));
    v[2] = max(v[2], __shfl_xor_sync(0xffffffffu, v[2], o));
    v[3] = min(v[3], __shfl_xor_sync(0xffffffffu, v[3], o));
  }
  if (threadIdx.x % 32 == 0)
    for (int i = 0; i < 4; ++i) red[i][threadIdx.x / 32] = v[i];
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kAttnTile / 32; ++w) {
      v[0] = min(v[0], red[0][w]);
      v[1] = max(v[1], red[1][w]);
      v[2] = max(v[2], red[2][w]);
      v[3] = min(v[3], red[3][w]);
    }
    plan.q_tiles[blockIdx.x] = make_int4(v[0], v[1], v[2], v[3]);
  }
}

// The query tiles that may see a key of each tile of 128 keys: one warp a
// key tile.
__global__ void __launch_bounds__(kAttnTile) mask_tiles_kernel(MaskPlan plan, int32_t tiles) {
  pdl_wait();
  pdl_launch_dependents();
  const int32_t j = blockIdx.x * (kAttnTile / 32) + threadIdx.x / 32, lane = threadIdx.x % 32;
  if (j >= tiles) return;
  int32_t first = INT_MAX, last = -1;
  for (int32_t i = lane; i < tiles; i += 32) {
    const int4 s = plan.q_tiles[i];
    if (s.x < s.y && s.x / kAttnTile <= j && (s.y - 1) / kAttnTile >= j) {
      first = min(first, i);
      last = max(last, i);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o /= 2) {
    first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
    last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
  }
  if (lane == 0) plan.k_tiles[j] = last < 0 ? make_int2(0, 0) : make_int2(first, last + 1);
}

template <int MODE>
tp_status launch_mode(const LaunchCtx& c, const ScoredParams& prm, const CUtensorMap& mQ,
                      const CUtensorMap& mK, const CUtensorMap& mV) {
  static uint64_t attr_epoch[64] = {};
  static std::mutex mu;
  {
    std::lock_guard<std::mutex> lk(mu);
    const int dev = c.device & 63;
    if (attr_epoch[dev] != c.epoch) {
      if (cudaFuncSetAttribute(tc_attn_scored_kernel<MODE>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               SMEM_BYTES) != cudaSuccess) {
        set_error_detail("cudaFuncSetAttribute failed: %s", cudaGetErrorString(cudaGetLastError()));
        return TP_ERR_CUDA;
      }
      attr_epoch[dev] = c.epoch;
    }
  }
  const int grid = prm.num_units < c.num_sms ? prm.num_units : c.num_sms;
  const cudaError_t e = launch_pdl(tc_attn_scored_kernel<MODE>, dim3(grid), dim3(NUM_THREADS),
                                   SMEM_BYTES, c.stream, mQ, mK, mV, prm);
  note_launch();
  if (e != cudaSuccess) {
    set_error_detail("scored attention launch failed: %s", cudaGetErrorString(e));
    return TP_ERR_CUDA;
  }
  return TP_OK;
}

}  // namespace

cudaError_t launch_attention_mask(const LaunchCtx& c, const int32_t* off, int n_docs,
                                  const int32_t* prefix, bool causal, void* mask, int64_t T) {
  const MaskPlan plan = mask_plan(mask, T);
  const int32_t tiles = ceil_div(T, kAttnTile);
  cudaError_t e = launch_pdl(mask_rows_kernel, dim3(tiles), dim3(kAttnTile), 0, c.stream, off,
                             static_cast<int32_t>(n_docs), prefix, causal ? 1 : 0, plan,
                             static_cast<int32_t>(T));
  note_launch();
  if (e != cudaSuccess) return e;
  e = launch_pdl(mask_tiles_kernel, dim3(ceil_div(tiles, kAttnTile / 32)), dim3(kAttnTile), 0,
                 c.stream, plan, tiles);
  note_launch();
  return e;
}

tp_status launch_attention_scored(const LaunchCtx& c, const ScoreCall& a) {
  CUtensorMap mQ, mK, mV;
  if (!make_map_a(&mQ, a.Q, static_cast<int64_t>(a.hq) * DH, a.T, a.p) ||
      !make_map_a(&mK, a.K, static_cast<int64_t>(a.hkv) * DH, a.T, a.p) ||
      !make_map_a(&mV, a.V, static_cast<int64_t>(a.hkv) * DH, a.T, a.p))
    return TP_ERR_CUDA;
  ScoredParams prm{};
  prm.T = static_cast<int32_t>(a.T);
  prm.p = a.p;
  prm.hq = a.hq;
  prm.hkv = a.hkv;
  prm.group = a.hq / a.hkv;
  prm.q_blocks = ceil_div(a.T, BQ);
  prm.q_pairs = ceil_div(prm.q_blocks, NQT);
  prm.num_units = a.p * a.hq * prm.q_pairs;
  prm.causal = a.causal ? 1 : 0;
  prm.mask = mask_plan(a.mask, a.T);
  prm.s = score_consts(a.scale, a.cap);
  prm.slopes = a.slopes;
  prm.O = static_cast<__nv_bfloat16*>(a.O);
  prm.LSE = a.LSE;
  prm.wait.err = c.err_word;
  prm.wait.timeout_ns = c.timeout_ns;
  prm.debug_drop = c.debug_drop;
  if (a.cap > 0.0f) {
    if (a.slopes == nullptr && prm.s.cap_log2 <= kBoundLog2) return launch_mode<kCap>(c, prm, mQ, mK, mV);
    return launch_mode<kCapAny>(c, prm, mQ, mK, mV);
  }
  if (a.slopes != nullptr) return launch_mode<kBias>(c, prm, mQ, mK, mV);
  return launch_mode<kPlain>(c, prm, mQ, mK, mV);
}

}  // namespace tpk
