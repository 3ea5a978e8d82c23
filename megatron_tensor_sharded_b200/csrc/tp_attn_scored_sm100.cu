// Attention with capped scores, a distance bias, and document, prefix or
// causal masks: the forward pass, one persistent tcgen05 launch (sm_100a),
// and the mask's plan.
//
//   z_ij = cap tanh(scale q_i.k_j / cap) - slope |i - j|   over the keys that
//   row i sees, an interval [lo_i, hi_i);  O_i = sum_j softmax(z_i)_j v_j,
//   LSE_i = log sum_j exp z_ij.
//
// Bound by the tensor cores (4 * 128 flops a visible pair) and, with the cap,
// by the softmax's arithmetic beside them.  A unit is a (shard, query head,
// tile of 128 query rows); it walks blocks of 128 keys.  Sixteen warps do the
// softmax (a thread is a row and half of a block's columns: 64 scores) in two
// groups that take alternate blocks, so one group's waits and round trips to
// TMEM are covered by the other's arithmetic; three score buffers in TMEM let
// the tensor core run Q K^T up to three blocks ahead of P V.  (The form with
// two query tiles that share the K/V blocks, each with one score buffer,
// waited for the next scores after every block: 2780 clocks a tile and block
// with the cap, of 1040 of products.)  The probabilities stay in TMEM, over
// the scores they came from, as the A operand of P V.  A tensor-core
// instruction is issued only when the pipe takes it, so whatever else the
// issuing thread does adds to the products' time (90 clocks for a commit and a
// wait after eight of them): Q K^T and P V have a warp each, and one's waits
// run beside the other's products.  4096 causal tokens, 64 heads, cap: 353 us,
// 778 TFLOP/s; 2300 clocks a tile and block, of 1040 of products.
// Roles (640 threads): warp 0 loads Q, K (two slots) and V (three), warp 1
// issues Q K^T, warp 3 P V, warp 2 looks at V where a mask cuts a block, warps
// 4..11 and 12..19 are the two softmax groups.
//
// Running maximum (shared by a row's four threads): block by block, each
// group takes over the other's value as soon as it has its block's own
// maximum, moves it only when it grows by more than 2^8, and hands it on
// before its exponentials.  A group's sum follows when it next sees a larger
// maximum; sums and O meet at the unit's end, which each group does behind its
// first block of the next unit.
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
// Then there is no maximum pass over the scores and O is never rescaled.  The
// price is range: probabilities of 2^-80 to 2^80 leave V 2^128 / (2^80 T) upwards
// and 2^-46 downwards before O's fp32 sum ends (at a cap of 50 2^56 / T and
// 2^-54); the form with a maximum takes 390 to 410 us where this one takes 300.
//
// A key that a row does not see adds nothing to it, whatever K and V hold
// there: its score is replaced by -inf before the softmax, and where a mask
// cuts a block warp 2 zeroes the rows of V that hold an infinity or NaN
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
constexpr int NK = 2;                        // ring slots of K
constexpr int NV = 3;                        // ring slots of V
constexpr int NS = 3;                        // score buffers in TMEM
static_assert(NV == NS, "a group finds a block's score buffer and V slot at one index");
constexpr int TILE_BYTES = 128 * 128 * 2;
constexpr int HALF_BYTES = TILE_BYTES / 2;
constexpr int TILES_BYTES = (1 + NK + NV) * TILE_BYTES;
// floats: [group][half][row] maxima, [group][row] running maximum, and
// [unit parity][sum, maximum, mark][part][row] for the unit's end
constexpr int XCH_FLOATS = 2 * 2 * BQ + 2 * BQ + 2 * 3 * 4 * BQ;
constexpr int SMEM_BYTES = 1024 + TILES_BYTES + XCH_FLOATS * 4 + 512 + 2 * kOrderTiles * 2;
constexpr int NUM_THREADS = 640;
constexpr uint32_t IDESC_S = idesc_bf16_f32(BQ, BKV, 0, 0);
constexpr uint32_t IDESC_O = idesc_bf16_f32(BQ, DH, 0, 1);
constexpr uint32_t O_COL0 = NS * BKV, TMEM_COLS = 512;
constexpr float RESCALE_LOG2 = 8.0f;
constexpr float kBoundLog2 = 80.0f;          // |z| in log2 that needs no running maximum

// kCap: no bias, bounded; kCapAny: with a maximum; kCapFine: the same in the finer form
enum { kPlain = 0, kBias = 1, kCap = 2, kCapAny = 3, kCapFine = 4 };
static_assert(kCoarseCapLog2 <= kBoundLog2, "kCap: the caps of the coarse form need no maximum");

struct ScoredParams {
  int32_t T, p, hq, hkv, group, q_blocks, num_units, causal;
  MaskPlan mask;
  ScoreConsts s;
  const float* slopes;
  __nv_bfloat16* O;
  float* LSE;
  WaitCtl wait;
  int64_t debug_drop;
};

struct Unit {
  int32_t shard, head, kvh, qb;
  TileSpan t;
};

__device__ __forceinline__ Unit decode_unit(const ScoredParams& P, int32_t u, const uint16_t* order) {
  Unit x;
  const int32_t heads = P.p * P.hq;
  const int32_t level = u / heads, hh = u - level * heads;
  x.qb = order != nullptr ? order[level] : P.q_blocks - 1 - level;   // causal: the longest first
  x.shard = hh / P.hq;
  x.head = hh - x.shard * P.hq;
  x.kvh = x.head / P.group;
  x.t = tile_span(P.mask, x.qb, P.q_blocks, P.T, P.causal);
  return x;
}

// Rounds of gridDim.x units, alternately forwards and backwards over the CTAs.
__device__ __forceinline__ int32_t unit_of(int32_t r) {
  const int32_t g = static_cast<int32_t>(gridDim.x), b = static_cast<int32_t>(blockIdx.x);
  return r * g + ((r & 1) ? g - 1 - b : b);
}

// A walk over the blocks of the CTA's units (units without a block left out).
// With a bias a unit's last keys come first: near keys weigh most, so the
// maximum stands after the first block, and O is not rescaled block by block
// (4096 causal tokens, 64 heads: 375 us, 497 the other way round).  Without one
// the first keys do: causal rows see a whole block of them, not a corner, and
// their maximum hardly grows after it (294 us, 344 the other way round).
template <bool DOWN>
struct Walk {
  Unit x;
  int32_t r, u, j;   // round, unit, block
  uint32_t n, nu;    // blocks and units before this one
  bool first, done;  // the unit's first block; the walk is over
  const uint16_t* order;
  __device__ __forceinline__ void find(const ScoredParams& P) {
    for (; u < P.num_units; u = unit_of(++r)) {
      x = decode_unit(P, u, order);
      if (x.t.jb < x.t.je) {
        j = DOWN ? x.t.je - 1 : x.t.jb;
        first = true;
        return;
      }
    }
    done = true;
  }
  __device__ __forceinline__ void begin(const ScoredParams& P, const uint16_t* tiles) {
    order = tiles;
    r = 0;
    u = unit_of(0);
    n = nu = 0;
    done = false;
    find(P);
  }
  __device__ __forceinline__ bool last() const { return DOWN ? j == x.t.jb : j + 1 == x.t.je; }
  __device__ __forceinline__ void next(const ScoredParams& P) {
    ++n;
    first = false;
    if (DOWN ? --j >= x.t.jb : ++j < x.t.je) return;
    ++nu;
    u = unit_of(++r);
    find(P);
  }
};

// Of every eight pairs of probabilities, those whose 2^x runs as a polynomial
// on the FMA pipe, so that it and the MUFU unit (16 a clock and SM) are busy
// for about as long: an element costs the FMA pipe 6 clocks of a scheduler
// with the cap and 2 to 3 without, 9 more where 2^x is there too, and the MUFU
// unit 8 where it is not.
template <int MODE>
constexpr int kPolyPairs = MODE >= kCap ? 0 : 2;

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
                                            float dist0, int side, bool whole, uint32_t seen,
                                            bool& lost) {
  bool slow = false;
  if (MODE >= kCap)
    slow = cap_chunk<MODE == kCapFine, false>(v, S, !whole, seen);
  if (MODE == kBias || MODE >= kCapAny)
    bias_chunk<MODE == kBias>(v, S.scale_log2, slope2, dist0, side);
  if (!whole) mask_chunk(v, seen);
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
  const uint32_t sQ = base;
  auto sK = [&](uint32_t n) { return base + (1 + n % NK) * TILE_BYTES; };
  auto sV = [&](uint32_t n) { return base + (1 + NK + n % NV) * TILE_BYTES; };
  volatile float* const xch = reinterpret_cast<volatile float*>(smem_raw + (base - raw) + TILES_BYTES);
  volatile float* const run_m = xch + 2 * 2 * BQ;
  volatile float* const ends = run_m + 2 * BQ;
  uint8_t* const ctrl = smem_raw + (base - raw) + TILES_BYTES + XCH_FLOATS * 4;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(ctrl);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const uint32_t q_full = bar(0), q_empty = bar(1);
  auto k_full = [&](uint32_t n) { return bar(2 + n % NK); };
  auto k_empty = [&](uint32_t n) { return bar(4 + n % NK); };
  auto v_full = [&](uint32_t n) { return bar(6 + n % NV); };
  auto v_empty = [&](uint32_t n) { return bar(9 + n % NV); };
  auto s_full = [&](uint32_t n) { return bar(12 + n % NS); };
  // Barriers of a block are as many as it can be ahead of the block whose phase
  // somebody may still be waiting for: one a score buffer for p_full (a group
  // may finish block n + 2 while a load holds P V of block n up) and for
  // pv_done (a load may hold Q K^T up while P V of all its buffers completes).
  auto p_full = [&](uint32_t n) { return bar(15 + n % NS); };
  auto pv_done = [&](uint32_t n) { return bar(18 + n % NS); };
  auto v_seen = [&](uint32_t n) { return bar(21 + n % NV); };
  auto x_full = [&](uint32_t n) { return bar(24 + (n & 1)); };
  auto m_ready = [&](uint32_t n) { return bar(26 + (n & 1)); };
  const uint32_t o_full = bar(28), o_empty = bar(29), e_full = bar(30), drain = bar(31);
  constexpr int NBARS = 33;   // (drain: one for each issuing thread)
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 8 * NBARS);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* const bad = tmem_slot + 2;   // [NV][4]: keys of a block whose V is not finite

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < NK; ++i) {
      mbar_init(k_full(i), 1);
      mbar_init(k_empty(i), 1);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(v_full(i), 1);
      mbar_init(v_empty(i), 2);   // the issuing thread's commit, warp 2
      mbar_init(v_seen(i), 32);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), 256);
      mbar_init(pv_done(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(x_full(i), 256);
      mbar_init(m_ready(i), 256);
    }
    mbar_init(o_full, 1);
    mbar_init(o_empty, 512);
    mbar_init(e_full, 512);
    mbar_init(drain, 1);
    mbar_init(drain + 8, 1);
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
  uint16_t* const order_smem = reinterpret_cast<uint16_t*>(ctrl + 512);
  const uint16_t* const order =
      order_tiles(P.mask, P.q_blocks, P.T, P.causal, P.num_units <= static_cast<int32_t>(gridDim.x),
                  order_smem, order_smem + kOrderTiles);

  constexpr bool DOWN = MODE == kBias || MODE >= kCapAny;
  Walk<DOWN> w;
  // 96 registers a thread at launch: 128 x 64 + 512 x 104 <= 640 x 96
  if (warp < 4) {
    regs_shrink<64>();
    if (warp == 0) {
      if (lane == 0) {
        // ------------------------------------------------- Q, K and V loads
        // K runs NK blocks ahead of V: a walk each.
        Walk<DOWN> a;
        a.begin(P, order);
        int64_t nk = 0;
        uint32_t nv = 0, units = 0;
        auto load_k = [&]() {
          if (a.done) return true;
          if (a.first) {
            if (!wait_asleep(q_empty, (a.nu & 1) ^ 1u, abort_flag, P.wait, kErrWaitAttn)) return false;
            mbar_arrive_expect_tx(q_full, TILE_BYTES);
            for (int c = 0; c < 2; ++c)
              tma_load_3d(sQ + c * HALF_BYTES, &mapQ, q_full, a.x.head * DH + c * 64, a.x.qb * BQ,
                          a.x.shard);
            ++units;
          }
          if (!wait_asleep(k_empty(a.n), ((a.n / NK) & 1) ^ 1u, abort_flag, P.wait, kErrWaitEmpty))
            return false;
          if (nk != P.debug_drop) {
            mbar_arrive_expect_tx(k_full(a.n), TILE_BYTES);
            for (int c = 0; c < 2; ++c)
              tma_load_3d(sK(a.n) + c * HALF_BYTES, &mapK, k_full(a.n), a.x.kvh * DH + c * 64,
                          a.j * BKV, a.x.shard);
          }
          ++nk;
          a.next(P);
          return true;
        };
        bool ok = true;
        for (int i = 0; ok && i < NK; ++i) ok = load_k();
        for (w.begin(P, order); ok && !w.done; w.next(P)) {
          if (!wait_asleep(v_empty(w.n), ((w.n / NV) & 1) ^ 1u, abort_flag, P.wait, kErrWaitEmpty)) break;
          mbar_arrive_expect_tx(v_full(w.n), TILE_BYTES);
          for (int c = 0; c < 2; ++c)
            tma_load_3d(sV(w.n) + c * HALF_BYTES, &mapV, v_full(w.n), w.x.kvh * DH + c * 64, w.j * BKV,
                        w.x.shard);
          ++nv;
          ok = load_k();
        }
        // Teardown: let the last loads land before shared memory is released.
        if (units > 0) wait_teardown(q_full, (units - 1) & 1, P.wait);
        for (int64_t i = nk > NK ? nk - NK : 0; i < nk; ++i)
          if (i != P.debug_drop)
            wait_teardown(k_full(static_cast<uint32_t>(i)), static_cast<uint32_t>((i / NK) & 1), P.wait);
        for (uint32_t i = nv > NV ? nv - NV : 0; i < nv; ++i) wait_teardown(v_full(i), (i / NV) & 1, P.wait);
      }
      __syncwarp();
    } else if (warp == 1) {
      {
        // --------------------------------------------------- S = Q K^T issuer
        // The whole warp goes through the loop and one lane issues: what the
        // products' operands are made of is then the same for the warp, and
        // stays in uniform registers.
        const bool leader = elect_one();
        auto await = [&](uint32_t bar, uint32_t parity, unsigned code) {
          return __all_sync(0xffffffffu, wait_asleep(bar, parity, abort_flag, P.wait, code)) != 0;
        };
        for (w.begin(P, order); !w.done; w.next(P)) {
          if ((w.first && !await(q_full, w.nu & 1, kErrWaitFull)) ||
              !await(k_full(w.n), (w.n / NK) & 1, kErrWaitFull) ||
              // the buffer's last probabilities have been used
              (w.n >= NS && !await(pv_done(w.n - NS), ((w.n - NS) / NS) & 1, kErrWaitAttn)))
            break;
          tc_fence_after();
          const uint32_t q = desc_lo(sQ, 16), k = desc_lo(sK(w.n), 16);
          const uint32_t d = tmem_base + (w.n % NS) * BKV;
#pragma unroll
          for (int kk = 0; leader && kk < DH / 16; ++kk) {
            const uint32_t off = desc_step((kk >> 2) * HALF_BYTES + (kk & 3) * 32);
            tc_mma_f16_lo(d, q + off, k + off, IDESC_S, kk > 0 ? 1u : 0u);
          }
          if (leader) tc_commit(s_full(w.n));
          if (leader) tc_commit(k_empty(w.n));
          if (leader && w.last()) tc_commit(q_empty);
        }
        if (leader) tc_commit(drain);
        wait_teardown(drain, 0, P.wait);
      }
      __syncwarp();
    } else if (warp == 3) {
      {
        // ------------------------------------------------- O += P V issuer
        // (the same way)
        const bool leader = elect_one();
        auto await = [&](uint32_t bar, uint32_t parity, unsigned code) {
          return __all_sync(0xffffffffu, wait_asleep(bar, parity, abort_flag, P.wait, code)) != 0;
        };
        for (w.begin(P, order); !w.done; w.next(P)) {
          if ((w.first && w.nu > 0 &&
               !await(o_empty, (w.nu - 1) & 1, kErrWaitAttn)) ||
              !await(v_seen(w.n), (w.n / NV) & 1, kErrWaitFull) ||
              !await(p_full(w.n), (w.n / NS) & 1, kErrWaitAttn))
            break;
          tc_fence_after();
          const uint32_t v = desc_lo(sV(w.n), HALF_BYTES), pa = tmem_base + (w.n % NS) * BKV;
#pragma unroll
          for (int kk = 0; leader && kk < BKV / 16; ++kk)
            tc_mma_f16_ts_lo(tmem_base + O_COL0, pa + (kk >> 2) * 64 + (kk & 3) * 8,
                             v + desc_step(kk * 16 * 128), IDESC_O, (!w.first || kk > 0) ? 1u : 0u);
          if (leader) tc_commit(pv_done(w.n));
          if (leader) tc_commit(v_empty(w.n));
          if (leader && w.last()) tc_commit(o_full);
        }
        if (leader) tc_commit(drain + 8);
        wait_teardown(drain + 8, 0, P.wait);
      }
      __syncwarp();
    } else {
      // ----------------------------------- values in blocks that a mask cuts
      for (w.begin(P, order); !w.done; w.next(P)) {
        bool ok = wait_asleep(v_full(w.n), (w.n / NV) & 1, abort_flag, P.wait, kErrWaitFull);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (!w.x.t.whole(w.j)) {
#pragma unroll 1
          for (int h = 0; h < 4; ++h) {
            const int row = h * 32 + lane;
            const bool is_bad = row_not_finite(sV(w.n), row);
            const uint32_t m = __ballot_sync(0xffffffffu, is_bad);
            if (is_bad) zero_row(sV(w.n), row);
            if (lane == 0) bad[(w.n % NV) * 4 + h] = m;
          }
          fence_proxy_async_smem();
        }
        mbar_arrive(v_seen(w.n));
        __syncwarp();
        if (lane == 0) mbar_arrive(v_empty(w.n));
      }
    }
  } else {
    regs_grow<104>();
    // ------------------------------------------------------- softmax / output
    // thread = row and column half: scores [64 half, 64 half + 64) of its
    // group's blocks, and 32 columns of O
    const int g = (warp - 4) / 8;
    const int half = ((warp - 4) / 4) & 1;
    const int part = g * 2 + half;
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tO = tmem_base + lane_off + O_COL0;
    constexpr bool HAS_MAX = MODE != kCap;
    const ScoreConsts& S = P.s;
    bool ok = true;
    float m = HAS_MAX ? -INFINITY : 0.0f, l = 0.0f;
    bool poison = false, lost = false;
    // the unit whose end is still to be done
    bool pending = false;
    uint32_t p_nu = 0;
    int64_t p_row = -1;       // its row in O [.. * head_dim], -1: not stored
    int64_t p_lse = 0;
    auto wait = [&](uint32_t b, uint32_t parity) {
      const bool got = wait_asleep(b, parity, abort_flag, P.wait, kErrWaitAttn);
      return __all_sync(0xffffffffu, got) != 0;
    };
    auto finish = [&]() {
      pending = false;
      if (!wait(e_full, p_nu & 1) || !wait(o_full, p_nu & 1)) return false;
      tc_fence_after();
      const volatile float* e = ends + (p_nu & 1) * 3 * 4 * BQ + row;
      // the row's sum over its four threads, each under its own last maximum
      float M = 0.0f;
      if (HAS_MAX) {
        M = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i) M = max3_nan(M, e[(4 + i) * BQ], M);
      }
      float L = 0.0f, mark = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float mi = HAS_MAX ? e[(4 + i) * BQ] : 0.0f, li = e[i * BQ];
        L += mi == M ? li : li * ex2(mi - M);
        mark += e[(8 + i) * BQ];
      }
      // (M = inf: some score is, the softmax is NaN and its polynomial 2^x would
      // hide it; M = -inf: all are, and nothing has a weight)
      const bool none = L == 0.0f || (HAS_MAX && M == -INFINITY), over = HAS_MAX && M == INFINITY;
      const float inv_l = mark != 0.0f || over ? NAN : none ? 0.0f : 1.0f / L;
      uint32_t v[32];
      tmem_ld_32x32b_x32(tO + part * 32, v);
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(o_empty);
      if (p_row >= 0) {
        __nv_bfloat16* dst = P.O + p_row + part * 32;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            o[i] = pack2(__uint_as_float(v[q * 8 + 2 * i]) * inv_l,
                         __uint_as_float(v[q * 8 + 2 * i + 1]) * inv_l);
          *reinterpret_cast<uint4*>(dst + q * 8) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        if (part == 0 && P.LSE != nullptr)
          P.LSE[p_lse] = over ? INFINITY : none ? -INFINITY : 0.6931471805599453f * M + logf(L);
      }
      return true;
    };
    // Blocks are counted through the CTA's units; a group's are every second
    // one, so from one to the next the score buffer moves on by two.
    uint32_t slot = g, phase = 0;      // n % NS and (n / NS) & 1 of the group's next block
    uint32_t turn = 0;                 // (n >> 1) & 1
    uint32_t nu = 0, parity0 = 0;      // units, and the parity of a unit's first block
    bool started = g == 1;             // a block came before (of either group)
    int32_t r = 0;
    for (int32_t u = unit_of(0); ok && u < P.num_units; u = unit_of(++r)) {
      const Unit x = decode_unit(P, u, order);
      const int32_t blocks = x.t.je - x.t.jb;
      if (blocks <= 0) continue;
      const int32_t q = x.qb * BQ + row;
      const int2 seen = row_span(P.mask, q, P.T, P.causal);
      float slope2 = 0.0f;
      if (MODE == kBias || MODE >= kCapAny)
        slope2 = P.slopes != nullptr ? 1.4426950408889634f * P.slopes[x.shard * P.hq + x.head] : 0.0f;
      for (int32_t i = (static_cast<uint32_t>(g) ^ parity0) & 1; i < blocks; i += 2) {
        // (a group that enters the unit with its second block does the previous
        // unit's end first, since the first block's P V waits for it; with a
        // maximum its block comes first, and measured 7% better)
        if (!HAS_MAX && pending && i > 0 && !finish()) {
          ok = false;
          break;
        }
        const int32_t j = DOWN ? x.t.je - 1 - i : x.t.jb + i;
        const uint32_t tS = tmem_base + lane_off + slot * BKV + half * 64;
        const bool whole = x.t.whole(j);
        const int32_t key0 = j * BKV + half * 64;
        if (!wait(s_full(slot), phase)) {
          ok = false;
          break;
        }
        tc_fence_after();
        auto columns = [&](int c) {   // that the row sees, of a chunk of a cut block
          return columns_in(seen.x - key0 - c * 32, seen.y - key0 - c * 32);
        };
        float dist0 = 0.0f;
        int side = 0;
        if (MODE == kBias || MODE >= kCapAny) {
          dist0 = static_cast<float>(key0 - q);
          side = j * BKV + BKV - 1 <= x.qb * BQ ? -1 : j * BKV >= x.qb * BQ + BQ - 1 ? 1 : 0;
        }
        uint64_t sum2[2] = {f2_pack(0.0f, 0.0f), f2_pack(0.0f, 0.0f)};
        // (loops kept rolled: the instruction cache holds one chunk's code)
        if (HAS_MAX) {
          float acc[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(tS + c * 32, v);
            tmem_ld_wait();
            score_chunk<MODE>(v, S, slope2, dist0 + c * 32.0f, side, whole, columns(c), lost);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              acc[0] = max3_nan(acc[0], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
              acc[1] = max3_nan(acc[1], __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
            }
            if (MODE >= kCapAny) tmem_st_32x32b_x32(tS + c * 32, v);   // (else computed again below)
          }
          if (MODE >= kCapAny) tmem_st_wait();
          float m_cand = max3_nan(acc[0], acc[1], acc[1]);
          // the other group's maximum first: its arrival also says that this
          // group's last exchange has been read
          if (started && !wait(m_ready(g ^ 1), turn ^ (g ^ 1))) {
            ok = false;
            break;
          }
          const float m_prev = i == 0 ? -INFINITY : run_m[(g ^ 1) * BQ + row];
          xch[part * BQ + row] = m_cand;
          mbar_arrive(x_full(g));
          if (!wait(x_full(g), turn)) {
            ok = false;
            break;
          }
          const float other = xch[(part ^ 1) * BQ + row];
          m_cand = max3_nan(m_cand, other, other);
          if (MODE == kPlain) m_cand *= S.scale_log2;
          const bool grow = !(m_cand <= m_prev + RESCALE_LOG2);   // NaN too: it then stays
          const float m_new = grow ? m_cand : m_prev;
          if (half == 0) run_m[g * BQ + row] = m_new;
          mbar_arrive(m_ready(g));
          if (m != m_new) l *= ex2(m - m_new);
          m = m_new;
          if (i > 0 && __any_sync(0xffffffffu, grow)) {
            // O is whole once P V of the block before this one is done, which
            // itself waits for the end of the previous unit
            const uint32_t before = slot == 0 ? NS - 1 : slot - 1;
            if ((pending && !finish()) || !wait(pv_done(before), slot == 0 ? phase ^ 1u : phase)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const float alpha = grow ? ex2(m_prev - m_new) : 1.0f;
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              uint32_t v[32];
              tmem_ld_32x32b_x32(tO + half * 64 + c * 32, v);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
              tmem_st_32x32b_x32(tO + half * 64 + c * 32, v);
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
          if (MODE == kPlain && !whole) mask_chunk(v, columns(c));
          if (MODE == kCap || MODE == kBias)
            score_chunk<MODE>(v, S, slope2, dist0 + c * 32.0f, side, whole, columns(c), lost);
          exp_chunk<kPolyPairs<MODE>, HAS_MAX>(v, f2_pack(scale, scale), f2_pack(off, off), sum2, pk);
          tmem_st_32x32b_x16(tS + c * 16, pk);
        }
        tmem_st_wait();
        if (!whole) {   // keys in sight whose value is not finite
          if (!wait(v_seen(slot), phase)) {
            ok = false;
            break;
          }
          const volatile uint32_t* b = bad + slot * 4 + half * 2;
          const uint32_t b0 = b[0], b1 = b[1];
          if (b0 | b1) poison |= ((b0 & columns(0)) | (b1 & columns(1))) != 0;
        }
        tc_fence_before();
        mbar_arrive(p_full(slot));
        float s0, s1, s2, s3;
        f2_unpack(sum2[0], s0, s1);
        f2_unpack(sum2[1], s2, s3);
        l += (s0 + s1) + (s2 + s3);
        slot += 2;
        if (slot >= NS) {
          slot -= NS;
          phase ^= 1u;
        }
        turn ^= 1u;
        started = true;
        if (pending && !finish()) {
          ok = false;
          break;
        }
      }
      if (!ok || (pending && !finish())) break;
      parity0 ^= blocks & 1;
      // this unit's sums; its end follows
      volatile float* e = ends + (nu & 1) * 3 * 4 * BQ + row;
      e[part * BQ] = lost ? NAN : l;
      if (HAS_MAX) e[(4 + part) * BQ] = m;
      e[(8 + part) * BQ] = poison ? 1.0f : 0.0f;
      mbar_arrive(e_full);
      pending = true;
      p_nu = nu++;
      const bool store = q < P.T && seen.y >= 0;   // rows of no document stay as they were
      p_row = store ? ((static_cast<int64_t>(x.shard) * P.T + q) * P.hq + x.head) * DH : -1;
      p_lse = (static_cast<int64_t>(x.shard) * P.hq + x.head) * P.T + q;
      m = HAS_MAX ? -INFINITY : 0.0f;
      l = 0.0f;
      poison = lost = false;
    }
    if (ok && pending) finish();
  }

  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// ------------------------------------------------------------- mask's plan
// One CTA per tile of 128 rows: each row finds its document (binary search of
// the offsets) and writes the keys it sees and the queries that see it; the
// tile's summary as queries and as keys follows.
__global__ void __launch_bounds__(kAttnTile)
    mask_plan_kernel(const int32_t* __restrict__ off, int32_t n_docs,
                     const int32_t* __restrict__ prefix, int32_t causal, MaskPlan plan, int32_t T) {
  __shared__ int32_t red[6][kAttnTile / 32];
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
  // least and greatest of each, as minima
  int32_t v[6] = {in ? lo : INT_MAX, in ? -hi : 0,  t < T ? -lo : 0,
                  t < T ? hi : INT_MAX, in ? by.x : INT_MAX, in ? -by.y : 0};
#pragma unroll
  for (int i = 0; i < 6; ++i) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v[i] = min(v[i], __shfl_xor_sync(0xffffffffu, v[i], o));
    if (threadIdx.x % 32 == 0) red[i][threadIdx.x / 32] = v[i];
  }
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < 6; ++i)
      for (int w = 1; w < kAttnTile / 32; ++w) v[i] = min(v[i], red[i][w]);
    plan.q_tiles[blockIdx.x] = make_int4(v[0], -v[1], -v[2], v[3]);
    plan.k_tiles[blockIdx.x] = v[4] < -v[5] ? make_int2(v[4] / kAttnTile, (-v[5] - 1) / kAttnTile + 1)
                                            : make_int2(0, 0);
  }
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
  const cudaError_t e = launch_pdl(mask_plan_kernel, dim3(tiles), dim3(kAttnTile), 0, c.stream, off,
                                   static_cast<int32_t>(n_docs), prefix, causal ? 1 : 0, plan,
                                   static_cast<int32_t>(T));
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
  prm.num_units = a.p * a.hq * prm.q_blocks;
  prm.causal = a.causal ? 1 : 0;
  prm.mask = mask_plan(a.mask, a.T);
  prm.s = score_consts(a.scale, a.cap);
  prm.slopes = a.slopes;
  prm.O = static_cast<__nv_bfloat16*>(a.O);
  prm.LSE = a.LSE;
  prm.wait.err = c.err_word;
  prm.wait.timeout_ns = c.timeout_ns;
  prm.debug_drop = c.debug_drop;
  const int form = cap_form(prm.s);
  if (form == kFineCap) return launch_mode<kCapFine>(c, prm, mQ, mK, mV);
  if (form == kCoarseCap && a.slopes != nullptr) return launch_mode<kCapAny>(c, prm, mQ, mK, mV);
  if (form == kCoarseCap) return launch_mode<kCap>(c, prm, mQ, mK, mV);
  if (a.slopes != nullptr) return launch_mode<kBias>(c, prm, mQ, mK, mV);
  return launch_mode<kPlain>(c, prm, mQ, mK, mV);
}

}  // namespace tpk
