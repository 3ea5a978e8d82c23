// Backward of scored attention (sm_100a): three launches.
//
// With P = exp(z - LSE), D_i = sum_d dO_id O_id and t the cap's tanh,
//   dV_j = sum_i P_ij dO_i,   dS_ij = P_ij (dO_i.v_j - D_i) (1 - t_ij^2),
//   dQ_i = scale sum_j dS_ij k_j,   dK_j = scale sum_i dS_ij q_i,
// dK and dV summed over the query heads that share a key/value head.
//
// 1. score_delta_kernel: D, one pass over O and dO (HBM-bound).
// 2. tc_scored_dkv_kernel: a unit is (shard, key/value head, 128 keys) and
//    walks every query tile that sees them, for every query head of the
//    group: dK and dV stay in TMEM from the first to the last, so the sum
//    over heads costs nothing and has a fixed order.
// 3. tc_scored_dq_kernel: a unit is (shard, query head, 128 queries) and walks
//    its key blocks with dQ in TMEM.
// Scores and probabilities are recomputed in both: seven products a tile
// instead of the five that one kernel with atomic adds to dQ would need, in
// exchange for the same bits on every run, no fp32 dQ in memory and no pass
// that converts it.  Both are bound by the tensor cores (4 and 3 products of
// 128 x 128 x 128 a tile) with the softmax's arithmetic beside them.
//
// dkv computes the transposed tiles S^T = K Q^T and dP^T = V dO^T: a thread
// then owns a key row, and P^T and dS^T, left in TMEM as bf16, are the A
// operands of dV += P^T dO and dK += dS^T Q, whose B operands are the tiles
// that S^T and dP^T read: no operand is transposed or written to shared
// memory.  dq likewise: dQ += dS K.  The sixteen arithmetic warps split a tile
// by column quarters; each quarter's bf16 result goes over the first half of
// its own scores, so the quarters never wait for one another.  The tensor core runs dV and the next S^T while the warps form
// dS^T, and dK and the next dP^T while they form P^T.
//
// Masks, and rows that hold infinities or NaN outside what is seen, as in the
// forward kernel; here the tiles of Q and dO (dkv) and of K (dq) are looked at.
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
constexpr int NST = 2;                       // ring slots of the walked pair of tiles
constexpr int TILE_BYTES = 128 * 128 * 2;
constexpr int HALF_BYTES = TILE_BYTES / 2;
constexpr int VEC_BYTES = 4 * BT * 4;        // per slot: -LSE log2 e, D, first and last + 1 key in sight
constexpr int SMEM_BYTES = 1024 + 2 * TILE_BYTES + NST * 2 * TILE_BYTES + NST * VEC_BYTES + 512;   // + barriers, flags
constexpr int NUM_THREADS = 640;
constexpr int ARITH = 512;                   // threads that form P and dS
constexpr uint32_t IDESC_KK = idesc_bf16_f32(BT, BT, 0, 0);   // both operands along head_dim
constexpr uint32_t IDESC_KN = idesc_bf16_f32(BT, DH, 0, 1);   // A in TMEM, B rows x head_dim
// Of every eight pairs of probabilities, those whose 2^x runs on the FMA pipe:
// none with the cap, whose own arithmetic there (11 clocks of a scheduler an
// element against the MUFU unit's 8) is the longer already.
template <bool CAP>
constexpr int kPolyPairs = CAP ? 0 : 2;
constexpr float kLog2e = 1.4426950408889634f;

struct BwdParams {
  int32_t T, p, hq, hkv, group, tiles, num_units, causal;
  MaskPlan mask;
  ScoreConsts s;
  float neg_inv_cap2;       // -(cap log2 e)^-2: 1 - tanh^2 = 1 + z^2 times it
  const float* slopes;
  const float* LSE;
  const float* delta;
  __nv_bfloat16 *dQ, *dK, *dV;
  WaitCtl wait;
  int64_t debug_drop;
};

__device__ __forceinline__ int32_t unit_of(int32_t r) {
  const int32_t g = static_cast<int32_t>(gridDim.x), b = static_cast<int32_t>(blockIdx.x);
  return r * g + ((r & 1) ? g - 1 - b : b);
}

// A product of two shared-memory tiles along head_dim: D = A B^T.
__device__ __forceinline__ void mma_tiles(uint32_t d, uint32_t a, uint32_t b) {
#pragma unroll
  for (int kk = 0; kk < DH / 16; ++kk) {
    const uint32_t off = (kk >> 2) * HALF_BYTES + (kk & 3) * 32;
    tc_mma_f16(d, smem_desc_sw128(a + off, 16, 1024), smem_desc_sw128(b + off, 16, 1024), IDESC_KK,
               kk > 0 ? 1u : 0u);
  }
}
// D (+)= A B with A (bf16, each column quarter at its 32 columns' start) in
// TMEM and B's 128 rows the contraction.
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint32_t b, bool add) {
#pragma unroll
  for (int kk = 0; kk < BT / 16; ++kk)
    tc_mma_f16_ts(d, a + (kk >> 1) * 32 + (kk & 1) * 8,
                  smem_desc_sw128(b + kk * 16 * 128, HALF_BYTES, 1024), IDESC_KN,
                  (add || kk > 0) ? 1u : 0u);
}

__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                          int32_t head, int32_t row, int32_t shard) {
  for (int c = 0; c < 2; ++c)
    tma_load_3d(dst + c * HALF_BYTES, map, bar, head * DH + c * 64, row, shard);
}

// 32 raw products -> P as bf16 pairs in pk and w = P (1 - tanh^2).  nl(e):
// -LSE log2 e of columns e and e + 1; seen(e): whether the pair counts.
template <bool CAP, bool BIAS, typename NegLse, typename Seen>
__device__ __forceinline__ void prob_chunk(uint32_t (&v)[32], float (&w)[32], uint32_t (&pk)[16],
                                           const BwdParams& P, float slope2, float dist0, int side,
                                           bool cut, NegLse nl, Seen seen) {
  if (CAP) {
    cap_chunk(v, P.s);
    const uint64_t ic = f2_pack(P.neg_inv_cap2, P.neg_inv_cap2), one = f2_pack(1.0f, 1.0f);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const uint64_t z = f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
      f2_unpack(f2_fma(f2_mul(z, z), ic, one), w[e], w[e + 1]);
    }
  }
  if (BIAS) bias_chunk<!CAP>(v, P.s.scale_log2, slope2, dist0, side);
  const uint64_t sc2 = f2_pack(P.s.scale_log2, P.s.scale_log2);
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    uint64_t x = f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
    x = CAP || BIAS ? f2_add(x, nl(e)) : f2_fma(x, sc2, nl(e));
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
      if (!seen(e)) {
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

// 32 products dP -> dS = w (dP - D) as bf16 pairs; nd(e): -D of columns e, e + 1.
template <typename NegDelta, typename Seen>
__device__ __forceinline__ void grad_chunk(uint32_t (&v)[32], const float (&w)[32],
                                           uint32_t (&pk)[16], bool cut, NegDelta nd, Seen seen) {
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const uint64_t x = f2_add(f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), nd(e));
    float a, b;
    f2_unpack(f2_mul(x, f2_pack(w[e], w[e + 1])), a, b);
    v[e] = __float_as_uint(a);
    v[e + 1] = __float_as_uint(b);
  }
  if (cut) {   // 0 * NaN from what is not seen
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!seen(e)) v[e] = 0;
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

__device__ __forceinline__ float lds(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint64_t lds2(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// ------------------------------------------------------------------ delta
// D[shard][head][t] = sum over the head of dO * O: 16 lanes a row.
__global__ void __launch_bounds__(256)
    score_delta_kernel(const __nv_bfloat16* __restrict__ O, const __nv_bfloat16* __restrict__ dO,
                       float* __restrict__ delta, int64_t rows, int32_t T, int32_t hq) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 16 + threadIdx.x / 16;   // [shard][t][head]
  const int lane = threadIdx.x % 16;
  float s = 0.0f;
  if (row < rows) {
    const uint4 a = *reinterpret_cast<const uint4*>(O + row * DH + lane * 8);
    const uint4 b = *reinterpret_cast<const uint4*>(dO + row * DH + lane * 8);
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s += __uint_as_float(x[i] << 16) * __uint_as_float(y[i] << 16);
      s += __uint_as_float(x[i] & 0xffff0000u) * __uint_as_float(y[i] & 0xffff0000u);
    }
  }
#pragma unroll
  for (int o = 8; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (row < rows && lane == 0) {
    const int64_t st = row / hq;            // shard * T + t
    const int64_t shard = st / T;
    delta[(shard * hq + row % hq) * T + (st - shard * T)] = s;
  }
}

// ---------------------------------------------------------------- dK and dV
struct KeyUnit {
  int32_t shard, kvh, kb, ia, ib;   // query tiles [ia, ib)
};
__device__ __forceinline__ KeyUnit key_unit(const BwdParams& P, int32_t u) {
  KeyUnit x;
  const int32_t heads = P.p * P.hkv;
  x.kb = u / heads;                 // causal: the first keys are seen by most
  const int32_t hh = u % heads;
  x.shard = hh / P.hkv;
  x.kvh = hh % P.hkv;
  if (P.mask.rows != nullptr) {
    const int2 t = P.mask.k_tiles[x.kb];
    x.ia = t.x;
    x.ib = t.y;
  } else {
    x.ia = P.causal ? x.kb : 0;
    x.ib = P.tiles;
  }
  return x;
}

template <bool CAP, bool BIAS>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    tc_scored_dkv_kernel(const __grid_constant__ CUtensorMap mapQ,
                         const __grid_constant__ CUtensorMap mapK,
                         const __grid_constant__ CUtensorMap mapV,
                         const __grid_constant__ CUtensorMap mapdO,
                         const __grid_constant__ BwdParams P) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t sK = base, sV = base + TILE_BYTES;
  auto sQ = [&](uint32_t st) { return base + 2 * TILE_BYTES + st * 2 * TILE_BYTES; };
  auto sdO = [&](uint32_t st) { return sQ(st) + TILE_BYTES; };
  constexpr int RING_END = 2 * TILE_BYTES + NST * 2 * TILE_BYTES;
  auto vec = [&](uint32_t st, int which) { return base + RING_END + st * VEC_BYTES + which * BT * 4; };
  uint8_t* const ctrl = smem_raw + (base - raw) + RING_END + NST * VEC_BYTES;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(ctrl);
  const uint32_t kv_full = smem_u32(&bars[0]), kv_empty = smem_u32(&bars[1]);
  auto qd_full = [&](uint32_t s) { return smem_u32(&bars[2 + s]); };
  auto qd_empty = [&](uint32_t s) { return smem_u32(&bars[4 + s]); };
  auto vec_full = [&](uint32_t s) { return smem_u32(&bars[6 + s]); };
  const uint32_t s_full = smem_u32(&bars[8]), dp_full = smem_u32(&bars[9]);
  const uint32_t p_full = smem_u32(&bars[10]), ds_full = smem_u32(&bars[11]);
  const uint32_t acc_full = smem_u32(&bars[12]), acc_empty = smem_u32(&bars[13]);
  const uint32_t drain = smem_u32(&bars[14]);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 8 * 15);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* const cut_flag = tmem_slot + 2;   // [NST]: the step's tile is cut by a mask
  volatile uint32_t* const bad = tmem_slot + 4;        // [NST][4]: its rows of dO or Q that are not finite
  // [3][4]: keys that see one, by unit number mod 3 (set by any column
  // quarter's thread of the key, read by all at the unit's end; cleared two
  // units ahead, when the last reader of the slot has moved on)
  uint32_t* const hit = tmem_slot + 4 + NST * 4;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    mbar_init(kv_empty, 1);
    for (int s = 0; s < NST; ++s) {
      mbar_init(qd_full(s), 1);
      mbar_init(qd_empty(s), 3);   // the MMA thread's commit, warps 2 and 3
      mbar_init(vec_full(s), 64);
    }
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(p_full, ARITH);
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
  // The dq kernel behind this one reads only what was complete before this
  // point; it may start on SMs that this one leaves (it waits at its end).
  pdl_wait();
  pdl_launch_dependents();

  // 96 registers a thread at launch: 128 x 64 + 512 x 104 <= 640 x 96
  if (warp < 4) {
    regs_shrink<64>();
    if (warp == 0) {
      if (lane == 0) {
        // ---------------------------------------------------------- producer
        uint32_t nu = 0;
        int64_t n = 0;
        bool ok = true;
        int32_t r = 0;
        for (int32_t u = unit_of(0); ok && u < P.num_units; u = unit_of(++r)) {
          const KeyUnit x = key_unit(P, u);
          if (x.ia >= x.ib) continue;
          if (!wait_bounded(kv_empty, (nu & 1) ^ 1u, abort_flag, P.wait, kErrWaitAttn)) break;
          mbar_arrive_expect_tx(kv_full, 2 * TILE_BYTES);
          load_tile(sK, &mapK, kv_full, x.kvh, x.kb * BT, x.shard);
          load_tile(sV, &mapV, kv_full, x.kvh, x.kb * BT, x.shard);
          ++nu;
          for (int32_t g = 0; ok && g < P.group; ++g) {
            const int32_t head = x.kvh * P.group + g;
            for (int32_t i = x.ia; i < x.ib; ++i, ++n) {
              const uint32_t st = n % NST;
              if (!wait_bounded(qd_empty(st), ((n / NST) & 1) ^ 1u, abort_flag, P.wait,
                                kErrWaitEmpty)) {
                ok = false;
                break;
              }
              if (n != P.debug_drop) {
                mbar_arrive_expect_tx(qd_full(st), 2 * TILE_BYTES);
                load_tile(sQ(st), &mapQ, qd_full(st), head, i * BT, x.shard);
                load_tile(sdO(st), &mapdO, qd_full(st), head, i * BT, x.shard);
              }
            }
          }
        }
        // Teardown: let the last loads land before shared memory is released.
        if (nu > 0) wait_teardown(kv_full, (nu - 1) & 1, P.wait);
        for (int64_t q = n > NST ? n - NST : 0; q < n; ++q)
          if (q != P.debug_drop)
            wait_teardown(qd_full(static_cast<uint32_t>(q % NST)),
                          static_cast<uint32_t>((q / NST) & 1), P.wait);
      }
      __syncwarp();
    } else if (warp == 1) {
      if (lane == 0) {
        // -------------------------------------------------------- MMA issuer
        uint32_t n = 0, nu = 0;
        bool ok = true;
        auto wait_qd = [&](uint32_t m) {
          return wait_bounded(qd_full(m % NST), (m / NST) & 1, abort_flag, P.wait, kErrWaitFull);
        };
        int32_t r = 0;
        for (int32_t u = unit_of(0); ok && u < P.num_units; u = unit_of(++r)) {
          const KeyUnit x = key_unit(P, u);
          const int32_t steps = P.group * (x.ib - x.ia);
          if (x.ia >= x.ib) continue;
          if (!wait_bounded(kv_full, nu & 1, abort_flag, P.wait, kErrWaitFull) || !wait_qd(n)) break;
          tc_fence_after();
          mma_tiles(tS, sK, sQ(n % NST));
          tc_commit(s_full);
          mma_tiles(tdP, sV, sdO(n % NST));
          tc_commit(dp_full);
          if (steps == 1) tc_commit(kv_empty);
          for (int32_t s = 0; s < steps; ++s, ++n) {
            const uint32_t st = n % NST, nx = (n + 1) % NST;
            const bool more = s + 1 < steps;
            if (!wait_bounded(p_full, n & 1, abort_flag, P.wait, kErrWaitAttn) ||
                (s == 0 && nu > 0 &&
                 !wait_bounded(acc_empty, (nu - 1) & 1, abort_flag, P.wait, kErrWaitAttn))) {
              ok = false;
              break;
            }
            tc_fence_after();
            mma_rows(tdV, tS, sdO(st), s > 0);
            if (more) {
              if (!wait_qd(n + 1)) {
                ok = false;
                break;
              }
              tc_fence_after();
              mma_tiles(tS, sK, sQ(nx));
              tc_commit(s_full);
            }
            if (!wait_bounded(ds_full, n & 1, abort_flag, P.wait, kErrWaitAttn)) {
              ok = false;
              break;
            }
            tc_fence_after();
            mma_rows(tdK, tdP, sQ(st), s > 0);
            tc_commit(qd_empty(st));
            if (more) {
              mma_tiles(tdP, sV, sdO(nx));
              tc_commit(dp_full);
              if (s + 2 == steps) tc_commit(kv_empty);   // K and V are read by S^T and dP^T alone
            }
          }
          if (!ok) break;
          tc_commit(acc_full);
          ++nu;
        }
        tc_commit(drain);
        wait_teardown(drain, 0, P.wait);
      }
      __syncwarp();
    } else {
      // --------------- per-query numbers of each step, and the look at its rows
      uint32_t n = 0;
      bool ok = true;
      int32_t r = 0;
      const int me = (warp - 2) * 32 + lane;   // 0..63: rows me and me + 64 of the tile
      for (int32_t u = unit_of(0); ok && u < P.num_units; u = unit_of(++r)) {
        const KeyUnit x = key_unit(P, u);
        for (int32_t g = 0; ok && g < P.group; ++g) {
          const int64_t row0 =
              (static_cast<int64_t>(x.shard) * P.hq + x.kvh * P.group + g) * P.T;
          for (int32_t i = x.ia; i < x.ib; ++i, ++n) {
            const uint32_t st = n % NST;
            const bool cut = !tile_span(P.mask, i, P.tiles, P.T, P.causal).whole(x.kb);
            float lse[2], dl[2];
            int2 span[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int32_t q = i * BT + h * 64 + me;
              const bool in = q < P.T;
              lse[h] = in ? -kLog2e * P.LSE[row0 + q] : -INFINITY;   // P = 0 behind the last row
              dl[h] = in ? -P.delta[row0 + q] : 0.0f;
              span[h] = in ? row_span(P.mask, q, P.T, P.causal) : make_int2(0, -1);
            }
            ok = wait_bounded(qd_empty(st), ((n / NST) & 1) ^ 1u, abort_flag, P.wait, kErrWaitEmpty);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t o = (h * 64 + me) * 4;
              sts(vec(st, 0) + o, lse[h]);
              sts(vec(st, 1) + o, dl[h]);
              sts(vec(st, 2) + o, __int_as_float(span[h].x));
              sts(vec(st, 3) + o, __int_as_float(span[h].y));
            }
            if (me == 0) cut_flag[st] = cut;
            if (cut) {
              ok = wait_bounded(qd_full(st), (n / NST) & 1, abort_flag, P.wait, kErrWaitFull);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int row = h * 64 + me;
                const bool b0 = row_not_finite(sQ(st), row), b1 = row_not_finite(sdO(st), row);
                if (b0) zero_row(sQ(st), row);
                if (b1) zero_row(sdO(st), row);
                const uint32_t w = __ballot_sync(0xffffffffu, b0 || b1);
                if (lane == 0) bad[st * 4 + h * 2 + (warp - 2)] = w;
              }
              fence_proxy_async_smem();
            }
            mbar_arrive(vec_full(st));
            __syncwarp();
            if (lane == 0) mbar_arrive(qd_empty(st));
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
    int32_t r = 0;
    for (int32_t u = unit_of(0); ok && u < P.num_units; u = unit_of(++r)) {
      const KeyUnit x = key_unit(P, u);
      if (x.ia >= x.ib) continue;
      const int32_t key = x.kb * BT + quad * 32 + lane;
      for (int32_t g = 0; ok && g < P.group; ++g) {
        float slope2 = 0.0f;
        if (BIAS) slope2 = kLog2e * P.slopes[x.shard * P.hq + x.kvh * P.group + g];
        for (int32_t i = x.ia; i < x.ib; ++i, ++n) {
          const uint32_t st = n % NST;
          ok = wait_bounded(vec_full(st), (n / NST) & 1, abort_flag, P.wait, kErrWaitAttn) &&
               wait_bounded(s_full, n & 1, abort_flag, P.wait, kErrWaitAttn);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const bool cut = cut_flag[st] != 0;
          const uint32_t vl = vec(st, 0) + part * 128, vd = vec(st, 1) + part * 128;
          const uint32_t va = vec(st, 2) + part * 128, vb = vec(st, 3) + part * 128;
          const float dist0 = static_cast<float>(i * BT + part * 32 - key);
          const int side = i * BT >= x.kb * BT + BT - 1 ? 1 : i * BT + BT - 1 <= x.kb * BT ? -1 : 0;
          float w[32];
          uint32_t seen = 0xffffffffu;   // columns that see this key
          if (cut) {
            seen = 0;
            for (int e = 0; e < 32; ++e) {
              const int32_t a = __float_as_int(lds(va + e * 4)), b = __float_as_int(lds(vb + e * 4));
              seen |= static_cast<uint32_t>(key >= a && key < b) << e;
            }
            if (seen & bad[st * 4 + part]) atomicOr(&hit[(nu % 3) * 4 + quad], 1u << lane);
          }
          uint32_t v[32], pk[16];
          auto sees = [&](int e) { return ((seen >> e) & 1u) != 0; };
          tmem_ld_32x32b_x32(tS + off, v);
          tmem_ld_wait();
          prob_chunk<CAP, BIAS>(v, w, pk, P, slope2, dist0, side, cut,
                                [&](int e) { return lds2(vl + e * 4); }, sees);
          tmem_st_32x32b_x16(tS + off, pk);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(p_full);
          ok = wait_bounded(dp_full, n & 1, abort_flag, P.wait, kErrWaitAttn);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          tmem_ld_32x32b_x32(tdP + off, v);
          tmem_ld_wait();
          grad_chunk(v, w, pk, cut, [&](int e) { return lds2(vd + e * 4); }, sees);
          tmem_st_32x32b_x16(tdP + off, pk);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(ds_full);
        }
      }
      if (!ok) break;
      ok = wait_bounded(acc_full, nu & 1, abort_flag, P.wait, kErrWaitAttn);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      // keys of no document stay as they were
      const bool store = key < P.T && row_span(P.mask, key, P.T, P.causal).y >= 0;
      const int64_t row =
          ((static_cast<int64_t>(x.shard) * P.T + key) * P.hkv + x.kvh) * DH + part * 32;
      const uint32_t hits = *const_cast<volatile uint32_t*>(&hit[(nu % 3) * 4 + quad]);
      const float f = (hits >> lane) & 1u ? NAN : 1.0f;
      if (part == 0 && lane == 0) hit[((nu + 2) % 3) * 4 + quad] = 0;
      store_part_row(tdV + off, f, store, P.dV + row);
      store_part_row(tdK + off, f * P.s.scale, store, P.dK + row);
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

// --------------------------------------------------------------------- dQ
struct QueryUnit {
  int32_t shard, head, kvh, qb;
  TileSpan t;
};
__device__ __forceinline__ QueryUnit query_unit(const BwdParams& P, int32_t u) {
  QueryUnit x;
  const int32_t heads = P.p * P.hq, hh = u % heads;
  x.qb = P.tiles - 1 - u / heads;   // causal: the longest first
  x.shard = hh / P.hq;
  x.head = hh % P.hq;
  x.kvh = x.head / P.group;
  x.t = tile_span(P.mask, x.qb, P.tiles, P.T, P.causal);
  return x;
}

template <bool CAP, bool BIAS>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    tc_scored_dq_kernel(const __grid_constant__ CUtensorMap mapQ,
                        const __grid_constant__ CUtensorMap mapK,
                        const __grid_constant__ CUtensorMap mapV,
                        const __grid_constant__ CUtensorMap mapdO,
                        const __grid_constant__ BwdParams P) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t sQ = base, sdO = base + TILE_BYTES;
  auto sK = [&](uint32_t st) { return base + 2 * TILE_BYTES + st * 2 * TILE_BYTES; };
  auto sV = [&](uint32_t st) { return sK(st) + TILE_BYTES; };
  uint8_t* const ctrl = smem_raw + (base - raw) + 2 * TILE_BYTES + NST * 2 * TILE_BYTES;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(ctrl);
  const uint32_t qd_full = smem_u32(&bars[0]), qd_empty = smem_u32(&bars[1]);
  auto kv_full = [&](uint32_t s) { return smem_u32(&bars[2 + s]); };
  auto kv_empty = [&](uint32_t s) { return smem_u32(&bars[4 + s]); };
  auto s_full = [&](uint32_t b) { return smem_u32(&bars[6 + b]); };
  const uint32_t dp_full = smem_u32(&bars[8]), dp_free = smem_u32(&bars[9]);
  const uint32_t ds_full = smem_u32(&bars[10]);
  const uint32_t acc_full = smem_u32(&bars[11]), acc_empty = smem_u32(&bars[12]);
  auto k_seen = [&](uint32_t i) { return smem_u32(&bars[13 + i]); };
  const uint32_t drain = smem_u32(&bars[15]);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 8 * 16);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    mbar_init(qd_full, 1);
    mbar_init(qd_empty, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(kv_full(s), 1);
      mbar_init(kv_empty(s), 3);   // the MMA thread's commit, warps 2 and 3
      mbar_init(s_full(s), 1);
      mbar_init(k_seen(s), 64);
    }
    mbar_init(dp_full, 1);
    mbar_init(dp_free, ARITH);
    mbar_init(ds_full, ARITH);
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

  // 96 registers a thread at launch: 128 x 64 + 512 x 104 <= 640 x 96
  if (warp < 4) {
    regs_shrink<64>();
    if (warp == 0) {
      if (lane == 0) {
        // ---------------------------------------------------------- producer
        uint32_t nu = 0;
        int64_t n = 0;
        bool ok = true;
        int32_t r = 0;
        for (int32_t u = unit_of(0); ok && u < P.num_units; u = unit_of(++r)) {
          const QueryUnit x = query_unit(P, u);
          if (x.t.jb >= x.t.je) continue;
          if (!wait_bounded(qd_empty, (nu & 1) ^ 1u, abort_flag, P.wait, kErrWaitAttn)) break;
          mbar_arrive_expect_tx(qd_full, 2 * TILE_BYTES);
          load_tile(sQ, &mapQ, qd_full, x.head, x.qb * BT, x.shard);
          load_tile(sdO, &mapdO, qd_full, x.head, x.qb * BT, x.shard);
          ++nu;
          for (int32_t j = x.t.jb; j < x.t.je; ++j, ++n) {
            const uint32_t st = n % NST;
            if (!wait_bounded(kv_empty(st), ((n / NST) & 1) ^ 1u, abort_flag, P.wait, kErrWaitEmpty)) {
              ok = false;
              break;
            }
            if (n != P.debug_drop) {
              mbar_arrive_expect_tx(kv_full(st), 2 * TILE_BYTES);
              load_tile(sK(st), &mapK, kv_full(st), x.kvh, j * BT, x.shard);
              load_tile(sV(st), &mapV, kv_full(st), x.kvh, j * BT, x.shard);
            }
          }
        }
        if (nu > 0) wait_teardown(qd_full, (nu - 1) & 1, P.wait);
        for (int64_t q = n > NST ? n - NST : 0; q < n; ++q)
          if (q != P.debug_drop)
            wait_teardown(kv_full(static_cast<uint32_t>(q % NST)),
                          static_cast<uint32_t>((q / NST) & 1), P.wait);
      }
      __syncwarp();
    } else if (warp == 1) {
      if (lane == 0) {
        // -------------------------------------------------------- MMA issuer
        uint32_t n = 0, nu = 0;
        bool ok = true;
        auto wait_kv = [&](uint32_t m) {
          return wait_bounded(kv_full(m % NST), (m / NST) & 1, abort_flag, P.wait, kErrWaitFull);
        };
        auto issue_s = [&](uint32_t m) {
          mma_tiles(tm + (m & 1) * 128, sQ, sK(m % NST));
          tc_commit(s_full(m & 1));
        };
        int32_t r = 0;
        for (int32_t u = unit_of(0); ok && u < P.num_units; u = unit_of(++r)) {
          const QueryUnit x = query_unit(P, u);
          const int32_t steps = x.t.je - x.t.jb;
          if (steps <= 0) continue;
          if (!wait_bounded(qd_full, nu & 1, abort_flag, P.wait, kErrWaitFull) || !wait_kv(n)) break;
          tc_fence_after();
          issue_s(n);
          mma_tiles(tdP, sdO, sV(n % NST));
          tc_commit(dp_full);
          if (steps == 1) {
            tc_commit(qd_empty);
          } else {
            if (!wait_kv(n + 1)) break;
            tc_fence_after();
            issue_s(n + 1);
          }
          for (int32_t s = 0; s < steps; ++s, ++n) {
            if (s + 1 < steps) {
              // the warps have read dP of this step
              if (!wait_bounded(dp_free, n & 1, abort_flag, P.wait, kErrWaitAttn)) {
                ok = false;
                break;
              }
              tc_fence_after();
              mma_tiles(tdP, sdO, sV((n + 1) % NST));
              tc_commit(dp_full);
              if (s + 2 == steps) tc_commit(qd_empty);
            }
            if (!wait_bounded(ds_full, n & 1, abort_flag, P.wait, kErrWaitAttn) ||
                (s == 0 && nu > 0 &&
                 !wait_bounded(acc_empty, (nu - 1) & 1, abort_flag, P.wait, kErrWaitAttn))) {
              ok = false;
              break;
            }
            tc_fence_after();
            mma_rows(tdQ, tm + (n & 1) * 128, sK(n % NST), s > 0);
            tc_commit(kv_empty(n % NST));
            if (s + 2 < steps) {
              if (!wait_kv(n + 2)) {
                ok = false;
                break;
              }
              tc_fence_after();
              issue_s(n + 2);
            }
          }
          if (!ok) break;
          tc_commit(acc_full);
          ++nu;
        }
        tc_commit(drain);
        wait_teardown(drain, 0, P.wait);
      }
      __syncwarp();
    } else {
      // ------------------------------------- keys in blocks that a mask cuts
      uint32_t n = 0, looked = 0;
      bool ok = true;
      int32_t r = 0;
      for (int32_t u = unit_of(0); ok && u < P.num_units; u = unit_of(++r)) {
        const QueryUnit x = query_unit(P, u);
        for (int32_t j = x.t.jb; j < x.t.je; ++j, ++n) {
          const uint32_t st = n % NST;
          ok = wait_bounded(kv_full(st), (n / NST) & 1, abort_flag, P.wait, kErrWaitFull);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (!x.t.whole(j)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int row = h * 64 + (warp - 2) * 32 + lane;
              if (row_not_finite(sK(st), row)) zero_row(sK(st), row);
            }
            fence_proxy_async_smem();
            mbar_arrive(k_seen(looked & 1));
            ++looked;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(kv_empty(st));
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
      const QueryUnit x = query_unit(P, u);
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
        ok = wait_bounded(s_full(b), (n >> 1) & 1, abort_flag, P.wait, kErrWaitAttn);
        if (cut) {
          ok = ok && wait_bounded(k_seen(looked & 1), (looked >> 1) & 1, abort_flag, P.wait, kErrWaitAttn);
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
        auto sees = [&](int e) { return e >= rl && e < rh; };
        tmem_ld_32x32b_x32(tS, v);
        tmem_ld_wait();
        // (P itself is not stored: dQ needs dS alone)
        prob_chunk<CAP, BIAS>(v, w, pk, P, slope2, dist0, side, cut, [&](int) { return nlse; }, sees);
        ok = wait_bounded(dp_full, n & 1, abort_flag, P.wait, kErrWaitAttn);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        tmem_ld_32x32b_x32(tdP + off, v);
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive(dp_free);
        grad_chunk(v, w, pk, cut, [&](int) { return ndl; }, sees);
        tmem_st_32x32b_x16(tS, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(ds_full);
      }
      if (!ok) break;
      ok = wait_bounded(acc_full, nu & 1, abort_flag, P.wait, kErrWaitAttn);
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
  // this grid must not be complete before the one it ran beside
  pdl_wait();
  pdl_launch_dependents();
}

template <bool CAP, bool BIAS>
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
  prm.num_units = prm.p * prm.hkv * prm.tiles;
  cudaError_t e = launch_pdl(tc_scored_dkv_kernel<CAP, BIAS>, grid(prm.num_units), dim3(NUM_THREADS),
                             SMEM_BYTES, c.stream, mQ, mK, mV, mdO, prm);
  note_launch();
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

}  // namespace

tp_status launch_attention_scored_bwd(const LaunchCtx& c, const ScoreCall& a) {
  CUtensorMap mQ, mK, mV, mdO;
  const int64_t wq = static_cast<int64_t>(a.hq) * DH, wk = static_cast<int64_t>(a.hkv) * DH;
  if (!make_map_a(&mQ, a.Q, wq, a.T, a.p) || !make_map_a(&mK, a.K, wk, a.T, a.p) ||
      !make_map_a(&mV, a.V, wk, a.T, a.p) || !make_map_a(&mdO, a.dO, wq, a.T, a.p))
    return TP_ERR_CUDA;
  const int64_t rows = a.T * a.p * a.hq;
  const cudaError_t e =
      launch_pdl(score_delta_kernel, dim3(static_cast<unsigned>((rows + 15) / 16)), dim3(256), 0,
                 c.stream, static_cast<const __nv_bfloat16*>(a.O),
                 static_cast<const __nv_bfloat16*>(a.dO), a.delta, rows, static_cast<int32_t>(a.T),
                 static_cast<int32_t>(a.hq));
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
  prm.dQ = static_cast<__nv_bfloat16*>(a.dQ);
  prm.dK = static_cast<__nv_bfloat16*>(a.dK);
  prm.dV = static_cast<__nv_bfloat16*>(a.dV);
  prm.wait.err = c.err_word;
  prm.wait.timeout_ns = c.timeout_ns;
  prm.debug_drop = c.debug_drop;
  const bool cap = a.cap > 0.0f, bias = a.slopes != nullptr;
  if (cap && bias) return launch_bwd<true, true>(c, prm, a, mQ, mK, mV, mdO);
  if (cap) return launch_bwd<true, false>(c, prm, a, mQ, mK, mV, mdO);
  if (bias) return launch_bwd<false, true>(c, prm, a, mQ, mK, mV, mdO);
  return launch_bwd<false, false>(c, prm, a, mQ, mK, mV, mdO);
}

}  // namespace tpk
