// Scored attention of one new token per sequence over its key/value cache.
//
// Bound by HBM: every cached key and value in sight is read once (512 bytes a
// key and key/value head), 4 * 128 flops a key and query head.  So the work
// is cut by bytes, not by rows: all (sequence, shard, key/value head) items'
// 64-key tiles form one line, which the CTAs share out evenly; a CTA walks its
// stretch without a pause between items.  An item that ends up on several
// CTAs leaves one partial (max, sum, O) each, and decode_join_kernel adds them
// in the order of the CTAs: the same bits on every run.
//
// A group's query heads run together, so the cache is read once for all of
// them: 8 or 16 to an item (more take several items that share their cache
// lines through L2).  Each of the four warps has its own 16 keys of a tile and
// its own three-slot ring, filled by 16-byte asynchronous copies, with its own
// running maximum: no barrier in the loop.  The products are warp-level MMAs
// (m16n8k16; a 128-row tensor-core tile would be nearly empty) of the
// transposed tiles, S^T = K Q^T and O^T = V^T P^T, so that the cache fills the
// MMA's 16 rows and the few heads its 8 columns: half the products and half
// the softmax of the form with padded head rows, which was bound by its
// instructions (735 a warp and tile; 79 us of 8192-token caches against 64 at
// HBM's rate).  Two CTAs an SM keep up to 192 KB in flight.
//
// Keys behind a sequence's length are never read (their copies are zero
// filled) and masked; the appended key and value come from the call's K_new
// and V_new and are written to the cache by the warp that uses them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

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
constexpr int TILE = kDecodeTile;        // keys of a tile, 16 a warp
constexpr int WARPS = 4;
constexpr int NST = 3;                   // ring slots of a warp
constexpr int MROWS = 16;                // most query heads of an item
constexpr int SUM_LD = DH + 4;           // floats between heads of the CTA's joined O
constexpr int WTILE_BYTES = 16 * DH * 2; // a warp's keys (or values) of a tile
constexpr int RING_BYTES = WARPS * NST * 2 * WTILE_BYTES;
constexpr int SMEM_BYTES = RING_BYTES + MROWS * SUM_LD * 4 + 2 * WARPS * MROWS * 4;
constexpr int CTAS_PER_SM = 2;
constexpr int PART_FLOATS = MROWS * (DH + 2);   // O rows, then max and sum of each
constexpr float kLog2e = 1.4426950408889634f;

struct DecodeParams {
  const __nv_bfloat16 *Q, *Kn, *Vn;
  __nv_bfloat16 *Kc, *Vc, *O;
  float *LSE, *part;
  const int32_t* len;
  const float* slopes;
  int32_t B, p, hq, hkv, group, rows, mtiles, heads, ctas;   // rows: heads of an item, 8 or 16;
                                                             // heads: items of a sequence
  int64_t capacity;
  ScoreConsts s;
  unsigned* err;
};

// Keys in sight of sequence b's token, the appended one included; -1: the
// slot is unused, -2: the length does not fit the cache.
__device__ __forceinline__ int32_t keys_of(const DecodeParams& P, int32_t b) {
  const int32_t n = __ldcg(P.len + b);   // (from L2: the join reads it before it waits)
  if (n < 0) return -1;
  const int64_t keys = static_cast<int64_t>(n) + (P.Kn != nullptr ? 1 : 0);
  return keys > P.capacity ? -2 : static_cast<int32_t>(keys);
}
__device__ __forceinline__ int64_t tiles_of(int32_t keys) {
  return keys <= 0 ? 0 : (keys + TILE - 1) / TILE;
}

// First tile of CTA c's share of `total` tiles (both below 2^31 in sum with
// the CTAs' number in almost every call: 32-bit division then).
__device__ __forceinline__ int64_t share_of(int64_t total, int64_t c, int32_t ctas) {
  const uint64_t x = static_cast<uint64_t>(total) * static_cast<uint64_t>(c);
  if (x >> 32) return static_cast<int64_t>(x / static_cast<uint32_t>(ctas));
  return static_cast<uint32_t>(x) / static_cast<uint32_t>(ctas);
}

// Sum of v over the CTA's threads; every thread gets it (and, in *before, the
// sum over the threads of a lower number).
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* before, int64_t* scratch) {
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (threadIdx.x % 32 >= o) x += y;
  }
  __syncthreads();
  if (threadIdx.x % 32 == 31) scratch[threadIdx.x / 32] = x;
  __syncthreads();
  int64_t total = 0, base = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) {
    if (w < static_cast<int>(threadIdx.x) / 32) base += scratch[w];
    total += scratch[w];
  }
  *before = base + x - v;
  return total;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool read) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(read ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8 x 8 tile of bf16 held as fragments, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// 16-byte chunk c of row r of a warp's 16 x 256-byte tile, swizzled so that
// eight rows' chunks of one column lie in different banks.
__device__ __forceinline__ uint32_t chunk_at(uint32_t tile, int r, int c) {
  return tile + r * 256 + ((c ^ (r & 7)) * 16);
}

// Where a CTA stands on the line of tiles.
struct Place {
  int32_t b, h, keys;     // sequence, item of it, its keys
  int64_t tile, tiles;    // tile of the item
};
__device__ __forceinline__ void advance(const DecodeParams& P, Place& x) {
  if (++x.tile < x.tiles) return;
  x.tile = 0;
  if (++x.h < P.heads) return;
  x.h = 0;
  do {
    if (++x.b >= P.B) return;
    x.keys = keys_of(P, x.b);
    x.tiles = tiles_of(x.keys);
  } while (x.tiles == 0);
}

// NT: 8-head column tiles of an item.
template <int CAP, bool BIAS, int NT>
__global__ void __launch_bounds__(WARPS * 32, CTAS_PER_SM)
    decode_kernel(const __grid_constant__ DecodeParams P) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t scratch[WARPS];
  __shared__ Place start;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t ring = smem_u32(smem) + warp * NST * 2 * WTILE_BYTES;
  float* const sum_o = reinterpret_cast<float*>(smem + RING_BYTES);          // [16][128]
  float* const warp_m = sum_o + MROWS * SUM_LD;                              // [warp][16]
  float* const warp_l = warp_m + WARPS * MROWS;
  pdl_wait();
  pdl_launch_dependents();

  // The line's length, then the place of this CTA's first tile on it (one
  // pass over the lengths where there are no more than threads).
  int64_t total = 0, before = 0;
  int32_t keys = 0;
  bool bad = false;
  for (int32_t b0 = 0; b0 < P.B; b0 += WARPS * 32) {
    const int32_t b = b0 + threadIdx.x;
    keys = b < P.B ? keys_of(P, b) : 0;
    bad |= keys == -2;
    total += block_sum(tiles_of(keys) * P.heads, &before, scratch);
  }
  if (bad && blockIdx.x == 0) atomicOr(P.err, kErrLength);
  const int64_t w0 = share_of(total, blockIdx.x, P.ctas), w1 = share_of(total, blockIdx.x + 1, P.ctas);
  if (w0 >= w1) return;
  int64_t done = 0;
  for (int32_t b0 = 0; b0 < P.B && done <= w0; b0 += WARPS * 32) {
    const int32_t b = b0 + threadIdx.x;
    int64_t sum = total;
    if (P.B > WARPS * 32) {
      keys = b < P.B ? keys_of(P, b) : 0;
      sum = block_sum(tiles_of(keys) * P.heads, &before, scratch);
    }
    const int64_t tiles = tiles_of(keys), at = w0 - (done + before);
    if (tiles > 0 && at >= 0 && at < tiles * P.heads) {
      const int32_t h = static_cast<int32_t>(static_cast<uint32_t>(at) / static_cast<uint32_t>(tiles));
      start = Place{b, h, keys, at - h * tiles, tiles};
    }
    done += sum;
  }
  __syncthreads();
  Place use = start, get = start;

  // Copies of one tile of the walk into ring slot st (nothing past w1).
  auto fetch = [&](int64_t w, int st) {
    if (w < w1) {
      const int32_t hk = get.h / P.mtiles;
      const int32_t shard = hk / P.hkv, kvh = hk - shard * P.hkv;
      const int64_t key0 = get.tile * TILE + warp * 16;
      const int64_t pitch = static_cast<int64_t>(P.hkv) * DH;
      const int64_t seq = static_cast<int64_t>(shard) * P.B + get.b;
      const int64_t off = (seq * P.capacity + key0) * pitch + kvh * DH;
      const int64_t off_new = seq * pitch + kvh * DH;
      const int fresh = P.Kn != nullptr ? get.keys - 1 - static_cast<int>(key0) : -1;
      const int left = get.keys - static_cast<int>(key0);
      const uint32_t kt = ring + st * 2 * WTILE_BYTES, vt = kt + WTILE_BYTES;
      const int c = lane % 16, r0 = lane / 16;
      if (left > 16 || (left == 16 && fresh < 0)) {   // cached rows only
        const __nv_bfloat16* k = P.Kc + off + r0 * pitch + c * 8;
        const __nv_bfloat16* v = P.Vc + off + r0 * pitch + c * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          cp_async16(chunk_at(kt, i * 2 + r0, c), k, true);
          cp_async16(chunk_at(vt, i * 2 + r0, c), v, true);
          k += 2 * pitch;
          v += 2 * pitch;
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          const int r = i * 2 + r0;
          const bool own = r == fresh, read = r < left;
          // (an address in range also where nothing is read)
          const int64_t src = own ? off_new : off + r * pitch;
          const __nv_bfloat16* k = read ? (own ? P.Kn : P.Kc) + src + c * 8 : P.Kc;
          const __nv_bfloat16* v = read ? (own ? P.Vn : P.Vc) + src + c * 8 : P.Vc;
          cp_async16(chunk_at(kt, r, c), k, read);
          cp_async16(chunk_at(vt, r, c), v, read);
          if (own && get.h % P.mtiles == 0) {
            const int64_t to = off + r * pitch + c * 8;
            *reinterpret_cast<uint4*>(P.Kc + to) = *reinterpret_cast<const uint4*>(k);
            *reinterpret_cast<uint4*>(P.Vc + to) = *reinterpret_cast<const uint4*>(v);
          }
        }
      }
      advance(P, get);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

#pragma unroll
  for (int st = 0; st < NST - 1; ++st) fetch(w0 + st, st);

  // a thread's heads: columns 2 (lane % 4) and the next one of each 8-head tile
  uint32_t q[NT][8][2];
  float o[NT][8][4], m[NT][2], l[NT][2], slope2[NT][2];
  bool first = true;        // the item at hand began before this CTA
  bool open = false;        // q, o, m, l hold an item
  int slot = 0;
  for (int64_t w = w0; w < w1; ++w) {
    if (!open) {
      const int32_t hk = use.h / P.mtiles, mt = use.h - hk * P.mtiles;
      const int32_t shard = hk / P.hkv, kvh = hk - shard * P.hkv;
      const __nv_bfloat16* Q =
          P.Q + ((static_cast<int64_t>(shard) * P.B + use.b) * P.hq + kvh * P.group) * DH;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int r = mt * P.rows + t * 8 + lane / 4;   // query head of the group
        const uint32_t* a = reinterpret_cast<const uint32_t*>(Q + static_cast<int64_t>(r) * DH) + lane % 4;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          q[t][kk][0] = r < P.group ? a[kk * 8] : 0u;
          q[t][kk][1] = r < P.group ? a[kk * 8 + 4] : 0u;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int rh = mt * P.rows + t * 8 + (lane % 4) * 2 + h;
          if (BIAS)
            slope2[t][h] = rh < P.group ? kLog2e * P.slopes[shard * P.hq + kvh * P.group + rh] : 0.0f;
          m[t][h] = -INFINITY;
          l[t][h] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][i][e] = 0.0f;
      }
      open = true;
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(NST - 2) : "memory");
    __syncwarp();
    fetch(w + NST - 1, slot == 0 ? NST - 1 : slot - 1);   // the slot of the tile before this one
    const uint32_t kt = ring + slot * 2 * WTILE_BYTES, vt = kt + WTILE_BYTES;

    // scores of 16 keys x 8 heads a tile: keys lane / 4 and + 8 of a thread
    float s[NT][4] = {};
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      uint32_t k4[4];
      ldsm4(k4, chunk_at(kt, (lane & 7) + ((lane >> 3) & 1) * 8, kk * 2 + (lane >> 4)));
#pragma unroll
      for (int t = 0; t < NT; ++t) mma16816(s[t], k4, q[t][kk][0], q[t][kk][1]);
    }
    const int32_t key0 = static_cast<int32_t>(use.tile * TILE) + warp * 16 + lane / 4;
    const bool ends = key0 - lane / 4 + 16 > use.keys;   // (same for the warp)
    float mx[NT][2];
    bool grow = false;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float z;
        if (CAP != kNoCap) {
          z = cap_score<CAP == kFineCap>(s[t][e], P.s);
        } else {
          z = s[t][e] * P.s.scale_log2;
        }
        const int32_t key = key0 + (e >> 1) * 8;
        if (BIAS) z = fmaf(slope2[t][e & 1], static_cast<float>(key - (use.keys - 1)), z);
        if (ends && key >= use.keys) z = -INFINITY;
        s[t][e] = z;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = max3_nan(s[t][h], s[t][h + 2], s[t][h]);
#pragma unroll
        for (int d = 4; d < 32; d *= 2) x = max3_nan(x, __shfl_xor_sync(0xffffffffu, x, d), x);
        mx[t][h] = x;
        grow |= !(x <= m[t][h]);
      }
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mn = max3_nan(m[t][h], mx[t][h], mx[t][h]);
          const float alpha = mn == -INFINITY ? 1.0f : ex2(m[t][h] - mn);
          m[t][h] = mn;
          l[t][h] *= alpha;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[t][i][h] *= alpha;
            o[t][i][2 + h] *= alpha;
          }
        }
      }
    }
    uint32_t pb[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float m0 = m[t][0] == -INFINITY ? 0.0f : m[t][0], m1 = m[t][1] == -INFINITY ? 0.0f : m[t][1];
      const float e0 = ex2(s[t][0] - m0), e1 = ex2(s[t][1] - m1);
      const float e2 = ex2(s[t][2] - m0), e3 = ex2(s[t][3] - m1);
      l[t][0] += e0 + e2;
      l[t][1] += e1 + e3;
      pb[t][0] = transpose8x8(pack2(e0, e1));   // [key][head] -> [head][key]
      pb[t][1] = transpose8x8(pack2(e2, e3));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t v4[4];   // 16 elements x 16 keys, transposed on the way
      ldsm4_t(v4, chunk_at(vt, (lane & 7) + (lane >> 4) * 8, i * 2 + ((lane >> 3) & 1)));
#pragma unroll
      for (int t = 0; t < NT; ++t) mma16816(o[t][i], v4, pb[t][0], pb[t][1]);
    }
    __syncwarp();   // every lane is done with the slot
    slot = slot + 1 == NST ? 0 : slot + 1;

    const bool item_ends = use.tile + 1 == use.tiles;
    if (item_ends || w + 1 == w1) {
      // join the warps: heads' maxima and sums, then O warp by warp
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int d = 4; d < 32; d *= 2) l[t][h] += __shfl_xor_sync(0xffffffffu, l[t][h], d);
          if (lane < 4) {
            warp_m[warp * MROWS + t * 8 + lane * 2 + h] = m[t][h];
            warp_l[warp * MROWS + t * 8 + lane * 2 + h] = l[t][h];
          }
        }
      }
      __syncthreads();
      float f[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float M = -INFINITY;
#pragma unroll
          for (int i = 0; i < WARPS; ++i) {
            const float x = warp_m[i * MROWS + t * 8 + (lane % 4) * 2 + h];
            M = max3_nan(M, x, x);
          }
          f[t][h] = m[t][h] == -INFINITY ? 0.0f : ex2(m[t][h] - M);
        }
      }
      for (int i = 0; i < WARPS; ++i) {
        if (warp == i) {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int n = 0; n < 8; ++n) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float* at = sum_o + (t * 8 + (lane % 4) * 2 + (e & 1)) * SUM_LD + n * 16 + lane / 4 + (e >> 1) * 8;
                const float x = o[t][n][e] * f[t][e & 1];
                *at = i > 0 ? *at + x : x;
              }
            }
          }
        }
        __syncthreads();
      }
      const int32_t hk = use.h / P.mtiles, mt = use.h - hk * P.mtiles;
      const int32_t shard = hk / P.hkv, kvh = hk - shard * P.hkv;
      const bool whole = item_ends && !(first && start.tile != 0);
      const int rows = min(P.rows, P.group - mt * P.rows);
      float* const part =
          P.part + (static_cast<int64_t>(blockIdx.x) * 2 + (first ? 0 : 1)) * PART_FLOATS;
      for (int row = warp; row < rows; row += WARPS) {
        float Mr = -INFINITY, L = 0.0f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) {
          const float x = warp_m[i * MROWS + row];
          Mr = max3_nan(Mr, x, x);
        }
#pragma unroll
        for (int i = 0; i < WARPS; ++i) {
          const float x = warp_m[i * MROWS + row];
          if (x != -INFINITY) L += warp_l[i * MROWS + row] * ex2(x - Mr);
        }
        const float4 x = *reinterpret_cast<const float4*>(sum_o + row * SUM_LD + lane * 4);
        if (whole) {
          const int32_t head = kvh * P.group + mt * P.rows + row;
          const float inv = L == 0.0f ? 0.0f : 1.0f / L;
          *reinterpret_cast<uint2*>(
              P.O + ((static_cast<int64_t>(shard) * P.B + use.b) * P.hq + head) * DH + lane * 4) =
              make_uint2(pack2(x.x * inv, x.y * inv), pack2(x.z * inv, x.w * inv));
          if (P.LSE != nullptr && lane == 0)
            P.LSE[(static_cast<int64_t>(shard) * P.hq + head) * P.B + use.b] =
                L == 0.0f ? -INFINITY : 0.6931471805599453f * Mr + logf(L);
        } else {
          *reinterpret_cast<float4*>(part + row * DH + lane * 4) = x;
          if (lane == 0) {
            part[MROWS * DH + row] = Mr;
            part[MROWS * DH + MROWS + row] = L;
          }
        }
      }
      __syncthreads();   // sum_o and the rows' numbers are free again
      open = false;
      first = false;
    }
    advance(P, use);
  }
}

// Adds the partials of an item that lay on several CTAs, in their order, and
// writes zeros for sequences without keys.  One CTA a (item, query head); eight
// groups of lanes share the parts, then add up in order.
constexpr int JOIN_THREADS = 256;
__global__ void __launch_bounds__(JOIN_THREADS) decode_join_kernel(const __grid_constant__ DecodeParams P) {
  __shared__ int64_t scratch[JOIN_THREADS / 32];
  __shared__ float grp_m[8];
  __shared__ float grp_l[8];
  __shared__ __align__(16) float grp_o[8][DH];
  const int32_t item = blockIdx.x;
  const int32_t b = item / P.heads, h = item - b * P.heads;
  const int32_t hk = h / P.mtiles, mt = h - hk * P.mtiles;
  const int32_t shard = hk / P.hkv, kvh = hk - shard * P.hkv;
  const int32_t in_group = mt * P.rows + blockIdx.y;
  if (in_group >= P.group) return;
  // The lengths were complete before the decode kernel, which this one waits
  // for, let it start: where the parts lie is worked out beside it.
  const int32_t keys = keys_of(P, b);
  const int32_t head = kvh * P.group + in_group, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  __nv_bfloat16* const out = P.O + ((static_cast<int64_t>(shard) * P.B + b) * P.hq + head) * DH;
  float* const lse =
      P.LSE != nullptr ? P.LSE + (static_cast<int64_t>(shard) * P.hq + head) * P.B + b : nullptr;
  int64_t total = 0, ahead = 0, before;
  for (int32_t b0 = 0; b0 < P.B; b0 += JOIN_THREADS) {
    const int32_t i = b0 + threadIdx.x;
    const int64_t t = i < P.B ? tiles_of(keys_of(P, i)) * P.heads : 0;
    total += block_sum(t, &before, scratch);
    ahead += block_sum(i < b ? t : 0, &before, scratch);
  }
  const int64_t tiles = tiles_of(keys), a = ahead + h * tiles, z = a + tiles - 1;
  // the CTA of tile w: the last c with total * c / ctas <= w
  auto cta_of = [&](int64_t w) {
    const uint64_t x = static_cast<uint64_t>(w + 1) * P.ctas - 1;
    if ((x | static_cast<uint64_t>(total)) >> 32) return static_cast<int64_t>(x / total);
    return static_cast<int64_t>(static_cast<uint32_t>(x) / static_cast<uint32_t>(total));
  };
  const int64_t c0 = keys > 0 ? cta_of(a) : 0, c1 = keys > 0 ? cta_of(z) : 0;
  pdl_wait();
  pdl_launch_dependents();
  if (keys < 0) return;
  if (keys == 0) {
    if (warp == 0) *reinterpret_cast<uint2*>(out + lane * 4) = make_uint2(0, 0);
    if (threadIdx.x == 0 && lse != nullptr) *lse = -INFINITY;
    return;
  }
  if (c0 == c1) return;   // written whole
  float m = -INFINITY, l = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  constexpr int GROUPS = JOIN_THREADS / 32, AHEAD = 4;   // parts of a warp loaded together
  for (int64_t cb = c0 + warp; cb <= c1; cb += GROUPS * AHEAD) {
    float pm[AHEAD], pl[AHEAD];
    float4 x[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int64_t c = cb + i * GROUPS;
      pm[i] = -INFINITY;
      pl[i] = 0.0f;
      x[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      const int64_t first = share_of(total, c, P.ctas);
      // (a CTA without a tile, where there are fewer tiles than CTAs, left none)
      if (c <= c1 && first < share_of(total, c + 1, P.ctas)) {
        // a CTA's first item is its slot 0; the item begins inside c0 unless it
        // begins with it
        const bool second = c == c0 && first != a;
        const float* part = P.part + (c * 2 + (second ? 1 : 0)) * PART_FLOATS;
        pm[i] = part[MROWS * DH + blockIdx.y];
        pl[i] = part[MROWS * DH + MROWS + blockIdx.y];
        x[i] = *reinterpret_cast<const float4*>(part + blockIdx.y * DH + lane * 4);
      }
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const float mn = max3_nan(m, pm[i], pm[i]);
      const float fa = m == -INFINITY ? 0.0f : ex2(m - mn);
      const float fb = pm[i] == -INFINITY ? 0.0f : ex2(pm[i] - mn);
      l = l * fa + pl[i] * fb;
      o.x = o.x * fa + x[i].x * fb;
      o.y = o.y * fa + x[i].y * fb;
      o.z = o.z * fa + x[i].z * fb;
      o.w = o.w * fa + x[i].w * fb;
      m = mn;
    }
  }
  if (lane == 0) {
    grp_m[warp] = m;
    grp_l[warp] = l;
  }
  *reinterpret_cast<float4*>(&grp_o[warp][lane * 4]) = o;
  __syncthreads();
  if (threadIdx.x < DH) {
    float M = -INFINITY, L = 0.0f, v = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) M = max3_nan(M, grp_m[i], grp_m[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = grp_m[i] == -INFINITY ? 0.0f : ex2(grp_m[i] - M);
      L += grp_l[i] * f;
      v += grp_o[i][threadIdx.x] * f;
    }
    out[threadIdx.x] = __float2bfloat16_rn(L == 0.0f ? 0.0f : v / L);
    if (threadIdx.x == 0 && lse != nullptr)
      *lse = L == 0.0f ? -INFINITY : 0.6931471805599453f * M + logf(L);
  }
}

template <int CAP, bool BIAS, int NT>
tp_status launch_decode(const LaunchCtx& c, const DecodeParams& prm) {
  static uint64_t attr_epoch[64] = {};
  static std::mutex mu;
  {
    std::lock_guard<std::mutex> lk(mu);
    const int dev = c.device & 63;
    if (attr_epoch[dev] != c.epoch) {
      if (cudaFuncSetAttribute(decode_kernel<CAP, BIAS, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               SMEM_BYTES) != cudaSuccess) {
        set_error_detail("cudaFuncSetAttribute failed: %s", cudaGetErrorString(cudaGetLastError()));
        return TP_ERR_CUDA;
      }
      attr_epoch[dev] = c.epoch;
    }
  }
  cudaError_t e = launch_pdl(decode_kernel<CAP, BIAS, NT>, dim3(prm.ctas), dim3(WARPS * 32), SMEM_BYTES,
                             c.stream, prm);
  note_launch();
  if (e == cudaSuccess) {
    e = launch_pdl(decode_join_kernel, dim3(prm.B * prm.heads, prm.group < prm.rows ? prm.group : prm.rows),
                   dim3(JOIN_THREADS), 0, c.stream, prm);
    note_launch();
  }
  if (e != cudaSuccess) {
    set_error_detail("decode launch failed: %s", cudaGetErrorString(e));
    return TP_ERR_CUDA;
  }
  return TP_OK;
}

template <int CAP, int NT>
tp_status launch_form(const LaunchCtx& c, const DecodeParams& prm) {
  if (prm.slopes != nullptr) return launch_decode<CAP, true, NT>(c, prm);
  return launch_decode<CAP, false, NT>(c, prm);
}

}  // namespace

// CTAs that share the line of tiles: two an SM, fewer where the caches could
// not give each a tile.
int64_t decode_ctas(int num_sms, int64_t B, int64_t capacity, int p, int hq, int hkv) {
  const int64_t most = B * p * decode_items(hq, hkv) * ((capacity + TILE - 1) / TILE);
  int64_t full = static_cast<int64_t>(num_sms) * CTAS_PER_SM;
  if (full > kMaxDecodeCtas) full = kMaxDecodeCtas;
  return most < full ? most : full;
}
size_t decode_part_bytes(int64_t ctas) {
  return static_cast<size_t>(ctas) * 2 * PART_FLOATS * sizeof(float);
}

tp_status launch_attention_decode(const LaunchCtx& c, const DecodeCall& a) {
  DecodeParams prm{};
  prm.Q = static_cast<const __nv_bfloat16*>(a.Q);
  prm.Kn = static_cast<const __nv_bfloat16*>(a.Kn);
  prm.Vn = static_cast<const __nv_bfloat16*>(a.Vn);
  prm.Kc = static_cast<__nv_bfloat16*>(a.Kc);
  prm.Vc = static_cast<__nv_bfloat16*>(a.Vc);
  prm.O = static_cast<__nv_bfloat16*>(a.O);
  prm.LSE = a.LSE;
  prm.part = a.part;
  prm.len = a.len;
  prm.slopes = a.slopes;
  prm.B = static_cast<int32_t>(a.B);
  prm.p = a.p;
  prm.hq = a.hq;
  prm.hkv = a.hkv;
  prm.group = a.hq / a.hkv;
  prm.rows = decode_rows(prm.group);
  prm.mtiles = (prm.group + prm.rows - 1) / prm.rows;
  prm.heads = static_cast<int32_t>(a.p * decode_items(a.hq, a.hkv));
  prm.capacity = a.capacity;
  prm.s = score_consts(a.scale, a.cap);
  prm.err = c.err_word;
  prm.ctas = static_cast<int32_t>(decode_ctas(c.num_sms, a.B, a.capacity, a.p, a.hq, a.hkv));
  const int cap = cap_form(prm.s);
  if (prm.rows == 8) {
    if (cap == kFineCap) return launch_form<kFineCap, 1>(c, prm);
    if (cap == kCoarseCap) return launch_form<kCoarseCap, 1>(c, prm);
    return launch_form<kNoCap, 1>(c, prm);
  }
  if (cap == kFineCap) return launch_form<kFineCap, 2>(c, prm);
  if (cap == kCoarseCap) return launch_form<kCoarseCap, 2>(c, prm);
  return launch_form<kNoCap, 2>(c, prm);
}

}  // namespace tpk
