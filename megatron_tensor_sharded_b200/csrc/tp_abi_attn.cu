// C ABI of the attention-side operators (declared in include/tp_mlp.h):
// rotary positions, head norms and scored attention.  Argument checks and
// dispatch; no device memory is allocated here.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "tp_internal.h"
#include "tp_launch.cuh"
#include "tp_score.h"
#include "tp_mlp.h"

namespace tpk {
namespace {

#define TP_FAIL(status, ...)        \
  do {                              \
    set_error_detail(__VA_ARGS__);  \
    return status;                  \
  } while (0)
#define TP_TRY(expr)               \
  do {                             \
    const tp_status st_ = (expr);  \
    if (st_ != TP_OK) return st_;  \
  } while (0)

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

tp_status cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return TP_OK;
  TP_FAIL(TP_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// A buffer of the call: `self` names the input (and no other that happens to
// lie there) that an output may share its whole buffer with.
struct Buf {
  const char* name;
  const void* ptr;
  size_t bytes;
  const char* self;
};

bool overlap(const Buf& a, const Buf& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.ptr), y = reinterpret_cast<uintptr_t>(b.ptr);
  return a.ptr != nullptr && b.ptr != nullptr && x < y + b.bytes && y < x + a.bytes;
}

tp_status check_overlaps(std::initializer_list<Buf> outs, std::initializer_list<Buf> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (const Buf& i : ins)
      if (overlap(*o, i) && !(o->ptr == i.ptr && o->self != nullptr && std::strcmp(o->self, i.name) == 0))
        TP_FAIL(TP_ERR_INVALID_ARG, "%s overlaps %s", o->name, i.name);
    for (auto q = o + 1; q != outs.end(); ++q)
      if (overlap(*o, *q)) TP_FAIL(TP_ERR_INVALID_ARG, "%s overlaps %s", o->name, q->name);
  }
  return TP_OK;
}

tp_status check_workspace(const void* ws, size_t have, size_t need) {
  if (ws == nullptr || have < need)
    TP_FAIL(TP_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need,
            ws == nullptr ? size_t(0) : have);
  if (!aligned(ws, 256)) TP_FAIL(TP_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  return TP_OK;
}

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

// Shards, heads and head size of a call; a head count is checked only where
// its tensor is there.
tp_status check_layout(int64_t T, int p, int n_heads, int n_kv_heads, int head_dim, bool q, bool k) {
  if (p < 1) TP_FAIL(TP_ERR_INVALID_ARG, "p = %d, must be >= 1", p);
  if (T < 0) TP_FAIL(TP_ERR_INVALID_ARG, "T = %lld", (long long)T);
  if ((q && n_heads < 1) || (k && n_kv_heads < 1) || head_dim < 1)
    TP_FAIL(TP_ERR_INVALID_ARG, "heads %d / %d, head_dim %d", n_heads, n_kv_heads, head_dim);
  if ((q && n_heads % p != 0) || (k && n_kv_heads % p != 0))
    TP_FAIL(TP_ERR_INDIVISIBLE,
            "number of attention heads (%d) and key/value heads (%d) must be divisible by "
            "tensor_parallel_size (%d)",
            n_heads, n_kv_heads, p);
  const int64_t heads = (q ? static_cast<int64_t>(n_heads) : 0) + (k ? n_kv_heads : 0);
  if (T > INT32_MAX || heads > (1 << 20) || T * heads > (int64_t(1) << 40))
    TP_FAIL(TP_ERR_UNSUPPORTED, "sizes too large (T = %lld, %lld heads)", (long long)T,
            (long long)heads);
  return TP_OK;
}

tp_status check_rope(const RopeCall& a, int n_heads, int n_kv_heads, bool backward) {
  if (a.dtype != TP_F32 && a.dtype != TP_BF16) TP_FAIL(TP_ERR_INVALID_ARG, "dtype %d", a.dtype);
  const bool q = a.Q != nullptr, k = a.K != nullptr;
  if (q != (a.Qo != nullptr) || k != (a.Ko != nullptr) ||
      (backward && (q != (a.dYq != nullptr) || k != (a.dYk != nullptr))))
    TP_FAIL(TP_ERR_INVALID_ARG, "the buffers of Q (and those of K) are given together or not at all");
  if (!q && !k && a.T > 0) TP_FAIL(TP_ERR_INVALID_ARG, "neither Q nor K is given");
  TP_TRY(check_layout(a.T, a.p, n_heads, n_kv_heads, a.dh, q, k));
  if (a.dh < 2 || a.dh > 256)
    TP_FAIL(TP_ERR_UNSUPPORTED, "head_dim %d (2 to 256 are provided)", a.dh);
  if (a.plan != nullptr) {
    const tp_rope_plan& pl = *a.plan;
    if (pl.rotary_dim < 2 || pl.rotary_dim % 2 != 0 || pl.rotary_dim > a.dh)
      TP_FAIL(TP_ERR_INVALID_ARG, "rotary_dim %d of head_dim %d", pl.rotary_dim, a.dh);
    if (pl.layout != TP_ROPE_HALF && pl.layout != TP_ROPE_INTERLEAVED)
      TP_FAIL(TP_ERR_INVALID_ARG, "layout %d", pl.layout);
  }
  const uintptr_t es = a.dtype == TP_BF16 ? 2 : 4;
  for (const void* b : {a.Q, a.K, static_cast<const void*>(a.Qo), static_cast<const void*>(a.Ko),
                        a.dYq, a.dYk})
    if (!aligned(b, es)) TP_FAIL(TP_ERR_ALIGNMENT, "buffers must be aligned to their element");
  for (const void* b : {static_cast<const void*>(a.wq), static_cast<const void*>(a.wk),
                        static_cast<const void*>(a.pos), static_cast<const void*>(a.dwq),
                        static_cast<const void*>(a.dwk)})
    if (!aligned(b, 4))
      TP_FAIL(TP_ERR_ALIGNMENT, "weights and positions must be 4-byte aligned");
  return TP_OK;
}

tp_status rope_impl(RopeCall a, int n_heads, int n_kv_heads, void* stream) {
  TP_TRY(check_rope(a, n_heads, n_kv_heads, false));
  if (a.norm && !(a.eps > 0.0f)) TP_FAIL(TP_ERR_INVALID_ARG, "eps must be > 0");
  if (a.T == 0) return TP_OK;
  a.hq = a.Q != nullptr ? n_heads / a.p : 0;
  a.hk = a.K != nullptr ? n_kv_heads / a.p : 0;
  const size_t es = a.dtype == TP_BF16 ? 2 : 4, row = static_cast<size_t>(a.T) * a.dh * a.p * es;
  const size_t w = static_cast<size_t>(a.dh) * 4;
  TP_TRY(check_overlaps({{"Q_out", a.Qo, row * a.hq, "Q"}, {"K_out", a.Ko, row * a.hk, "K"}},
                        {{"Q", a.Q, row * a.hq, nullptr},
                         {"K", a.K, row * a.hk, nullptr},
                         {"wq", a.wq, w, nullptr},
                         {"wk", a.wk, w, nullptr},
                         {"positions", a.pos, static_cast<size_t>(a.T) * 4, nullptr}}));
  LaunchCtx c{};
  TP_TRY(make_launch_ctx(stream, false, &c));
  return cuda_status(launch_rope(c, a), "rotary launch");
}

size_t norm_rope_ws(int64_t T, int dh) {
  return align256(static_cast<size_t>(norm_rope_bwd_ctas(T)) * 2 * dh * 4);
}

// Heads and options of a scored-attention call into `a`.
tp_status score_call(ScoreCall* a, int64_t T, int p, int n_heads, int n_kv_heads, int head_dim,
                     const tp_score_params* s) {
  TP_TRY(check_layout(T, p, n_heads, n_kv_heads, head_dim, true, true));
  if (n_heads % n_kv_heads != 0)
    TP_FAIL(TP_ERR_INVALID_ARG, "n_heads (%d) must be a multiple of n_kv_heads (%d)", n_heads,
            n_kv_heads);
  if (head_dim != 128) TP_FAIL(TP_ERR_UNSUPPORTED, "head_dim %d (128 is provided)", head_dim);
  // unit counts and TMA coordinates stay in int32
  if (T > (int64_t(1) << 30) ||
      static_cast<int64_t>(n_heads) * (T / kAttnTile + 2) > (int64_t(1) << 30))
    TP_FAIL(TP_ERR_UNSUPPORTED, "sizes too large (T = %lld, %d heads)", (long long)T, n_heads);
  a->T = T;
  a->p = p;
  a->hq = n_heads / p;
  a->hkv = n_kv_heads / p;
  a->scale = 1.0f / std::sqrt(static_cast<float>(head_dim));
  if (s == nullptr) return TP_OK;
  if (s->scale != 0.0f) {
    if (!(s->scale > 0.0f) || !std::isfinite(s->scale))
      TP_FAIL(TP_ERR_INVALID_ARG, "scale must be > 0 (or 0 for 1/sqrt(head_dim))");
    a->scale = s->scale;
  }
  if (!std::isfinite(score_consts(a->scale, 0.0f).scale_log2))
    TP_FAIL(TP_ERR_UNSUPPORTED, "scale %g (up to 2.3e38 is provided)", a->scale);
  if (!(s->softcap >= 0.0f) || !std::isfinite(s->softcap))
    TP_FAIL(TP_ERR_INVALID_ARG, "softcap must be >= 0");
  if (s->softcap > 0.0f && (s->softcap < 1e-3f || s->softcap > 1e6f ||
                            a->scale / s->softcap < 1e-9f || a->scale / s->softcap > 1e6f))
    TP_FAIL(TP_ERR_UNSUPPORTED, "softcap 1e-3 to 1e6 and scale/softcap 1e-9 to 1e6 are provided");
  if (!aligned(s->slopes, 4)) TP_FAIL(TP_ERR_ALIGNMENT, "slopes must be 4-byte aligned");
  if (!aligned(s->mask, 256)) TP_FAIL(TP_ERR_ALIGNMENT, "mask must be 256-byte aligned");
  a->cap = s->softcap;
  a->slopes = s->slopes;
  a->mask = s->mask;
  a->causal = s->causal != 0;
  return TP_OK;
}

// Backward workspace: D, a number a query row and head, a byte a key row and
// head, then the partial dK and dV.  (The mask and the causal option do not
// change its size.)
size_t score_delta_ws(const ScoreCall& a) { return align256(static_cast<size_t>(a.T) * a.p * a.hq * 4); }
size_t score_bad_ws(const ScoreCall& a) { return align256(static_cast<size_t>(a.T) * a.p * a.hkv); }
size_t score_bwd_ws(ScoreCall a) {
  a.causal = false;
  return score_delta_ws(a) + score_bad_ws(a) + align256(score_dkv_bytes(a));
}

// Heads and options of a backward call into `a`: a CTA counts the steps of dK
// and dV that are its share in 32 bits.
tp_status score_bwd_call(ScoreCall* a, int64_t T, int p, int n_heads, int n_kv_heads, int head_dim,
                         const tp_score_params* s) {
  TP_TRY(score_call(a, T, p, n_heads, n_kv_heads, head_dim, s));
  const double tiles = static_cast<double>(ceil_div(T, kAttnTile));
  const double seen = a->causal && a->mask == nullptr ? (tiles + 1) / 2 : tiles;
  if (n_heads * tiles * (seen + kUnitCost) / kScoreDkvCtas >= 0x1p31)
    TP_FAIL(TP_ERR_UNSUPPORTED, "sizes too large (T = %lld, %d heads)", (long long)T, n_heads);
  return TP_OK;
}

// Sizes and options of a decode call into `a` (its T is the batch).
tp_status decode_sizes(ScoreCall* a, int64_t B, int64_t capacity, int p, int n_heads,
                       int n_kv_heads, int head_dim, const tp_score_params* s) {
  TP_TRY(score_call(a, B, p, n_heads, n_kv_heads, head_dim, s));
  if (a->mask != nullptr)
    TP_FAIL(TP_ERR_UNSUPPORTED, "a single token's call takes lengths, not a mask");
  if (capacity < 1) TP_FAIL(TP_ERR_INVALID_ARG, "capacity = %lld", (long long)capacity);
  if (capacity > (int64_t(1) << 30) || B > (1 << 20) || B * n_heads > (int64_t(1) << 30) ||
      B * n_kv_heads * capacity > (int64_t(1) << 44))
    TP_FAIL(TP_ERR_UNSUPPORTED, "sizes too large (B = %lld, capacity = %lld)", (long long)B,
            (long long)capacity);
  // a CTA finds its place among all sequences' tiles of a head in 32 bits
  const int64_t tiles = capacity / kDecodeTile + 1;
  if (tiles * a->p * decode_items(a->hq, a->hkv) > (int64_t(1) << 31))
    TP_FAIL(TP_ERR_UNSUPPORTED, "sizes too large (%d / %d heads, capacity = %lld)", n_heads, n_kv_heads,
            (long long)capacity);
  return TP_OK;
}
size_t decode_ws(const ScoreCall& a, int64_t B, int64_t capacity) {
  // (for any number of SMs: the caller may ask on a machine without a GPU)
  return align256(decode_part_bytes(decode_ctas(kMaxDecodeCtas, B, capacity, a.p, a.hq, a.hkv)));
}

tp_status check_bf16(const void* p, const char* name) {
  if (p == nullptr) TP_FAIL(TP_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(p, 16)) TP_FAIL(TP_ERR_ALIGNMENT, "%s must be 16-byte aligned", name);
  return TP_OK;
}

}  // namespace
}  // namespace tpk

using namespace tpk;

extern "C" {

tp_status tp_rope_plan_init(const tp_rope_config* cfg, tp_rope_plan* plan) {
  set_error_detail("%s", "");
  if (cfg == nullptr || plan == nullptr) TP_FAIL(TP_ERR_INVALID_ARG, "config or plan is NULL");
  const int r = cfg->rotary_dim;
  if (r < 2 || r % 2 != 0 || r > 2 * TP_ROPE_MAX_PAIRS)
    TP_FAIL(TP_ERR_INVALID_ARG, "rotary_dim %d (even, 2 to %d)", r, 2 * TP_ROPE_MAX_PAIRS);
  if (cfg->layout != TP_ROPE_HALF && cfg->layout != TP_ROPE_INTERLEAVED)
    TP_FAIL(TP_ERR_INVALID_ARG, "layout %d", cfg->layout);
  if (cfg->scaling < TP_ROPE_SCALE_NONE || cfg->scaling > TP_ROPE_SCALE_RAMP)
    TP_FAIL(TP_ERR_INVALID_ARG, "scaling %d", cfg->scaling);
  if (!(cfg->base > 1.0) || !std::isfinite(cfg->base))
    TP_FAIL(TP_ERR_INVALID_ARG, "base must be > 1");
  const int scaling = cfg->scaling;
  const double f = scaling == TP_ROPE_SCALE_NONE ? 1.0 : cfg->factor;
  if (!(f >= 1.0) || !std::isfinite(f)) TP_FAIL(TP_ERR_INVALID_ARG, "factor must be >= 1");
  const bool bands = scaling == TP_ROPE_SCALE_BANDS, ramp = scaling == TP_ROPE_SCALE_RAMP;
  if ((bands || ramp) && (!(cfg->original_len > 0.0) || !std::isfinite(cfg->original_len) ||
                          !(cfg->low > 0.0) || !(cfg->high > cfg->low) || !std::isfinite(cfg->high)))
    TP_FAIL(TP_ERR_INVALID_ARG, "this scaling needs original_len > 0 and 0 < low < high");
  if (!(cfg->amplitude >= 0.0) || !std::isfinite(cfg->amplitude))
    TP_FAIL(TP_ERR_INVALID_ARG, "amplitude must be >= 0");
  // In long double: at 2^31 the angle then is off by less than 2^-30 turns.
  using real = long double;
  const real two_pi = 6.283185307179586476925286766559L, len = cfg->original_len;
  real base = cfg->base, lo = 0, span = 1;
  if (scaling == TP_ROPE_SCALE_BASE && r > 2) base *= std::pow(real(f), r / (r - real(2)));
  if (ramp) {
    // pair index at which a frequency turns n times in original_len
    auto at = [&](real n) { return r * std::log(len / (two_pi * n)) / (2 * std::log(base)); };
    lo = std::max(std::floor(at(cfg->high)), real(0));
    span = std::min(std::ceil(at(cfg->low)), real(r - 1)) - lo;
    if (!(span > 0)) span = 0.001L;   // a step
  }
  *plan = tp_rope_plan{};
  plan->rotary_dim = r;
  plan->layout = cfg->layout;
  plan->amplitude = static_cast<float>(
      cfg->amplitude > 0.0 ? cfg->amplitude : ramp ? 0.1 * std::log(f) + 1.0 : 1.0);
  for (int i = 0; i < r / 2; ++i) {
    real w = std::pow(base, real(-2) * i / r);
    if (scaling == TP_ROPE_SCALE_LINEAR) {
      w /= f;
    } else if (bands) {
      const real n = len * w / two_pi;
      const real s = std::min(real(1), std::max(real(0), (n - cfg->low) / (cfg->high - cfg->low)));
      w = w * s + w / f * (1 - s);
    } else if (ramp) {
      const real g = std::min(real(1), std::max(real(0), (i - lo) / span));
      w = w * (1 - g) + w / f * g;
    }
    // to the nearest (w <= 1: below 2^62)
    plan->turn[i] = static_cast<uint64_t>(std::floor(std::ldexp(w / two_pi, 64) + real(0.5)));
  }
  return TP_OK;
}

tp_status tp_rope(const void* Q, const void* K, const int32_t* positions, void* Q_out, void* K_out,
                  int64_t T, int p, int n_heads, int n_kv_heads, int head_dim,
                  const tp_rope_plan* plan, tp_dtype dtype, int inverse, void* stream) {
  set_error_detail("%s", "");
  if (plan == nullptr) TP_FAIL(TP_ERR_INVALID_ARG, "plan is NULL");
  RopeCall a{};
  a.Q = Q;
  a.K = K;
  a.Qo = Q_out;
  a.Ko = K_out;
  a.pos = positions;
  a.plan = plan;
  a.T = T;
  a.p = p;
  a.dh = head_dim;
  a.dtype = dtype;
  a.back = inverse != 0;
  return rope_impl(a, n_heads, n_kv_heads, stream);
}

tp_status tp_qk_norm_rope(const void* Q, const void* K, const float* wq, const float* wk,
                          const int32_t* positions, void* Q_out, void* K_out, int64_t T, int p,
                          int n_heads, int n_kv_heads, int head_dim, const tp_rope_plan* plan,
                          float eps, tp_dtype dtype, void* stream) {
  set_error_detail("%s", "");
  RopeCall a{};
  a.Q = Q;
  a.K = K;
  a.Qo = Q_out;
  a.Ko = K_out;
  a.wq = wq;
  a.wk = wk;
  a.pos = positions;
  a.plan = plan;
  a.T = T;
  a.p = p;
  a.dh = head_dim;
  a.dtype = dtype;
  a.norm = true;
  a.eps = eps;
  return rope_impl(a, n_heads, n_kv_heads, stream);
}

size_t tp_qk_norm_rope_backward_workspace_size(int64_t T, int p, int n_heads, int n_kv_heads,
                                               int head_dim) {
  if (check_layout(T, p, n_heads, n_kv_heads, head_dim, n_heads > 0, n_kv_heads > 0) != TP_OK ||
      head_dim > 256 || head_dim < 2)
    return 0;
  return norm_rope_ws(T, head_dim);
}

tp_status tp_qk_norm_rope_backward(const void* Q, const void* K, const float* wq, const float* wk,
                                   const int32_t* positions, const void* dQ_out,
                                   const void* dK_out, void* dQ, void* dK, float* dwq, float* dwk,
                                   void* workspace, size_t workspace_bytes, int64_t T, int p,
                                   int n_heads, int n_kv_heads, int head_dim,
                                   const tp_rope_plan* plan, float eps, tp_dtype dtype,
                                   void* stream) {
  set_error_detail("%s", "");
  RopeCall a{};
  a.Q = Q;
  a.K = K;
  a.dYq = dQ_out;
  a.dYk = dK_out;
  a.Qo = dQ;
  a.Ko = dK;
  a.wq = wq;
  a.wk = wk;
  a.dwq = dwq;
  a.dwk = dwk;
  a.pos = positions;
  a.plan = plan;
  a.T = T;
  a.p = p;
  a.dh = head_dim;
  a.dtype = dtype;
  a.norm = a.back = true;
  a.eps = eps;
  TP_TRY(check_rope(a, n_heads, n_kv_heads, true));
  if (!(eps > 0.0f)) TP_FAIL(TP_ERR_INVALID_ARG, "eps must be > 0");
  a.hq = Q != nullptr ? n_heads / p : 0;
  a.hk = K != nullptr ? n_kv_heads / p : 0;
  const size_t es = dtype == TP_BF16 ? 2 : 4, row = static_cast<size_t>(T) * head_dim * p * es;
  const size_t w = static_cast<size_t>(head_dim) * 4, need = norm_rope_ws(T, head_dim);
  if (T == 0) {
    for (float* d : {dwq, dwk}) {
      if (d == nullptr) continue;
      TP_TRY(cuda_status(cudaMemsetAsync(d, 0, w, static_cast<cudaStream_t>(stream)), "dw"));
    }
    return TP_OK;
  }
  TP_TRY(check_workspace(workspace, workspace_bytes, need));
  TP_TRY(check_overlaps({{"dQ", dQ, row * a.hq, "dQ_out"},
                         {"dK", dK, row * a.hk, "dK_out"},
                         {"dwq", dwq, w, nullptr},
                         {"dwk", dwk, w, nullptr},
                         {"workspace", workspace, need, nullptr}},
                        {{"Q", Q, row * a.hq, nullptr},
                         {"K", K, row * a.hk, nullptr},
                         {"dQ_out", dQ_out, row * a.hq, nullptr},
                         {"dK_out", dK_out, row * a.hk, nullptr},
                         {"wq", wq, w, nullptr},
                         {"wk", wk, w, nullptr},
                         {"positions", positions, static_cast<size_t>(T) * 4, nullptr}}));
  a.partial = static_cast<float*>(workspace);
  LaunchCtx c{};
  TP_TRY(make_launch_ctx(stream, false, &c));
  return cuda_status(launch_norm_rope_bwd(c, a), "head norm backward launch");
}

size_t tp_attention_mask_size(int64_t T) {
  return T < 0 || T > (int64_t(1) << 30) ? 0 : T == 0 ? 256 : mask_bytes(T);
}

tp_status tp_attention_mask(const int32_t* doc_offsets, int n_docs, const int32_t* prefix,
                            int causal, void* mask, size_t mask_size, int64_t T, void* stream) {
  set_error_detail("%s", "");
  if (T < 0) TP_FAIL(TP_ERR_INVALID_ARG, "T = %lld", (long long)T);
  if (T > (int64_t(1) << 30)) TP_FAIL(TP_ERR_UNSUPPORTED, "T = %lld", (long long)T);
  if (n_docs < 1 || n_docs > (1 << 30)) TP_FAIL(TP_ERR_INVALID_ARG, "n_docs = %d", n_docs);
  if (prefix != nullptr && !causal)
    TP_FAIL(TP_ERR_INVALID_ARG, "a prefix needs causal: without it every token of a document is seen");
  if (T == 0) return TP_OK;
  if (doc_offsets == nullptr) TP_FAIL(TP_ERR_INVALID_ARG, "doc_offsets is NULL");
  if (!aligned(doc_offsets, 4) || !aligned(prefix, 4))
    TP_FAIL(TP_ERR_ALIGNMENT, "doc_offsets and prefix must be 4-byte aligned");
  if (mask == nullptr || mask_size < mask_bytes(T))
    TP_FAIL(TP_ERR_WORKSPACE, "the mask plan needs %zu bytes, got %zu", mask_bytes(T),
            mask == nullptr ? size_t(0) : mask_size);
  if (!aligned(mask, 256)) TP_FAIL(TP_ERR_ALIGNMENT, "mask must be 256-byte aligned");
  const size_t n = static_cast<size_t>(n_docs) * 4;
  TP_TRY(check_overlaps({{"mask", mask, mask_bytes(T), nullptr}},
                        {{"doc_offsets", doc_offsets, n + 4, nullptr},
                         {"prefix", prefix, n, nullptr}}));
  LaunchCtx c{};
  TP_TRY(make_launch_ctx(stream, false, &c));
  return cuda_status(launch_attention_mask(c, doc_offsets, n_docs, prefix, causal != 0, mask, T),
                     "mask launch");
}

tp_status tp_attention_scored(const void* Q, const void* K, const void* V, void* O, float* LSE,
                              int64_t T, int p, int n_heads, int n_kv_heads, int head_dim,
                              const tp_score_params* score, void* stream) {
  set_error_detail("%s", "");
  ScoreCall a{};
  TP_TRY(score_call(&a, T, p, n_heads, n_kv_heads, head_dim, score));
  if (T == 0) return TP_OK;
  TP_TRY(check_bf16(Q, "Q"));
  TP_TRY(check_bf16(K, "K"));
  TP_TRY(check_bf16(V, "V"));
  TP_TRY(check_bf16(O, "O"));
  if (!aligned(LSE, 4)) TP_FAIL(TP_ERR_ALIGNMENT, "LSE must be 4-byte aligned");
  const size_t t = static_cast<size_t>(T), q = t * n_heads * 256, kv = t * n_kv_heads * 256;
  const size_t lse = t * n_heads * 4;
  TP_TRY(check_overlaps({{"O", O, q, nullptr}, {"LSE", LSE, lse, nullptr}},
                        {{"Q", Q, q, nullptr},
                         {"K", K, kv, nullptr},
                         {"V", V, kv, nullptr},
                         {"slopes", a.slopes, static_cast<size_t>(n_heads) * 4, nullptr},
                         {"mask", a.mask, mask_bytes(T), nullptr}}));
  a.Q = Q;
  a.K = K;
  a.V = V;
  a.O = O;
  a.LSE = LSE;
  LaunchCtx c{};
  TP_TRY(make_launch_ctx(stream, true, &c));
  return launch_attention_scored(c, a);
}

size_t tp_attention_scored_backward_workspace_size(int64_t T, int p, int n_heads, int n_kv_heads,
                                                   int head_dim) {
  ScoreCall a{};
  tp_score_params least{};   // (the mask that leaves the fewest steps)
  least.causal = 1;
  if (score_bwd_call(&a, T, p, n_heads, n_kv_heads, head_dim, &least) != TP_OK) return 0;
  return T == 0 ? 256 : score_bwd_ws(a);
}

tp_status tp_attention_scored_backward(const void* Q, const void* K, const void* V, const void* O,
                                       const float* LSE, const void* dO, void* dQ, void* dK,
                                       void* dV, void* workspace, size_t workspace_bytes,
                                       int64_t T, int p, int n_heads, int n_kv_heads, int head_dim,
                                       const tp_score_params* score, void* stream) {
  set_error_detail("%s", "");
  ScoreCall a{};
  TP_TRY(score_bwd_call(&a, T, p, n_heads, n_kv_heads, head_dim, score));
  if (T == 0) return TP_OK;
  TP_TRY(check_bf16(Q, "Q"));
  TP_TRY(check_bf16(K, "K"));
  TP_TRY(check_bf16(V, "V"));
  TP_TRY(check_bf16(O, "O"));
  TP_TRY(check_bf16(dO, "dO"));
  TP_TRY(check_bf16(dQ, "dQ"));
  TP_TRY(check_bf16(dK, "dK"));
  TP_TRY(check_bf16(dV, "dV"));
  if (LSE == nullptr) TP_FAIL(TP_ERR_INVALID_ARG, "LSE is NULL");
  if (!aligned(LSE, 4)) TP_FAIL(TP_ERR_ALIGNMENT, "LSE must be 4-byte aligned");
  const size_t need = score_bwd_ws(a);
  TP_TRY(check_workspace(workspace, workspace_bytes, need));
  const size_t t = static_cast<size_t>(T), q = t * n_heads * 256, kv = t * n_kv_heads * 256;
  TP_TRY(check_overlaps({{"dQ", dQ, q, nullptr},
                         {"dK", dK, kv, nullptr},
                         {"dV", dV, kv, nullptr},
                         {"workspace", workspace, need, nullptr}},
                        {{"Q", Q, q, nullptr},
                         {"K", K, kv, nullptr},
                         {"V", V, kv, nullptr},
                         {"O", O, q, nullptr},
                         {"dO", dO, q, nullptr},
                         {"LSE", LSE, t * n_heads * 4, nullptr},
                         {"slopes", a.slopes, static_cast<size_t>(n_heads) * 4, nullptr},
                         {"mask", a.mask, mask_bytes(T), nullptr}}));
  a.Q = Q;
  a.K = K;
  a.V = V;
  a.O = const_cast<void*>(O);
  a.LSE = const_cast<float*>(LSE);
  a.dO = dO;
  a.dQ = dQ;
  a.dK = dK;
  a.dV = dV;
  a.delta = static_cast<float*>(workspace);
  a.k_bad = static_cast<uint8_t*>(workspace) + score_delta_ws(a);
  a.part = reinterpret_cast<float*>(a.k_bad + score_bad_ws(a));
  LaunchCtx c{};
  TP_TRY(make_launch_ctx(stream, true, &c));
  return launch_attention_scored_bwd(c, a);
}

size_t tp_attention_decode_workspace_size(int64_t B, int64_t capacity, int p, int n_heads,
                                          int n_kv_heads, int head_dim) {
  ScoreCall a{};
  if (decode_sizes(&a, B, capacity, p, n_heads, n_kv_heads, head_dim, nullptr) != TP_OK) return 0;
  return B == 0 ? 256 : decode_ws(a, B, capacity);
}

tp_status tp_attention_decode(const void* Q, const void* K_new, const void* V_new, void* K_cache,
                              void* V_cache, const int32_t* lengths, void* O, float* LSE,
                              void* workspace, size_t workspace_bytes, int64_t B,
                              int64_t capacity, int p, int n_heads, int n_kv_heads, int head_dim,
                              const tp_score_params* score, void* stream) {
  set_error_detail("%s", "");
  ScoreCall a{};
  TP_TRY(decode_sizes(&a, B, capacity, p, n_heads, n_kv_heads, head_dim, score));
  if (B == 0) return TP_OK;
  TP_TRY(check_bf16(Q, "Q"));
  if ((K_new == nullptr) != (V_new == nullptr))
    TP_FAIL(TP_ERR_INVALID_ARG, "K_new and V_new are given together or not at all");
  if (K_new != nullptr) {
    TP_TRY(check_bf16(K_new, "K_new"));
    TP_TRY(check_bf16(V_new, "V_new"));
  }
  TP_TRY(check_bf16(K_cache, "K_cache"));
  TP_TRY(check_bf16(V_cache, "V_cache"));
  TP_TRY(check_bf16(O, "O"));
  if (lengths == nullptr) TP_FAIL(TP_ERR_INVALID_ARG, "lengths is NULL");
  if (!aligned(lengths, 4) || !aligned(LSE, 4))
    TP_FAIL(TP_ERR_ALIGNMENT, "lengths and LSE must be 4-byte aligned");
  const size_t need = decode_ws(a, B, capacity);
  TP_TRY(check_workspace(workspace, workspace_bytes, need));
  const size_t b = static_cast<size_t>(B), q = b * n_heads * 256, kv = b * n_kv_heads * 256;
  const size_t cache = kv * static_cast<size_t>(capacity);
  TP_TRY(check_overlaps({{"O", O, q, nullptr},
                         {"LSE", LSE, b * n_heads * 4, nullptr},
                         {"K_cache", K_cache, cache, nullptr},
                         {"V_cache", V_cache, cache, nullptr},
                         {"workspace", workspace, need, nullptr}},
                        {{"Q", Q, q, nullptr},
                         {"K_new", K_new, kv, nullptr},
                         {"V_new", V_new, kv, nullptr},
                         {"lengths", lengths, b * 4, nullptr},
                         {"slopes", a.slopes, static_cast<size_t>(n_heads) * 4, nullptr}}));
  DecodeCall d{};
  d.Q = Q;
  d.Kn = K_new;
  d.Vn = V_new;
  d.Kc = K_cache;
  d.Vc = V_cache;
  d.O = O;
  d.LSE = LSE;
  d.part = static_cast<float*>(workspace);
  d.len = lengths;
  d.B = B;
  d.capacity = capacity;
  d.p = a.p;
  d.hq = a.hq;
  d.hkv = a.hkv;
  d.scale = a.scale;
  d.cap = a.cap;
  d.slopes = a.slopes;
  LaunchCtx c{};
  TP_TRY(make_launch_ctx(stream, false, &c));
  return launch_attention_decode(c, d);
}

}  // extern "C"
