// C ABI of the operators around the layer: argument validation and launches. The contract
// of each entry point is stated in include/moe355_block.h.
#include <hip/hip_runtime.h>
#include <rocprofiler-sdk-roctx/roctx.h>

#include <cmath>
#include <initializer_list>

#include "common.h"
#include "kernels.h"

namespace moe {

// a named roctx range around one entry point's launches (seen by rocprofv3 --marker-trace)
struct BlockRange {
  explicit BlockRange(const char* name) { roctxRangePushA(name); }
  ~BlockRange() { roctxRangePop(); }
};

static bool misaligned(std::initializer_list<const void*> ps, uintptr_t to) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % to != 0) return true;
  return false;
}

constexpr int32_t kMaxWidth = 32768;

// shape, weight type and quantised format of the norm, in the order the contract lists them
static int check_norm(const void* weight, int32_t weight_dtype, int32_t T, int32_t H) {
  if (!weight || T < 0 || H < 8 || (weight_dtype != MOE_BF16 && weight_dtype != MOE_F32)) return MOE_ERR_INVALID;
  if (misaligned({weight}, 16)) return MOE_ERR_INVALID;
  if (H % 8 != 0 || H > kMaxWidth) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// the two norms around the residual's addition, their gate and scales
static int check_sandwich(const void* post_weight, const void* weight, int32_t weight_dtype, const void* gate,
                          const moe_sandwich_config* c, int32_t T, int32_t H) {
  if (!c || T < 0 || H < 8 || (weight_dtype != MOE_BF16 && weight_dtype != MOE_F32)) return MOE_ERR_INVALID;
  if (misaligned({post_weight, weight}, 16)) return MOE_ERR_INVALID;
  if (!(c->eps >= 0.0) || !std::isfinite(c->eps) || !(c->post_eps >= 0.0) || !std::isfinite(c->post_eps)) return MOE_ERR_INVALID;
  if (!std::isfinite(c->res_scale) || !std::isfinite(c->branch_scale)) return MOE_ERR_INVALID;
  if (c->gate < MOE_GATE_NONE || c->gate > MOE_GATE_FULL) return MOE_ERR_INVALID;
  if (c->gate_act < MOE_GATE_IDENTITY || c->gate_act > MOE_GATE_TANH) return MOE_ERR_INVALID;
  if (c->gate_dtype != MOE_BF16 && c->gate_dtype != MOE_F32) return MOE_ERR_INVALID;
  if (c->gate == MOE_GATE_NONE ? gate != nullptr : (!gate && (T > 0 || c->gate == MOE_GATE_CHANNEL))) return MOE_ERR_INVALID;
  if (misaligned({gate}, c->gate != MOE_GATE_ROW ? 16 : c->gate_dtype == MOE_F32 ? 4 : 2)) return MOE_ERR_INVALID;
  if (H % 8 != 0 || H > kMaxWidth) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// adapters of a call: their table, the rows' grouping, and the pitches of its row arrays (in elements)
static int check_adapter(const void* a, const void* b, const float* scale, const int32_t* ranks, int32_t n, int32_t T,
                         int32_t K, int32_t N, int32_t R) {
  if (!a || !b || n < 1 || n > 1024 || T < 0 || K < 8 || N < 8 || R < 8) return MOE_ERR_INVALID;
  if (misaligned({a, b}, 16) || misaligned({scale, ranks}, 4)) return MOE_ERR_INVALID;
  if (K % 8 != 0 || N % 8 != 0 || R % 8 != 0 || K > kMaxWidth || N > kMaxWidth || R > 256) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
static int check_adapter_plan(const moe_plan_t* p, int32_t n, int32_t T) {
  const int rc = check_plan(p);
  if (rc != MOE_OK) return rc;
  return p->T == T && p->K == 1 && p->E_local == n ? MOE_OK : MOE_ERR_INVALID;
}
static bool bad_pitch(int32_t ld, int32_t width) { return ld < width || ld % 8 != 0; }

static int check_router(int32_t logits_dtype, int32_t T, int32_t E, int32_t K, const moe_router_config* c) {
  if (!c || T < 0 || E < 1 || E > 1024 || K < 1 || K > 16) return MOE_ERR_INVALID;
  if (logits_dtype != MOE_BF16 && logits_dtype != MOE_F32) return MOE_ERR_INVALID;
  if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID;
  if (c->normalize != 0 && c->normalize != 1) return MOE_ERR_INVALID;
  if (c->groups < 1 || c->groups > 64 || E % c->groups != 0) return MOE_ERR_INVALID;
  if (c->topk_groups < 1 || c->topk_groups > c->groups) return MOE_ERR_INVALID;
  if (c->group_top != 1 && c->group_top != 2) return MOE_ERR_INVALID;
  if (K > c->topk_groups * (E / c->groups)) return MOE_ERR_INVALID;
  if (!std::isfinite(c->scale)) return MOE_ERR_INVALID;
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" {

MOE355_API int moe_rmsnorm(const void* x, const void* res, const void* weight, int32_t weight_dtype, int32_t T,
                           int32_t H, double eps, void* s_out, void* y, float* rstd, int32_t q_dtype, void* q,
                           void* q_s, void* stream) {
  BlockRange trace("moe_rmsnorm");
  int rc = check_norm(weight, weight_dtype, T, H);
  if (rc == MOE_ERR_INVALID) return rc;
  if (!(eps >= 0.0) || !std::isfinite(eps)) return MOE_ERR_INVALID;
  if (q_dtype != MOE_BF16 && q_dtype != MOE_FP8_E4M3_G128 && q_dtype != MOE_MXFP4) return MOE_ERR_INVALID;
  if (T > 0) {
    if (!x || (!y && !q)) return MOE_ERR_INVALID;
    if (q_dtype == MOE_BF16 ? (q || q_s) : (!q || !q_s)) return MOE_ERR_INVALID;
    if (s_out && (!res || s_out == y)) return MOE_ERR_INVALID;
    if (misaligned({x, res, s_out, y, q}, 16) || misaligned({rstd, q_s}, 4)) return MOE_ERR_INVALID;
  }
  if (rc != MOE_OK) return rc;
  if ((q_dtype == MOE_FP8_E4M3_G128 && H % 128 != 0) || (q_dtype == MOE_MXFP4 && H % 32 != 0))
    return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  return launch_rmsnorm(x, res, weight, weight_dtype == MOE_F32, T, H, eps, s_out, y, rstd, q_dtype, q, q_s,
                        static_cast<hipStream_t>(stream));
}

MOE355_API size_t moe_rmsnorm_backward_workspace_bytes(int32_t T, int32_t H) {
  if (T < 1 || H < 8 || H % 8 != 0 || H > kMaxWidth) return 0;
  return (size_t)rmsnorm_backward_blocks(T, H) * H * sizeof(float);
}

MOE355_API int moe_rmsnorm_backward(const void* dy, const void* s, const void* weight, int32_t weight_dtype,
                                    const float* rstd, const void* d_res, int32_t T, int32_t H, void* dx,
                                    float* dweight, void* ws, size_t ws_bytes, void* stream) {
  BlockRange trace("moe_rmsnorm_backward");
  int rc = check_norm(weight, weight_dtype, T, H);
  if (rc == MOE_ERR_INVALID) return rc;
  if (misaligned({dweight}, 4)) return MOE_ERR_INVALID;
  if (T > 0) {
    if (!dy || !s || !rstd || !dx) return MOE_ERR_INVALID;
    if (misaligned({dy, s, d_res, dx}, 16) || misaligned({rstd}, 4)) return MOE_ERR_INVALID;
  }
  if (rc != MOE_OK) return rc;
  if (T > 0 && dweight &&
      (!ws || misaligned({ws}, 16) || ws_bytes < moe_rmsnorm_backward_workspace_bytes(T, H)))
    return MOE_ERR_INVALID;
  return launch_rmsnorm_backward(dy, s, weight, weight_dtype == MOE_F32, rstd, d_res, T, H, dx, dweight, ws,
                                 static_cast<hipStream_t>(stream));
}

MOE355_API int moe_sandwich_norm(const void* x, const void* res, const void* post_weight, const void* weight,
                                 int32_t weight_dtype, const void* gate, const moe_sandwich_config* cfg, int32_t T,
                                 int32_t H, void* s_out, void* y, float* post_rstd, float* rstd, int32_t q_dtype,
                                 void* q, void* q_s, void* stream) {
  BlockRange trace("moe_sandwich_norm");
  const int rc = check_sandwich(post_weight, weight, weight_dtype, gate, cfg, T, H);
  if (rc == MOE_ERR_INVALID) return rc;
  if (q_dtype != MOE_BF16 && q_dtype != MOE_FP8_E4M3_G128 && q_dtype != MOE_MXFP4) return MOE_ERR_INVALID;
  if (T > 0) {
    if (!x || !s_out || s_out == y) return MOE_ERR_INVALID;
    if (weight ? (!y && !q) : (y || rstd)) return MOE_ERR_INVALID;
    if (!post_weight && post_rstd) return MOE_ERR_INVALID;
    if (q_dtype == MOE_BF16 ? (q || q_s) : (!q || !q_s || !weight)) return MOE_ERR_INVALID;
    if (misaligned({x, res, s_out, y, q}, 16) || misaligned({post_rstd, rstd, q_s}, 4)) return MOE_ERR_INVALID;
  }
  if (rc != MOE_OK) return rc;
  if ((q_dtype == MOE_FP8_E4M3_G128 && H % 128 != 0) || (q_dtype == MOE_MXFP4 && H % 32 != 0))
    return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  return launch_sandwich_norm({x, res, post_weight, weight, weight_dtype == MOE_F32, gate, *cfg, T, H, s_out, y, post_rstd, rstd,
                               q_dtype, q, q_s},
                              static_cast<hipStream_t>(stream));
}

MOE355_API size_t moe_sandwich_norm_backward_workspace_bytes(int32_t T, int32_t H) {
  if (T < 1 || H < 8 || H % 8 != 0 || H > kMaxWidth) return 0;
  return (size_t)3 * sandwich_backward_blocks(T, H) * H * sizeof(float);   // two weights and a channel gate
}

MOE355_API int moe_sandwich_norm_backward(const void* dy, const void* d_s, const void* x, const void* s,
                                          const void* post_weight, const void* weight, int32_t weight_dtype,
                                          const void* gate, const moe_sandwich_config* cfg, const float* post_rstd,
                                          const float* rstd, int32_t T, int32_t H, void* dx, void* d_res,
                                          float* dweight, float* d_post_weight, void* d_gate, void* ws,
                                          size_t ws_bytes, void* stream) {
  BlockRange trace("moe_sandwich_norm_backward");
  const int rc = check_sandwich(post_weight, weight, weight_dtype, gate, cfg, T, H);
  if (rc == MOE_ERR_INVALID) return rc;
  if ((dweight && !weight) || (d_post_weight && !post_weight) || (d_gate && cfg->gate == MOE_GATE_NONE)) return MOE_ERR_INVALID;
  const bool channel = cfg->gate == MOE_GATE_CHANNEL;
  if (misaligned({dweight, d_post_weight}, 4)) return MOE_ERR_INVALID;
  if (misaligned({d_gate}, channel ? 4 : cfg->gate == MOE_GATE_FULL ? 16 : cfg->gate_dtype == MOE_F32 ? 4 : 2)) return MOE_ERR_INVALID;
  const bool sums = dweight || d_post_weight || (channel && d_gate);
  if (T > 0) {
    if (!dx || dx == d_res) return MOE_ERR_INVALID;
    if (weight ? (!dy || !s || !rstd) : (dy || !d_s)) return MOE_ERR_INVALID;
    if ((post_weight || d_gate) && !x) return MOE_ERR_INVALID;
    if (post_weight && !post_rstd) return MOE_ERR_INVALID;
    if (misaligned({dy, d_s, x, s, dx, d_res}, 16) || misaligned({post_rstd, rstd}, 4)) return MOE_ERR_INVALID;
  }
  if (rc != MOE_OK) return rc;
  if (T > 0 && sums && (!ws || misaligned({ws}, 16) || ws_bytes < moe_sandwich_norm_backward_workspace_bytes(T, H)))
    return MOE_ERR_INVALID;
  return launch_sandwich_norm_backward({dy, d_s, x, s, post_weight, weight, weight_dtype == MOE_F32, gate, *cfg, post_rstd, rstd, T, H,
                                        dx, d_res, dweight, d_post_weight, d_gate, ws},
                                       static_cast<hipStream_t>(stream));
}

MOE355_API int moe_router_topk(const void* logits, int32_t logits_dtype, const float* bias, int32_t T, int32_t E,
                               int32_t K, const moe_router_config* cfg, int32_t* topk_idx, float* topk_weights,
                               void* stream) {
  BlockRange trace("moe_router_topk");
  const int rc = check_router(logits_dtype, T, E, K, cfg);
  if (rc != MOE_OK) return rc;
  if (misaligned({bias}, 4)) return MOE_ERR_INVALID;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_weights) return MOE_ERR_INVALID;
  if (misaligned({topk_idx, topk_weights}, 4) || misaligned({logits}, logits_dtype == MOE_BF16 ? 16 : 4))
    return MOE_ERR_INVALID;
  return launch_router_topk(logits, logits_dtype == MOE_BF16, bias, T, E, K, *cfg, topk_idx, topk_weights,
                            static_cast<hipStream_t>(stream));
}

MOE355_API int moe_router_topk_backward(const float* d_topk_weights, const void* logits, int32_t logits_dtype,
                                        const int32_t* topk_idx, int32_t T, int32_t E, int32_t K,
                                        const moe_router_config* cfg, void* d_logits, void* stream) {
  BlockRange trace("moe_router_topk_backward");
  const int rc = check_router(logits_dtype, T, E, K, cfg);
  if (rc != MOE_OK) return rc;
  if (T == 0) return MOE_OK;
  if (!d_topk_weights || !logits || !topk_idx || !d_logits) return MOE_ERR_INVALID;
  if (misaligned({topk_idx, d_topk_weights}, 4) ||
      misaligned({logits, d_logits}, logits_dtype == MOE_BF16 ? 16 : 4))
    return MOE_ERR_INVALID;
  return launch_router_topk_backward(d_topk_weights, logits, logits_dtype == MOE_BF16, topk_idx, T, E, K, *cfg,
                                     d_logits, static_cast<hipStream_t>(stream));
}

MOE355_API size_t moe_adapter_workspace_bytes(int32_t T, int32_t K, int32_t R) {
  if (T < 1 || K < 8 || K % 8 != 0 || K > kMaxWidth || R < 8 || R % 8 != 0 || R > 256) return 0;
  return (size_t)adapter_splits(T, K, R) * T * R * sizeof(float) + (size_t)T * R * 6;   // v's partial results, v in 2-byte parts
}

MOE355_API int moe_adapter(const void* x, int32_t ldx, const void* a, const void* b, const float* scale,
                           const int32_t* ranks, int32_t n, int32_t T, int32_t K, int32_t N, int32_t R,
                           const int32_t* ids, int32_t id_begin, const moe_plan_t* plan, const void* base,
                           int32_t ld_base, void* out, int32_t ld_out, float* v, void* ws, size_t ws_bytes,
                           void* stream) {
  BlockRange trace("moe_adapter");
  const int rc = check_adapter(a, b, scale, ranks, n, T, K, N, R);
  if (rc == MOE_ERR_INVALID) return rc;
  if (T > 0) {
    if (!x || !out || !ws || (ids == nullptr) == (plan == nullptr) || id_begin < 0) return MOE_ERR_INVALID;
    if (misaligned({x, base, out, v, ws}, 16) || misaligned({ids}, 4)) return MOE_ERR_INVALID;
    if (bad_pitch(ldx, K) || bad_pitch(ld_out, N) || (base && bad_pitch(ld_base, N))) return MOE_ERR_INVALID;
    if (base == out && ld_base != ld_out) return MOE_ERR_INVALID;
    if (plan && check_adapter_plan(plan, n, T) != MOE_OK) return MOE_ERR_INVALID;
  }
  if (rc != MOE_OK) return rc;
  if (T == 0) return MOE_OK;
  if (ids && T > 64) return MOE_ERR_UNSUPPORTED;
  if (ws_bytes < moe_adapter_workspace_bytes(T, K, R)) return MOE_ERR_INVALID;
  return launch_adapter({x, ldx, a, b, scale, ranks, n, T, K, N, R, ids, id_begin, plan, base, ld_base, out, ld_out, v, ws},
                        static_cast<hipStream_t>(stream));
}

MOE355_API size_t moe_adapter_backward_workspace_bytes(int32_t T, int32_t n, int32_t K, int32_t N, int32_t R) {
  if (n < 1 || n > 1024 || N < 8 || N % 8 != 0 || N > kMaxWidth || moe_adapter_workspace_bytes(T, K, R) == 0) return 0;
  // dv's partial results, dv in two 2-byte parts, dv and v in three each, partial results of da and db
  return moe_adapter_workspace_bytes(T, N, R) + (size_t)T * R * 12 + (size_t)adapter_grad_slots(T) * R * (K + N) * sizeof(float);
}

MOE355_API int moe_adapter_backward(const void* dout, int32_t ld_dout, const void* x, int32_t ldx, const float* v,
                                    const void* a, const void* b, const float* scale, const int32_t* ranks, int32_t n,
                                    int32_t T, int32_t K, int32_t N, int32_t R, const moe_plan_t* plan,
                                    const void* dx_base, int32_t ld_base, void* dx, int32_t ld_dx, float* da, float* db,
                                    void* ws, size_t ws_bytes, void* stream) {
  BlockRange trace("moe_adapter_backward");
  const int rc = check_adapter(a, b, scale, ranks, n, T, K, N, R);
  if (rc == MOE_ERR_INVALID) return rc;
  if (misaligned({da, db}, 16)) return MOE_ERR_INVALID;
  if (T > 0) {
    if (!dout || !ws || (!dx && !da && !db)) return MOE_ERR_INVALID;
    if ((da && !x) || (db && !v)) return MOE_ERR_INVALID;
    if (misaligned({dout, x, v, dx_base, dx, ws}, 16)) return MOE_ERR_INVALID;
    if (bad_pitch(ld_dout, N) || (da && bad_pitch(ldx, K)) || (dx && bad_pitch(ld_dx, K))) return MOE_ERR_INVALID;
    if (dx_base && (!dx || bad_pitch(ld_base, K) || (dx_base == dx && ld_base != ld_dx))) return MOE_ERR_INVALID;
    if (check_adapter_plan(plan, n, T) != MOE_OK) return MOE_ERR_INVALID;
  }
  if (rc != MOE_OK) return rc;
  if (T > 0 && ws_bytes < moe_adapter_backward_workspace_bytes(T, n, K, N, R)) return MOE_ERR_INVALID;
  AdapterLaunch l{};
  l.x = x;
  l.ldx = ldx;
  l.a = a;
  l.b = b;
  l.scale = scale;
  l.ranks = ranks;
  l.n = n;
  l.T = T;
  l.K = K;
  l.N = N;
  l.R = R;
  l.plan = plan;
  l.v = const_cast<float*>(v);
  l.ws = ws;
  return launch_adapter_backward(l, {dout, ld_dout, dx_base, ld_base, dx, ld_dx, da, db}, static_cast<hipStream_t>(stream));
}

MOE355_API int moe_dispatch_quantized(const void* q, const void* q_s, int32_t H, int32_t act_dtype,
                                      const moe_plan_t* plan, int32_t pool_rows, void* pool, void* pool_s,
                                      uint32_t epoch, void* ws, size_t ws_bytes, void* stream) {
  BlockRange trace("moe_dispatch_quantized");
  int rc = check_plan(plan);
  if (rc != MOE_OK) return rc;
  if (!q || !q_s || !pool || !pool_s || !ws || epoch == 0 || H < 8 || pool_rows < 0) return MOE_ERR_INVALID;
  if (act_dtype != MOE_FP8_E4M3_G128 && act_dtype != MOE_MXFP4) return MOE_ERR_INVALID;
  if (misaligned({q, pool}, 16) || misaligned({q_s, pool_s}, 4)) return MOE_ERR_INVALID;
  if (pool_rows % plan->tile != 0) return MOE_ERR_INVALID;   // a row of a partial tile has no scale words
  if (H % (act_dtype == MOE_FP8_E4M3_G128 ? 128 : 32) != 0) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)H * 2 > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
  const WsLayout L = ws_layout(plan->T, plan->K, plan->E_local, plan->tile, 0, 0, MOE_BF16);
  if (ws_bytes < L.plan_end) return MOE_ERR_INVALID;
  return launch_dispatch_quantized(q, q_s, H, *plan, pool_rows, pool, pool_s, epoch, L, static_cast<char*>(ws),
                         static_cast<hipStream_t>(stream));
}

MOE355_API size_t moe_expert_ffn_decode_workspace_bytes(int32_t T, int32_t K, int32_t I) {
  if (T < 1 || T > 64 || K < 1 || K > 16 || I < 1 || I % 128 != 0 || I > kMaxWidth) return 0;
  return decode_ws_bytes(T, K, I);
}

MOE355_API int moe_expert_ffn_decode(const void* x, const void* x_s, int32_t x_dtype, int32_t T, int32_t H, int32_t I,
                                     int32_t K, int32_t expert_begin, int32_t E_local, const int32_t* topk_idx,
                                     const float* topk_weights, const void* w1, const void* w1_s, const void* w2,
                                     const void* w2_s, void* ws, size_t ws_bytes, void* out, void* stream) {
  BlockRange trace("moe_expert_ffn_decode");
  if (T < 0 || K < 1 || K > 16 || E_local < 1 || E_local > 1024 || expert_begin < 0 || H < 1 || I < 1)
    return MOE_ERR_INVALID;
  if (x_dtype != MOE_BF16 && x_dtype != MOE_MXFP4) return MOE_ERR_INVALID;
  if (!w1 || !w1_s || !w2 || !w2_s || misaligned({w1, w1_s, w2, w2_s}, 16)) return MOE_ERR_INVALID;
  if (T > 0) {
    if (!x || !topk_idx || !topk_weights || !ws || !out) return MOE_ERR_INVALID;
    if ((x_dtype == MOE_BF16) != (x_s == nullptr)) return MOE_ERR_INVALID;
    if (misaligned({x, ws, out}, 16) || misaligned({x_s, topk_idx, topk_weights}, 4)) return MOE_ERR_INVALID;
  }
  if (T > 64 || H % 128 != 0 || I % 128 != 0 || H > kMaxWidth || I > kMaxWidth) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  // out is scratch while x is still read
  const char* from = static_cast<const char*>(x);
  const char* to = static_cast<const char*>(out);
  if (from < to + (size_t)T * H * 2 && to < from + (size_t)T * H * (x_dtype == MOE_BF16 ? 2 : 1)) return MOE_ERR_INVALID;
  if (ws_bytes < decode_ws_bytes(T, K, I)) return MOE_ERR_INVALID;
  return launch_expert_ffn_decode(x, x_s, T, H, I, K, expert_begin, E_local, topk_idx, topk_weights, w1, w1_s, w2,
                                  w2_s, ws, out, static_cast<hipStream_t>(stream));
}

}  // extern "C"
