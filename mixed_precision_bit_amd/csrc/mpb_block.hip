// Host side of the operators around the packed experts: argument validation
// and launches. Every export validates before anything is enqueued and lets no
// C++ exception escape.
#include <cmath>
#include <string>

#include "mpb.h"
#include "mpb_internal.h"

namespace {

int fail(int code, const std::string& msg) { return mpb::set_error(code, msg.c_str()); }

int hip_fail(hipError_t e, const char* where) {
  return fail(MPB_E_HIP, std::string(where) + ": " + hipGetErrorString(e));
}

// The kernels read rows in 16-byte vectors.
bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
template <class... P>
bool all_aligned16(P... p) {
  return (aligned16(p) && ...);
}

int check_rows(const std::string& n, int x_dtype, int T, int H) {
  if (x_dtype != MPB_F16 && x_dtype != MPB_BF16) return fail(MPB_E_ARG, n + ": bad x_dtype");
  if (T < 0) return fail(MPB_E_ARG, n + ": T < 0");
  if (T > (1 << 20)) return fail(MPB_E_SHAPE, n + ": T above 2^20");
  if (H <= 0 || H % 64 || H > 65536) return fail(MPB_E_SHAPE, n + ": H must be a multiple of 64 in 64..65536");
  return MPB_OK;
}

int check_norm(const std::string& n, int gate_kind, float scale, float eps) {
  if (gate_kind != MPB_GATE_NONE && gate_kind != MPB_GATE_TOKEN && gate_kind != MPB_GATE_FULL)
    return fail(MPB_E_ARG, n + ": bad gate_kind");
  if (!std::isfinite(scale)) return fail(MPB_E_ARG, n + ": scale must be finite");
  if (!(eps > 0.0f) || !std::isfinite(eps)) return fail(MPB_E_ARG, n + ": eps must be positive and finite");
  return MPB_OK;
}

int check_router(const std::string& n, int x_dtype, int T, int H, int E, int K, float alpha, float beta) {
  const int rc = check_rows(n, x_dtype, T, H);
  if (rc) return rc;
  if (E < 1 || E > 512) return fail(MPB_E_SHAPE, n + ": E must be in 1..512");
  if (K < 1 || K > 16 || K > E) return fail(MPB_E_SHAPE, n + ": K must be in 1..min(E,16)");
  if (!std::isfinite(alpha) || !std::isfinite(beta)) return fail(MPB_E_ARG, n + ": alpha and beta must be finite");
  return MPB_OK;
}

int check_ws(const std::string& n, const void* ws, size_t bytes, size_t need) {
  if (!ws) return fail(MPB_E_ARG, n + ": null workspace");
  if (!aligned16(ws)) return fail(MPB_E_ARG, n + ": the workspace must be 16-byte aligned");
  if (bytes < need) return fail(MPB_E_WS, n + ": workspace " + std::to_string(bytes) + " < " + std::to_string(need));
  return MPB_OK;
}

mpb::RouterLossParams router_params(const void* X, const float* W, const int32_t* idx, const uint8_t* mask, int T, int H,
                                    int E, int K, float alpha, float beta, void* ws_dev) {
  const mpb::RouterLossWs w = mpb::router_loss_ws(T, H, E);
  char* ws = (char*)ws_dev;
  mpb::RouterLossParams p{};
  p.X = X; p.W = W; p.idx = idx; p.mask = mask;
  p.T = T; p.H = H; p.E = E; p.K = K; p.alpha = alpha; p.beta = beta;
  p.part = (float*)(ws + w.part);
  p.stat = (int2*)(ws + w.stat);
  p.dl_a = (uint16_t*)(ws + w.dl_a);
  p.dl_s = (float*)(ws + w.dl_s);
  p.dl_t = (uint16_t*)(ws + w.dl_t);
  p.on = (uint8_t*)(ws + w.on);
  p.db_part = (float*)(ws + w.db_part);
  p.dw_part = (float*)(ws + w.dw_part);
  p.splits = w.splits; p.groups = w.groups; p.chunks = w.chunks; p.dx_ranges = w.dx_ranges;
  p.Tp = w.Tp; p.Ep = w.Ep;
  p.mt = w.mt; p.et = w.et;
  return p;
}

}  // namespace

extern "C" {

int moe_block_norm(const float* o_dev, const void* r_dev, int x_dtype, int T, int H, const void* gate_dev,
                   int gate_kind, const float* gamma_post_dev, const float* gamma_next_dev, float scale, float eps,
                   void* r_out_dev, void* x_out_dev, void* stream) try {
  const std::string n("moe_block_norm");
  int rc = check_rows(n, x_dtype, T, H);
  if (!rc) rc = check_norm(n, gate_kind, scale, eps);
  if (rc) return rc;
  if (T == 0) return MPB_OK;
  if ((gate_kind != MPB_GATE_NONE) != (gate_dev != nullptr))
    return fail(MPB_E_ARG, n + ": gate and gate_kind disagree");
  if ((gamma_next_dev != nullptr) != (x_out_dev != nullptr))
    return fail(MPB_E_ARG, n + ": gamma_next and x_out go together");
  if ((o_dev != nullptr) != (r_out_dev != nullptr)) return fail(MPB_E_ARG, n + ": o and r_out go together");
  if (!o_dev && (gamma_post_dev || gate_dev)) return fail(MPB_E_ARG, n + ": a gate or gamma_post needs o");
  if (!o_dev && !x_out_dev) return fail(MPB_E_ARG, n + ": neither o nor x_out");
  if (!r_dev) return fail(MPB_E_ARG, n + ": null pointer");
  if (!all_aligned16(o_dev, r_dev, gamma_post_dev, gamma_next_dev, r_out_dev, x_out_dev) ||
      (gate_kind == MPB_GATE_FULL && !aligned16(gate_dev)))
    return fail(MPB_E_ARG, n + ": rows must be 16-byte aligned");
  mpb::BlockNormParams p{o_dev, r_dev, gate_dev, gamma_post_dev, gamma_next_dev, r_out_dev, x_out_dev,
                         scale, eps, gate_kind, T, H};
  const hipError_t e = mpb::launch_block_norm(p, x_dtype == MPB_BF16, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "moe_block_norm");
  return MPB_OK;
} catch (...) {
  return mpb::set_error(MPB_E_HIP, "moe_block_norm: unexpected exception");
}

size_t moe_block_norm_grad_workspace_bytes(int T, int H) {
  if (T < 0 || T > (1 << 20) || H <= 0 || H % 64 || H > 65536) return 0;
  const size_t b = (size_t)2 * mpb::block_norm_grad_groups(T) * H * sizeof(float);
  return b < 256 ? 256 : b;
}

int moe_block_norm_grad(const float* o_dev, const void* y_dev, int x_dtype, int T, int H, const void* gate_dev,
                        int gate_kind, const float* gamma_post_dev, const float* gamma_next_dev, float scale,
                        float eps, const void* dr_out_dev, const void* dx_dev, void* dr_dev, float* do_dev,
                        void* dgate_dev, float* dgamma_post_dev, float* dgamma_next_dev, void* ws_dev,
                        size_t ws_bytes, void* stream) try {
  const std::string n("moe_block_norm_grad");
  int rc = check_rows(n, x_dtype, T, H);
  if (!rc) rc = check_norm(n, gate_kind, scale, eps);
  if (rc) return rc;
  if (!all_aligned16(o_dev, y_dev, gamma_post_dev, gamma_next_dev, dr_out_dev, dx_dev, dr_dev, do_dev, dgamma_post_dev,
                     dgamma_next_dev, ws_dev) ||
      (gate_kind == MPB_GATE_FULL && !all_aligned16(gate_dev, dgate_dev)))
    return fail(MPB_E_ARG, n + ": rows must be 16-byte aligned");
  if (T > 0) {  // an empty batch has no rows to point at
    if ((gate_kind != MPB_GATE_NONE) != (gate_dev != nullptr))
      return fail(MPB_E_ARG, n + ": gate and gate_kind disagree");
    if ((gamma_next_dev != nullptr) != (dx_dev != nullptr))
      return fail(MPB_E_ARG, n + ": gamma_next and dx go together");
    if (!dr_out_dev && !dx_dev) return fail(MPB_E_ARG, n + ": neither dr_out nor dx");
    if (dgamma_next_dev && !gamma_next_dev) return fail(MPB_E_ARG, n + ": dgamma_next needs gamma_next");
    if (dgamma_post_dev && !gamma_post_dev) return fail(MPB_E_ARG, n + ": dgamma_post needs gamma_post");
    if (dgate_dev && !gate_dev) return fail(MPB_E_ARG, n + ": dgate needs a gate");
    if ((gamma_post_dev || gate_dev) && !o_dev) return fail(MPB_E_ARG, n + ": a gate or gamma_post needs o");
    if (!dr_dev || (dx_dev && !y_dev)) return fail(MPB_E_ARG, n + ": null pointer");
    if (dgamma_post_dev || dgamma_next_dev) {
      if (!ws_dev) return fail(MPB_E_ARG, n + ": null workspace");
      const size_t need = moe_block_norm_grad_workspace_bytes(T, H);
      if (ws_bytes < need)
        return fail(MPB_E_WS, n + ": workspace " + std::to_string(ws_bytes) + " < " + std::to_string(need));
    }
  } else if (!dgamma_post_dev && !dgamma_next_dev) {
    return MPB_OK;
  }
  // o is read only where the gate or the norm needs it
  mpb::BlockNormGradParams p{gamma_post_dev || gate_dev ? o_dev : nullptr, y_dev, gate_dev, gamma_post_dev,
                             gamma_next_dev, dr_out_dev, dx_dev, dr_dev, do_dev, dgate_dev, dgamma_post_dev,
                             dgamma_next_dev, (float*)ws_dev, scale, eps, gate_kind, T, H};
  const hipError_t e = mpb::launch_block_norm_grad(p, x_dtype == MPB_BF16, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "moe_block_norm_grad");
  return MPB_OK;
} catch (...) {
  return mpb::set_error(MPB_E_HIP, "moe_block_norm_grad: unexpected exception");
}

size_t moe_router_loss_workspace_bytes(int T, int H, int E) {
  if (T < 0 || T > (1 << 20) || H <= 0 || H % 64 || H > 65536 || E < 1 || E > 512) return 0;
  return mpb::router_loss_ws(T, H, E).total;
}

int moe_router_loss(const void* X_dev, int x_dtype, const float* W_router_dev, const float* bias_dev,
                    const int32_t* topk_idx_dev, const uint8_t* mask_dev, int T, int H, int E, int K, float alpha,
                    float beta, float* logits_dev, float* lse_dev, int32_t* counts_dev, float* prob_dev,
                    float* loss_dev, void* ws_dev, size_t ws_bytes, void* stream) try {
  const std::string n("moe_router_loss");
  int rc = check_router(n, x_dtype, T, H, E, K, alpha, beta);
  if (rc) return rc;
  if (!counts_dev || !prob_dev || !loss_dev) return fail(MPB_E_ARG, n + ": null pointer");
  if (T > 0 && (!X_dev || !W_router_dev || !topk_idx_dev || !logits_dev || !lse_dev))
    return fail(MPB_E_ARG, n + ": null pointer");
  if (!all_aligned16(X_dev, W_router_dev)) return fail(MPB_E_ARG, n + ": rows must be 16-byte aligned");
  rc = check_ws(n, ws_dev, ws_bytes, moe_router_loss_workspace_bytes(T, H, E));
  if (rc) return rc;
  mpb::RouterLossParams p = router_params(X_dev, W_router_dev, topk_idx_dev, mask_dev, T, H, E, K, alpha, beta, ws_dev);
  p.bias = bias_dev;
  p.logits = logits_dev; p.lse = lse_dev; p.counts = counts_dev; p.prob = prob_dev; p.loss = loss_dev;
  const hipError_t e = mpb::launch_router_loss(p, x_dtype == MPB_BF16, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "moe_router_loss");
  return MPB_OK;
} catch (...) {
  return mpb::set_error(MPB_E_HIP, "moe_router_loss: unexpected exception");
}

int moe_router_loss_grad(const void* X_dev, int x_dtype, const float* W_router_dev, const int32_t* topk_idx_dev,
                         const uint8_t* mask_dev, const float* logits_dev, const float* lse_dev,
                         const int32_t* counts_dev, int T, int H, int E, int K, float alpha, float beta,
                         const float* gw_dev, const float* gloss_dev, float* dX_dev, float* dW_dev, float* dbias_dev,
                         void* ws_dev, size_t ws_bytes, void* stream) try {
  const std::string n("moe_router_loss_grad");
  int rc = check_router(n, x_dtype, T, H, E, K, alpha, beta);
  if (rc) return rc;
  if (T > 0 && (!logits_dev || !lse_dev || !counts_dev || (dX_dev && !W_router_dev) || (dW_dev && !X_dev) ||
                (gw_dev && !topk_idx_dev)))
    return fail(MPB_E_ARG, n + ": null pointer");
  if (!all_aligned16(X_dev, W_router_dev, dX_dev, dW_dev)) return fail(MPB_E_ARG, n + ": rows must be 16-byte aligned");
  if (!dX_dev && !dW_dev && !dbias_dev) {
    if (T > 0) return fail(MPB_E_ARG, n + ": no gradient asked for");
    return MPB_OK;
  }
  rc = check_ws(n, ws_dev, ws_bytes, moe_router_loss_workspace_bytes(T, H, E));
  if (rc) return rc;
  mpb::RouterLossParams p = router_params(X_dev, W_router_dev, topk_idx_dev, mask_dev, T, H, E, K, alpha, beta, ws_dev);
  p.logits = const_cast<float*>(logits_dev);
  p.lse = const_cast<float*>(lse_dev);
  p.counts = const_cast<int32_t*>(counts_dev);
  p.gw = gw_dev; p.gloss = gloss_dev; p.dX = T > 0 ? dX_dev : nullptr; p.dW = dW_dev; p.dbias = dbias_dev;
  const hipError_t e = mpb::launch_router_loss_grad(p, x_dtype == MPB_BF16, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "moe_router_loss_grad");
  return MPB_OK;
} catch (...) {
  return mpb::set_error(MPB_E_HIP, "moe_router_loss_grad: unexpected exception");
}

size_t moe_adapters_workspace_bytes(int T, int Kd, int n, int R) {
  if (T < 0 || T > (1 << 20) || Kd <= 0 || Kd % 64 || Kd > 65536 || n < 1 || n > mpb::kAdapterMaxN || R < 8 || R > 128 ||
      R % 8)
    return 0;
  return mpb::adapter_ws(T, Kd, n, R).total;
}

int moe_adapters(const void* X_dev, int x_dtype, int T, int Kd, const void* A_dev, const void* B_dev,
                 const int32_t* ranks_dev, const float* scales_dev, int n, int R, int N, const int32_t* adapter_dev,
                 const float* base_dev, float* out_dev, void* ws_dev, size_t ws_bytes, void* stream) try {
  const std::string nm("moe_adapters");
  int rc = check_rows(nm, x_dtype, T, Kd);
  if (rc) return rc;
  if (N <= 0 || N % 64 || N > 131072) return fail(MPB_E_SHAPE, nm + ": N must be a multiple of 64 in 64..131072");
  if (n < 1 || n > mpb::kAdapterMaxN) return fail(MPB_E_SHAPE, nm + ": n must be in 1..4096");
  if (R < 8 || R > 128 || R % 8) return fail(MPB_E_SHAPE, nm + ": R must be a multiple of 8 in 8..128");
  if (T == 0) return MPB_OK;
  if (!X_dev || !A_dev || !B_dev || !adapter_dev || !out_dev) return fail(MPB_E_ARG, nm + ": null pointer");
  if (!all_aligned16(X_dev, A_dev, B_dev, base_dev, out_dev))
    return fail(MPB_E_ARG, nm + ": rows must be 16-byte aligned");
  const mpb::AdapterWs w = mpb::adapter_ws(T, Kd, n, R);
  rc = check_ws(nm, ws_dev, ws_bytes, w.total);
  if (rc) return rc;
  char* ws = (char*)ws_dev;
  mpb::AdapterParams p{X_dev, A_dev, B_dev, ranks_dev, scales_dev, adapter_dev, base_dev, out_dev, T, Kd, N, n, R,
                       (float*)(ws + w.z), w.scan ? nullptr : (int32_t*)(ws + w.perm),
                       w.scan ? nullptr : (int32_t*)(ws + w.tiles), w.ranges};
  const hipError_t e = mpb::launch_adapters(p, w, x_dtype == MPB_BF16, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "moe_adapters");
  return MPB_OK;
} catch (...) {
  return mpb::set_error(MPB_E_HIP, "moe_adapters: unexpected exception");
}

}  // extern "C"
