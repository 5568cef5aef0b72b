// Host side of the dense operators beside the packed experts (projections, head
// norms, distillation): argument validation and launches. Every export validates
// before anything is enqueued and lets no C++ exception escape.
#include <cmath>
#include <string>

#include "mpb.h"
#include "mpb_internal.h"

namespace {

int fail(int code, const std::string& msg) { return mpb::set_error(code, msg.c_str()); }

int hip_fail(hipError_t e, const std::string& where) {
  return fail(MPB_E_HIP, where + ": " + hipGetErrorString(e));
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
template <class... P>
bool all_aligned16(P... p) {
  return (aligned16(p) && ...);
}

int check_batch(const std::string& n, int x_dtype, int T) {
  if (x_dtype != MPB_F16 && x_dtype != MPB_BF16) return fail(MPB_E_ARG, n + ": bad x_dtype");
  if (T < 0) return fail(MPB_E_ARG, n + ": T < 0");
  if (T > (1 << 20)) return fail(MPB_E_SHAPE, n + ": T above 2^20");
  return MPB_OK;
}

int check_ws(const std::string& n, const void* ws, size_t bytes, size_t need) {
  if (!ws) return fail(MPB_E_ARG, n + ": null workspace");
  if (!aligned16(ws)) return fail(MPB_E_ARG, n + ": the workspace must be 16-byte aligned");
  if (bytes < need) return fail(MPB_E_WS, n + ": workspace " + std::to_string(bytes) + " < " + std::to_string(need));
  return MPB_OK;
}

bool linear_shape(int T, int Kd, int N) {
  return T >= 0 && T <= (1 << 20) && Kd > 0 && Kd % 64 == 0 && Kd <= 65536 && N > 0 && N % 8 == 0 && N <= 524288;
}

int check_linear(const std::string& n, int x_dtype, int act, int T, int Kd, int N) {
  const int rc = check_batch(n, x_dtype, T);
  if (rc) return rc;
  if (Kd <= 0 || Kd % 64 || Kd > 65536) return fail(MPB_E_SHAPE, n + ": Kd must be a multiple of 64 in 64..65536");
  if (N <= 0 || N % 8 || N > 524288) return fail(MPB_E_SHAPE, n + ": N must be a multiple of 8 in 8..524288");
  if (act < MPB_ACT_NONE || act > MPB_ACT_GELU_TANH) return fail(MPB_E_ARG, n + ": bad act");
  return MPB_OK;
}

size_t up(size_t b) { return (b + 255) / 256 * 256; }

size_t partial_bytes(const mpb::LinearPlan& p, int64_t M, int64_t N) {
  return p.splits > 1 ? up((size_t)p.splits * M * N * sizeof(float)) : 0;
}

// Regions of moe_linear_grad's workspace. dz is formed where it is not dy itself, as
// fp16 parts, and bf16 X and W become fp16 beside them.
struct GradWs {
  size_t part1, part2, x16, w16, maxima, exp2, db_part, partial_x, partial_w, total;
  int rows;
  bool formed;
};
GradWs grad_ws(int T, int Kd, int N, int act, bool dy32, bool bf16) {
  GradWs w{};
  w.formed = act != MPB_ACT_NONE || dy32;
  // one group up to 256 tokens, else some 1024 workgroups of 512 columns
  const int64_t cols = (N + 511) / 512;
  int64_t groups = T <= 256 ? 1 : 1024 / cols;
  if (groups < 1) groups = 1;
  w.rows = (int)((T + groups - 1) / groups);
  if (w.rows < 16) w.rows = 16;
  size_t at = 0;
  auto take = [&](size_t b) {
    const size_t o = at;
    at += up(b);
    return o;
  };
  const size_t part = (size_t)T * N * 2;
  const int parts = w.formed ? 2 : 1;
  w.part1 = take(w.formed ? part : 0);
  w.part2 = take(w.formed ? part : 0);
  w.x16 = take(w.formed && bf16 ? (size_t)T * Kd * 2 : 0);
  w.w16 = take(w.formed && bf16 && T > 0 ? (size_t)N * Kd * 2 : 0);
  w.maxima = take(3 * mpb::kMaxima * sizeof(float));
  w.exp2 = take(3 * sizeof(int32_t));
  w.db_part = take((size_t)((T + w.rows - 1) / w.rows) * N * sizeof(float));
  w.partial_x = take(T > 0 ? partial_bytes(mpb::linear_plan(T, Kd, N, parts), T, Kd) : 0);
  w.partial_w = take(partial_bytes(mpb::linear_plan(N, Kd, T, parts), N, Kd));
  w.total = at;
  return w;
}

int check_heads(const std::string& n, int x_dtype, int T, int Hq, int Hk, int D, float eps, const int32_t* pos, int A,
                const int32_t* axis, const float* freq, int Dr, int pairs) {
  const int rc = check_batch(n, x_dtype, T);
  if (rc) return rc;
  if (Hq < 1 || Hq > 1024 || Hk < 0 || Hk > 1024) return fail(MPB_E_SHAPE, n + ": Hq must be in 1..1024, Hk in 0..1024");
  if (D < 16 || D > 512 || D % 16) return fail(MPB_E_SHAPE, n + ": D must be a multiple of 16 in 16..512");
  if (Dr < 0 || Dr > D || Dr % 16) return fail(MPB_E_SHAPE, n + ": Dr must be a multiple of 16 in 0..D");
  if (!(eps > 0.0f) || !std::isfinite(eps)) return fail(MPB_E_ARG, n + ": eps must be positive and finite");
  if (pairs != MPB_PAIRS_HALVES && pairs != MPB_PAIRS_NEIGHBOURS) return fail(MPB_E_ARG, n + ": bad pairs");
  if (Dr > 0) {
    if (A < 1 || A > 8) return fail(MPB_E_SHAPE, n + ": A must be in 1..8");
    if (!freq || (T > 0 && !pos)) return fail(MPB_E_ARG, n + ": null pointer");
    if (!all_aligned16(freq, axis)) return fail(MPB_E_ARG, n + ": freq and axis must be 16-byte aligned");
  }
  return MPB_OK;
}

int check_stride(const std::string& n, const char* what, const void* p, int64_t stride, int heads, int D) {
  if (!p) return MPB_OK;
  if (!aligned16(p)) return fail(MPB_E_ARG, n + ": " + what + " must be 16-byte aligned");
  if (stride % 8 || stride < (int64_t)heads * D)
    return fail(MPB_E_SHAPE, n + ": the stride of " + what + " must be a multiple of 8 that holds its heads");
  if (stride > ((int64_t)1 << 40)) return fail(MPB_E_SHAPE, n + ": the stride of " + what + " is above 2^40");
  return MPB_OK;
}

int check_distill(const std::string& n, const void* S, int s_dtype, int64_t stride, const void* ids, const void* teacher,
                  int T, int V, int k, float tau, const void* stats, const void* dS) {
  if (s_dtype != MPB_F16 && s_dtype != MPB_BF16 && s_dtype != MPB_F32) return fail(MPB_E_ARG, n + ": bad s_dtype");
  if (T < 0) return fail(MPB_E_ARG, n + ": T < 0");
  if (T > (1 << 20)) return fail(MPB_E_SHAPE, n + ": T above 2^20");
  if (V < 1 || V > 400000) return fail(MPB_E_SHAPE, n + ": V must be in 1..400000");
  if (k < 1 || k > mpb::kDistillMaxK) return fail(MPB_E_SHAPE, n + ": k must be in 1..256");
  if (!(tau >= 1e-3f && tau <= 1e3f)) return fail(MPB_E_ARG, n + ": tau must be in 1e-3..1e3");
  if (T == 0) return MPB_OK;
  if (stride < V || stride > ((int64_t)1 << 40)) return fail(MPB_E_SHAPE, n + ": s_stride must be in V..2^40");
  if (!S || !ids || !teacher || !stats) return fail(MPB_E_ARG, n + ": null pointer");
  if ((uintptr_t)S % (s_dtype == MPB_F32 ? 4 : 2)) return fail(MPB_E_ARG, n + ": S must be aligned to its elements");
  if (!aligned16(stats)) return fail(MPB_E_ARG, n + ": stats must be 16-byte aligned");
  if (dS && ((uintptr_t)dS - (uintptr_t)S) % 16)
    return fail(MPB_E_ARG, n + ": dS and S must lie at the same offset from a 16-byte boundary");
  return MPB_OK;
}

}  // namespace

extern "C" {

size_t moe_linear_workspace_bytes(int T, int Kd, int N) {
  if (!linear_shape(T, Kd, N)) return 0;
  const size_t b = T == 0 || mpb::linear_skinny(T, N, Kd) ? 0 : partial_bytes(mpb::linear_plan(T, N, Kd, 1), T, N);
  return b < 256 ? 256 : b;
}

int moe_linear(const void* X_dev, int x_dtype, const void* W_dev, const float* bias_dev, int act, const void* res_dev,
               int T, int Kd, int N, void* z_dev, void* y_dev, int y_dtype, void* ws_dev, size_t ws_bytes,
               void* stream) try {
  const std::string n("moe_linear");
  int rc = check_linear(n, x_dtype, act, T, Kd, N);
  if (rc) return rc;
  if (y_dtype != x_dtype && y_dtype != MPB_F32) return fail(MPB_E_ARG, n + ": y_dtype must be x_dtype or MPB_F32");
  if (T == 0) return MPB_OK;
  if (!X_dev || !W_dev || !y_dev) return fail(MPB_E_ARG, n + ": null pointer");
  if (!all_aligned16(X_dev, W_dev, bias_dev, res_dev, z_dev, y_dev))
    return fail(MPB_E_ARG, n + ": rows must be 16-byte aligned");
  rc = check_ws(n, ws_dev, ws_bytes, moe_linear_workspace_bytes(T, Kd, N));
  if (rc) return rc;
  mpb::LinearProduct p{};
  p.A = p.A2 = X_dev; p.B = W_dev; p.lda = p.ldb = Kd;
  p.M = T; p.N = N; p.K = Kd;
  p.out = mpb::LinearOut{bias_dev, res_dev, z_dev, y_dev, nullptr, nullptr, act, y_dtype == MPB_F32, N};
  const hipError_t e = mpb::launch_linear(p, x_dtype == MPB_BF16, (float*)ws_dev, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, n);
  return MPB_OK;
} catch (...) {
  return mpb::set_error(MPB_E_HIP, "moe_linear: unexpected exception");
}

size_t moe_linear_grad_workspace_bytes(int T, int Kd, int N, int act, int dy_dtype) {
  if (!linear_shape(T, Kd, N) || act < MPB_ACT_NONE || act > MPB_ACT_GELU_TANH) return 0;
  return grad_ws(T, Kd, N, act, dy_dtype == MPB_F32, true).total;  // of either activation type
}

int moe_linear_grad(const void* X_dev, int x_dtype, const void* W_dev, int act, const void* z_dev, const void* dy_dev,
                    int dy_dtype, int T, int Kd, int N, void* dX_dev, float* dW_dev, float* dbias_dev, void* ws_dev,
                    size_t ws_bytes, void* stream) try {
  const std::string n("moe_linear_grad");
  int rc = check_linear(n, x_dtype, act, T, Kd, N);
  if (rc) return rc;
  if (dy_dtype != x_dtype && dy_dtype != MPB_F32) return fail(MPB_E_ARG, n + ": dy_dtype must be x_dtype or MPB_F32");
  if (T == 0 && !dW_dev && !dbias_dev) return MPB_OK;
  if (!dX_dev && !dW_dev && !dbias_dev) return fail(MPB_E_ARG, n + ": no gradient asked for");
  if (T > 0 && (!dy_dev || (dX_dev && !W_dev) || (dW_dev && !X_dev) || (act != MPB_ACT_NONE && !z_dev)))
    return fail(MPB_E_ARG, n + ": null pointer");
  if (!all_aligned16(X_dev, W_dev, z_dev, dy_dev, dX_dev, dW_dev, dbias_dev))
    return fail(MPB_E_ARG, n + ": rows must be 16-byte aligned");
  const bool bf16 = x_dtype == MPB_BF16;
  const GradWs w = grad_ws(T, Kd, N, act, dy_dtype == MPB_F32, bf16);
  rc = check_ws(n, ws_dev, ws_bytes, moe_linear_grad_workspace_bytes(T, Kd, N, act, dy_dtype));
  if (rc) return rc;
  char* ws = (char*)ws_dev;
  mpb::LinearGradParams p{};
  p.X = X_dev; p.W = W_dev; p.z = z_dev; p.dy = dy_dev;
  p.dX = dX_dev; p.dW = dW_dev; p.dbias = dbias_dev;
  const bool parts = w.formed && (dX_dev || dW_dev);
  p.part1 = parts ? ws + w.part1 : nullptr;
  p.part2 = parts ? ws + w.part2 : nullptr;
  p.x16 = parts && bf16 && dW_dev ? ws + w.x16 : nullptr;
  p.w16 = parts && bf16 && dX_dev ? ws + w.w16 : nullptr;
  p.maxima = (float*)(ws + w.maxima);
  p.exp2 = (int32_t*)(ws + w.exp2);
  p.db_part = (float*)(ws + w.db_part);
  p.partial_x = (float*)(ws + w.partial_x);
  p.partial_w = (float*)(ws + w.partial_w);
  p.T = T; p.Kd = Kd; p.N = N; p.act = act; p.dy32 = dy_dtype == MPB_F32;
  p.rows = w.rows;
  const hipError_t e = mpb::launch_linear_grad(p, bf16, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, n);
  return MPB_OK;
} catch (...) {
  return mpb::set_error(MPB_E_HIP, "moe_linear_grad: unexpected exception");
}

int moe_head_norm(const void* q_dev, int64_t q_stride, const void* k_dev, int64_t k_stride, int x_dtype, int T, int Hq,
                  int Hk, int D, const float* gamma_q_dev, const float* gamma_k_dev, float eps, const int32_t* pos_dev,
                  int A, const int32_t* axis_dev, const float* freq_dev, int Dr, int pairs, void* q_out_dev,
                  int64_t q_out_stride, void* k_out_dev, int64_t k_out_stride, void* stream) try {
  const std::string n("moe_head_norm");
  int rc = check_heads(n, x_dtype, T, Hq, Hk, D, eps, pos_dev, A, axis_dev, freq_dev, Dr, pairs);
  if (!rc && !all_aligned16(gamma_q_dev, gamma_k_dev)) rc = fail(MPB_E_ARG, n + ": gammas must be 16-byte aligned");
  if (rc) return rc;
  if (T == 0) return MPB_OK;
  if (!q_dev || !q_out_dev || (Hk > 0 && (!k_dev || !k_out_dev))) return fail(MPB_E_ARG, n + ": null pointer");
  rc = check_stride(n, "q", q_dev, q_stride, Hq, D);
  if (!rc) rc = check_stride(n, "q_out", q_out_dev, q_out_stride, Hq, D);
  if (!rc && Hk) rc = check_stride(n, "k", k_dev, k_stride, Hk, D);
  if (!rc && Hk) rc = check_stride(n, "k_out", k_out_dev, k_out_stride, Hk, D);
  if (rc) return rc;
  mpb::HeadNormParams p{q_dev, k_dev, gamma_q_dev, gamma_k_dev, pos_dev, axis_dev, freq_dev, q_out_dev, k_out_dev,
                        q_stride, k_stride, q_out_stride, k_out_stride, eps, T, Hq, Hk, D, Dr, A, pairs, 1};
  const hipError_t e = mpb::launch_head_norm(p, x_dtype == MPB_BF16, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, n);
  return MPB_OK;
} catch (...) {
  return mpb::set_error(MPB_E_HIP, "moe_head_norm: unexpected exception");
}

size_t moe_head_norm_grad_workspace_bytes(int T, int Hq, int Hk, int D) {
  if (T < 0 || T > (1 << 20) || Hq < 1 || Hq > 1024 || Hk < 0 || Hk > 1024 || D < 16 || D > 512 || D % 16) return 0;
  const size_t b = (size_t)2 * mpb::head_norm_grad_groups(T, Hq, Hk, D) * D * sizeof(float);
  return b < 256 ? 256 : b;
}

int moe_head_norm_grad(const void* q_dev, int64_t q_stride, const void* k_dev, int64_t k_stride, int x_dtype, int T,
                       int Hq, int Hk, int D, const float* gamma_q_dev, const float* gamma_k_dev, float eps,
                       const int32_t* pos_dev, int A, const int32_t* axis_dev, const float* freq_dev, int Dr, int pairs,
                       const void* dq_out_dev, int64_t dq_out_stride, const void* dk_out_dev, int64_t dk_out_stride,
                       void* dq_dev, int64_t dq_stride, void* dk_dev, int64_t dk_stride, float* dgamma_q_dev,
                       float* dgamma_k_dev, void* ws_dev, size_t ws_bytes, void* stream) try {
  const std::string n("moe_head_norm_grad");
  int rc = check_heads(n, x_dtype, T, Hq, Hk, D, eps, pos_dev, A, axis_dev, freq_dev, Dr, pairs);
  if (!rc && !all_aligned16(gamma_q_dev, gamma_k_dev)) rc = fail(MPB_E_ARG, n + ": gammas must be 16-byte aligned");
  if (rc) return rc;
  if (T > 0) {  // an empty batch has no heads to point at
    if (!dq_out_dev || !dq_dev || (gamma_q_dev && !q_dev) ||
        (Hk > 0 && (!dk_out_dev || !dk_dev || (gamma_k_dev && !k_dev))))
      return fail(MPB_E_ARG, n + ": null pointer");
    if ((dgamma_q_dev && !gamma_q_dev) || (dgamma_k_dev && !gamma_k_dev))
      return fail(MPB_E_ARG, n + ": a gradient of gamma needs gamma");
    rc = check_stride(n, "dq_out", dq_out_dev, dq_out_stride, Hq, D);
    if (!rc) rc = check_stride(n, "dq", dq_dev, dq_stride, Hq, D);
    if (!rc && gamma_q_dev) rc = check_stride(n, "q", q_dev, q_stride, Hq, D);
    if (!rc && Hk) rc = check_stride(n, "dk_out", dk_out_dev, dk_out_stride, Hk, D);
    if (!rc && Hk) rc = check_stride(n, "dk", dk_dev, dk_stride, Hk, D);
    if (!rc && Hk && gamma_k_dev) rc = check_stride(n, "k", k_dev, k_stride, Hk, D);
    if (!rc && (dgamma_q_dev || dgamma_k_dev))
      rc = check_ws(n, ws_dev, ws_bytes, moe_head_norm_grad_workspace_bytes(T, Hq, Hk, D));
    if (rc) return rc;
  } else if (!dgamma_q_dev && !dgamma_k_dev) {
    return MPB_OK;
  }
  mpb::HeadNormGradParams p{};
  p.f = mpb::HeadNormParams{q_dev, k_dev, gamma_q_dev, gamma_k_dev, pos_dev, axis_dev, freq_dev, nullptr, nullptr,
                            q_stride, k_stride, dq_out_stride, dk_out_stride, eps, T, Hq, Hk, D, Dr, A, pairs, 1};
  p.dq_out = dq_out_dev; p.dk_out = dk_out_dev;
  p.dq = dq_dev; p.dk = dk_dev; p.dq_ld = dq_stride; p.dk_ld = dk_stride;
  p.dg_q = dgamma_q_dev; p.dg_k = dgamma_k_dev;
  p.part = (float*)ws_dev;
  const hipError_t e = mpb::launch_head_norm_grad(p, x_dtype == MPB_BF16, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, n);
  return MPB_OK;
} catch (...) {
  return mpb::set_error(MPB_E_HIP, "moe_head_norm_grad: unexpected exception");
}

int moe_distill_loss(const void* S_dev, int s_dtype, int64_t s_stride, const int32_t* ids_dev, const float* teacher_dev,
                     const float* teacher_lse_dev, const float* weight_dev, int T, int V, int k, float tau,
                     float* stats_dev, float* kl_dev, float* loss_dev, void* dS_dev, const float* gloss_dev,
                     void* stream) try {
  const std::string n("moe_distill_loss");
  const int rc = check_distill(n, S_dev, s_dtype, s_stride, ids_dev, teacher_dev, T, V, k, tau, stats_dev, dS_dev);
  if (rc) return rc;
  if (!loss_dev || (T > 0 && !kl_dev)) return fail(MPB_E_ARG, n + ": null pointer");
  mpb::DistillParams p{S_dev, ids_dev, teacher_dev, teacher_lse_dev, weight_dev, gloss_dev, stats_dev, kl_dev, loss_dev,
                       dS_dev, s_stride, tau, T, V, k, 0};
  const hipError_t e = mpb::launch_distill(p, s_dtype, true, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, n);
  return MPB_OK;
} catch (...) {
  return mpb::set_error(MPB_E_HIP, "moe_distill_loss: unexpected exception");
}

int moe_distill_loss_grad(const void* S_dev, int s_dtype, int64_t s_stride, const int32_t* ids_dev,
                          const float* teacher_dev, const float* teacher_lse_dev, const float* weight_dev, int T, int V,
                          int k, float tau, const float* stats_dev, void* dS_dev, const float* gloss_dev,
                          void* stream) try {
  const std::string n("moe_distill_loss_grad");
  const int rc = check_distill(n, S_dev, s_dtype, s_stride, ids_dev, teacher_dev, T, V, k, tau, stats_dev, dS_dev);
  if (rc) return rc;
  if (T == 0) return MPB_OK;
  if (!dS_dev) return fail(MPB_E_ARG, n + ": null pointer");
  mpb::DistillParams p{S_dev, ids_dev, teacher_dev, teacher_lse_dev, weight_dev, gloss_dev,
                       const_cast<float*>(stats_dev), nullptr, nullptr, dS_dev, s_stride, tau, T, V, k, 0};
  const hipError_t e = mpb::launch_distill(p, s_dtype, false, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, n);
  return MPB_OK;
} catch (...) {
  return mpb::set_error(MPB_E_HIP, "moe_distill_loss_grad: unexpected exception");
}

}  // extern "C"
