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
  const size_t b = (size_t)2 * mpb::block_norm_grad_groups(T, H) * H * sizeof(float);
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

}  // extern "C"
