// Norms before and after a block, fused with its gate and residual scale, and
// their backward pass.
//
//   rms(v) = 1 / sqrt(mean(v^2) + eps)
//   u = o rms(o) g_post (or o)      what the block adds, normed
//   y = r + s sigmoid(gate) u       the residual stream after the block
//   x = y rms(y) g_next             the next block's normed input
//
// One pass over the rows: a workgroup holds a row in registers (2 vectors of 8
// elements per thread), so every input is read once and every output written
// once; the two means are two workgroup sums. All arithmetic and both sums are
// fp32; y is rounded once for r_out, and x is formed from the unrounded y.
//
// Backward, from y (the stored stream), with d = dx g_next:
//   dy = dr_out + rms(y) (d - yh mean(d yh)),  yh = y rms(y);  dg_next = sum_t dx yh
//   dv = s dy;  dgate = sigmoid'(gate) dv u;  du = sigmoid(gate) dv
//   do = rms(o) (du g_post - oh mean(du g_post oh));  dg_post = sum_t du oh
// The column sums stay in registers over the rows of a workgroup, which writes
// one partial row; k_col_sum adds the partials in workgroup order, so results
// do not depend on timing.
#include "k_block_common.h"
#include "mpb.h"
#include "mpb_internal.h"

namespace mpb {

namespace {

template <class D, int NV>
__global__ __launch_bounds__(1024) void k_block_norm(BlockNormParams p) {
  typedef typename D::vec vec;
  typedef typename D::elem elem;
  __shared__ float buf[2][16];
  const int tid = threadIdx.x, nt = blockDim.x, nvec = p.H / 8;
  const bool post = p.g_post != nullptr, next = p.x != nullptr, added = p.o != nullptr;
  const float inv_h = 1.0f / (float)p.H;
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    const size_t row = (size_t)t * p.H;
    fx8 y[NV], o[NV];
    float ss[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = tid + j * nt;
      y[j] = o[j] = (fx8)(0.0f);
      if (v < nvec) {
        y[j] = widen<D>(*(const vec*)((const elem*)p.r + row + 8 * v));
        if (added) o[j] = load8(p.o + row + 8 * v);
      }
      if (post) {
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] += o[j][i] * o[j][i];
      }
    }
    if (added) {
      float k = p.scale;
      if (p.gate_kind == 1) k *= sigmoid(((const float*)p.gate)[t]);
      if (post) {
        block_sum<1>(ss, buf[0]);
        k *= rsqrtf(ss[0] * inv_h + p.eps);
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int v = tid + j * nt;
        if (v < nvec) {
          fx8 u = o[j] * k;
          if (post) u *= load8(p.g_post + 8 * v);
          if (p.gate_kind == 2) {
            const fx8 g = widen<D>(*(const vec*)((const elem*)p.gate + row + 8 * v));
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] *= sigmoid(g[i]);
          }
          y[j] += u;
          *(vec*)((elem*)p.r_out + row + 8 * v) = narrow<D>(y[j]);
        }
      }
    }
    if (next) {
      ss[0] = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] += y[j][i] * y[j][i];
      }
      block_sum<1>(ss, buf[1]);
      const float ry = rsqrtf(ss[0] * inv_h + p.eps);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int v = tid + j * nt;
        if (v < nvec) *(vec*)((elem*)p.x + row + 8 * v) = narrow<D>(y[j] * ry * load8(p.g_next + 8 * v));
      }
    }
    // buf[0] of this row was read before every thread passed buf[1]'s barrier,
    // and buf[1] before buf[0]'s of the next row; without one of the two sums
    // the other's buffer needs a barrier of its own
    if (post != next) __syncthreads();
  }
}

template <class D, int NV>
__global__ __launch_bounds__(1024) void k_block_norm_grad(BlockNormGradParams p) {
  typedef typename D::vec vec;
  typedef typename D::elem elem;
  __shared__ float buf[2][3 * 16];
  const int tid = threadIdx.x, nt = blockDim.x, nvec = p.H / 8;
  const bool post = p.g_post != nullptr, next = p.dx != nullptr, need_o = p.o != nullptr;
  const float inv_h = 1.0f / (float)p.H;
  fx8 gp[NV], gn[NV];  // column sums of dg_post, dg_next
#pragma unroll
  for (int j = 0; j < NV; ++j) gp[j] = gn[j] = (fx8)(0.0f);
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    const size_t row = (size_t)t * p.H;
    fx8 o[NV], y[NV], d[NV], dy[NV];
    float s1[3] = {0.0f, 0.0f, 0.0f};  // sums of y^2, d y, o^2
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = tid + j * nt;
      o[j] = y[j] = d[j] = dy[j] = (fx8)(0.0f);
      if (v < nvec) {
        if (p.dr_out) dy[j] = widen<D>(*(const vec*)((const elem*)p.dr_out + row + 8 * v));
        if (next) {
          y[j] = widen<D>(*(const vec*)((const elem*)p.y + row + 8 * v));
          d[j] = widen<D>(*(const vec*)((const elem*)p.dx + row + 8 * v));
        }
        if (need_o) o[j] = load8(p.o + row + 8 * v);
        if (next) {
          const fx8 e = d[j] * load8(p.g_next + 8 * v);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            s1[0] += y[j][i] * y[j][i];
            s1[1] += e[i] * y[j][i];
          }
        }
        if (post) {
#pragma unroll
          for (int i = 0; i < 8; ++i) s1[2] += o[j][i] * o[j][i];
        }
      }
    }
    block_sum<3>(s1, buf[0]);
    const float ry = rsqrtf(s1[0] * inv_h + p.eps), ro = post ? rsqrtf(s1[2] * inv_h + p.eps) : 1.0f;
    const float my = s1[1] * ry * inv_h;  // mean(d yh)
    float k = p.scale, dsig = 0.0f;
    if (p.gate_kind == 1) {
      const float g = ((const float*)p.gate)[t], sg = sigmoid(g);
      k *= sg;
      dsig = sigmoid(-g);  // sigmoid' = sigmoid(g) sigmoid(-g)
    }
    float s2[1] = {0.0f};  // sum of du g_post o, and with a token gate of du u
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = tid + j * nt;
      if (v < nvec) {
        if (next) {
          const fx8 yh = y[j] * ry;
          gn[j] += d[j] * yh;
          dy[j] += (d[j] * load8(p.g_next + 8 * v) - yh * my) * ry;
        }
        *(vec*)((elem*)p.dr + row + 8 * v) = narrow<D>(dy[j]);
        fx8 w = (fx8)(1.0f);
        if (post) w = load8(p.g_post + 8 * v);
        fx8 du = dy[j] * k;  // with a token gate's sigmoid
        if (p.gate_kind == 2) {
          const fx8 g = widen<D>(*(const vec*)((const elem*)p.gate + row + 8 * v));
          fx8 dg;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            du[i] *= sigmoid(g[i]);
            dg[i] = du[i] * o[j][i] * ro * w[i] * sigmoid(-g[i]);
          }
          if (p.dgate) *(vec*)((elem*)p.dgate + row + 8 * v) = narrow<D>(dg);
        }
        if (post) gp[j] += du * o[j] * ro;
        dy[j] = du * w;
#pragma unroll
        for (int i = 0; i < 8; ++i) s2[0] += dy[j][i] * o[j][i];
      }
    }
    if (post || p.gate_kind == 1) {
      block_sum<1>(s2, buf[1]);
      if (p.gate_kind == 1 && p.dgate && tid == 0) ((float*)p.dgate)[t] = s2[0] * ro * dsig;
    }
    if (p.d_o) {
      const float mo = post ? s2[0] * ro * inv_h * ro : 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int v = tid + j * nt;
        if (v < nvec) store8(p.d_o + row + 8 * v, post ? (dy[j] - o[j] * mo) * ro : dy[j]);
      }
    }
    if (!(post || p.gate_kind == 1)) __syncthreads();  // buf[0], as in the forward kernel
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int v = tid + j * nt;
    if (v < nvec) {
      if (p.dg_post) store8(p.part + (size_t)blockIdx.x * p.H + 8 * v, gp[j]);
      if (p.dg_next) store8(p.part + (size_t)(gridDim.x + blockIdx.x) * p.H + 8 * v, gn[j]);
    }
  }
}

// dg[h] = sum over n partial rows, 64 columns per workgroup: wave w adds every
// 16th row from w on, then the waves' sums are added in wave order.
__global__ __launch_bounds__(1024) void k_col_sum(const float* part, int n, int H, float* dg0, float* dg1) {
  __shared__ float buf[16][64];
  float* dg = blockIdx.y ? dg1 : dg0;
  if (!dg) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = blockIdx.x * 64 + lane;
  const float* src = part + (size_t)blockIdx.y * n * H + h;
  float s = 0.0f;
  for (int i = wave; i < n; i += 16) s += src[(size_t)i * H];
  buf[wave][lane] = s;
  __syncthreads();
  if (wave == 0) {
    for (int w = 1; w < 16; ++w) s += buf[w][lane];
    dg[h] = s;
  }
}

// Threads of a workgroup: NV vectors each, whole waves.
inline int norm_threads(int H, int nv) { return ((H / 8 + nv - 1) / nv + 63) / 64 * 64; }

}  // namespace

hipError_t launch_block_norm(const BlockNormParams& p, bool bf16, hipStream_t s) {
  const int grid = p.T < 4096 ? p.T : 4096;
  if (p.H <= 16384) {
    const int nt = norm_threads(p.H, 2);
    if (bf16) k_block_norm<BF16, 2><<<grid, nt, 0, s>>>(p);
    else k_block_norm<F16, 2><<<grid, nt, 0, s>>>(p);
  } else {
    const int nt = norm_threads(p.H, 8);
    if (bf16) k_block_norm<BF16, 8><<<grid, nt, 0, s>>>(p);
    else k_block_norm<F16, 8><<<grid, nt, 0, s>>>(p);
  }
  return hipGetLastError();
}

int block_norm_grad_groups(int T, int H) {
  const int most = 512;
  (void)H;
  return T < most ? T : most;
}

hipError_t launch_block_norm_grad(const BlockNormGradParams& p, bool bf16, hipStream_t s) {
  const int grid = block_norm_grad_groups(p.T, p.H);
  if (grid) {
    if (p.H <= 16384) {
      const int nt = norm_threads(p.H, 2);
      if (bf16) k_block_norm_grad<BF16, 2><<<grid, nt, 0, s>>>(p);
      else k_block_norm_grad<F16, 2><<<grid, nt, 0, s>>>(p);
    } else {
      const int nt = norm_threads(p.H, 8);
      if (bf16) k_block_norm_grad<BF16, 8><<<grid, nt, 0, s>>>(p);
      else k_block_norm_grad<F16, 8><<<grid, nt, 0, s>>>(p);
    }
  }
  if (p.dg_post || p.dg_next) k_col_sum<<<dim3(p.H / 64, 2), 1024, 0, s>>>(p.part, grid, p.H, p.dg_post, p.dg_next);
  return hipGetLastError();
}

}  // namespace mpb
