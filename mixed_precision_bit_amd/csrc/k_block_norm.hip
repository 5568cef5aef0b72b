// Norms before and after a block, fused with its gate and residual scale, and
// their backward pass.
//
//   rms(v) = 1 / sqrt(mean(v^2) + eps)
//   u = o rms(o) g_post (or o)      what the block adds, normed
//   y = r + s sigmoid(gate) u       the residual stream after the block
//   x = y rms(y) g_next             the next block's normed input
//
// One pass over the rows: a workgroup holds a row in registers (vectors of 8
// elements, one or two per thread), so every input is read once and every output written
// once; the two means are two workgroup sums. All arithmetic and both sums are
// fp32; y is rounded once for r_out, and x is formed from the unrounded y.
// Bound by HBM: 4096 x 2816 bf16 with a full gate takes 31.7 us a call among others
// (33 by itself under a trace), 4.37 TB/s of the 4.9 TB/s that a large copy reaches; up
// to some hundred rows the launch itself (3.1 us for one row of 2048). Times below
// are traced ones.
//
// Backward, from y (the stored stream), with d = dx g_next:
//   dy = dr_out + rms(y) (d - yh mean(d yh)),  yh = y rms(y);  dg_next = sum_t dx yh
//   dv = s dy;  dgate = sigmoid'(gate) dv u;  du = sigmoid(gate) dv
//   do = rms(o) (du g_post - oh mean(du g_post oh));  dg_post = sum_t du oh
// The column sums stay in registers over the rows of a workgroup, which writes
// one partial row; k_col_sum adds the partials in workgroup order, so results
// do not depend on timing. 4093 x 2816 takes 50 + 4.7 us (3.7 TB/s: eight rows a
// workgroup leave a ramp at both ends), 8192 x 4096 with a full gate 144 + 4.8
// (4.7 TB/s).
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

// One row of the backward pass's inputs as loaded.
template <class D, int NV>
struct GradRow {
  fx8 o[NV];
  typename D::vec y[NV], dx[NV], dr[NV], gate[NV];

  __device__ __forceinline__ void load(const BlockNormGradParams& p, int t) {
    typedef typename D::vec vec;
    typedef typename D::elem elem;
    const size_t row = (size_t)t * p.H;
    const int nvec = p.H / 8;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = threadIdx.x + j * blockDim.x;
      o[j] = (fx8)(0.0f);
      y[j] = dx[j] = dr[j] = gate[j] = (vec)(typename D::elem)0.0f;
      if (v < nvec) {
        const size_t at = row + 8 * v;
        if (p.dx) {
          y[j] = *(const vec*)((const elem*)p.y + at);
          dx[j] = *(const vec*)((const elem*)p.dx + at);
        }
        if (p.o) o[j] = load8(p.o + at);
        if (p.dr_out) dr[j] = *(const vec*)((const elem*)p.dr_out + at);
        if (p.gate_kind == 2) gate[j] = *(const vec*)((const elem*)p.gate + at);
      }
    }
  }
};

// THREADS: most threads a launch may have. AHEAD: a row's loads are issued
// before the row before it is worked on, so that memory stays busy through the
// two workgroup sums.
template <class D, int NV, int THREADS, bool AHEAD>
__global__ __launch_bounds__(THREADS) void k_block_norm_grad(BlockNormGradParams p) {
  typedef typename D::vec vec;
  typedef typename D::elem elem;
  __shared__ float buf[2][3 * 16];
  const int tid = threadIdx.x, nt = blockDim.x, nvec = p.H / 8;
  const bool post = p.g_post != nullptr, next = p.dx != nullptr;
  const float inv_h = 1.0f / (float)p.H;
  fx8 gp[NV], gn[NV];  // column sums of dg_post, dg_next
#pragma unroll
  for (int j = 0; j < NV; ++j) gp[j] = gn[j] = (fx8)(0.0f);
  const auto work = [&](int t, const GradRow<D, NV>& in) {
    const size_t row = (size_t)t * p.H;
    float s1[3] = {0.0f, 0.0f, 0.0f};  // sums of y^2, d y, o^2
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = tid + j * nt;
      if (next && v < nvec) {
        const fx8 y = widen<D>(in.y[j]), e = widen<D>(in.dx[j]) * load8(p.g_next + 8 * v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s1[0] += y[i] * y[i];
          s1[1] += e[i] * y[i];
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) s1[2] += in.o[j][i] * in.o[j][i];
    }
    block_sum<3>(s1, buf[0]);
    const float ry = rsqrtf(s1[0] * inv_h + p.eps), ro = post ? rsqrtf(s1[2] * inv_h + p.eps) : 1.0f;
    const float my = s1[1] * ry * inv_h;  // mean(d yh)
    float k = p.scale, dsig = 0.0f;
    if (p.gate_kind == 1) {
      const float g = ((const float*)p.gate)[t];
      k *= sigmoid(g);
      dsig = sigmoid(-g);  // sigmoid' = sigmoid(g) sigmoid(-g)
    }
    float s2[1] = {0.0f};  // sum of du g_post o (with a token gate also that of dv u, but for factors)
    fx8 dw[NV];            // du g_post
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = tid + j * nt;
      dw[j] = (fx8)(0.0f);
      if (v < nvec) {
        fx8 dy = widen<D>(in.dr[j]);
        if (next) {
          const fx8 yh = widen<D>(in.y[j]) * ry, d = widen<D>(in.dx[j]);
          gn[j] += d * yh;
          dy += (d * load8(p.g_next + 8 * v) - yh * my) * ry;
        }
        stream_store((vec*)((elem*)p.dr + row + 8 * v), narrow<D>(dy));
        fx8 w = (fx8)(1.0f);
        if (post) w = load8(p.g_post + 8 * v);
        fx8 du = dy * k;  // with a token gate's sigmoid
        if (p.gate_kind == 2) {
          const fx8 g = widen<D>(in.gate[j]);
          fx8 dg;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            du[i] *= sigmoid(g[i]);
            dg[i] = du[i] * in.o[j][i] * ro * w[i] * sigmoid(-g[i]);
          }
          if (p.dgate) stream_store((vec*)((elem*)p.dgate + row + 8 * v), narrow<D>(dg));
        }
        if (post) gp[j] += du * in.o[j] * ro;
        dw[j] = du * w;
#pragma unroll
        for (int i = 0; i < 8; ++i) s2[0] += dw[j][i] * in.o[j][i];
      }
    }
    if (post || p.gate_kind == 1) {
      block_sum<1>(s2, buf[1]);
      if (p.gate_kind == 1 && p.dgate && tid == 0) ((float*)p.dgate)[t] = s2[0] * ro * dsig;
    } else {
      __syncthreads();  // buf[0] is free again, as in the forward kernel
    }
    if (p.d_o) {
      const float mo = post ? s2[0] * ro * inv_h * ro : 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int v = tid + j * nt;
        if (v < nvec) stream_store8(p.d_o + row + 8 * v, post ? (dw[j] - in.o[j] * mo) * ro : dw[j]);
      }
    }
  };
  GradRow<D, NV> in;
  if (AHEAD) {
    // two register sets in turn (a copy from one to the other would wait for the
    // row's stores as well); past the last row the last one is loaded again
    GradRow<D, NV> in2;
    const int step = gridDim.x, last = blockIdx.x + (p.T - 1 - blockIdx.x) / step * step;
    in.load(p, blockIdx.x);
    for (int t = blockIdx.x;; t += 2 * step) {
      in2.load(p, t + step < last ? t + step : last);
      work(t, in);
      if (t + step > last) break;
      in.load(p, t + 2 * step < last ? t + 2 * step : last);
      work(t + step, in2);
      if (t + 2 * step > last) break;
    }
  } else {
    for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
      in.load(p, t);
      work(t, in);
    }
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
  int i = wave;
  for (; i + 7 * 16 < n; i += 8 * 16) {  // eight loads in flight
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = src[(size_t)(i + 16 * j) * H];
#pragma unroll
    for (int j = 0; j < 8; ++j) s += v[j];
  }
  for (; i < n; i += 16) s += src[(size_t)i * H];
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

// One vector a thread up to H = 4096 (one row of 2048: 3.1 us against 3.5 with
// two; 4096 x 2816: 33.0 against 33.2), then two; past 16384 the eight vectors a
// thread spill 75 registers, which only such rows pay.
template <class D>
static void norm_rows(const BlockNormParams& p, hipStream_t s) {
  const int grid = p.T < 4096 ? p.T : 4096;
  if (p.H <= 4096) k_block_norm<D, 1><<<grid, norm_threads(p.H, 1), 0, s>>>(p);
  else if (p.H <= 16384) k_block_norm<D, 2><<<grid, norm_threads(p.H, 2), 0, s>>>(p);
  else k_block_norm<D, 8><<<grid, norm_threads(p.H, 8), 0, s>>>(p);
}

hipError_t launch_block_norm(const BlockNormParams& p, bool bf16, hipStream_t s) {
  if (bf16) norm_rows<BF16>(p, s);
  else norm_rows<F16>(p, s);
  return hipGetLastError();
}

// Two workgroups a CU (512): more would add partial rows of 8 H bytes each, and
// take turns on the CUs (4093 x 2816: 55 us in all against 63 with 768, 58 with 1024;
// 8192 x 4096 with a full gate 148 against 158, 154).
int block_norm_grad_groups(int T) { return T < 512 ? T : 512; }

// Two vectors a thread; rows past 8192 elements leave no registers for a second
// row and spill 10 to 13 of them, and past 16384 the eight vectors a thread spill
// some 590, which only such rows pay.
template <class D>
static void grad_rows(const BlockNormGradParams& p, int grid, hipStream_t s) {
  if (p.H <= 8192) k_block_norm_grad<D, 2, 512, true><<<grid, norm_threads(p.H, 2), 0, s>>>(p);
  else if (p.H <= 16384) k_block_norm_grad<D, 2, 1024, false><<<grid, norm_threads(p.H, 2), 0, s>>>(p);
  else k_block_norm_grad<D, 8, 1024, false><<<grid, norm_threads(p.H, 8), 0, s>>>(p);
}

hipError_t launch_block_norm_grad(const BlockNormGradParams& p, bool bf16, hipStream_t s) {
  const int grid = block_norm_grad_groups(p.T);
  if (grid) {
    if (bf16) grad_rows<BF16>(p, grid, s);
    else grad_rows<F16>(p, grid, s);
  }
  if (p.dg_post || p.dg_next) k_col_sum<<<dim3(p.H / 64, 2), 1024, 0, s>>>(p.part, grid, p.H, p.dg_post, p.dg_next);
  return hipGetLastError();
}

}  // namespace mpb
