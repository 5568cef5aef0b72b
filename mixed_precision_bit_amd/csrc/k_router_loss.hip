// Router losses and their gradients.
//
// Forward, over the live tokens (mask != 0 and some logit above -inf):
//   l = X W^T + bias, lse = log sum_e exp l, p = exp(l - lse)
//   c_e = live (token, slot) pairs with expert e, N = live tokens, P_e = sum_t p_te
//   balance = E / (K N^2) sum_e c_e P_e,  z = 1/N sum_t lse^2
//   loss = alpha balance + beta z
// Backward (c_e taken as a constant):
//   dl_te = g p_te (alpha E / N (f_e - sum_j f_j p_tj) + 2 beta / N lse_t),  f_e = c_e / (K N)
//         + sum over slots k with expert e of w_k (gw_k - sum_j w_j gw_j)
//   dX = dl W, dW = dl^T X, dbias = sum_t dl
//
// The three T x E x H products run on the bf16 matrix cores at fp32 accuracy:
// an fp32 operand is cut into three bf16 parts (8 bits each, 24 together, by
// truncation: exact, and no part overflows), an fp16 activation into two, a
// bf16 one is its own part; products of parts are exact in fp32 and accumulate
// in fp32, and only products below 2^-24 of the whole are left out. Against
// the fp32 matrix instructions (1/16 of the bf16 rate) three to six bf16
// products are still 2.5 to 5 times cheaper.
#include "k_block_common.h"
#include "mpb.h"
#include "mpb_internal.h"

namespace mpb {

namespace {

__device__ __forceinline__ bool is_live(const RouterLossParams& p, int t) {
  return t < p.T && (!p.mask || p.mask[t]);
}

// Whether token t takes part in the loss, after the forward pass.
__device__ __forceinline__ bool is_on(const RouterLossParams& p, int t) {
  return is_live(p, t) && !(p.lse[t] == -INFINITY);
}

// ---------------------------------------------------------------- logits
// 64 tokens x 64 experts x one range of H per workgroup of 4 waves; a wave
// holds 16 experts, whose W it reads straight into fragments and cuts there
// (each W value is read by one wave of the workgroup); the tokens' activations
// are staged in LDS for all four waves, 64 elements of H at a time, the next
// stage's loads in flight during the products. Partial sums go to
// part[range][T][E].
constexpr int kLT = 64, kLE = 64, kLK = 64, kLRow = kLK + 8;  // 16 bytes of padding per LDS row

template <class D>
__global__ __launch_bounds__(256) void k_router_logits(RouterLossParams p) {
  typedef typename D::vec vec;
  typedef typename D::elem elem;
  constexpr int NP = Parts<D>::N;
  __shared__ __align__(16) __bf16 xs[2][NP][kLT * kLRow];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, g = lane >> 4;
  const int t0 = blockIdx.x * kLT, e = blockIdx.y * kLE + wave * 16 + n;
  const int steps = p.H / kLK, s0 = (int)((long long)steps * blockIdx.z / gridDim.z),
            s1 = (int)((long long)steps * (blockIdx.z + 1) / gridDim.z);
  const float* wrow = p.W + (size_t)(e < p.E ? e : 0) * p.H + 8 * g;
  // a thread stages two vectors: rows tid/8 and tid/8 + 32, columns 8 (tid % 8)
  const int r0 = tid >> 3, c0 = (tid & 7) * 8;
  const bool live[2] = {is_live(p, t0 + r0), is_live(p, t0 + r0 + 32)};
  const elem* xrow[2] = {(const elem*)p.X + (size_t)(t0 + r0) * p.H + c0,
                         (const elem*)p.X + (size_t)(t0 + r0 + 32) * p.H + c0};
  vec xv[2];
  fx8 wv[2];
  auto load = [&](int s) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      xv[i] = (vec)(elem)0.0f;
      if (live[i]) xv[i] = *(const vec*)(xrow[i] + s * kLK);
      wv[i] = (fx8)(0.0f);
      if (e < p.E) wv[i] = load8(wrow + s * kLK + 32 * i);
    }
  };
  auto stage = [&](int b) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      bx8 q[NP];
      Parts<D>::of(xv[i], q);
#pragma unroll
      for (int k = 0; k < NP; ++k) *(bx8*)&xs[b][k][(r0 + 32 * i) * kLRow + c0] = q[k];
    }
  };
  acc4 acc[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) acc[m] = (acc4)(0.0f);
  load(s0);
  for (int s = s0; s < s1; ++s) {
    const int b = (s - s0) & 1;
    stage(b);
    bx8 w[2][3];
    cut<3>(wv[0], w[0]);
    cut<3>(wv[1], w[1]);
    if (s + 1 < s1) load(s + 1);
    __syncthreads();  // xs[b] is written; the other half was read before the barrier of the step before
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
#pragma unroll
        for (int k = NP - 1; k >= 0; --k) {
          const bx8 x = *(const bx8*)&xs[b][k][(16 * m + n) * kLRow + 32 * i + 8 * g];
#pragma unroll
          for (int j = 2 - k; j >= 0; --j) acc[m] = mfma(x, w[i][j], acc[m]);  // smallest parts first
        }
      }
    }
  }
  if (e < p.E) {
    float* out = p.part + (size_t)blockIdx.z * p.T * p.E + e;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = t0 + 16 * m + 4 * g + r;
        if (t < p.T) out[(size_t)t * p.E] = acc[m][r];
      }
    }
  }
}

// ---------------------------------------------------------------- softmax, counts
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 32; m; m >>= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}

constexpr int kEJ = 8;  // experts of a lane: e = lane + 64 j, E <= 512

// One wave per token: adds the ranges of H, writes logits and lse, and keeps
// its share of P_e, z and N in registers; a workgroup (8 waves) writes one row
// of each to stat_f [groups][E + 1] and stat_i [groups][E + 1].
template <int EJ>
__global__ __launch_bounds__(512) void k_router_stats(RouterLossParams p) {
  __shared__ int cnt[513];
  __shared__ float pr[8][513];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = p.E;
  for (int i = tid; i <= E; i += 512) cnt[i] = 0;
  __syncthreads();
  float psum[EJ], z = 0.0f;
#pragma unroll
  for (int j = 0; j < EJ; ++j) psum[j] = 0.0f;
  for (int t = blockIdx.x * 8 + wave; t < p.T; t += gridDim.x * 8) {
    const bool on = is_live(p, t);
    float l[EJ], m = -INFINITY;
#pragma unroll
    for (int j = 0; j < EJ; ++j) {
      const int e = lane + 64 * j;
      l[j] = -INFINITY;
      if (e < E) {
        float v = 0.0f;
        if (on) {
          const float* src = p.part + (size_t)t * E + e;
          for (int s = 0; s < p.splits; ++s) v += src[(size_t)s * p.T * E];
          if (p.bias) v += p.bias[e];
        }
        p.logits[(size_t)t * E + e] = v;
        l[j] = v;
        m = fmaxf(m, v);
      }
    }
    if (!on) {
      if (lane == 0) p.lse[t] = 0.0f;
      continue;
    }
    m = wave_max(m);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < EJ; ++j)
      if (lane + 64 * j < E) s += expf(l[j] - m);
    s = wave_sum(s);
    const float lse = m == -INFINITY && !(s == s && s > 0.0f) ? -INFINITY : m + logf(s);
    bool nan = false;  // fmaxf drops nan: the row's own values decide
#pragma unroll
    for (int j = 0; j < EJ; ++j) nan |= l[j] != l[j];
    const bool any_nan = __ballot(nan) != 0;
    const float out = any_nan ? NAN : lse;
    if (lane == 0) p.lse[t] = out;
    if (out == -INFINITY) continue;  // no expert left: the token does not count
    z += out * out;
#pragma unroll
    for (int j = 0; j < EJ; ++j)
      if (lane + 64 * j < E) psum[j] += expf(l[j] - out);
    if (lane < p.K) {
      const int id = p.idx[(size_t)t * p.K + lane];
      if (id >= 0 && id < E) atomicAdd(&cnt[id], 1);
    }
    if (lane == 0) atomicAdd(&cnt[E], 1);
  }
#pragma unroll
  for (int j = 0; j < EJ; ++j)
    if (lane + 64 * j < E) pr[wave][lane + 64 * j] = psum[j];
  if (lane == 0) pr[wave][E] = z;
  __syncthreads();
  for (int i = tid; i <= E; i += 512) {
    float s = pr[0][i];
    for (int w = 1; w < 8; ++w) s += pr[w][i];
    p.stat_f[(size_t)blockIdx.x * (E + 1) + i] = s;
    p.stat_i[(size_t)blockIdx.x * (E + 1) + i] = cnt[i];
  }
}

// Adds the groups' rows (fp64, group order per slice, slices in order) and
// forms the losses. One workgroup.
__global__ __launch_bounds__(1024) void k_router_finish(RouterLossParams p) {
  __shared__ double fs[1024];
  __shared__ int is[1024];
  __shared__ double zsum;
  __shared__ int nlive;
  const int tid = threadIdx.x, E = p.E, W = E + 1;
  double part = 0.0;
  // columns of 64, 16 slices of the groups each
  for (int c0 = 0; c0 < W; c0 += 64) {
    const int c = c0 + (tid & 63), sl = tid >> 6;
    double f = 0.0;
    int n = 0;
    if (c < W) {
      for (int i = sl; i < p.groups; i += 16) {
        f += (double)p.stat_f[(size_t)i * W + c];
        n += p.stat_i[(size_t)i * W + c];
      }
    }
    fs[tid] = f;
    is[tid] = n;
    __syncthreads();
    if (tid < 64 && c < W) {
      for (int k = 1; k < 16; ++k) {
        f += fs[tid + 64 * k];
        n += is[tid + 64 * k];
      }
      p.counts[c] = n;
      if (c < E) {
        p.prob[c] = (float)f;
        part += f * (double)n;
      } else {
        zsum = f;
        nlive = n;
      }
    }
    __syncthreads();
  }
  if (tid < 64) {
#pragma unroll
    for (int m = 32; m; m >>= 1) part += __shfl_xor(part, m);
  }
  if (tid == 0) {
    const double N = nlive > 0 ? (double)nlive : 1.0;
    const double bal = (double)E * part / ((double)p.K * N * N), z = zsum / N;
    p.loss[0] = (float)((double)p.alpha * bal + (double)p.beta * z);
    p.loss[1] = (float)bal;
    p.loss[2] = (float)z;
  }
}

// ---------------------------------------------------------------- gradients
// Operand fragments of the two gradient products, in the order that a wave's
// lanes read them (16 bytes a lane, 1 KiB a fragment):
//   dl_a [part][token / 16][expert / 32]   lane (n, g): token n, experts 8g..8g+7
//   dl_t [part][expert / 16][token / 32]   lane (n, g): expert n, tokens 8g..8g+7
//   w_t  [part][h / 16][expert / 32]       lane (n, g): column n, experts 8g..8g+7
__device__ __forceinline__ size_t frag(size_t tiles, size_t part, size_t tile) { return (part * tiles + tile) * 512; }

// Workgroups 0 .. Tp/32 - 1: dl of 32 tokens, one wave per 4 of them, held in
// LDS and written as both operands. The rest: w_t of 32 experts x 64 columns.
__global__ __launch_bounds__(512) void k_router_dl(RouterLossParams p) {
  extern __shared__ __align__(16) float ds[];  // [32][Ep + 4], or [32][68]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, g = lane >> 4;
  const int E = p.E, Ep = p.Ep;
  const int tok_wgs = p.Tp / 32;
  if ((int)blockIdx.x >= tok_wgs) {
    const int b = blockIdx.x - tok_wgs, e0 = 32 * (b % (Ep / 32)), h0 = 64 * (b / (Ep / 32));
    const int r = tid >> 4, c = (tid & 15) * 4;
    fx4 v = (fx4)(0.0f);
    if (e0 + r < E) v = *(const fx4*)(p.W + (size_t)(e0 + r) * p.H + h0 + c);
    *(fx4*)(ds + r * 68 + c) = v;
    __syncthreads();
    if (wave < 4) {
      fx8 x;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = ds[(8 * g + i) * 68 + 16 * wave + n];
      bx8 q[3];
      cut<3>(x, q);
      const size_t tiles = (size_t)(p.H / 16) * (Ep / 32), tile = (size_t)(h0 / 16 + wave) * (Ep / 32) + e0 / 32;
#pragma unroll
      for (int k = 0; k < 3; ++k) *(bx8*)(p.w_t + frag(tiles, k, tile) + 8 * lane) = q[k];
    }
    return;
  }
  const int t0 = blockIdx.x * 32, row = Ep + 4;
  const int N = p.counts[E];
  const float gl = p.gloss ? *p.gloss : 1.0f, inv_n = N > 0 ? 1.0f / (float)N : 0.0f;
  const float ca = gl * p.alpha * (float)E * inv_n, cb = gl * 2.0f * p.beta * inv_n, cf = inv_n / (float)p.K;
  for (int i = 0; i < 4; ++i) {
    const int r = wave * 4 + i, t = t0 + r;
    const float lse = is_live(p, t) ? p.lse[t] : -INFINITY;
    const bool on = !(lse == -INFINITY);  // nan stays on and spreads
    float pr[kEJ], dot = 0.0f;
#pragma unroll
    for (int j = 0; j < kEJ; ++j) {
      const int e = lane + 64 * j;
      pr[j] = 0.0f;
      if (e < E && on) {
        pr[j] = expf(p.logits[(size_t)t * E + e] - lse);
        dot += (float)p.counts[e] * cf * pr[j];
      }
    }
    dot = wave_sum(dot);
    float c = 0.0f;
    int id = -1;
    if (on && p.gw) {
      float l = -INFINITY, gw = 0.0f;
      if (lane < p.K) {
        id = p.idx[(size_t)t * p.K + lane];
        if (id < 0 || id >= E) id = -1;
        if (id >= 0) {
          l = p.logits[(size_t)t * E + id];
          gw = p.gw[(size_t)t * p.K + lane];
        }
      }
      const float m = wave_max(l);
      const float x = id >= 0 && m > -INFINITY ? expf(l - m) : 0.0f;
      const float s = wave_sum(x), w = s > 0.0f ? x / s : x;
      const float mean = wave_sum(id >= 0 ? w * gw : 0.0f);
      c = id >= 0 ? w * (gw - mean) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < kEJ; ++j) {
      const int e = lane + 64 * j;
      if (e < Ep) {
        float d = 0.0f;
        if (e < E && on) d = pr[j] * (ca * ((float)p.counts[e] * cf - dot) + cb * lse);
        if (p.gw) {
          for (int k = 0; k < p.K; ++k) {  // slots in order, also where one expert is named twice
            const int ik = __shfl(id, k);
            const float ck = __shfl(c, k);
            if (ik == e) d += ck;
          }
        }
        ds[r * row + e] = d;
      }
    }
  }
  __syncthreads();
  const int kt = Ep / 32;
  const size_t ta = (size_t)(p.Tp / 16) * kt, tt = (size_t)(Ep / 16) * (p.Tp / 32);
  for (int f = wave; f < 2 * kt; f += 8) {  // dl_a: 2 token tiles x kt expert tiles
    const int m = f & 1, k32 = f >> 1;
    const fx8 x = load8(ds + (16 * m + n) * row + 32 * k32 + 8 * g);
    bx8 q[3];
    cut<3>(x, q);
#pragma unroll
    for (int k = 0; k < 3; ++k)
      *(bx8*)(p.dl_a + frag(ta, k, (size_t)(t0 / 16 + m) * kt + k32) + 8 * lane) = q[k];
  }
  for (int f = wave; f < Ep / 16; f += 8) {  // dl_t: Ep / 16 expert tiles
    fx8 x;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = ds[(8 * g + i) * row + 16 * f + n];
    bx8 q[3];
    cut<3>(x, q);
#pragma unroll
    for (int k = 0; k < 3; ++k)
      *(bx8*)(p.dl_t + frag(tt, k, (size_t)f * (p.Tp / 32) + t0 / 32) + 8 * lane) = q[k];
  }
  for (int e = tid; e < E; e += 512) {
    float s = 0.0f;
    for (int r = 0; r < 32; ++r) s += ds[r * row + e];
    p.db_part[(size_t)blockIdx.x * E + e] = s;
  }
}

// dX = dl W: a wave holds 64 tokens x 64 columns, a workgroup 128 x 128. The
// columns are the products' rows, so that a lane ends with four of a token's
// consecutive columns.
__global__ __launch_bounds__(256) void k_router_dx(RouterLossParams p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
  const int kt = p.Ep / 32;
  const int t0 = blockIdx.x * 128 + (wave & 1) * 64, h0 = blockIdx.y * 128 + (wave >> 1) * 64;
  if (t0 >= p.Tp || h0 >= p.H) return;
  const size_t ta = (size_t)(p.Tp / 16) * kt, tw = (size_t)(p.H / 16) * kt;
  acc4 acc[4][4];
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[m][c] = (acc4)(0.0f);
  for (int k = 0; k < kt; ++k) {
    bx8 a[4][3], b[4][3];
#pragma unroll
    for (int q = 0; q < 3; ++q) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        a[m][q] = *(const bx8*)(p.dl_a + frag(ta, q, (size_t)(t0 / 16 + m) * kt + k) + 8 * lane);
        b[m][q] = *(const bx8*)(p.w_t + frag(tw, q, (size_t)(h0 / 16 + m) * kt + k) + 8 * lane);
      }
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int s = 2; s >= 0; --s) {  // parts i, j with i + j = s: the smallest first
#pragma unroll
          for (int i = s; i >= 0; --i) acc[m][c] = mfma(b[c][s - i], a[m][i], acc[m][c]);
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int t = t0 + 16 * m + n;
    if (t < p.T) {
      const bool on = is_on(p, t);
      float* out = p.dX + (size_t)t * p.H + h0 + 4 * g;
#pragma unroll
      for (int c = 0; c < 4; ++c) *(acc4*)(out + 16 * c) = on ? acc[m][c] : (acc4)(0.0f);
    }
  }
}

// dW = dl^T X: a workgroup holds 64 experts x 128 columns over one range of
// tokens, its four waves taking 32 tokens in turn. A lane loads 8 tokens x 8
// columns of X and turns them round in registers, which gives the 8 column
// fragments of a step (fragment j: columns 8 n + j). The waves' sums meet in
// LDS in wave order.
template <class D>
__global__ __launch_bounds__(256, 2) void k_router_dw(RouterLossParams p) {
  typedef typename D::vec vec;
  typedef typename D::elem elem;
  constexpr int NP = Parts<D>::N;
  __shared__ __align__(16) float sum[64][128 + 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, g = lane >> 4;
  const int e0 = blockIdx.x * 64, h = blockIdx.y * 128 + 8 * n;
  const int nt = p.Tp / 32;
  const int b0 = (int)((long long)nt * blockIdx.z / gridDim.z), b1 = (int)((long long)nt * (blockIdx.z + 1) / gridDim.z);
  const size_t tt = (size_t)(p.Ep / 16) * nt;
  acc4 acc[4][8];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[a][j] = (acc4)(0.0f);
  for (int b = b0 + wave; b < b1; b += 4) {
    vec x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = 32 * b + 8 * g + i;
      x[i] = (vec)(elem)0.0f;
      if (h < p.H && is_on(p, t)) x[i] = *(const vec*)((const elem*)p.X + (size_t)t * p.H + h);
    }
    bx8 a[4][3];
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int q = 0; q < 3; ++q)
        a[m][q] = *(const bx8*)(p.dl_t + frag(tt, q, (size_t)(e0 / 16 + m) * nt + b) + 8 * lane);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      vec c;
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = x[i][j];
      bx8 q[NP];
      Parts<D>::of(c, q);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
#pragma unroll
        for (int k = NP - 1; k >= 0; --k)
#pragma unroll
          for (int i = 2 - k; i >= 0; --i) acc[m][j] = mfma(a[m][i], q[k], acc[m][j]);
      }
    }
  }
  for (int w = 0; w < 4; ++w) {
    if (wave == w) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          fx8 v;
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = acc[m][j][r];
          float* at = &sum[16 * m + 4 * g + r][8 * n];
          if (w) v += load8(at);
          store8(at, v);
        }
      }
    }
    __syncthreads();
  }
  float* out = p.dw_part + (size_t)blockIdx.z * p.E * p.H;
  for (int i = tid; i < 64 * 16; i += 256) {
    const int e = i >> 4, c = (i & 15) * 8, col = blockIdx.y * 128 + c;
    if (e0 + e < p.E && col < p.H) store8(out + (size_t)(e0 + e) * p.H + col, load8(&sum[e][c]));
  }
}

// Adds the token ranges of dW (workgroups below `dw_wgs`, 4 values a thread)
// and the token tiles of dbias (64 experts a workgroup, 16 slices).
__global__ __launch_bounds__(1024) void k_router_add(RouterLossParams p, int dw_wgs) {
  __shared__ double buf[1024];
  const int tid = threadIdx.x;
  if ((int)blockIdx.x < dw_wgs) {
    const size_t n = (size_t)p.E * p.H, i = ((size_t)blockIdx.x * 1024 + tid) * 4;
    if (i >= n) return;
    fx4 s = (fx4)(0.0f);
    for (int c = 0; c < p.chunks; ++c) s += *(const fx4*)(p.dw_part + (size_t)c * n + i);
    *(fx4*)(p.dW + i) = s;
    return;
  }
  const int e = (blockIdx.x - dw_wgs) * 64 + (tid & 63);
  double s = 0.0;
  if (e < p.E)
    for (int i = tid >> 6; i < p.Tp / 32; i += 16) s += (double)p.db_part[(size_t)i * p.E + e];
  buf[tid] = s;
  __syncthreads();
  if (tid < 64 && e < p.E) {
    for (int k = 1; k < 16; ++k) s += buf[tid + 64 * k];
    p.dbias[e] = (float)s;
  }
}

}  // namespace

static size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

RouterLossWs router_loss_ws(int T, int H, int E) {
  RouterLossWs w{};
  const int tiles = ((T + kLT - 1) / kLT) * ((E + kLE - 1) / kLE);
  // ranges of H for the logits: about 512 workgroups, whole stages of 64
  w.splits = tiles > 0 ? 512 / tiles : 1;
  if (w.splits > 32) w.splits = 32;
  if (w.splits > H / kLK) w.splits = H / kLK;
  if (w.splits < 1) w.splits = 1;
  w.groups = (T + 15) / 16 < 256 ? (T + 15) / 16 : 256;
  if (w.groups < 1) w.groups = 1;
  size_t off = 0;
  w.part = off;   off += up256((size_t)w.splits * T * E * 4);
  w.stat_f = off; off += up256((size_t)w.groups * (E + 1) * 4);
  w.stat_i = off; off += up256((size_t)w.groups * (E + 1) * 4);
  const size_t fwd = off;
  w.Tp = (T + 63) / 64 * 64;
  w.Ep = (E + 63) / 64 * 64;
  const int wt = (w.Ep / 64) * ((H + 127) / 128), nt = w.Tp / 32;
  // ranges of tokens for dW: about 512 workgroups, at least 8 tiles of 32 tokens each
  w.chunks = 512 / wt;
  if (w.chunks > nt / 8) w.chunks = nt / 8;
  if (w.chunks < 1) w.chunks = 1;
  off = 0;
  w.dl_a = off;    off += up256((size_t)3 * w.Tp * w.Ep * 2);
  w.dl_t = off;    off += up256((size_t)3 * w.Tp * w.Ep * 2);
  w.w_t = off;     off += up256((size_t)3 * H * w.Ep * 2);
  w.db_part = off; off += up256((size_t)(w.Tp / 32) * E * 4);
  w.dw_part = off; off += up256((size_t)w.chunks * E * H * 4);
  w.total = fwd > off ? fwd : off;
  return w;
}

hipError_t launch_router_loss(const RouterLossParams& p, bool bf16, hipStream_t s) {
  if (p.T > 0) {
    const dim3 grid((p.T + kLT - 1) / kLT, (p.E + kLE - 1) / kLE, p.splits);
    if (bf16) k_router_logits<BF16><<<grid, 256, 0, s>>>(p);
    else k_router_logits<F16><<<grid, 256, 0, s>>>(p);
  }
  if (p.E <= 64) k_router_stats<1><<<p.groups, 512, 0, s>>>(p);
  else if (p.E <= 128) k_router_stats<2><<<p.groups, 512, 0, s>>>(p);
  else k_router_stats<8><<<p.groups, 512, 0, s>>>(p);
  k_router_finish<<<1, 1024, 0, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_router_loss_grad(const RouterLossParams& p, bool bf16, hipStream_t s) {
  static unsigned long long raised = 0;
  const int lds = 32 * (p.Ep + 4) * 4;
  if (lds > 64 * 1024) {
    const hipError_t e = raise_lds_limit((const void*)k_router_dl, 32 * (512 + 4) * 4, raised);
    if (e != hipSuccess) return e;
  }
  const int w_wgs = p.dX ? (p.Ep / 32) * (p.H / 64) : 0;
  const int tok_wgs = p.Tp / 32;
  if (tok_wgs + w_wgs)
    k_router_dl<<<tok_wgs + w_wgs, 512, lds, s>>>(p);
  if (p.dX && p.T > 0) k_router_dx<<<dim3((p.T + 127) / 128, (p.H + 127) / 128), 256, 0, s>>>(p);
  int dw_wgs = 0;
  if (p.dW) {
    const dim3 grid(p.Ep / 64, (p.H + 127) / 128, p.chunks);
    if (bf16) k_router_dw<BF16><<<grid, 256, 0, s>>>(p);
    else k_router_dw<F16><<<grid, 256, 0, s>>>(p);
    dw_wgs = (int)(((size_t)p.E * p.H / 4 + 1023) / 1024);
  }
  const int db_wgs = p.dbias ? (p.E + 63) / 64 : 0;
  if (dw_wgs + db_wgs) k_router_add<<<dw_wgs + db_wgs, 1024, 0, s>>>(p, dw_wgs);
  return hipGetLastError();
}

}  // namespace mpb
