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
// in fp32, and only products below 2^-24 of the whole are left out (dX takes
// fp16 halves instead, see halves). Against the fp32 matrix instructions (1/16
// of the 16-bit rate) three to five products are still 3 to 5 times cheaper.
#include <type_traits>

#include "k_block_common.h"
#include "mpb.h"
#include "mpb_internal.h"

namespace mpb {

namespace {

__device__ __forceinline__ bool is_live(const RouterLossParams& p, int t) {
  return t < p.T && (!p.mask || p.mask[t]);
}

// Workgroups go round the 8 XCDs by their linear index. The n expert tiles that
// read the same activations are given to one XCD, one after the other, so that
// its L2 serves all but the first: splits linear index b of `count * n` into
// (tile, rest).
__device__ __forceinline__ void xcd_pairs(int b, int n, int count, int& tile, int& rest) {
  const int full = count / 8 * 8 * n;
  if (b < full) {
    tile = (b >> 3) % n;
    rest = (b >> 3) / n * 8 + (b & 7);
  } else {  // the last count % 8
    tile = (b - full) % n;
    rest = full / n + (b - full) / n;
  }
}

// ---------------------------------------------------------------- logits
// 16 MT tokens x 64 ET experts x one range of H per workgroup of 4 waves; a
// wave holds 16 ET experts, whose W it reads straight into fragments and cuts
// there (each W value is read by one wave of the workgroup, so that the cutting
// is shared by MT products); the tokens' activations are staged in LDS for all
// four waves, 64 elements of H at a time, the next stage's loads in flight
// during the products. Partial sums go to part[range][T][E].
// 128 tokens x 128 experts (64 where there are no more) from 8192 tokens, 64 x 64
// below. The whole forward call, us with 64- and with 128-token tiles:
//   tokens             4096        6000        8192        10000       16381
//   2048 x 60, bf16    21.3/24.5   25.3/26.0   25.6/25.8   29.3/31.9   34.9/35.1
//   2816 x 128, bf16   30.1/34.1   41.0/40.9   42.5/42.4   63.2/52.0   72.0/71.8
//   2816 x 128, fp16   34.8/36.8   48.7/46.5   50.9/48.6   77.5/62.8   88.1/85.0
//   2816 x 300, bf16   89.9/79.9   94.1/95.5   118/109     145/118     185/172
// (16381 x 4096 x 128: the kernel 63 us against 95; with 128 tokens x 64 experts 75;
// 4096 x 2816 x 128: 18.6 against 22). The matrix cores
// are busy a third of the time: the cutting (as many VALU cycles) and the reads of
// W, 16 bytes a cycle as a fragment's lanes lie in 16 rows, do not overlap enough
// with them. Staging W in LDS as well (18.3 and 73 us) and loading two stages
// ahead (19.2 and 75) did not help.
constexpr int kLK = 64, kLRow = kLK + 8;  // 16 bytes of padding per LDS row

template <class D, int MT, int ET>
__global__ __launch_bounds__(256, 2) void k_router_logits(RouterLossParams p) {
  typedef typename D::vec vec;
  typedef typename D::elem elem;
  constexpr int NP = Parts<D>::N, NX = MT / 2;  // vectors that a thread stages
  __shared__ __align__(16) __bf16 xs[2][NP][16 * MT * kLRow];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, g = lane >> 4;
  const int et = (p.E + 64 * ET - 1) / (64 * ET);
  int ey, tx;
  xcd_pairs(blockIdx.x, et, gridDim.x / et, ey, tx);
  const int t0 = tx * 16 * MT, e0 = ey * 64 * ET + wave * 16 * ET + n;
  const int steps = p.H / kLK, s0 = (int)((long long)steps * blockIdx.y / gridDim.y),
            s1 = (int)((long long)steps * (blockIdx.y + 1) / gridDim.y);
  const float* wrow = p.W + (size_t)(e0 < p.E ? e0 : 0) * p.H + 8 * g;
  // a thread stages rows tid / 8 + 32 i, columns 8 (tid % 8)
  const int r0 = tid >> 3, c0 = (tid & 7) * 8;
  unsigned live = 0;
#pragma unroll
  for (int i = 0; i < NX; ++i) live |= (is_live(p, t0 + r0 + 32 * i) ? 1u : 0u) << i;
  const elem* xrow = (const elem*)p.X + (size_t)(t0 + r0) * p.H + c0;
  vec xv[NX];
  fx8 wv[2][ET];
  auto load = [&](int s) {
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      xv[i] = (vec)(elem)0.0f;
      if (live >> i & 1) xv[i] = *(const vec*)(xrow + (size_t)(32 * i) * p.H + s * kLK);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int e = 0; e < ET; ++e) {
        wv[i][e] = (fx8)(0.0f);
        if (e0 + 16 * e < p.E) wv[i][e] = load8(wrow + (size_t)(16 * e) * p.H + s * kLK + 32 * i);
      }
    }
  };
  acc4 acc[MT][ET];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int e = 0; e < ET; ++e) acc[m][e] = (acc4)(0.0f);
  load(s0);
  for (int s = s0; s < s1; ++s) {
    const int b = (s - s0) & 1;
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      bx8 q[NP];
      Parts<D>::of(xv[i], q);
#pragma unroll
      for (int k = 0; k < NP; ++k) *(bx8*)&xs[b][k][(r0 + 32 * i) * kLRow + c0] = q[k];
    }
    bx8 w[2][ET][3];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < ET; ++e) cut<3>(wv[i][e], w[i][e]);
    if (s + 1 < s1) load(s + 1);
    __syncthreads();  // xs[b] is written; the other half was read before the barrier of the step before
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int k = NP - 1; k >= 0; --k) {
          const bx8 x = *(const bx8*)&xs[b][k][(16 * m + n) * kLRow + 32 * i + 8 * g];
#pragma unroll
          for (int j = 2 - k; j >= 0; --j)  // smallest parts first
#pragma unroll
            for (int e = 0; e < ET; ++e) acc[m][e] = mfma(x, w[i][e][j], acc[m][e]);
        }
      }
    }
  }
  float* out = p.part + (size_t)blockIdx.y * p.T * p.E;
#pragma unroll
  for (int e = 0; e < ET; ++e) {
    if (e0 + 16 * e < p.E) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = t0 + 16 * m + 4 * g + r;
          if (t < p.T) out[(size_t)t * p.E + e0 + 16 * e] = acc[m][e][r];
        }
      }
    }
  }
}

// ---------------------------------------------------------------- softmax, counts
// One wave per token: adds the ranges of H, writes logits and lse, and keeps
// its share of P_e, z and N in registers; a workgroup (16 waves) writes one row
// of them to stat [groups][E + 1] (sum and count of each expert, then z and N).
// EJ: experts of a lane, e = lane + 64 j. Bound by the chain of a token's loads,
// reductions and exponentials, a few tokens a wave: 6.7 us for 4096 tokens, 20 for
// 16381 (42 MB).
template <int EJ>
__global__ __launch_bounds__(1024) void k_router_stats(RouterLossParams p) {
  __shared__ int cnt[513];
  __shared__ float pr[16][64 * EJ + 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = p.E;
  for (int i = tid; i <= E; i += 1024) cnt[i] = 0;
  __syncthreads();
  float psum[EJ], z = 0.0f;
#pragma unroll
  for (int j = 0; j < EJ; ++j) psum[j] = 0.0f;
  float bias[EJ];
#pragma unroll
  for (int j = 0; j < EJ; ++j) bias[j] = p.bias && lane + 64 * j < E ? p.bias[lane + 64 * j] : 0.0f;
  for (int t = blockIdx.x * 16 + wave; t < p.T; t += gridDim.x * 16) {
    // all of a token's loads go out together
    const int alive = p.mask ? p.mask[t] : 1;
    const int id = p.idx[(size_t)t * p.K + (lane < p.K ? lane : 0)];
    float l[EJ], m = -INFINITY;
    bool nan = false;  // fmaxf drops nan
#pragma unroll
    for (int j = 0; j < EJ; ++j) {
      const int e = lane + 64 * j;
      const float* src = p.part + (size_t)t * E + (e < E ? e : 0);
      float v = 0.0f;
#pragma unroll 8
      for (int s = 0; s < p.splits; ++s) v += src[(size_t)s * p.T * E];
      l[j] = alive ? v + bias[j] : 0.0f;
      if (e < E) {
        p.logits[(size_t)t * E + e] = l[j];
        m = fmaxf(m, l[j]);
        nan |= l[j] != l[j];
      }
    }
    m = wave_max(m);
    float s = 0.0f, x[EJ];
#pragma unroll
    for (int j = 0; j < EJ; ++j) {
      x[j] = lane + 64 * j < E ? expf(l[j] - m) : 0.0f;
      s += x[j];
    }
    s = wave_sum(s);
    float lse = m == -INFINITY ? -INFINITY : m + logf(s);
    if (__ballot(nan)) lse = NAN;
    if (lane == 0) p.lse[t] = alive ? lse : 0.0f;
    if (!alive || lse == -INFINITY) continue;  // padding, or no expert left: the token does not count
    z += lse * lse;
    const float r = lse == lse ? 1.0f / s : NAN;
#pragma unroll
    for (int j = 0; j < EJ; ++j) psum[j] += x[j] * r;
    if (lane < p.K && id >= 0 && id < E) atomicAdd(&cnt[id], 1);
    if (lane == 0) atomicAdd(&cnt[E], 1);
  }
#pragma unroll
  for (int j = 0; j < EJ; ++j)
    if (lane + 64 * j < E) pr[wave][lane + 64 * j] = psum[j];
  if (lane == 0) pr[wave][E] = z;
  __syncthreads();
  for (int i = tid; i <= E; i += 1024) {
    float s = pr[0][i];
    for (int w = 1; w < 16; ++w) s += pr[w][i];
    p.stat[(size_t)blockIdx.x * (E + 1) + i] = make_int2(__float_as_int(s), cnt[i]);
  }
}

// Adds the groups' rows (fp64; 16 slices in group order, then the slices in
// order) and forms the losses. One workgroup; every load of a thread is
// independent of the others. EJ: columns of 64.
template <int EJ>
__global__ __launch_bounds__(1024) void k_router_finish(RouterLossParams p) {
  __shared__ double fs[16][64];
  __shared__ int is[16][64];
  const int tid = threadIdx.x, lane = tid & 63, sl = tid >> 6, E = p.E, W = E + 1;
  // z and N: the last column, one group a thread (at most 256 groups)
  const int2 last = tid < p.groups ? p.stat[(size_t)tid * W + E] : make_int2(0, 0);
  double f[EJ];
  int n[EJ];
#pragma unroll
  for (int j = 0; j < EJ; ++j) {
    f[j] = 0.0;
    n[j] = 0;
  }
#pragma unroll 4
  for (int i = sl; i < p.groups; i += 16) {
#pragma unroll
    for (int j = 0; j < EJ; ++j) {
      const int2 v = p.stat[(size_t)i * W + (lane + 64 * j < E ? lane + 64 * j : 0)];
      f[j] += (double)__int_as_float(v.x);
      n[j] += v.y;
    }
  }
  double part = 0.0;
#pragma unroll
  for (int j = 0; j < EJ; ++j) {
    fs[sl][lane] = f[j];
    is[sl][lane] = n[j];
    __syncthreads();
    if (sl == 0 && lane + 64 * j < E) {
      for (int k = 1; k < 16; ++k) {
        f[j] += fs[k][lane];
        n[j] += is[k][lane];
      }
      p.counts[lane + 64 * j] = n[j];
      p.prob[lane + 64 * j] = (float)f[j];
      part += f[j] * (double)n[j];
    }
    __syncthreads();
  }
  // wave 0: sum over the experts; waves 0..3: z and N over the groups
  double z = (double)__int_as_float(last.x);
  int live = last.y;
#pragma unroll
  for (int m = 32; m; m >>= 1) {
    part += __shfl_xor(part, m);
    z += __shfl_xor(z, m);
    live += __shfl_xor(live, m);
  }
  if (lane == 0) {
    fs[sl][0] = z;
    is[sl][0] = live;
  }
  __syncthreads();
  if (tid == 0) {
    for (int k = 1; k < 4; ++k) {
      z += fs[k][0];
      live += is[k][0];
    }
    p.counts[E] = live;
    const double N = live > 0 ? (double)live : 1.0;
    const double bal = (double)E * part / ((double)p.K * N * N);
    z /= N;
    p.loss[0] = (float)((double)p.alpha * bal + (double)p.beta * z);
    p.loss[1] = (float)bal;
    p.loss[2] = (float)z;
  }
}

// ---------------------------------------------------------------- gradients
// dl is kept in two forms, both cut into parts and laid out as operand
// fragments in the order that a wave's lanes read them (16 bytes a lane, 1 KiB a
// fragment):
//   dl_t [3][expert / 16][token / 32]   lane (n, g): expert n, tokens 8g..8g+7;
//        bf16 parts, as bf16 activations need them on the other side
//   dl_a [2][token / 16][expert / 32]   lane (n, g): token n, experts 8g..8g+7;
//        fp16 halves (see halves) of dl scaled by its token's power of two,
//        whose inverse is dl_s [Tp]
// on [Tp]: whether a token takes part.
// The power of two that brings a largest magnitude m into [2^13, 2^14) (at most
// 2^126; 1 for zero, inf and nan).
__device__ __forceinline__ float scale_for(float m) {
  const int e = (int)(__float_as_uint(m) >> 23);  // biased exponent
  const int k = e == 0 || e == 255 ? (e ? 0 : m > 0.0f ? 126 : 0) : 127 + 13 - e;
  return ldexpf(1.0f, k > 126 ? 126 : k);
}

// x = hi + lo / kLo in fp16, both rounded to nearest: 22 bits of x. Without kLo,
// lo would fall below fp16's smallest step (2^-24) where x is under 2^-17 of its
// row's largest value (scale_for), and leave errors of 2^-38 of that; with it they
// stay below 2^-49 of it. Three products of halves, hi hi + (hi lo + lo hi) / kLo,
// are then within 12 x 2^-24 of the exact product (and of 2^-49 of the row's or
// column's largest value): half the matrix work of three bf16 parts, where a power
// of two per row and per column can be taken out of the product.
constexpr float kLo = 2048.0f;

__device__ __forceinline__ void halves(fx8 x, hx8 (&q)[2]) {
  q[0] = narrow<F16>(x);
  q[1] = narrow<F16>((x - widen<F16>(q[0])) * kLo);
}

__device__ __forceinline__ size_t frag(size_t tiles, size_t part, size_t tile) { return (part * tiles + tile) * 512; }

// dl of 32 tokens per workgroup, two per wave, held in LDS and written in both
// forms, with the tile's column sums. EJ: experts of a lane, e = lane + 64 j. The
// logits, not the activations, are read: 7.7 us for 4096 tokens, 18.8 for 16381.
template <int EJ>
__global__ __launch_bounds__(1024) void k_router_dl(RouterLossParams p) {
  extern __shared__ __align__(16) float ds[];  // [32][Ep + 4]
  __shared__ float scl[32];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, g = lane >> 4;
  const int E = p.E, Ep = p.Ep;
  const int t0 = blockIdx.x * 32, row = Ep + 4;
  const int N = p.counts[E];
  const float gl = p.gloss ? *p.gloss : 1.0f, inv_n = N > 0 ? 1.0f / (float)N : 0.0f;
  const float ca = gl * p.alpha * (float)E * inv_n, cb = gl * 2.0f * p.beta * inv_n, cf = inv_n / (float)p.K;
  float f[EJ];  // f_e
#pragma unroll
  for (int j = 0; j < EJ; ++j) f[j] = lane + 64 * j < E ? (float)p.counts[lane + 64 * j] * cf : 0.0f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = wave * 2 + i, t = t0 + r, tc = t < p.T ? t : p.T - 1;
    // all of a token's loads go out together
    float lse = p.lse[tc];
    const bool alive = is_live(p, t);
    int id = -1;
    float gw = 0.0f;
    if (p.gw && lane < p.K) {
      id = p.idx[(size_t)tc * p.K + lane];
      gw = p.gw[(size_t)tc * p.K + lane];
    }
    float l[EJ], pr[EJ], dot = 0.0f;
#pragma unroll
    for (int j = 0; j < EJ; ++j) l[j] = p.logits[(size_t)tc * E + (lane + 64 * j < E ? lane + 64 * j : 0)];
    const bool on = alive && !(lse == -INFINITY);  // nan stays on and spreads
    if (lane == 0) p.on[t] = on ? 1 : 0;
    if (!on) lse = 0.0f;
#pragma unroll
    for (int j = 0; j < EJ; ++j) {
      pr[j] = on && lane + 64 * j < E ? expf(l[j] - lse) : 0.0f;
      dot += f[j] * pr[j];
    }
    dot = wave_sum(dot);
    float c = 0.0f;
    if (p.gw) {
      if (!on || id < 0 || id >= E) id = -1;
      float lk = -INFINITY;  // the slot's logit, from the lane that holds its expert
#pragma unroll
      for (int j = 0; j < EJ; ++j) {
        const float v = __shfl(l[j], id & 63);
        if (id >= 0 && id >> 6 == j) lk = v;
      }
      const float m = wave_max(lk);
      const float x = id >= 0 && m > -INFINITY ? expf(lk - m) : 0.0f;
      const float s = wave_sum(x), w = s > 0.0f ? x / s : x;
      const float mean = wave_sum(id >= 0 ? w * gw : 0.0f);
      c = id >= 0 ? w * (gw - mean) : 0.0f;
    }
    float d[EJ], most = 0.0f;
#pragma unroll
    for (int j = 0; j < EJ; ++j) {
      const int e = lane + 64 * j;
      d[j] = on && e < E ? pr[j] * (ca * (f[j] - dot) + cb * lse) : 0.0f;
      if (p.gw) {
        for (int k = 0; k < p.K; ++k) {  // slots in order, also where one expert is named twice
          const int ik = __builtin_amdgcn_readlane(id, k);
          const float ck = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(c), k));
          if (ik == e) d[j] += ck;
        }
      }
      if (e < Ep) ds[r * row + e] = d[j];
      most = fmaxf(most, fabsf(d[j]));
    }
    const float up = scale_for(wave_max(most));
    if (lane == 0) {
      scl[r] = up;
      p.dl_s[t] = 1.0f / up;
    }
  }
  __syncthreads();
  const int kt = Ep / 32;
  const size_t ta = (size_t)(p.Tp / 16) * kt;
  for (int i = wave; i < 2 * kt; i += 16) {  // dl_a: 2 token tiles x kt expert tiles
    const int m = i & 1, k32 = i >> 1;
    hx8 q[2];
    halves(load8(ds + (16 * m + n) * row + 32 * k32 + 8 * g) * scl[16 * m + n], q);
#pragma unroll
    for (int k = 0; k < 2; ++k) *(hx8*)(p.dl_a + frag(ta, k, (size_t)(t0 / 16 + m) * kt + k32) + 8 * lane) = q[k];
  }
  const size_t tt = (size_t)(Ep / 16) * (p.Tp / 32);
  for (int et = wave; et < Ep / 16; et += 16) {  // dl_t: Ep / 16 expert tiles
    fx8 x;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = ds[(8 * g + i) * row + 16 * et + n];
    bx8 q[3];
    cut<3>(x, q);
#pragma unroll
    for (int k = 0; k < 3; ++k)
      *(bx8*)(p.dl_t + frag(tt, k, (size_t)et * (p.Tp / 32) + t0 / 32) + 8 * lane) = q[k];
  }
  for (int e = tid; e < E; e += 1024) {
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < 32; ++r) s += ds[r * row + e];
    p.db_part[(size_t)blockIdx.x * E + e] = s;
  }
}

// dX = dl W: a workgroup keeps W of 64 columns and up to 128 experts in LDS, as
// two fp16 halves (32 KiB, cut once, each column scaled by a power of two), and
// goes over its range of tokens, 256 at a time; a wave holds 64 tokens x 64
// columns. The columns are the products' rows, so that a lane ends with four of
// a token's consecutive columns. Ranges of tokens are dealt to the XCDs, so that
// each L2 holds its own part of dl. 16381 x 4096 x 128: 77 us for 268 MB written
// (3.5 TB/s) and 52 GFLOP of products; without kLo, which takes the products with
// a second half apart, 73. Measured without it: with plain stores 75 (and 65 instead
// of 57 for dW behind it, whose operands they push out), with stores of 64 bytes a
// row 82, with three bf16 parts 115, with both operands read from L2 as bf16
// fragments 135.
__global__ __launch_bounds__(256, 2) void k_router_dx(RouterLossParams p) {
  __shared__ __align__(16) _Float16 wl[2 * 4 * 4 * 512];  // [half][column / 16][expert / 32] fragments
  __shared__ __align__(16) float down[64];                // inverse scales of the columns
  __shared__ __align__(16) float turn[4][16][64 + 4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
  const int cols = p.H / 64, blocks = (p.Tp + 255) / 256, kt = p.Ep / 32;
  const size_t ta = (size_t)(p.Tp / 16) * kt;
  int cg, range;
  xcd_pairs(blockIdx.x, cols, p.dx_ranges, cg, range);
  const int h0 = cg * 64;
  const int b0 = (int)((long long)blocks * range / p.dx_ranges), b1 = (int)((long long)blocks * (range + 1) / p.dx_ranges);
  const auto w_at = [&](int k) {  // column 16 wave + n, experts 32 k + 8 g ..
    fx8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = 32 * k + 8 * g + i;
      v[i] = p.W[(size_t)(e < p.E ? e : 0) * p.H + h0 + 16 * wave + n];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 32 * k + 8 * g + i < p.E ? v[i] : 0.0f;
    return v;
  };
  float up = 0.0f;
  const auto load_w = [&](int k0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      hx8 q[2];
      halves(w_at(k0 + k) * up, q);
#pragma unroll
      for (int i = 0; i < 2; ++i) *(hx8*)(wl + ((i * 4 + wave) * 4 + k) * 512 + 8 * lane) = q[i];
    }
  };
  hx8 d[4][2];  // dl of the next step
  const auto load_d = [&](int b, int k) {
    const int t0 = b * 256 + wave * 64, tile = (t0 < p.Tp ? t0 : 0) / 16;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int m = 0; m < 4; ++m) d[m][q] = *(const hx8*)(p.dl_a + frag(ta, q, (size_t)(tile + m) * kt + k) + 8 * lane);
  };
  load_d(b0, 0);
  float most = 0.0f;
  for (int k = 0; k < kt; ++k) {
    const fx8 v = w_at(k);
#pragma unroll
    for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(v[i]));
  }
  most = fmaxf(most, __shfl_xor(most, 16));
  most = fmaxf(most, __shfl_xor(most, 32));
  up = scale_for(most);
  if (g == 0) down[16 * wave + n] = 1.0f / up;
  if (kt <= 4) load_w(0);
  __syncthreads();
  // FULL: every token of the block is below T, so that nothing stands between the
  // stores and the next block's products but a wait for its dl, loaded before them
  const auto block = [&](int b, auto FULL) {
    const int t0 = b * 256 + wave * 64;
    acc4 acc[4][4];
    float ts[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int t = t0 + 16 * m + n;
      ts[m] = 0.0f;
      if (FULL.value || t < p.Tp) ts[m] = p.on[t] ? p.dl_s[t] : 0.0f;
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[m][c] = (acc4)(0.0f);
    }
    for (int k = 0; k < kt; ++k) {
      if (kt > 4 && k % 4 == 0) {
        __syncthreads();
        load_w(k);
        __syncthreads();
      }
      hx8 a[4][2];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        a[m][0] = d[m][0];
        a[m][1] = d[m][1];
      }
      const bool same = k + 1 < kt;
      load_d(same || b + 1 >= b1 ? b : b + 1, same ? k + 1 : 0);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        hx8 w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) w[i] = *(const hx8*)(wl + ((i * 4 + c) * 4 + k % 4) * 512 + 8 * lane);
        acc4 lo[4];  // the products with a second half, times kLo
#pragma unroll
        for (int s = 0; s < 3; ++s)  // lo hi, hi lo, hi hi
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            acc4& to = s < 2 ? lo[m] : acc[m][c];
            to = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[s == 0], a[m][s == 1], s ? to : (acc4)(0.0f), 0, 0, 0);
          }
#pragma unroll
        for (int m = 0; m < 4; ++m) acc[m][c] += lo[m] * (1.0f / kLo);
      }
    }
    // through LDS (one wave's accesses run in order), to store whole lines
#pragma unroll
    for (int m = 0; m < 4; ++m) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const acc4 v = acc[m][c] * *(const acc4*)(down + 16 * c + 4 * g) * ts[m];
        *(acc4*)&turn[wave][n][16 * c + 4 * g] = ts[m] > 0.0f ? v : (acc4)(0.0f);
      }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = t0 + 16 * m + 4 * i + g;
        if (FULL.value || t < p.T)
          stream_store((acc4*)(p.dX + (size_t)t * p.H + h0 + 4 * n), *(const acc4*)&turn[wave][4 * i + g][4 * n]);
      }
      __builtin_amdgcn_wave_barrier();
    }
  };
  int b = b0;
  for (; b < b1 && (b + 1) * 256 <= p.T; ++b) block(b, std::true_type{});
  if (b < b1) block(b, std::false_type{});
}

// dW = dl^T X: a workgroup holds 64 experts x 128 columns over one range of
// tokens, its four waves taking 32 tokens in turn. A lane loads 8 tokens x 8
// columns of X and turns them round in registers, which gives the 8 column
// fragments of a step (fragment j: columns 8 n + j). The waves' sums meet in
// LDS in wave order. One wave a SIMD with the next step's operands in flight
// (338 registers): 16381 x 4096 x 128 takes 57 us, 0.9 PFLOP/s of the 1.18 that a
// large bf16 product reaches; two waves without that 152, and 212 with loads that
// wait for their token's mask.
template <class D>
__global__ __launch_bounds__(256, 1) void k_router_dw(RouterLossParams p) {
  typedef typename D::vec vec;
  typedef typename D::elem elem;
  constexpr int NP = Parts<D>::N;
  __shared__ __align__(16) float sum[64][128 + 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, g = lane >> 4;
  const int ht = (p.H + 127) / 128;
  int ex, rest;
  xcd_pairs(blockIdx.x, p.Ep / 64, ht * p.chunks, ex, rest);
  const int e0 = ex * 64, h0 = rest % ht * 128, chunk = rest / ht, h = h0 + 8 * n;
  const int nt = p.Tp / 32;
  const int b0 = (int)((long long)nt * chunk / p.chunks), b1 = (int)((long long)nt * (chunk + 1) / p.chunks);
  const size_t tt = (size_t)(p.Ep / 16) * nt;
  acc4 acc[4][8];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[a][j] = (acc4)(0.0f);
  vec x[8];
  bx8 a[4][3];
  unsigned long long on;  // 8 tokens' bytes
  const elem* xcol = (const elem*)p.X + (h < p.H ? h : 0);
  // every load goes out at once: rows past the batch read its last one, and the
  // tokens that do not take part are cleared when their bytes have come
  auto load = [&](int b) {
    on = *(const unsigned long long*)(p.on + 32 * b + 8 * g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = 32 * b + 8 * g + i;
      x[i] = *(const vec*)(xcol + (size_t)(t < p.T ? t : p.T - 1) * p.H);
    }
#pragma unroll
    for (int q = 0; q < 3; ++q)
#pragma unroll
      for (int m = 0; m < 4; ++m)
        a[m][q] = *(const bx8*)(p.dl_t + frag(tt, q, (size_t)(e0 / 16 + m) * nt + b) + 8 * lane);
  };
  if (b0 + wave < b1) load(b0 + wave);
  for (int b = b0 + wave; b < b1; b += 4) {
    vec c[8];  // the 8 x 8 block turned round
    bx8 d[4][3];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = on >> (8 * i) & 1 ? x[i] : (vec)(elem)0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) c[j][i] = x[i][j];
#pragma unroll
    for (int q = 0; q < 3; ++q)
#pragma unroll
      for (int m = 0; m < 4; ++m) d[m][q] = a[m][q];
    if (b + 4 < b1) load(b + 4);  // the next step's operands come in during the products
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      bx8 q[NP];
      Parts<D>::of(c[j], q);
#pragma unroll
      for (int k = NP - 1; k >= 0; --k)
#pragma unroll
        for (int i = 2 - k; i >= 0; --i)
#pragma unroll
          for (int m = 0; m < 4; ++m) acc[m][j] = mfma(d[m][i], q[k], acc[m][j]);
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
  float* out = p.dw_part + (size_t)chunk * p.E * p.H;
  for (int i = tid; i < 64 * 16; i += 256) {
    const int e = i >> 4, c = (i & 15) * 8, col = h0 + c;
    if (e0 + e < p.E && col < p.H) store8(out + (size_t)(e0 + e) * p.H + col, load8(&sum[e][c]));
  }
}

// Adds the token ranges of dW (workgroups below `dw_wgs`, 4 values a thread)
// and the token tiles of dbias (16 experts a workgroup, 16 slices).
__global__ __launch_bounds__(256) void k_router_add(RouterLossParams p, int dw_wgs) {
  __shared__ double buf[256];
  const int tid = threadIdx.x;
  if ((int)blockIdx.x < dw_wgs) {
    const size_t n = (size_t)p.E * p.H, i = ((size_t)blockIdx.x * 256 + tid) * 4;
    if (i >= n) return;
    fx4 s = (fx4)(0.0f);
#pragma unroll 8
    for (int c = 0; c < p.chunks; ++c) s += *(const fx4*)(p.dw_part + (size_t)c * n + i);
    *(fx4*)(p.dW + i) = s;
    return;
  }
  const int e = (blockIdx.x - dw_wgs) * 16 + (tid & 15);
  double s = 0.0;
  if (e < p.E)
#pragma unroll 8
    for (int i = tid >> 4; i < p.Tp / 32; i += 16) s += (double)p.db_part[(size_t)i * p.E + e];
  buf[tid] = s;
  __syncthreads();
  if (tid < 16 && e < p.E) {
    for (int k = 1; k < 16; ++k) s += buf[tid + 16 * k];
    p.dbias[e] = (float)s;
  }
}

}  // namespace

static size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

RouterLossWs router_loss_ws(int T, int H, int E) {
  RouterLossWs w{};
  // 128-token tiles where the batch fills the chip with them, else 64
  w.mt = T >= 8192 ? 8 : 4;
  w.et = w.mt == 8 && E > 64 ? 2 : 1;
  const int tiles = ((T + 16 * w.mt - 1) / (16 * w.mt)) * ((E + 64 * w.et - 1) / (64 * w.et));
  // ranges of H for the logits: about 512 workgroups, whole stages of 64
  w.splits = tiles > 0 ? 512 / tiles : 1;
  if (w.splits > 16) w.splits = 16;
  if (w.splits > H / kLK) w.splits = H / kLK;
  if (w.splits < 1) w.splits = 1;
  w.groups = (T + 15) / 16 < 256 ? (T + 15) / 16 : 256;
  if (w.groups < 1) w.groups = 1;
  size_t off = 0;
  w.part = off;   off += up256((size_t)w.splits * T * E * 4);
  w.stat = off;   off += up256((size_t)w.groups * (E + 1) * 8);
  const size_t fwd = off;
  w.Tp = (T + 63) / 64 * 64;
  w.Ep = (E + 63) / 64 * 64;
  const int wt = (w.Ep / 64) * ((H + 127) / 128), nt = w.Tp / 32;
  // ranges of tokens for dW: about 256 workgroups, at least 8 tiles of 32 tokens each
  w.chunks = 256 / wt;
  if (w.chunks > nt / 8) w.chunks = nt / 8;
  if (w.chunks < 1) w.chunks = 1;
  // ranges of tokens for dX, whole blocks of 256 tokens: one block each up to
  // 1024 workgroups, else 512 workgroups (two per CU)
  const int blocks = (w.Tp + 255) / 256, cols = H / 64;
  w.dx_ranges = blocks;
  if ((long long)blocks * cols > 1024) w.dx_ranges = (512 + cols - 1) / cols;
  if (w.dx_ranges > blocks) w.dx_ranges = blocks;
  if (w.dx_ranges < 1) w.dx_ranges = 1;
  off = 0;
  w.dl_a = off;    off += up256((size_t)2 * w.Tp * w.Ep * 2);
  w.dl_s = off;    off += up256((size_t)w.Tp * 4);
  w.dl_t = off;    off += up256((size_t)3 * w.Tp * w.Ep * 2);
  w.on = off;      off += up256((size_t)w.Tp);
  w.db_part = off; off += up256((size_t)(w.Tp / 32) * E * 4);
  w.dw_part = off; off += up256((size_t)w.chunks * E * H * 4);
  w.total = fwd > off ? fwd : off;
  return w;
}

template <class D>
static void logits(const RouterLossParams& p, hipStream_t s) {
  const dim3 grid(((p.T + 16 * p.mt - 1) / (16 * p.mt)) * ((p.E + 64 * p.et - 1) / (64 * p.et)), p.splits);
  // 128 experts only beside 128 tokens
  if (p.et == 2) k_router_logits<D, 8, 2><<<grid, 256, 0, s>>>(p);
  else if (p.mt == 8) k_router_logits<D, 8, 1><<<grid, 256, 0, s>>>(p);
  else k_router_logits<D, 4, 1><<<grid, 256, 0, s>>>(p);
}

hipError_t launch_router_loss(const RouterLossParams& p, bool bf16, hipStream_t s) {
  if (p.T > 0) {
    if (bf16) logits<BF16>(p, s);
    else logits<F16>(p, s);
  }
  if (p.E <= 64) {
    k_router_stats<1><<<p.groups, 1024, 0, s>>>(p);
    k_router_finish<1><<<1, 1024, 0, s>>>(p);
  } else if (p.E <= 128) {
    k_router_stats<2><<<p.groups, 1024, 0, s>>>(p);
    k_router_finish<2><<<1, 1024, 0, s>>>(p);
  } else {
    k_router_stats<8><<<p.groups, 1024, 0, s>>>(p);
    k_router_finish<8><<<1, 1024, 0, s>>>(p);
  }
  return hipGetLastError();
}

hipError_t launch_router_loss_grad(const RouterLossParams& p, bool bf16, hipStream_t s) {
  static unsigned long long raised = 0;
  const int lds = 32 * (p.Ep + 4) * 4;
  if (lds > 64 * 1024) {
    const hipError_t e = raise_lds_limit((const void*)k_router_dl<8>, 32 * (512 + 4) * 4, raised);
    if (e != hipSuccess) return e;
  }
  const int dl_wgs = p.Tp / 32;
  if (dl_wgs) {
    if (p.Ep == 64) k_router_dl<1><<<dl_wgs, 1024, lds, s>>>(p);
    else if (p.Ep == 128) k_router_dl<2><<<dl_wgs, 1024, lds, s>>>(p);
    else k_router_dl<8><<<dl_wgs, 1024, lds, s>>>(p);
  }
  if (p.dX) {
    k_router_dx<<<p.H / 64 * p.dx_ranges, 256, 0, s>>>(p);
  }
  int dw_wgs = 0;
  if (p.dW) {
    const int grid = (p.Ep / 64) * ((p.H + 127) / 128) * p.chunks;
    if (bf16) k_router_dw<BF16><<<grid, 256, 0, s>>>(p);
    else k_router_dw<F16><<<grid, 256, 0, s>>>(p);
    dw_wgs = (int)(((size_t)p.E * p.H / 4 + 255) / 256);
  }
  const int db_wgs = p.dbias ? (p.E + 15) / 16 : 0;
  if (dw_wgs + db_wgs) k_router_add<<<dw_wgs + db_wgs, 256, 0, s>>>(p, dw_wgs);
  return hipGetLastError();
}

}  // namespace mpb
