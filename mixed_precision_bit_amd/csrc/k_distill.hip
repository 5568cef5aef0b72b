// Distillation of a teacher's top logits: the loss of student logits s against k
// stored teacher logits a row, and its gradient.
//
//   q_j = exp(t_j / tau - L), L the teacher's logsumexp (over all its logits where
//   the caller gives it, else over the k entries);  p = softmax(s / tau)
//   kl = sum_j q_j (log q_j - log p_j) + q_r (log q_r - log p_r)
//   q_r = 1 - sum_j q_j, p_r = the student's probability outside the entries
//   (the last term only where L is given)
//   ds_v = g w tau (p_v Q - q_v) for an entry, g w tau p_v (Q - q_r / p_r) else,
//   Q = sum_j q_j + q_r
//
// A workgroup takes a row. The entries' ids become a bitmap in LDS; one pass over
// the row keeps the running maximum and sum of exponentials of what is not an
// entry (so that p_r is a sum of its own, not 1 minus the rest), the entries are
// gathered by a thread each, and the few sums over them run in fp64. The gradient
// in the same launch reads the row again, from the Infinity Cache: 256 CUs hold
// rows of 80 MB at most sizes. Nothing is written twice: the pass over the row leaves the
// entries out, and each entry's thread writes its own.
//
// Rows may begin at any element: up to 7 elements before the first 16-byte
// boundary and after the last are taken one by one.
#include <cfloat>

#include "k_block_common.h"
#include "mpb.h"
#include "mpb_internal.h"

namespace mpb {

namespace {

struct F32 {
  typedef float elem;
  typedef fx8 vec;
};

template <class D>
__device__ __forceinline__ fx8 read8(const typename D::elem* p) {
  return widen<D>(*(const typename D::vec*)p);
}
template <>
__device__ __forceinline__ fx8 read8<F32>(const float* p) {
  return load8(p);
}
template <class D>
__device__ __forceinline__ void write8(typename D::elem* p, fx8 v) {
  stream_store((typename D::vec*)p, narrow<D>(v));
}
template <>
__device__ __forceinline__ void write8<F32>(float* p, fx8 v) {
  stream_store8(p, v);
}

constexpr float kLog2e = 1.44269504f;

// A running maximum and the sum of exp((s - max) / tau) under it (c = log2(e) / tau).
// It starts at the lowest finite value: rows of -inf keep l = 0 and nothing is nan.
struct Running {
  float m = -FLT_MAX, l = 0.0f;
  __device__ __forceinline__ void raise(float to, float c) {
    if (to > m) {
      l *= __builtin_amdgcn_exp2f((m - to) * c);
      m = to;
    }
  }
  __device__ __forceinline__ void join(float om, float ol, float c) {
    const float to = fmaxf(m, om);
    l = l * __builtin_amdgcn_exp2f((m - to) * c) + ol * __builtin_amdgcn_exp2f((om - to) * c);
    m = to;
  }
};

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < 64; m *= 2) v += __shfl_xor(v, m);
  return v;
}

// Where a row lies: h elements before the first 16-byte boundary, nv vectors of 8.
struct Row {
  int h, nv;
};
template <class D>
__device__ __forceinline__ Row row_of(const typename D::elem* s, int V) {
  int h = (int)((16 - ((uintptr_t)s & 15)) & 15) / (int)sizeof(typename D::elem);
  h = min(h, V);
  return {h, (V - h) / 8};
}

// Bit of element v: the elements before the first boundary fill the end of byte 0,
// vector i has byte i + 1.
__device__ __forceinline__ int bit_of(const Row& r, int v) { return v - r.h + 8; }

template <class D, bool LOSS, bool GRAD>
__global__ __launch_bounds__(1024) void k_distill(DistillParams p) {
  typedef typename D::elem elem;
  extern __shared__ uint32_t bits[];
  __shared__ float red_m[16], red_l[16];
  __shared__ double red_d[4][4];
  __shared__ int s_ids[kDistillMaxK];
  __shared__ double s_q[kDistillMaxK];
  __shared__ int s_dup;
  const int tid = threadIdx.x, nt = blockDim.x, wave = tid >> 6, t = blockIdx.x, V = p.V, k = p.k;
  const elem* S = (const elem*)p.S + (size_t)t * p.ld;
  elem* dS = GRAD ? (elem*)p.dS + (size_t)t * p.ld : nullptr;
  const Row r = row_of<D>(S, V);
  const int tail = r.h + 8 * r.nv;  // first element after the vectors
  const float w = p.weight ? p.weight[t] : 1.0f / (float)p.T;

  if (w == 0.0f) {  // padding: what the row holds is not looked at
    if (LOSS && tid == 0) {
      p.kl[t] = 0.0f;
      *(fx4*)(p.stats + 4 * (size_t)t) = (fx4)(0.0f);
    }
    if constexpr (GRAD) {
      for (int v = tid; v < r.h; v += nt) dS[v] = (elem)0.0f;
      for (int i = tid; i < r.nv; i += nt) write8<D>(dS + r.h + 8 * i, (fx8)(0.0f));
      for (int v = tail + tid; v < V; v += nt) dS[v] = (elem)0.0f;
    }
    return;
  }

  // the entries: bitmap, ids and the student's logits at them
  for (int i = tid; i < p.words; i += nt) bits[i] = 0;
  if (tid == 0) s_dup = 0;
  __syncthreads();
  int id = -1;
  float st = -FLT_MAX;
  if (tid < k) {
    id = p.ids[(size_t)t * k + tid];
    if ((unsigned)id >= (unsigned)V) id = -1;
    s_ids[tid] = id;
    if (id >= 0) {
      st = (float)S[id];
      const int b = bit_of(r, id);
      if (atomicOr(&bits[b >> 5], 1u << (b & 31)) >> (b & 31) & 1) s_dup = 1;
    }
  }
  __syncthreads();
  const uint8_t* bytes = (const uint8_t*)bits;
  const float c = kLog2e / p.tau;

  // the row without its entries
  Running rest;
  if constexpr (LOSS) {
    constexpr int U = 4;  // vectors in flight
    auto take = [&](fx8 x, unsigned skip) {
      if (skip) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (skip >> i & 1) x[i] = -INFINITY;
      }
      float mx = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
      rest.raise(mx, c);
      float l = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) l += __builtin_amdgcn_exp2f((x[i] - rest.m) * c);
      rest.l += l;
    };
    auto one = [&](int v) {
      const int b = bit_of(r, v);
      if (bits[b >> 5] >> (b & 31) & 1) return;
      const float x = (float)S[v];
      rest.raise(x, c);
      rest.l += __builtin_amdgcn_exp2f((x - rest.m) * c);
    };
    int i = tid;
    for (; i + (U - 1) * nt < r.nv; i += U * nt) {
      fx8 x[U];
#pragma unroll
      for (int j = 0; j < U; ++j) x[j] = read8<D>(S + r.h + 8 * (size_t)(i + j * nt));
#pragma unroll
      for (int j = 0; j < U; ++j) take(x[j], bytes[i + j * nt + 1]);
    }
    for (; i < r.nv; i += nt) take(read8<D>(S + r.h + 8 * (size_t)i), bytes[i + 1]);
    if (tid < r.h) one(tid);
    if (tail + tid < V) one(tail + tid);  // fewer than 8 of each
    const float wm = mpb::wave_max(rest.m);
    const float wl = mpb::wave_sum(rest.l * __builtin_amdgcn_exp2f((rest.m - wm) * c));
    if ((tid & 63) == 0) red_m[wave] = wm, red_l[wave] = wl;
  }

  // the teacher's probabilities, by the first 4 waves (k entries at most 256)
  const bool with_rest = p.t_lse != nullptr;
  double y = 0.0, q = 0.0, L = 0.0;
  const double inv_tau = 1.0 / (double)p.tau;
  if (id >= 0) y = (double)p.teacher[(size_t)t * k + tid] * inv_tau;
  if (with_rest) {
    L = p.t_lse[t];
    if (id >= 0) q = exp(y - L);
  } else {  // over the entries themselves
    float m = id >= 0 ? (float)y : -INFINITY;
    if (wave < 4) {
      m = mpb::wave_max(m);
      if ((tid & 63) == 0) red_d[0][wave] = m;
    }
    __syncthreads();
    const int nw = nt >> 6;
    double top = red_d[0][0];
    for (int i = 1; i < 4 && i < nw; ++i) top = fmax(top, red_d[0][i]);
    if (id >= 0 && top > -INFINITY) q = exp(y - top);  // nothing but -inf: no entry counts
    const double e = wave_sum(q);
    if (wave < 4 && (tid & 63) == 0) red_d[1][wave] = e;
    __syncthreads();
    double sum = 0.0;
    for (int i = 0; i < 4 && i < nw; ++i) sum += red_d[1][i];
    if (sum > 0.0) q /= sum;
  }
  // entries of one id stand together: the first of them carries the sum
  if (tid < k) s_q[tid] = q;
  __syncthreads();
  bool first = id >= 0;
  if (s_dup && id >= 0) {
    q = 0.0;
    for (int j = 0; j < k; ++j) {
      if (s_ids[j] != id) continue;
      if (j < tid) first = false;
      q += s_q[j];
    }
  }
  if (!first) q = 0.0;

  // the row's sums: all of it, and without its entries
  float mr, lr, m, l;
  if constexpr (LOSS) {
    Running all;
    for (int i = 0; i < nt >> 6; ++i) all.join(red_m[i], red_l[i], c);
    mr = all.m;
    lr = all.l;
  } else {
    const fx4 v = *(const fx4*)(p.stats + 4 * (size_t)t);
    mr = v[0], lr = v[1], m = v[2], l = v[3];
  }
  __syncthreads();  // red_d is free again
  if (wave < 4) {
    const double sq = wave_sum(q), n = wave_sum(first ? 1.0 : 0.0);
    const float tm = mpb::wave_max(first ? st : -FLT_MAX);
    if ((tid & 63) == 0) red_d[0][wave] = sq, red_d[1][wave] = n, red_d[2][wave] = tm;
  }
  __syncthreads();
  double sq = 0.0, listed = 0.0;
  float tm = -FLT_MAX;
  for (int i = 0; i < 4 && i < nt >> 6; ++i) sq += red_d[0][i], listed += red_d[1][i], tm = fmaxf(tm, (float)red_d[2][i]);
  const bool unlisted = listed < (double)V;
  const double qr = with_rest && unlisted ? fmax(0.0, 1.0 - sq) : 0.0;
  if constexpr (LOSS) {
    m = fmaxf(mr, tm);
    __syncthreads();
    if (wave < 4) {
      const double e = wave_sum(first ? exp(((double)st - (double)m) * inv_tau) : 0.0);
      if ((tid & 63) == 0) red_d[0][wave] = e;
    }
    __syncthreads();
    double sum = (double)lr * exp(((double)mr - (double)m) * inv_tau);
    for (int i = 0; i < 4 && i < nt >> 6; ++i) sum += red_d[0][i];
    l = (float)sum;
    // kl, with log p = (s - m) / tau - log l
    double kl = 0.0;
    if (q > 0.0) kl = q * (log(q) - (((double)st - (double)m) * inv_tau - log(sum)));
    else if (q != q) kl = q;
    __syncthreads();
    if (wave < 4) {
      kl = wave_sum(kl);
      if ((tid & 63) == 0) red_d[0][wave] = kl;
    }
    __syncthreads();
    if (tid == 0) {
      kl = 0.0;
      for (int i = 0; i < 4 && i < nt >> 6; ++i) kl += red_d[0][i];
      if (qr > 0.0) kl += qr * (log(qr) - (((double)mr - (double)m) * inv_tau + log((double)lr) - log(sum)));
      if (sum == 0.0) kl = 0.0;  // every logit is -inf: the row takes no part
      p.kl[t] = (float)kl;
      *(fx4*)(p.stats + 4 * (size_t)t) = fx4{mr, lr, m, l};
    }
  }

  if constexpr (GRAD) {
    const float scale = l == 0.0f ? 0.0f : w * p.tau * (p.gloss ? *p.gloss : 1.0f);
    const double Q = sq + qr;
    // p_v (Q - q_r / p_r) = exp((s - mr) / tau) (Q p_r - q_r) / lr
    const double pr = (double)lr / (double)l * exp(((double)mr - (double)m) * inv_tau);
    const float coef = lr == 0.0f ? 0.0f : scale * (float)((Q * pr - qr) / (double)lr);
    if (first) {
      const double pv = exp(((double)st - (double)m) * inv_tau) / (double)l;
      dS[id] = (elem)(l == 0.0f ? 0.0f : scale * (float)(pv * Q - q));
    }
    auto put = [&](int i, fx8 x) {
      const unsigned skip = bytes[i + 1];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = coef * __builtin_amdgcn_exp2f((x[j] - mr) * c);
      elem* d = dS + r.h + 8 * (size_t)i;
      if (!skip) {
        write8<D>(d, x);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!(skip >> j & 1)) d[j] = (elem)x[j];
      }
    };
    auto one = [&](int v) {
      const int b = bit_of(r, v);
      if (!(bits[b >> 5] >> (b & 31) & 1)) dS[v] = (elem)(coef * __builtin_amdgcn_exp2f(((float)S[v] - mr) * c));
    };
    constexpr int U = 4;
    int i = tid;
    for (; i + (U - 1) * nt < r.nv; i += U * nt) {
      fx8 x[U];
#pragma unroll
      for (int j = 0; j < U; ++j) x[j] = read8<D>(S + r.h + 8 * (size_t)(i + j * nt));
#pragma unroll
      for (int j = 0; j < U; ++j) put(i + j * nt, x[j]);
    }
    for (; i < r.nv; i += nt) put(i, read8<D>(S + r.h + 8 * (size_t)i));
    if (tid < r.h) one(tid);
    if (tail + tid < V) one(tail + tid);
  }
}

// loss = tau^2 sum_t w_t kl_t, in fp64 and a fixed order, by one workgroup.
__global__ __launch_bounds__(1024) void k_distill_sum(DistillParams p) {
  __shared__ double red[16];
  const int tid = threadIdx.x;
  double s = 0.0;
  for (int t = tid; t < p.T; t += 1024) {
    const float w = p.weight ? p.weight[t] : 1.0f / (float)p.T;
    if (w != 0.0f) s += (double)w * (double)p.kl[t];
  }
  s = wave_sum(s);
  if ((tid & 63) == 0) red[tid >> 6] = s;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < 16; ++i) s += red[i];
    *p.loss = (float)(s * (double)p.tau * (double)p.tau);
  }
}

template <class D>
hipError_t launch(const DistillParams& p, bool loss, hipStream_t s) {
  if (p.T > 0) {
    // 8 vectors a thread at the longest rows, whole waves, 4 of them at least (256 entries)
    const int n = (p.V + 63) / 64, nt = n >= 1024 ? 1024 : n <= 256 ? 256 : (n + 63) / 64 * 64;
    const size_t lds = 4 * (size_t)p.words;
    auto* k = loss ? (p.dS ? k_distill<D, true, true> : k_distill<D, true, false>) : k_distill<D, false, true>;
    k<<<p.T, nt, lds, s>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (loss) k_distill_sum<<<1, 1024, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_distill(DistillParams p, int dtype, bool loss, hipStream_t s) {
  p.words = (p.V + 16 + 31) / 32;
  return dtype == MPB_F32 ? launch<F32>(p, loss, s) : dtype == MPB_BF16 ? launch<BF16>(p, loss, s) : launch<F16>(p, loss, s);
}

}  // namespace mpb
