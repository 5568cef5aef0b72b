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
// entry (so that p_r is a sum of its own, not 1 minus the rest). The entries belong to
// wave 0, four a lane, which forms the teacher's side while the others read; the
// logarithms are differences of logits, and they and the sums over the entries are fp64.
// Nothing is written twice: the pass over the row leaves the entries out, and each
// entry's lane writes its own.
//
// The loss alone is bound by HBM (1021 x 65536 fp16 29 us, 4.7 TB/s). With the gradient a row is
// read twice, the second time backwards and mostly from the Infinity Cache, and
// written once: 2048 x 151677 bf16 296 us, 4.2 TB/s of one read and the write (302
// forwards). 9 x 32003 fp32 takes 7.4 + 1.6 us, a chain of latencies; a wave each for
// every step of the end of a row, with eight barriers and fp64 exponentials, took 10.3.
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

template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xf, 0xf, true);
  const uint32_t hi = __builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CTRL, 0xf, 0xf, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Over the wave, the same bits in every lane (see wave_all).
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp<0xb1>(v);
  v += dpp<0x4e>(v);
  v += dpp<0x141>(v);
  v += dpp<0x140>(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
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

constexpr int kPerLane = kDistillMaxK / 64;  // entries of a lane of wave 0

template <class D, bool LOSS, bool GRAD>
__global__ __launch_bounds__(1024, 8) void k_distill(DistillParams p) {
  typedef typename D::elem elem;
  extern __shared__ uint32_t bits[];
  __shared__ float red_m[16], red_l[16], s_coef, s_mr;
  // the entries' while the row is read (registers would cost the second workgroup of a CU)
  __shared__ int s_ids[kDistillMaxK];
  __shared__ float s_st[kDistillMaxK];
  __shared__ double s_q[kDistillMaxK], s_lq[kDistillMaxK];
  __shared__ int s_dup;
  const int tid = threadIdx.x, nt = blockDim.x, wave = tid >> 6, lane = tid & 63, t = blockIdx.x, V = p.V, k = p.k;
  const elem* S = (const elem*)p.S + (size_t)t * p.ld;
  elem* dS = GRAD ? (elem*)p.dS + (size_t)t * p.ld : nullptr;
  const Row r = row_of<D>(S, V);
  const int tail = r.h + 8 * r.nv;  // first element after the vectors
  const float w = p.weight ? p.weight[t] : 1.0f / (float)p.T;
  int id[kPerLane];
  float yt[kPerLane];
  if (wave == 0) {
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) {
      const int j = lane + 64 * e;
      id[e] = -1;
      yt[e] = 0.0f;
      if (j < k) {
        id[e] = p.ids[(size_t)t * k + j];
        yt[e] = p.teacher[(size_t)t * k + j];
        if ((unsigned)id[e] >= (unsigned)V) id[e] = -1;
      }
    }
  }

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
  if (wave == 0) {
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) {
      s_ids[lane + 64 * e] = id[e];
      if (id[e] < 0) continue;
      s_st[lane + 64 * e] = (float)S[id[e]];
      const int b = bit_of(r, id[e]);
      if (atomicOr(&bits[b >> 5], 1u << (b & 31)) >> (b & 31) & 1) s_dup = 1;
    }
  }
  __syncthreads();
  const uint8_t* bytes = (const uint8_t*)bits;
  const float c = kLog2e / p.tau;
  const double inv_tau = 1.0 / (double)p.tau;

  // the teacher's side, by wave 0: q and log q of every id once (its first entry has the
  // sum of all of them), their sum and number
  const bool with_rest = p.t_lse != nullptr;
  if (wave == 0) {
    double q[kPerLane], lq[kPerLane], L = with_rest ? (double)p.t_lse[t] : 0.0;
    if (!with_rest) {  // over the entries themselves
      float top = -INFINITY;
#pragma unroll
      for (int e = 0; e < kPerLane; ++e)
        if (id[e] >= 0) top = fmaxf(top, yt[e]);
      top = mpb::wave_max(top);
      double sum = 0.0;
#pragma unroll
      for (int e = 0; e < kPerLane; ++e)
        if (id[e] >= 0 && top > -INFINITY) sum += expf((float)(((double)yt[e] - (double)top) * inv_tau));
      L = (double)top * inv_tau + log(wave_sum(sum));
    }
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) {
      lq[e] = (double)yt[e] * inv_tau - L;
      q[e] = id[e] >= 0 && yt[e] != -INFINITY ? (double)expf((float)lq[e]) : 0.0;
      s_q[lane + 64 * e] = q[e];
    }
    if (s_dup) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      bool first[kPerLane];
#pragma unroll
      for (int e = 0; e < kPerLane; ++e) {
        first[e] = true;
        if (id[e] < 0) continue;
        q[e] = 0.0;
        for (int j = 0; j < k; ++j) {
          if (s_ids[j] != id[e]) continue;
          if (j < lane + 64 * e) first[e] = false;
          q[e] += s_q[j];
        }
        lq[e] = log(q[e]);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();  // every lane has read the ids and sums
#pragma unroll
      for (int e = 0; e < kPerLane; ++e) {
        if (!first[e]) s_ids[lane + 64 * e] = -1, q[e] = 0.0;
        s_q[lane + 64 * e] = q[e];
      }
    }
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) s_lq[lane + 64 * e] = lq[e];
  }

  // the row without its entries
  if constexpr (LOSS) {
    Running rest;
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
    if (lane == 0) red_m[wave] = wm, red_l[wave] = wl;
    __syncthreads();
  }

  // the row's sums and results, by wave 0
  if (wave == 0) {
    float mr, lr, m, l, st[kPerLane];
    double q[kPerLane], lq[kPerLane], sq = 0.0;
    int listed = 0;
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) {
      const int j = lane + 64 * e;
      id[e] = s_ids[j];
      q[e] = s_q[j];
      lq[e] = s_lq[j];
      st[e] = id[e] < 0 ? -FLT_MAX : s_st[j];
      sq += q[e];
      listed += __popcll(__ballot(id[e] >= 0));
    }
    sq = wave_sum(sq);
    const double qr = with_rest && listed < V ? fmax(0.0, 1.0 - sq) : 0.0;
    if constexpr (LOSS) {
      const bool on = lane < nt >> 6;
      const float wm = on ? red_m[lane] : -FLT_MAX;
      mr = mpb::wave_max(wm);
      lr = mpb::wave_sum(on ? red_l[lane] * __builtin_amdgcn_exp2f((wm - mr) * c) : 0.0f);
      float tm = -FLT_MAX;
#pragma unroll
      for (int e = 0; e < kPerLane; ++e) tm = fmaxf(tm, st[e]);
      m = fmaxf(mr, mpb::wave_max(tm));
      double sum = 0.0;
#pragma unroll
      for (int e = 0; e < kPerLane; ++e)
        if (id[e] >= 0) sum += expf((float)(((double)st[e] - (double)m) * inv_tau));
      sum = wave_sum(sum) + (double)lr * expf((float)(((double)mr - (double)m) * inv_tau));
      l = (float)sum;
      // log p = (s - m) / tau - log(sum)
      const double ls = log(sum);
      double kl = 0.0;
#pragma unroll
      for (int e = 0; e < kPerLane; ++e) {
        if (q[e] > 0.0) kl += q[e] * (lq[e] - (((double)st[e] - (double)m) * inv_tau - ls));
        else if (q[e] != q[e]) kl = q[e];
      }
      kl = wave_sum(kl);
      if (qr > 0.0) kl += qr * (log(qr) - (((double)mr - (double)m) * inv_tau + log((double)lr) - ls));
      if (sum == 0.0) kl = 0.0;  // every logit is -inf: the row takes no part
      if (lane == 0) {
        p.kl[t] = (float)kl;
        *(fx4*)(p.stats + 4 * (size_t)t) = fx4{mr, lr, m, l};
      }
    } else {
      const fx4 v = *(const fx4*)(p.stats + 4 * (size_t)t);
      mr = v[0], lr = v[1], m = v[2], l = v[3];
    }
    if constexpr (GRAD) {
      const float scale = l == 0.0f ? 0.0f : w * p.tau * (p.gloss ? *p.gloss : 1.0f);
      const double Q = sq + qr;
      // p_v (Q - q_r / p_r) = exp((s - mr) / tau) (Q p_r - q_r) / lr
      const double pr = (double)lr / (double)l * exp(((double)mr - (double)m) * inv_tau);
      if (lane == 0) {
        s_coef = lr == 0.0f ? 0.0f : scale * (float)((Q * pr - qr) / (double)lr);
        s_mr = mr;
      }
#pragma unroll
      for (int e = 0; e < kPerLane; ++e) {
        if (id[e] < 0) continue;
        const double pv = (double)expf((float)(((double)st[e] - (double)m) * inv_tau)) / (double)l;
        dS[id[e]] = (elem)(l == 0.0f ? 0.0f : scale * (float)(pv * Q - q[e]));
      }
    }
  }

  if constexpr (GRAD) {
    __syncthreads();
    const float coef = s_coef, mr = s_mr;
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
    // backwards: what was read last is nearest
    constexpr int U = 4;
    int i = r.nv - 1 - tid;
    for (; i - (U - 1) * nt >= 0; i -= U * nt) {
      fx8 x[U];
#pragma unroll
      for (int j = 0; j < U; ++j) x[j] = read8<D>(S + r.h + 8 * (size_t)(i - j * nt));
#pragma unroll
      for (int j = 0; j < U; ++j) put(i - j * nt, x[j]);
    }
    for (; i >= 0; i -= nt) put(i, read8<D>(S + r.h + 8 * (size_t)i));
    if (tid < r.h) one(tid);
    if (tail + tid < V) one(tail + tid);
  }
}

// loss = tau^2 sum_t w_t kl_t, in fp64 and a fixed order, by one workgroup.
__global__ __launch_bounds__(1024) void k_distill_sum(DistillParams p) {
  __shared__ double red[16];
  const int tid = threadIdx.x;
  double s = 0.0;
#pragma unroll 4
  for (int t = tid; t < p.T; t += 1024)  // kl is 0 where the weight is
    s += (double)(p.weight ? p.weight[t] : 1.0f / (float)p.T) * (double)p.kl[t];
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
    // Up to 512 threads, four rows a CU, which hide each other's ends (1021 x 65536 fp16:
    // loss 34 us, 44 with 1024); 1024 where there are no four rows for every CU, or where
    // the gradient's second reading would not find them in the 256 MB Infinity Cache (2048 x
    // 151677 bf16 with the gradient: 294 us with 1024 threads, 334 with 512). The loss alone
    // takes as many threads as with its gradient, so that its bits are the same (2048 x 151677
    // bf16 105 us with 1024, 110 with 512; 700 x 250001 68 and 64).
    const bool wide = p.T <= 512 || (loss && (double)p.V * sizeof(typename D::elem) * 1024 > 2e8);
    const int n = (p.V + 31) / 32, most = wide ? 1024 : 512, nt = n >= most ? most : n <= 256 ? 256 : (n + 63) / 64 * 64;
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
