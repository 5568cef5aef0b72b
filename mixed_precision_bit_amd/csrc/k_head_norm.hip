// Norms of query and key heads with their position rotation, in one pass, and the
// backward pass.
//
//   n = x rms(x) gamma           over the D elements of a head (n = x without gamma)
//   (a, b) -> (a cos f - b sin f, a sin f + b cos f)   for the pairs of the first Dr elements,
//   f = pos[axis_i][t] freq_i    for pair i
//
// A lane holds 16 elements of a head: 8 pairs, so both partners of a rotation are
// in one lane, and NL lanes hold a head (the smallest power of two for D / 16).
// A wave takes a token and works through its heads, 64 / NL at a time: the 8
// angles of a lane are the same for all of them and are formed once, as turns in
// fp64 (a position of 2^20 times a frequency keeps 2^-33 of a turn; an fp32
// product is off by 2^-7 turns there). Few tokens: the heads of a token go to
// several waves. Everything else is fp32, each output rounded once.
// Bound by HBM: 4093 tokens of 40 heads of 128, bf16, three axes, 18.7 us (4.5 TB/s of
// the 5.2 that a large copy reaches; 21.6 without streaming stores); 64 tokens of 32 heads 4.8, most of it
// the launch.
//
// Backward: d = the rotation by -f of the output's gradient, then the norm's
//   dx = rms(x) (d gamma - xh mean(d gamma xh)),  xh = x rms(x);  dgamma = sum d xh
// dgamma stays in registers over a workgroup's tokens and heads, one partial row
// a workgroup, added in workgroup order (no float atomics). 8192 tokens of 24 heads of
// 256: 68 + 4.9 us, 4.4 TB/s. A wave loads its next group before it works on one (75
// us without), which takes 138 registers: three workgroups a CU, and no more are launched (87 us
// with a fourth waiting).
#include "k_block_common.h"
#include "mpb.h"
#include "mpb_internal.h"

namespace mpb {

namespace {

// Sum over the NL consecutive lanes that hold a head, in every one of them.
template <int NL>
__device__ __forceinline__ float head_sum(float v) {
  if constexpr (NL >= 2) v += dpp<0xb1>(v);
  if constexpr (NL >= 4) v += dpp<0x4e>(v);
  if constexpr (NL >= 8) v += dpp<0x141>(v);
  if constexpr (NL >= 16) v += dpp<0x140>(v);
  if constexpr (NL >= 32) v += __shfl_xor(v, 16);
  return v;
}

__device__ __forceinline__ float sum_sq(const fx8& a, const fx8& b) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += a[i] * a[i] + b[i] * b[i];
  return s;
}

__device__ __forceinline__ float dot(const fx8& a, const fx8& b, const fx8& c, const fx8& d) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += a[i] * c[i] + b[i] * d[i];
  return s;
}

// Where lane p of a head finds its two vectors of 8. Pairs in halves: 8 elements
// of the rotated part's first half and their partners in its second. Neighbours
// as pairs, and what is not rotated: 16 consecutive elements.
__device__ __forceinline__ void lane_offsets(const HeadNormParams& p, int l, int& a, int& b) {
  const bool halves = p.pairs == MPB_PAIRS_HALVES && 16 * l < p.Dr;
  a = halves ? 8 * l : 16 * l;
  b = halves ? p.Dr / 2 + 8 * l : 16 * l + 8;
}

// cos and sin of the 8 angles of lane p at token t (1 and 0 for what is not rotated).
__device__ __forceinline__ void lane_angles(const HeadNormParams& p, int l, int t, fx8& cs, fx8& sn) {
  cs = (fx8)(1.0f);
  sn = (fx8)(0.0f);
  if (16 * l >= p.Dr) return;
  const fx8 f = load8(p.freq + 8 * l);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int axis = p.axis ? p.axis[8 * l + i] : 0;
    const int pos = (unsigned)axis < (unsigned)p.A ? p.pos[(size_t)axis * p.T + t] : 0;
    // in turns; the fraction is exact
    const double turns = (double)pos * (double)f[i] * 0.15915494309189535;
    float s, c;
    sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
    cs[i] = c;
    sn[i] = s;
  }
}

// The rotation of a lane's 8 pairs: (a_i, b_i), or neighbours within a and within b.
template <bool HALVES>
__device__ __forceinline__ void turn(fx8& a, fx8& b, const fx8& cs, const fx8& sn) {
  if constexpr (HALVES) {
    const fx8 x = a * cs - b * sn, y = a * sn + b * cs;
    a = x;
    b = y;
  } else {
    fx8 x = a, y = b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = a[2 * i] * cs[i] - a[2 * i + 1] * sn[i];
      x[2 * i + 1] = a[2 * i] * sn[i] + a[2 * i + 1] * cs[i];
      y[2 * i] = b[2 * i] * cs[4 + i] - b[2 * i + 1] * sn[4 + i];
      y[2 * i + 1] = b[2 * i] * sn[4 + i] + b[2 * i + 1] * cs[4 + i];
    }
    a = x;
    b = y;
  }
}

constexpr int kWaves = 4;  // waves of a workgroup, each with an item of its own

// Item (token, part): the wave's token and its groups of 64 / NL heads. The
// groups of the query heads come first, then those of the key heads.
struct Groups {
  int nq, nk;  // groups of each side
};
template <int NL>
__device__ __forceinline__ Groups groups(const HeadNormParams& p) {
  constexpr int HG = 64 / NL;
  return {(p.Hq + HG - 1) / HG, (p.Hk + HG - 1) / HG};
}

template <class D, int NL, bool HALVES>
__global__ __launch_bounds__(64 * kWaves) void k_head_norm(HeadNormParams p) {
  typedef typename D::vec vec;
  typedef typename D::elem elem;
  constexpr int HG = 64 / NL;
  const int lane = threadIdx.x & 63, l = lane & (NL - 1);
  const int64_t item = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (item >= (int64_t)p.T * p.parts) return;
  const int t = (int)(item / p.parts), part = (int)(item - (int64_t)t * p.parts);
  const bool mine = 16 * l < p.D;
  const Groups n = groups<NL>(p);
  int oa, ob;
  lane_offsets(p, l, oa, ob);
  fx8 cs, sn;
  if (mine) lane_angles(p, l, t, cs, sn);
  const float inv_d = 1.0f / (float)p.D;
  for (int g = part; g < n.nq + n.nk; g += p.parts) {
    const bool key = g >= n.nq;
    const int h = (key ? g - n.nq : g) * HG + lane / NL;
    const bool on = mine && h < (key ? p.Hk : p.Hq);
    const float* gamma = key ? p.g_k : p.g_q;
    const size_t in = (size_t)t * (key ? p.k_ld : p.q_ld) + (size_t)h * p.D;
    const elem* src = (const elem*)(key ? p.k : p.q);
    fx8 a = (fx8)(0.0f), b = (fx8)(0.0f);
    if (on) {
      a = widen<D>(*(const vec*)(src + in + oa));
      b = widen<D>(*(const vec*)(src + in + ob));
    }
    if (gamma) {
      const float r = rsqrtf(head_sum<NL>(sum_sq(a, b)) * inv_d + p.eps);
      if (on) {
        a *= r * load8(gamma + oa);
        b *= r * load8(gamma + ob);
      }
    }
    if (on) {
      if (16 * l < p.Dr) turn<HALVES>(a, b, cs, sn);
      const size_t out = (size_t)t * (key ? p.ko_ld : p.qo_ld) + (size_t)h * p.D;
      elem* dst = (elem*)(key ? p.k_out : p.q_out);
      stream_store((vec*)(dst + out + oa), narrow<D>(a));
      stream_store((vec*)(dst + out + ob), narrow<D>(b));
    }
  }
}

// Adds a lane's 16 sums of gamma's gradient over the lanes of the wave that hold
// the same elements, and the workgroup's waves, into one partial row.
template <int NL>
__device__ __forceinline__ void store_dgamma(const fx8& a, const fx8& b, float* row, int D, int oa, int ob, int l, float* lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float v[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = a[i], v[8 + i] = b[i];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
#pragma unroll
    for (int m = NL; m < 64; m *= 2) v[i] += __shfl_xor(v[i], m);
  }
  if (lane < NL) {
#pragma unroll
    for (int i = 0; i < 16; ++i) lds[(wave * NL + l) * 16 + i] = v[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < NL * 16; i += 64 * kWaves) {
    float s = lds[i];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) s += lds[w * NL * 16 + i];
    lds[i] = s;  // no other thread reads this wave-0 entry
  }
  __syncthreads();
  if (wave == 0 && lane < NL && 16 * l < D) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      row[oa + i] = lds[l * 16 + i];
      row[ob + i] = lds[l * 16 + 8 + i];
    }
  }
  __syncthreads();
}

// A wave's share of one group of heads as loaded: the gradient's and x's two vectors.
template <class D>
struct GradGroup {
  typename D::vec a, b, xa, xb;
};

template <class D, int NL, bool HALVES>
__global__ __launch_bounds__(64 * kWaves, 3) void k_head_norm_grad(HeadNormGradParams q) {
  typedef typename D::vec vec;
  typedef typename D::elem elem;
  constexpr int HG = 64 / NL;
  __shared__ float lds[kWaves * NL * 16];
  const HeadNormParams& p = q.f;
  const int lane = threadIdx.x & 63, l = lane & (NL - 1);
  const bool mine = 16 * l < p.D;
  const Groups n = groups<NL>(p);
  int oa, ob;
  lane_offsets(p, l, oa, ob);
  const float inv_d = 1.0f / (float)p.D;
  fx8 gqa = (fx8)(0.0f), gqb = gqa, gka = gqa, gkb = gqa;
  const int64_t items = (int64_t)p.T * p.parts, step = (int64_t)gridDim.x * kWaves;
  int64_t item = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  int t = 0, g = 0;
  auto begin = [&]() {
    t = (int)(item / p.parts);
    g = (int)(item - (int64_t)t * p.parts);
  };
  auto head = [&](int g, bool& key, bool& on) {
    key = g >= n.nq;
    const int h = (key ? g - n.nq : g) * HG + lane / NL;
    on = mine && h < (key ? p.Hk : p.Hq);
    return h;
  };
  auto load = [&](GradGroup<D>& v, int t, int g) {
    bool key, on;
    const int h = head(g, key, on);
    v.a = v.b = v.xa = v.xb = (vec)(0);
    if (!on) return;
    const size_t at = (size_t)t * (key ? p.ko_ld : p.qo_ld) + (size_t)h * p.D;
    const elem* d = (const elem*)(key ? q.dk_out : q.dq_out);
    v.a = *(const vec*)(d + at + oa);
    v.b = *(const vec*)(d + at + ob);
    if (key ? p.g_k : p.g_q) {
      const size_t in = (size_t)t * (key ? p.k_ld : p.q_ld) + (size_t)h * p.D;
      const elem* x = (const elem*)(key ? p.k : p.q);
      v.xa = *(const vec*)(x + in + oa);
      v.xb = *(const vec*)(x + in + ob);
    }
  };
  GradGroup<D> next;
  fx8 cs, sn;
  bool fresh = true;  // a token's first group
  if (item < items) {
    begin();
    load(next, t, g);
  }
  while (item < items) {
    const GradGroup<D> now = next;
    const int ti = t, gi = g;
    const bool first = fresh;
    // the next group's loads go out before this one is worked on
    g += p.parts;
    fresh = g >= n.nq + n.nk;
    if (fresh) {
      item += step;
      if (item < items) begin();
    }
    if (item < items) load(next, t, g);
    if (first && mine) lane_angles(p, l, ti, cs, sn);
    bool key, on;
    const int h = head(gi, key, on);
    const float* gamma = key ? p.g_k : p.g_q;
    fx8 a = widen<D>(now.a), b = widen<D>(now.b);
    if (on && 16 * l < p.Dr) turn<HALVES>(a, b, cs, -sn);
    if (gamma) {
      fx8 xa = widen<D>(now.xa), xb = widen<D>(now.xb);
      const float r = rsqrtf(head_sum<NL>(sum_sq(xa, xb)) * inv_d + p.eps);
      xa *= r;
      xb *= r;
      if (key) {
        gka += a * xa;
        gkb += b * xb;
      } else {
        gqa += a * xa;
        gqb += b * xb;
      }
      if (on) {
        a *= load8(gamma + oa);
        b *= load8(gamma + ob);
      }
      const float m = head_sum<NL>(dot(a, b, xa, xb)) * inv_d;
      a = r * (a - xa * m);
      b = r * (b - xb * m);
    }
    if (on) {
      const size_t out = (size_t)ti * (key ? q.dk_ld : q.dq_ld) + (size_t)h * p.D;
      elem* dst = (elem*)(key ? q.dk : q.dq);
      stream_store((vec*)(dst + out + oa), narrow<D>(a));
      stream_store((vec*)(dst + out + ob), narrow<D>(b));
    }
  }
  if (q.dg_q) store_dgamma<NL>(gqa, gqb, q.part + (size_t)blockIdx.x * p.D, p.D, oa, ob, l, lds);
  if (q.dg_k) store_dgamma<NL>(gka, gkb, q.part + ((size_t)gridDim.x + blockIdx.x) * p.D, p.D, oa, ob, l, lds);
}

// dgamma = the sum of the workgroups' partial rows, in a fixed order: 16 waves
// take every 16th row of 64 columns, then wave 0 adds the 16 sums.
__global__ __launch_bounds__(1024) void k_dgamma(HeadNormGradParams q, int rows) {
  __shared__ float lds[16][64];
  const int side = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float* dg = side ? q.dg_k : q.dg_q;
  if (!dg) return;
  const int D = q.f.D, c = blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < D) {
    const float* part = q.part + (size_t)side * rows * D + c;
#pragma unroll 8
    for (int r = wave; r < rows; r += 16) s += part[(size_t)r * D];
  }
  lds[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < D) {
    for (int w = 1; w < 16; ++w) s += lds[w][lane];
    dg[c] = s;
  }
}

template <class D, int NL>
void launch_nl(const HeadNormParams& p, hipStream_t s) {
  const int64_t blocks = ((int64_t)p.T * p.parts + kWaves - 1) / kWaves;
  if (p.pairs == MPB_PAIRS_HALVES)
    k_head_norm<D, NL, true><<<(unsigned)blocks, 64 * kWaves, 0, s>>>(p);
  else
    k_head_norm<D, NL, false><<<(unsigned)blocks, 64 * kWaves, 0, s>>>(p);
}

template <class D, int NL>
void launch_grad_nl(const HeadNormGradParams& p, int blocks, hipStream_t s) {
  if (p.f.pairs == MPB_PAIRS_HALVES)
    k_head_norm_grad<D, NL, true><<<blocks, 64 * kWaves, 0, s>>>(p);
  else
    k_head_norm_grad<D, NL, false><<<blocks, 64 * kWaves, 0, s>>>(p);
}

int lanes_of(int D) {
  int nl = 1;
  while (nl * 16 < D) nl *= 2;
  return nl;
}

// Waves that share a token's heads: as many as bring the launch to 2048 waves (8
// a CU), at most one group of heads each.
int parts_of(int T, int Hq, int Hk, int D) {
  const int hg = 64 / lanes_of(D), n = (Hq + hg - 1) / hg + (Hk + hg - 1) / hg;
  const int want = (2048 + T - 1) / (T > 0 ? T : 1);
  return want < n ? want : n;
}

#define MPB_HEADS(CALL)                                                                                     \
  switch (lanes_of(D)) {                                                                                    \
    case 1: CALL(1); break;                                                                                 \
    case 2: CALL(2); break;                                                                                 \
    case 4: CALL(4); break;                                                                                 \
    case 8: CALL(8); break;                                                                                 \
    case 16: CALL(16); break;                                                                               \
    default: CALL(32); break;                                                                               \
  }

}  // namespace

int head_norm_grad_groups(int T, int Hq, int Hk, int D) {
  const int64_t blocks = ((int64_t)T * parts_of(T, Hq, Hk, D) + kWaves - 1) / kWaves;
  return (int)(blocks < 768 ? blocks : 768);  // three a CU are resident
}

hipError_t launch_head_norm(HeadNormParams p, bool bf16, hipStream_t s) {
  const int D = p.D;
  p.parts = parts_of(p.T, p.Hq, p.Hk, D);
#define MPB_FWD(NL) (bf16 ? launch_nl<BF16, NL>(p, s) : launch_nl<F16, NL>(p, s))
  MPB_HEADS(MPB_FWD)
#undef MPB_FWD
  return hipGetLastError();
}

hipError_t launch_head_norm_grad(HeadNormGradParams p, bool bf16, hipStream_t s) {
  const int D = p.f.D;
  p.f.parts = parts_of(p.f.T, p.f.Hq, p.f.Hk, D);
  const int blocks = p.f.T > 0 ? head_norm_grad_groups(p.f.T, p.f.Hq, p.f.Hk, D) : 0;
  if (blocks > 0) {
#define MPB_BWD(NL) (bf16 ? launch_grad_nl<BF16, NL>(p, blocks, s) : launch_grad_nl<F16, NL>(p, blocks, s))
    MPB_HEADS(MPB_BWD)
#undef MPB_BWD
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (p.dg_q || p.dg_k) k_dgamma<<<dim3((D + 63) / 64, 2), 1024, 0, s>>>(p, blocks);
  return hipGetLastError();
}

}  // namespace mpb
