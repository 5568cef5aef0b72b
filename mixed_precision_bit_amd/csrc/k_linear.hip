// Matrix products with bias, activation and residual in their epilogue, and their
// gradients.
//
//   z = X W^T + bias,  y = res + act(z)              X [T][Kd], W [N][Kd]
//   dz = dy act'(z);  dX = dz W;  dW = dz^T X;  dbias = sum_t dz
//
// One product kernel, C[m][n] = sum_k A(m, k) B(n, k), for all three: an operand
// lies with its reduction contiguous (X and W forward, dz in dX) or as the rows of
// the other index (W in dX, dz and X in dW), which LDS's transposing reads turn on
// the way into the registers. Stages of 32 of the reduction go straight from memory to
// LDS, four in flight, and a wave holds its part of the output in registers and
// multiplies 16 x 16 x 32 at a time. Accumulation is fp32, every sum has a fixed
// order (reductions split over workgroups leave partial sums that a second launch
// adds in order).
//
// Large products are bound by the matrix cores under the card's power (they are busy 65 %
// of dX's cycles): 8192 x 4096 x 4096 bf16 takes dX 200 us and dW 203, 1.37 and 1.35 PFLOP/s,
// after 200 passes that settle the clock; a library product of those layouts takes 200
// and 223 (with bf16 dW), the forward one 174 where this takes 202, and one of 8192^3 reaches
// 1.64 PFLOP/s where this reaches 1.34. Figures that compare two variants of this file are of a
// few passes, 5 to 13 % longer. What did not help, against dX of 221 to 227 at the time: one
// buffer of 64 ahead instead of four of 32 (236), reads interleaved with the products in
// every wave instead of halves of the waves in turn (232), waves of 128 x 128, one a SIMD
// (252), two workgroups of 128 x 256 a CU with three buffers each (312).
//
// A batch of few tokens reads W once and has little to share: k_skinny, W straight
// into the registers.
//
// dz is formed once for both gradients. Where it is not exactly dy (an activation, or
// fp32 dy) it becomes fp16 parts, whatever the activations are, scaled by a power of two
// that brings the largest value to 2^13 (the gradients of a mean, below fp16's range,
// keep their bits): two parts, of 22 bits together, for dX and dW alike. bf16 X and W become
// scaled fp16 beside them. dX could do with one part half the time, but not with its 11 bits:
// fp16 dX would be 2.9e-4 of its norm off, its own rounding being 2.1e-4, and bf16 dX
// 8.6e-4 of its norm from the product of the unrounded dz.
// bf16 parts cost the same and lose more: dW 2.6e-6 with two instead of 7e-7 (an fp32
// library product: 1.2e-6; 4093 tokens).
#include <type_traits>

#include "k_block_common.h"
#include "mpb.h"
#include "mpb_internal.h"

namespace mpb {

namespace {

typedef short sx4 __attribute__((ext_vector_type(4)));
typedef short sx8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) void lds_void;

template <class D>
__device__ __forceinline__ acc4 product(typename D::vec a, typename D::vec b, acc4 c);
template <>
__device__ __forceinline__ acc4 product<F16>(hx8 a, hx8 b, acc4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
template <>
__device__ __forceinline__ acc4 product<BF16>(bx8 a, bx8 b, acc4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// ---------------------------------------------------------------- activations
constexpr float kSqrtHalf = 0.707106781f, kInvSqrt2Pi = 0.398942280f;
constexpr float kTanhA = 0.797884561f, kTanhB = 0.044715f;  // sqrt(2 / pi)

// For results of 16 bits: within (6 + |x|) 2^-24 of itself (the roundings of the exponent, the
// exponential and the reciprocal), in half the operations: 4093 x 5632 x 2816 with silu,
// residual and z 136 us, 143 with the other. Below -88.7, where sigmoid is under 2^-128,
// the exponential overflows and this is 0.
__device__ __forceinline__ float sigmoid16(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269502f * x));
}

// Phi(-a) for a >= 0, given e = exp(-a^2 / 2): e t Q(t) with t = 1 / (1 + C a), where
// Phi(-a) / (e t) is so smooth in t that a polynomial of degree 8, fitted for the least
// largest relative error over a in [0, 20], stays within 2^-25 of it. With the
// roundings of fp32 it is within (18 + 1.1 a^2) 2^-24 of itself, up to 13, where e leaves the
// range of fp32. dz of 4093 x 2816 24 us, 36 to 40 with erfcf; 4093 x 5632 x 2816
// forward with gelu, residual and z 141, 156 with it.
__device__ __forceinline__ float normal_tail(float a, float e) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.268700570f, a, 1.0f));
  float q = fmaf(0.0290484875f, t, -0.129195794f);
  q = fmaf(q, t, 0.178268000f);
  q = fmaf(q, t, -0.0769507661f);
  q = fmaf(q, t, 0.112688191f);
  q = fmaf(q, t, 0.0701929182f);
  q = fmaf(q, t, 0.101762444f);
  q = fmaf(q, t, 0.106982090f);
  q = fmaf(q, t, 0.107204415f);
  return e * (t * q);
}
// exp(-z^2 / 2)
__device__ __forceinline__ float bell(float z) { return __builtin_amdgcn_exp2f(-0.721347520f * (z * z)); }

// gelu_tanh is z sigmoid(2 u), u = a (z + b z^3): 1 + tanh(u) = 2 sigmoid(2 u),
// which keeps its relative accuracy where tanh is close to -1.
template <bool NARROW>
__device__ __forceinline__ float act_of(float z, int act) {
  auto sig = [](float x) { return NARROW ? sigmoid16(x) : sigmoid(x); };
  switch (act) {
    case MPB_ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
    case MPB_ACT_SILU: return z * sig(z);
    case MPB_ACT_GELU: {
      if constexpr (!NARROW) return 0.5f * z * erfcf(-z * kSqrtHalf);
      const float tail = normal_tail(fabsf(z), bell(z));
      return z * (z > 0.0f ? 1.0f - tail : tail);
    }
    case MPB_ACT_GELU_TANH: return z * sig(2.0f * kTanhA * (z + kTanhB * z * z * z));
    default: return z;
  }
}
// sigmoid(x) and sigmoid(-x), each within 6 x 2^-24 of itself (see sigmoid).
struct Sigmoids {
  float of, of_minus;
};
__device__ __forceinline__ Sigmoids sigmoids(float x) {
  const float a = fabsf(x), t = a * 1.44269502f;
  const float rest = fmaf(a, 1.92596303e-8f, fmaf(a, 1.44269502f, -t));
  const float p = __builtin_amdgcn_exp2f(-t), e = fmaf(p * rest, -0.693147182f, p), d = 1.0f + e;
  const float y = __builtin_amdgcn_rcpf(d), r = fmaf(fmaf(-d, y, 1.0f), y, y), er = e * r;
  return x < 0.0f ? Sigmoids{er, r} : Sigmoids{r, er};
}
// z is limited where the derivative has long been 0 or 1, so that no inf meets a 0.
__device__ __forceinline__ float act_grad(float z, int act) {
  switch (act) {
    case MPB_ACT_RELU: return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    case MPB_ACT_SILU: {
      const float x = z != z ? z : fminf(fmaxf(z, -120.0f), 120.0f);
      const Sigmoids s = sigmoids(x);
      return s.of * fmaf(x, s.of_minus, 1.0f);
    }
    case MPB_ACT_GELU: {
      const float x = z != z ? z : fminf(fmaxf(z, -20.0f), 20.0f);
      const float e = bell(x), tail = normal_tail(fabsf(x), e);
      return fmaf(x * kInvSqrt2Pi, e, x > 0.0f ? 1.0f - tail : tail);
    }
    case MPB_ACT_GELU_TANH: {
      const float x = z != z ? z : fminf(fmaxf(z, -20.0f), 20.0f), x2 = x * x;
      const Sigmoids s = sigmoids(2.0f * kTanhA * x * fmaf(kTanhB, x2, 1.0f));
      return fmaf(x * s.of * s.of_minus, 2.0f * kTanhA * fmaf(3.0f * kTanhB, x2, 1.0f), s.of);
    }
    default: return 1.0f;
  }
}

// ---------------------------------------------------------------- epilogue
// What becomes of a product: a gradient in the operands' type, in bf16 (of fp16
// operands) or fp32, times a scale, or moe_linear's epilogue with y of 16 bits or fp32.
enum { kGrad16, kGradBf, kGrad32, kOut16, kOut32 };

// NV (4 or 8) consecutive columns of a row, as they are loaded from the residual: the
// load of one group goes out before the group in front of it is stored.
template <class D, int NV, int KIND>
struct Residual {
  typedef typename std::conditional<KIND == kGradBf, BF16, D>::type::elem elem;
  typedef elem evec __attribute__((ext_vector_type(NV)));
  typedef float fvec __attribute__((ext_vector_type(NV), aligned(16)));  // rows are 16-byte aligned
  evec narrow_;
  fvec wide_;
  __device__ __forceinline__ void load(const LinearOut& o, int64_t m, int n) {
    const size_t at = (size_t)m * o.N + n;
    if constexpr (KIND == kOut16) {
      if (o.res) narrow_ = *(const evec*)((const elem*)o.res + at);
    } else if constexpr (KIND == kOut32) {
      if (o.res) wide_ = *(const fvec*)((const float*)o.res + at);
    }
  }
};

// NV results of row m from column n on.
template <class D, int NV, int KIND>
__device__ __forceinline__ void finish(const LinearOut& o, int64_t m, int n, float (&v)[NV], const Residual<D, NV, KIND>& res) {
  typedef typename Residual<D, NV, KIND>::elem elem;
  typedef typename Residual<D, NV, KIND>::evec evec;
  typedef typename Residual<D, NV, KIND>::fvec fvec;
  const size_t at = (size_t)m * o.N + n;
  fvec w;
#pragma unroll
  for (int i = 0; i < NV; ++i) w[i] = v[i];
  constexpr bool kNarrow = KIND != kGrad32 && KIND != kOut32;
  if constexpr (KIND <= kGrad32) {
    if (o.exp2) {
      // at once: 2 to one of them may be out of range, and so may the result in between
      const int e = *o.exp2 + (o.exp2_b ? *o.exp2_b : 0);
#pragma unroll
      for (int i = 0; i < NV; ++i) w[i] = __builtin_ldexpf(w[i], e);
    }
  } else {
    if (o.bias) w += *(const fvec*)(o.bias + n);
    if (o.z) *(evec*)((elem*)o.z + at) = __builtin_convertvector(w, evec);
    if (o.act != MPB_ACT_NONE) {
#pragma unroll
      for (int i = 0; i < NV; ++i) w[i] = act_of<kNarrow>(w[i], o.act);
    }
    if (o.res) w += kNarrow ? __builtin_convertvector(res.narrow_, fvec) : res.wide_;
  }
  if constexpr (kNarrow) *(evec*)((elem*)o.y + at) = __builtin_convertvector(w, evec);
  else *(fvec*)((float*)o.y + at) = w;
}

// ---------------------------------------------------------------- operands in LDS
// 16 bytes a lane from src + off to LDS at byte `lds` + 16 lane (src and lds are the
// wave's). The load has no register of its own that could be reused early, and
// its address registers are read when it issues; before the barrier that hands a buffer over
// the caller waits until no more loads are outstanding than those of later buffers. The builtin
// of this load makes the compiler wait for it before any transposing read of LDS, of the
// other buffers too. m0 is
// reserved to such instructions: nothing else in these kernels counts on its value.
__device__ __forceinline__ void load_lds16(const char* src, uint32_t off, uint32_t lds) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass cannot parse the operands
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(src) : "memory");
#endif
}
// A pointer that is the same in every lane, in scalar registers.
__device__ __forceinline__ const char* wave_uniform(const char* p) {
  const uint64_t v = (uint64_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (const char*)((uint64_t)hi << 32 | lo);
}
// All but the wave's last N loads have arrived.
template <int N>
__device__ __forceinline__ void loads_but() {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
#endif
}

// A stage is 32 of the reduction. R rows (of A or B) take 64 R bytes of it, in one of two forms:
//  rows   row r at 64 r, its 16-byte pieces c at c ^ swz_row(r)
//  turned reduction index k at 2 R k, its 32-byte pieces (16 rows) s at s ^ swz_k(k)
// so that what a fragment reads at once takes turns on the banks. A direct load writes a wave's 1 KiB
// (lane i the i-th 16 bytes), so the swizzle is in the addresses that it loads from.
template <int R, bool TURNED, int SH>
struct Operand {
  static __device__ __forceinline__ int swz_row(int r) { return (r >> 1 & 1) | (r >> SH & 1) << 1; }
  // (rows of 384 bytes shift by half the banks already: two bits are left to change)
  static __device__ __forceinline__ int swz_k(int kk) {
    return R % 128 == 0 ? (kk & 3) | ((kk >> 3 & 1) << 2) : (kk & 3) ^ (kk >> 3 & 1);
  }
  // Reduction index of the bytes o of a stage.
  static __device__ __forceinline__ int k_of(int o) { return TURNED ? o / (2 * R) : 8 * ((o >> 4 & 3) ^ swz_row(o >> 6)); }
  // Offset in the source of the bytes o of a stage. Rows past the `left` that there are
  // repeat the last: their results are not stored.
  static __device__ __forceinline__ uint32_t source(int o, int64_t stride, int left) {
    if constexpr (TURNED) {
      const int col = 16 * ((o % (2 * R) / 32) ^ swz_k(k_of(o))) + 8 * (o >> 4 & 1);
      return (uint32_t)(k_of(o) * stride + 2 * min(col, left - 8));
    } else {
      return (uint32_t)(min(o >> 6, left - 1) * stride + 2 * k_of(o));
    }
  }
  // The tile's first byte at reduction index 0, and the bytes of a stage's advance.
  static __device__ __forceinline__ const char* first(const void* p, int64_t r0, int64_t stride) {
    return (const char*)p + (TURNED ? 2 * r0 : r0 * stride);
  }
  static __device__ __forceinline__ int64_t advance(int64_t stride) { return TURNED ? 32 * stride : 64; }
};

// A fragment: lane l holds row (first + its row among 16) at reduction indices 8 (l / 16) ... + 7.
__device__ __forceinline__ ux4 read_rows(const lds_char* a) { return *(const __attribute__((address_space(3))) ux4*)a; }
// Turned: each read gives the lane its row at 4 indices; its 16 lanes address 4
// rows of 16 elements, 8 bytes each.
__device__ __forceinline__ ux4 read_turned(lds_char* a, int step4) {
  typedef __attribute__((address_space(3))) sx4 lds_sx4;
  const sx4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_sx4*)a);
  const sx4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_sx4*)(a + step4));
  sx8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = lo[i], v[4 + i] = hi[i];
  return __builtin_bit_cast(ux4, v);
}

// ---------------------------------------------------------------- the product
// Workgroup b works on unit() b: the dispatcher hands b to XCD b % 8, and an XCD takes
// neighbouring tiles (8 rows of tiles at a time), so that its L2 holds the operands that they share.
__device__ __forceinline__ int unit(int b, int n) {
  const int x = b & 7, q = n >> 3, r = n & 7;
  return x * q + min(x, r) + (b >> 3);
}

// The share of workgroup `block` of `blocks` in product p.
template <class D, int BM, int BN, int WM, int WN, bool AT, bool BT, int KIND>
__device__ __forceinline__ void product_tile(const LinearProduct& p, int block, int blocks, char* smem) {
  typedef typename D::vec vec;
  constexpr int NWN = BN / WN, NW = (BM / WM) * NWN, MF = WM / 16, NF = WN / 16;
  constexpr int kStages = 5;  // buffers
  // Columns of C in a lane (row r of 16, g of 4) once its products are done: 8 in a row for
  // every two fragments of B, 32 with its neighbours, so that what a wave stores in two
  // instructions at most are whole lines of fp32 and half lines of 16 bits. Where B lies in rows, fragment j's
  // row r is column 32 (j / 2) + 8 (r / 4) + 4 (j % 2) + r % 4; where it is turned, a
  // fragment is 16 consecutive columns, and lanes 16 apart exchange theirs at the end.
  // 4096 x 8192 x 2048 with fp32 y takes 150 us, 163 with 4 columns a lane, 253 with 16;
  // 8192 x 4096 x 4096 dX 211, 219 with 4.
  constexpr int SHB = 3;
  static_assert(NF % 2 == 0, "");
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int id = unit(block, blocks), tiles = p.tm * p.tn;
  const int split = id / tiles, tile = id - split * tiles;
  const int grp = tile / (8 * p.tn), rest = tile - grp * 8 * p.tn, gm = min(8, p.tm - 8 * grp);
  const int64_t m0 = (int64_t)(8 * grp + rest % gm) * BM;
  const int64_t n0 = (int64_t)(rest / gm) * BN;

  typedef Operand<BM, AT, 2> OA;
  typedef Operand<BN, BT, SHB> OB;
  // A stage comes as pieces of 1 KiB, A's PA and then B's; wave w loads pieces w, w + NW, ...
  constexpr int PA = BM / 16, PB = BN / 16, NP = (PA + PB + NW - 1) / NW, SPARE = (PA + PB) % NW;
  constexpr uint32_t kA = 64 * BM, kStage = 64 * (BM + BN);
  const int64_t sa = 2 * p.lda, sb = 2 * p.ldb;
  uint32_t off[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int q = i * NW + wave, o = 1024 * q + 16 * lane;
    off[i] = q < PA        ? OA::source(o, sa, (int)min((int64_t)BM, p.M - m0))
             : q < PA + PB ? OB::source(o - kA, sb, (int)min((int64_t)BN, p.N - n0))
                           : 0;
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char*)smem;

  // stages of this workgroup: the reduction once, or twice with A's two parts (first A, then A2)
  const int stages = p.stages, s0 = split * p.per, s1 = min(s0 + p.per, stages * p.parts);
  int next = s0 < stages ? s0 : s0 - stages, left = (int)p.K - 32 * next;  // of its part; reduction left
  const char* pa = OA::first(s0 < stages ? p.A : p.A2, m0, sa) + next * OA::advance(sa);
  const char* pb = OB::first(p.B, n0, sb) + next * OB::advance(sb);
  auto of_a = [&](int i) { return (i + 1) * NW <= PA || (i * NW < PA && i * NW + wave < PA); };
  auto issue_whole = [&](uint32_t lds) {
    const char *a = wave_uniform(pa), *b = wave_uniform(pb);
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (!SPARE || i < NP - 1 || wave < SPARE) load_lds16(of_a(i) ? a : b, off[i], lds + 1024 * (i * NW + wave));
    pa += OA::advance(sa);
    pb += OB::advance(sb);
    left -= 32;
    ++next;
  };
  auto issue = [&](uint32_t lds) {
    if (left >= 32) {
      issue_whole(lds);
    } else {  // the reduction ends inside the stage: zeros behind its end
      // arrived_but counts whole stages only; this one has no direct loads, and waves
      // all of whose pieces lie behind the end would not wait at all
      loads_but<0>();
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if (SPARE && i == NP - 1 && wave >= SPARE) break;
        const int o = 1024 * (i * NW + wave) + 16 * lane;
        ux4 v = (ux4)(0u);
        if ((of_a(i) ? OA::k_of(o) : OB::k_of(o - kA)) < left)
          v = *(const __attribute__((address_space(1))) ux4*)(uintptr_t)((of_a(i) ? pa : pb) + off[i]);
        *(__attribute__((address_space(3))) ux4*)(uintptr_t)(lds + o) = v;
        __builtin_amdgcn_sched_barrier(0);  // one at a time: the registers are taken
      }
      ++next;
    }
    if (next == stages) {
      next = 0;
      left = (int)p.K;
      pa = OA::first(p.A2, m0, sa);
      pb = OB::first(p.B, n0, sb);
    }
  };
  // All but the last N stages that the wave issued have arrived (those before one that
  // ends the reduction had when that was issued).
  auto arrived_but = [&](auto n) {
    constexpr int N = decltype(n)::value;
    if (SPARE == 0 || wave < SPARE)
      loads_but<N * NP>();
    else
      loads_but<N * (NP - 1)>();
  };

  const int wm = (wave / NWN) * WM, wn = (wave % NWN) * WN, r = lane & 15, g = lane >> 4;
  // fragment addresses within a stage
  uint32_t fa[AT ? MF : 1], fb[BT ? NF : 1];
  const int kk = 8 * g + (r >> 2);
  if constexpr (AT) {
#pragma unroll
    for (int i = 0; i < MF; ++i) fa[i] = 2 * BM * kk + 32 * ((wm / 16 + i) ^ OA::swz_k(kk)) + 8 * (r & 3);
  } else {
    fa[0] = 64 * (wm + r) + 16 * (g ^ (r >> 1 & 3));
  }
  if constexpr (BT) {
#pragma unroll
    for (int j = 0; j < NF; ++j) fb[j] = kA + 2 * BN * kk + 32 * ((wn / 16 + j) ^ OB::swz_k(kk)) + 8 * (r & 3);
  } else {
    fb[0] = kA + 64 * (wn + 8 * (r >> 2) + (r & 3)) + 16 * (g ^ (r >> 1 & 3));
  }

  acc4 acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = (acc4)(0.0f);

  // A stage has two phases: its fragments are read (and a later stage is issued), then
  // multiplied. With 8 waves, two a SIMD, waves 4 to 7 run one phase behind waves 0 to 3: the
  // matrix cores work for one half while the other reads.
  constexpr bool kTwoHalves = NW == 8;
  constexpr int kAhead = kStages - 1;  // stages in flight
  ux4 a[MF], b[NF];
  auto at = [&](uint32_t buf, uint32_t o) { return (lds_char*)(uintptr_t)(buf + o); };
  uint32_t buf = lds0, free = lds0 + kAhead * kStage;  // of stage s, of stage s - 1
  auto stage = [&](auto steady, int s) {
#pragma unroll
    for (int j = 0; j < NF; ++j) b[j] = BT ? read_turned(at(buf, fb[BT ? j : 0]), 8 * BN) : read_rows(at(buf, fb[0]) + 2048 * (j / 2) + 256 * (j % 2));
#pragma unroll
    for (int i = 0; i < MF; ++i) a[i] = AT ? read_turned(at(buf, fa[AT ? i : 0]), 8 * BM) : read_rows(at(buf, fa[0]) + 1024 * i);
    if (steady) issue_whole(free);
    else if (s + kAhead < s1) issue(free);
    // stage s + 1 has arrived
    if (steady || s + kAhead < s1) arrived_but(std::integral_constant<int, kAhead - 1>());
    else loads_but<0>();
    __syncthreads();  // ... for every wave, and every wave of this half has read stage s
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j)
        acc[i][j] = product<D>(__builtin_bit_cast(vec, b[j]), __builtin_bit_cast(vec, a[i]), acc[i][j]);
    __builtin_amdgcn_s_setprio(0);
    if (kTwoHalves) __syncthreads();
    free = buf;
    buf = buf + kStage == lds0 + kStages * kStage ? lds0 : buf + kStage;
  };
  if (s0 < s1) {
    for (int i = 0; i < kAhead && s0 + i < s1; ++i) issue(lds0 + i * kStage);
    if (s0 + kAhead <= s1) arrived_but(std::integral_constant<int, kAhead - 1>());
    else loads_but<0>();
    __syncthreads();
    if (kTwoHalves && wave >= NW / 2) __syncthreads();
    for (int s = s0; s < s1;) {
      for (; s + kAhead < s1 && left >= 64; ++s) stage(std::true_type(), s);
      if (s < s1) stage(std::false_type(), s++);
    }
    if (kTwoHalves && wave < NW / 2) __syncthreads();
  }

  const int64_t m = m0 + wm + r;
  if (p.partial) {
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        const int64_t n = n0 + wn + (BT ? 16 * j + 4 * g : 32 * (j / 2) + 8 * g + 4 * (j % 2));
        if (m + 16 * i < p.M && n < p.N) *(acc4*)(p.partial + ((size_t)split * p.M + m + 16 * i) * p.N + n) = acc[i][j];
      }
    return;
  }
  constexpr int NV = 8, NG = NF / 2;  // columns of a group, groups of a lane's row
  if constexpr (BT) {
    // of fragments 2 k and 2 k + 1, lanes of even g keep the first and get their neighbour's
    // four columns of it, those of odd g the second's
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int j = 0; j < NF; j += 2)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const auto v = __builtin_amdgcn_permlane16_swap(__float_as_uint(acc[i][j][e]), __float_as_uint(acc[i][j + 1][e]), false, false);
          acc[i][j][e] = __uint_as_float(v[0]);
          acc[i][j + 1][e] = __uint_as_float(v[1]);
        }
  }
  auto column = [&](int k) {
    return n0 + wn + 32 * k + (BT ? 16 * (g & 1) + 8 * (g >> 1) : 8 * g);
  };
  Residual<D, NV, KIND> res[2][NG];
  auto load_row = [&](int i) {
#pragma unroll
    for (int k = 0; k < NG; ++k)
      if (m + 16 * i < p.M && column(k) < p.N) res[i & 1][k].load(p.out, m + 16 * i, (int)column(k));
  };
  load_row(0);
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    if (i + 1 < MF) load_row(i + 1);
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      if (m + 16 * i >= p.M || column(k) >= p.N) continue;
      float v[NV];
#pragma unroll
      for (int e = 0; e < NV; ++e) v[e] = acc[i][2 * k + e / 4][e & 3];
      finish<D, NV, KIND>(p.out, m + 16 * i, (int)column(k), v, res[i & 1][k]);
    }
  }
}

template <class D, int BM, int BN, int WM, int WN, bool AT, bool BT, int KIND>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN)) void k_product(LinearProduct p) {
  extern __shared__ __align__(16) char smem[];
  product_tile<D, BM, BN, WM, WN, AT, BT, KIND>(p, blockIdx.x, gridDim.x, smem);
}

// ---------------------------------------------------------------- dz
// The largest finite |v| of each workgroup's share of dy (blockIdx.y 0), and of X (1)
// and W (2) where they are to become fp16.
template <class D>
__global__ __launch_bounds__(256) void k_max(LinearGradParams p) {
  typedef typename D::vec vec;
  typedef typename D::elem elem;
  __shared__ float red[4];
  const int of = blockIdx.y;
  if ((of == 1 && !p.x16) || (of == 2 && !p.w16)) return;
  const int64_t n8 = (of == 0 ? (int64_t)p.T * p.N : of == 1 ? (int64_t)p.T * p.Kd : (int64_t)p.N * p.Kd) / 8;
  const elem* src = (const elem*)(of == 0 ? p.dy : of == 1 ? p.X : p.W);
  float m = 0.0f;
  auto take = [&](const fx8& d) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = fabsf(d[j]);
      if (a < INFINITY) m = fmaxf(m, a);
    }
  };
  const int64_t step = (int64_t)gridDim.x * 256;
#pragma unroll 4
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += step) {
    if (of == 0 && p.dy32) take(load8((const float*)p.dy + 8 * i));
    else take(widen<D>(*(const vec*)(src + 8 * i)));
  }
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x == 0) p.maxima[of * kMaxima + blockIdx.x] = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}

// The exponent e of the scale that brings the largest of k_max's values into [2^13,
// 2^14): an activation's slope of up to 1.13 and the rounding to fp16 stay in range.
__device__ __forceinline__ int scale_of(const float* maxima, float (&red)[4]) {
  float m = 0.0f;
  for (int i = threadIdx.x; i < kMaxima; i += 256) m = fmaxf(m, maxima[i]);
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  __syncthreads();
  if (m == 0.0f) return 0;
  int e = 0;
  (void)frexpf(m, &e);  // m = f 2^e, f in [1/2, 1)
  return min(max(14 - e, -126), 126);
}

// dz in one or two parts, and the sums over a group of rows for dbias. A
// thread has 8 columns, LC threads a row: whole waves where there are several groups,
// whose sums k_dbias adds; 4 threads and 64 rows at a time where one group has all rows
// and its sums are dbias.
template <class D, int LC>
__device__ __forceinline__ void dz_rows(const LinearGradParams& p, int bx, int by, int groups, float* smem) {
  typedef typename D::vec vec;
  typedef typename D::elem elem;
  constexpr int R = 256 / LC;  // rows at a time
  float(*red)[8 * LC] = (float(*)[8 * LC])smem;  // [R]
  const int col = 8 * (threadIdx.x % LC), slot = threadIdx.x / LC;
  const int64_t n = (int64_t)bx * (8 * LC) + col;
  float scale = 1.0f;
  if (p.part1) {
    const int e = scale_of(p.maxima, *(float(*)[4])smem);
    scale = ldexpf(1.0f, e);
    if (bx == 0 && by == 0 && threadIdx.x == 0) p.exp2[0] = -e;
  }
  fx8 sum = (fx8)(0.0f);
  // U rows a thread are loaded before the first is worked on (none is behind the last);
  // left to the compiler, the loads of one waited for the stores of the one before
  constexpr int U = 4;
  auto rows = [&](auto wide, auto with_z) {
    const int t0 = by * p.rows, t1 = min(p.T, t0 + p.rows);
    for (int t = t0 + slot; t < t1; t += U * R) {
      fx8 dy32[U];
      vec dy[U], z[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const size_t at = (size_t)min(t + u * R, t1 - 1) * p.N + n;
        if constexpr (wide) dy32[u] = load8((const float*)p.dy + at);
        else dy[u] = *(const vec*)((const elem*)p.dy + at);
        if constexpr (with_z) z[u] = *(const vec*)((const elem*)p.z + at);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t + u * R >= t1) break;
        fx8 d;
        if constexpr (wide) d = dy32[u];
        else d = widen<D>(dy[u]);
        if constexpr (with_z) {
          const fx8 x = widen<D>(z[u]);
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] *= act_grad(x[i], p.act);
        }
        sum += d;
        if constexpr (wide || with_z) {
          if (!p.part1) continue;
          const size_t at = (size_t)(t + u * R) * p.N + n;
          const fx8 x = d * scale;
          const hx8 h = narrow<F16>(x);
          *(hx8*)((_Float16*)p.part1 + at) = h;
          fx8 left = x - widen<F16>(h);
#pragma unroll
          for (int i = 0; i < 8; ++i) left[i] = fabsf(x[i]) < INFINITY ? left[i] : 0.0f;  // inf - inf
          *(hx8*)((_Float16*)p.part2 + at) = narrow<F16>(left);
        }
      }
    }
  };
  if (n < p.N) {
    using std::false_type, std::true_type;
    if (p.act != MPB_ACT_NONE) {
      if (p.dy32) rows(true_type(), true_type());
      else rows(false_type(), true_type());
    } else {
      if (p.dy32) rows(true_type(), false_type());
      else rows(false_type(), false_type());
    }
  }
  if (!p.dbias) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) red[slot][col + i] = sum[i];
  __syncthreads();
  float* to = groups == 1 ? p.dbias : p.db_part + (size_t)by * p.N;
  if constexpr (LC < 64) {  // 8 threads a column, then those 8
    const int c = threadIdx.x & 31, part = threadIdx.x >> 5;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < R / 8; ++i) s += red[part * (R / 8) + i][c];
    __syncthreads();
    red[part][c] = s;
    __syncthreads();
    const int64_t at = (int64_t)bx * 32 + c;
    if (part == 0 && at < p.N) {
#pragma unroll
      for (int i = 1; i < 8; ++i) s += red[i][c];
      to[at] = s;
    }
  } else {
    for (int c = threadIdx.x; c < 512; c += 256) {
      const int64_t at = (int64_t)bx * 512 + c;
      if (at < p.N) to[at] = red[0][c] + red[1][c] + red[2][c] + red[3][c];
    }
  }
}

template <class D, int LC>
__global__ __launch_bounds__(256) void k_dz(LinearGradParams p) {
  __shared__ __align__(16) float smem[2048];
  dz_rows<D, LC>(p, blockIdx.x, blockIdx.y, gridDim.y, smem);
}

// dX and dW in one launch, where both have small tiles and neither fills the chip
// alone, and dbias of a few tokens (blocks_b workgroups): 200 x 2048 x 2048 with its
// join 21 us a pass, in a launch each 36.
template <class D, int KIND>
__global__ __launch_bounds__(256) void k_gradients(LinearProduct x, LinearProduct w, LinearGradParams p, int blocks_x,
                                                   int blocks_b) {
  extern __shared__ __align__(16) char smem[];
  const int b = blockIdx.x, bw = gridDim.x - blocks_x - blocks_b;
  if (b < blocks_x) product_tile<D, 128, 128, 64, 64, false, true, KIND>(x, b, blocks_x, smem);
  else if (b < blocks_x + bw) product_tile<D, 128, 128, 64, 64, true, true, kGrad32>(w, b - blocks_x, bw, smem);
  else dz_rows<D, 4>(p, b - blocks_x - bw, 0, 1, (float*)smem);
}

// Adds the partial sums of a split reduction in their order, 8 columns a thread.
template <class D, int KIND>
__global__ __launch_bounds__(256) void k_join(LinearProduct p, int splits) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n8 = p.N / 8;
  if (i >= p.M * n8) return;
  const int64_t m = i / n8;
  const int n = (int)(i - m * n8) * 8;
  const float* src = p.partial + (size_t)m * p.N + n;
  const size_t step = (size_t)p.M * p.N;
  fx8 s = load8(src);
  for (int k = 1; k < splits; k += 8) {  // eight loads in flight
    fx8 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (k + j < splits) v[j] = load8(src + (k + j) * step);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (k + j < splits) s += v[j];
  }
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = s[j];
  Residual<D, 8, KIND> res;
  res.load(p.out, m, n);
  finish<D, 8, KIND>(p.out, m, n, v, res);
}

// ---------------------------------------------------------------- few tokens
constexpr int kSkinnyWaves = 16;

// 16 rows of W a workgroup and up to 16 MF tokens; its 16 waves take every 16th piece
// of 64 of the reduction (whole 128-byte lines of W, once), both operands straight into
// registers, U halves of pieces in flight. Their sums meet in LDS: waves 8 to 15
// hand theirs to waves 0 to 7, whose sums are added in wave order. Bound by HBM: one
// token of 16384 x 4096 27 us (4.9 TB/s), of 4096 x 4096 8.9 (3.8: the launch and one chain of latencies).
template <class D, int KIND, int MF>
__global__ __launch_bounds__(64 * kSkinnyWaves) void k_skinny(LinearProduct p) {
  typedef typename D::vec vec;
  constexpr int U = MF == 1 ? 8 : MF == 2 ? 6 : MF <= 4 ? 4 : 2, kHalfWaves = kSkinnyWaves / 2;
  __shared__ float sums[kHalfWaves][16 * MF][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int T = (int)p.M;
  const char* w = (const char*)p.B + ((n0 + r < p.N ? n0 + r : p.N - 1) * p.ldb + 8 * g) * 2;
  const char* x = (const char*)p.A + 16 * g;
  uint32_t xo[MF];  // rows past the last repeat it: their results are not stored
#pragma unroll
  for (int i = 0; i < MF; ++i) xo[i] = (uint32_t)(min(16 * i + r, T - 1) * p.lda * 2);
  const int pieces = (int)(p.K / 64);
  acc4 acc[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) acc[i] = (acc4)(0.0f);
  int c = wave;
  auto run = [&](auto n) {  // n halves of pieces
    constexpr int N = decltype(n)::value;
    vec b[N], a[N][MF];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const uint32_t at = (uint32_t)(c + u / 2 * kSkinnyWaves) * 128 + 64 * (u & 1);
      b[u] = stream_load((const vec*)(w + at));
#pragma unroll
      for (int i = 0; i < MF; ++i) a[u][i] = *(const vec*)(x + at + xo[i]);
    }
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int i = 0; i < MF; ++i) acc[i] = product<D>(b[u], a[u][i], acc[i]);
    c += N / 2 * kSkinnyWaves;
  };
  while (c + (U / 2 - 1) * kSkinnyWaves < pieces) run(std::integral_constant<int, U>());
  if constexpr (U > 2) {
    while (c < pieces) run(std::integral_constant<int, 2>());
  }
  if (wave >= kHalfWaves) {
#pragma unroll
    for (int i = 0; i < MF; ++i) *(acc4*)&sums[wave - kHalfWaves][16 * i + r][4 * g] = acc[i];
  }
  __syncthreads();
  if (wave < kHalfWaves) {
#pragma unroll
    for (int i = 0; i < MF; ++i) *(acc4*)&sums[wave][16 * i + r][4 * g] += acc[i];
  }
  __syncthreads();
  // 4 columns a thread
  const int t = threadIdx.x >> 2, q = 4 * (threadIdx.x & 3);
  if (t < T && t < 16 * MF && n0 + q < p.N) {
    fx4 s = *(const fx4*)&sums[0][t][q];
#pragma unroll
    for (int i = 1; i < kHalfWaves; ++i) s += *(const fx4*)&sums[i][t][q];
    float v[4] = {s[0], s[1], s[2], s[3]};
    Residual<D, 4, KIND> res;
    res.load(p.out, t, (int)(n0 + q));
    finish<D, 4, KIND>(p.out, t, (int)(n0 + q), v, res);
  }
}

// ---------------------------------------------------------------- fp16 operands
// bf16 X (blockIdx.y 0) and W (1) as scaled fp16, and the exponent that takes the scale
// out again. A value's 8 bits fit unless it is below 2^-30 of the largest.
__global__ __launch_bounds__(256) void k_half(LinearGradParams p) {
  __shared__ float s_max[4];
  const int of = 1 + blockIdx.y;
  _Float16* to = (_Float16*)(of == 1 ? p.x16 : p.w16);
  if (!to) return;
  const int e = scale_of(p.maxima + of * kMaxima, s_max);
  if (blockIdx.x == 0 && threadIdx.x == 0) p.exp2[of] = -e;
  const float scale = ldexpf(1.0f, e);
  const __bf16* src = (const __bf16*)(of == 1 ? p.X : p.W);
  const int64_t n8 = (int64_t)(of == 1 ? p.T : p.N) * p.Kd / 8, step = (int64_t)gridDim.x * 256;
#pragma unroll 4
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += step)
    *(hx8*)(to + 8 * i) = narrow<F16>(widen<BF16>(*(const bx8*)(src + 8 * i)) * scale);
}

// dbias: the groups' sums in their order.
__global__ __launch_bounds__(256) void k_dbias(const float* part, int groups, int N, float* db) {
  __shared__ float red[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (n < N) {
#pragma unroll 8
    for (int i = wave; i < groups; i += 4) s += part[(size_t)i * N + n];
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && n < N) db[n] = red[0][lane] + red[1][lane] + red[2][lane] + red[3][lane];
}

// ---------------------------------------------------------------- launches
template <class D, int BM, int BN, int WM, int WN, bool AT, bool BT, int KIND>
hipError_t launch_tiles(LinearProduct& p, hipStream_t s) {
  static unsigned long long raised = 0;
  constexpr int lds = 5 * 64 * (BM + BN);
  const hipError_t e = raise_lds_limit((const void*)&k_product<D, BM, BN, WM, WN, AT, BT, KIND>, lds, raised);
  if (e != hipSuccess) return e;
  k_product<D, BM, BN, WM, WN, AT, BT, KIND><<<p.tm * p.tn * p.splits, 64 * (BM / WM) * (BN / WN), lds, s>>>(p);
  return hipGetLastError();
}

// p with the plan's launch shape; a split reduction's sums go to `partial`.
void set_plan(LinearProduct& p, const LinearPlan& plan, float* partial) {
  p.tm = plan.tm;
  p.tn = plan.tn;
  p.per = plan.per;
  p.splits = plan.splits;
  p.stages = plan.stages;
  p.parts = plan.parts;
  p.partial = plan.splits > 1 ? partial : nullptr;
}

template <class D, int KIND>
hipError_t join(const LinearProduct& p, hipStream_t s) {
  if (p.splits == 1) return hipSuccess;
  const int64_t n = p.M * (p.N / 8);
  k_join<D, KIND><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(p, p.splits);
  return hipGetLastError();
}

template <class D, bool AT, bool BT, int KIND>
hipError_t launch_product(LinearProduct p, const LinearPlan& plan, float* partial, hipStream_t s) {
  set_plan(p, plan, partial);
  const hipError_t e = plan.rows == 256   ? launch_tiles<D, 256, 256, 128, 64, AT, BT, KIND>(p, s)
                       : plan.rows == 192 ? launch_tiles<D, 192, 256, 96, 64, AT, BT, KIND>(p, s)
                                          : launch_tiles<D, 128, 128, 64, 64, AT, BT, KIND>(p, s);
  return e != hipSuccess ? e : join<D, KIND>(p, s);
}

// dX and dW, in one launch where both have small tiles.
template <class D, int KIND>
hipError_t launch_gradients(LinearProduct x, const LinearPlan& px, LinearProduct w, const LinearPlan& pw,
                            const LinearGradParams& p, bool with_dbias, hipStream_t s) {
  if (px.rows != 128 || pw.rows != 128) {
    const hipError_t e = launch_product<D, false, true, KIND>(x, px, p.partial_x, s);
    return e != hipSuccess ? e : launch_product<D, true, true, kGrad32>(w, pw, p.partial_w, s);
  }
  set_plan(x, px, p.partial_x);
  set_plan(w, pw, p.partial_w);
  static unsigned long long raised = 0;
  constexpr int lds = 5 * 64 * 256;
  hipError_t e = raise_lds_limit((const void*)&k_gradients<D, KIND>, lds, raised);
  if (e != hipSuccess) return e;
  const int bx = x.tm * x.tn * x.splits, bw = w.tm * w.tn * w.splits, bb = with_dbias ? (p.N + 31) / 32 : 0;
  k_gradients<D, KIND><<<bx + bw + bb, 256, lds, s>>>(x, w, p, bx, bb);
  if ((e = hipGetLastError()) != hipSuccess || (e = join<D, KIND>(x, s)) != hipSuccess) return e;
  return join<D, kGrad32>(w, s);
}

template <class D, int KIND>
hipError_t forward(const LinearProduct& p, float* ws, hipStream_t s) {
  if (linear_skinny(p.M, p.N, p.K)) {
    const unsigned grid = (unsigned)((p.N + 15) / 16);
    constexpr int threads = 64 * kSkinnyWaves;
    switch ((p.M + 15) / 16) {
      case 1: k_skinny<D, KIND, 1><<<grid, threads, 0, s>>>(p); break;
      case 2: k_skinny<D, KIND, 2><<<grid, threads, 0, s>>>(p); break;
      case 3: k_skinny<D, KIND, 3><<<grid, threads, 0, s>>>(p); break;
      case 4: k_skinny<D, KIND, 4><<<grid, threads, 0, s>>>(p); break;
      case 5: k_skinny<D, KIND, 5><<<grid, threads, 0, s>>>(p); break;
      case 6: k_skinny<D, KIND, 6><<<grid, threads, 0, s>>>(p); break;
      default: k_skinny<D, KIND, 8><<<grid, threads, 0, s>>>(p); break;
    }
    return hipGetLastError();
  }
  return launch_product<D, false, false, KIND>(p, linear_plan(p.M, p.N, p.K, 1), ws, s);
}

template <class D>
hipError_t gradients(LinearGradParams p, hipStream_t s) {
  hipError_t e = hipSuccess;
  const bool formed = p.part1 != nullptr, dx = p.dX && p.T > 0;
  const int groups = (p.T + p.rows - 1) / p.rows;
  const int parts = formed ? 2 : 1;
  const LinearPlan pw = linear_plan(p.N, p.Kd, p.T, parts), px = dx ? linear_plan(p.T, p.Kd, p.N, parts) : pw;
  // dbias of a few tokens beside the products
  const bool beside = p.dbias && !formed && groups == 1 && dx && p.dW && px.rows == 128 && pw.rows == 128;
  if (p.T > 0 && (formed || (p.dbias && !beside))) {
    if (formed) {
      k_max<D><<<dim3(kMaxima, p.w16 ? 3 : p.x16 ? 2 : 1), 256, 0, s>>>(p);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (groups == 1) k_dz<D, 4><<<(p.N + 31) / 32, 256, 0, s>>>(p);
    else k_dz<D, 64><<<dim3((p.N + 511) / 512, groups), 256, 0, s>>>(p);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (p.x16 || p.w16) {
      k_half<<<dim3(1024, p.w16 ? 2 : 1), 256, 0, s>>>(p);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  if (p.dbias && groups != 1) {
    k_dbias<<<(p.N + 63) / 64, 256, 0, s>>>(p.db_part, groups, p.N, p.dbias);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const bool scaled = formed && p.T > 0;  // the scales are there
  LinearProduct g{};
  g.out.N = g.ldb = p.Kd;
  g.out.exp2 = scaled ? p.exp2 : nullptr;
  g.lda = p.N;
  g.N = p.Kd;
  g.A = formed ? p.part1 : p.dy;
  g.A2 = formed ? p.part2 : p.dy;
  LinearProduct x = g, w = g;
  x.B = p.w16 ? p.w16 : p.W;
  x.M = p.T; x.K = p.N;
  x.out.y = p.dX;
  x.out.exp2_b = p.w16 ? p.exp2 + 2 : nullptr;
  w.B = p.x16 ? p.x16 : p.X;
  w.M = p.N; w.K = p.T;
  w.out.y = p.dW;
  w.out.exp2_b = scaled && p.x16 ? p.exp2 + 1 : nullptr;
  // parts are fp16 whatever the activations are
  if (dx && p.dW) {
    if (p.w16) return launch_gradients<F16, kGradBf>(x, px, w, pw, p, false, s);
    return launch_gradients<D, kGrad16>(x, px, w, pw, p, beside, s);
  }
  if (dx) return p.w16 ? launch_product<F16, false, true, kGradBf>(x, px, p.partial_x, s) : launch_product<D, false, true, kGrad16>(x, px, p.partial_x, s);
  if (p.dW) return formed ? launch_product<F16, true, true, kGrad32>(w, pw, p.partial_w, s) : launch_product<D, true, true, kGrad32>(w, pw, p.partial_w, s);
  return hipSuccess;
}

}  // namespace

// Tiles of 256 x 256 or 192 x 256, one workgroup a CU, or of 128 x 128, two a CU,
// whichever needs the least time by its rounds over the 256 CUs; small tiles feed the
// matrix cores from LDS at some three quarters of the rate. With fewer than 256 small
// tiles the reduction is split until there are about as many, in pieces of at least 8
// stages of 32 (72 x 5120 x 4096 19.1 us with 240 workgroups, 22.4 with 440; 500 x 2048 x
// 2048 20.5 with 256, 26.4 with 512: partial sums and their join cost more than the second workgroup of a CU
// gives).
LinearPlan linear_plan(int64_t M, int64_t N, int64_t K, int parts) {
  LinearPlan q{};
  q.stages = (int)((K + 31) / 32);
  q.parts = parts;
  const int64_t total = (int64_t)q.stages * parts;
  auto tiles = [&](int64_t bm, int64_t bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); };  // M and N are positive
  auto rounds = [](int64_t n, int64_t a) { return (n + a - 1) / a; };
  const int64_t c256 = rounds(tiles(256, 256), 256) * 256 * 256, c192 = rounds(tiles(192, 256), 256) * 192 * 256;
  int64_t splits = 256 / tiles(128, 128);
  if (splits > total / 8) splits = total / 8;
  if (splits > 16) splits = 16;
  if (splits < 1) splits = 1;
  const int64_t c128 = rounds(tiles(128, 128) * splits, 512) * 2 * 128 * 128 * 4 / 3 / splits;
  const int64_t wide = c256 <= c192 ? c256 : c192;
  q.rows = wide > c128 ? 128 : c256 <= c192 ? 256 : 192;
  const int64_t bn = q.rows == 128 ? 128 : 256;
  q.tm = (int)((M + q.rows - 1) / q.rows);
  q.tn = (int)((N + bn - 1) / bn);
  if (q.rows != 128) splits = 1;
  q.per = (int)((total + splits - 1) / splits);
  if (q.per < 1) q.per = 1;
  q.splits = (int)((total + q.per - 1) / q.per);
  if (q.splits < 1) q.splits = 1;
  return q;
}

hipError_t launch_linear(const LinearProduct& p, bool bf16, float* ws, hipStream_t s) {
  if (p.out.y32) return bf16 ? forward<BF16, kOut32>(p, ws, s) : forward<F16, kOut32>(p, ws, s);
  return bf16 ? forward<BF16, kOut16>(p, ws, s) : forward<F16, kOut16>(p, ws, s);
}

hipError_t launch_linear_grad(const LinearGradParams& p, bool bf16, hipStream_t s) {
  return bf16 ? gradients<BF16>(p, s) : gradients<F16>(p, s);
}

}  // namespace mpb
