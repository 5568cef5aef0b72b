// Device helpers shared by the operators around the packed experts (block
// norms, router losses, request adapters): 8-element vectors of the two
// activation types and workgroup sums.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mpb {

typedef float fx4 __attribute__((ext_vector_type(4)));
typedef float fx8 __attribute__((ext_vector_type(8)));
typedef _Float16 hx8 __attribute__((ext_vector_type(8)));
typedef __bf16 bx8 __attribute__((ext_vector_type(8)));

struct F16 {
  typedef _Float16 elem;
  typedef hx8 vec;
};
struct BF16 {
  typedef __bf16 elem;
  typedef bx8 vec;
};

// 8 consecutive activations as fp32 (exact) and back (one rounding, to nearest even).
template <class D>
__device__ __forceinline__ fx8 widen(typename D::vec v) {
  return __builtin_convertvector(v, fx8);
}
template <class D>
__device__ __forceinline__ typename D::vec narrow(fx8 v) {
  return __builtin_convertvector(v, typename D::vec);
}

__device__ __forceinline__ fx8 load8(const float* p) {
  const fx4 a = *(const fx4*)p, b = *(const fx4*)(p + 4);
  return fx8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
// Results of a whole pass, which the caches could not keep anyway, are stored
// (and inputs read once loaded) as streams, so that they do not push out what the
// other workgroups read again.
template <class V>
__device__ __forceinline__ void stream_store(V* p, V v) {
  __builtin_nontemporal_store(v, p);
}
template <class V>
__device__ __forceinline__ V stream_load(const V* p) {
  return __builtin_nontemporal_load(p);
}
__device__ __forceinline__ void stream_store8(float* p, fx8 v) {
  stream_store((fx4*)p, fx4{v[0], v[1], v[2], v[3]});
  stream_store((fx4*)(p + 4), fx4{v[4], v[5], v[6], v[7]});
}
__device__ __forceinline__ void store8(float* p, fx8 v) {
  *(fx4*)p = fx4{v[0], v[1], v[2], v[3]};
  *(fx4*)(p + 4) = fx4{v[4], v[5], v[6], v[7]};
}

// v of another lane: DPP patterns within rows of 16 lanes (a register move,
// where a shuffle goes through the LDS unit).
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}

// op over the wave, the same bits in every lane: pairs, quads, 8, 16 lanes by
// DPP (quad permutes, then mirrors), 32 and 64 by shuffles.
template <class Op>
__device__ __forceinline__ float wave_all(float v, Op op) {
  v = op(v, dpp<0xb1>(v));   // quad_perm 1 0 3 2
  v = op(v, dpp<0x4e>(v));   // quad_perm 2 3 0 1
  v = op(v, dpp<0x141>(v));  // row_half_mirror
  v = op(v, dpp<0x140>(v));  // row_mirror
  v = op(v, __shfl_xor(v, 16));
  return op(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float wave_sum(float v) {
  return wave_all(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_all(v, [](float a, float b) { return fmaxf(a, b); });
}

// Sums of N values over the workgroup, the same bits in every thread (each
// wave's sum by butterflies, then the waves' sums in wave order). buf holds
// N * 16 floats and is free again after the next barrier.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* buf) {
  const int wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (nw == 1) return;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) buf[i * 16 + wave] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = buf[i * 16];
    for (int w = 1; w < nw; ++w) s += buf[i * 16 + w];
    v[i] = s;
  }
}

// Sigmoid within 6 x 2^-24 of itself at any gate (0 from -88 on). e^-|x| is the
// hardware's power of two with what its argument t = |x| log2(e) lost by rounding,
// up to |x| 2^-24 of the result, put back to first order; nothing overflows, and
// 1 + e in [1, 2] has its reciprocal from one Newton step. sigmoid(-x) shares all
// but the last product. 8192 x 4096 norm gradients with a full gate: 144 us, 165
// with expf and a division, 155 with __expf and a division (and far gates up to
// 62 x 2^-24 off); 4096 x 2816 forward 33.1, 34.5 and 32.6.
__device__ __forceinline__ float sigmoid(float x) {
  const float a = fabsf(x), t = a * 1.44269502f;  // log2(e) = 1.44269502 + 1.92596303e-8
  // |x| = inf makes the rest nan, which the maximum drops
  const float rest = fmaxf(fmaf(a, 1.92596303e-8f, fmaf(a, 1.44269502f, -t)), -1.0f);
  const float p = __builtin_amdgcn_exp2f(-t), e = fmaf(p * rest, -0.693147182f, p), d = 1.0f + e;
  const float y = __builtin_amdgcn_rcpf(d), r = fmaf(fmaf(-d, y, 1.0f), y, y);
  return x < 0.0f ? e * r : r;
}

// ---------------------------------------------------------------- fp32 products on the bf16 matrix cores
typedef unsigned int ux4 __attribute__((ext_vector_type(4)));
typedef float acc4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ acc4 mfma(bx8 a, bx8 b, acc4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Cuts 8 fp32 values into N bf16 parts each: part i holds the next 8 bits, cut
// off by truncation, so x - part is exact. What is not finite stays so: inf
// leaves nan for its second part (and a nan whose first part reads as inf, too).
template <int N>
__device__ __forceinline__ void cut(fx8 x, bx8 (&part)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    ux4 u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned a = __float_as_uint(x[2 * i]), b = __float_as_uint(x[2 * i + 1]);
      u[i] = __builtin_amdgcn_perm(b, a, 0x07060302u);
      if (n + 1 < N) {
        x[2 * i] -= __uint_as_float(a & 0xffff0000u);
        x[2 * i + 1] -= __uint_as_float(b & 0xffff0000u);
      }
    }
    part[n] = __builtin_bit_cast(bx8, u);
  }
}

template <class D>
struct Parts;  // parts of an activation
template <>
struct Parts<BF16> {
  static constexpr int N = 1;
  static __device__ __forceinline__ void of(bx8 v, bx8 (&p)[1]) { p[0] = v; }
};
template <>
struct Parts<F16> {
  static constexpr int N = 2;
  static __device__ __forceinline__ void of(hx8 v, bx8 (&p)[2]) { cut<2>(widen<F16>(v), p); }
};

}  // namespace mpb
