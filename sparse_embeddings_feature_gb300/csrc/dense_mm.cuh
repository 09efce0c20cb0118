// Products of bf16 matrices on the tensor cores, with the dense layers' epilogue: what dense.cu asks of dense_mm.cu.
#pragma once

#include "common.cuh"

namespace ctr {

// A matrix as an operand: [outer][inner] elements, inner contiguous, rows ld apart; fp32 matrices as three planes
// of bf16, `plane` elements apart, that add up to them.  Rows are 16-byte aligned.
struct MmOperand {
  const void* p;
  int64_t inner, outer, ld, plane;
};

// out[i, j] = epilogue(sum over r of A(i, r) B(j, r)), i < m, j < n.
//   major 0: A is [m][r], B is [n][r]     (x W^T)
//   major 1: A is [m][r], B is [r][n]     (dz W)
//   major 2: A is [r][m], B is [r][n]     (dz^T x)
struct MmCall {
  int major, planes;
  int64_t m, n, r;
  MmOperand a, b;
  // out, residual and pre are of one type, fp32 or bf16; bias of the inputs' (major 0 alone has any of the three)
  const void* bias = nullptr;
  const void* residual = nullptr;
  void* pre = nullptr;
  void* out = nullptr;
  int64_t ld_res = 0, ld_pre = 0, ldo = 0;
  int act = 0;
  bool out_f32 = false;
  int* err = nullptr;
};

// How a product is taken apart: CTA pairs on 256 x 256 tiles, or CTAs on 128 x 128 or 128 x 32; where share is not 0, sums
// in `parts` of `share` blocks of 64, which leave as fp32 (whole tiles, in the workspace) and are added up by a second
// kernel.
struct MmPlan {
  int columns = 128;  // of a tile
  int64_t share = 0, parts = 1;
  int side() const { return columns == 256 ? 256 : 128; }  // its rows
};
MmPlan mm_plan(int major, int planes, int64_t m, int64_t n, int64_t r);

// Bytes of the parts' places of a sum (major 2), enough for any r up to this one.
size_t mm_room(int64_t m, int64_t n, int64_t r);

// Runs the product; `part` has mm_room(..) bytes, 256-byte aligned.  A ctr_status.
int mm_run(const MmCall& c, float* part, cudaStream_t s);

// Activations (ctr_activation) and their derivatives, of layers of type T, by the hardware's exponential (within 2^-22) and
// reciprocal (1 ulp).
//
// bf16: e^x is 2^(x log2 e) with the product rounded, within (|x| + 4) 2^-24; in gelu, erf within 1.5e-7 by Abramowitz and
// Stegun, Handbook of Mathematical Functions, 7.1.26.  Far below a result's rounding, but not in fp32's tails.
//
// fp32: what that product drops comes back as a factor, so that e^-x is within 5 2^-24 whatever x; the smaller of the two
// sigmoids is taken from it, not from the larger one; gelu's tail of the normal distribution is bell t P(t), t = 1 / (1 +
// 0.34 |z|), P of degree 8 fitted to erfcx(|z| / sqrt 2) / 2 (Lawson's weights on Chebyshev nodes, within 2^-24 of its value
// for |z| up to 14.5, where bell is 0 in fp32).
//
// 65536 x 1024 x 1024 bf16 with silu: expf and divisions 229 us, without an activation 84.  16384 x 1024 x 1024 fp32 with
// gelu and pre: 187 us, by bf16's way 177 (3.7e-6 off at z = -2), without an activation 167; two values an instruction
// do not help, as such operations take their constants from registers, which the sums fill (193 us).
__device__ __forceinline__ float exp2_hw(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_hw(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {  // NaN of NaN
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// e^-x for x from 0 to 110: 2^-h and e^-(x - h ln 2), ln 2 to 48 bits; REST: e^-(x + rest), of a rest far below x.
template <bool REST>
__device__ __forceinline__ float exp_below(float x, float rest = 0.f) {
  const float h = x * 1.44269504f, r = exp2_hw(-h);
  float left = fmaf(h, 1.90465421e-9f, fmaf(-h, 0.693147182f, x));
  if (REST) left += rest;
  return fmaf(-left, r, r);
}

// 1 / (1 + e^-z), and one less that.
template <typename T>
__device__ __forceinline__ float sigmoid_of(float z, float& other) {
  if constexpr (sizeof(T) == 4) {
    const float e = exp_below<false>(min_nan(fabsf(z), 104.f)), r = rcp_hw(1.f + e), small = e * r;
    other = z < 0.f ? r : small;
    return z < 0.f ? small : r;
  } else {
    const float s = rcp_hw(1.f + exp2_hw(-1.44269504f * z));
    other = 1.f - s;
    return s;
  }
}

// The normal distribution's integral up to z, and exp(-z^2 / 2).
template <typename T>
__device__ __forceinline__ float normal_below(float z, float& bell) {
  float tail;
  if constexpr (sizeof(T) == 4) {
    const float a = min_nan(fabsf(z), 14.5f), half = 0.5f * a, sq = half * a;
    bell = exp_below<true>(sq, fmaf(half, a, -sq));
    const float t = rcp_hw(fmaf(0.34f, a, 1.f));
    float y = fmaf(-0.025876375f, t, 0.13835679f);
    y = fmaf(y, t, -0.27087051f);
    y = fmaf(y, t, 0.19971704f);
    y = fmaf(y, t, -0.043105949f);
    y = fmaf(y, t, 0.11471348f);
    y = fmaf(y, t, 0.11535173f);
    y = fmaf(y, t, 0.13609223f);
    y = fmaf(y, t, 0.13562158f);
    tail = (y * t) * bell;
  } else {
    bell = exp2_hw(-0.72134752f * z * z);
    const float t = rcp_hw(fmaf(0.3275911f * 0.70710678f, fabsf(z), 1.f));
    float y = fmaf(1.061405429f, t, -1.453152027f);
    y = fmaf(y, t, 1.421413741f);
    y = fmaf(y, t, -0.284496736f);
    y = fmaf(y, t, 0.254829592f);
    tail = 0.5f * (y * t) * bell;
  }
  return z < 0.f ? tail : 1.f - tail;
}

template <typename T>
__device__ __forceinline__ float activation(int act, float z) {
  float other, bell;
  switch (act) {
    case CTR_ACT_RELU: return z < 0.f ? 0.f : z;
    case CTR_ACT_SILU: return z * sigmoid_of<T>(z, other);
    case CTR_ACT_GELU: return z * normal_below<T>(z, bell);
    case CTR_ACT_SIGMOID: return sigmoid_of<T>(z, other);
    default: return z;
  }
}

template <typename T>
__device__ __forceinline__ float derivative(int act, float z) {
  float other, bell;
  switch (act) {
    case CTR_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case CTR_ACT_SILU: {
      const float s = sigmoid_of<T>(z, other);
      return s * fmaf(z, other, 1.f);
    }
    case CTR_ACT_GELU: {
      const float below = normal_below<T>(z, bell);
      return fmaf(0.39894228040143268f * z, bell, below);
    }
    case CTR_ACT_SIGMOID: {
      const float s = sigmoid_of<T>(-fabsf(z), other);  // the smaller of both: 1 less the larger has lost what that rounded away
      return s * other;
    }
    default: return 1.f;
  }
}

// The same for N values, the choice made once.
template <typename T, int N>
__device__ __forceinline__ void activate(int act, float (&z)[N]) {
  if (act == CTR_ACT_SILU || act == CTR_ACT_SIGMOID) {
    float other;
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = (act == CTR_ACT_SILU ? z[i] : 1.f) * sigmoid_of<T>(z[i], other);
  } else if (act == CTR_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = activation<T>(CTR_ACT_GELU, z[i]);
  } else if (act == CTR_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = activation<T>(CTR_ACT_RELU, z[i]);
  }
}
// v *= the derivative at z.
template <typename T, int N>
__device__ __forceinline__ void times_derivative(int act, float (&v)[N], const float (&z)[N]) {
  if (act == CTR_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= derivative<T>(CTR_ACT_SILU, z[i]);
  } else if (act == CTR_ACT_SIGMOID) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= derivative<T>(CTR_ACT_SIGMOID, z[i]);
  } else if (act == CTR_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= derivative<T>(CTR_ACT_GELU, z[i]);
  } else if (act == CTR_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= derivative<T>(CTR_ACT_RELU, z[i]);
  }
}

}  // namespace ctr
