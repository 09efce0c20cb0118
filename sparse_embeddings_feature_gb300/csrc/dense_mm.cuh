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

// Activations (ctr_activation) and their derivatives, by the hardware's exponential and reciprocal (within 2 and 1 ulp)
// and, in gelu, erf within 1.5e-7 by Abramowitz and Stegun, Handbook of Mathematical Functions, 7.1.26: within 10 2^-24
// (|z| + 1).  With expf, erff and divisions the epilogue took twice as long as the products (65536 x 1024 x 1024 with
// silu 229 us, without an activation 84).
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

__device__ __forceinline__ float sigmoid_of(float z) { return rcp_hw(1.f + exp2_hw(-1.44269504f * z)); }

// The normal distribution's integral up to z, and exp(-z^2 / 2).
__device__ __forceinline__ float normal_below(float z, float& bell) {
  bell = exp2_hw(-0.72134752f * z * z);
  const float t = rcp_hw(fmaf(0.3275911f * 0.70710678f, fabsf(z), 1.f));
  float y = fmaf(1.061405429f, t, -1.453152027f);
  y = fmaf(y, t, 1.421413741f);
  y = fmaf(y, t, -0.284496736f);
  y = fmaf(y, t, 0.254829592f);
  const float tail = 0.5f * (y * t) * bell;
  return z < 0.f ? tail : 1.f - tail;
}

__device__ __forceinline__ float activation(int act, float z) {
  switch (act) {
    case CTR_ACT_RELU: return z < 0.f ? 0.f : z;
    case CTR_ACT_SILU: return z * sigmoid_of(z);
    case CTR_ACT_GELU: {
      float bell;
      return z * normal_below(z, bell);
    }
    case CTR_ACT_SIGMOID: return sigmoid_of(z);
    default: return z;
  }
}

__device__ __forceinline__ float derivative(int act, float z) {
  switch (act) {
    case CTR_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case CTR_ACT_SILU: {
      const float s = sigmoid_of(z);
      return s * fmaf(z, 1.f - s, 1.f);
    }
    case CTR_ACT_GELU: {
      float bell;
      const float below = normal_below(z, bell);
      return fmaf(0.39894228040143268f * z, bell, below);
    }
    case CTR_ACT_SIGMOID: {
      const float s = sigmoid_of(-fabsf(z));  // the smaller of both: 1 less the larger has lost what that rounded away
      return s * (1.f - s);
    }
    default: return 1.f;
  }
}

// The same for N values, the choice made once.
template <int N>
__device__ __forceinline__ void activate(int act, float (&z)[N]) {
  if (act == CTR_ACT_SILU || act == CTR_ACT_SIGMOID) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = (act == CTR_ACT_SILU ? z[i] : 1.f) * sigmoid_of(z[i]);
  } else if (act == CTR_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = activation(CTR_ACT_GELU, z[i]);
  } else if (act == CTR_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = activation(CTR_ACT_RELU, z[i]);
  }
}
// v *= the derivative at z.
template <int N>
__device__ __forceinline__ void times_derivative(int act, float (&v)[N], const float (&z)[N]) {
  if (act == CTR_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= derivative(CTR_ACT_SILU, z[i]);
  } else if (act == CTR_ACT_SIGMOID) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= derivative(CTR_ACT_SIGMOID, z[i]);
  } else if (act == CTR_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= derivative(CTR_ACT_GELU, z[i]);
  } else if (act == CTR_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= derivative(CTR_ACT_RELU, z[i]);
  }
}

}  // namespace ctr
