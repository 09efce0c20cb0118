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

// How a product is taken apart: CTA pairs on 256 x 256 tiles or CTAs on 128 x 128, and sums in `splits` parts of
// `seg` blocks of 64, which leave as fp32 planes of m x ld and are added up by a second kernel.
struct MmPlan {
  bool pair = false;
  int32_t seg = 0, splits = 1;
  int64_t ld = 0;
  size_t bytes(int64_t m) const { return splits > 1 ? (size_t)splits * m * ld * 4 : 0; }
};
MmPlan mm_plan(int major, int planes, int64_t m, int64_t n, int64_t r);

// Runs the product; `part` has mm_plan(..).bytes(m) bytes, 256-byte aligned.  A ctr_status.
int mm_run(const MmCall& c, float* part, cudaStream_t s);

// The value of an activation (ctr_activation).
__device__ __forceinline__ float sigmoid_of(float z) { return 1.f / (1.f + expf(-z)); }

__device__ __forceinline__ float activation(int act, float z) {
  switch (act) {
    case CTR_ACT_RELU: return z < 0.f ? 0.f : z;
    case CTR_ACT_SILU: return z * sigmoid_of(z);
    case CTR_ACT_GELU: return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    case CTR_ACT_SIGMOID: return sigmoid_of(z);
    default: return z;
  }
}

}  // namespace ctr
