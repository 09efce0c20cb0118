// e4m3 codes of blocks of 128 values: the scale's arithmetic and the conversion, shared by the quantisers
// and by the kernels that write codes of what they compute.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace ctr {

constexpr float kTop = 448.f;         // largest e4m3 value
constexpr float kFloor = 0x1p-100f;

// NaN stays NaN (the comparison is false for it).
__device__ __forceinline__ float at_least_floor(float m) { return m < kFloor ? kFloor : m; }

// The larger magnitude, NaN winning.
__device__ __forceinline__ float max_mag(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

template <int N>
__device__ __forceinline__ float max_mag(const float (&v)[N]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) m = max_mag(m, v[i]);
  return m;
}

// (x, y) * inv, each rounded to fp32, in one instruction.
__device__ __forceinline__ float2 times(float x, float y, float inv) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c;\n\t"
      "mov.b64 a, {%2, %3};\n\t"
      "mov.b64 b, {%4, %4};\n\t"
      "mul.rn.f32x2 c, a, b;\n\t"
      "mov.b64 {%0, %1}, c;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x), "f"(y), "f"(inv));
  return r;
}

// Four codes, put together as halves of a word.
__device__ __forceinline__ uint32_t codes4(const float* v, float inv) {
  const float2 a = times(v[0], v[1], inv), b = times(v[2], v[3], inv);
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

}  // namespace ctr
