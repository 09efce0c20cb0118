// Typed vector access to rows of fp32 or bf16 elements, shared by the expert
// layer's kernels: VB bytes (16, 8, 4 or 2) at a time, converted to fp32.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace ctr {

template <int VB>
struct RawOf;
template <>
struct RawOf<16> {
  using type = uint4;
};
template <>
struct RawOf<8> {
  using type = uint2;
};
template <>
struct RawOf<4> {
  using type = uint32_t;
};
template <>
struct RawOf<2> {
  using type = uint16_t;
};

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// VB bytes of T elements as fp32 values, and back (each value rounded once).  bf16 pairs are taken
// apart as words (a shift, a mask) and put together two at a time: element by element the compiler
// spent about twice the instructions.
template <typename T, int VB>
struct Chunk {
  static constexpr int n = VB / (int)sizeof(T);
  static constexpr int words = VB / 4;
  using Raw = typename RawOf<VB>::type;
  union Bits {
    Raw raw;
    uint32_t w[words > 0 ? words : 1];
    uint16_t h;
    __device__ Bits() {}
  };
  static __device__ __forceinline__ void unpack(const Raw& raw, float (&f)[n]) {
    Bits b;
    b.raw = raw;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < n; ++i) f[i] = __uint_as_float(b.w[i]);
    } else if constexpr (VB == 2) {
      f[0] = __uint_as_float((uint32_t)b.h << 16);
    } else {
#pragma unroll
      for (int i = 0; i < words; ++i) {
        f[2 * i] = __uint_as_float(b.w[i] << 16);
        f[2 * i + 1] = __uint_as_float(b.w[i] & 0xffff0000u);
      }
    }
  }
  static __device__ __forceinline__ Raw pack(const float (&f)[n]) {
    Bits b;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < n; ++i) b.w[i] = __float_as_uint(f[i]);
    } else if constexpr (VB == 2) {
      b.h = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
    } else {
#pragma unroll
      for (int i = 0; i < words; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        b.w[i] = *(const uint32_t*)&p;
      }
    }
    return b.raw;
  }
};

// Widest access (16, 8, 4 or 2 bytes, at least one element) that divides every
// argument: base addresses, row strides and row lengths in bytes.
inline int vector_bytes(std::initializer_list<uint64_t> parts, int elem) {
  uint64_t all = 16;
  for (uint64_t p : parts) all |= p;
  const int low = (int)(all & (~all + 1));  // the lowest set bit, at most 16
  return low < elem ? elem : low;
}

inline bool dtype_ok(int dtype) { return dtype == CTR_F32 || dtype == CTR_BF16; }
inline int dtype_bytes(int dtype) { return dtype == CTR_F32 ? 4 : 2; }

}  // namespace ctr
