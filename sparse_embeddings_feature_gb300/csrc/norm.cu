// c1. Root-mean-square norm on a residual stream, its 8-bit codes, and its gradient.
//
// Source: "DHEN" notes, section 2.2 (a layer's output is Norm(Ensemble(...) +
// ShortCut)); the page names no norm, the formulas are stated in include/ctr.h.
//
// A row is held in registers by a group of lanes (8 lanes up to 128 columns, a
// warp up to 1024, up to 16 warps beyond), read once and written once: sum, sum of
// squares, result and codes need no second pass.  A warp owns a contiguous run of
// 32 EPT columns, so that a block of 128 columns never crosses warps and its
// largest magnitude is a few shuffles.  Sums are fp32; bound by HBM.
//
// Backward.  With u = s rstd:  dx = ds + rstd (g - u mean(g u)), g = dy gamma, and
// dgamma = sum over rows of dy u.  A block walks rows with its columns' sums in
// registers, adds its warps' up through shared memory in their order, and leaves
// one partial row; a second kernel adds those in their order.  No atomics, so the
// result is the same in every run.
#include <cuda_bf16.h>

#include <algorithm>
#include <initializer_list>

#include "codes.cuh"
#include "common.cuh"
#include "rows.cuh"

namespace ctr {
namespace {

constexpr int kNormMaxCols = CTR_MAX_NORM_WIDTH;  // 16 warps of 1024 columns
static_assert(kNormMaxCols <= 16 * 1024, "a row has 16 warps at most");
constexpr int kNormParts = 304;      // blocks of the backward, at most: two an SM of 152
constexpr int kJoinCols = 32, kJoinRows = 16;

struct NormArgs {
  const void* x;
  const void* residual;  // forward: NULL without; backward: the gradient that arrives on the stream
  const void* dy;        // backward
  const float* gamma;    // NULL: all 1
  void* s;               // NULL: not wanted
  void* y;               // forward: NULL for codes alone; backward: dx
  uint8_t* q;
  float* scale;
  float* part;           // backward: partial sums of dgamma
  int64_t rows, ldx, ldr, lds, ldy, ld_dy, ld_scale;
  int32_t d, qcols, wpr; // qcols: d rounded up to blocks; wpr: warps to a row
  int32_t gvec;          // gamma is 16-byte aligned
  float eps;
};

// Where a thread's elements are: chunk c of a lane holds columns col(c) .. col(c) + n - 1.
template <int N, int LANES, int EPT>
struct Place {
  static constexpr int span = LANES * EPT;  // columns of a lane group
  int first, sub;
  __device__ __forceinline__ Place(int warp_in_row, int lane)
      : first(warp_in_row * span + (lane & (LANES - 1)) * N), sub(lane & (LANES - 1)) {}
  __device__ __forceinline__ int col(int c) const { return first + c * (LANES * N); }
};

// A thread's elements are kept as pairs: most of the arithmetic is two operations an instruction.
template <typename T, int VB, int EPT>
struct Raw {
  using C = Chunk<T, VB>;
  static constexpr int N = C::n, chunks = EPT / N;
  typename C::Raw c[chunks];
  template <typename P>
  __device__ __forceinline__ void load(const P& at, const T* row, int d, bool mine) {
#pragma unroll
    for (int i = 0; i < chunks; ++i) {
      c[i] = typename C::Raw{};
      if (mine && at.col(i) < d) c[i] = *(const typename C::Raw*)(row + at.col(i));
    }
  }
  template <typename P>
  __device__ __forceinline__ void store(const P& at, T* row, int d) const {
#pragma unroll
    for (int i = 0; i < chunks; ++i)
      if (at.col(i) < d) *(typename C::Raw*)(row + at.col(i)) = c[i];
  }
  __device__ __forceinline__ void get(float2 (&f)[EPT / 2]) const {
#pragma unroll
    for (int i = 0; i < chunks; ++i) {
      float v[N];
      C::unpack(c[i], v);
#pragma unroll
      for (int j = 0; j < N; ++j) ((j + i * N) & 1 ? f[(i * N + j) / 2].y : f[(i * N + j) / 2].x) = v[j];
    }
  }
  __device__ __forceinline__ void set(const float2 (&f)[EPT / 2]) {
#pragma unroll
    for (int i = 0; i < chunks; ++i) {
      float v[N];
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = (j + i * N) & 1 ? f[(i * N + j) / 2].y : f[(i * N + j) / 2].x;
      c[i] = C::pack(v);
    }
  }
};

// f *= gamma's values at a thread's columns.
template <int N, int EPT, typename P>
__device__ __forceinline__ void times_gamma(const P& at, const NormArgs& a, float2 (&f)[EPT / 2]) {
  if (!a.gamma) return;
#pragma unroll
  for (int c = 0; c < EPT / N; ++c) {
    float g[N];
    if (N >= 4 && a.gvec) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const float4 v = at.col(c) < a.d ? *(const float4*)(a.gamma + at.col(c) + i) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4 && i + j < N; ++j) g[i + j] = w[j];
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) g[i] = at.col(c) < a.d ? a.gamma[at.col(c) + i] : 0.f;
    }
    if constexpr (N >= 2) {
#pragma unroll
      for (int i = 0; i < N; i += 2) f[(c * N + i) / 2] = mul2(f[(c * N + i) / 2], make_float2(g[i], g[i + 1]));
    } else {
      if (c & 1) f[c / 2].y *= g[0];
      else f[c / 2].x *= g[0];
    }
  }
}

// Sum over a row's lanes, the same in all of them.  wpr > 1: the row's warps meet at a barrier of their own; `sums` has a
// word a warp of the block, and is not used again before another of the row's sums.
template <int LANES>
__device__ __forceinline__ float row_sum(float v, int wpr, float* sums) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) v += __shfl_xor_sync(kFull, v, o);
  if (wpr > 1) {
    const int warp = threadIdx.x >> 5, first = warp & ~(wpr - 1);
    if ((threadIdx.x & 31) == 0) sums[warp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + first / wpr), "r"(32 * wpr) : "memory");
    v = 0.f;
    for (int w = 0; w < wpr; ++w) v += sums[first + w];
  }
  return v;
}

// 1 / sqrt(mean(f^2) + eps) over a row.  Squares that leave fp32's range (or all but do, against a small eps)
// are taken again of scaled values (2^-80: kNormMaxCols squares of fp32's largest number are 2^110); a NaN or an infinity in the row gives NaN or 0, and NaN results.
template <int LANES, int EPT>
__device__ __forceinline__ float row_rstd(const float2 (&f)[EPT / 2], const NormArgs& a, float (*sums)[16]) {
  float2 sq = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < EPT / 2; ++i) sq = fma2(f[i], f[i], sq);
  const float total = row_sum<LANES>(sq.x + sq.y, a.wpr, sums[0]);
  const float mean = total / (float)a.d + a.eps;
  float rstd = 1.f / sqrtf(mean);
  const bool odd = !(mean < 1e37f) || mean < 1e-30f;  // the same in all of a row's threads
  if (__any_sync(kFull, odd)) {
    const float by = mean < 1e-30f ? 0x1p70f : 0x1p-80f;
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < EPT / 2; ++i) {
      t = fmaf(f[i].x * by, f[i].x * by, t);
      t = fmaf(f[i].y * by, f[i].y * by, t);
    }
    t = row_sum<LANES>(t, a.wpr, sums[1]);
    if (odd) rstd = (float)((double)by / sqrt((double)t / a.d + (double)a.eps * by * by));
  }
  return rstd;
}

// The largest of three magnitudes, NaN winning.
__device__ __forceinline__ float max_mag3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Codes of a thread's values: the largest magnitude of each block of 128 columns, its scale and the bytes.
template <int N, int LANES, int EPT, typename P>
__device__ __forceinline__ void store_codes(const P& at, const NormArgs& a, int64_t r, bool mine, const float2 (&f)[EPT / 2]) {
  constexpr int kChunks = EPT / N;
  constexpr int kWide = LANES * N;                       // columns of a chunk over the lanes
  constexpr int kPer = kWide >= 128 ? 1 : (LANES == 32 ? 128 / kWide : kChunks);  // chunks of a block
  constexpr int kLanes = kWide >= 128 ? 128 / N : LANES;  // lanes of a block
#pragma unroll
  for (int c0 = 0; c0 < kChunks; c0 += kPer) {
    float m = 0.f;
#pragma unroll
    for (int i = c0 * N / 2; i < (c0 + kPer) * N / 2; ++i) m = max_mag3(m, f[i].x, f[i].y);
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) m = max_mag(m, __shfl_xor_sync(kFull, m, o));
    m = at_least_floor(m);
    const float inv = __fdiv_rn(kTop, m);
    if (!mine) continue;
    if ((at.sub & (kLanes - 1)) == 0 && at.col(c0) < a.qcols)
      a.scale[(int64_t)(at.col(c0) / 128) * a.ld_scale + r] = __fdiv_rn(m, kTop);
    uint8_t* row = a.q + r * a.qcols;
#pragma unroll
    for (int c = c0; c < c0 + kPer; ++c) {
      if (at.col(c) >= a.qcols) continue;
      if constexpr (N >= 4) {
        uint32_t w[N / 4];
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          const float2 lo = f[(c * N + i) / 2], hi = f[(c * N + i) / 2 + 1];
          const float v[4] = {lo.x, lo.y, hi.x, hi.y};
          w[i / 4] = codes4(v, inv);
        }
        if constexpr (N == 8) *(uint2*)(row + at.col(c)) = make_uint2(w[0], w[1]);
        else *(uint32_t*)(row + at.col(c)) = w[0];
      } else {
        static_assert(N == 1, "whole parts or single elements");
        const float one[4] = {c & 1 ? f[c / 2].y : f[c / 2].x, 0.f, 0.f, 0.f};
        row[at.col(c)] = (uint8_t)codes4(one, inv);
      }
    }
  }
}

// qcols may be past what 8 lanes hold of a narrow row: a group of 8 lanes covers 64 or 128 columns, and the
// codes' row is 128; the rest is zeros.
template <int LANES, int EPT, typename P>
__device__ __forceinline__ void zero_codes(const P& at, const NormArgs& a, int64_t r, bool mine) {
  if constexpr (LANES * EPT < 128) {
    if (mine)
      for (int c = LANES * EPT + at.sub * 4; c < a.qcols; c += LANES * 4) *(uint32_t*)(a.q + r * a.qcols + c) = 0;
  }
}

// THREADS: 512 where a row has 16 warps, else 256.  Blocks of an SM: bf16 rows want more threads at once than fp32 ones,
// whose loads are twice as wide.
template <typename T>
constexpr int kNormThreads = sizeof(T) == 2 ? 1024 : 768;

template <typename T, int VB, int LANES, int EPT, int THREADS>
__global__ void __launch_bounds__(THREADS, kNormThreads<T> / THREADS) rms_norm_kernel(const NormArgs a) {
  constexpr int N = Chunk<T, VB>::n;
  using Row = Raw<T, VB, EPT>;
  __shared__ float sums[2][16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_block = THREADS / (LANES * a.wpr);  // rows of a block
  const Place<N, LANES, EPT> at(warp & (a.wpr - 1), lane);
  const int64_t r = (int64_t)blockIdx.x * per_block + (int)threadIdx.x / (LANES * a.wpr);
  const bool mine = r < a.rows;
  grid_wait();
  float2 f[EPT / 2];
  {
    Row x, p;
    x.load(at, (const T*)a.x + r * a.ldx, a.d, mine);
    if (a.residual) {
      p.load(at, (const T*)a.residual + r * a.ldr, a.d, mine);
      float2 g[EPT / 2];
      x.get(f);
      p.get(g);
#pragma unroll
      for (int i = 0; i < EPT / 2; ++i) f[i] = add2(f[i], g[i]);
      x.set(f);  // the stream's value is what its type holds
    }
    if (a.s && mine) x.store(at, (T*)a.s + r * a.lds, a.d);
    x.get(f);
  }
  const float rstd = row_rstd<LANES, EPT>(f, a, sums);
  const float2 by = make_float2(rstd, rstd);
#pragma unroll
  for (int i = 0; i < EPT / 2; ++i) f[i] = mul2(f[i], by);
  times_gamma<N, EPT>(at, a, f);
  if (a.y && mine) {
    Row y;
    y.set(f);
    y.store(at, (T*)a.y + r * a.ldy, a.d);
  }
  if (a.q) {
    store_codes<N, LANES, EPT>(at, a, r, mine, f);
    zero_codes<LANES, EPT>(at, a, r, mine);
  }
}

template <typename T, int VB, int LANES, int EPT, int THREADS>
__global__ void __launch_bounds__(THREADS, 512 / THREADS) rms_norm_bwd_kernel(const NormArgs a) {
  constexpr int N = Chunk<T, VB>::n;
  using Row = Raw<T, VB, EPT>;
  extern __shared__ float total[];  // a column's sum over the block's rows
  __shared__ float sums[3][16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_block = THREADS / (LANES * a.wpr);
  const Place<N, LANES, EPT> at(warp & (a.wpr - 1), lane);
  float2 acc[EPT / 2];
#pragma unroll
  for (int i = 0; i < EPT / 2; ++i) acc[i] = make_float2(0.f, 0.f);
  grid_wait();
  const int64_t step = (int64_t)gridDim.x * per_block;
  const int64_t trips = ceil_div(a.rows, step);  // the same in every thread: sums over a row need all of them
  int64_t r = (int64_t)blockIdx.x * per_block + (int)threadIdx.x / (LANES * a.wpr);
  // bf16 rows, half as many registers as fp32 ones, are asked for while the row before is worked on.
  constexpr bool kAhead = sizeof(T) == 2;
  Row x, y, p;
  auto fetch = [&](int64_t row) {
    const bool mine = row < a.rows;  // nothing past the last row
    x.load(at, (const T*)a.x + row * a.ldx, a.d, mine);
    y.load(at, (const T*)a.dy + row * a.ld_dy, a.d, mine);
    if (kAhead && a.residual) p.load(at, (const T*)a.residual + row * a.ldr, a.d, mine);
  };
  if (kAhead) fetch(r);
  for (int64_t trip = 0; trip < trips; ++trip, r += step) {
    const bool mine = r < a.rows;
    float2 u[EPT / 2], g[EPT / 2];
    Row arrived;  // the gradient on the stream
    if (!kAhead) fetch(r);
    x.get(u);
    y.get(g);
    if (kAhead) {
      arrived = p;
      fetch(r + step);
    }
    const float rstd = row_rstd<LANES, EPT>(u, a, sums);
    const float2 by = make_float2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < EPT / 2; ++i) {
      u[i] = mul2(u[i], by);
      acc[i] = fma2(g[i], u[i], acc[i]);  // rows past the last are zeros
    }
    times_gamma<N, EPT>(at, a, g);
    float2 dot2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < EPT / 2; ++i) dot2 = fma2(g[i], u[i], dot2);
    const float dot = -row_sum<LANES>(dot2.x + dot2.y, a.wpr, sums[2]) / (float)a.d;
    const float2 less = make_float2(dot, dot);
#pragma unroll
    for (int i = 0; i < EPT / 2; ++i) g[i] = mul2(fma2(u[i], less, g[i]), by);
    if (a.residual) {
      if (!kAhead) arrived.load(at, (const T*)a.residual + r * a.ldr, a.d, mine);
      arrived.get(u);
#pragma unroll
      for (int i = 0; i < EPT / 2; ++i) g[i] = add2(g[i], u[i]);
    }
    if (mine) {
      Row out;
      out.set(g);
      out.store(at, (T*)a.y + r * a.ldy, a.d);
    }
  }
  if (!a.part) return;
  // lane groups of a warp in the order of their rows, then the warps
#pragma unroll
  for (int o = LANES; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < EPT / 2; ++i) {
      acc[i].x += __shfl_xor_sync(kFull, acc[i].x, o);
      acc[i].y += __shfl_xor_sync(kFull, acc[i].y, o);
    }
  const int groups = (int)(blockDim.x >> 5) / a.wpr;  // warps that hold the same columns
  for (int w = 0; w < groups; ++w) {
    if (warp / a.wpr == w && lane < LANES) {
#pragma unroll
      for (int c = 0; c < EPT / N; ++c)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int col = at.col(c) + i;
          const float v = (c * N + i) & 1 ? acc[(c * N + i) / 2].y : acc[(c * N + i) / 2].x;
          if (col < a.d) total[col] = (w ? total[col] : 0.f) + v;
        }
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < a.d; c += blockDim.x) a.part[(int64_t)blockIdx.x * a.d + c] = total[c];
}

// dgamma[c] = the sum of the partial rows, kJoinRows strands of them and then the strands, in their order.
__global__ void __launch_bounds__(kJoinCols* kJoinRows) join_rows_kernel(const float* part, int parts, int d, float* out) {
  __shared__ float strand[kJoinRows][kJoinCols + 1];
  grid_wait();
  const int x = threadIdx.x % kJoinCols, y = threadIdx.x / kJoinCols;
  const int c = blockIdx.x * kJoinCols + x;
  float sum = 0.f;
  if (c < d) {
#pragma unroll 4
    for (int p = y; p < parts; p += kJoinRows) sum += part[(int64_t)p * d + c];
  }
  strand[y][x] = sum;
  __syncthreads();
  if (y == 0 && c < d) {
    for (int i = 1; i < kJoinRows; ++i) sum += strand[i][x];
    out[c] = sum;
  }
}

// Lanes and elements of a thread by the row's width.  most: elements of a thread of wide rows, which take more warps
// instead: 32, but for bf16 rows in the backward kernel, which holds three of them, the next three and the columns' sums
// (65536 x 2048: 198 us; 32 and the next row not asked for, 238; 16 and three blocks an SM, 253).
template <template <typename, int, int, int, int> class K, typename T, int VB>
auto pick_width(int d) {
  constexpr int kMost = K<T, VB, 32, 8, 256>::most;
  return d <= 64 ? K<T, VB, 8, 8, 256>::get() : d <= 128 ? K<T, VB, 8, 16, 256>::get()
       : d <= 256 ? K<T, VB, 32, 8, 256>::get() : d <= 512 ? K<T, VB, 32, 16, 256>::get()
       : d <= 8 * 32 * kMost ? K<T, VB, 32, kMost, 256>::get()
       : d <= 16 * 32 * kMost ? K<T, VB, 32, kMost, 512>::get() : K<T, VB, 32, 32, 512>::get();
}
template <typename T, int VB, int LANES, int EPT, int THREADS>
struct Forward {
  static constexpr int most = 32;
  static auto get() { return rms_norm_kernel<T, VB, LANES, EPT, THREADS>; }
};
template <typename T, int VB, int LANES, int EPT, int THREADS>
struct Backward {
  static constexpr int most = sizeof(T) == 2 ? 16 : 32;
  static auto get() { return rms_norm_bwd_kernel<T, VB, LANES, EPT, THREADS>; }
};
template <template <typename, int, int, int, int> class K>
auto pick(ctr_dtype dtype, bool wide, int d) {
  if (dtype == CTR_F32) return wide ? pick_width<K, float, 16>(d) : pick_width<K, float, 4>(d);
  return wide ? pick_width<K, __nv_bfloat16, 16>(d) : pick_width<K, __nv_bfloat16, 2>(d);
}

struct NormPlan {
  int lanes, wpr = 1, threads = 256, per_block;
  NormPlan(int d, bool backward, int dtype) {
    const int most = !backward ? Forward<float, 16, 32, 8, 256>::most
                     : dtype == CTR_F32 ? Backward<float, 16, 32, 8, 256>::most : Backward<__nv_bfloat16, 16, 32, 8, 256>::most;
    lanes = d <= 128 ? 8 : 32;
    while (wpr < 16 && wpr * 32 * most < d) wpr *= 2;
    if (wpr > 8) threads = 512;
    per_block = threads / (lanes * wpr);
  }
};

int norm_parts(int64_t rows, int d, int dtype) {
  return (int)imin64(kNormParts, ceil_div(rows, NormPlan(d, true, dtype).per_block));
}

bool misaligned(const void* p, int by) { return ((uintptr_t)p % by) != 0; }

int check_norm(ctr_dtype dtype, int64_t rows, int32_t d, float eps) {
  if (!dtype_ok(dtype) || rows < 0 || d < 1 || !(eps > 0.f) || !(eps < INFINITY)) return CTR_ERR_INVALID_ARG;
  if (d > kNormMaxCols || rows > INT32_MAX - 65536) return CTR_ERR_UNSUPPORTED;
  return CTR_OK;
}

}  // namespace
}  // namespace ctr

using namespace ctr;

extern "C" size_t ctr_rms_norm_workspace_size(int64_t rows, int32_t d) {
  if (rows < 0 || d < 1 || d > kNormMaxCols) return 0;
  WsSizer z;
  z.take<float>((size_t)std::max(norm_parts(rows, d, CTR_F32), norm_parts(rows, d, CTR_BF16)) * d);
  return z.used;
}

extern "C" int ctr_rms_norm(const void* x, ctr_dtype dtype, int64_t rows, int32_t d, int64_t ldx, const void* residual,
                            int64_t ld_residual, const float* gamma, float eps, void* s, int64_t ld_s, void* y,
                            int64_t ld_y, uint8_t* q, float* scale, int64_t ld_scale, void* ws, size_t ws_bytes,
                            ctr_stream_t stream) {
  const int st = check_norm(dtype, rows, d, eps);
  if (st != CTR_OK) return st;
  if ((q == nullptr) != (scale == nullptr) || (!y && !q && rows > 0)) return CTR_ERR_INVALID_ARG;
  if (ldx < d || (residual && ld_residual < d) || (s && ld_s < d) || (y && ld_y < d) || (q && ld_scale < rows))
    return CTR_ERR_INVALID_ARG;
  const int eb = dtype_bytes(dtype);
  if (rows > 0 && !x) return CTR_ERR_INVALID_ARG;
  for (const void* p : {x, residual, (const void*)s, (const void*)y})
    if (misaligned(p, eb)) return CTR_ERR_INVALID_ARG;
  if (misaligned(gamma, 4) || misaligned(scale, 4) || misaligned(q, 16)) return CTR_ERR_INVALID_ARG;
  if (!ws_valid(ws, ws_bytes, kWsHeader)) return CTR_ERR_WORKSPACE;
  if (rows == 0) return CTR_OK;
  const NormPlan plan(d, false, dtype);
  NormArgs a = {};
  a.x = x;
  a.residual = residual;
  a.gamma = gamma;
  a.s = s;
  a.y = y;
  a.q = q;
  a.scale = scale;
  a.rows = rows;
  a.ldx = ldx;
  a.ldr = ld_residual;
  a.lds = ld_s;
  a.ldy = ld_y;
  a.ld_scale = ld_scale;
  a.d = d;
  a.qcols = (d + 127) / 128 * 128;
  a.wpr = plan.wpr;
  a.gvec = !misaligned(gamma, 16);
  a.eps = eps;
  uint64_t parts = (uint64_t)x | (uint64_t)(ldx * eb) | (uint64_t)d * eb;
  if (residual) parts |= (uint64_t)residual | (uint64_t)(ld_residual * eb);
  if (s) parts |= (uint64_t)s | (uint64_t)(ld_s * eb);
  if (y) parts |= (uint64_t)y | (uint64_t)(ld_y * eb);
  const cudaError_t e = launch_after(pick<Forward>(dtype, parts % 16 == 0, d),
                                     dim3((unsigned)ceil_div(rows, plan.per_block)), plan.threads, 0,
                                     (cudaStream_t)stream, 1, a);
  return e == cudaSuccess ? launch_status() : CTR_ERR_CUDA;
}

extern "C" int ctr_rms_norm_bwd(const void* dy, ctr_dtype dtype, int64_t rows, int32_t d, int64_t ld_dy, const void* ds,
                                int64_t ld_ds, const void* s, int64_t ld_s, const float* gamma, float eps, void* dx,
                                int64_t ld_dx, float* dgamma, void* ws, size_t ws_bytes, ctr_stream_t stream) {
  const int st = check_norm(dtype, rows, d, eps);
  if (st != CTR_OK) return st;
  if (ld_dy < d || (ds && ld_ds < d) || ld_s < d || ld_dx < d) return CTR_ERR_INVALID_ARG;
  if (rows > 0 && (!dy || !s || !dx)) return CTR_ERR_INVALID_ARG;
  const int eb = dtype_bytes(dtype);
  for (const void* p : {dy, ds, s, (const void*)dx})
    if (misaligned(p, eb)) return CTR_ERR_INVALID_ARG;
  if (misaligned(gamma, 4) || misaligned(dgamma, 4)) return CTR_ERR_INVALID_ARG;
  if (!ws_valid(ws, ws_bytes, dgamma ? ctr_rms_norm_workspace_size(rows, d) : kWsHeader)) return CTR_ERR_WORKSPACE;
  const cudaStream_t stm = (cudaStream_t)stream;
  const NormPlan plan(d, true, dtype);
  const int parts = norm_parts(rows, d, dtype);
  WsCarver c(ws, ws_bytes);
  float* part = dgamma ? c.take<float>((size_t)parts * d) : nullptr;
  if (rows > 0) {
    NormArgs a = {};
    a.x = s;
    a.residual = ds;
    a.dy = dy;
    a.gamma = gamma;
    a.y = dx;
    a.part = part;
    a.rows = rows;
    a.ldx = ld_s;
    a.ldr = ld_ds;
    a.ld_dy = ld_dy;
    a.ldy = ld_dx;
    a.d = d;
    a.wpr = plan.wpr;
    a.gvec = !misaligned(gamma, 16);
    a.eps = eps;
    uint64_t all = (uint64_t)dy | (uint64_t)s | (uint64_t)dx | (uint64_t)(ld_dy * eb) | (uint64_t)(ld_s * eb) |
                   (uint64_t)(ld_dx * eb) | (uint64_t)d * eb;
    if (ds) all |= (uint64_t)ds | (uint64_t)(ld_ds * eb);
    const auto k = pick<Backward>(dtype, all % 16 == 0, d);
    const size_t smem = (size_t)d * 4;
    if (smem > 48 * 1024 && !allow_smem(k, smem)) return CTR_ERR_CUDA;
    if (launch_after(k, dim3((unsigned)parts), plan.threads, smem, stm, 1, a) != cudaSuccess) return CTR_ERR_CUDA;
  }
  if (dgamma &&
      launch_after(join_rows_kernel, dim3((unsigned)ceil_div(d, kJoinCols)), kJoinCols * kJoinRows, 0, stm, 1,
                   (const float*)part, parts, (int)d, dgamma) != cudaSuccess)
    return CTR_ERR_CUDA;
  return launch_status();
}
