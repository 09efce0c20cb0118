// b4. Global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum g^2),  out = g * (norm > max_norm ? max_norm / norm : 1)
//
// The tensors are cut into chunks of kChunk elements, handed to the blocks in a
// fixed order.  A thread squares and adds its part of a chunk in fp32 (four
// accumulators), adds up to kFlush chunks in fp32 and then moves the sum into
// fp64; joins are fp64 in a fixed order, so the result does not change from run
// to run.  A part whose sum of squares comes near either end of fp32's range is
// read again and squared in fp64 by its warp (fp64 in the common path, even
// predicated off, tripled the pass: 724 us against 248 for 5e8 elements), unless
// all of it is zero, as the weight gradient of an expert without rows is (2.5e8
// fp32 zeros 150 us; in fp64 973).  Every
// block of the second pass adds the first one's sums up for itself, in the same
// order: no counter, and no launch between the two.  Two passes over the data,
// bound by HBM: the second walks the chunks in reverse, so what the first read
// last is still in L2.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "rows.cuh"

namespace ctr {
namespace {

constexpr int kClipThreads = 256;
constexpr int kChunk = 8192;        // elements of a chunk
constexpr int kListMax = 256;       // tensors of one launch
constexpr int kClipBlocksPerSm = 6;
constexpr int kMaxBlocks = 2048;    // bound of a launch's grid
constexpr int kMaxSums = 16384;     // bound of all launches' blocks, for the workspace
constexpr int kFlush = 8;           // chunks between moves of the fp32 sums into fp64
// A thread's sum over its part of a chunk is used within these bounds: above, a sum of them could
// overflow; below, squares that fall under fp32's smallest numbers would weigh in (at or above it
// they are under 2^-149 x 32 of 2^-100).
constexpr float kBig = 0x1p100f;
constexpr float kSmall = 0x1p-100f;

struct ClipList {
  const void* g[kListMax];
  void* out[kListMax];
  int64_t n[kListMax];
  int64_t first[kListMax + 1];  // chunks before each tensor
  uint8_t dtype[kListMax];
  int32_t count;
};

__device__ __forceinline__ int tensor_of(const ClipList& l, int64_t chunk) {
  int lo = 0, hi = l.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (l.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Sum of squares of this thread's part of a chunk: 16-byte pieces where the chunk is aligned.  nonzero: whether
// any of its magnitudes has a bit set, which tells zeros from squares that were too small for fp32.
template <typename T>
__device__ __forceinline__ float chunk_squares(const T* g, int n, bool& nonzero) {
  constexpr int per = 16 / (int)sizeof(T);
  constexpr int pieces = kChunk / per / kClipThreads;
  constexpr uint32_t kMagnitude = sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  uint32_t bits = 0;
  int i0 = 0;
  if (((uintptr_t)g & 15) == 0) {
    const int full = n / per;
    i0 = full * per;
    uint4 raw[pieces];
#pragma unroll
    for (int p = 0; p < pieces; ++p) {
      const int i = threadIdx.x + p * kClipThreads;
      raw[p] = i < full ? ((const uint4*)g)[i] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int p = 0; p < pieces; ++p) {
      float f[per];
      Chunk<T, 16>::unpack(raw[p], f);
      bits |= (raw[p].x | raw[p].y | raw[p].z | raw[p].w) & kMagnitude;
#pragma unroll
      for (int i = 0; i < per; ++i) acc[i & 3] = fmaf(f[i], f[i], acc[i & 3]);
    }
  }
#pragma unroll 4
  for (int i = i0 + threadIdx.x; i < n; i += kClipThreads) {
    const float f = to_f32<T>(g[i]);
    acc[0] = fmaf(f, f, acc[0]);
    bits |= __float_as_uint(f) & 0x7fffffffu;
  }
  nonzero = bits != 0;
  return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

// The same elements of the same thread in fp64.
template <typename T>
__device__ __noinline__ double chunk_squares_wide(const T* g, int n) {
  constexpr int per = 16 / (int)sizeof(T);
  double s = 0.0;
  int i0 = 0;
  if (((uintptr_t)g & 15) == 0) {
    i0 = n / per * per;
    for (int p = threadIdx.x * per; p < i0; p += kClipThreads * per)
      for (int e = 0; e < per; ++e) {
        const float f = to_f32<T>(g[p + e]);
        if (f != 0.f) s += (double)f * (double)f;  // true for NaN
      }
  }
  for (int i = i0 + threadIdx.x; i < n; i += kClipThreads) {
    const float f = to_f32<T>(g[i]);
    if (f != 0.f) s += (double)f * (double)f;
  }
  return s;
}

// Sum over the block's threads, valid in thread 0.
__device__ __forceinline__ double block_sum(double v, double* warp_sum) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_down_sync(kFull, v, o);
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < kClipThreads / 32; ++w) s += warp_sum[w];
  return s;
}

__global__ void __launch_bounds__(kClipThreads) norm_kernel(const __grid_constant__ ClipList l, double* part) {
  __shared__ double warp_sum[kClipThreads / 32];
  grid_wait();
  float acc = 0.f;
  double wide = 0.0;
  int since = 0;
  for (int64_t c = blockIdx.x; c < l.first[l.count]; c += gridDim.x) {
    const int t = tensor_of(l, c);
    const int64_t e0 = (c - l.first[t]) * kChunk;
    const int n = (int)imin64(kChunk, l.n[t] - e0);
    const bool f32 = l.dtype[t] == CTR_F32;
    const float* g32 = (const float*)l.g[t] + e0;
    const __nv_bfloat16* g16 = (const __nv_bfloat16*)l.g[t] + e0;
    bool nonzero;
    const float sum = f32 ? chunk_squares(g32, n, nonzero) : chunk_squares(g16, n, nonzero);
    const bool odd = !(sum <= kBig) || (sum < kSmall && nonzero);
    if (__any_sync(kFull, odd)) {
      wide += f32 ? chunk_squares_wide(g32, n) : chunk_squares_wide(g16, n);
    } else {
      acc += sum;
    }
    if (++since == kFlush) {
      wide += (double)acc;
      acc = 0.f;
      since = 0;
    }
  }
  wide += (double)acc;
  wide = block_sum(wide, warp_sum);
  if (threadIdx.x == 0) part[blockIdx.x] = wide;
}

// The factor of the n sums in part; the first block of a launch that is told to writes the norm.
__device__ __forceinline__ float clip_factor(const double* part, int n, float max_norm, float* norm) {
  __shared__ double warp_sum[kClipThreads / 32];
  __shared__ float factor;
  double s = 0.0;
  for (int b = threadIdx.x; b < n; b += kClipThreads) s += part[b];
  s = block_sum(s, warp_sum);
  if (threadIdx.x == 0) {
    const float v = (float)sqrt(s);
    if (norm && blockIdx.x == 0) *norm = v;
    factor = v > max_norm && v < INFINITY ? max_norm / v : 1.f;  // NaN and inf leave the gradients as they are
  }
  __syncthreads();
  return factor;
}

__global__ void __launch_bounds__(kClipThreads) norm_only_kernel(const double* part, int n, float* norm) {
  grid_wait();
  clip_factor(part, n, 0.f, norm);
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T* g, T* out, int n, float f) {
  constexpr int per = 16 / (int)sizeof(T);
  int i0 = 0;
  if ((((uintptr_t)g | (uintptr_t)out) & 15) == 0) {
    i0 = n / per * per;
    constexpr int pieces = kChunk / per / kClipThreads;
    const int full = n / per;
    if (n == kChunk) {
      uint4 raw[pieces];
#pragma unroll
      for (int p = 0; p < pieces; ++p) raw[p] = ((const uint4*)g)[threadIdx.x + p * kClipThreads];
#pragma unroll
      for (int p = 0; p < pieces; ++p) {
        float v[per];
        Chunk<T, 16>::unpack(raw[p], v);
#pragma unroll
        for (int i = 0; i < per; ++i) v[i] *= f;
        __stcs((uint4*)out + threadIdx.x + p * kClipThreads, Chunk<T, 16>::pack(v));
      }
    } else {
      for (int p = threadIdx.x; p < full; p += kClipThreads) {
        float v[per];
        Chunk<T, 16>::unpack(((const uint4*)g)[p], v);
#pragma unroll
        for (int i = 0; i < per; ++i) v[i] *= f;
        ((uint4*)out)[p] = Chunk<T, 16>::pack(v);
      }
    }
  }
  for (int i = i0 + threadIdx.x; i < n; i += kClipThreads) out[i] = from_f32<T>(to_f32<T>(g[i]) * f);
}

__global__ void __launch_bounds__(kClipThreads) scale_kernel(const __grid_constant__ ClipList l, const double* part, int n_sums,
                                                             float max_norm, float* norm) {
  grid_wait();
  const float f = clip_factor(part, n_sums, max_norm, norm);
  for (int64_t c = l.first[l.count] - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
    const int t = tensor_of(l, c);
    if (f == 1.f && l.out[t] == l.g[t]) continue;  // in place and nothing to change
    const int64_t e0 = (c - l.first[t]) * kChunk;
    const int n = (int)imin64(kChunk, l.n[t] - e0);
    if (l.dtype[t] == CTR_F32) chunk_scale((const float*)l.g[t] + e0, (float*)l.out[t] + e0, n, f);
    else chunk_scale((const __nv_bfloat16*)l.g[t] + e0, (__nv_bfloat16*)l.out[t] + e0, n, f);
  }
}

// Tensors [i0, i1) as one launch's list; returns its number of chunks.
int64_t fill_list(ClipList* l, const void* const* grads, void* const* outs, const int32_t* dtypes,
                  const int64_t* counts, int i0, int i1) {
  int64_t chunks = 0;
  l->count = i1 - i0;
  for (int i = i0; i < i1; ++i) {
    const int j = i - i0;
    l->g[j] = grads[i];
    l->out[j] = outs ? outs[i] : nullptr;
    l->n[j] = counts[i];
    l->dtype[j] = (uint8_t)dtypes[i];
    l->first[j] = chunks;
    chunks += ceil_div(counts[i], kChunk);
  }
  l->first[l->count] = chunks;
  return chunks;
}

int clip_grid(int64_t chunks, int64_t most) {
  return (int)imax64(1, imin64(imin64(chunks, (int64_t)num_sms() * kClipBlocksPerSm), most));
}

}  // namespace
}  // namespace ctr

using namespace ctr;

extern "C" size_t ctr_clip_grads_workspace_size(void) {
  WsSizer z;
  z.take<double>(kMaxSums);
  return z.used;
}

extern "C" int ctr_clip_grads(const void* const* grads, void* const* outs, const int32_t* dtypes,
                              const int64_t* counts, int32_t n_tensors, float max_norm, float* norm, void* ws,
                              size_t ws_bytes, ctr_stream_t stream) {
  if (n_tensors < 0 || !norm || !(max_norm >= 0.f)) return CTR_ERR_INVALID_ARG;
  if (n_tensors > 0 && (!grads || !dtypes || !counts)) return CTR_ERR_INVALID_ARG;
  for (int i = 0; i < n_tensors; ++i) {
    if (!dtype_ok(dtypes[i]) || counts[i] < 0) return CTR_ERR_INVALID_ARG;
    if (counts[i] == 0) continue;
    const int eb = dtype_bytes(dtypes[i]);
    if (!grads[i] || ((uintptr_t)grads[i] % eb) != 0) return CTR_ERR_INVALID_ARG;
    if (outs && (!outs[i] || ((uintptr_t)outs[i] % eb) != 0)) return CTR_ERR_INVALID_ARG;
  }
  if (!ws_valid(ws, ws_bytes, ctr_clip_grads_workspace_size())) return CTR_ERR_WORKSPACE;
  // launches of up to kListMax tensors, with the workspace's sums shared out between them
  const int batches = std::max(1, (n_tensors + kListMax - 1) / kListMax);
  if (batches > kMaxSums) return CTR_ERR_UNSUPPORTED;
  const int64_t most = std::min(kMaxBlocks, kMaxSums / batches);
  WsCarver c(ws, ws_bytes);
  double* part = c.take<double>(kMaxSums);
  cudaStream_t s = (cudaStream_t)stream;
  ClipList l;
  int sums = 0;
  for (int b = 0; b < batches; ++b) {
    const int i0 = b * kListMax, i1 = std::min(n_tensors, i0 + kListMax);
    const int grid = clip_grid(fill_list(&l, grads, outs, dtypes, counts, i0, i1), most);
    launch_after(norm_kernel, dim3(grid), kClipThreads, 0, s, 1, l, part + sums);
    sums += grid;
  }
  bool told = false;
  for (int b = batches - 1; outs && b >= 0; --b) {
    const int i0 = b * kListMax, i1 = std::min(n_tensors, i0 + kListMax);
    if (batches > 1) fill_list(&l, grads, outs, dtypes, counts, i0, i1);
    const int64_t chunks = l.first[l.count];
    if (chunks == 0) continue;
    launch_after(scale_kernel, dim3(clip_grid(chunks, most)), kClipThreads, 0, s, 1, l, part, sums, max_norm,
                 told ? (float*)nullptr : norm);
    told = true;
  }
  if (!told) {
    launch_after(norm_only_kernel, dim3(1), kClipThreads, 0, s, 1, part, sums, norm);
  }
  return launch_status();
}
