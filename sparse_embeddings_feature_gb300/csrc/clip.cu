// b4. Global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum g^2),  out = g * (norm > max_norm ? max_norm / norm : 1)
//
// The tensors are cut into chunks of kChunk elements, handed to the blocks in a
// fixed order.  A thread squares and adds 16-byte pieces in fp32 (four
// accumulators), moves them into fp64 every few chunks, and joins are fp64 in a
// fixed order, so the result does not change from run to run.  A piece whose
// largest magnitude would leave fp32's range when squared (or lose its square
// below it) is squared in fp64 instead; for gradients of ordinary size that
// branch is never taken.  The last block to finish adds the blocks' sums up.
// Two passes over the data, bound by HBM: the second walks the chunks in
// reverse, so what the first read last is still in L2.
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
constexpr int kMaxBlocks = 2048;    // bound of the grid, for the workspace
constexpr int kFlush = 8;           // chunks between moves of the fp32 sums into fp64
constexpr float kBig = 0x1p50f;     // squares of larger values (2^100) could overflow in a sum
constexpr float kSmall = 0x1p-55f;  // squares of smaller ones (2^-110) lose accuracy near fp32's floor

struct ClipList {
  const void* g[kListMax];
  void* out[kListMax];
  int64_t n[kListMax];
  int64_t first[kListMax + 1];  // chunks before each tensor
  uint8_t dtype[kListMax];
  int32_t count;
};

// Workspace after the header.  `sum` runs over the launches of one call.
struct ClipState {
  double sum;
  float factor;
  uint32_t done;
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

template <int N>
__device__ __forceinline__ void add_squares(const float (&f)[N], float (&acc)[4], double& wide) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(f[i]));
  if (m > kBig || (m < kSmall && m > 0.f)) {
#pragma unroll
    for (int i = 0; i < N; ++i) wide += (double)f[i] * (double)f[i];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i & 3] = fmaf(f[i], f[i], acc[i & 3]);
  }
}

template <typename T>
__device__ __forceinline__ void chunk_squares(const T* g, int n, float (&acc)[4], double& wide) {
  constexpr int per = 16 / (int)sizeof(T);
  int i0 = 0;
  if (((uintptr_t)g & 15) == 0) {
    i0 = n / per * per;
    constexpr int pieces = kChunk / per / kClipThreads;
    const int full = n / per;
    if (n == kChunk) {
      uint4 raw[pieces];
#pragma unroll
      for (int p = 0; p < pieces; ++p) raw[p] = ((const uint4*)g)[threadIdx.x + p * kClipThreads];
#pragma unroll
      for (int p = 0; p < pieces; ++p) {
        float f[per];
        Chunk<T, 16>::unpack(raw[p], f);
        add_squares(f, acc, wide);
      }
    } else {
      for (int p = threadIdx.x; p < full; p += kClipThreads) {
        float f[per];
        Chunk<T, 16>::unpack(((const uint4*)g)[p], f);
        add_squares(f, acc, wide);
      }
    }
  }
  for (int i = i0 + threadIdx.x; i < n; i += kClipThreads) {
    const float f[1] = {to_f32<T>(g[i])};
    add_squares(f, acc, wide);
  }
}

__global__ void __launch_bounds__(kClipThreads) norm_kernel(const __grid_constant__ ClipList l, ClipState* st,
                                                            double* part, float* norm, float max_norm, int first,
                                                            int last) {
  __shared__ double warp_sum[kClipThreads / 32];
  __shared__ bool am_last;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  double wide = 0.0;
  int since = 0;
  for (int64_t c = blockIdx.x; c < l.first[l.count]; c += gridDim.x) {
    const int t = tensor_of(l, c);
    const int64_t e0 = (c - l.first[t]) * kChunk;
    const int n = (int)imin64(kChunk, l.n[t] - e0);
    if (l.dtype[t] == CTR_F32) chunk_squares((const float*)l.g[t] + e0, n, acc, wide);
    else chunk_squares((const __nv_bfloat16*)l.g[t] + e0, n, acc, wide);
    if (++since == kFlush) {
      wide += (double)((acc[0] + acc[1]) + (acc[2] + acc[3]));
      acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
      since = 0;
    }
  }
  wide += (double)((acc[0] + acc[1]) + (acc[2] + acc[3]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) wide += __shfl_down_sync(kFull, wide, o);
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = wide;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < kClipThreads / 32; ++w) s += warp_sum[w];
    part[blockIdx.x] = s;
    __threadfence();
    am_last = atomicAdd(&st->done, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!am_last) return;
  __threadfence();
  double s = 0.0;
  for (int b = threadIdx.x; b < (int)gridDim.x; b += kClipThreads) s += __ldcg(part + b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_down_sync(kFull, s, o);
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double all = first ? 0.0 : st->sum;
    for (int w = 0; w < kClipThreads / 32; ++w) all += warp_sum[w];
    st->sum = all;
    st->done = 0;
    if (last) {
      const float v = (float)sqrt(all);
      *norm = v;
      st->factor = v > max_norm && v < INFINITY ? max_norm / v : 1.f;  // NaN and inf leave the gradients as they are
    }
  }
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

__global__ void __launch_bounds__(kClipThreads) scale_kernel(const __grid_constant__ ClipList l, const ClipState* st) {
  const float f = st->factor;
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

int clip_grid(int64_t chunks) {
  return (int)imax64(1, imin64(imin64(chunks, (int64_t)num_sms() * kClipBlocksPerSm), kMaxBlocks));
}

}  // namespace
}  // namespace ctr

using namespace ctr;

extern "C" size_t ctr_clip_grads_workspace_size(void) {
  WsSizer z;
  z.take<ClipState>(1);
  z.take<double>(kMaxBlocks);
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
  WsCarver c(ws, ws_bytes);
  ClipState* st = c.take<ClipState>(1);
  double* part = c.take<double>(kMaxBlocks);
  cudaStream_t s = (cudaStream_t)stream;
  ClipList l;
  const int batches = std::max(1, (n_tensors + kListMax - 1) / kListMax);
  for (int b = 0; b < batches; ++b) {
    const int i0 = b * kListMax, i1 = std::min(n_tensors, i0 + kListMax);
    const int64_t chunks = fill_list(&l, grads, outs, dtypes, counts, i0, i1);
    norm_kernel<<<clip_grid(chunks), kClipThreads, 0, s>>>(l, st, part, norm, max_norm, b == 0, b == batches - 1);
    count_launch();
  }
  if (outs) {
    for (int b = batches - 1; b >= 0; --b) {
      const int i0 = b * kListMax, i1 = std::min(n_tensors, i0 + kListMax);
      const int64_t chunks = fill_list(&l, grads, outs, dtypes, counts, i0, i1);
      if (chunks == 0) continue;
      scale_kernel<<<clip_grid(chunks), kClipThreads, 0, s>>>(l, st);
      count_launch();
    }
  }
  return launch_status();
}
