// c2. Dense layers: z = x W^T + bias, y = act(z) + residual, and their gradients.
//
// Source: "Meta DLRM", section 02 (the dense stacks below and above the interaction), and "DHEN" notes, section
// 3.1 (linear modules, projected shortcuts); the formulas are stated in include/ctr.h.
//
// The products run on the tensor cores (dense_mm.cu), which want rows of bf16 on 16 bytes.  What is not that is laid
// out first, in the workspace: fp32 as three planes of bf16 that add up to it (each the rounding of what is left),
// bf16 rows off 16 bytes as a copy.  Bound by HBM.
//
// Backward: dz = dy act'(pre), rounded to bf16 (or split in planes) for both products, and dbias from it before that
// rounding, in one read of dy and pre: a thread holds its columns' sums over a strip of rows, the strips are added
// in their order by a second kernel.
//
// A few rows are not worth a tensor core's tile: a warp reads one to four rows of W, as they lie in memory, and multiplies
// them with all of x's, kept as fp32 in shared memory.  Bound by W's bytes (one row x 4096 -> 4096 bf16 9.7 us, 3.5 TB/s),
// and below some megabytes by latency.
#include <cuda_bf16.h>

#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "common.cuh"
#include "dense_mm.cuh"
#include "rows.cuh"
#include "tc.cuh"

namespace ctr {
namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------
// rows as the products want them
// ---------------------------------------------------------------------------
// x = p[0] + p[1] + p[2], each the rounding to bf16 of what is left.  A number that would round to an infinity is cut
// off instead; an infinity or a NaN is its first plane alone.
__device__ __forceinline__ void split3(float x, float (&p)[3]) {
  p[0] = __bfloat162float(__float2bfloat16_rn(x));
  if (!(fabsf(p[0]) < INFINITY)) {
    const bool finite = fabsf(x) < INFINITY;
    p[0] = finite ? __uint_as_float(__float_as_uint(x) & 0xffff0000u) : x;
    if (!finite) {
      p[1] = p[2] = 0.f;
      return;
    }
  }
  const float r = x - p[0];
  p[1] = __bfloat162float(__float2bfloat16_rn(r));
  p[2] = r - p[1];  // rounded to bf16 where it is stored
}

// N columns of a row into the planes `plane` elements apart.
template <int PLANES, int N>
__device__ __forceinline__ void store_planes(__nv_bfloat16* to, int64_t plane, const float (&v)[N]) {
  if constexpr (PLANES == 1) {
    *(typename RawOf<2 * N>::type*)to = Chunk<__nv_bfloat16, 2 * N>::pack(v);
  } else {
    float p[3][N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float one[3];
      split3(v[i], one);
#pragma unroll
      for (int q = 0; q < 3; ++q) p[q][i] = one[q];
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) *(typename RawOf<2 * N>::type*)(to + q * plane) = Chunk<__nv_bfloat16, 2 * N>::pack(p[q]);
  }
}

// Columns that a thread takes at once: 16 bytes of either type.
template <typename T>
constexpr int kPart = 16 / (int)sizeof(T);

// The kPart columns from c on as fp32; zeros past the end.
template <typename T, bool VEC>
__device__ __forceinline__ void load_part(const T* row, int c, int cols, float (&v)[kPart<T>]) {
  if constexpr (VEC) {
    if (c + kPart<T> <= cols) {
      Chunk<T, 16>::unpack(*(const uint4*)(row + c), v);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < kPart<T>; ++i) v[i] = c + i < cols ? to_f32<T>(row[c + i]) : 0.f;
}

template <typename T, int PLANES, bool VEC>
__global__ void __launch_bounds__(kThreads) pack_kernel(const T* x, int64_t rows, int cols, int64_t ldx, __nv_bfloat16* out,
                                                        int64_t ld, int64_t plane) {
  grid_wait();
  constexpr int N = kPart<T>;
  const int64_t parts = ld / N, total = rows * parts, step = (int64_t)gridDim.x * kThreads;
  for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < total; e += step) {
    const int64_t r = e / parts;
    const int c = (int)(e - r * parts) * N;
    float v[N];
    load_part<T, VEC>(x + r * ldx, c, cols, v);
    store_planes<PLANES>(out + r * ld + c, plane, v);
  }
}

// ---------------------------------------------------------------------------
// dz = dy act'(pre), and its column sums
// ---------------------------------------------------------------------------
struct DzArgs {
  const void* dy;
  const void* pre;          // NULL without an activation
  __nv_bfloat16* dz;        // NULL: not wanted
  float* part;              // [strips][n]; NULL: not wanted
  int64_t rows, ld_dy, ld_pre, ld, plane;
  int32_t n, strip, act;    // strip: rows of a block
};
constexpr int kDzCols = 256;  // columns of a block

// Blocks of an SM: six of aligned rows, whose loads are few and wide (65536 x 1024 bf16 with silu, sums alone: four blocks
// and two rows at once 79 us, six and one 65; eight, 66 and 18 us more with dz), four of others.
template <bool VEC>
constexpr int kDzBlocks = VEC ? 6 : 4;

template <typename T, int PLANES, bool VEC>
__global__ void __launch_bounds__(kThreads, kDzBlocks<VEC>) dz_kernel(const DzArgs a) {
  constexpr int N = kPart<T>, kAcross = kDzCols / N, kLanes = kThreads / kAcross;  // threads of a row, rows at a time
  __shared__ float sums[kLanes][kDzCols];
  const int part = threadIdx.x % kAcross, lane = threadIdx.x / kAcross;
  const int c = blockIdx.x * kDzCols + part * N;
  const int64_t r0 = (int64_t)blockIdx.y * a.strip, r1 = imin64(a.rows, r0 + a.strip);
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
  grid_wait();
  if (c < a.ld) {
#pragma unroll(VEC ? 1 : 2)
    for (int64_t r = r0 + lane; r < r1; r += kLanes) {
      float v[N], z[N];
      load_part<T, VEC>((const T*)a.dy + r * a.ld_dy, c, a.n, v);
      if (a.pre) {
        load_part<T, VEC>((const T*)a.pre + r * a.ld_pre, c, a.n, z);
        times_derivative<T>(a.act, v, z);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] += v[i];
      if (a.dz) store_planes<PLANES>(a.dz + r * a.ld + c, a.plane, v);
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int i = 0; i < N; ++i) sums[lane][part * N + i] = acc[i];
  __syncthreads();
  const int col = blockIdx.x * kDzCols + threadIdx.x;
  if (col >= a.n) return;
  float sum = 0.f;
#pragma unroll
  for (int l = 0; l < kLanes; ++l) sum += sums[l][threadIdx.x];
  a.part[(int64_t)blockIdx.y * a.n + col] = sum;
}
static_assert(kThreads == kDzCols, "a column to a thread in the end");

// dbias[c] = the sum of the strips' rows, 16 strands of them and then the strands, in their order.
constexpr int kJoinCols = 32, kJoinRows = 16;
template <typename T>
__global__ void __launch_bounds__(kJoinCols* kJoinRows) join_strips_kernel(const float* part, int strips, int n, T* out) {
  __shared__ float strand[kJoinRows][kJoinCols + 1];
  grid_wait();
  const int x = threadIdx.x % kJoinCols, y = threadIdx.x / kJoinCols;
  const int c = blockIdx.x * kJoinCols + x;
  float sum = 0.f;
  if (c < n) {
#pragma unroll 4
    for (int p = y; p < strips; p += kJoinRows) sum += part[(int64_t)p * n + c];
  }
  strand[y][x] = sum;
  __syncthreads();
  if (y == 0 && c < n) {
    for (int i = 1; i < kJoinRows; ++i) sum += strand[i][x];
    out[c] = from_f32<T>(sum);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) zero_rows_kernel(T* out, int64_t rows, int64_t cols, int64_t ld) {
  grid_wait();
  for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < rows * cols; e += (int64_t)gridDim.x * kThreads)
    out[e / cols * ld + e % cols] = from_f32<T>(0.f);
}

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------
constexpr int kFewRows = 8;      // at most
constexpr int kFewWords = 4096;  // of x in shared memory at a time

struct FewArgs {
  const void* x;
  const void* w;
  const void* bias;
  const void* residual;
  void* y;
  void* pre;
  int64_t ldx, ldw, ldr, ldy, ldp;
  int32_t rows, n, k, act;
};

// COLS rows of W to a warp: of more rows of x, what is read of it in shared memory serves more products (8 rows x 4096
// x 4096 bf16, one row of W to a warp, 65 us).
template <typename T, int VB, int ROWS, int COLS>
__global__ void __launch_bounds__(kThreads) dense_few_kernel(const FewArgs a) {
  using C = Chunk<T, VB>;
  constexpr int N = C::n, kChunk = kFewWords / ROWS;
  constexpr int kHeld = N == 1 ? 8 : 8 / COLS;  // parts of a row of W on their way at once
  constexpr int kStep = kHeld * 32 * N;
  __shared__ float x[ROWS][kChunk];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col0 = (blockIdx.x * (kThreads / 32) + warp) * COLS;
  // eight columns of a lane are two parts of four, 128 words apart, so that lanes read consecutive words
  auto place = [](int c) { return N == 8 ? (c & ~255) + ((c >> 2) & 1) * 128 + ((c >> 3) & 31) * 4 + (c & 3) : c; };
  float2 acc[ROWS][COLS];
#pragma unroll
  for (int t = 0; t < ROWS; ++t)
#pragma unroll
    for (int j = 0; j < COLS; ++j) acc[t][j] = make_float2(0.f, 0.f);
  grid_wait();
  for (int k0 = 0; k0 < a.k; k0 += kChunk) {
    const int len = min(kChunk, a.k - k0);
    typename C::Raw held[COLS][kHeld];
    auto fetch = [&](int c0) {
#pragma unroll
      for (int j = 0; j < COLS; ++j) {
        const T* row = (const T*)a.w + (int64_t)min(col0 + j, a.n - 1) * a.ldw + k0;
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
          const int c = c0 + (h * 32 + lane) * N;
          held[j][h] = typename C::Raw{};
          if (c < len) held[j][h] = *(const typename C::Raw*)(row + c);
        }
      }
    };
    fetch(0);  // W is on its way while x is laid out
    if (k0 > 0) __syncthreads();
    const int cover = (len + 255) & ~255;  // what the lanes may read
    for (int e = threadIdx.x; e < ROWS * cover; e += kThreads) {
      const int t = e / cover, c = e - t * cover;
      x[t][place(c)] = t < a.rows && c < len ? to_f32<T>(((const T*)a.x)[t * a.ldx + k0 + c]) : 0.f;
    }
    __syncthreads();
    for (int c0 = 0; c0 < len; c0 += kStep) {
      if (c0 > 0) fetch(c0);
#pragma unroll
      for (int h = 0; h < kHeld; ++h) {
        const int c = c0 + (h * 32 + lane) * N;
        if (c >= len) continue;
        float w[COLS][N];
#pragma unroll
        for (int j = 0; j < COLS; ++j) C::unpack(held[j][h], w[j]);
#pragma unroll
        for (int t = 0; t < ROWS; ++t) {
          if constexpr (N == 1) {
            const float v = x[t][c];
#pragma unroll
            for (int j = 0; j < COLS; ++j) acc[t][j].x = fmaf(v, w[j][0], acc[t][j].x);
          } else {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
              const float4 v = *(const float4*)&x[t][place(c + i)];
#pragma unroll
              for (int j = 0; j < COLS; ++j) {
                acc[t][j] = fma2(make_float2(v.x, v.y), make_float2(w[j][i], w[j][i + 1]), acc[t][j]);
                acc[t][j] = fma2(make_float2(v.z, v.w), make_float2(w[j][i + 2], w[j][i + 3]), acc[t][j]);
              }
            }
          }
        }
      }
    }
  }
  // lane t + ROWS j gets the sum of row t and column j
  float z = 0.f;
#pragma unroll
  for (int j = 0; j < COLS; ++j)
#pragma unroll
    for (int t = 0; t < ROWS; ++t) {
      float v = acc[t][j].x + acc[t][j].y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
      z = lane == t + ROWS * j ? v : z;
    }
  const int t = lane % ROWS, col = col0 + lane / ROWS;
  if (lane >= ROWS * COLS || t >= a.rows || col >= a.n) return;
  if (a.bias) z += to_f32<T>(((const T*)a.bias)[col]);
  if (a.pre) ((T*)a.pre)[t * a.ldp + col] = from_f32<T>(z);
  z = activation<T>(a.act, z);
  if (a.residual) z += to_f32<T>(((const T*)a.residual)[t * a.ldr + col]);
  ((T*)a.y)[t * a.ldy + col] = from_f32<T>(z);
}

// Rows of W to a warp of a call with `rows` rows.
int few_cols(int64_t rows) { return rows <= 1 ? 1 : rows <= 4 ? 2 : 4; }

template <typename T, int VB>
auto few_kernel(int64_t rows) {
  return rows <= 1 ? dense_few_kernel<T, VB, 1, 1> : rows <= 2 ? dense_few_kernel<T, VB, 2, 2>
       : rows <= 4 ? dense_few_kernel<T, VB, 4, 2> : dense_few_kernel<T, VB, 8, 4>;
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
int64_t up8(int64_t n) { return ceil_div(n, 8) * 8; }

// The distance between rows: of a single row whatever suits the products.
int64_t row_distance(int64_t rows, int64_t cols, int64_t ld) { return rows == 1 ? up8(cols) : ld; }

// Whether the products can read a matrix as it lies.
bool direct(const void* p, ctr_dtype dtype, int64_t rows, int64_t ld) {
  return dtype == CTR_BF16 && ((uintptr_t)p % 16) == 0 && ld % 8 == 0 && ld * 2 * imax64(rows, 1) < (1ll << 40);
}

size_t packed_elems(ctr_dtype dtype, int64_t rows, int64_t cols) {
  return (size_t)(dtype == CTR_F32 ? 3 : 1) * (size_t)rows * (size_t)up8(cols);
}

// Rows of a strip of dz_kernel: as many blocks as run at once on 152 SMs, at least kMinStrip rows each.
constexpr int kMinStrip = 32;
int64_t most_strips(int64_t n, bool vec) {
  return imax64(1, 152 * (vec ? kDzBlocks<true> : kDzBlocks<false>) / ceil_div(up8(n), kDzCols));
}
int strip_rows(int64_t rows, int64_t n, bool vec) { return (int)imax64(kMinStrip, ceil_div(rows, most_strips(n, vec))); }

// What a call takes from the workspace: no less than a call of fewer rows, so that one sized for the largest batch has room
// for every smaller one.
struct Room {
  __nv_bfloat16 *x = nullptr, *w = nullptr, *dz = nullptr;
  float *part = nullptr, *strips = nullptr;
};

template <typename Z, typename T>
T* take(Z& z, size_t count) {
  if constexpr (std::is_same_v<Z, WsSizer>) {
    z.template take<T>(count);
    return nullptr;
  } else {
    return z.template take<T>(count);
  }
}

struct Wants {
  bool x, w, dz, dw, strips;
};

template <typename Z>
Room carve(Z& z, ctr_dtype dtype, int64_t rows, int64_t n, int64_t k, const Wants& want) {
  Room r;
  if (want.x) r.x = take<Z, __nv_bfloat16>(z, packed_elems(dtype, rows, k));
  if (want.w) r.w = take<Z, __nv_bfloat16>(z, packed_elems(dtype, n, k));
  if (want.dz) r.dz = take<Z, __nv_bfloat16>(z, packed_elems(dtype, rows, n));
  if (want.dw) r.part = take<Z, float>(z, mm_room(n, k, rows) / 4);
  if (want.strips) r.strips = take<Z, float>(z, (size_t)imin64(ceil_div(imax64(rows, 1), kMinStrip), most_strips(n, true)) * n);
  return r;
}

bool fine(cudaError_t e) { return e == cudaSuccess; }

// A matrix as the products want it: as it lies, or laid out in `room`.
bool operand(MmOperand* o, const void* p, ctr_dtype dtype, int64_t rows, int64_t cols, int64_t ld, __nv_bfloat16* room,
             cudaStream_t s) {
  o->inner = cols;
  o->outer = rows;
  o->p = p;
  o->ld = ld;
  o->plane = 0;
  if (!room) return true;
  o->p = room;
  o->ld = up8(cols);
  o->plane = rows * o->ld;
  const dim3 grid((unsigned)imax64(1, imin64(ceil_div(rows * o->ld * dtype_bytes(dtype) / 16, kThreads), (int64_t)num_sms() * 16)));
  const int eb = dtype_bytes(dtype);
  const bool vec = ((uintptr_t)p % 16) == 0 && (ld * eb) % 16 == 0;
  if (dtype == CTR_F32) {
    auto k = vec ? pack_kernel<float, 3, true> : pack_kernel<float, 3, false>;
    return fine(launch_after(k, grid, kThreads, 0, s, 1, (const float*)p, rows, (int)cols, ld, room, o->ld, o->plane));
  }
  auto k = vec ? pack_kernel<__nv_bfloat16, 1, true> : pack_kernel<__nv_bfloat16, 1, false>;
  return fine(launch_after(k, grid, kThreads, 0, s, 1, (const __nv_bfloat16*)p, rows, (int)cols, ld, room, o->ld, o->plane));
}

// Whether a forward call goes to the kernel for few rows.  bf16 matrices that the tensor cores can read as they lie: one or
// two rows (4 rows of 1024 -> 2048 7.8 us against 7.6, of 4096 -> 4096 26 against 19).  Others would have W laid out first:
// up to eight (fp32 1024 -> 2048 14 us against 19, 4096 -> 4096 51 against 76; bf16 479 -> 512 6.0 against 8.0).
bool few_rows(int64_t rows, bool as_they_lie) { return rows <= (as_they_lie ? 2 : kFewRows); }

bool off(const void* p, int by) { return ((uintptr_t)p % by) != 0; }

int check_dense(ctr_dtype dtype, int64_t rows, int64_t n, int64_t k, int act) {
  if (!dtype_ok(dtype) || rows < 0 || n < 1 || k < 1 || act < CTR_ACT_NONE || act > CTR_ACT_SIGMOID)
    return CTR_ERR_INVALID_ARG;
  if (rows > INT32_MAX - 65536 || n > INT32_MAX / 4 || k > INT32_MAX / 4) return CTR_ERR_UNSUPPORTED;
  return CTR_OK;
}

}  // namespace
}  // namespace ctr

using namespace ctr;

extern "C" size_t ctr_dense_workspace_size(int64_t rows, int64_t n, int64_t k, ctr_dtype dtype, int train, int packed) {
  if (check_dense(dtype, rows, n, k, CTR_ACT_NONE) != CTR_OK) return 0;
  const bool pack = packed != 0 || dtype == CTR_F32;
  WsSizer z;
  carve(z, dtype, rows, n, k, Wants{pack, pack, train != 0, train != 0, train != 0});
  return z.used;
}

extern "C" int ctr_dense(const void* x, ctr_dtype dtype, int64_t rows, int64_t k, int64_t ldx, const void* w, int64_t n,
                         int64_t ldw, const void* bias, int act, const void* residual, int64_t ld_residual, void* y,
                         int64_t ld_y, void* pre, int64_t ld_pre, void* ws, size_t ws_bytes, ctr_stream_t stream) {
  const int st = check_dense(dtype, rows, n, k, act);
  if (st != CTR_OK) return st;
  if (ldx < k || ldw < k || (residual && ld_residual < n) || ld_y < n || (pre && ld_pre < n)) return CTR_ERR_INVALID_ARG;
  if (!w || (rows > 0 && (!x || !y))) return CTR_ERR_INVALID_ARG;
  const int eb = dtype_bytes(dtype);
  for (const void* p : {x, w, bias, residual, (const void*)y, (const void*)pre})
    if (off(p, eb)) return CTR_ERR_INVALID_ARG;
  if (!ws_valid(ws, ws_bytes, kWsHeader)) return CTR_ERR_WORKSPACE;
  if (rows == 0) return CTR_OK;
  ldx = row_distance(rows, k, ldx);
  ldw = row_distance(n, k, ldw);
  cudaStream_t s = (cudaStream_t)stream;
  if (few_rows(rows, direct(x, dtype, rows, ldx) && direct(w, dtype, n, ldw))) {
    FewArgs a = {x, w, bias, residual, y, pre, ldx, ldw, ld_residual, ld_y, ld_pre, (int32_t)rows, (int32_t)n, (int32_t)k, act};
    const bool vec = !off(w, 16) && (ldw * eb) % 16 == 0 && (k * eb) % 16 == 0;
    auto kernel = dtype == CTR_F32 ? (vec ? few_kernel<float, 16>(rows) : few_kernel<float, 4>(rows))
                                   : (vec ? few_kernel<__nv_bfloat16, 16>(rows) : few_kernel<__nv_bfloat16, 2>(rows));
    return fine(launch_after(kernel, dim3((unsigned)ceil_div(n, kThreads / 32 * few_cols(rows))), kThreads, 0, s, 1, a))
               ? launch_status()
               : CTR_ERR_CUDA;
  }
  WsCarver c(ws, ws_bytes);
  const Room room = carve(c, dtype, rows, n, k, Wants{!direct(x, dtype, rows, ldx), !direct(w, dtype, n, ldw), false, false, false});
  if (!c.ok()) return CTR_ERR_WORKSPACE;
  MmCall m = {};
  m.major = 0;
  m.planes = dtype == CTR_F32 ? 3 : 1;
  m.m = rows;
  m.n = n;
  m.r = k;
  if (!operand(&m.a, x, dtype, rows, k, ldx, room.x, s) || !operand(&m.b, w, dtype, n, k, ldw, room.w, s)) return CTR_ERR_CUDA;
  m.bias = bias;
  m.act = act;
  m.residual = residual;
  m.ld_res = ld_residual;
  m.pre = pre;
  m.ld_pre = ld_pre;
  m.out = y;
  m.ldo = ld_y;
  m.out_f32 = dtype == CTR_F32;
  m.err = (int*)ws;
  return mm_run(m, nullptr, s);
}

extern "C" int ctr_dense_bwd(const void* dy, ctr_dtype dtype, int64_t rows, int64_t n, int64_t ld_dy, const void* x,
                             int64_t k, int64_t ldx, const void* w, int64_t ldw, const void* pre, int64_t ld_pre, int act,
                             void* dx, int64_t ld_dx, ctr_dtype grad_dtype, void* dw, int64_t ld_dw, void* dbias, void* ws,
                             size_t ws_bytes, ctr_stream_t stream) {
  const int st = check_dense(dtype, rows, n, k, act);
  if (st != CTR_OK) return st;
  if (grad_dtype != CTR_F32 && grad_dtype != dtype) return CTR_ERR_INVALID_ARG;
  if (ld_dy < n || (dw && ldx < k) || (dx && ldw < k) || (act != CTR_ACT_NONE && ld_pre < n) || (dx && ld_dx < k) ||
      (dw && ld_dw < k))
    return CTR_ERR_INVALID_ARG;
  if (rows > 0 && (!dy || (act != CTR_ACT_NONE && !pre) || (dw && !x) || (dx && !w))) return CTR_ERR_INVALID_ARG;
  const int eb = dtype_bytes(dtype), gb = dtype_bytes(grad_dtype);
  for (const void* p : {dy, x, w, pre, (const void*)dx})
    if (off(p, eb)) return CTR_ERR_INVALID_ARG;
  if (off(dw, gb) || off(dbias, gb)) return CTR_ERR_INVALID_ARG;
  if (!ws_valid(ws, ws_bytes, kWsHeader)) return CTR_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  if (rows == 0) {  // sums of nothing
    const dim3 grid((unsigned)imin64(ceil_div(n * k, kThreads), (int64_t)num_sms() * 16)), few((unsigned)ceil_div(n, kThreads));
    bool ok = true;
    if (grad_dtype == CTR_F32) {
      if (dw) ok = fine(launch_after(zero_rows_kernel<float>, grid, kThreads, 0, s, 1, (float*)dw, n, k, ld_dw));
      if (ok && dbias) ok = fine(launch_after(zero_rows_kernel<float>, few, kThreads, 0, s, 1, (float*)dbias, (int64_t)1, n, n));
    } else {
      if (dw) ok = fine(launch_after(zero_rows_kernel<__nv_bfloat16>, grid, kThreads, 0, s, 1, (__nv_bfloat16*)dw, n, k, ld_dw));
      if (ok && dbias)
        ok = fine(launch_after(zero_rows_kernel<__nv_bfloat16>, few, kThreads, 0, s, 1, (__nv_bfloat16*)dbias, (int64_t)1, n, n));
    }
    return ok ? launch_status() : CTR_ERR_CUDA;
  }
  ld_dy = row_distance(rows, n, ld_dy);
  ld_pre = row_distance(rows, n, ld_pre);
  ldx = row_distance(rows, k, ldx);
  ldw = row_distance(n, k, ldw);
  // without an activation dz is dy, which the products may be able to read as it lies
  const bool make_dz = (dx || dw) && (act != CTR_ACT_NONE || !direct(dy, dtype, rows, ld_dy));
  const Wants want = {dw && !direct(x, dtype, rows, ldx), dx && !direct(w, dtype, n, ldw), make_dz, dw != nullptr,
                      dbias != nullptr};
  WsCarver c(ws, ws_bytes);
  const Room room = carve(c, dtype, rows, n, k, want);
  if (!c.ok()) return CTR_ERR_WORKSPACE;
  MmOperand dz = {dy, n, rows, ld_dy, 0};
  if (make_dz || dbias) {
    DzArgs a = {};
    a.dy = dy;
    a.pre = act != CTR_ACT_NONE ? pre : nullptr;
    a.dz = make_dz ? room.dz : nullptr;
    a.part = room.strips;
    a.rows = rows;
    a.ld_dy = ld_dy;
    a.ld_pre = ld_pre;
    a.ld = up8(n);
    a.plane = rows * a.ld;
    a.n = (int32_t)n;
    a.act = act;
    if (make_dz) dz = MmOperand{room.dz, n, rows, a.ld, a.plane};
    const bool vec = !off(dy, 16) && (ld_dy * eb) % 16 == 0 && (!a.pre || (!off(pre, 16) && (ld_pre * eb) % 16 == 0));
    a.strip = strip_rows(rows, n, vec);
    const int strips = (int)ceil_div(rows, a.strip);
    const dim3 grid((unsigned)ceil_div(a.ld, kDzCols), (unsigned)strips);
    auto kernel = dtype == CTR_F32 ? (vec ? dz_kernel<float, 3, true> : dz_kernel<float, 3, false>)
                                   : (vec ? dz_kernel<__nv_bfloat16, 1, true> : dz_kernel<__nv_bfloat16, 1, false>);
    if (!fine(launch_after(kernel, grid, kThreads, 0, s, 1, a))) return CTR_ERR_CUDA;
    if (dbias) {
      const dim3 jg((unsigned)ceil_div(n, kJoinCols));
      const bool ok = grad_dtype == CTR_F32
                          ? fine(launch_after(join_strips_kernel<float>, jg, kJoinCols * kJoinRows, 0, s, 1,
                                              (const float*)room.strips, strips, (int)n, (float*)dbias))
                          : fine(launch_after(join_strips_kernel<__nv_bfloat16>, jg, kJoinCols * kJoinRows, 0, s, 1,
                                              (const float*)room.strips, strips, (int)n, (__nv_bfloat16*)dbias));
      if (!ok) return CTR_ERR_CUDA;
    }
  }
  MmCall m = {};
  m.planes = dtype == CTR_F32 ? 3 : 1;
  m.a = dz;
  m.err = (int*)ws;
  if (dx) {
    m.major = 1;
    m.m = rows;
    m.n = k;
    m.r = n;
    if (!operand(&m.b, w, dtype, n, k, ldw, room.w, s)) return CTR_ERR_CUDA;
    m.out = dx;
    m.ldo = ld_dx;
    m.out_f32 = dtype == CTR_F32;
    const int e = mm_run(m, nullptr, s);
    if (e != CTR_OK) return e;
  }
  if (dw) {
    m.major = 2;
    m.m = n;
    m.n = k;
    m.r = rows;
    if (!operand(&m.b, x, dtype, rows, k, ldx, room.x, s)) return CTR_ERR_CUDA;
    m.out = dw;
    m.ldo = ld_dw;
    m.out_f32 = grad_dtype == CTR_F32;
    const int e = mm_run(m, room.part, s);
    if (e != CTR_OK) return e;
  }
  return launch_status();
}
