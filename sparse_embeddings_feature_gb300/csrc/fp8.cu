// b3. e4m3 codes with a scale per block of 128: rows, rows + columns, blocks.
//
// With m = max(largest |x| of the block, 2^-100):  scale = m / 448,  code =
// e4m3(x * (448 / m)), all in fp32 (two correctly rounded divisions a block, one
// multiplication and one conversion a value).  The floor of 2^-100 keeps 448 / m
// finite: values below it are zero for the product's purposes.
//
// Rows: 16 lanes hold a block of 128 values, 8 each (one or two 16-byte loads),
// the maximum is four xor-shuffles, and the 128 codes leave as one 128-byte
// store of 8 bytes a lane.  A lane group takes two to four blocks of one row at
// once, has the next row's loads in flight while it converts, and divides once
// for all of them.  65536 x 1024 bf16 39 us in a row of calls (201 MB at 5.1 TB/s);
// bound by latency and occupancy (0.55 of the cycles issue, 31% of the warps are
// active).
//
// Tiles (rows + columns, blocks): a CTA reads a 128 x 128 tile once, keeps it in
// shared memory in its own type, and writes both orders of codes from it, each
// as 128 consecutive bytes: a second pass over x would cost as much as the
// first.  For the column order a thread holds 32 rows of two neighbouring columns
// in registers (one shared-memory read of both columns' values per row) for the
// maximum and for the codes, which leave in 16-byte stores.  Bound by latency and
// issue (0.67 of the cycles issue, 58% of the warps are active; 65536 x 1024 bf16,
// both orders, 53 us in a row of calls: 268 MB at 5.0 TB/s).
#include <cuda_bf16.h>

#include <algorithm>
#include <initializer_list>

#include "codes.cuh"
#include "common.cuh"
#include "rows.cuh"

namespace ctr {
namespace {

constexpr int kQThreads = 256;

// Columns c0 .. c0 + 7 of a row of `cols` elements as fp32; zeros past the end.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int64_t c0, int64_t cols, bool vec, float (&v)[8]) {
  constexpr int per = 16 / (int)sizeof(T);
  if (vec && c0 + 8 <= cols) {
#pragma unroll
    for (int i = 0; i < 8; i += per) {
      float f[per];
      Chunk<T, 16>::unpack(*(const uint4*)(row + c0 + i), f);
#pragma unroll
      for (int q = 0; q < per; ++q) v[i + q] = f[q];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c0 + i < cols ? to_f32<T>(row[c0 + i]) : 0.f;
  }
}

// Row of x for row r of the codes: row_index[r], or r; -1 for a zero row.
__device__ __forceinline__ int64_t source_row(const int32_t* row_index, int64_t r, int64_t x_rows, int* err) {
  if (!row_index) return r;
  const int64_t i = row_index[r];
  if (i >= x_rows) {
    set_error(err, CTR_ERR_INDEX_OUT_OF_RANGE);
    return -1;
  }
  return i;
}

// Largest magnitudes, NaN winning, two values at a time: bf16 pairs stay packed.
template <typename T>
struct MaxPair;
template <>
struct MaxPair<float> {
  float x = 0.f, y = 0.f;
  __device__ __forceinline__ void add(const float* p) {
    const float2 v = *(const float2*)p;
    x = max_mag(x, v.x);
    y = max_mag(y, v.y);
  }
  __device__ __forceinline__ float2 get() const { return make_float2(x, y); }
};
template <>
struct MaxPair<__nv_bfloat16> {
  uint32_t m = 0;  // magnitudes as unsigned 16-bit numbers: their order is the values', NaN above all
  __device__ __forceinline__ void add(const __nv_bfloat16* p) { m = __vmaxu2(m, *(const uint32_t*)p & 0x7fff7fffu); }
  __device__ __forceinline__ float2 get() const {
    return make_float2(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
};

// Blocks of one row that a lane group takes at once: 64 bytes of loads a lane.
template <typename T>
constexpr int row_blocks() {
  return 8 / (int)sizeof(T);
}

template <typename T>
struct RowPart {
  static constexpr int kBlocks = row_blocks<T>();
  uint4 raw[kBlocks][sizeof(T) / 2];  // 8 values of each block
};

// The lane's 8 values of blocks kb0, kb0 + 1, .. of row src (-1: zeros); zeros past the row's end.
template <typename T>
__device__ __forceinline__ void load_part(RowPart<T>& p, const T* x, int64_t ldx, int64_t src, int kb0, int lane16,
                                          int64_t cols, bool vec) {
  constexpr int per = 16 / (int)sizeof(T);
#pragma unroll
  for (int b = 0; b < RowPart<T>::kBlocks; ++b) {
    const int64_t c = (int64_t)(kb0 + b) * 128 + lane16 * 8;
    const T* row = x + src * ldx + c;
#pragma unroll
    for (int h = 0; h < 8 / per; ++h) {
      if (vec && src >= 0 && c + (h + 1) * per <= cols) {
        p.raw[b][h] = *(const uint4*)(row + h * per);
      } else {
        float f[per];
#pragma unroll
        for (int i = 0; i < per; ++i) f[i] = src >= 0 && c + h * per + i < cols ? to_f32<T>(row[h * per + i]) : 0.f;
        p.raw[b][h] = Chunk<T, 16>::pack(f);
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kQThreads) quantize_rows_kernel(const T* x, int64_t x_rows, int64_t rows,
                                                                  int64_t cols, int64_t ldx, int vec,
                                                                  const int32_t* row_index, uint8_t* q, float* scale,
                                                                  int64_t ld_scale, int blocks, int* err) {
  constexpr int kBlocks = row_blocks<T>(), per = 16 / (int)sizeof(T);
  const int lane16 = threadIdx.x & 15;
  const int kb0 = blockIdx.y * kBlocks;
  const int64_t step = (int64_t)gridDim.x * (kQThreads / 16);
  const int64_t trips = ceil_div(rows, step);  // the same in every lane: the shuffles need all of them
  int64_t r = (int64_t)blockIdx.x * (kQThreads / 16) + (threadIdx.x >> 4);
  RowPart<T> cur, next;
  grid_wait();
  load_part(cur, x, ldx, r < rows ? source_row(row_index, r, x_rows, err) : -1, kb0, lane16, cols, vec != 0);
  for (int64_t trip = 0; trip < trips; ++trip, r += step) {
    // the next row's loads fly while this one is converted
    if (trip + 1 < trips)
      load_part(next, x, ldx, r + step < rows ? source_row(row_index, r + step, x_rows, err) : -1, kb0, lane16, cols,
                vec != 0);
    // a block's two divisions are one lane's: lane b of the group has block b's
    float mine = 0.f;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      MaxPair<T> mp;
#pragma unroll
      for (int h = 0; h < 8 / per; ++h)
#pragma unroll
        for (int e = 0; e < per; e += 2) mp.add((const T*)&cur.raw[b][h] + e);
      const float2 m2 = mp.get();
      float m = max_mag(m2.x, m2.y);
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) m = max_mag(m, __shfl_xor_sync(kFull, m, o));
      if (lane16 == b) mine = m;
    }
    const float amax = at_least_floor(mine);
    const float inv_mine = __fdiv_rn(kTop, amax);
    const float s = __fdiv_rn(amax, kTop);
    if (r < rows && lane16 < kBlocks && kb0 + lane16 < blocks) scale[(kb0 + lane16) * ld_scale + r] = s;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      const float inv = __shfl_sync(kFull, inv_mine, b, 16);
      float v[8];
#pragma unroll
      for (int h = 0; h < 8 / per; ++h) {
        float f[per];
        Chunk<T, 16>::unpack(cur.raw[b][h], f);
#pragma unroll
        for (int i = 0; i < per; ++i) v[h * per + i] = f[i];
      }
      if (r < rows && kb0 + b < blocks)
        *(uint2*)(q + (r * blocks + kb0 + b) * 128 + lane16 * 8) = make_uint2(codes4(v, inv), codes4(v + 4, inv));
    }
    cur = next;
  }
}

struct TileArgs {
  const void* x;
  int64_t x_rows, rows, cols, ldx;
  const int32_t* row_index;
  const int32_t* offsets;  // NULL: `groups` groups of `rows` rows each
  int32_t groups, unit, col_blocks;  // unit: bytes that every row can be read in
  uint8_t* q;
  float* scale;
  int64_t ldq, ld_scale;  // scale: [col block][row], or with blocks [group][row block][col block]
  uint8_t* qt;
  float* scale_t;
  int64_t ldt, ld_scale_t;  // qt: [col][ldt]; scale_t: [tile][cols] by column, [col block][tile] by block
  int* err;
};

// Values of two neighbouring columns of a tile row.
__device__ __forceinline__ float2 two(const float* p) { return *(const float2*)p; }
__device__ __forceinline__ float2 two(const __nv_bfloat16* p) {
  const uint32_t w = *(const uint32_t*)p;
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// A tile row is 128 elements and 16 bytes more: 16-byte accesses stay aligned and a row's do not
// meet the next one's banks.
template <typename T>
constexpr int tile_ld() {
  return 128 + 16 / (int)sizeof(T);
}

// Threads of a tile's CTA: fp32 tiles are twice as large, so only three CTAs fit an SM, and get twice
// the threads to keep as many warps (65536 x 479 fp32, both orders: 59 us, with 256 threads 64).
template <typename T>
constexpr int tile_threads() {
  return sizeof(T) == 4 ? 512 : 256;
}

// B bytes into shared memory without waiting, of which the first `take` come from src and the rest
// are zeros.
template <int B>
__device__ __forceinline__ void copy_async(void* dst, const void* src, int take) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  if constexpr (B == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(take) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(d), "l"(src), "r"(take), "n"(B) : "memory");
}

// A 128 x 128 tile from the rows source(i) of x (-1: zeros), by asynchronous copies of B bytes: nothing
// waits in registers, so that all of a CTA's reads are in flight.
template <typename T, int B, typename Source>
__device__ __forceinline__ void stage_tile(T* tile, const T* x, int64_t ldx, int col0, int ncols, Source source) {
  constexpr int per = B / (int)sizeof(T), parts = 128 / per;
  constexpr int kLanes = parts < 32 ? parts : 32, kTurns = parts / kLanes, kStep = tile_threads<T>() / kLanes;
  const int c0 = ((int)threadIdx.x % kLanes) * per;
  constexpr int kRows = kTurns == 1 ? 4 : 1;  // rows whose places are looked up together
#pragma unroll 1
  for (int i0 = (int)threadIdx.x / kLanes; i0 < 128; i0 += kRows * kStep) {
    int64_t src[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) src[u] = source(i0 + u * kStep);
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const T* row = x + (src[u] >= 0 ? src[u] * ldx + col0 : 0);
      const int have = src[u] >= 0 ? ncols : 0;
#pragma unroll
      for (int h = 0; h < kTurns; ++h) {
        const int c = c0 + h * kLanes * per;
        int take = c < have ? B : 0;
        if constexpr (per > 1) take = min(take, max(0, (have - c) * (int)sizeof(T)));
        copy_async<B>(tile + (i0 + u * kStep) * tile_ld<T>() + c, take ? row + c : x, take);
      }
    }
  }
}

// The same where rows start at odd elements, which no asynchronous copy can take: four rows' elements
// in registers at once (a row at a time, the reads' latency was the kernel's: 23 x 1407 x 973, both
// orders, 51 us against 41).
template <typename T, typename Source>
__device__ __forceinline__ void stage_elements(T* tile, const T* x, int64_t ldx, int col0, int ncols, Source source) {
  constexpr int kWarps = tile_threads<T>() / 32, kRows = 4;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int i0 = threadIdx.x >> 5; i0 < 128; i0 += kWarps * kRows) {
    int64_t src[kRows];
    T v[kRows][4];
#pragma unroll
    for (int u = 0; u < kRows; ++u) src[u] = source(i0 + u * kWarps);
#pragma unroll
    for (int u = 0; u < kRows; ++u)
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int c = h * 32 + lane;
        v[u][h] = src[u] >= 0 && c < ncols ? x[src[u] * ldx + col0 + c] : from_f32<T>(0.f);
      }
#pragma unroll
    for (int u = 0; u < kRows; ++u)
#pragma unroll
      for (int h = 0; h < 4; ++h) tile[(i0 + u * kWarps) * tile_ld<T>() + h * 32 + lane] = v[u][h];
  }
}

// One 128 x 128 tile.  ROW_BLOCK: the row codes have one scale for the tile (else one a row);
// COL_BLOCK: the column codes have (else one a column).
template <typename T, bool ROW_BLOCK, bool COL_BLOCK>
__global__ void __launch_bounds__(tile_threads<T>(), sizeof(T) == 2 ? 5 : 3) quantize_tile_kernel(const TileArgs a) {
  constexpr int kLd = tile_ld<T>(), kThreads = tile_threads<T>();
  constexpr int kPartRows = 64 * 128 / kThreads, kParts = 128 / kPartRows;  // rows of two columns that a thread takes
  extern __shared__ __align__(16) uint8_t smem[];
  T* tile = (T*)smem;
  __shared__ float col_max[kParts][128];  // then [0]: the columns' multipliers
  __shared__ float row_max[128];     // then the rows' multipliers
  __shared__ float warp_max[kThreads / 32];
  __shared__ int where[4];  // group, first row, rows, tile number (of all groups)
  const int col0 = blockIdx.y * 128;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_wait();
  if (a.offsets) {
    // the groups' tiles come one after another: find this block's (one warp, 32 groups at a time)
    if (warp == 0) {
      if (lane == 0) where[2] = 0;
      __syncwarp();
      int seen = 0;
      bool ok = a.offsets[0] == 0;
      for (int g0 = 0; g0 < a.groups; g0 += 32) {
        const int g = g0 + lane;
        int lo = 0, hi = 0;
        if (g < a.groups) {
          lo = a.offsets[g];
          hi = a.offsets[g + 1];
          ok = ok && lo >= 0 && hi >= lo && hi <= a.rows;
        }
        const int mine = ok ? (hi - lo + 127) / 128 : 0;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(kFull, incl, o);
          if (lane >= o) incl += y;
        }
        const int t = (int)blockIdx.x - (seen + incl - mine);
        if (t >= 0 && t < mine) {
          where[0] = g;
          where[1] = lo + t * 128;
          where[2] = min(128, hi - lo - t * 128);
          where[3] = blockIdx.x;
        }
        seen += __shfl_sync(kFull, incl, 31);
      }
      const bool good = __all_sync(kFull, ok);
      __syncwarp();
      if (!good) {
        if (lane == 0) {
          set_error(a.err, CTR_ERR_BAD_OFFSETS);
          where[2] = 0;
        }
      }
    }
  } else if (threadIdx.x == 0) {
    const int per = (int)((a.rows + 127) / 128);
    const int g = blockIdx.x / per, t = blockIdx.x - g * per;
    where[0] = g;
    where[1] = t * 128;
    where[2] = (int)imin64(128, a.rows - t * 128);
    where[3] = t;
  }
  __syncthreads();
  const int g = where[0], row0 = where[1], n = where[2], tnum = where[3];
  if (n <= 0) return;
  const int64_t xbase = a.offsets ? 0 : (int64_t)g * a.rows;  // rows of earlier groups

  // The tile into shared memory; rows past n and columns past the end are zeros.
  const int lane16 = threadIdx.x & 15;
  const int ncols = (int)imin64(128, a.cols - col0);
  auto source = [&](int i) -> int64_t {
    if (i >= n) return -1;
    const int64_t r = source_row(a.row_index, row0 + i, a.x_rows, a.err);
    return r >= 0 ? xbase + r : -1;
  };
  if (a.unit == 16) stage_tile<T, 16>(tile, (const T*)a.x, a.ldx, col0, ncols, source);
  else if (a.unit == 8) stage_tile<T, 8>(tile, (const T*)a.x, a.ldx, col0, ncols, source);
  else if (a.unit == 4) stage_tile<T, 4>(tile, (const T*)a.x, a.ldx, col0, ncols, source);
  else if constexpr (sizeof(T) == 2) stage_elements(tile, (const T*)a.x, a.ldx, col0, ncols, source);
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();

  // Maxima.  Rows: 16 lanes a row, 8 values each; columns: two and 32 of their rows to a thread.  The
  // loops are unrolled in part: in full, a small call with cold caches spent its time on instruction
  // fetches (the training step of 6 rows of 376 x 560 bf16 42.6 us against 38.6), and large ones gained
  // nothing.
  const int64_t qcol = col0 + lane16 * 8;
  const int c = (threadIdx.x & 63) * 2, part = threadIdx.x >> 6;
  const T* mine = tile + part * kPartRows * kLd + c;
  float tile_max = 0.f;
#pragma unroll 2
  for (int p = 0; p < 128 * 16 / kThreads; ++p) {
    const int i = p * (kThreads / 16) + (threadIdx.x >> 4);
    MaxPair<T> mp;
#pragma unroll
    for (int e = 0; e < 8; e += 2) mp.add(tile + i * kLd + lane16 * 8 + e);
    const float2 m2 = mp.get();
    float m = max_mag(m2.x, m2.y);
    if constexpr (ROW_BLOCK || COL_BLOCK) tile_max = max_mag(tile_max, m);
    if constexpr (!ROW_BLOCK) {
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) m = max_mag(m, __shfl_xor_sync(kFull, m, o));
      if (lane16 == 0) row_max[i] = m;
    }
  }
  if constexpr (!COL_BLOCK) {
    MaxPair<T> mp;
#pragma unroll 8
    for (int i = 0; i < kPartRows; ++i) mp.add(mine + i * kLd);
    *(float2*)&col_max[part][c] = mp.get();
  }
  float block_amax = 0.f, block_inv = 0.f;
  if constexpr (ROW_BLOCK || COL_BLOCK) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) tile_max = max_mag(tile_max, __shfl_xor_sync(kFull, tile_max, o));
    if (lane == 0) warp_max[warp] = tile_max;
  }
  __syncthreads();
  // Scales and multipliers: a row or a column to a thread.
  if constexpr (ROW_BLOCK || COL_BLOCK) {
    tile_max = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) tile_max = max_mag(tile_max, warp_max[w]);
    block_amax = at_least_floor(tile_max);
    block_inv = __fdiv_rn(kTop, block_amax);
  }
  if constexpr (ROW_BLOCK) {
    if (threadIdx.x == 0) {
      const int64_t row_blocks = (a.rows + 127) / 128;
      const float s = __fdiv_rn(block_amax, kTop);
      a.scale[((int64_t)g * row_blocks + tnum) * a.col_blocks + blockIdx.y] = s;
      if (a.qt) a.scale_t[((int64_t)g * a.col_blocks + blockIdx.y) * row_blocks + tnum] = s;
    }
  } else {
    const int i = threadIdx.x & 127;
    if (threadIdx.x < 128) {
      const float m = at_least_floor(row_max[i]);
      row_max[i] = __fdiv_rn(kTop, m);
      if (i < n) a.scale[(int64_t)blockIdx.y * a.ld_scale + row0 + i] = __fdiv_rn(m, kTop);
    } else if (threadIdx.x >= 256) {
    } else if constexpr (!COL_BLOCK) {
      float m = 0.f;
#pragma unroll
      for (int p = 0; p < kParts; ++p) m = max_mag(m, col_max[p][i]);
      m = at_least_floor(m);
      col_max[0][i] = __fdiv_rn(kTop, m);
      if (i < ncols) a.scale_t[(int64_t)tnum * a.ld_scale_t + col0 + i] = __fdiv_rn(m, kTop);
    } else if (i == 0) {
      a.scale_t[(int64_t)blockIdx.y * a.ld_scale_t + tnum] = __fdiv_rn(block_amax, kTop);
    }
    __syncthreads();
  }
  // Row codes.
  uint8_t* q = a.q + ((ROW_BLOCK ? xbase : 0) + row0 + (threadIdx.x >> 4)) * a.ldq + qcol;
#pragma unroll 2
  for (int p = 0; p < 128 * 16 / kThreads; ++p) {
    const int i = p * (kThreads / 16) + (threadIdx.x >> 4);
    float v[8];
    load8(tile + i * kLd, lane16 * 8, 128, true, v);
    const float inv = ROW_BLOCK ? block_inv : row_max[i];
    if (i < n) *(uint2*)q = make_uint2(codes4(v, inv), codes4(v + 4, inv));
    q += (kThreads / 16) * a.ldq;
  }
  if (!a.qt) return;
  const float inv0 = COL_BLOCK ? block_inv : col_max[0][c], inv1 = COL_BLOCK ? block_inv : col_max[0][c + 1];
  // The codes go through shared memory (over the tile, which is in registers by then), so that eight
  // lanes write a column's 128 bytes together.
  uint32_t w[2][kPartRows / 4];
#pragma unroll
  for (int b = 0; b < kPartRows / 4; ++b) {
    float f0[4], f1[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 v = two(mine + (4 * b + e) * kLd);
      f0[e] = v.x;
      f1[e] = v.y;
    }
    w[0][b] = codes4(f0, inv0);
    w[1][b] = codes4(f1, inv1);
  }
  constexpr int kCodeLd = 144;
  uint8_t* codes = smem;
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint4* dst = (uint4*)(codes + (c + h) * kCodeLd + part * kPartRows);
#pragma unroll
    for (int b = 0; b < kPartRows / 16; ++b)
      dst[b] = make_uint4(w[h][4 * b], w[h][4 * b + 1], w[h][4 * b + 2], w[h][4 * b + 3]);
  }
  __syncthreads();
  const int64_t qrow = (ROW_BLOCK ? (int64_t)g * a.cols : 0) + col0;
#pragma unroll
  for (int p = 0; p < 128 * 8 / kThreads; ++p) {
    const int cc = p * (kThreads / 8) + (threadIdx.x >> 3), piece = threadIdx.x & 7;
    if (col0 + cc < a.cols)
      *(uint4*)(a.qt + (qrow + cc) * a.ldt + (int64_t)tnum * 128 + piece * 16) =
          *(const uint4*)(codes + cc * kCodeLd + piece * 16);
  }
}

template <typename T, bool ROW_BLOCK, bool COL_BLOCK>
int launch_tiles(const TileArgs& a, int64_t tiles, cudaStream_t s) {
  auto k = quantize_tile_kernel<T, ROW_BLOCK, COL_BLOCK>;
  const int smem = 128 * tile_ld<T>() * (int)sizeof(T);
  static std::atomic<uint64_t> ready{0};
  if (!once_per_device(ready, [&] {
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess;
      }))
    return CTR_ERR_CUDA;
  launch_after(k, dim3((unsigned)tiles, (unsigned)a.col_blocks), tile_threads<T>(), smem, s, 1, a);
  return launch_status();
}

bool aligned16(const void* p) { return ((uintptr_t)p % 16) == 0; }

}  // namespace
}  // namespace ctr

using namespace ctr;

extern "C" int64_t ctr_fp8_padded_rows(int64_t rows, int32_t groups) {
  if (rows < 0 || groups < 1) return -1;
  // a group of c rows takes ceil(c / 128) <= c tiles
  return 128 * imax64(1, imin64((rows + 127 * (int64_t)groups) / 128, rows));
}

extern "C" int ctr_fp8_quantize_rows(const void* x, ctr_dtype dtype, int64_t x_rows, int64_t rows, int64_t cols,
                                     int64_t ldx, const int32_t* row_index, uint8_t* q, float* scale,
                                     int64_t ld_scale, void* ws, size_t ws_bytes, ctr_stream_t stream) {
  if (!dtype_ok(dtype) || x_rows < 0 || rows < 0 || cols < 1 || ldx < cols || ld_scale < rows)
    return CTR_ERR_INVALID_ARG;
  if (!row_index && rows > x_rows) return CTR_ERR_INVALID_ARG;
  if (rows > INT32_MAX || cols > 65535 * 256) return CTR_ERR_UNSUPPORTED;
  if (!ws_valid(ws, ws_bytes, kWsHeader)) return CTR_ERR_WORKSPACE;
  if (rows == 0) return CTR_OK;
  const int eb = dtype_bytes(dtype);
  if (!x || !q || !scale || ((uintptr_t)x % eb) || !aligned16(q)) return CTR_ERR_INVALID_ARG;
  const int vec = aligned16(x) && (ldx * eb) % 16 == 0;
  const int kb = (int)ceil_div(cols, 128);
  const int64_t parts = ceil_div(kb, dtype == CTR_F32 ? row_blocks<float>() : row_blocks<__nv_bfloat16>());
  // rows are walked by as many CTAs as are resident, so that a lane group has a next row to load
  const int64_t resident = imax64(1, ceil_div((int64_t)num_sms() * 5, parts));
  const dim3 grid((unsigned)imin64(ceil_div(rows, kQThreads / 16), resident), (unsigned)parts);
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == CTR_F32)
    launch_after(quantize_rows_kernel<float>, grid, kQThreads, 0, s, 1, (const float*)x, x_rows, rows, cols, ldx, vec,
                 row_index, q, scale, ld_scale, kb, (int*)ws);
  else
    launch_after(quantize_rows_kernel<__nv_bfloat16>, grid, kQThreads, 0, s, 1, (const __nv_bfloat16*)x, x_rows, rows,
                 cols, ldx, vec, row_index, q, scale, ld_scale, kb, (int*)ws);
  return launch_status();
}

extern "C" int ctr_fp8_quantize_rows_cols(const void* x, ctr_dtype dtype, int64_t x_rows, int64_t rows, int64_t cols,
                                          int64_t ldx, const int32_t* row_index, const int32_t* offsets,
                                          int32_t groups, int cols_by_block, uint8_t* q, float* scale,
                                          int64_t ld_scale, uint8_t* qc, float* scale_c, void* ws, size_t ws_bytes,
                                          ctr_stream_t stream) {
  if (!dtype_ok(dtype) || x_rows < 0 || rows < 0 || cols < 1 || ldx < cols || ld_scale < rows || groups < 1)
    return CTR_ERR_INVALID_ARG;
  if (!offsets || (!row_index && rows > x_rows) || (cols_by_block != 0 && cols_by_block != 1))
    return CTR_ERR_INVALID_ARG;
  // the kernel rounds a group's rows up to tiles in 32 bits; the products take no more rows either
  if (rows > INT32_MAX - 65536 || cols > INT32_MAX || groups > CTR_MAX_EXPERTS) return CTR_ERR_UNSUPPORTED;
  if (!ws_valid(ws, ws_bytes, kWsHeader)) return CTR_ERR_WORKSPACE;
  if (rows == 0) return CTR_OK;
  const int eb = dtype_bytes(dtype);
  if (!x || !q || !scale || !qc || !scale_c || ((uintptr_t)x % eb) || !aligned16(q) || !aligned16(qc))
    return CTR_ERR_INVALID_ARG;
  const int64_t padded = ctr_fp8_padded_rows(rows, groups), tiles = padded / 128;
  if (tiles > INT32_MAX || ceil_div(cols, 128) > 65535) return CTR_ERR_UNSUPPORTED;
  TileArgs a = {};
  a.x = x;
  a.x_rows = x_rows;
  a.rows = rows;
  a.cols = cols;
  a.ldx = ldx;
  a.row_index = row_index;
  a.offsets = offsets;
  a.groups = groups;
  a.unit = vector_bytes({(uint64_t)(uintptr_t)x, (uint64_t)(ldx * eb)}, eb);
  a.col_blocks = (int32_t)ceil_div(cols, 128);
  a.q = q;
  a.scale = scale;
  a.ldq = (int64_t)a.col_blocks * 128;
  a.ld_scale = ld_scale;
  a.qt = qc;
  a.scale_t = scale_c;
  a.ldt = padded;
  a.ld_scale_t = cols_by_block ? tiles : cols;
  a.err = (int*)ws;
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == CTR_F32)
    return cols_by_block ? launch_tiles<float, false, true>(a, tiles, s) : launch_tiles<float, false, false>(a, tiles, s);
  return cols_by_block ? launch_tiles<__nv_bfloat16, false, true>(a, tiles, s)
                       : launch_tiles<__nv_bfloat16, false, false>(a, tiles, s);
}

extern "C" int ctr_fp8_quantize_blocks(const void* w, ctr_dtype dtype, int32_t groups, int64_t n, int64_t k,
                                       uint8_t* q, float* scale, uint8_t* qt, float* scale_t, void* ws,
                                       size_t ws_bytes, ctr_stream_t stream) {
  if (!dtype_ok(dtype) || groups < 1 || n < 1 || k < 1 || (qt == nullptr) != (scale_t == nullptr))
    return CTR_ERR_INVALID_ARG;
  if (n > INT32_MAX || k > INT32_MAX || groups > CTR_MAX_EXPERTS) return CTR_ERR_UNSUPPORTED;
  if (!ws_valid(ws, ws_bytes, kWsHeader)) return CTR_ERR_WORKSPACE;
  const int eb = dtype_bytes(dtype);
  if (!w || !q || !scale || ((uintptr_t)w % eb) || !aligned16(q) || !aligned16(qt)) return CTR_ERR_INVALID_ARG;
  const int64_t tiles = groups * ceil_div(n, 128);
  if (tiles > INT32_MAX || ceil_div(k, 128) > 65535) return CTR_ERR_UNSUPPORTED;
  TileArgs a = {};
  a.x = w;
  a.x_rows = n;
  a.rows = n;
  a.cols = k;
  a.ldx = k;
  a.groups = groups;
  a.unit = vector_bytes({(uint64_t)(uintptr_t)w, (uint64_t)(k * eb)}, eb);
  a.col_blocks = (int32_t)ceil_div(k, 128);
  a.q = q;
  a.scale = scale;
  a.ldq = (int64_t)a.col_blocks * 128;
  a.qt = qt;
  a.scale_t = scale_t;
  a.ldt = ceil_div(n, 128) * 128;
  a.err = (int*)ws;
  cudaStream_t s = (cudaStream_t)stream;
  return dtype == CTR_F32 ? launch_tiles<float, true, true>(a, tiles, s)
                          : launch_tiles<__nv_bfloat16, true, true>(a, tiles, s);
}
