// b1/b2. Expert routing, and rows into expert order and back.
//
// Source: "DHEN" notes, the mixture-of-experts section (a gate sends each
// sample to a few experts); the formulas and the row order are stated in
// include/ctr.h.
//
// Routing.  A token's scores are spread over a group of lanes (at least k), EPL
// consecutive scores to a lane.  fp32: the k choices are k rounds of "best score
// not yet taken" (in-lane maximum, then xor-shuffles; ties go to the lower index).
// bf16 scores carry their index in the low half of an ordered 32-bit key, so that
// integer maxima and minima are all it takes; three or four choices come from
// sorting networks (131072 x 64, k 4, with the order: 36 us before, 26 with both).
// Then lane j has choice j, its exponential and its stores.  Bound by latency and
// issue (0.57 of the cycles issue, 41% of the warps are active).  The stable order by expert is a counting sort without atomics on
// counts: a block's tile of up to 256 tokens is a bit matrix [expert][token]
// in shared memory, so a choice's rank within the tile is a population count
// of the bits before it, and the tile's count of an expert the count of all.
// Three launches: choices + tile counts; exclusive sums of the counts over the
// tiles (one warp column per expert); ranks and the two maps.  Up to kTileTokens
// x 16 tokens run as one launch, a block or a cluster of up to sixteen blocks that
// read each other's counts (2048 x 26, k 4: 6.1 us), where the device can place it.
//
// Rows.  A token's group of lanes reads its row once and writes its k rows (or
// reads k rows and writes one): every byte crosses HBM once, and rows of 1 KB
// and more keep scattered writes whole.  Bound by HBM.
#include <cuda_bf16.h>

#include <algorithm>
#include <initializer_list>

#include "common.cuh"
#include "rows.cuh"

namespace ctr {
namespace {

constexpr int kRouteThreads = 512;
constexpr int kTileTokens = 256;      // tokens of a tile, at most
// One block does it all up to this many scores (tokens x experts) and kTileTokens tokens.
constexpr int64_t kOneBlockScores = 16384;

struct RouteArgs {
  const void* scores;
  int64_t tokens, ld;
  int32_t experts, k, lanes, tile, tiles;  // lanes: per token; tile: tokens of a tile
  int32_t renormalize, vec;                // vec: rows start 16-byte aligned
  int32_t* expert;
  float* weight;
  int32_t* slot;
  int32_t* token;
  int32_t* offsets;
  int32_t* counts;  // [tiles][experts], then [experts] totals
  int* err;
};

// Scores base .. base + EPL - 1 of a row; -inf past the last expert.
template <typename T, int EPL>
__device__ __forceinline__ void load_scores(const T* row, int base, int experts, bool vec, float (&v)[EPL]) {
  constexpr int per = 16 / (int)sizeof(T);
  if (vec && base + EPL <= experts) {
#pragma unroll
    for (int i = 0; i < EPL; i += per) {
      float f[per];
      Chunk<T, 16>::unpack(*(const uint4*)(row + base + i), f);
#pragma unroll
      for (int q = 0; q < per; ++q) v[i + q] = f[q];
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = base + i < experts ? to_f32<T>(row[base + i]) : -INFINITY;
  }
}

// Exclusive sum of totals[0 .. experts) into start (shared); returns the sum.  All threads.
static_assert(kRouteThreads >= CTR_MAX_EXPERTS, "an expert to a thread");
__device__ __forceinline__ int expert_starts(const int* totals, int experts, int* start, int* warp_sum) {
  const int e = threadIdx.x;
  const int mine = e < experts ? totals[e] : 0;
  int x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if ((threadIdx.x & 31) >= o) x += y;
  }
  if ((threadIdx.x & 31) == 31) warp_sum[threadIdx.x >> 5] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kRouteThreads / 32; ++w) {
    if (w < (int)(threadIdx.x >> 5)) before += warp_sum[w];
    all += warp_sum[w];
  }
  if (e < experts) start[e] = before + x - mine;
  __syncthreads();
  return all;
}

// What a lane learns of its group's token: choice `sub`'s score and expert (-1: none), the best score,
// and, where the weights are over the whole row, the sum of exp(score - best).
struct Choice {
  float value = -INFINITY, best = 0.f, total = 0.f;
  int expert = -1;
};

// fp32: a round a choice, the value first, then the lowest index that has it.
template <typename T, int EPL, int KMAX>
struct Chooser {
  static __device__ __forceinline__ Choice run(const RouteArgs& a, const T* row, bool mine, int sub) {
    const int base = sub * EPL;
    float v[EPL];
    if (mine) {
      load_scores<T, EPL>(row, base, a.experts, a.vec != 0, v);
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[i] = -INFINITY;
    }
    bool odd = false;  // NaN or +inf: the token is routed nowhere
#pragma unroll
    for (int i = 0; i < EPL; ++i) odd |= !(v[i] < INFINITY);
    const int lane = threadIdx.x & 31;
    const uint32_t group = (a.lanes == 32 ? kFull : ((1u << a.lanes) - 1)) << (lane & ~(a.lanes - 1));
    const bool bad = (__ballot_sync(kFull, odd) & group) != 0;
    if (bad) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[i] = -INFINITY;
      if (sub == 0) set_error(a.err, CTR_ERR_BAD_VALUE);
    }
    Choice c;
    if (!a.renormalize) {
      float m = v[0];
#pragma unroll
      for (int i = 1; i < EPL; ++i) m = fmaxf(m, v[i]);
      for (int o = 1; o < a.lanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
      if (!(m > -INFINITY)) m = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) c.total += expf(v[i] - m);  // exp(-inf) = 0: masked scores add nothing
      for (int o = 1; o < a.lanes; o <<= 1) c.total += __shfl_xor_sync(kFull, c.total, o);
    }
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      if (j < a.k) {
        float best = v[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) best = fmaxf(best, v[i]);
        for (int o = 1; o < a.lanes; o <<= 1) best = fmaxf(best, __shfl_xor_sync(kFull, best, o));
        int at = 0x7fffffff;
#pragma unroll
        for (int i = EPL - 1; i >= 0; --i) at = v[i] == best ? base + i : at;
        for (int o = 1; o < a.lanes; o <<= 1) at = min(at, __shfl_xor_sync(kFull, at, o));
        if (best > -INFINITY) {
          if (j == 0) c.best = best;
          if (j == sub) {
            c.value = best;
            c.expert = at;
          }
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) v[i] = base + i == at ? -INFINITY : v[i];
      }
    }
    return c;
  }
};

// bf16: a score is a 32-bit key, its 16 bits made to order as an unsigned number (negative ones
// complemented, else the sign set) above the complement of the index, so that integer maxima find value
// and lowest index together.  -inf is 0x007f, below every number; +inf and, as adding zero makes them all
// positive, NaNs are 0xff80 and above and come out as the best.
template <int EPL, int KMAX>
struct Chooser<__nv_bfloat16, EPL, KMAX> {
  static constexpr uint32_t kLeast = 0x00800000u, kBad = 0xff800000u;  // keys of numbers lie between

  static __device__ __forceinline__ float value(uint32_t key) {
    return __uint_as_float((key & 0xffff0000u) ^ (key & 0x80000000u ? 0x80000000u : 0xffff0000u));
  }
  static __device__ __forceinline__ void order(uint32_t& x, uint32_t& y) {
    const uint32_t hi = max(x, y);
    y = min(x, y);
    x = hi;
  }
  // a and b in falling order: a becomes the four largest of both, in falling order
  static __device__ __forceinline__ void merge4(uint32_t* a, const uint32_t* b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = max(a[i], b[3 - i]);
    order(a[0], a[2]);
    order(a[1], a[3]);
    order(a[0], a[1]);
    order(a[2], a[3]);
  }
  // The group's k largest keys.  Three and four by sorting networks: fours within the lane, then the best
  // four of two lists until one is left.  Else a round a choice.
  static __device__ __forceinline__ void largest(uint32_t (&key)[EPL], int lanes, int k, uint32_t (&top)[KMAX]) {
    if (KMAX == 4 && k > 2) {
#pragma unroll
      for (int i = 0; i < EPL; i += 4) {
        order(key[i], key[i + 1]);
        order(key[i + 2], key[i + 3]);
        order(key[i], key[i + 2]);
        order(key[i + 1], key[i + 3]);
        order(key[i + 1], key[i + 2]);
      }
#pragma unroll
      for (int w = 4; w < EPL; w *= 2)
#pragma unroll
        for (int i = 0; i < EPL; i += 2 * w) merge4(key + i, key + i + w);
      for (int o = 1; o < lanes; o <<= 1) {
        uint32_t other[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) other[i] = __shfl_xor_sync(kFull, key[i], o);
        merge4(key, other);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) top[j] = key[j];
    } else {
#pragma unroll
      for (int j = 0; j < KMAX; ++j) {
        top[j] = 0;
        if (j < k) {
          uint32_t best = key[0];
#pragma unroll
          for (int i = 1; i < EPL; ++i) best = max(best, key[i]);
          for (int o = 1; o < lanes; o <<= 1) best = max(best, __shfl_xor_sync(kFull, best, o));
          top[j] = best;
          if (j + 1 < k) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) key[i] = key[i] == best ? 0u : key[i];
          }
        }
      }
    }
  }

  static __device__ __forceinline__ Choice run(const RouteArgs& a, const __nv_bfloat16* row, bool mine, int sub) {
    const int base = sub * EPL;
    uint32_t w[EPL / 2];  // pairs of scores
    if (mine && a.vec && base + EPL <= a.experts) {
#pragma unroll
      for (int i = 0; i < EPL / 8; ++i) *(uint4*)(w + 4 * i) = *(const uint4*)(row + base + 8 * i);
    } else {
#pragma unroll
      for (int i = 0; i < EPL / 2; ++i) {
        const int e = base + 2 * i;
        const uint32_t lo = mine && e < a.experts ? __bfloat16_as_ushort(row[e]) : 0xff80u;
        const uint32_t hi = mine && e + 1 < a.experts ? __bfloat16_as_ushort(row[e + 1]) : 0xff80u;
        w[i] = lo | (hi << 16);
      }
    }
    uint32_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL / 2; ++i) {
      uint32_t x, sign;
      asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(w[i]), "r"(0u));  // -0 becomes +0
      asm("prmt.b32 %0, %1, 0, 0xbb99;" : "=r"(sign) : "r"(x));         // all ones for a negative half
      x ^= sign | 0x80008000u;
      const uint32_t index = 0xfffeffffu - 0x00010001u * (uint32_t)(base + 2 * i);  // complements, two
      key[2 * i] = __byte_perm(x, index, 0x1054);
      key[2 * i + 1] = __byte_perm(x, index, 0x3276);
    }
    uint32_t top[KMAX];
    largest(key, a.lanes, a.k, top);
    const bool bad = top[0] >= kBad;
    if (bad && sub == 0) set_error(a.err, CTR_ERR_BAD_VALUE);
    uint32_t own = 0;
#pragma unroll
    for (int j = 0; j < KMAX; ++j) own = j == sub ? top[j] : own;
    Choice c;
    if (!bad && top[0] >= kLeast) c.best = value(top[0]);
    if (!bad && own >= kLeast && sub < a.k) {
      c.value = value(own);
      c.expert = 0xffff - (int)(own & 0xffffu);
    }
    if (!a.renormalize) {
#pragma unroll
      for (int i = 0; i < EPL / 2; ++i)  // exp(-inf) = 0: masked scores add nothing
        c.total += expf(__uint_as_float(w[i] << 16) - c.best) + expf(__uint_as_float(w[i] & 0xffff0000u) - c.best);
      for (int o = 1; o < a.lanes; o <<= 1) c.total += __shfl_xor_sync(kFull, c.total, o);
    }
    return c;
  }
};

// i / k for the choices of a tile, i < kTileTokens * k: with m = ceil(2^16 / k), i m / 2^16 is too large by
// less than i / 2^16 < 1 / k.
struct TokenOf {
  uint32_t m;
  __device__ __forceinline__ explicit TokenOf(int k) : m((65535u + (uint32_t)k) / (uint32_t)k) {}
  __device__ __forceinline__ int operator()(int i) const { return (int)(((uint32_t)i * m) >> 16); }
};
static_assert(kTileTokens * CTR_MAX_CHOICES * CTR_MAX_CHOICES <= 65536, "a tile's choices leave the bound of TokenOf");

// Ranks of the tile's choices from its bit matrix: slot and token of each, given the first row of
// every expert's choices in this tile.  `before` gets each word's count of earlier tokens.
__device__ __forceinline__ void write_slots(const RouteArgs& a, int64_t t0, int n, const uint32_t* bits,
                                            uint16_t* before, const int* first) {
  const int words = a.tile / 32;
  for (int e = threadIdx.x; e < a.experts; e += kRouteThreads) {
    int c = 0;
    for (int w = 0; w < words; ++w) {
      before[e * words + w] = (uint16_t)c;
      c += __popc(bits[e * words + w]);
    }
  }
  __syncthreads();
  const TokenOf token_of(a.k);
  for (int i = threadIdx.x; i < n * a.k; i += kRouteThreads) {
    const int64_t at = t0 * a.k + i;
    const int e = a.expert[at];
    int s = -1;
    if (e >= 0) {
      const int t = token_of(i), w = e * words + (t >> 5);
      s = first[e] + before[w] + __popc(bits[w] & ((1u << (t & 31)) - 1));
      a.token[s] = (int32_t)(t0 + t);
    }
    a.slot[at] = s;
  }
}

template <typename T, int EPL, int KMAX, bool CLUSTER>
__global__ void __launch_bounds__(kRouteThreads) route_choose_kernel(const RouteArgs a) {
  extern __shared__ uint32_t bits[];  // [experts][tile / 32], then uint16 before[...] and int first[experts]
  const int words = a.tile / 32;
  const int64_t t0 = (int64_t)blockIdx.x * a.tile;
  const int n = (int)imin64(a.tile, a.tokens - t0);
  for (int i = threadIdx.x; i < a.experts * words; i += kRouteThreads) bits[i] = 0;
  __syncthreads();
  grid_wait();
  const int lane = threadIdx.x & 31, sub = lane & (a.lanes - 1);
  const int per_pass = kRouteThreads / a.lanes;
  for (int p0 = 0; p0 < n; p0 += per_pass) {  // the same trips in every lane: the shuffles need all of them
    const int tl = p0 + (int)threadIdx.x / a.lanes;
    const bool mine = tl < n;
    // lane j of the group has choice j
    const Choice c = Chooser<T, EPL, KMAX>::run(a, (const T*)a.scores + (t0 + tl) * a.ld, mine, sub);
    const float z = c.expert >= 0 ? expf(c.value - c.best) : 0.f;
    float total = c.total;
    if (a.renormalize) {
      total = z;
      for (int o = 1; o < a.lanes; o <<= 1) total += __shfl_xor_sync(kFull, total, o);
    }
    if (mine && sub < a.k) {
      const int64_t at = (t0 + tl) * a.k + sub;
      a.expert[at] = c.expert;
      a.weight[at] = c.expert >= 0 ? z / total : 0.f;
      if (c.expert >= 0) atomicOr(&bits[c.expert * words + (tl >> 5)], 1u << (tl & 31));
    }
  }
  __syncthreads();
  if (!CLUSTER && a.tiles > 1) {
    for (int e = threadIdx.x; e < a.experts; e += kRouteThreads) {
      int c = 0;
      for (int w = 0; w < words; ++w) c += __popc(bits[e * words + w]);
      a.counts[(int64_t)blockIdx.x * a.experts + e] = c;
    }
    return;
  }
  // all tiles are this block's, or this cluster's: an expert to a thread
  __shared__ int warp_sum[kRouteThreads / 32];
  uint16_t* before = (uint16_t*)(bits + a.experts * words);
  int* first = (int*)(before + ((a.experts * words + 1) & ~1));
  int* mine = first + a.experts;
  int* totals = mine + a.experts;
  const int e = threadIdx.x;
  if (e < a.experts) {
    int c = 0;
    for (int w = 0; w < words; ++w) c += __popc(bits[e * words + w]);
    mine[e] = c;
  }
  __syncthreads();
  if constexpr (CLUSTER) cluster_sync();
  int earlier = 0;  // the expert's choices in the tiles before this one
  if (e < a.experts) {
    int all = 0;
    for (int r = 0; r < a.tiles; ++r) {
      int c;
      if constexpr (CLUSTER)
        asm volatile("ld.shared::cluster.s32 %0, [%1];"
                     : "=r"(c)
                     : "r"(in_cta((uint32_t)__cvta_generic_to_shared(mine + e), r))
                     : "memory");
      else
        c = mine[e];
      if (r < (int)blockIdx.x) earlier += c;
      all += c;
    }
    totals[e] = all;
  }
  __syncthreads();
  const int all = expert_starts(totals, a.experts, first, warp_sum);
  if (blockIdx.x == 0) {
    if (e < a.experts) a.offsets[e] = first[e];
    if (e == 0) a.offsets[a.experts] = all;
  }
  __syncthreads();
  if (e < a.experts) first[e] += earlier;
  __syncthreads();
  write_slots(a, t0, n, bits, before, first);
  for (int64_t r = all + (int64_t)blockIdx.x * kRouteThreads + threadIdx.x; r < a.tokens * a.k;
       r += (int64_t)gridDim.x * kRouteThreads)
    a.token[r] = -1;
  __syncthreads();
  if constexpr (CLUSTER) cluster_sync();  // no block leaves while another reads its counts
}

// counts[tile][e] -> exclusive sum over the tiles, and the totals: 32 experts to a block, one to a
// lane, the tiles cut into one segment a warp.
__global__ void __launch_bounds__(1024) route_scan_kernel(const RouteArgs a) {
  __shared__ int seg[32][33];
  grid_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + lane;
  const int per = (a.tiles + 31) / 32;
  const int b0 = min(a.tiles, warp * per), b1 = min(a.tiles, b0 + per);
  int sum = 0;
  if (e < a.experts) {
#pragma unroll 8
    for (int b = b0; b < b1; ++b) sum += a.counts[(int64_t)b * a.experts + e];
  }
  seg[warp][lane] = sum;
  __syncthreads();
  int run = 0, all = 0;
  for (int w = 0; w < 32; ++w) {
    if (w < warp) run += seg[w][lane];
    all += seg[w][lane];
  }
  if (e >= a.experts) return;
  for (int b = b0; b < b1; b += 8) {
    int x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = b + i < b1 ? a.counts[(int64_t)(b + i) * a.experts + e] : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (b + i < b1) a.counts[(int64_t)(b + i) * a.experts + e] = run;
      run += x[i];
    }
  }
  if (warp == 0) a.counts[(int64_t)a.tiles * a.experts + e] = all;
}

__global__ void __launch_bounds__(kRouteThreads) route_rank_kernel(const RouteArgs a) {
  extern __shared__ uint32_t bits[];
  __shared__ int warp_sum[kRouteThreads / 32];
  const int words = a.tile / 32;
  uint16_t* before = (uint16_t*)(bits + a.experts * words);
  int* first = (int*)(before + ((a.experts * words + 1) & ~1));
  const int64_t t0 = (int64_t)blockIdx.x * a.tile;
  const int n = (int)imin64(a.tile, a.tokens - t0);
  for (int i = threadIdx.x; i < a.experts * words; i += kRouteThreads) bits[i] = 0;
  __syncthreads();
  grid_wait();
  const TokenOf token_of(a.k);
  for (int i = threadIdx.x; i < n * a.k; i += kRouteThreads) {
    const int e = a.expert[t0 * a.k + i], t = token_of(i);
    if (e >= 0) atomicOr(&bits[e * words + (t >> 5)], 1u << (t & 31));
  }
  const int all = expert_starts(a.counts + (int64_t)a.tiles * a.experts, a.experts, first, warp_sum);
  if (blockIdx.x == 0) {
    for (int e = threadIdx.x; e < a.experts; e += kRouteThreads) a.offsets[e] = first[e];
    if (threadIdx.x == 0) a.offsets[a.experts] = all;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kRouteThreads)
    first[e] += a.counts[(int64_t)blockIdx.x * a.experts + e];
  __syncthreads();
  write_slots(a, t0, n, bits, before, first);
  for (int64_t r = all + (int64_t)blockIdx.x * kRouteThreads + threadIdx.x; r < a.tokens * a.k;
       r += (int64_t)gridDim.x * kRouteThreads)
    a.token[r] = -1;
}

__global__ void route_empty_kernel(int32_t* offsets, int experts) {
  grid_wait();
  for (int e = threadIdx.x; e <= experts; e += blockDim.x) offsets[e] = 0;
}

// Writes a lane's EPL values of a row (base + EPL may pass the last expert).
template <typename T, int EPL>
__device__ __forceinline__ void store_scores(T* out, int base, int experts, bool vec, const float (&v)[EPL]) {
  constexpr int per = 16 / (int)sizeof(T);
  if (vec && base + EPL <= experts) {
#pragma unroll
    for (int i = 0; i < EPL; i += per) {
      float f[per];
#pragma unroll
      for (int q = 0; q < per; ++q) f[q] = v[i + q];
      *(uint4*)(out + i) = Chunk<T, 16>::pack(f);
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (base + i < experts) out[i] = from_f32<T>(v[i]);
  }
}

// Softmax over the choices: lane j of a token's lanes (as few as hold its choices) reads choice j's score
// alone.  The other scores' gradient is zero: the lanes write the row's zeros first, then each its choice
// over them (selecting the values' places in registers took twice the instructions: 131072 x 64 bf16, k 4,
// 18.4 us against 14.3; 256, k 8, 61 against 29).
template <typename T>
__global__ void __launch_bounds__(kRouteThreads) route_bwd_choices_kernel(const RouteArgs a, const float* dweight,
                                                                          T* dscores, int64_t ldd, int vec_out) {
  constexpr int per = 16 / (int)sizeof(T);
  const int lane = threadIdx.x & 31, sub = lane & (a.lanes - 1);
  const int64_t groups = (int64_t)gridDim.x * (kRouteThreads / a.lanes);
  int64_t t = ((int64_t)blockIdx.x * kRouteThreads + threadIdx.x) / a.lanes;
  const int64_t trips = ceil_div(a.tokens, groups);  // the same in every lane
  grid_wait();
  for (int64_t trip = 0; trip < trips; ++trip, t += groups) {
    const bool mine = t < a.tokens;
    T* out = dscores + t * ldd;
    const int e = mine && sub < a.k ? a.expert[t * a.k + sub] : -1;
    const bool live = e >= 0 && e < a.experts;
    const float l = live ? to_f32<T>(((const T*)a.scores)[t * a.ld + e]) : -INFINITY;
    const float g = live ? dweight[t * a.k + sub] : 0.f;
    if (mine) {
      int done = 0;
      if (vec_out) {
        done = a.experts & ~(per - 1);
        for (int i = sub * per; i < done; i += a.lanes * per) *(uint4*)(out + i) = make_uint4(0, 0, 0, 0);
      }
      for (int i = done + sub; i < a.experts; i += a.lanes) out[i] = from_f32<T>(0.f);
    }
    float m = l;
    for (int o = 1; o < a.lanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    const float z = live ? expf(l - m) : 0.f;
    float total = z, dot = z * g;
    for (int o = 1; o < a.lanes; o <<= 1) {
      total += __shfl_xor_sync(kFull, total, o);
      dot += __shfl_xor_sync(kFull, dot, o);
    }
    __syncwarp();  // the row's zeros come before its choices
    if (live) {    // then total >= its own exponential > 0
      const float inv = 1.f / total;
      out[e] = from_f32<T>(z * inv * (g - dot * inv));
    }
  }
}

// Softmax over the whole row: d score_i = p_i (g_i - sum p g), g of the scores not chosen 0.
template <typename T, int EPL>
__global__ void __launch_bounds__(kRouteThreads) route_bwd_kernel(const RouteArgs a, const float* dweight, T* dscores,
                                                                  int64_t ldd, int vec_out) {
  const int lane = threadIdx.x & 31, sub = lane & (a.lanes - 1);
  const int base = sub * EPL;
  const int64_t groups = (int64_t)gridDim.x * (kRouteThreads / a.lanes);
  int64_t t = ((int64_t)blockIdx.x * kRouteThreads + threadIdx.x) / a.lanes;
  const int64_t trips = ceil_div(a.tokens, groups);  // the same in every lane
  grid_wait();
  for (int64_t trip = 0; trip < trips; ++trip, t += groups) {
    const bool mine = t < a.tokens;
    const T* row = (const T*)a.scores + t * a.ld;
    // lane j has choice j
    const int e = mine && sub < a.k ? a.expert[t * a.k + sub] : -1;
    const bool live = e >= 0 && e < a.experts;
    const float g = live ? dweight[t * a.k + sub] : 0.f;
    const uint32_t group = (a.lanes == 32 ? kFull : ((1u << a.lanes) - 1)) << (lane & ~(a.lanes - 1));
    // a token with no choice (all masked, or flagged by the routing) has no gradient
    const bool routed = (__ballot_sync(kFull, live) & group) != 0;
    float out[EPL];
    float v[EPL], gi[EPL];
    if (mine) {
      load_scores<T, EPL>(row, base, a.experts, a.vec != 0, v);
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[i] = -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) gi[i] = 0.f;
    for (int j = 0; j < a.k; ++j) {
      const int at = __shfl_sync(kFull, live ? e : -1, j, a.lanes) - base;
      const float gj = __shfl_sync(kFull, g, j, a.lanes);
#pragma unroll
      for (int i = 0; i < EPL; ++i) gi[i] = at == i ? gj : gi[i];
    }
    float m = v[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) m = fmaxf(m, v[i]);
    for (int o = 1; o < a.lanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    float total = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      v[i] = routed ? expf(v[i] - m) : 0.f;
      total += v[i];
      dot += v[i] * gi[i];
    }
    for (int o = 1; o < a.lanes; o <<= 1) {
      total += __shfl_xor_sync(kFull, total, o);
      dot += __shfl_xor_sync(kFull, dot, o);
    }
    const float inv = routed ? 1.f / total : 0.f;
    dot *= inv;
#pragma unroll
    for (int i = 0; i < EPL; ++i) out[i] = v[i] * inv * (gi[i] - dot);
    if (mine) store_scores<T, EPL>(dscores + t * ldd + base, base, a.experts, vec_out != 0, out);
  }
}

// Lanes per token: `per` scores a lane and a lane for each choice, a power of two.
int route_lanes(int experts, int k, int per) {
  int lanes = 1;
  while (lanes < 32 && (lanes * per < experts || lanes < k)) lanes *= 2;
  return lanes;
}

// Scores of a lane: work within a lane is cheaper than between lanes, down to four lanes a token (131072
// x 64, k 4, 16 scores against 8: bf16 25.6 us against 29.7, fp32 33.8 against 37.9; x 128, k 2, fp32 40
// against 48).
int lane_scores(int experts) { return experts > 32 ? 16 : 8; }

// Blocks of the largest cluster that a kernel may ask for (eight without asking: 2048 x 26 7.7 us against
// 6.1, 4096 x 26 in three launches 12.6 against 8.6; both k 4).
constexpr int kClusterTiles = 16;

// Tokens of a tile: small batches are cut finer so that they spread over SMs, those that fit one
// launch over the blocks of one cluster.
int route_tile(int64_t tokens, int experts) {
  if (tokens <= kTileTokens && tokens * experts <= kOneBlockScores) return kTileTokens;
  const int64_t parts = tokens <= kClusterTiles * kTileTokens ? kClusterTiles : num_sms();
  int tile = kTileTokens;
  while (tile > 32 && ceil_div(tokens, tile / 2) <= parts) tile /= 2;
  return tile;
}

size_t route_smem(int experts, int tile) {
  const size_t cells = (size_t)experts * (tile / 32);
  return cells * 4 + align_up(cells, 2) * 2 + (size_t)experts * 12;
}

int check_route(const void* scores, ctr_dtype dtype, int64_t tokens, int32_t experts, int64_t ld, int32_t k) {
  if (!dtype_ok(dtype) || tokens < 0 || experts < 1 || k < 1 || k > experts || ld < experts) return CTR_ERR_INVALID_ARG;
  if (tokens > 0 && !scores) return CTR_ERR_INVALID_ARG;
  if (((uintptr_t)scores % dtype_bytes(dtype)) != 0) return CTR_ERR_INVALID_ARG;
  if (experts > CTR_MAX_EXPERTS || k > CTR_MAX_CHOICES || tokens > INT32_MAX / k) return CTR_ERR_UNSUPPORTED;
  return CTR_OK;
}

std::atomic<int> g_route_cluster{1};  // ctr_set_route_cluster

// Whether the current device can place the kernel's largest cluster, asked once for each device: clusters of more
// than eight blocks are not portable, and a process may be given part of a GPU.
template <auto k>
bool largest_cluster_fits() {
  static std::atomic<uint64_t> asked{0}, fits{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  const uint64_t bit = 1ull << dev;
  if (!(asked.load(std::memory_order_acquire) & bit)) {
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = kClusterTiles;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kClusterTiles);
    cfg.blockDim = dim3(kRouteThreads);
    cfg.dynamicSmemBytes = route_smem(CTR_MAX_EXPERTS, kTileTokens);
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&clusters, k, &cfg) == cudaSuccess && clusters > 0)
      fits.fetch_or(bit, std::memory_order_relaxed);
    else
      cudaGetLastError();  // not a failure of this call
    asked.fetch_or(bit, std::memory_order_release);
  }
  return (fits.load(std::memory_order_relaxed) & bit) != 0;
}

// cluster: whether one is wanted, then whether the launch was one.
template <typename T, int EPL, int KMAX>
bool launch_choose(const RouteArgs& a, size_t smem, bool& cluster, cudaStream_t s) {
  cluster = cluster && largest_cluster_fits<route_choose_kernel<T, EPL, KMAX, true>>();
  auto k = cluster ? route_choose_kernel<T, EPL, KMAX, true> : route_choose_kernel<T, EPL, KMAX, false>;
  return launch_after(k, dim3((unsigned)a.tiles), kRouteThreads, smem, s, cluster ? (unsigned)a.tiles : 1u, a) ==
         cudaSuccess;
}

template <typename T, int EPL>
bool launch_choose(const RouteArgs& a, size_t smem, bool& cluster, cudaStream_t s) {
  return a.k <= 4 ? launch_choose<T, EPL, 4>(a, smem, cluster, s)
                  : launch_choose<T, EPL, CTR_MAX_CHOICES>(a, smem, cluster, s);
}

// Lanes of a token whose softmax is over its choices: one for each, and enough that the row's zeros leave
// in pieces of 64 bytes a lane (131072 rows of 64 bf16, k 1: 2 lanes 12.3 us, one 16.4, 8 16.4; 128 fp32, k
// 2: 8 lanes 22.5, 2 24.6), of 32 where rows are not 16-byte aligned (63 fp32, k 2: 8 lanes 18.4, 4 22.5, 2
// 53).  More than 8 gained nothing (512 bf16, k 4: 8 lanes 36.9, 16 38.9).
int choice_lanes(int row_bytes, int k, int vec_out) {
  return route_lanes((int)imin64(row_bytes, vec_out ? 512 : 256), k, vec_out ? 64 : 32);
}

template <typename T>
void launch_bwd(RouteArgs& a, const float* dweight, T* dscores, int64_t ldd, int vec_out, cudaStream_t s) {
  const int per = lane_scores(a.experts);
  a.lanes = a.renormalize ? choice_lanes(a.experts * (int)sizeof(T), a.k, vec_out) : route_lanes(a.experts, a.k, per);
  auto k = a.renormalize ? route_bwd_choices_kernel<T> : per == 16 ? route_bwd_kernel<T, 16> : route_bwd_kernel<T, 8>;
  const int grid = (int)imin64(ceil_div(a.tokens * a.lanes, kRouteThreads), (int64_t)num_sms() * 8);
  launch_after(k, dim3(grid), kRouteThreads, 0, s, 1, a, dweight, dscores, ldd, vec_out);
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;
// Chunks of a row that a lane holds at once: what it has in flight is what hides the reads' latency.  Rows
// that can only be read in small parts want more of them (65536 x 478 bf16, two rows a token, 4-byte parts:
// dispatch 41 us with 4, 37 with 8, the gradients 80 and 71; 479, 2 bytes: 53 with 4, 45 with 16, and
// 100 and 89).
template <int VB>
constexpr int row_unroll() {
  return VB >= 8 ? 4 : VB == 4 ? 8 : 16;
}
// Sums, where a lane reads two rows at once: 55 us with 4 against 66 with 8, and 76 with 4 against 72 with 16.
template <int VB>
constexpr int sum_unroll() {
  return VB >= 4 ? 4 : 16;
}

struct RowArgs {
  const char* x;     // token rows (dispatch: read; backward: dy)
  const char* rows;  // expert-ordered rows that are read
  char* out;         // dispatch, backward: expert-ordered rows; combine: token rows
  int64_t tokens, total;  // total = tokens * k rows
  int64_t ldx, ldr, ldo;  // bytes
  int32_t k, chunks, lanes;
  const int32_t* slot;
  const int32_t* token;
  const float* weight;
  float* dweight;
  int* err;
};

__device__ __forceinline__ int checked_slot(const RowArgs& a, int64_t i) {
  const int s = a.slot[i];
  if (s >= a.total) {
    set_error(a.err, CTR_ERR_INDEX_OUT_OF_RANGE);
    return -1;
  }
  return s;
}

// Zeros in the rows that no token has: 32 rows to a warp.
template <typename Raw>
__device__ __forceinline__ void zero_unused(const RowArgs& a, const Raw& zero) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kRowThreads / 32);
  for (int64_t r0 = (int64_t)(blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5)) * 32; r0 < a.total;
       r0 += warps * 32) {
    const bool unused = r0 + lane < a.total && a.token[r0 + lane] < 0;
    unsigned todo = __ballot_sync(kFull, unused);
    while (todo) {
      const int b = __ffs(todo) - 1;
      todo &= todo - 1;
      Raw* out = (Raw*)(a.out + (r0 + b) * a.ldo);
      for (int c = lane; c < a.chunks; c += 32) out[c] = zero;
    }
  }
}

// Blocks of an SM (0: the compiler's choice) where the compiler, left alone, takes fewer registers than the
// loads in flight want, or more than leave room for blocks: dispatch of 65536 x 1024 bf16 68.2 us against 66.2
// with five, of 65536 x 479 fp32 71.7 against 70.3, its gradients 119.4 against 115.4 with four, its sums 94 us
// against 83 with six (2048 rows 5.0 against 6.2).
template <int VB>
__global__ void __launch_bounds__(kRowThreads, VB == 2 ? 0 : VB == 8 ? 6 : 5) dispatch_kernel(const RowArgs a) {
  using Raw = typename RawOf<VB>::type;
  constexpr int kUnroll = row_unroll<VB>();
  grid_wait();
  const int sub = threadIdx.x & (a.lanes - 1);
  const int64_t groups = (int64_t)gridDim.x * (kRowThreads / a.lanes);
  for (int64_t t = (blockIdx.x * kRowThreads + threadIdx.x) / (uint32_t)a.lanes; t < a.tokens; t += groups) {
    const Raw* x = (const Raw*)(a.x + t * a.ldx);
    for (int c0 = sub; c0 < a.chunks; c0 += kUnroll * a.lanes) {
      Raw v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (c0 + u * a.lanes < a.chunks) v[u] = __ldcs(x + c0 + u * a.lanes);
      for (int j = 0; j < a.k; ++j) {
        const int s = checked_slot(a, t * a.k + j);
        if (s < 0) continue;
        Raw* out = (Raw*)(a.out + s * a.ldo);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (c0 + u * a.lanes < a.chunks) out[c0 + u * a.lanes] = v[u];
      }
    }
  }
  zero_unused<Raw>(a, Raw{});
}

template <typename T, int VB>
__global__ void __launch_bounds__(kRowThreads, sizeof(T) == 4 && VB == 4 ? 6 : 0) combine_kernel(const RowArgs a) {
  using Ch = Chunk<T, VB>;
  using Raw = typename Ch::Raw;
  constexpr int kUnroll = sum_unroll<VB>();
  grid_wait();
  const int sub = threadIdx.x & (a.lanes - 1);
  const int64_t groups = (int64_t)gridDim.x * (kRowThreads / a.lanes);
  for (int64_t t = (blockIdx.x * kRowThreads + threadIdx.x) / (uint32_t)a.lanes; t < a.tokens; t += groups) {
    Raw* y = (Raw*)(a.out + t * a.ldo);
    for (int c0 = sub; c0 < a.chunks; c0 += kUnroll * a.lanes) {
      float acc[kUnroll][Ch::n];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
#pragma unroll
        for (int i = 0; i < Ch::n; ++i) acc[u][i] = 0.f;
#pragma unroll 1  // two choices at a time: 67.7 us against 66.7 for 65536 x 1024 bf16, k 2
      for (int j = 0; j < a.k; ++j) {
        const int s = checked_slot(a, t * a.k + j);
        if (s < 0) continue;
        const float w = a.weight ? a.weight[t * a.k + j] : 1.f;
        const Raw* r = (const Raw*)(a.rows + s * a.ldr);
        Raw v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (c0 + u * a.lanes < a.chunks) v[u] = __ldcs(r + c0 + u * a.lanes);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (c0 + u * a.lanes < a.chunks) {
            float f[Ch::n];
            Ch::unpack(v[u], f);
#pragma unroll
            for (int i = 0; i < Ch::n; ++i) acc[u][i] = fmaf(w, f[i], acc[u][i]);
          }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (c0 + u * a.lanes < a.chunks) y[c0 + u * a.lanes] = Ch::pack(acc[u]);
    }
  }
}

template <typename T, int VB>
__global__ void __launch_bounds__(kRowThreads, sizeof(T) == 4 && VB < 16 ? 4 : 0) combine_bwd_kernel(const RowArgs a) {
  using Ch = Chunk<T, VB>;
  using Raw = typename Ch::Raw;
  constexpr int kUnroll = row_unroll<VB>();
  grid_wait();
  const int sub = threadIdx.x & (a.lanes - 1);
  const int64_t groups = (int64_t)gridDim.x * (kRowThreads / a.lanes);
  const int64_t trips = ceil_div(a.tokens, groups);  // the same in every lane: the shuffles need all of them
  int64_t t = (blockIdx.x * kRowThreads + threadIdx.x) / (uint32_t)a.lanes;
  for (int64_t trip = 0; trip < trips; ++trip, t += groups) {
    const bool mine = t < a.tokens;
    const Raw* dy = (const Raw*)(a.x + t * a.ldx);
    for (int j = 0; j < a.k; ++j) {
      const int s = mine ? checked_slot(a, t * a.k + j) : -1;
      float dot = 0.f;
      if (s >= 0) {
        const float w = a.weight[t * a.k + j];
        const Raw* r = (const Raw*)(a.rows + s * a.ldr);
        Raw* out = (Raw*)(a.out + s * a.ldo);
        for (int c0 = sub; c0 < a.chunks; c0 += kUnroll * a.lanes) {
          Raw v[kUnroll], g[kUnroll];
#pragma unroll
          for (int u = 0; u < kUnroll; ++u)
            if (c0 + u * a.lanes < a.chunks) {
              v[u] = __ldcs(r + c0 + u * a.lanes);
              g[u] = dy[c0 + u * a.lanes];  // read once per choice: from L1 after the first
            }
#pragma unroll
          for (int u = 0; u < kUnroll; ++u)
            if (c0 + u * a.lanes < a.chunks) {
              float f[Ch::n], d[Ch::n];
              Ch::unpack(v[u], f);
              Ch::unpack(g[u], d);
#pragma unroll
              for (int i = 0; i < Ch::n; ++i) {
                dot = fmaf(d[i], f[i], dot);
                d[i] *= w;
              }
              out[c0 + u * a.lanes] = Ch::pack(d);
            }
        }
      }
      for (int o = 1; o < a.lanes; o <<= 1) dot += __shfl_xor_sync(kFull, dot, o);
      if (mine && sub == 0) a.dweight[t * a.k + j] = dot;
    }
  }
  zero_unused<Raw>(a, Raw{});
}

int check_rows(ctr_dtype dtype, int64_t tokens, int32_t d, int32_t k, void* ws, size_t ws_bytes) {
  if (!dtype_ok(dtype) || tokens < 0 || d < 1 || k < 1) return CTR_ERR_INVALID_ARG;
  if (k > CTR_MAX_CHOICES || tokens > INT32_MAX / k) return CTR_ERR_UNSUPPORTED;
  if (!ws_valid(ws, ws_bytes, kWsHeader)) return CTR_ERR_WORKSPACE;
  return CTR_OK;
}

// Chunk count, lanes per row and grid of a row kernel.  A row gets as few lanes as hold it at once,
// unless too few threads had one (65536 rows of 256 bf16, two rows a token, 8 lanes against 32: dispatch
// 20 us against 25, combine 25 against 49, its gradients 37 against 72; 20000 rows of 480, 16 lanes
// against 32, combine 18 against 25; 5000 rows of 256, 16 lanes: 8.2 against 10.2).
int plan_rows(RowArgs* a, int64_t row_bytes, int vb) {
  a->chunks = (int32_t)(row_bytes / vb);
  const int unroll = vb >= 8 ? row_unroll<8>() : vb == 4 ? row_unroll<4>() : row_unroll<2>();
  a->lanes = 1;
  while (a->lanes < 32 && a->lanes < a->chunks &&
         (a->lanes * unroll < a->chunks || a->tokens * a->lanes < (int64_t)num_sms() * 512))
    a->lanes *= 2;
  const int64_t blocks = ceil_div(a->tokens * a->lanes, kRowThreads);
  return (int)imax64(1, imin64(blocks, (int64_t)num_sms() * 16));
}

#define CTR_LAUNCH_TYPED(kernel, dtype, vb, grid, stream, args)                                       \
  do {                                                                                                \
    auto k = kernel<float, 4>;                                                                        \
    if ((dtype) == CTR_F32) k = (vb) == 16 ? kernel<float, 16> : (vb) == 8 ? kernel<float, 8> : k;    \
    else k = (vb) == 16 ? kernel<__nv_bfloat16, 16> : (vb) == 8 ? kernel<__nv_bfloat16, 8>            \
             : (vb) == 4 ? kernel<__nv_bfloat16, 4> : kernel<__nv_bfloat16, 2>;                       \
    launch_after(k, dim3(grid), kRowThreads, 0, stream, 1, args);                                     \
  } while (0)

}  // namespace
}  // namespace ctr

using namespace ctr;

extern "C" size_t ctr_expert_workspace_size(void) { return kWsHeader; }

extern "C" size_t ctr_expert_route_workspace_size(int64_t tokens, int32_t experts, int32_t k) {
  if (tokens < 0 || experts < 1 || k < 1) return 0;
  WsSizer z;
  z.take<int32_t>((size_t)(ceil_div(tokens, 32) + 1) * experts);  // tiles hold at least 32 tokens
  return z.used;
}

extern "C" int ctr_set_route_cluster(int on) { return g_route_cluster.exchange(on ? 1 : 0); }

extern "C" int ctr_expert_route(const void* scores, ctr_dtype dtype, int64_t tokens, int32_t experts,
                                int64_t ld_scores, int32_t k, int renormalize, int32_t* expert, float* weight,
                                int32_t* slot, int32_t* token, int32_t* offsets, void* ws, size_t ws_bytes,
                                ctr_stream_t stream) {
  const int st = check_route(scores, dtype, tokens, experts, ld_scores, k);
  if (st != CTR_OK) return st;
  if (!offsets || (tokens > 0 && (!expert || !weight || !slot || !token))) return CTR_ERR_INVALID_ARG;
  if (!ws_valid(ws, ws_bytes, ctr_expert_route_workspace_size(tokens, experts, k))) return CTR_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  if (tokens == 0) {
    launch_after(route_empty_kernel, dim3(1), 128, 0, s, 1, offsets, experts);
    return launch_status();
  }
  RouteArgs a = {};
  a.scores = scores;
  a.tokens = tokens;
  a.ld = ld_scores;
  a.experts = experts;
  a.k = k;
  const int per = lane_scores(experts);
  a.lanes = route_lanes(experts, k, per);
  a.tile = route_tile(tokens, experts);
  a.tiles = (int32_t)ceil_div(tokens, a.tile);
  a.renormalize = renormalize != 0;
  const int eb = dtype_bytes(dtype);
  a.vec = ((uintptr_t)scores % 16) == 0 && (ld_scores * eb) % 16 == 0;
  a.expert = expert;
  a.weight = weight;
  a.slot = slot;
  a.token = token;
  a.offsets = offsets;
  WsCarver c(ws, ws_bytes);
  a.counts = c.take<int32_t>((size_t)(a.tiles + 1) * experts);
  a.err = (int*)ws;
  const size_t smem = route_smem(experts, a.tile);
  bool cluster = a.tiles > 1 && a.tiles <= kClusterTiles && g_route_cluster.load(std::memory_order_relaxed) != 0;
  const bool ok = dtype == CTR_F32 ? (per == 8 ? launch_choose<float, 8>(a, smem, cluster, s)
                                               : launch_choose<float, 16>(a, smem, cluster, s))
                                   : (per == 8 ? launch_choose<__nv_bfloat16, 8>(a, smem, cluster, s)
                                               : launch_choose<__nv_bfloat16, 16>(a, smem, cluster, s));
  if (!ok) return CTR_ERR_CUDA;
  if (a.tiles > 1 && !cluster) {
    launch_after(route_scan_kernel, dim3((unsigned)ceil_div(experts, 32)), 1024, 0, s, 1, a);
    launch_after(route_rank_kernel, dim3((unsigned)a.tiles), kRouteThreads, smem, s, 1, a);
  }
  return launch_status();
}

extern "C" int ctr_expert_route_bwd(const float* dweight, const void* scores, ctr_dtype dtype, int64_t tokens,
                                    int32_t experts, int64_t ld_scores, int32_t k, int renormalize,
                                    const int32_t* expert, void* dscores, int64_t ld_dscores, void* ws,
                                    size_t ws_bytes, ctr_stream_t stream) {
  const int st = check_route(scores, dtype, tokens, experts, ld_scores, k);
  if (st != CTR_OK) return st;
  if (ld_dscores < experts || (tokens > 0 && (!dweight || !expert || !dscores))) return CTR_ERR_INVALID_ARG;
  if (((uintptr_t)dscores % dtype_bytes(dtype)) != 0) return CTR_ERR_INVALID_ARG;
  if (!ws_valid(ws, ws_bytes, kWsHeader)) return CTR_ERR_WORKSPACE;
  if (tokens == 0) return CTR_OK;
  RouteArgs a = {};
  a.scores = scores;
  a.tokens = tokens;
  a.ld = ld_scores;
  a.experts = experts;
  a.k = k;
  a.renormalize = renormalize != 0;
  const int eb = dtype_bytes(dtype);
  a.vec = ((uintptr_t)scores % 16) == 0 && (ld_scores * eb) % 16 == 0;
  const int vec_out = ((uintptr_t)dscores % 16) == 0 && (ld_dscores * eb) % 16 == 0;
  a.expert = const_cast<int32_t*>(expert);
  a.err = (int*)ws;
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == CTR_F32) launch_bwd(a, dweight, (float*)dscores, ld_dscores, vec_out, s);
  else launch_bwd(a, dweight, (__nv_bfloat16*)dscores, ld_dscores, vec_out, s);
  return launch_status();
}

extern "C" int ctr_expert_dispatch(const void* x, ctr_dtype dtype, int64_t tokens, int32_t d, int64_t ldx, int32_t k,
                                   const int32_t* slot, const int32_t* token, void* out, int64_t ldo, void* ws,
                                   size_t ws_bytes, ctr_stream_t stream) {
  const int st = check_rows(dtype, tokens, d, k, ws, ws_bytes);
  if (st != CTR_OK) return st;
  if (ldx < d || ldo < d) return CTR_ERR_INVALID_ARG;
  if (tokens == 0) return CTR_OK;
  const int eb = dtype_bytes(dtype);
  if (!x || !slot || !token || !out || ((uintptr_t)x % eb) || ((uintptr_t)out % eb)) return CTR_ERR_INVALID_ARG;
  RowArgs a = {};
  a.x = (const char*)x;
  a.out = (char*)out;
  a.tokens = tokens;
  a.total = tokens * k;
  a.ldx = ldx * eb;
  a.ldo = ldo * eb;
  a.k = k;
  a.slot = slot;
  a.token = token;
  a.err = (int*)ws;
  const int64_t row = (int64_t)d * eb;
  const int vb = vector_bytes({(uint64_t)(uintptr_t)x, (uint64_t)(uintptr_t)out, (uint64_t)a.ldx, (uint64_t)a.ldo,
                               (uint64_t)row}, eb);
  const int grid = plan_rows(&a, row, vb);
  cudaStream_t s = (cudaStream_t)stream;
  if (vb == 16) launch_after(dispatch_kernel<16>, dim3(grid), kRowThreads, 0, s, 1, a);
  else if (vb == 8) launch_after(dispatch_kernel<8>, dim3(grid), kRowThreads, 0, s, 1, a);
  else if (vb == 4) launch_after(dispatch_kernel<4>, dim3(grid), kRowThreads, 0, s, 1, a);
  else launch_after(dispatch_kernel<2>, dim3(grid), kRowThreads, 0, s, 1, a);
  return launch_status();
}

extern "C" int ctr_expert_combine(const void* rows, ctr_dtype dtype, int64_t tokens, int32_t d, int64_t ld_rows,
                                  int32_t k, const int32_t* slot, const float* weight, void* y, int64_t ldy, void* ws,
                                  size_t ws_bytes, ctr_stream_t stream) {
  const int st = check_rows(dtype, tokens, d, k, ws, ws_bytes);
  if (st != CTR_OK) return st;
  if (ld_rows < d || ldy < d) return CTR_ERR_INVALID_ARG;
  if (tokens == 0) return CTR_OK;
  const int eb = dtype_bytes(dtype);
  if (!rows || !slot || !y || ((uintptr_t)rows % eb) || ((uintptr_t)y % eb)) return CTR_ERR_INVALID_ARG;
  RowArgs a = {};
  a.rows = (const char*)rows;
  a.out = (char*)y;
  a.tokens = tokens;
  a.total = tokens * k;
  a.ldr = ld_rows * eb;
  a.ldo = ldy * eb;
  a.k = k;
  a.slot = slot;
  a.weight = weight;
  a.err = (int*)ws;
  const int64_t row = (int64_t)d * eb;
  const int vb = vector_bytes({(uint64_t)(uintptr_t)rows, (uint64_t)(uintptr_t)y, (uint64_t)a.ldr, (uint64_t)a.ldo,
                               (uint64_t)row}, eb);
  const int grid = plan_rows(&a, row, vb);
  cudaStream_t s = (cudaStream_t)stream;
  CTR_LAUNCH_TYPED(combine_kernel, dtype, vb, grid, s, a);
  return launch_status();
}

extern "C" int ctr_expert_combine_bwd(const void* dy, ctr_dtype dtype, int64_t tokens, int32_t d, int64_t ld_dy,
                                      int32_t k, const void* rows, int64_t ld_rows, const int32_t* slot,
                                      const float* weight, const int32_t* token, void* drows, int64_t ld_drows,
                                      float* dweight, void* ws, size_t ws_bytes, ctr_stream_t stream) {
  const int st = check_rows(dtype, tokens, d, k, ws, ws_bytes);
  if (st != CTR_OK) return st;
  if (ld_dy < d || ld_rows < d || ld_drows < d) return CTR_ERR_INVALID_ARG;
  if (tokens == 0) return CTR_OK;
  const int eb = dtype_bytes(dtype);
  if (!dy || !rows || !slot || !weight || !token || !drows || !dweight) return CTR_ERR_INVALID_ARG;
  if (((uintptr_t)dy % eb) || ((uintptr_t)rows % eb) || ((uintptr_t)drows % eb)) return CTR_ERR_INVALID_ARG;
  RowArgs a = {};
  a.x = (const char*)dy;
  a.rows = (const char*)rows;
  a.out = (char*)drows;
  a.tokens = tokens;
  a.total = tokens * k;
  a.ldx = ld_dy * eb;
  a.ldr = ld_rows * eb;
  a.ldo = ld_drows * eb;
  a.k = k;
  a.slot = slot;
  a.token = token;
  a.weight = weight;
  a.dweight = dweight;
  a.err = (int*)ws;
  const int64_t row = (int64_t)d * eb;
  const int vb = vector_bytes({(uint64_t)(uintptr_t)dy, (uint64_t)(uintptr_t)rows, (uint64_t)(uintptr_t)drows,
                               (uint64_t)a.ldx, (uint64_t)a.ldr, (uint64_t)a.ldo, (uint64_t)row}, eb);
  const int grid = plan_rows(&a, row, vb);
  cudaStream_t s = (cudaStream_t)stream;
  CTR_LAUNCH_TYPED(combine_bwd_kernel, dtype, vb, grid, s, a);
  return launch_status();
}
