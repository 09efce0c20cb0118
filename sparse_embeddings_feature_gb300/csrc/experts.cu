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
  float factor;                            // of the weights
  // balanced routing
  const float* bias;                       // NULL without
  int32_t sigmoid, groups, group_k, seg;   // seg: lanes of a group of experts, 0 where groups end inside lanes
  int32_t f32, cluster;                    // type of the scores; whether the launch is one cluster
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

// What a choice's weight is in proportion to, by its score s and the choices' largest score m.  Sigmoids' proportions are taken
// less e^m where m is negative: the sigmoids themselves may be below fp32's numbers, the weights are not.
__device__ __forceinline__ float choice_value(const RouteArgs& a, float s, float m) {
  if (!a.sigmoid) return expf(s - m);
  const float r = 1.f / (1.f + expf(-fabsf(s)));
  return s > 0.f ? r : expf(s - (a.renormalize ? fminf(m, 0.f) : 0.f)) * r;
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

// The order of a tile whose choices are in `bits`: its counts for the scan, or, where all tiles are this block's or
// this cluster's, its choices' rows.
template <bool CLUSTER>
__device__ __forceinline__ void finish_tile(const RouteArgs& a, int64_t t0, int n, uint32_t* bits) {
  const int words = a.tile / 32;
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
  finish_tile<CLUSTER>(a, t0, n, bits);
}

// ---------------------------------------------------------------------------
// Balanced routing: keys (score function + bias), groups, weights from the score function
// ---------------------------------------------------------------------------
// Keys are compared to 64 bits' precision.  All of them are computed in fp32 and packed: 23 bits of the keys' range above
// the complement of the expert's index (without a bias, choices go by the upper 23 bits of the scores, made to order as
// unsigned numbers), so that integer maxima and minima find keys and lowest indexes together: a lane sorts its keys
// (Batcher's odd-even merge sort), a round a choice takes the largest of the lanes' first ones.  Where two that have to be
// told apart are nearer than the bound on what packed keys may be off by (one token in 500; equal scores with equal
// biases are ties and told apart by their indexes), the warp does its tokens again, with the keys that matter in 64 bits: a
// group's two best, and as many choices as there are lanes.  Where that is not enough (another key that may be larger than
// those and is not their equal), all keys in 64 bits, of which a warp's instruction takes 64 cycles (all tokens of 65536 x
// 256 so: 3.1 ms).
// 65536 x 256, k 8, 4 of 8 groups, all tokens in fp32 with a round a choice for the key and one for its index: 196 us.
// e^x in 64 bits for x from -700 to 709.7 (beyond, as at the ends): 2^(j / 64) from a table, the rest, below ln 2 / 128, by five
// terms of the series: a third of the 64-bit instructions of exp, which a warp is bound by.
__device__ const double kPowers[64] = {
    1.0, 1.0108892860517005, 1.0218971486541166, 1.0330248790212284,
    1.0442737824274138, 1.0556451783605572, 1.0671404006768237, 1.0787607977571199,
    1.0905077326652577, 1.102382583307841, 1.1143867425958924, 1.1265216186082418,
    1.1387886347566916, 1.1511892299529827, 1.1637248587775775, 1.1763969916502812,
    1.189207115002721, 1.202156731452703, 1.215247359980469, 1.22848053610687,
    1.241857812073484, 1.255380757024691, 1.2690509571917332, 1.2828700160787783,
    1.2968395546510096, 1.3109612115247644, 1.3252366431597413, 1.339667524053303,
    1.3542555469368927, 1.3690024229745905, 1.383909881963832, 1.3989796725383112,
    1.4142135623730951, 1.42961333839197, 1.4451808069770467, 1.460917794180647,
    1.4768261459394993, 1.4929077282912648, 1.5091644275934228, 1.5255981507445384,
    1.5422108254079407, 1.559004400237837, 1.5759808451078865, 1.593142151342267,
    1.6104903319492543, 1.6280274218573478, 1.645755478153965, 1.6636765803267364,
    1.681792830507429, 1.7001063537185235, 1.718619298122478, 1.7373338352737062,
    1.7562521603732995, 1.7753764925265212, 1.7947090750031072, 1.8142521755003989,
    1.8340080864093424, 1.8539791250833855, 1.8741676341103, 1.8945759815869656,
    1.9152065613971474, 1.9360617934922943, 1.9571441241754002, 1.978456026387951};
__device__ __forceinline__ double exp_64(double x) {
  x = fmin(fmax(x, -700.0), 709.7);
  const double shifted = x * 92.33248261689366 + 0x1.8p52;  // the nearest whole number of 64ths of ln 2, in the low bits
  const int n = __double2loint(shifted);
  const double k = shifted - 0x1.8p52;
  double r = fma(k, -0.01083042468962958, x);  // the first factor has 31 bits: its product is exact
  r = fma(k, -6.619564634077006e-12, r);
  double p = fma(r, 1.0 / 120, 1.0 / 24);
  p = fma(p, r, 1.0 / 6);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0) * r;
  const double t = kPowers[n & 63];
  const double y = fma(t, p, t);
  return __hiloint2double(__double2hiint(y) + ((n >> 6) << 20), __double2loint(y));
}
// The same down to 64 bits' smallest numbers, below which it is 0.
__device__ __forceinline__ double exp_64_down(double x) {
  return x < -700.0 ? exp_64(x + 700.0) * 9.85967654375977e-305 : exp_64(x);  // e^-700
}
// 1 / (1 + e^-x); where 64 bits hold no difference, e^x, which has a value longer.
__device__ __forceinline__ double sigmoid_64(double x) { return x < -40.0 ? exp_64_down(x) : 1 / (1 + exp_64(-x)); }

template <typename K>
__device__ __forceinline__ K exp_of(K x);
template <>
__device__ __forceinline__ float exp_of<float>(float x) {
  return expf(x);
}
template <>
__device__ __forceinline__ double exp_of<double>(double x) {
  return x > -700.0 ? exp_64(x) : 0.0;  // nothing beside a sum of 1 and more
}

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A softmax's shift and sum over a row, from a lane's scores (-inf: masked).
template <typename K, int EPL>
__device__ __forceinline__ K row_softmax(const float (&v)[EPL], int lanes, float& m) {
  m = v[0];
#pragma unroll
  for (int i = 1; i < EPL; ++i) m = fmaxf(m, v[i]);
  for (int o = 1; o < lanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  if (!(m > -INFINITY)) m = 0.f;
  K total = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) total += exp_of<K>((K)v[i] - (K)m);
  for (int o = 1; o < lanes; o <<= 1) total += __shfl_xor_sync(kFull, total, o);
  return total;
}

// The expert of choice `sub` of the lanes' token, -1: none, with all keys in 64 bits.  v: the lane's scores (-inf: masked,
// all of them for a token that is routed nowhere); b: its experts' biases.
template <int EPL>
__device__ __forceinline__ int choose_exact(const RouteArgs& a, const float (&v)[EPL], const float (&b)[EPL], int sub) {
  const double none = -INFINITY;
  const int base = sub * EPL, per = a.experts / a.groups;
  float m = 0.f;
  double total = 1, key[EPL];
  if (!a.sigmoid) total = row_softmax<double, EPL>(v, a.lanes, m);
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const double p = a.sigmoid ? sigmoid_64(v[i]) : exp_64_down((double)v[i] - m) / total;
    key[i] = v[i] > -INFINITY && b[i] > -INFINITY ? p + b[i] : none;
  }
  auto take = [](double& x0, double& x1, double x) {
    x1 = fmax(x1, fmin(x0, x));
    x0 = fmax(x0, x);
  };
  if (a.group_k < a.groups) {
    double worth = none;  // lane g: of group g
    for (int g = 0; g < a.groups; ++g) {
      double x0 = none, x1 = none;
#pragma unroll
      for (int i = 0; i < EPL; ++i) take(x0, x1, base + i >= g * per && base + i < (g + 1) * per ? key[i] : none);
      for (int o = 1; o < a.lanes; o <<= 1) {
        const double y0 = __shfl_xor_sync(kFull, x0, o), y1 = __shfl_xor_sync(kFull, x1, o);
        take(x0, x1, y0);
        take(x0, x1, y1);
      }
      if (g == sub) worth = x1 > none ? x0 + x1 : x0;
    }
    int place = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double other = __shfl_sync(kFull, worth, g, a.lanes);
      place += other > worth || (other == worth && g < sub);
    }
    const int lane = threadIdx.x & 31;
    const uint32_t kept = __ballot_sync(kFull, worth > none && place < a.group_k) >> (lane & ~(a.lanes - 1));
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (base + i < a.experts && !((kept >> ((base + i) / per)) & 1)) key[i] = none;
  }
  if (!a.bias) {  // the scores are in the keys' order, without rounding
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = key[i] > none ? (double)v[i] : none;
  }
  int expert = -1;
  for (int j = 0; j < a.k; ++j) {
    double best = key[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) best = fmax(best, key[i]);
    for (int o = 1; o < a.lanes; o <<= 1) best = fmax(best, __shfl_xor_sync(kFull, best, o));
    int at = 0x7fffffff;
#pragma unroll
    for (int i = EPL - 1; i >= 0; --i) at = key[i] == best ? base + i : at;
    for (int o = 1; o < a.lanes; o <<= 1) at = min(at, __shfl_xor_sync(kFull, at, o));
    if (best > none && j == sub) expert = at;
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = base + i == at ? none : key[i];
  }
  return expert;
}

// Scores of a row in either type.
template <int EPL>
__device__ __forceinline__ void load_scores(const RouteArgs& a, int64_t t, int base, float (&v)[EPL]) {
  if (a.f32) load_scores<float, EPL>((const float*)a.scores + t * a.ld, base, a.experts, a.vec != 0, v);
  else load_scores<__nv_bfloat16, EPL>((const __nv_bfloat16*)a.scores + t * a.ld, base, a.experts, a.vec != 0, v);
}
__device__ __forceinline__ float score_at(const RouteArgs& a, int64_t t, int e) {
  return a.f32 ? ((const float*)a.scores)[t * a.ld + e] : to_f32(((const __nv_bfloat16*)a.scores)[t * a.ld + e]);
}

// A number as an integer in the same order (64-bit comparisons of integers are not slow); -0 as +0.
__device__ __forceinline__ int64_t in_order(double x) {
  const int64_t b = __double_as_longlong(x + 0.0);
  return b ^ ((b >> 63) & INT64_MAX);
}

// Whether two packed keys are of equal scores with equal biases.
__device__ __noinline__ bool same_inputs(const RouteArgs& a, int64_t t, uint32_t x, uint32_t y) {
  const int e = 511 - (int)(x & 511u), f = 511 - (int)(y & 511u);
  return score_at(a, t, e) == score_at(a, t, f) && (!a.bias || a.bias[e] == a.bias[f]);
}

// Falling order, by Batcher's odd-even merge sort (Sorting networks and their applications, 1968).
template <int N>
__device__ __forceinline__ void sort_falling(uint32_t (&x)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t hi = max(x[i + j], x[i + j + k]);
            x[i + j + k] = min(x[i + j], x[i + j + k]);
            x[i + j] = hi;
          }
}

template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t x) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) x = max(x, __shfl_xor_sync(kFull, x, o));
  return x;
}

// Packed keys: the keys' range from the smallest bias on is cut into kParts parts of 1 / scale, numbered from 1.
// What a key may be off by besides p's own error, in parts (2^-24 of a range is half a part): three roundings of the
// bias's part number and one of the sum, half a part each, and one part for cutting off.
// Biases further apart than kSpread (experts pushed out by -1e9, or lifted, say) would make the parts as coarse as that is.
// Their gaps of more than kGap are closed to that: p is at most 1, so keys on either side of such a gap keep their order, and
// by more parts than a comparison asks for; keys with no such gap between them keep their distance (65536 x 256 bf16, k 8, 4 of
// 8 groups, sigmoids and softmax: biases of 0.05 96 and 125 us, a tenth of them -1e9 109 and 142, one of them +10 108 and
// 156; in parts of the whole range -1e9 takes 3.1 ms, +10 106 and 234).  Closing takes a block 1.7 us, so biases spread by less
// are left as they are.
struct Packing {
  float scale;
  bool cut;         // whether gaps have been closed
  bool top_coarse;  // the largest bias is past kLarge
  static constexpr float off = 3.f;
};
struct PackedBias {            // shared
  float at[CTR_MAX_EXPERTS];   // each expert's part number at p = 0; -inf: never chosen
  float lift[CTR_MAX_EXPERTS]; // where gaps have been closed: a key less the largest bias's, in parts, less the same of part numbers
  int low, high;               // keys of smaller parts, and of these and larger ones, have biases past kLarge
};
constexpr float kParts = 8388592.f;  // a few below 2^23, which p may pass 1 by
constexpr float kSpread = 6.f;
constexpr float kGap = 1.0625f;
constexpr float kLarge = 1073741824.f;  // 2^30: past it a 64-bit key's last bit is more than a part
static_assert(CTR_MAX_EXPERTS <= 512, "an index has 9 bits");

// `to` of biases b whose gaps are closed; some: whether the thread's expert may be chosen.  Distances are added up as whole
// numbers of 2^-40: what a distance is off by are the gaps' own roundings, 2^-24 of it (in 64-bit numbers the same took 7 us).
__device__ __noinline__ Packing pack_apart(PackedBias& to, int experts, float b, bool some) {
  __shared__ int64_t sums[kRouteThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = threadIdx.x;
  if (e < experts) to.at[e] = some ? b : INFINITY;
  const int n = __syncthreads_count(some);
  int rank = 0;  // by bias, then index
  if (some) {
#pragma unroll 8
    for (int j = 0; j < experts; ++j) rank += to.at[j] < b || (to.at[j] == b && j < e);
    to.lift[rank] = b;
  }
  __syncthreads();
  // thread r: the r-th smallest, its distance from the smallest with the gaps closed
  const int r = e;
  const float mine = r < n ? to.lift[r] : 0.f, before = r > 0 && r < n ? to.lift[r - 1] : mine, top = to.lift[n - 1];
  const bool cut = __syncthreads_or(mine - before > kGap);  // and the next write to `lift` comes after all reads
  int64_t c = (int64_t)(fminf(mine - before, kGap) * 0x1p40f);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(kFull, c, o);
    if (lane >= o) c += y;
  }
  if (lane == 31) sums[warp] = c;
  if (e == 0) to.low = to.high = 1 << 23;
  __syncthreads();
  int64_t all = 0;
#pragma unroll
  for (int w = 0; w < kRouteThreads / 32; ++w) {
    if (w < warp) c += sums[w];
    all += sums[w];
  }
  const float scale = kParts / (1.f + (float)all * 0x1p-40f);
  const float at = fmaf((float)c * 0x1p-40f, scale, 1.f), lift = ((mine - top) + (float)(all - c) * 0x1p-40f) * scale;
  if (r < n) {
    to.at[r] = at;
    to.lift[r] = lift;
    if (mine > -kLarge && (r == 0 || before <= -kLarge)) to.low = (int)at;
    if (mine >= kLarge && (r == 0 || before < kLarge)) to.high = (int)at;
  }
  __syncthreads();
  const float my_at = some ? to.at[rank] : -INFINITY, my_lift = some ? to.lift[rank] : 0.f;
  __syncthreads();
  to.at[e] = my_at;
  to.lift[e] = my_lift;
  return {scale, cut, fabsf(top) >= kLarge};
}
static_assert(kRouteThreads == CTR_MAX_EXPERTS, "a rank, and an expert, to a thread");

// `to` filled by all threads of the block.
__device__ __forceinline__ Packing pack_range(const RouteArgs& a, PackedBias& to, float* ends) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = threadIdx.x;
  float b = a.bias && e < a.experts ? a.bias[e] : 0.f;
  if (!(b < INFINITY)) {  // NaN, +inf: as -inf, and flagged
    b = -INFINITY;
    set_error(a.err, CTR_ERR_BAD_VALUE);
  }
  const bool some = e < a.experts && b > -INFINITY;
  float lo = some ? b : INFINITY, hi = some ? b : -INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
  }
  if (lane == 0) {
    ends[2 * warp] = lo;
    ends[2 * warp + 1] = hi;
  }
  __syncthreads();
  for (int w = 0; w < kRouteThreads / 32; ++w) {
    lo = fminf(lo, ends[2 * w]);
    hi = fmaxf(hi, ends[2 * w + 1]);
  }
  if (!(lo <= hi)) lo = hi = 0.f;
  Packing pack = {kParts / (1.f + (hi - lo)), false, fabsf(hi) >= kLarge};
  if (hi - lo > kSpread) {  // the same in all threads
    pack = pack_apart(to, a.experts, b, some);
  } else {
    to.at[e] = some ? fmaf(b - lo, pack.scale, 1.f) : -INFINITY;
    if (e == 0) {
      to.low = pack.top_coarse ? 1 << 23 : 0;
      to.high = 1 << 23;
    }
  }
  __syncthreads();
  return pack;
}

// The expert of choice `sub` of the lanes' token t, -1: none; near: this could not tell.  KMAX: choices at most.  REFINE:
// the keys that matter are computed in 64 bits.
template <int EPL, int KMAX, int LANES, bool REFINE>
__device__ __forceinline__ int choose_packed(const RouteArgs& a, const float (&v)[EPL], const PackedBias& bias, const Packing& pack,
                                             int64_t t, int sub, float shift, float total, bool& near) {
  constexpr float kLog2e = 1.44269504f;
  const int base = sub * EPL, per = a.experts / a.groups;
  const bool plain = !a.bias, grouped = a.group_k < a.groups;
  const int lane = threadIdx.x & 31, first = lane & ~(LANES - 1);
  near = false;
  uint32_t key[EPL];
  int apart;  // keys whose parts are no further apart have to be told apart
  uint32_t kept = kFull;
  double sum = 1;  // of a softmax, in 64 bits
  if (REFINE && !a.sigmoid && (!plain || grouped)) sum = row_softmax<double, EPL>(v, LANES, shift);
  auto exact = [&](uint32_t x) {  // a packed key's value in 64 bits
    const int e = 511 - (int)(x & 511u);
    const double l = score_at(a, t, e), b = a.bias ? a.bias[e] : 0.f;
    return (a.sigmoid ? sigmoid_64(l) : exp_64_down(l - shift) / sum) + b;
  };
  if (plain) {
    // scores of one upper part differ in what was cut off, but for bf16 ones, which have nothing there
    apart = a.f32 ? 0 : -1;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      uint32_t u = __float_as_uint(v[i] + 0.f);  // -0 becomes +0
      u ^= (uint32_t)((int32_t)u >> 31) | 0x80000000u;
      key[i] = v[i] > -INFINITY ? (u & 0xfffffe00u) | (uint32_t)(511 - base - i) : 0u;
    }
  } else {
    // p's error in parts (two of 2^-24), sigmoid: exponential 4 of 2^-24 and its argument's rounding, sum, reciprocal 4:
    // 8; softmax, of its largest p: exponential 4, its argument's rounding 1, a sum of 16 + 5 additions of such terms and
    // its division, product: 33
    const float times = 1.f / total;
    apart = 1 + (int)fminf(2.f * (Packing::off + (a.sigmoid ? 4.f : 17.f * times)), 1e8f);
    auto part = [&](int i, float p) {
      // -inf, of a bias, becomes 0: no key
      const uint32_t q = (uint32_t)fmaf(p, pack.scale, bias.at[base + i]);
      key[i] = v[i] > -INFINITY && q > 0 ? q * 512u + (uint32_t)(511 - base - i) : 0u;
    };
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) part(i, __fdividef(1.f, 1.f + exp2_fast(-v[i] * kLog2e)));
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) part(i, exp2_fast((v[i] - shift) * kLog2e) * times);
    }
  }
  const int low = plain ? 0 : bias.low, high = plain ? 1 << 23 : bias.high;
  auto nearby = [&](uint32_t x, uint32_t y) {  // whether y, the smaller packed key, may be the larger one
    return y != 0 && ((int)((x >> 9) - (y >> 9)) <= apart || (int)(x >> 9) < low || (int)(y >> 9) >= high);
  };
  auto unclear = [&](uint32_t x, uint32_t y) { return nearby(x, y) && !same_inputs(a, t, x, y); };
  if (grouped) {
    uint32_t k0 = 0, k1 = 0, k2 = 0;  // lane g learns group g's two (REFINE: three) best keys
    auto take = [](uint32_t& x0, uint32_t& x1, uint32_t& x2, uint32_t x) {
      const uint32_t y = min(x0, x);
      x0 = max(x0, x);
      if (REFINE) x2 = max(x2, min(x1, y));
      x1 = max(x1, y);
    };
    auto join = [&](uint32_t& x0, uint32_t& x1, uint32_t& x2, int o) {
      const uint32_t y0 = __shfl_xor_sync(kFull, x0, o), y1 = __shfl_xor_sync(kFull, x1, o);
      const uint32_t y2 = REFINE ? __shfl_xor_sync(kFull, x2, o) : 0;
      take(x0, x1, x2, y0);
      take(x0, x1, x2, y1);
      if (REFINE) take(x0, x1, x2, y2);
    };
    if (a.seg) {
      uint32_t x0 = 0, x1 = 0, x2 = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) take(x0, x1, x2, key[i]);
      for (int o = 1; o < a.seg; o <<= 1) join(x0, x1, x2, o);
      k0 = __shfl_sync(kFull, x0, sub * a.seg, LANES);
      k1 = __shfl_sync(kFull, x1, sub * a.seg, LANES);
      if (REFINE) k2 = __shfl_sync(kFull, x2, sub * a.seg, LANES);
    } else {
      for (int g = 0; g < a.groups; ++g) {
        uint32_t x0 = 0, x1 = 0, x2 = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) take(x0, x1, x2, base + i >= g * per && base + i < (g + 1) * per ? key[i] : 0u);
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) join(x0, x1, x2, o);
        if (g == sub) {
          k0 = x0;
          k1 = x1;
          k2 = x2;
        }
      }
    }
    const bool some = sub < a.groups && k0 != 0;
    int place = 0;
    bool close = false;
    // near: on either side of the border; equal pairs are ties where packed keys are exact, so that the pairs are the best
    if (!plain) {
      // In parts; where gaps have been closed, what they hid is added again (a sum past fp32's range is below all others).  A
      // lift is off by 3 of 2^-24 of itself and a part, two of them and the parts' sum by one more each: two groups' worths by
      // 10 of 2^-24 of the larger one's lifts, which are within 2^24 parts of it, and 4 parts.
      float worth = some ? (float)((k0 >> 9) + (k1 >> 9)) : -INFINITY;
      float least = 2.f * (float)apart, rel = 0.f;
      if (pack.cut) {
        least += 32.f;
        rel = 0x1p-20f;
        if (some)
          worth = fmaxf(worth + (bias.lift[511 - (k0 & 511u)] + (k1 ? bias.lift[511 - (k1 & 511u)] : 0.f)), -3e38f);
      }
      auto apart_from = [&](float other) {  // a group without keys from any other
        return fabsf(worth - other) > fmaf(rel, fmaxf(fabsf(worth), fabsf(other)), least) || other == -INFINITY;
      };
      float gap = INFINITY;  // to the nearest other group
      for (int g = 0; g < a.groups; ++g) {
        const float other = __shfl_sync(kFull, worth, g, LANES);
        place += other > worth || (other == worth && g < sub);
        if (g != sub) gap = fminf(gap, fabsf(worth - other));
      }
      const bool tight = gap <= fmaf(rel, fabsf(worth) + gap, least);  // or no other one can be near
      // a sum of one key is not to be compared with one of two in parts
      const uint32_t all = LANES == 32 ? kFull : (1u << (LANES & 31)) - 1;
      const uint32_t ones = __ballot_sync(kFull, some && k1 == 0) >> first & all;
      const uint32_t twos = __ballot_sync(kFull, some && k1 != 0) >> first & all;
      close = (ones != 0 && twos != 0) || (some && pack.top_coarse);
      if (__any_sync(kFull, some && tight)) {
        for (int g = 0; g < a.groups; ++g) {
          const float other = __shfl_sync(kFull, worth, g, LANES);
          const int there = __shfl_sync(kFull, place, g, LANES);
          close |= some && (place < a.group_k) != (there < a.group_k) && !apart_from(other);
        }
      }
    } else {
      // What a group is worth, from the scores, as a number whose error is relative, so that the small sums of peaked scores
      // are told apart too: a softmax's p0 + p1; of sigmoids, which crowd at 1 as well as at 0, the ratio to what is missing
      // from 2.  Relative errors, twice for the other side's: an exponential's 8 of 2^-24 and twice its argument's x, four
      // of those in a ratio; what was cut off, up to 2^-14 of a score, twice in a ratio.
      float worth = -INFINITY, rel = 0.f;
      if (some) {
        const float l0 = score_at(a, t, 511 - (int)(k0 & 511u)), l1 = k1 ? score_at(a, t, 511 - (int)(k1 & 511u)) : -INFINITY;
        const float largest = fmaxf(fabsf(l0), k1 ? fabsf(l1) : 0.f);
        if (a.sigmoid) {
          const float p = __fdividef(1.f, 1.f + exp2_fast(-l0 * kLog2e)) + __fdividef(1.f, 1.f + exp2_fast(-l1 * kLog2e));
          const float q = __fdividef(1.f, 1.f + exp2_fast(l0 * kLog2e)) + __fdividef(1.f, 1.f + exp2_fast(l1 * kLog2e));
          worth = p / q;
        } else {
          worth = exp2_fast((l0 - shift) * kLog2e) + exp2_fast((l1 - shift) * kLog2e);
        }
        rel = 0x1p-24f * (128.f + 16.f * (a.sigmoid ? largest : fabsf(shift) + largest)) + (a.f32 ? 0x1p-12f * largest : 0.f);
        // nearer to 2 than 64 bits' sums can be compared with this error, or past fp32
        if (a.sigmoid && !(worth < 0x1p30f)) rel = 2.f;
      }
      // NaN: no; the smallest numbers lose bits, or all of them
      auto apart_from = [&](float other) { return fabsf(worth - other) > fmaf(rel, fmaxf(worth, other), 0x1p-118f); };
      bool tight = false;
      for (int g = 0; g < a.groups; ++g) {
        const float other = __shfl_sync(kFull, worth, g, LANES);
        place += other > worth || (other == worth && g < sub);
        if (g != sub) tight |= !apart_from(other);
      }
      if (__any_sync(kFull, some && tight)) {
        for (int g = 0; g < a.groups; ++g) {
          const float other = __shfl_sync(kFull, worth, g, LANES);
          const int there = __shfl_sync(kFull, place, g, LANES);
          const uint32_t y0 = __shfl_sync(kFull, k0, g, LANES), y1 = __shfl_sync(kFull, k1, g, LANES);
          close |= some && y0 != 0 && (place < a.group_k) != (there < a.group_k) && !apart_from(other) &&
                   !(apart < 0 && k0 >> 9 == y0 >> 9 && k1 >> 9 == y1 >> 9);
        }
      }
    }
    if constexpr (REFINE) {
      if (__any_sync(kFull, close)) {
        // the two best are the two best unless another one may be larger than either
        if (__any_sync(kFull, some && nearby(k1, k2))) {
          for (int g = 0; g < a.groups; ++g) {
            const uint32_t y0 = __shfl_sync(kFull, k0, g, LANES), y1 = __shfl_sync(kFull, k1, g, LANES);
#pragma unroll
            for (int i = 0; i < EPL; ++i)
              if (base + i >= g * per && base + i < (g + 1) * per && key[i] != y0 && key[i] != y1)
                near |= unclear(y0, key[i]) || unclear(y1, key[i]);
          }
        }
        const int64_t value = some ? in_order(exact(k0) + (k1 ? exact(k1) : 0.0)) : INT64_MIN;
        place = 0;
        for (int g = 0; g < a.groups; ++g) {
          const int64_t other = __shfl_sync(kFull, value, g, LANES);
          place += other > value || (other == value && g < sub);
        }
      }
    } else {
      near = close;
    }
    kept = __ballot_sync(kFull, some && place < a.group_k) >> first;
  }
  if (grouped) {
    if (a.seg) {
      const uint32_t in = (uint32_t)-(int32_t)((kept >> (sub / a.seg)) & 1);  // lanes past the last group have no keys
#pragma unroll
      for (int i = 0; i < EPL; ++i) key[i] &= in;
    } else {
      int g = base / per, left = per - base % per;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if (g >= a.groups || !((kept >> g) & 1)) key[i] = 0;
        if (--left == 0) {
          ++g;
          left = per;
        }
      }
    }
  }
  sort_falling(key);
  uint32_t mine = 0;  // lane j gets the j-th largest key
  if constexpr (REFINE) {
    for (int j = 0; j < LANES; ++j) {
      const uint32_t best = lanes_max<LANES>(key[0]);
      mine = j == sub ? best : mine;
      const bool pop = key[0] == best;
#pragma unroll
      for (int i = 0; i < EPL - 1; ++i) key[i] = pop ? key[i + 1] : key[i];
      if (pop) key[EPL - 1] = 0;
    }
    int64_t value = INT64_MIN;
    if (mine != 0) value = in_order(plain ? (double)score_at(a, t, 511 - (int)(mine & 511u)) : exact(mine));
    int rank = 0;
    for (int j = 0; j < LANES; ++j) {
      const int64_t other = __shfl_sync(kFull, value, j, LANES);
      const uint32_t there = __shfl_sync(kFull, mine, j, LANES);
      rank += other > value || (other == value && (there & 511u) > (mine & 511u));  // the larger complement first
    }
    uint32_t chosen = 0;
    for (int j = 0; j < LANES; ++j) {
      const int r = __shfl_sync(kFull, mine != 0 ? rank : -1, j, LANES);
      const uint32_t there = __shfl_sync(kFull, mine, j, LANES);
      if (r == sub) chosen = there;
    }
    // unless one that is left may be larger than the last of them
    const uint32_t last = __shfl_sync(kFull, chosen, a.k - 1, LANES);
    if (nearby(last, lanes_max<LANES>(key[0]))) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) near |= unclear(last, key[i]);
    }
    return sub < a.k && chosen != 0 ? 511 - (int)(chosen & 511u) : -1;
  } else {
    uint32_t after = 0;  // the best one left
#pragma unroll
    for (int j = 0; j <= KMAX; ++j) {
      if (j > a.k) break;
      const uint32_t best = lanes_max<LANES>(key[0]);
      mine = j == sub ? best : mine;
      after = best;
      const bool pop = key[0] == best;
#pragma unroll
      for (int i = 0; i < EPL - 1 && i < KMAX - j; ++i) key[i] = pop ? key[i + 1] : key[i];
      if (EPL - 1 < KMAX - j && pop) key[EPL - 1] = 0;
    }
    const uint32_t below = __shfl_down_sync(kFull, mine, 1, LANES), next = sub + 1 == a.k ? after : below;
    // equal ones are ties, but for the last choice and the best one left: what is left behind it may be larger than either
    if (sub < a.k) near |= sub + 1 == a.k ? nearby(mine, next) : unclear(mine, next);
    return sub < a.k && mine != 0 ? 511 - (int)(mine & 511u) : -1;
  }
}

// The same again with 64 bits, from the row itself.  Not inlined: few tokens come here.
template <int EPL, int LANES>
__device__ __noinline__ int choose_again(const RouteArgs& a, const PackedBias& bias, Packing pack, int64_t t,
                                         bool mine, int sub) {
  float v[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = sub * EPL + i;
    v[i] = mine && e < a.experts ? score_at(a, t, e) : -INFINITY;
  }
  float shift = 0.f, total = 1.f;
  if (!a.sigmoid) total = row_softmax<float, EPL>(v, LANES, shift);
  bool near;
  int expert = choose_packed<EPL, CTR_MAX_CHOICES, LANES, true>(a, v, bias, pack, t, sub, shift, total, near);
  if (__any_sync(kFull, near)) {
    float b[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = sub * EPL + i;
      b[i] = a.bias && e < a.experts ? a.bias[e] : 0.f;
      if (!(b[i] < INFINITY)) b[i] = -INFINITY;
    }
    expert = choose_exact<EPL>(a, v, b, sub);
  }
  return expert;
}

template <int EPL, int KMAX, int LANES>
__global__ void __launch_bounds__(kRouteThreads, 2) route_balanced_kernel(const __grid_constant__ RouteArgs a) {
  extern __shared__ uint32_t bits[];  // as in route_choose_kernel
  __shared__ PackedBias bias;
  __shared__ float ends[kRouteThreads / 16];
  const int words = a.tile / 32;
  const int64_t t0 = (int64_t)blockIdx.x * a.tile;
  const int n = (int)imin64(a.tile, a.tokens - t0);
  for (int i = threadIdx.x; i < a.experts * words; i += kRouteThreads) bits[i] = 0;
  grid_wait();
  const Packing pack = pack_range(a, bias, ends);
  const int lane = threadIdx.x & 31, sub = lane & (LANES - 1);
  const uint32_t group = (LANES == 32 ? kFull : (1u << (LANES & 31)) - 1) << (lane & ~(LANES - 1));
  constexpr int per_pass = kRouteThreads / LANES;
  for (int p0 = 0; p0 < n; p0 += per_pass) {  // the same trips in every lane: the shuffles need all of them
    const int tl = p0 + (int)threadIdx.x / LANES;
    const bool mine = tl < n;
    float v[EPL];
    if (mine) {
      load_scores<EPL>(a, t0 + tl, sub * EPL, v);
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[i] = -INFINITY;
    }
    bool odd = false;  // NaN or +inf: the token is routed nowhere
#pragma unroll
    for (int i = 0; i < EPL; ++i) odd |= !(v[i] < INFINITY);
    const bool bad = (__ballot_sync(kFull, odd) & group) != 0;
    if (bad) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[i] = -INFINITY;
      if (sub == 0) set_error(a.err, CTR_ERR_BAD_VALUE);
    }
    float shift = 0.f, total = 1.f;
    if (!a.sigmoid) total = row_softmax<float, EPL>(v, LANES, shift);
    bool near;
    int expert = choose_packed<EPL, KMAX, LANES, false>(a, v, bias, pack, t0 + tl, sub, shift, total, near);
    if (__any_sync(kFull, near))
      expert = choose_again<EPL, LANES>(a, bias, pack, t0 + tl, mine && !bad, sub);
    // weights: lane j has choice j
    const bool live = expert >= 0;
    const float s = live ? score_at(a, t0 + tl, expert) : -INFINITY;
    float z = 0.f, sum = total;
    if (a.renormalize) {
      float m = s;
#pragma unroll
      for (int o = 1; o < LANES; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
      if (live) z = choice_value(a, s, m);
      sum = z;
#pragma unroll
      for (int o = 1; o < LANES; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
    } else if (live) {
      z = choice_value(a, s, shift);
    }
    if (mine && sub < a.k) {
      const int64_t place = (t0 + tl) * a.k + sub;
      a.expert[place] = expert;
      a.weight[place] = live ? a.factor * (z / sum) : 0.f;
      if (live) atomicOr(&bits[expert * words + (tl >> 5)], 1u << (tl & 31));
    }
  }
  if (a.cluster) finish_tile<true>(a, t0, n, bits);
  else finish_tile<false>(a, t0, n, bits);
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

// Softmax over the choices, or sigmoids: lane j of a token's lanes (as few as hold its choices) reads choice j's score
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
    const float g = live ? a.factor * dweight[t * a.k + sub] : 0.f;
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
    const float z = live ? choice_value(a, l, m) : 0.f;
    float total = z, dot = z * g;
    for (int o = 1; o < a.lanes; o <<= 1) {
      total += __shfl_xor_sync(kFull, total, o);
      dot += __shfl_xor_sync(kFull, dot, o);
    }
    float w = z;  // sigmoids renormalised: the weight itself, which is 1 of a single choice, whose gradient is 0
    if (a.sigmoid && a.renormalize) {
      w = live ? z / total : 0.f;
      dot = w * g;
      for (int o = 1; o < a.lanes; o <<= 1) dot += __shfl_xor_sync(kFull, dot, o);
    }
    __syncwarp();  // the row's zeros come before its choices
    if (live) {    // then total >= its own exponential > 0
      const float inv = 1.f / total;
      float d = !a.renormalize ? z * g : a.sigmoid ? w * (g - dot) : z * inv * (g - dot * inv);
      if (a.sigmoid) d *= 1.f / (1.f + expf(l));  // d ln p / dl = 1 - p
      out[e] = from_f32<T>(d);
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
    const float g = live ? a.factor * dweight[t * a.k + sub] : 0.f;
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

template <int EPL, int KMAX, int LANES>
bool launch_balanced(RouteArgs& a, size_t smem, bool& cluster, cudaStream_t s) {
  constexpr auto k = route_balanced_kernel<EPL, KMAX, LANES>;
  cluster = cluster && largest_cluster_fits<k>();
  a.cluster = cluster;
  return launch_after(k, dim3((unsigned)a.tiles), kRouteThreads, smem, s, cluster ? (unsigned)a.tiles : 1u, a) ==
         cudaSuccess;
}

template <int EPL, int KMAX>
bool launch_balanced(RouteArgs& a, size_t smem, bool& cluster, cudaStream_t s) {
  return a.lanes == 8 ? launch_balanced<EPL, KMAX, 8>(a, smem, cluster, s)
         : a.lanes == 16 ? launch_balanced<EPL, KMAX, 16>(a, smem, cluster, s)
                         : launch_balanced<EPL, KMAX, 32>(a, smem, cluster, s);
}

template <int EPL>
bool launch_balanced(RouteArgs& a, size_t smem, bool& cluster, cudaStream_t s) {
  return a.k <= 8 ? launch_balanced<EPL, 8>(a, smem, cluster, s)
                  : launch_balanced<EPL, CTR_MAX_CHOICES>(a, smem, cluster, s);
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
  const bool choices = a.renormalize || a.sigmoid;
  a.lanes = choices ? choice_lanes(a.experts * (int)sizeof(T), a.k, vec_out) : route_lanes(a.experts, a.k, per);
  auto k = choices ? route_bwd_choices_kernel<T> : per == 16 ? route_bwd_kernel<T, 16> : route_bwd_kernel<T, 8>;
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

namespace ctr {
namespace {

// Score function, bias and groups of a routing; the default is none of them.
struct Balance {
  bool on = false, sigmoid = false;
  const float* bias = nullptr;
  int32_t groups = 1, group_k = 1;
  float factor = 1.f;
};

int route(const void* scores, ctr_dtype dtype, int64_t tokens, int32_t experts, int64_t ld_scores, int32_t k, int renormalize,
          const Balance& b, int32_t* expert, float* weight, int32_t* slot, int32_t* token, int32_t* offsets, void* ws,
          size_t ws_bytes, ctr_stream_t stream) {
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
  int per = lane_scores(experts);
  const int members = experts / b.groups;
  const bool grouped = b.group_k < b.groups;
  if (grouped && members % per != 0 && members % 8 == 0 && experts <= 256) per = 8;  // groups of whole lanes, if they can be
  a.lanes = route_lanes(experts, k, per);
  while (b.on && (a.lanes < 8 || (grouped && a.lanes < b.groups))) a.lanes *= 2;  // 8, 16 or 32; one for each group
  if (grouped && members % per == 0 && ((members / per) & (members / per - 1)) == 0) a.seg = members / per;
  a.tile = route_tile(tokens, experts);
  // two blocks an SM: finer tiles even them out (65536 x 256, tiles of 256, 128 and 64 tokens: 108, 101 and 102 us)
  if (b.on && tokens > kClusterTiles * kTileTokens) a.tile = std::min(a.tile, 128);
  a.tiles = (int32_t)ceil_div(tokens, a.tile);
  a.renormalize = renormalize != 0;
  const int eb = dtype_bytes(dtype);
  a.vec = ((uintptr_t)scores % 16) == 0 && (ld_scores * eb) % 16 == 0;
  a.f32 = dtype == CTR_F32;
  a.factor = b.factor;
  a.bias = b.bias;
  a.sigmoid = b.sigmoid;
  a.groups = b.groups;
  a.group_k = b.group_k;
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
  bool ok;
  if (b.on)
    ok = per == 8 ? launch_balanced<8>(a, smem, cluster, s) : launch_balanced<16>(a, smem, cluster, s);
  else
    ok = dtype == CTR_F32 ? (per == 8 ? launch_choose<float, 8>(a, smem, cluster, s)
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

int route_bwd(const float* dweight, const void* scores, ctr_dtype dtype, int64_t tokens, int32_t experts, int64_t ld_scores,
              int32_t k, int renormalize, bool sigmoid, float factor, const int32_t* expert, void* dscores,
              int64_t ld_dscores, void* ws, size_t ws_bytes, ctr_stream_t stream) {
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
  a.sigmoid = sigmoid;
  a.factor = factor;
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

bool score_ok(int score) { return score == CTR_SCORE_SOFTMAX || score == CTR_SCORE_SIGMOID; }

}  // namespace
}  // namespace ctr

extern "C" int ctr_expert_route(const void* scores, ctr_dtype dtype, int64_t tokens, int32_t experts,
                                int64_t ld_scores, int32_t k, int renormalize, int32_t* expert, float* weight,
                                int32_t* slot, int32_t* token, int32_t* offsets, void* ws, size_t ws_bytes,
                                ctr_stream_t stream) {
  return route(scores, dtype, tokens, experts, ld_scores, k, renormalize, Balance(), expert, weight, slot, token, offsets, ws,
               ws_bytes, stream);
}

extern "C" int ctr_expert_route_bwd(const float* dweight, const void* scores, ctr_dtype dtype, int64_t tokens,
                                    int32_t experts, int64_t ld_scores, int32_t k, int renormalize,
                                    const int32_t* expert, void* dscores, int64_t ld_dscores, void* ws,
                                    size_t ws_bytes, ctr_stream_t stream) {
  return route_bwd(dweight, scores, dtype, tokens, experts, ld_scores, k, renormalize, false, 1.f, expert, dscores, ld_dscores,
                   ws, ws_bytes, stream);
}

extern "C" int ctr_expert_route_balanced(const void* scores, ctr_dtype dtype, int64_t tokens, int32_t experts,
                                         int64_t ld_scores, int32_t k, int score, const float* bias, int32_t groups,
                                         int32_t group_k, int renormalize, float factor, int32_t* expert, float* weight,
                                         int32_t* slot, int32_t* token, int32_t* offsets, void* ws, size_t ws_bytes,
                                         ctr_stream_t stream) {
  const int st = check_route(scores, dtype, tokens, experts, ld_scores, k);
  if (st != CTR_OK) return st;
  if (!score_ok(score) || groups < 1 || group_k < 1 || group_k > groups || experts % groups != 0 ||
      k > group_k * (experts / groups) || !(factor < INFINITY) || !(factor > -INFINITY) || ((uintptr_t)bias % 4) != 0)
    return CTR_ERR_INVALID_ARG;
  if (groups > CTR_MAX_GROUPS) return CTR_ERR_UNSUPPORTED;
  Balance b;
  b.on = true;
  b.sigmoid = score == CTR_SCORE_SIGMOID;
  b.bias = bias;
  b.groups = groups;
  b.group_k = group_k;
  b.factor = factor;
  return route(scores, dtype, tokens, experts, ld_scores, k, renormalize, b, expert, weight, slot, token, offsets, ws, ws_bytes,
               stream);
}

extern "C" int ctr_expert_route_balanced_bwd(const float* dweight, const void* scores, ctr_dtype dtype, int64_t tokens,
                                             int32_t experts, int64_t ld_scores, int32_t k, int score, int renormalize,
                                             float factor, const int32_t* expert, void* dscores, int64_t ld_dscores,
                                             void* ws, size_t ws_bytes, ctr_stream_t stream) {
  if (!score_ok(score) || !(factor < INFINITY) || !(factor > -INFINITY)) return CTR_ERR_INVALID_ARG;
  return route_bwd(dweight, scores, dtype, tokens, experts, ld_scores, k, renormalize, score == CTR_SCORE_SIGMOID, factor,
                   expert, dscores, ld_dscores, ws, ws_bytes, stream);
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
