// b3. Products of e4m3 codes with a scale per block of 128, on the tensor cores.
//
//   out[r, i] = sum over blocks kb of  sa[r, kb] * sb[i / 128, kb] * S(r, i, kb),
//   S(r, i, kb) = sum over the block's 128 columns of a[r, c] * b[i, c]
//
// S is four tcgen05.mma (kind::f8f6f4, K = 32 each) into a fresh fp32 TMEM
// accumulator; the scaled sum over kb lives in registers.  Scales are arbitrary
// fp32 numbers, so they cannot ride in the instruction (which takes powers of
// two); what it costs is reading every block's accumulator back once, beside the
// next block's products.
//
// PAIR: two CTAs of a cluster (two SMs) share one 256 x 256 tile: each holds 128
// rows of either operand (32 KB a block of 128), the even one issues the
// cta_group::2 MMAs for both, and each keeps the 128 rows of the accumulator that
// are its own.  A single CTA takes 128 x 128.  The operand tiles come through L2,
// whose share of an SM (about 70 bytes a cycle) is what 128 x 256 tiles of one CTA
// ran into: 48 KB a block take 700 cycles, the products 512.
//
// Roles: warp 0 loads the operand tiles by TMA (128-byte swizzle, a ring of
// stages); warp 1 of the issuing CTA owns the MMAs, into two accumulators in turn;
// warp 2 copies the scales to shared memory, eight blocks at a time; 8 warps scale
// and add: a thread owns one row (TMEM lane) and half of the columns, and one
// packed multiply-add covers two values.  A tile's rows never leave their group: rows past it belong to the
// next group or lie outside the tensor (TMA fills zeros) and are not stored.
// Every mbarrier wait is bounded by a wall-clock limit; on expiry the kernel
// records CTR_ERR_TIMEOUT, waits (bounded) for its own copies and MMAs, frees
// TMEM and returns.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "rows.cuh"
#include "tc.cuh"

namespace ctr {
namespace {

constexpr int kScaleWarps = 8;
constexpr int kMmThreads = 128 + 32 * kScaleWarps;  // warps 0..3: loads, MMAs, scales, none; then scaling
// Registers: 384 threads are launched with 168 each (the most that three warps to a scheduler
// leave); the first four warps give some up so that a scaling thread can hold 128 sums and 64 values
// on their way.  56 x 128 + 224 x 256 = 168 x 384.
constexpr int kLaunchRegs = 168, kControlRegs = 56, kScaleRegs = 224;
static_assert(kControlRegs * 128 + kScaleRegs * 32 * kScaleWarps <= kLaunchRegs * kMmThreads,
              "more registers than launched");
constexpr int kBM = 128;                        // rows of either operand that a CTA holds
constexpr uint32_t kOperandBytes = kBM * 128;
constexpr uint32_t kStageBytes = 2 * kOperandBytes;
constexpr int kStages = 4;
constexpr int kSuper = 8;                       // row tiles that take the column tiles together
constexpr int kSorted = 128;                    // groups whose sums are sorted by length
constexpr int kChunk = 8;                       // blocks whose scales come together
// A scaling warp's pieces of the result on their way out: 32 rows of 128 bytes each, two of them, in
// the 128-byte swizzle (16-byte part i of row r at i ^ (r mod 8)).
constexpr uint32_t kPieceBytes = 32 * 128;
constexpr uint32_t kStagingBytes = 2 * kPieceBytes;
// Scales: two chunks of [block][row], then two of [128-column half][block].
constexpr uint32_t kScaleBytes = 2 * kChunk * (kBM + 2) * 4;
constexpr int kMmSmem = (int)(1024 + kStages * kStageBytes + kScaleWarps * kStagingBytes + kScaleBytes);

struct MmArgs {
  const float* sa;
  const float* sb;
  const int32_t* offsets;  // NULL: one group of all rows
  char* out;
  int* err;
  int64_t ld_sa, ld_sb, ldo;  // sa: [block][row]; sb: [128-column block][block]; ldo in elements
  int64_t rows;
  int32_t groups, m, n, kb;  // m: rows of a group's result (weight gradient); kb: blocks (product)
  int32_t nt, mt;            // column tiles; row tiles of a group (weight gradient)
  int32_t splits;            // few rows: CTAs that share a tile's blocks
  int32_t seg;               // weight gradient: blocks of a partial sum; 0: sums are whole
  int32_t out_f32, wide_rows;  // wide_rows: output rows start 16-byte aligned, and TMA may store them
};

// kind::f8f6f4 instruction descriptor: e4m3 x e4m3 -> fp32, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

template <bool PAIR>
__device__ __forceinline__ void mma_e4m3(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// The issued MMAs' completion arrives at the barrier `bar`, in both CTAs of a pair.
template <bool PAIR>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  else
    mma_commit(bar);
}

// Loads into this CTA's shared memory, counted at `bar` (of the pair's even CTA).
template <bool PAIR>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, int32_t c0, int32_t c1, uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"((uint64_t)map), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
  else
    tma_load_2d(dst, map, c0, c1, bar);
}

// Bounded wait of a whole warp.  The hint lets the hardware park the warp for up to 20 us a try:
// warps that poll take issue slots from the ones that scale.
__device__ __forceinline__ bool park(uint32_t bar, uint32_t parity) {
  uint64_t t0 = 0;
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (__all_sync(kFull, ok)) return true;
    if (t0 == 0) t0 = globaltimer();
    if (__any_sync(kFull, globaltimer() - t0 > kWaitLimitNs)) return false;
  }
}

// One lane of the warp, the same every time.  The roles' loops are run by whole warps, so that
// their values stay in uniform registers; only the copies, MMAs and arrivals are one lane's.
__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// Arrival at a barrier of either CTA.  Release at CTA scope (the default): what it orders are this
// thread's accumulator reads, which are complete; at cluster scope an arrival took 1500 cycles.
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// acc += f * v for 32 values, two at a time.  volatile: stays after the wait for the load of v.
__device__ __forceinline__ void scale_add32(uint64_t* acc, const uint32_t (&v)[32], uint64_t f2) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
    asm volatile(
        "{\n\t.reg .b64 t;\n\t"
        "mov.b64 t, {%1, %2};\n\t"
        "fma.rn.f32x2 %0, t, %3, %0;\n\t}"
        : "+l"(acc[i])
        : "r"(v[2 * i]), "r"(v[2 * i + 1]), "l"(f2));
}

// One fp32 number into shared memory, without waiting; zero where `take` is false (then `any` is a
// valid address that is not read).
__device__ __forceinline__ void copy_scale(uint32_t dst, const float* src, bool take, const float* any) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(take ? src : any), "r"(take ? 4 : 0)
               : "memory");
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *(const uint32_t*)&h;
}

struct Tile {
  int32_t nkb;        // blocks to sum
  int32_t rows;       // rows of this CTA's half of the tile inside the group (may be <= 0)
  int32_t a_row;      // first row of this CTA's left operand
  int32_t b_row;      // first row of this CTA's right operand
  int32_t k0;         // first block along the summed axis
  int32_t sb0;        // row of the block scales for the tile's first 128 columns
  int32_t col;        // first column of the result
  int64_t out_row;    // first output row of this CTA
};

// Tile t, as seen from CTA `rank` of a pair (0 alone).  Weight gradient: offs holds the groups, the
// one with most blocks first; of partial sums, the number of them before each group.
template <bool PAIR, bool WGRAD>
__device__ __forceinline__ Tile locate(const MmArgs& p, const int32_t* start, const int32_t* offs, int t, int rank) {
  constexpr int kTileM = PAIR ? 2 * kBM : kBM, kBN = PAIR ? 256 : 128;
  Tile x;
  int g, mi, ni;
  if constexpr (WGRAD) {
    const int per = p.mt * p.nt;
    const int q = t / per;
    const int l = t - q * per;
    ni = l / p.mt;
    mi = l - ni * p.mt;
    if (p.seg) {
      g = 0;
      while (offs[g + 1] <= q) ++g;
      x.k0 = start[g] + (q - offs[g]) * p.seg;
      x.nkb = min(p.seg, start[g + 1] - x.k0);
      g = q;  // the partial result's place
    } else {
      g = offs[q];
      x.k0 = start[g];
      x.nkb = start[g + 1] - start[g];
    }
    x.a_row = mi * kTileM + rank * kBM;
    x.rows = min(kBM, p.m - x.a_row);
    x.b_row = ni * kBN;
    x.sb0 = ni * (kBN / 128);
    x.out_row = (int64_t)g * p.m + x.a_row;
  } else {
    const int u = t / p.nt;
    int lo = 0, hi = p.groups - 1;  // the group whose row tiles [start[g], start[g+1]) hold u
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (start[mid] <= u) lo = mid;
      else hi = mid - 1;
    }
    g = lo;
    const int l = t - start[g] * p.nt;
    const int mts = start[g + 1] - start[g];
    const int per = kSuper * p.nt;
    const int sg = l / per;
    const int rem = l - sg * per;
    const int mm = min(kSuper, mts - sg * kSuper);
    ni = rem / mm;
    mi = sg * kSuper + rem - ni * mm;
    const int r0 = offs[g], r1 = offs[g + 1];
    x.nkb = p.kb;
    x.k0 = 0;
    x.a_row = r0 + mi * kTileM + rank * kBM;
    x.rows = min(kBM, r1 - x.a_row);
    x.b_row = g * p.n + ni * kBN;
    x.sb0 = g * ((p.n + 127) / 128) + ni * (kBN / 128);
    x.out_row = x.a_row;
  }
  if constexpr (PAIR) x.b_row += rank * kBM;
  x.col = ni * kBN;
  return x;
}

// Tiles of `size` rows before each group (start[groups] = all) and the groups' first rows, by one
// warp.  Bad offsets: all zero and flagged.
__device__ __forceinline__ void group_starts(const MmArgs& p, int32_t* start, int32_t* offs, int size) {
  const int lane = threadIdx.x & 31;
  if (!p.offsets) {
    if (lane == 0) {
      start[0] = offs[0] = 0;
      offs[1] = (int32_t)p.rows;
      start[1] = (int32_t)((p.rows + size - 1) / size);
    }
    return;
  }
  int seen = 0;
  bool ok = p.offsets[0] == 0;
  for (int g0 = 0; g0 < p.groups; g0 += 32) {
    const int g = g0 + lane;
    int lo = 0, hi = 0;
    if (g < p.groups) {
      lo = p.offsets[g];
      hi = p.offsets[g + 1];
      ok = ok && lo >= 0 && hi >= lo && hi <= p.rows;
    }
    int incl = ok ? (hi - lo + size - 1) / size : 0;
    const int mine = incl;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += y;
    }
    if (g < p.groups) {
      start[g] = seen + incl - mine;
      offs[g + 1] = hi;
    }
    seen += __shfl_sync(kFull, incl, 31);
  }
  if (lane == 0) {
    start[p.groups] = seen;
    offs[0] = 0;
  }
  const bool good = __all_sync(kFull, ok);
  __syncwarp();
  if (!good) {
    if (lane == 0) set_error(p.err, CTR_ERR_BAD_OFFSETS);
    for (int g = lane; g <= p.groups; g += 32) start[g] = offs[g] = 0;
  }
}

// Partial sums of the groups before g.
__device__ __forceinline__ int sums_before(const int32_t* start, int g, int seg) {
  int n = 0;
  for (int o = 0; o < g; ++o) n += (start[o + 1] - start[o] + seg - 1) / seg;
  return n;
}

template <bool PAIR, bool WGRAD>
__global__ void __launch_bounds__(kMmThreads, 1) fp8_matmul_kernel(const MmArgs p,
                                                                   const __grid_constant__ CUtensorMap amap,
                                                                   const __grid_constant__ CUtensorMap bmap,
                                                                   const __grid_constant__ CUtensorMap omap) {
  constexpr int kBN = PAIR ? 256 : 128;
  constexpr int kCols = kBN / 2;  // columns of a scaling thread
  constexpr int kCtas = PAIR ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[2 * kStages + 8];
  __shared__ uint32_t tmem_base_slot;
  __shared__ int32_t start[CTR_MAX_EXPERTS + 1], offs[CTR_MAX_EXPERTS + 1];
  __shared__ Tile info[2];  // a tile's place, with its first chunk of scales

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // swizzled tiles need 1024-byte alignment
  uint8_t* after_stages = smem_raw + (base - raw) + kStages * kStageBytes;
  float* row_scales = (float*)(after_stages + kScaleWarps * kStagingBytes);  // [2][kChunk][kBM]
  float* col_scales = row_scales + 2 * kChunk * kBM;                         // [2][2][kChunk]
  const uint32_t full0 = smem_u32(&bars[0]);                 // a stage's operands are there (pair: the even CTA's)
  const uint32_t empty0 = smem_u32(&bars[kStages]);          // a stage's MMAs are done
  const uint32_t tfull0 = smem_u32(&bars[2 * kStages]);      // an accumulator's MMAs and scales are there
  const uint32_t tempty0 = smem_u32(&bars[2 * kStages + 2]); // an accumulator has been read (pair: the even CTA's)
  const uint32_t cfull0 = smem_u32(&bars[2 * kStages + 4]);  // a chunk of scales is there
  const uint32_t cempty0 = smem_u32(&bars[2 * kStages + 6]); // and has been used
  uint32_t rank = 0;
  if constexpr (PAIR) asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, kCtas * kScaleWarps);
      mbar_init(cfull0 + 8 * b, 33);
      mbar_init(cempty0 + 8 * b, kScaleWarps);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_slot)),
                   "r"(2 * kBN)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_slot)),
                   "r"(2 * kBN)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  grid_wait();
  if (warp == 4) group_starts(p, start, offs, WGRAD ? 128 : kCtas * kBM);
  fence_before();
  __syncthreads();
  if constexpr (WGRAD) {
    // Partial sums in the order of the groups.  Whole ones: the long first, so that the last tiles to
    // start are short (experts are chosen unevenly).  A group's place is the number of groups before it;
    // beyond kSorted groups they keep their order.
    if (p.seg) {
      for (int g = threadIdx.x; g <= p.groups; g += kMmThreads) offs[g] = sums_before(start, g, p.seg);
    } else for (int g = threadIdx.x; g < p.groups; g += kMmThreads) {
      const int mine = start[g + 1] - start[g];
      int place = p.groups <= kSorted ? 0 : g;
      for (int o = 0; o < p.groups && p.groups <= kSorted; ++o) {
        const int other = start[o + 1] - start[o];
        place += other > mine || (other == mine && o < g);
      }
      offs[place] = g;
    }
    __syncthreads();
  }
  if constexpr (PAIR) cluster_sync();  // the other CTA's barriers are ready too
  fence_after();
  const uint32_t tmem = tmem_base_slot;
  const int ntiles = (!WGRAD ? start[p.groups] : (p.seg ? offs[p.groups] : p.groups) * p.mt) * p.nt;
  const int first = blockIdx.x / kCtas, step = gridDim.x / kCtas;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
    if (warp == 0) {
      // ---------------- TMA producer ----------------
      const uint32_t count_at = PAIR ? in_cta(full0, 0) : full0;
      int s = 0;
      uint32_t ph = 0, issued = 0;  // issued: blocks so far, at most kStages counted
      bool ok = true;
      for (int t = first; ok && t < ntiles; t += step) {
        const Tile x = locate<PAIR, WGRAD>(p, start, offs, t, (int)rank);
        for (int j = 0; j < x.nkb; ++j) {
          if (!park(empty0 + 8 * s, ph ^ 1)) {
            if (lane == 0) set_error(p.err, CTR_ERR_TIMEOUT);
            ok = false;
            break;
          }
          const uint32_t dst = base + (uint32_t)s * kStageBytes;
          const int32_t k = (x.k0 + j) * 128;
          if (elected()) {
            if (rank == 0) mbar_expect_tx(full0 + 8 * s, kCtas * kStageBytes);
            load_tile<PAIR>(dst, &amap, k, x.a_row, count_at + 8 * s);
            load_tile<PAIR>(dst + kOperandBytes, &bmap, k, x.b_row, count_at + 8 * s);
          }
          __syncwarp();
          if (issued < kStages) ++issued;
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      // drain: every issued load must have landed before the CTA can exit.  The last round's MMAs free
      // the stages; after a failure no MMA may come, and a stage's own barrier says that it is filled
      // (a pair's odd CTA has none and waits the limit out).
      for (uint32_t i = 0; i < issued; ++i) {
        s = s == 0 ? kStages - 1 : s - 1;
        if (s == kStages - 1) ph ^= 1;
        if (!park((ok || rank != 0 ? empty0 : full0) + 8 * s, ph) && lane == 0) set_error(p.err, CTR_ERR_TIMEOUT);
      }
    }
    if (warp == 1 && rank == 0) {
      // ---------------- MMA issuer ----------------
      constexpr uint32_t idesc = idesc_e4m3(kCtas * kBM, kBN);
      const uint64_t desc0 = smem_desc_sw128(base);
      int s = 0;
      uint32_t ph = 0, b = 0, bph = 0, issued = 0;  // issued: blocks so far, at most 2 counted
      bool ok = true;
      for (int t = first; ok && t < ntiles; t += step) {
        const int nkb = WGRAD ? locate<PAIR, WGRAD>(p, start, offs, t, 0).nkb : p.kb;
        for (int j = 0; j < nkb; ++j) {
          if (!park(full0 + 8 * s, ph) || !park(tempty0 + 8 * b, bph ^ 1)) {
            if (lane == 0) set_error(p.err, CTR_ERR_TIMEOUT);
            ok = false;
            break;
          }
          fence_after();
          const uint64_t da = desc0 + (uint64_t)((uint32_t)s * (kStageBytes >> 4));  // addresses in units of 16 bytes
          if (elected()) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_e4m3<PAIR>(tmem + b * kBN, da + 2 * k, da + (kOperandBytes >> 4) + 2 * k, idesc, k != 0);
            commit<PAIR>(empty0 + 8 * s);
            commit<PAIR>(tfull0 + 8 * b);
          }
          __syncwarp();
          if (issued < 2) ++issued;
          bph ^= b;
          b ^= 1;
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      // drain: the last commits must have arrived before TMEM is freed
      for (uint32_t i = 0; i < issued; ++i) {
        b ^= 1;
        bph ^= b;
        if (!park(tfull0 + 8 * b, bph) && lane == 0) set_error(p.err, CTR_ERR_TIMEOUT);
      }
    }
    if (warp == 2) {
      // ---------------- scales ----------------
      // kChunk blocks at a time by asynchronous copies of one scale each, which need no register and
      // stall no one (through registers, with a barrier a block, the reads' latency bounded the kernel).
      // Rows past the group and columns past the result get zeros.
      uint32_t b = 0, ph = 0;
      bool ok = true;
      for (int t = first; ok && t < ntiles; t += step) {
        const Tile x = locate<PAIR, WGRAD>(p, start, offs, t, (int)rank);
        const float* sa = p.sa + (int64_t)x.k0 * p.ld_sa + x.a_row + lane;
        const int h = lane / kChunk, u = lane % kChunk;  // 16 lanes: a block scale each
        const bool has_b = h < kCtas && x.col + 128 * h < p.n;
        const float* sb = p.sb + (int64_t)(x.sb0 + h) * p.ld_sb + x.k0 + u;
        // a tile without blocks has one empty chunk: its place has to reach the scaling warps
        for (int j0 = 0; j0 == 0 || j0 < x.nkb; j0 += kChunk) {
          if (!park(cempty0 + 8 * b, ph ^ 1)) {
            if (lane == 0) set_error(p.err, CTR_ERR_TIMEOUT);
            ok = false;
            break;
          }
          const uint32_t dst = smem_u32(row_scales + b * (kChunk * kBM) + lane);
          for (int j = j0; j < j0 + kChunk && j < x.nkb; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              copy_scale(dst + ((j - j0) * kBM + 32 * r) * 4, sa + (int64_t)j * p.ld_sa + 32 * r, lane + 32 * r < x.rows,
                         p.sa);
          if (h < 2)
            copy_scale(smem_u32(col_scales + (b * 2 + h) * kChunk + u), sb + j0, has_b && j0 + u < x.nkb, p.sb);
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(cfull0 + 8 * b) : "memory");
          if (lane == 0) {
            info[b] = x;
            mbar_arrive(cfull0 + 8 * b);
          }
          ph ^= b;
          b ^= 1;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kScaleRegs));
    // ---------------- scaling warps ----------------
    const int q = warp & 3;             // TMEM lane quarter this warp may read
    const int part = (warp - 4) >> 2;   // which half of the columns
    const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(part * kCols);
    const float* row_scale = row_scales + q * 32 + lane;
    const float* col_scale = col_scales + (part * kCols / 128) * kChunk;
    uint8_t* staging = after_stages + (size_t)(warp - 4) * kStagingBytes;
    const uint32_t tempty_at = PAIR ? in_cta(tempty0, 0) : tempty0;
    uint32_t b = 0, ph = 0, cb = 0, cph = 0;  // accumulator, chunk of scales
    bool ok = true;
    for (int t = first; ok && t < ntiles; t += step) {
      // the tile's place comes with its first scales: finding it here would hold the sums up
      if (!park(cfull0 + 8 * cb, cph)) {
        if (lane == 0) set_error(p.err, CTR_ERR_TIMEOUT);
        ok = false;
        break;
      }
      const int nkb = info[cb].nkb;
      uint64_t acc[kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) acc[i] = 0;
      for (int j = 0; j < nkb; ++j) {
        const int u = j % kChunk;
        if (u == 0 && j > 0) ok = park(cfull0 + 8 * cb, cph);
        const float f = row_scale[(cb * kChunk + u) * kBM] * col_scale[cb * (2 * kChunk) + u];
        ok = ok && park(tfull0 + 8 * b, ph);
        if (!ok) {
          if (lane == 0) set_error(p.err, CTR_ERR_TIMEOUT);
          break;
        }
        fence_after();
        uint64_t f2;
        asm("mov.b64 %0, {%1, %1};" : "=l"(f2) : "r"(__float_as_uint(f)));
#pragma unroll
        for (int c = 0; c < kCols; c += 64) {
          uint32_t v0[32], v1[32];
          tmem_ld32_async(lane_base + b * kBN + c, v0);
          tmem_ld32_async(lane_base + b * kBN + c + 32, v1);
          tmem_wait_ld();
          if (c + 64 == kCols) {  // the accumulator is in registers: the next MMAs may have it
            fence_before();
            __syncwarp();
            if (lane == 0) {
              if (rank == 0) mbar_arrive(tempty0 + 8 * b);
              else arrive_at(tempty_at + 8 * b);
            }
          }
          scale_add32(acc + c / 2, v0, f2);
          scale_add32(acc + c / 2 + 16, v1, f2);
        }
        if (u == kChunk - 1 && j + 1 < nkb) {
          __syncwarp();
          if (lane == 0) mbar_arrive(cempty0 + 8 * cb);
          cph ^= cb;
          cb ^= 1;
        }
        ph ^= b;
        b ^= 1;
      }
      if (!ok) break;
      // the place is read again: the registers are full while the blocks are summed
      const Tile x = info[cb];
      __syncwarp();
      if (lane == 0) mbar_arrive(cempty0 + 8 * cb);
      cph ^= cb;
      cb ^= 1;
      // ---- the rows leave through shared memory, 32 rows of 128 bytes to a piece (64 columns of bf16, 32
      // of fp32).  Where the output's rows are 16-byte aligned a piece of 32 rows leaves as one TMA store,
      // which drains while the next tile is summed (stores from the threads, or a bulk copy a row, held the
      // warps up for 3800 cycles a tile); else, and at a group's last rows and the result's last columns,
      // the warp stores elements, consecutive columns together.  bf16: both pieces under one fence; fp32:
      // four pieces in turn through the two places.
      const int nrows = min(32, x.rows - q * 32);
      const int col0 = x.col + part * kCols;
      if (nrows <= 0 || col0 >= p.n) continue;
      const bool whole = p.wide_rows && nrows == 32;
      auto leave = [&](const uint8_t* piece, int col) {
        const int width = p.out_f32 ? 32 : 64;
        if (whole && col + width <= p.n) {
          if (lane == 0)
            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                             (uint64_t)&omap),
                         "r"(col), "r"((int32_t)(x.out_row + q * 32)), "r"(smem_u32(piece))
                         : "memory");
        } else if (p.out_f32) {
          float* out = (float*)p.out + (x.out_row + q * 32) * p.ldo + col + lane;
          if (col + lane < p.n)
            for (int r = 0; r < nrows; ++r)
              out[r * p.ldo] = *(const float*)(piece + r * 128 + (((lane >> 2) ^ (r & 7)) * 16) + (lane & 3) * 4);
        } else {
          uint16_t* out = (uint16_t*)p.out + (x.out_row + q * 32) * p.ldo + col + lane;
#pragma unroll
          for (int e = 0; e < 64; e += 32)
            if (col + e + lane < p.n)
              for (int r = 0; r < nrows; ++r)
                out[r * p.ldo + e] =
                    *(const uint16_t*)(piece + r * 128 + ((((e + lane) >> 3) ^ (r & 7)) * 16) + (lane & 7) * 2);
        }
      };
      uint8_t* row = staging + lane * 128;
      if (p.out_f32) {
#pragma unroll
        for (int h = 0; h < kCols / 32; ++h) {
          if (col0 + 32 * h >= p.n) break;
          // The place is free: all of the last tile's pieces have left (an odd number of them ends in the first
          // place), then of this tile's all but the newest.
          if (lane == 0) {
            if (h == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            else asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 2; ++k)
              asm("mov.b64 {%0, %1}, %2;" : "=r"(w[2 * k]), "=r"(w[2 * k + 1]) : "l"(acc[16 * h + 2 * i + k]));
            *(uint4*)(row + (h & 1) * kPieceBytes + ((i ^ (lane & 7)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          if (whole) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          leave(staging + (h & 1) * kPieceBytes, col0 + 32 * h);
          if (lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
      } else {
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the last tile's pieces have left
        __syncwarp();
#pragma unroll
        for (int h = 0; h < kCols / 64; ++h)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t lo, hi;
              asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(acc[32 * h + 4 * i + k]));
              w[k] = bf16_pair(__uint_as_float(lo), __uint_as_float(hi));
            }
            *(uint4*)(row + h * kPieceBytes + ((i ^ (lane & 7)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        if (whole) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int h = 0; h < kCols / 64; ++h)
          if (col0 + 64 * h < p.n) leave(staging + h * kPieceBytes, col0 + 64 * h);
        if (lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (!WGRAD && p.offsets) {
      // rows past the last group: zeros
      const int64_t used = offs[p.groups];
      const int64_t stride = (int64_t)gridDim.x * kScaleWarps;
      for (int64_t r = used + (int64_t)blockIdx.x * kScaleWarps + (warp - 4); r < p.rows; r += stride)
        for (int c = lane; c < p.n; c += 32) {
          if (p.out_f32) ((float*)p.out)[r * p.ldo + c] = 0.f;
          else ((uint16_t*)p.out)[r * p.ldo + c] = 0;
        }
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // nothing of this CTA is the other's target any more
  if (warp == 1) {
    fence_after();
    if constexpr (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * kBN) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * kBN) : "memory");
  }
}

// ---------------------------------------------------------------------------
// Weight gradient in partial sums: the groups' planes of n x k, four columns of one row to a thread,
// added in their order.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kJoinThreads) join_sums_kernel(const MmArgs p, const float* part,
                                                                 int64_t ld, bool vec) {
  __shared__ int32_t start[CTR_MAX_EXPERTS + 1], offs[CTR_MAX_EXPERTS + 1];
  grid_wait();
  if (threadIdx.x < 32) group_starts(p, start, offs, 128);
  __syncthreads();
  const int g = blockIdx.y;
  const int count = (start[g + 1] - start[g] + p.seg - 1) / p.seg;
  const int quads = (int)(ld / 4), e = blockIdx.x * kJoinThreads + threadIdx.x;
  const int row = e / quads, c = (e - row * quads) * 4;
  if (row >= p.m) return;
  const int64_t plane = p.m * ld;
  const float* from = part + sums_before(start, g, p.seg) * plane + row * ld + c;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int s = 0; s < count; ++s) {
    const float4 v = *(const float4*)(from + s * plane);
    sum.x += v.x;
    sum.y += v.y;
    sum.z += v.z;
    sum.w += v.w;
  }
  T* out = (T*)p.out + ((int64_t)g * p.m + row) * p.n + c;
  if (vec) {
    if constexpr (sizeof(T) == 4) *(float4*)out = sum;
    else *(uint2*)out = make_uint2(bf16_pair(sum.x, sum.y), bf16_pair(sum.z, sum.w));
  } else {
    const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < p.n) out[i] = from_f32<T>(v[i]);
  }
}

// ---------------------------------------------------------------------------
// Few rows a group: the weights are the left operand (128 of their rows to a
// CTA), up to 32 of a group's rows the right one, so that a tile reads each
// weight once and multiplies no more than 32 columns.  The blocks are shared out
// over a cluster of up to eight CTAs, enough to keep every SM reading, and their
// sums joined through distributed shared memory in the order of the blocks.  Two
// CTAs an SM.  Bound by the weights' bytes, and below some megabytes by latency.
// ---------------------------------------------------------------------------
constexpr int kFewCols = 32;
constexpr int kFewThreads = 192;  // warp 0: loads, 1: MMAs, 2..5: scaling
constexpr int kFewStages = 5;
constexpr uint32_t kFewStageBytes = kOperandBytes + kFewCols * 128;
constexpr int kFewSmem = (int)(1024 + kFewStages * kFewStageBytes);
constexpr int kFewChunk = 8;      // blocks whose scales are read together

__global__ void __launch_bounds__(kFewThreads, 2) fp8_few_kernel(const MmArgs p,
                                                                 const __grid_constant__ CUtensorMap wmap,
                                                                 const __grid_constant__ CUtensorMap xmap) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[2 * kFewStages + 4];
  __shared__ uint32_t tmem_base_slot;
  __shared__ int32_t start[CTR_MAX_EXPERTS + 1], offs[CTR_MAX_EXPERTS + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  // [row of x][row of the weights]: this CTA's share of the sums, over the stages once they are used up
  float(*sums)[kBM] = (float(*)[kBM])(smem_raw + (base - raw));
  const uint32_t full0 = smem_u32(&bars[0]), empty0 = smem_u32(&bars[kFewStages]);
  const uint32_t tfull0 = smem_u32(&bars[2 * kFewStages]), tempty0 = smem_u32(&bars[2 * kFewStages + 2]);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kFewStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, 4);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_slot)),
                 "r"(2 * kFewCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  grid_wait();
  if (warp == 2) group_starts(p, start, offs, kFewCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_base_slot;

  // this cluster's tile: 128 rows of the weights of a group, and up to 32 of its rows
  const int split = (int)(blockIdx.x % p.splits), tile = (int)(blockIdx.x / p.splits);
  const int u = tile / p.nt, ni = tile - u * p.nt;
  const bool work = u < start[p.groups];
  int lo = 0, hi = p.groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (start[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  const int g = lo;
  const int row0 = offs[g] + (u - start[g]) * kFewCols;
  const int rows = work ? min(kFewCols, offs[g + 1] - row0) : 0;
  const int j0 = (int)((int64_t)p.kb * split / p.splits), j1 = (int)((int64_t)p.kb * (split + 1) / p.splits);
  const int nkb = work ? j1 - j0 : 0;

  if (warp == 0) {
    for (int j = 0; j < nkb; ++j) {
      const int s = j % kFewStages;
      if (j >= kFewStages && !park(empty0 + 8 * s, (uint32_t)((j / kFewStages - 1) & 1))) {
        if (lane == 0) set_error(p.err, CTR_ERR_TIMEOUT);
        break;
      }
      if (elected()) {
        mbar_expect_tx(full0 + 8 * s, kFewStageBytes);
        const uint32_t dst = base + (uint32_t)s * kFewStageBytes;
        tma_load_2d(dst, &wmap, (j0 + j) * 128, g * p.n + ni * kBM, full0 + 8 * s);
        tma_load_2d(dst + kOperandBytes, &xmap, (j0 + j) * 128, row0, full0 + 8 * s);
      }
      __syncwarp();
    }
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_e4m3(kBM, kFewCols);
    const uint64_t desc0 = smem_desc_sw128(base);
    int done = 0;
    for (int j = 0; j < nkb; ++j, ++done) {
      const int s = j % kFewStages, b = j & 1;
      if (!park(full0 + 8 * s, (uint32_t)((j / kFewStages) & 1)) ||
          (j >= 2 && !park(tempty0 + 8 * b, (uint32_t)((j / 2 - 1) & 1)))) {
        if (lane == 0) set_error(p.err, CTR_ERR_TIMEOUT);
        break;
      }
      fence_after();
      const uint64_t d = desc0 + (uint64_t)((uint32_t)s * (kFewStageBytes >> 4));
      if (elected()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_e4m3<false>(tmem + b * kFewCols, d + 2 * k, d + (kOperandBytes >> 4) + 2 * k, idesc, k != 0);
        mma_commit(empty0 + 8 * s);
        mma_commit(tfull0 + 8 * b);
      }
      __syncwarp();
    }
    // drain: the MMAs are done with shared memory and TMEM, and every load that was waited for has landed
    for (int j = max(0, done - 2); j < done; ++j)
      if (!park(tfull0 + 8 * (j & 1), (uint32_t)((j / 2) & 1)) && lane == 0) set_error(p.err, CTR_ERR_TIMEOUT);
    for (int j = done; j < min(nkb, done + kFewStages); ++j)  // after a failure: loads nobody used
      park(full0 + 8 * (j % kFewStages), (uint32_t)((j / kFewStages) & 1));
  } else {
    const int q = warp & 3, n = q * 32 + lane;  // row of the weights
    const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16);
    // lane t has row t of x; the other lanes read the last one's scales, so that the loads need no branch
    const float* sa = p.sa + (int64_t)j0 * p.ld_sa + row0 + min(lane, rows - 1);
    const float* sb = p.sb + (int64_t)(g * p.nt + ni) * p.ld_sb + j0;
    uint64_t acc[kFewCols / 2];
#pragma unroll
    for (int i = 0; i < kFewCols / 2; ++i) acc[i] = 0;
    bool ok = true;
    for (int c = 0; ok && c < nkb; c += kFewChunk) {
      float f[kFewChunk];
#pragma unroll
      for (int i = 0; i < kFewChunk; ++i) {
        const int j = min(c + i, nkb - 1);
        const float v = sa[(int64_t)j * p.ld_sa] * sb[j];
        f[i] = lane < rows ? v : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kFewChunk; ++i) {
        const int j = c + i, b = j & 1;
        if (j >= nkb) break;
        if (!park(tfull0 + 8 * b, (uint32_t)((j / 2) & 1))) {
          if (lane == 0) set_error(p.err, CTR_ERR_TIMEOUT);
          ok = false;
          break;
        }
        fence_after();
        uint32_t v[kFewCols];
        tmem_ld32(lane_base + b * kFewCols, v);
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty0 + 8 * b);
#pragma unroll
        for (int t = 0; t < kFewCols / 2; ++t) {
          const float f0 = __shfl_sync(kFull, f[i], 2 * t), f1 = __shfl_sync(kFull, f[i], 2 * t + 1);
          asm volatile(
              "{\n\t.reg .b64 t, w;\n\t"
              "mov.b64 t, {%1, %2};\n\t"
              "mov.b64 w, {%3, %4};\n\t"
              "fma.rn.f32x2 %0, t, w, %0;\n\t}"
              : "+l"(acc[t])
              : "r"(v[2 * t]), "r"(v[2 * t + 1]), "r"(__float_as_uint(f0)), "r"(__float_as_uint(f1)));
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kFewCols / 2; ++t) {
      uint32_t a0, a1;
      asm("mov.b64 {%0, %1}, %2;" : "=r"(a0), "=r"(a1) : "l"(acc[t]));
      sums[2 * t][n] = __uint_as_float(a0);
      sums[2 * t + 1][n] = __uint_as_float(a1);
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (p.splits > 1) cluster_sync();  // every CTA's sums are there
  if (warp >= 2) {
    const int n = (warp - 2) * 32 + lane, col = ni * kBM + n;
    if (col < p.n) {
      // the cluster's CTAs take the tile's rows in turn
#pragma unroll 4
      for (int t = split; t < rows; t += p.splits) {
        float v = 0.f;
        if (p.splits == 1) {
          v = sums[t][n];
        } else {
          for (int r = 0; r < p.splits; ++r) {
            float w;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(w) : "r"(in_cta(smem_u32(&sums[t][n]), r)) : "memory");
            v += w;
          }
        }
        const int64_t at = (int64_t)(row0 + t) * p.ldo + col;
        if (p.out_f32) ((float*)p.out)[at] = v;
        else ((__nv_bfloat16*)p.out)[at] = __float2bfloat16_rn(v);
      }
    }
    if (p.offsets) {  // rows past the last group: zeros
      const int64_t stride = (int64_t)gridDim.x * 4;
      for (int64_t r = offs[p.groups] + (int64_t)blockIdx.x * 4 + (warp - 2); r < p.rows; r += stride)
        for (int c = lane; c < p.n; c += 32) {
          if (p.out_f32) ((float*)p.out)[r * p.ldo + c] = 0.f;
          else ((uint16_t*)p.out)[r * p.ldo + c] = 0;
        }
    }
  }
  __syncthreads();
  if (p.splits > 1) cluster_sync();  // no CTA leaves while another reads its sums
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * kFewCols) : "memory");
  }
}

// Codes [rows, bytes per row] in tiles of 128 bytes x `box` rows.
bool code_map(CUtensorMap* map, const void* codes, int64_t rows, int64_t row_bytes, int box) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t gdim[2] = {(cuuint64_t)row_bytes, (cuuint64_t)rows};
  cuuint64_t gstride[1] = {(cuuint64_t)row_bytes};
  cuuint32_t bx[2] = {128, (cuuint32_t)box};
  cuuint32_t es[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), gdim, gstride, bx, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The output in pieces of 128 bytes x 32 rows.
bool out_map(CUtensorMap* map, const MmArgs& p, int64_t rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const int eb = p.out_f32 ? 4 : 2;
  cuuint64_t gdim[2] = {(cuuint64_t)p.n, (cuuint64_t)rows};
  cuuint64_t gstride[1] = {(cuuint64_t)(p.ldo * eb)};
  cuuint32_t bx[2] = {(cuuint32_t)(128 / eb), 32};
  cuuint32_t es[2] = {1, 1};
  return enc(map, p.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.out, gdim,
             gstride, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool PAIR, bool WGRAD>
int launch_mm(MmArgs& p, const uint8_t* a, int64_t a_rows, const uint8_t* b, int64_t b_rows, int64_t row_bytes,
              int64_t tiles_m, cudaStream_t s) {
  CUtensorMap amap, bmap;
  if (!code_map(&amap, a, a_rows, row_bytes, kBM) || !code_map(&bmap, b, b_rows, row_bytes, kBM)) return CTR_ERR_CUDA;
  CUtensorMap omap = amap;  // not used unless the output's rows are aligned
  const int64_t planes = p.seg ? tiles_m : p.groups;  // weight gradient: results of m rows
  if (p.wide_rows && !out_map(&omap, p, WGRAD ? planes * p.m : p.rows)) return CTR_ERR_CUDA;
  constexpr int kCtas = PAIR ? 2 : 1;
  p.nt = (int32_t)ceil_div(p.n, PAIR ? 256 : 128);
  if (WGRAD) p.mt = (int32_t)ceil_div(p.m, kCtas * kBM);
  auto k = fp8_matmul_kernel<PAIR, WGRAD>;
  // the split of registers between the warps waits for ever if the kernel was launched with fewer
  static std::atomic<uint64_t> ready{0};
  if (!once_per_device(ready, [&] {
        cudaFuncAttributes fa;
        return cudaFuncGetAttributes(&fa, k) == cudaSuccess && fa.numRegs == kLaunchRegs &&
               cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMmSmem) == cudaSuccess;
      }))
    return CTR_ERR_CUDA;
  const int64_t tiles = (WGRAD ? planes * p.mt : tiles_m) * p.nt;
  if (tiles > INT32_MAX - 65536) return CTR_ERR_UNSUPPORTED;
  const cudaError_t e = launch_after(k, dim3((unsigned)(kCtas * imax64(1, imin64(tiles, num_sms() / kCtas)))), kMmThreads,
                                     kMmSmem, s, kCtas, p, amap, bmap, omap);
  return e == cudaSuccess ? launch_status() : CTR_ERR_CUDA;
}

int launch_few(MmArgs& p, const uint8_t* a, int64_t a_rows, const uint8_t* b, int64_t b_rows, int64_t row_bytes,
               cudaStream_t s) {
  CUtensorMap wmap, xmap;
  if (!code_map(&wmap, b, b_rows, row_bytes, kBM) || !code_map(&xmap, a, a_rows, row_bytes, kFewCols))
    return CTR_ERR_CUDA;
  p.nt = (int32_t)ceil_div(p.n, kBM);
  const int64_t units = imin64((a_rows + (kFewCols - 1) * (int64_t)p.groups) / kFewCols, a_rows);  // row tiles, at most
  const int64_t tiles = imax64(1, p.offsets ? units : ceil_div(a_rows, kFewCols)) * p.nt;
  // CTAs to a tile: until two fill every SM, at least two blocks each
  p.splits = 1;
  while (p.splits < 8 && tiles * p.splits * 2 <= 2 * num_sms() && p.splits * 4 <= p.kb) p.splits *= 2;
  if (tiles * p.splits > INT32_MAX) return CTR_ERR_UNSUPPORTED;
  static std::atomic<uint64_t> ready{0};
  if (!once_per_device(ready, [&] {
        return cudaFuncSetAttribute(fp8_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem) == cudaSuccess;
      }))
    return CTR_ERR_CUDA;
  const cudaError_t e = launch_after(fp8_few_kernel, dim3((unsigned)(tiles * p.splits)), kFewThreads, kFewSmem, s,
                                     (unsigned)p.splits, p, wmap, xmap);
  return e == cudaSuccess ? launch_status() : CTR_ERR_CUDA;
}

// Up to 16 rows a group on average go to the kernel that streams the weights (device time of one
// call with cold caches, its launch included; few rows against 128 x 128 tiles): 1 row of 4096 x 4096
// 15.0 us against 21.2, 16 groups of 8 rows of 2048 x 1024 17.1 against 19.1, of 32 rows 19.1 against
// 19.1, of 64 rows 25.2 against 19.1; 32 rows of 1024 x 512 13.0 against 10.9.
bool few_rows(int64_t rows, int32_t groups) { return rows <= 16 * (int64_t)groups; }

// A pair of CTAs on 256 x 256 tiles where the groups fill a tile's rows and there are tiles for most of the
// pairs (as above, pairs against 128 x 128 tiles): 16 groups of 2048 x 1024 with 128 rows each 23.2 us
// against 19.1, 256 rows 23.2 against 25.2, 512 rows 31.4 against 35.5; one group of 8192 x 1024 with 256
// rows (32 pairs) 14.9 against 13.0, 512 rows (64) 15.1 against 17.1.
bool use_pair(int64_t rows, int64_t groups, int64_t n) {
  return n > 128 && rows >= 256 * groups && ceil_div(rows, 256) * ceil_div(n, 256) >= num_sms() / 3;
}

// How a weight gradient is taken apart (figures: device time of a call with cold caches).  A pair of CTAs
// has to have sums of some length, or more than a round of tiles, to be worth its setting up, and of
// several groups, which are as a rule uneven, enough tiles for every pair (pairs against 128 x 128 tiles):
// 16 groups of 2 to 3 blocks, 512 x 512, 15.0 us against 13.0, of 16 blocks 23.2 against 25.2 but uneven
// 37.5 against 35.5; 4 groups of 32, 2048 x 1024, 43.7 against 58.0, uneven 49.9 against 58.0; one of 64
// blocks, 2048 x 2048, 39.6 against 53.9.
// Where the tiles of whole sums would leave half of the SMs idle, each group's sum is cut into partial
// sums of `seg` blocks, as many as run at once, and a second kernel adds them up in their order: 65536
// rows of 1024 x 1024 175 -> 76 us, 16384 rows of 512 x 479 52 -> 25, 8 uneven groups of 65536 rows of
// 512 x 512 103 -> 46 (even ones 42 -> 48).  The parts and their kernel cost about as much as 8 blocks, so
// shorter sums stay whole: 12 blocks of 1024 x 1024 17.0 us whole against 21.1, 16 19.1 against 21.1, 32
// 25.2 against 23.2; 26 blocks of 512 x 479 25.2 against 21.1.
struct WgradPlan {
  bool pair;
  int32_t seg = 0;     // blocks of a partial sum; 0: sums are whole
  int64_t planes = 0;  // partial results of all groups, at most
  int64_t ld = 0;      // their rows' stride, in elements (16-byte aligned rows)
  size_t bytes() const { return (size_t)planes * ld * 4; }  // a row of each
};

// Blocks of a partial sum, at least: 4096 rows of 512 x 479 take 19.1 us with 4, 21.2 with 8 and 24.2 with
// 16; 16384 rows 27.3, 25.3 and 25.2.
constexpr int kMinSeg = 8;

WgradPlan plan_wgrad(int64_t rows, int64_t groups, int64_t n, int64_t k) {
  WgradPlan w;
  const int64_t blocks = ctr_fp8_padded_rows(rows, (int32_t)groups) / 128;
  const int64_t pairs = groups * ceil_div(n, 256) * ceil_div(k, 256);  // tiles of whole sums
  const bool wide = n > 128 && k > 128;
  w.pair = wide && (blocks >= 8 * groups || pairs >= num_sms());
  const int64_t side = w.pair ? 256 : 128, workers = num_sms() / (w.pair ? 2 : 1);
  const int64_t room = workers / (ceil_div(n, side) * ceil_div(k, side));  // planes that run at once
  const auto whole = [&] {
    w.pair = w.pair && (groups == 1 || pairs >= num_sms() / 2);
    return w;
  };
  if (room < 2 * groups) return whole();
  // a group's last partial sum may be short: as many are left over as there are groups
  const int64_t seg = imax64(kMinSeg, ceil_div(blocks, groups == 1 ? room : room - groups));
  if (blocks < groups * (seg + kMinSeg)) return whole();
  w.seg = (int32_t)seg;
  w.planes = groups == 1 ? ceil_div(blocks, seg) : room;
  w.ld = ceil_div(k, 4) * 4;
  return w;
}

int check_mm(const void* a, const float* sa, const void* b, const float* sb, const int32_t* offsets, int64_t rows,
             int32_t groups, int64_t n, int64_t k, const void* out, int out_dtype, void* ws, size_t ws_bytes) {
  if (!dtype_ok(out_dtype) || rows < 0 || groups < 1 || n < 1 || k < 1) return CTR_ERR_INVALID_ARG;
  if (!offsets && groups != 1) return CTR_ERR_INVALID_ARG;
  if (groups > CTR_MAX_EXPERTS || rows > INT32_MAX - 65536 || n > INT32_MAX / 2 / groups ||
      k > INT32_MAX / 2 / groups)
    return CTR_ERR_UNSUPPORTED;
  if (!ws_valid(ws, ws_bytes, kWsHeader)) return CTR_ERR_WORKSPACE;
  if (!b || !sb || ((uintptr_t)b % 16) != 0) return CTR_ERR_INVALID_ARG;
  if (rows > 0 && (!a || !sa || ((uintptr_t)a % 16) != 0)) return CTR_ERR_INVALID_ARG;
  if (!out || ((uintptr_t)out % dtype_bytes(out_dtype)) != 0) return CTR_ERR_INVALID_ARG;
  return CTR_OK;
}

}  // namespace
}  // namespace ctr

using namespace ctr;

extern "C" size_t ctr_fp8_matmul_workspace_size(int64_t rows, int32_t groups, int64_t n, int64_t k) {
  if (rows < 0 || groups < 1 || n < 1 || k < 1) return 0;
  return kWsHeader + plan_wgrad(rows, groups, n, k).bytes() * n;
}

extern "C" int ctr_fp8_matmul(const uint8_t* a, const float* a_scale, int64_t ld_scale, const uint8_t* b,
                              const float* b_scale, const int32_t* offsets, int64_t rows, int32_t groups, int64_t n,
                              int64_t k, void* out, ctr_dtype out_dtype, int64_t ldo, void* ws, size_t ws_bytes,
                              ctr_stream_t stream) {
  if (rows == 0 && n >= 1 && k >= 1 && groups >= 1) return CTR_OK;
  const int st = check_mm(a, a_scale, b, b_scale, offsets, rows, groups, n, k, out, out_dtype, ws, ws_bytes);
  if (st != CTR_OK) return st;
  if (ldo < n || ld_scale < rows) return CTR_ERR_INVALID_ARG;
  MmArgs p = {};
  p.sa = a_scale;
  p.sb = b_scale;
  p.offsets = offsets;
  p.out = (char*)out;
  p.err = (int*)ws;
  p.kb = (int32_t)ceil_div(k, 128);
  p.ld_sa = ld_scale;
  p.ld_sb = p.kb;
  p.ldo = ldo;
  p.rows = rows;
  p.groups = groups;
  p.n = (int32_t)n;
  p.out_f32 = out_dtype == CTR_F32;
  const int eb = dtype_bytes(out_dtype);
  p.wide_rows = ((uintptr_t)out % 16) == 0 && (ldo * eb) % 16 == 0 && ldo * eb < (1ll << 40);
  cudaStream_t s = (cudaStream_t)stream;
  const int64_t row_bytes = (int64_t)p.kb * 128;
  if (few_rows(rows, groups)) return launch_few(p, a, rows, b, groups * n, row_bytes, s);
  const int64_t m256 = ceil_div(rows + 255 * (int64_t)(groups - 1), 256);  // row tiles, at most
  const int64_t m128 = ceil_div(rows + 127 * (int64_t)(groups - 1), 128);
  if (use_pair(rows, groups, n))
    return launch_mm<true, false>(p, a, rows, b, groups * n, row_bytes, m256, s);
  return launch_mm<false, false>(p, a, rows, b, groups * n, row_bytes, m128, s);
}

extern "C" int ctr_fp8_matmul_wgrad(const uint8_t* d, const float* d_scale, const uint8_t* x, const float* x_scale,
                                    const int32_t* offsets, int64_t rows, int32_t groups, int64_t n, int64_t k,
                                    void* out, ctr_dtype out_dtype, void* ws, size_t ws_bytes, ctr_stream_t stream) {
  if (!offsets) return CTR_ERR_INVALID_ARG;
  const int st = check_mm(d, d_scale, x, x_scale, offsets, imax64(rows, 1), groups, n, k, out, out_dtype, ws, ws_bytes);
  if (st != CTR_OK) return st;
  const int64_t padded = ctr_fp8_padded_rows(rows, groups);
  if (rows < 0 || padded > INT32_MAX) return rows < 0 ? CTR_ERR_INVALID_ARG : CTR_ERR_UNSUPPORTED;
  MmArgs p = {};
  p.sa = d_scale;
  p.sb = x_scale;
  p.offsets = offsets;
  p.out = (char*)out;
  p.err = (int*)ws;
  p.ld_sa = n;
  p.ld_sb = padded / 128;
  p.ldo = k;
  p.rows = rows;
  p.groups = groups;
  p.m = (int32_t)n;
  p.n = (int32_t)k;
  p.out_f32 = out_dtype == CTR_F32;
  const int eb = dtype_bytes(out_dtype);
  p.wide_rows = ((uintptr_t)out % 16) == 0 && (k * eb) % 16 == 0 && groups * n < INT32_MAX;
  cudaStream_t s = (cudaStream_t)stream;
  const WgradPlan w = plan_wgrad(rows, groups, n, k);
  if (!w.seg)
    return w.pair ? launch_mm<true, true>(p, d, n, x, k, padded, 0, s) : launch_mm<false, true>(p, d, n, x, k, padded, 0, s);
  if (ws_bytes < kWsHeader + w.bytes() * n) return CTR_ERR_WORKSPACE;
  float* part = (float*)((char*)ws + kWsHeader);
  MmArgs q = p;
  q.seg = p.seg = w.seg;
  q.out = (char*)part;
  q.out_f32 = q.wide_rows = 1;
  q.ldo = w.ld;
  const int e = w.pair ? launch_mm<true, true>(q, d, n, x, k, padded, w.planes, s)
                       : launch_mm<false, true>(q, d, n, x, k, padded, w.planes, s);
  if (e != CTR_OK) return e;
  const dim3 grid((unsigned)ceil_div(n * (w.ld / 4), kJoinThreads), (unsigned)groups);
  const bool vec = k % 4 == 0 && ((uintptr_t)out % (4 * eb)) == 0;
  const cudaError_t j =
      out_dtype == CTR_F32
          ? launch_after(join_sums_kernel<float>, grid, kJoinThreads, 0, s, 1, p, (const float*)part, w.ld, vec)
          : launch_after(join_sums_kernel<__nv_bfloat16>, grid, kJoinThreads, 0, s, 1, p, (const float*)part, w.ld, vec);
  return j == cudaSuccess ? launch_status() : CTR_ERR_CUDA;
}
