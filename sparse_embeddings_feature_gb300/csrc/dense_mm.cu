// c2. Products of the dense layers on the tensor cores: forward with bias, activation and residual in the
// epilogue, input gradient, weight gradient.
//
//   out[i, j] = epilogue(sum over r of A(i, r) B(j, r))
//
// tcgen05.mma kind::f16 (bf16, fp32 accumulators in TMEM), 64 of r a block.  Operands come by TMA as they lie in
// memory: an operand whose rows run along r is K-major in shared memory, one whose rows run along i or j is
// MN-major (64 of i or j to a 128-byte row, 8 KB a chunk of 64), so that neither gradient needs a transpose.
//
// fp32 matrices are three planes of bf16 (x = x0 + x1 + x2, each the rounding of what is left: 24 bits and more).
// Of the nine products of planes the six largest are added up; what is dropped is below 2^-24 of |x| |w|.
//
// The tensor core's additions to an accumulator drop what fp32 cannot hold instead of rounding it: a sum of n
// instructions (16 of r each) comes out about 0.75 n 2^-24 too near to zero (measured: 56 of them 2.5e-6, 256 1.2e-5),
// which a bf16 result does not show and an fp32 one does.  So where results are fp32, or sums as long as a batch
// or past kLongSum (kFlush), an accumulator is read back every few blocks and added up in registers, with rounding.  With planes, the
// product of the first ones has an accumulator of its own, flushed every kMainBlocks; the five small ones, 2^-8 of it
// and less, share the other, flushed every kCrossBlocks.
//
// PAIR: two CTAs of a cluster share one 256 x 256 tile (cta_group::2), each holding 128 rows of either operand and
// 128 rows of the accumulator: 32 KB an SM for 512 cycles of products, what an SM's share of L2 can bring.  A single
// CTA takes 128 x 128.
//
// Roles: warp 0 loads the operand tiles into a ring of stages; warp 1 of the issuing CTA owns the MMAs, into two
// accumulators in turn; 8 warps read them back, a thread one row (TMEM lane) and half of the columns, 32 at a time.
// A warp's results pass through shared memory as pieces of 32 rows x 128 bytes and leave by TMA (stores from the threads:
// 65536 x 1024 x 1024 bf16 with silu and residual 119 us against 104); but those of an fp32 pre, whose place y waits for,
// by the threads, a line at a time: such a store waits behind the operands' loads, and its place is free 2000 cycles
// later.  Residual pieces come by TMA, a tile ahead.  Matrices whose rows are not 16-byte aligned go element by element,
// consecutive columns together.
// Every mbarrier wait is bounded by a wall-clock limit; on expiry the kernel records CTR_ERR_TIMEOUT, waits (bounded)
// for its own copies and MMAs, frees TMEM and returns.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "dense_mm.cuh"
#include "rows.cuh"
#include "tc.cuh"

namespace ctr {
namespace {

constexpr int kOutWarps = 8;
constexpr int kDmThreads = 128 + 32 * kOutWarps;  // warps 0..3: loads, MMAs, none, none; then the epilogue
constexpr int kRows = 128;                        // rows of either operand that a CTA holds
constexpr int kBlock = 64;                        // of r to a block: one 128-byte swizzled row of bf16
constexpr uint32_t kTileBytes = kRows * kBlock * 2;
constexpr uint32_t kChunkBytes = 64 * 128;        // MN-major: 64 of i or j times 64 of r
constexpr uint32_t kPiece = 32 * 128;             // a warp's piece of the result on its way: 32 rows of 128 bytes
constexpr int kSuper = 8;                         // row tiles that take the column tiles together
constexpr int kMinShare = 8;                      // blocks of a part of a sum, at least
constexpr int kPairBlocks = 64;                   // blocks of a sum that pairs cut up whatever the number of tiles
constexpr int kMainBlocks = 2, kCrossBlocks = 64; // blocks between two readings (planes): 8 and 1280 instructions
constexpr int kFlushBlocks = 8;                   // without planes: 32 instructions
// Forward and input gradient without planes sum up to this many terms in the accumulator alone: 1.8e-4 too near to zero at most, a
// tenth of a bf16 result's rounding (4096 x 4096 x 65536 1440 us, 64 more terms, read back, 1460).
constexpr int64_t kLongSum = 65536;
// Registers of a kFlush kernel: 384 threads are launched with 168 each; the first four warps give some up so that an
// epilogue thread can hold 128 sums beside the 64 values that it adds.  56 x 128 + 224 x 256 = 168 x 384.
constexpr int kLaunchRegs = 168, kControlRegs = 56, kOutRegs = 224;
static_assert(kControlRegs * 128 + kOutRegs * 32 * kOutWarps <= kLaunchRegs * kDmThreads, "more registers than launched");

// BN: columns of a tile: 256 of a pair, 128, or 32 (with 128 rows).
template <int PLANES, int BN>
struct Shape {
  static constexpr uint32_t b_bytes = (BN == 256 ? 128 : BN) * kBlock * 2;  // of the right operand that a CTA holds
  static constexpr int stages = BN == 32 ? (PLANES == 1 ? 16 : 8) : PLANES == 1 ? 4 : 2;  // at most
  static constexpr uint32_t stage_bytes = PLANES * (kTileBytes + b_bytes);
  static constexpr int parts = BN == 32 ? 1 : 2;  // epilogue warps that share a row
  // Places for pieces of an epilogue warp.  Three: pieces of y (and their residual) take the first two in turn, those of
  // pre the third.  One: each piece of pre leaves before that of y takes its place.
  static constexpr int places = PLANES == 1 ? 3 : 1;
  static constexpr int turns = PLANES == 1 ? 2 : 1;
  static constexpr uint32_t room = 4 * parts * places * kPiece;  // all epilogue warps'
  static constexpr int smem = BN == 32 ? 226 * 1024 : (int)(1024 + stages * stage_bytes + room);
};
static_assert(Shape<1, 256>::smem <= 231 * 1024 && Shape<3, 256>::smem <= 231 * 1024, "more shared memory than a CTA has");

struct DmArgs {
  char* out;
  const char* res;
  char* pre;
  const char* bias;
  int* err;
  int64_t ldo, ldr, ldp;      // in elements
  int32_t m, n, kb, mt, nt, tiles, act;
  int32_t share, parts;       // 0, or blocks of a part of a sum, and parts of a tile
  // Of a tile of 32 columns: rows of the left operand that are there (else 128), and how many stages fit.
  int32_t a_rows, stages;
  int32_t f32, bias_f32;      // type of out, residual and pre; of the bias
  // Rows are 16-byte aligned: TMA moves them.  It writes whole 16-byte parts, past the end of a row that ends inside
  // one: 1 where rows do, and the last columns go element by element; 2 where they do not, or may be written past.
  int32_t wide_out, wide_res, wide_pre;
};

// kind::f16 instruction descriptor: bf16 x bf16 -> fp32; bits 15 and 16: A and B MN-major.
__host__ __device__ constexpr uint32_t idesc_dense(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// MN-major operand, 128-byte swizzle: chunks of 64 kChunkBytes apart, groups of 8 of r 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
  uint64_t d = 0;
  d |= (uint64_t)((addr & 0x3FFFF) >> 4);
  d |= (uint64_t)(kChunkBytes >> 4) << 16;  // leading byte offset
  d |= (uint64_t)(1024 >> 4) << 32;         // stride byte offset
  d |= (uint64_t)1 << 46;                   // descriptor version
  d |= (uint64_t)2 << 61;                   // SWIZZLE_128B
  return d;
}

template <bool PAIR>
__device__ __forceinline__ void mma_dense(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// A box of a 3D map into this CTA's shared memory, counted at `bar` (of the pair's even CTA).
template <bool PAIR>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2,
                                         uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"((uint64_t)map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"((uint64_t)map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void store_box(const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"((uint64_t)map),
               "r"(c0), "r"(c1), "r"(c2), "r"(src)
               : "memory");
}
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// One operand's block of all planes: rows i0 .. i0 + 127, r0 .. r0 + 63.
template <bool PAIR, bool MN, int PLANES>
__device__ __forceinline__ void load_operand(uint32_t dst, uint32_t plane, const CUtensorMap* map, int32_t i0, int32_t r0,
                                             uint32_t bar) {
#pragma unroll
  for (int pl = 0; pl < PLANES; ++pl) {
    if constexpr (MN) {
      load_box<PAIR>(dst + pl * plane, map, i0, r0, pl, bar);
      load_box<PAIR>(dst + pl * plane + kChunkBytes, map, i0 + 64, r0, pl, bar);
    } else {
      load_box<PAIR>(dst + pl * plane, map, r0, i0, pl, bar);
    }
  }
}

struct DmTile {
  int32_t nkb, k0;            // blocks of r to sum, the first of them
  int32_t a_row, b_row, col;  // this CTA's first row of either operand; first column of the result
  int32_t slot;               // the part's place
};

// A worker's way through the tiles: every step-th one.  Where sums are cut, the tiles of the first `share` blocks of r
// come first, then those of the next: workers that run at once share what they read.  (Shares that end and begin inside
// tiles, so that all workers have the same, read it again and again: 65536 x 1024 x 1024 123 us against 100.)
template <int BN>
struct Walk {
  static constexpr bool PAIR = BN == 256;
  static constexpr int kSide = PAIR ? 256 : 128;  // rows of a tile
  const DmArgs& p;
  int rank, step, at, end;
  __device__ __forceinline__ Walk(const DmArgs& args, int r) : p(args), rank(r) {
    at = blockIdx.x / (PAIR ? 2 : 1);
    step = gridDim.x / (PAIR ? 2 : 1);
    end = p.tiles * (p.share ? p.parts : 1);
  }
  __device__ __forceinline__ bool more() const { return at < end; }
  __device__ __forceinline__ DmTile tile() const {
    DmTile x;
    const int cut = at / p.tiles, l = at - cut * p.tiles;
    x.k0 = cut * p.share;
    x.nkb = p.share ? min(p.share, p.kb - x.k0) : p.kb;
    x.slot = at;
    const int sg = l / (kSuper * p.nt);
    const int rem = l - sg * (kSuper * p.nt);
    const int mm = min(kSuper, p.mt - sg * kSuper);
    const int ni = rem / mm;
    const int mi = sg * kSuper + rem - ni * mm;
    x.a_row = mi * kSide + rank * kRows;
    x.col = ni * BN;
    x.b_row = x.col + (PAIR ? rank * kRows : 0);
    return x;
  }
  __device__ __forceinline__ void go() { at += step; }
};

// sum += v for 32 values, two at a time.  volatile: stays after the wait for the load of v.
__device__ __forceinline__ void add32(float* sum, const uint32_t (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 2)
    asm volatile(
        "{\n\t.reg .b64 a, t;\n\t"
        "mov.b64 a, {%0, %1};\n\t"
        "mov.b64 t, {%2, %3};\n\t"
        "add.rn.f32x2 a, a, t;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "+f"(sum[i]), "+f"(sum[i + 1])
        : "r"(v[i]), "r"(v[i + 1]));
}

__device__ __forceinline__ float bias_at(const DmArgs& p, int col) {
  if (!p.bias || col >= p.n) return 0.f;
  return p.bias_f32 ? ((const float*)p.bias)[col] : __bfloat162float(((const __nv_bfloat16*)p.bias)[col]);
}

// A piece to its matrix: rows row0 .. row0 + nrows - 1, columns from col on.  wide: rows are 16-byte aligned, and eight
// lanes store 128 bytes of a row; else a warp's lanes store consecutive columns.
template <typename E>
__device__ __forceinline__ void piece_out(const uint8_t* piece, char* to, int64_t ld, int64_t row0, int nrows, int col, int n,
                                          bool wide) {
  constexpr int width = 128 / (int)sizeof(E), per = 16 / (int)sizeof(E);
  const int lane = threadIdx.x & 31;
  if (wide) {
    const int part = lane & 7, c = col + part * per;
    E* out = (E*)to + (row0 + (lane >> 3)) * ld + c;
#pragma unroll
    for (int r = lane >> 3; r < 32; r += 4, out += 4 * ld) {
      const uint4 v = *(const uint4*)(piece + r * 128 + ((part ^ (r & 7)) * 16));
      if (r >= nrows) continue;
      if (c + per <= n) {
        *(uint4*)out = v;
      } else {
        const E* e = (const E*)&v;
#pragma unroll
        for (int i = 0; i < per; ++i)
          if (c + i < n) out[i] = e[i];
      }
    }
  } else {
    E* out = (E*)to + row0 * ld + col;
#pragma unroll
    for (int e = lane; e < width; e += 32)
      if (col + e < n)
        for (int r = 0; r < nrows; ++r)
          out[r * ld + e] = *(const E*)(piece + r * 128 + (((e / per) ^ (r & 7)) * 16) + (e % per) * sizeof(E));
  }
}
// A piece of a matrix whose rows are not 16-byte aligned.
template <typename E>
__device__ __forceinline__ void piece_in(uint8_t* piece, const char* from, int64_t ld, int64_t row0, int nrows, int col, int n) {
  constexpr int width = 128 / (int)sizeof(E), per = 16 / (int)sizeof(E);
  const int lane = threadIdx.x & 31;
  const E* in = (const E*)from + row0 * ld + col;
#pragma unroll
  for (int e = lane; e < width; e += 32)
#pragma unroll 8
    for (int r = 0; r < 32; ++r)
      *(E*)(piece + r * 128 + (((e / per) ^ (r & 7)) * 16) + (e % per) * sizeof(E)) =
          r < nrows && col + e < n ? in[r * ld + e] : (E)0;
}

constexpr bool flushes(int major, int planes) { return planes == 3 || major == 2; }

template <int BN, int MAJOR, int PLANES, bool LONG>
__global__ void __launch_bounds__(kDmThreads, 1)
    dense_mm_kernel(const DmArgs p, const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                    const __grid_constant__ CUtensorMap omap, const __grid_constant__ CUtensorMap rmap,
                    const __grid_constant__ CUtensorMap pmap) {
  using S = Shape<PLANES, BN>;
  constexpr bool PAIR = BN == 256;
  static_assert(BN != 32 || MAJOR == 0, "32 columns of an MN-major operand are half a row of its layout");
  constexpr bool kAmn = MAJOR == 2, kBmn = MAJOR >= 1;
  constexpr bool kFlush = flushes(MAJOR, PLANES) || LONG;
  constexpr int kBN = BN;
  constexpr int kCols = kBN / S::parts;  // columns of an epilogue thread
  constexpr int kCtas = PAIR ? 2 : 1;
  // Of few rows a stage holds those that are there, so that more of them are on their way.  The products read on past
  // them, into what comes next in shared memory: rows of the accumulator that nobody reads.
  const uint32_t a_bytes = BN == 32 ? (uint32_t)p.a_rows * (kBlock * 2) : kTileBytes;
  const uint32_t stage_bytes = BN == 32 ? PLANES * (a_bytes + S::b_bytes) : S::stage_bytes;
  const int stages = BN == 32 ? p.stages : S::stages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[2 * S::stages + 5 + 2 * kOutWarps];
  __shared__ uint32_t tmem_base_slot;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // swizzled tiles need 1024-byte alignment
  const uint32_t full0 = smem_u32(&bars[0]);                      // a stage's operands are there (pair: the even CTA's)
  const uint32_t empty0 = smem_u32(&bars[S::stages]);             // a stage's MMAs are done
  const uint32_t tfull0 = smem_u32(&bars[2 * S::stages]);         // an accumulator is complete
  const uint32_t tempty0 = smem_u32(&bars[2 * S::stages + 2]);    // an accumulator has been read (pair: the even CTA's)
  const uint32_t rfull0 = smem_u32(&bars[2 * S::stages + 4]);     // a piece of residual is there, two a warp
  const uint32_t drained = rfull0 + 16 * kOutWarps;               // all MMAs are done
  uint32_t rank = 0;
  if constexpr (PAIR) asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, kCtas * 4 * S::parts);
    }
    for (int w = 0; w < 2 * kOutWarps; ++w) mbar_init(rfull0 + 8 * w, 1);
    mbar_init(drained, 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc<PAIR>(smem_u32(&tmem_base_slot), 2 * kBN);
  grid_wait();
  fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // the other CTA's barriers are ready too
  fence_after();
  const uint32_t tmem = tmem_base_slot;

  if (warp < 4) {
    if constexpr (kFlush) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
    if (warp == 0) {
      // ---------------- TMA producer ----------------
      const uint32_t count_at = PAIR ? in_cta(full0, 0) : full0;
      int s = 0;
      uint32_t ph = 0, issued = 0;  // issued: blocks so far, at most stages counted
      bool ok = true;
      DmTile x;
      for (Walk<BN> way(p, (int)rank); ok && way.more(); way.go()) {
        x = way.tile();
        for (int j = 0; j < x.nkb; ++j) {
          if (!park(empty0 + 8 * s, ph ^ 1)) {
            if (lane == 0) set_error(p.err, CTR_ERR_TIMEOUT);
            ok = false;
            break;
          }
          const uint32_t dst = base + (uint32_t)s * stage_bytes;
          const int32_t r0 = (x.k0 + j) * kBlock;
          if (elected()) {
            if (rank == 0) mbar_expect_tx(full0 + 8 * s, kCtas * stage_bytes);
            load_operand<PAIR, kAmn, PLANES>(dst, a_bytes, &amap, x.a_row, r0, count_at + 8 * s);
            load_operand<PAIR, kBmn, PLANES>(dst + PLANES * a_bytes, S::b_bytes, &bmap, x.b_row, r0, count_at + 8 * s);
          }
          __syncwarp();
          if (issued < stages) ++issued;
          if (++s == stages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      // drain: every issued load must have landed before the CTA can exit.  The last round's MMAs free the stages;
      // after a failure no MMA may come, and a stage's own barrier says that it is filled (a pair's odd CTA has none
      // and waits the limit out).
      for (uint32_t i = 0; i < issued; ++i) {
        s = s == 0 ? stages - 1 : s - 1;
        if (s == stages - 1) ph ^= 1;
        if (!park((ok || rank != 0 ? empty0 : full0) + 8 * s, ph) && lane == 0) set_error(p.err, CTR_ERR_TIMEOUT);
      }
    } else if (warp == 1) {
      if (rank == 0) {
        // ---------------- MMA issuer ----------------
        constexpr uint32_t idesc = idesc_dense(kCtas * kRows, kBN, kAmn, kBmn);
        // planes of the small products, the smallest first
        constexpr int kPa[5] = {2, 0, 1, 1, 0}, kPb[5] = {0, 2, 1, 0, 1};
        // 16 of r further: 32 bytes along K-major rows, 16 rows of 128 bytes in MN-major chunks (in units of 16 bytes)
        constexpr uint32_t kStepA = kAmn ? 128 : 2, kStepB = kBmn ? 128 : 2;
        const uint64_t a0 = kAmn ? desc_mn(base) : smem_desc_sw128(base);
        const uint64_t b0 = kBmn ? desc_mn(base + PLANES * a_bytes) : smem_desc_sw128(base + PLANES * a_bytes);
        int s = 0;
        // Without planes the two accumulators take turns, b's phase bph.  With planes, the first (phase bph) has the main
        // products, the other (phase cph) the rest.
        uint32_t ph = 0, b = 0, bph = 0, cph = 0;
        bool ok = true;
        DmTile x;
        for (Walk<BN> way(p, 0); ok && way.more(); way.go()) {
          x = way.tile();
          const int nkb = x.nkb;
          for (int j = 0; ok && j < nkb; ++j) {
            const int every = !kFlush ? nkb : PLANES == 3 ? kMainBlocks : kFlushBlocks;
            const bool opens = j % every == 0, closes = (j + 1) % every == 0 || j + 1 == nkb;
            const bool copens = PLANES == 3 && j % kCrossBlocks == 0;
            const bool ccloses = PLANES == 3 && ((j + 1) % kCrossBlocks == 0 || j + 1 == nkb);
            if (copens) ok = park(tempty0 + 8, cph ^ 1);
            if (PLANES == 1 && opens) ok = ok && park(tempty0 + 8 * b, bph ^ 1);
            ok = ok && park(full0 + 8 * s, ph);
            if (!ok) break;
            fence_after();
            const uint64_t at = (uint64_t)((uint32_t)s * (stage_bytes >> 4));
            if constexpr (PLANES == 3) {
              // the small products first: they need not wait until the main accumulator has been read
              if (elected()) {
#pragma unroll
                for (int q = 0; q < 5; ++q)
#pragma unroll
                  for (int k = 0; k < kBlock / 16; ++k)
                    mma_dense<PAIR>(tmem + kBN, a0 + at + kPa[q] * (a_bytes >> 4) + k * kStepA,
                                    b0 + at + kPb[q] * (S::b_bytes >> 4) + k * kStepB, idesc, !copens || (q | k) != 0);
              }
              __syncwarp();
              if (opens) ok = park(tempty0, bph ^ 1);
              if (!ok) break;
              fence_after();
            }
            if (elected()) {
#pragma unroll
              for (int k = 0; k < kBlock / 16; ++k)
                mma_dense<PAIR>(tmem + b * kBN, a0 + at + k * kStepA, b0 + at + k * kStepB, idesc, !opens || k != 0);
              commit<PAIR>(empty0 + 8 * s);
              if (closes) commit<PAIR>(tfull0 + 8 * b);
              if (ccloses) commit<PAIR>(tfull0 + 8);
            }
            __syncwarp();
            if (closes) {
              bph ^= PLANES == 3 ? 1 : b;
              b ^= PLANES == 3 ? 0 : 1;
            }
            if (ccloses) cph ^= 1;
            if (++s == stages) {
              s = 0;
              ph ^= 1;
            }
          }
          if (!ok && lane == 0) set_error(p.err, CTR_ERR_TIMEOUT);
        }
        // drain: all MMAs must be done before TMEM is freed, those too that a failure left without a reader
        if (elected()) commit<PAIR>(drained);
        __syncwarp();
        if (!park(drained, 0) && lane == 0) set_error(p.err, CTR_ERR_TIMEOUT);
      }
    }
  } else {
    if constexpr (kFlush) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kOutRegs));
    // ---------------- epilogue ----------------
    const int q = warp & 3;            // TMEM lane quarter this warp may read
    const int part = (warp - 4) >> 2;  // which half of the columns
    const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(part * kCols);
    uint8_t* staging = smem_raw + (base - raw) + stages * stage_bytes + (warp - 4) * (S::places * kPiece);
    const uint32_t rfull = rfull0 + 16 * (warp - 4);
    const uint32_t tempty_at = PAIR ? in_cta(tempty0, 0) : tempty0;
    const bool f32 = MAJOR == 2 ? p.f32 != 0 : PLANES == 3;  // type of the results
    const int width = f32 ? 32 : 64;                         // columns of a piece
    const bool has_bias = MAJOR == 0 && p.bias, has_res = MAJOR == 0 && p.res, has_pre = MAJOR == 0 && p.pre;
    const bool wide_res = MAJOR == 0 && p.wide_res;
    uint32_t b = 0, ph = 0, cph = 0;  // accumulators, as the MMAs' issuer has them
    uint32_t rph = 0, flying = 0;     // phases of the residual's barriers, and which are awaited
    bool ok = true;
    // The warp's part of a tile.
    struct Part {
      int64_t row0;
      int nrows, col0, cols;  // cols: to do (may be <= 0)
    };
    auto part_of = [&](const DmTile& x) {
      Part r;
      if (p.share) {  // parts are whole tiles, one below the other
        r.row0 = (int64_t)x.slot * (kCtas * kRows) + rank * kRows + q * 32;
        r.nrows = 32;
        r.col0 = part * kCols;
        r.cols = kCols;
        return r;
      }
      r.row0 = x.a_row + q * 32;
      r.nrows = (int)imin64(32, p.m - r.row0);
      r.col0 = x.col + part * kCols;
      r.cols = r.nrows <= 0 ? 0 : min(kCols, p.n - r.col0);
      return r;
    };
    auto ask = [&](int place, int64_t row0, int col) {  // a piece of residual into a place that is free
      if (PLANES == 3) {  // whose last readers were threads
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }
      if (lane == 0) {
        mbar_expect_tx(rfull + 8 * place, kPiece);
        load_box<false>(smem_u32(staging + place * kPiece), &rmap, col, (int32_t)row0, 0, rfull + 8 * place);
      }
      flying |= 1u << place;
    };
    // A piece of residual for a place that is being read out: asked for when the next piece has begun.
    struct Later {
      int place, col;
      int64_t row0;
    } later = {-1, 0, 0};
    auto ask_later = [&] {
      if (lane == 0) bulk_wait_read<0>();
      __syncwarp();
      ask(later.place, later.row0, later.col);
      later.place = -1;
    };
    // The first pieces of residual.  Later ones, the next tile's too, are asked for as their places become free: asked for
    // at their tile's start, they took 1 us of every tile.
    Walk<BN> way(p, (int)rank);
    if (wide_res && part < S::parts && way.more()) {
      const Part f = part_of(way.tile());
      for (int h = 0; h < S::turns; ++h)
        if (h * width < f.cols) ask(h, f.row0, f.col0 + h * width);
    }
    while (ok && part < S::parts && way.more()) {
      const DmTile x = way.tile();
      way.go();
      const Part me = part_of(x);
      const int64_t row0 = me.row0;
      const int nrows = me.nrows, col0 = me.col0, cols = me.cols;
      Part ahead = {};
      if (wide_res && way.more()) ahead = part_of(way.tile());
      auto give = [&](uint32_t acc) {  // an accumulator has been read: the next MMAs may have it
        fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank == 0) mbar_arrive(tempty0 + 8 * acc);
          else arrive_at(tempty_at + 8 * acc);
        }
      };
      float sum[kFlush ? kCols : 1];
      if constexpr (kFlush) {
#pragma unroll
        for (int i = 0; i < kCols; ++i) sum[i] = 0.f;
        auto add = [&](uint32_t acc, uint32_t parity) {
          if (!park(tfull0 + 8 * acc, parity)) return false;
          fence_after();
          // 64 columns at once; with planes, or activations, whose epilogue has more to hold, 32 (spills go to L2: all but nothing is left of
          // L1 beside the operands)
          constexpr int kStep = PLANES == 3 || LONG || kCols < 64 ? 32 : 64;
#pragma unroll
          for (int c = 0; c < kCols; c += kStep) {
            uint32_t v0[32], v1[32];
            tmem_ld32_async(lane_base + acc * kBN + c, v0);
            if (kStep == 64) tmem_ld32_async(lane_base + acc * kBN + c + 32, v1);
            tmem_wait_ld();
            if (c + kStep == kCols) give(acc);
            add32(sum + c, v0);
            if (kStep == 64) add32(sum + c + 32, v1);
          }
          return true;
        };
        for (int j = 0; ok && j < x.nkb;) {
          if constexpr (PLANES == 3) {
            const int end = min(x.nkb, j + kCrossBlocks);
            for (; ok && j < end; j += kMainBlocks, ph ^= 1) ok = add(0, ph);
            j = end;
            ok = ok && add(1, cph);
            cph ^= 1;
          } else {
            ok = add(b, ph);
            ph ^= b;
            b ^= 1;
            j += kFlushBlocks;
          }
        }
      } else {
        ok = park(tfull0 + 8 * b, ph);
        fence_after();
      }
      if (!ok) {
        if (lane == 0) set_error(p.err, CTR_ERR_TIMEOUT);
        break;
      }
      int place = 0;
      // columns c .. c + 31 of the tile's part, whose sums are v once `get` has run
      auto leave32 = [&](int c, uint32_t (&v)[32], auto get) {
        const int col = col0 + c;
        const int half = f32 ? 0 : (c >> 5) & 1;
        uint8_t* piece = staging + place * kPiece;
        if (half == 0) {
          if (wide_res) {
            if (later.place == place) ask_later();
            ok = park(rfull + 8 * place, (rph >> place) & 1);
            if (!ok) {
              if (lane == 0) set_error(p.err, CTR_ERR_TIMEOUT);
              return;
            }
            rph ^= 1u << place;
            flying &= ~(1u << place);
          } else {
            // the place is free: all pieces have left, or (places in turn, within a tile) all but the newest
            if (lane == 0) {
              if (S::turns == 2 && c > 0) bulk_wait_read<1>();
              else bulk_wait_read<0>();
            }
            __syncwarp();
            if (has_res) {
              if (f32) piece_in<float>(piece, p.res, p.ldr, row0, nrows, col, p.n);
              else piece_in<uint16_t>(piece, p.res, p.ldr, row0, nrows, col, p.n);
              __syncwarp();
            }
          }
        }
        get();
        if (later.place >= 0) ask_later();
        const float bias = has_bias ? bias_at(p, col + lane) : 0.f;
        uint8_t* row = piece + lane * 128;
        auto leave = [&](const CUtensorMap* map, int wide, char* to, int64_t ld, const uint8_t* from, int at) {
          if (kCols < 64 && !f32) {  // half a piece
            __syncwarp();
            piece_out<uint16_t>(from, to, ld, row0, nrows, at, min(p.n, at + kCols), wide != 0);
          } else if (wide == 2 || (wide == 1 && at + width <= p.n)) {
            if (lane == 0) store_box(map, at, (int32_t)row0, 0, smem_u32(from));
          } else if (f32) {
            piece_out<float>(from, to, ld, row0, nrows, at, p.n, false);
          } else {
            piece_out<uint16_t>(from, to, ld, row0, nrows, at, p.n, false);
          }
        };
        // All 32 at once: a thread's chains of exponentials and reciprocals hide each other's latency (8 at a time:
        // 65536 x 1024 x 1024 with silu 110 us).
        float z[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) z[i] = __uint_as_float(v[i]);
        if (has_bias) {
#pragma unroll
          for (int i = 0; i < 32; ++i) z[i] += __shfl_sync(kFull, bias, i);
        }
        if (f32) {
          float4 res[8];
          if (has_res) {
#pragma unroll
            for (int i = 0; i < 8; ++i) res[i] = *(const float4*)(row + ((i ^ (lane & 7)) * 16));
          }
          if (has_pre) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *(float4*)(row + ((i ^ (lane & 7)) * 16)) = make_float4(z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]);
            // by the threads: y takes its place at once
            __syncwarp();
            piece_out<float>(piece, p.pre, p.ldp, row0, nrows, col, p.n, p.wide_pre != 0);
            __syncwarp();
          }
          if constexpr (MAJOR == 0) activate<std::conditional_t<PLANES == 3, float, __nv_bfloat16>>(p.act, z);
          if (has_res) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              z[4 * i] += res[i].x;
              z[4 * i + 1] += res[i].y;
              z[4 * i + 2] += res[i].z;
              z[4 * i + 3] += res[i].w;
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *(float4*)(row + ((i ^ (lane & 7)) * 16)) = make_float4(z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]);
        } else {
          auto pack8 = [&](int g) {
            return make_uint4(bf16_pair(z[8 * g], z[8 * g + 1]), bf16_pair(z[8 * g + 2], z[8 * g + 3]),
                              bf16_pair(z[8 * g + 4], z[8 * g + 5]), bf16_pair(z[8 * g + 6], z[8 * g + 7]));
          };
          const auto at = [&](int g) { return (uint32_t)(((4 * half + g) ^ (lane & 7)) * 16); };
          if (S::places == 3 && has_pre) {
            if (half == 0) {  // pre's place is free
              if (lane == 0) bulk_wait_read<0>();
              __syncwarp();
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) *(uint4*)(staging + 2 * kPiece + lane * 128 + at(g)) = pack8(g);
          }
          if constexpr (MAJOR == 0) activate<std::conditional_t<PLANES == 3, float, __nv_bfloat16>>(p.act, z);
          if (has_res) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              float r[8];
              Chunk<__nv_bfloat16, 16>::unpack(*(const uint4*)(row + at(g)), r);
#pragma unroll
              for (int i = 0; i < 8; ++i) z[8 * g + i] += r[i];
            }
          }
#pragma unroll
          for (int g = 0; g < 4; ++g) *(uint4*)(row + at(g)) = pack8(g);
        }
        if (half == 0 && !f32 && c + 32 < cols) return;
        // the piece is complete
        const int at = col - 32 * half;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        leave(&omap, p.wide_out, p.out, p.ldo, piece, at);
        if (S::places == 3 && has_pre) leave(&pmap, p.wide_pre, p.pre, p.ldp, staging + 2 * kPiece, at);
        if (lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        if (wide_res) {
          // what comes here next: this tile's piece after the next ones, or the next tile's of the same turn
          const int next = at - col0 + S::turns * width;
          const bool here = next < cols;
          const int col = here ? next : place * width;
          if (here || col < ahead.cols) later = {place, (here ? col0 : ahead.col0) + col, here ? row0 : ahead.row0};
        }
        if (S::turns == 2) place ^= 1;
      };
      if constexpr (kFlush) {
        // With activations one copy of the code, the sums moving up: four are more than the instruction cache holds (fp32
        // 16384 x 1024 x 1024 with gelu and pre 292 us).
        if constexpr (MAJOR == 0) {
#pragma unroll 1
          for (int c = 0; ok && c < cols; c += 32) {
            uint32_t v[32];
            leave32(c, v, [&] {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(sum[i]);
            });
#pragma unroll
            for (int i = 0; i < kCols - 32; ++i) sum[i] = sum[i + 32];
          }
        } else {
#pragma unroll
          for (int c = 0; c < kCols; c += 32)
            if (ok && c < cols) {
              uint32_t v[32];
              leave32(c, v, [&] {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(sum[c + i]);
              });
            }
        }
      } else {
        for (int c = 0; ok && c < cols; c += 32) {
          uint32_t v[32];
          leave32(c, v, [&] { tmem_ld32(lane_base + b * kBN + c, v); });
        }
      }
      if (!ok) break;
      // places that this tile had no piece for
      if (wide_res)
        for (int h = 0; h < S::turns; ++h)
          if (h * width >= cols && h * width < ahead.cols) {
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
            ask(h, ahead.row0, ahead.col0 + h * width);
          }
      if constexpr (!kFlush) {
        give(b);
        ph ^= b;
        b ^= 1;
      }
    }
    for (int place = 0; place < S::places; ++place)
      if ((flying >> place) & 1) {
        if (!park(rfull + 8 * place, (rph >> place) & 1) && lane == 0) set_error(p.err, CTR_ERR_TIMEOUT);
      }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // nothing of this CTA is the other's target any more
  if (warp == 1) {
    fence_after();
    tmem_free<PAIR>(tmem, 2 * kBN);
  }
}

// ---------------------------------------------------------------------------
// Sums in parts: a tile's parts added in their order, four columns of one row to a thread.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kJoinThreads) join_parts_kernel(const DmArgs p, const float* part, int side, T* out,
                                                                  int64_t ldo, int vec) {
  grid_wait();
  const int64_t quads = (p.n + 3) / 4, e = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;
  const int row = (int)(e / quads), c = (int)(e - row * quads) * 4;
  if (row >= p.m) return;
  const int mi = row / side, ni = c / side;
  // the tile's number, as Walk has it
  const int sg = mi / kSuper;
  const int64_t t = (int64_t)sg * kSuper * p.nt + ni * min(kSuper, p.mt - sg * kSuper) + (mi - sg * kSuper);
  const int64_t place = (int64_t)side * side, next = place * p.mt * p.nt;
  const float* from = part + t * place + (row - mi * side) * side + (c - ni * side);
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int i = 0; i < p.parts; ++i, from += next) {
    const float4 v = *(const float4*)from;
    sum.x += v.x;
    sum.y += v.y;
    sum.z += v.z;
    sum.w += v.w;
  }
  T* to = out + row * ldo + c;
  if (vec && c + 4 <= p.n) {
    if constexpr (sizeof(T) == 4) *(float4*)to = sum;
    else *(uint2*)to = make_uint2(bf16_pair(sum.x, sum.y), bf16_pair(sum.z, sum.w));
  } else {
    const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < p.n) to[i] = from_f32<T>(v[i]);
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
// Planes of [outer][inner] bf16 in boxes of 64 x `box`.
bool operand_map(CUtensorMap* map, const MmOperand& o, int planes, int box) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t gdim[3] = {(cuuint64_t)o.inner, (cuuint64_t)o.outer, (cuuint64_t)planes};
  cuuint64_t gstride[2] = {(cuuint64_t)(o.ld * 2), (cuuint64_t)((planes > 1 ? o.plane : o.ld * o.outer) * 2)};
  cuuint32_t bx[3] = {64, (cuuint32_t)box, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(o.p), gdim, gstride, bx, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A result matrix [m][n] in pieces of 32 rows of 128 bytes.
bool piece_map(CUtensorMap* map, const void* p, bool f32, int64_t m, int64_t n, int64_t ld) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const int eb = f32 ? 4 : 2;
  cuuint64_t gdim[3] = {(cuuint64_t)n, (cuuint64_t)m, 1};
  cuuint64_t gstride[2] = {(cuuint64_t)(ld * eb), (cuuint64_t)(ld * m * eb)};
  cuuint32_t bx[3] = {(cuuint32_t)(128 / eb), 32, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), gdim,
             gstride, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How TMA may move a matrix's rows (DmArgs): 16-byte aligned, and strides that a map can hold.
int wide(const void* p, int64_t rows, int64_t cols, int64_t ld, int eb) {
  if (!p || ((uintptr_t)p % 16) != 0 || (ld * eb) % 16 != 0 || ld * eb * rows >= (1ll << 40)) return 0;
  return (cols * eb) % 16 == 0 ? 2 : 1;
}

DmArgs dm_args(const MmCall& c, const MmPlan& plan) {
  const int side = plan.side();
  DmArgs p = {};
  p.m = (int32_t)c.m;
  p.n = (int32_t)c.n;
  p.kb = (int32_t)ceil_div(c.r, kBlock);
  p.mt = (int32_t)ceil_div(c.m, side);
  p.nt = (int32_t)ceil_div(c.n, plan.columns);
  p.share = (int32_t)plan.share;
  p.parts = (int32_t)plan.parts;
  p.err = c.err;
  p.act = c.act;
  p.bias = (const char*)c.bias;
  p.bias_f32 = c.planes == 3;
  return p;
}

template <int BN, int MAJOR, int PLANES, bool LONG>
int launch_dm(const MmCall& c, const MmPlan& plan, float* part, cudaStream_t s) {
  constexpr int kCtas = BN == 256 ? 2 : 1, kSide = BN == 256 ? 256 : 128;
  using S = Shape<PLANES, BN>;
  DmArgs p = dm_args(c, plan);
  const int64_t tiles = (int64_t)p.mt * p.nt;
  if (tiles > INT32_MAX - 65536) return CTR_ERR_UNSUPPORTED;
  p.tiles = (int32_t)tiles;
  const int64_t workers = imin64(tiles * (plan.share ? plan.parts : 1), num_sms() / kCtas);
  int64_t out_rows = c.m, out_cols = c.n;
  if (plan.share) {
    p.out = (char*)part;
    p.f32 = 1;
    p.wide_out = 2;
    p.ldo = out_cols = kSide;
    out_rows = tiles * plan.parts * kSide;
  } else {
    p.out = (char*)c.out;
    p.ldo = c.ldo;
    p.f32 = c.out_f32;
    p.res = (const char*)c.residual;
    p.ldr = c.ld_res;
    p.pre = (char*)c.pre;
    p.ldp = c.ld_pre;
    const int eb = c.out_f32 ? 4 : 2;
    p.wide_out = wide(p.out, c.m, c.n, p.ldo, eb);
    p.wide_res = wide(p.res, c.m, c.n, p.ldr, eb);
    p.wide_pre = wide(p.pre, c.m, c.n, p.ldp, eb);
  }
  p.a_rows = BN == 32 ? (int)imin64(kRows, ceil_div(c.m, 8) * 8) : kRows;
  p.stages = (int)imin64(S::stages, (S::smem - 1024 - S::room) / (PLANES * (p.a_rows * kBlock * 2 + (int)S::b_bytes)));
  CUtensorMap amap, bmap;
  if (!operand_map(&amap, c.a, PLANES, MAJOR == 2 ? 64 : p.a_rows) || !operand_map(&bmap, c.b, PLANES, MAJOR >= 1 ? 64 : std::min(BN, kRows)))
    return CTR_ERR_CUDA;
  CUtensorMap omap = amap, rmap = amap, pmap = amap;  // not used unless the rows are aligned
  if (p.wide_out && !piece_map(&omap, p.out, p.f32 != 0, out_rows, out_cols, p.ldo)) return CTR_ERR_CUDA;
  if (p.wide_res && !piece_map(&rmap, p.res, p.f32 != 0, c.m, c.n, p.ldr)) return CTR_ERR_CUDA;
  if (p.wide_pre && !piece_map(&pmap, p.pre, p.f32 != 0, c.m, c.n, p.ldp)) return CTR_ERR_CUDA;
  auto k = dense_mm_kernel<BN, MAJOR, PLANES, LONG>;
  static std::atomic<uint64_t> ready{0};
  if (!once_per_device(ready, [&] {
        // the split of registers between the warps waits for ever if the kernel was launched with fewer
        cudaFuncAttributes fa;
        if (cudaFuncGetAttributes(&fa, k) != cudaSuccess || ((flushes(MAJOR, PLANES) || LONG) && fa.numRegs != kLaunchRegs)) return false;
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, S::smem) == cudaSuccess;
      }))
    return CTR_ERR_CUDA;
  const cudaError_t e = launch_after(k, dim3((unsigned)(kCtas * imax64(1, workers))), kDmThreads, S::smem, s, kCtas,
                                     p, amap, bmap, omap, rmap, pmap);
  return e == cudaSuccess ? launch_status() : CTR_ERR_CUDA;
}

template <int BN, int MAJOR>
int launch_dm(const MmCall& c, const MmPlan& plan, float* part, cudaStream_t s) {
  if (c.planes == 3) return launch_dm<BN, MAJOR, 3, false>(c, plan, part, s);
  if constexpr (MAJOR != 2 && BN != 32)
    if (c.r > kLongSum) return launch_dm<BN, MAJOR, 1, true>(c, plan, part, s);
  return launch_dm<BN, MAJOR, 1, false>(c, plan, part, s);
}

template <int MAJOR>
int launch_dm(const MmCall& c, const MmPlan& plan, float* part, cudaStream_t s) {
  if constexpr (MAJOR == 0)
    if (plan.columns == 32) return launch_dm<32, MAJOR>(c, plan, part, s);
  return plan.columns == 256 ? launch_dm<256, MAJOR>(c, plan, part, s) : launch_dm<128, MAJOR>(c, plan, part, s);
}

// CTA pairs, or CTAs, that run at once.
int64_t mm_workers(bool pair) { return imax64(1, num_sms() / (pair ? 2 : 1)); }

// Parts of a sum of kb blocks, at most: no fewer than kMinShare blocks each, and no more parts of all tiles than four
// rounds of the workers take.
int64_t most_parts(int64_t kb, int64_t tiles, int64_t workers) {
  return imax64(1, imin64(kb / kMinShare, 3 * workers / tiles + 1));
}

}  // namespace

MmPlan mm_plan(int major, int planes, int64_t m, int64_t n, int64_t r) {
  MmPlan w;
  const int64_t kb = ceil_div(r, kBlock);
  const int64_t pairs = ceil_div(m, 256) * ceil_div(n, 256);
  const int64_t sms = num_sms();
  const bool pair = m > 128 && n > 128 && (pairs >= sms / 3 || (major == 2 && kb >= kPairBlocks));
  if (pair) w.columns = 256;
  const int64_t side = w.side(), most = mm_workers(pair);
  const int64_t tiles = ceil_div(m, side) * ceil_div(n, side);
  // few rows: more and narrower tiles, so that more SMs read the weights
  const bool readback = planes == 1 && r > kLongSum;  // which those tiles have not
  if (!pair && major == 0 && 2 * tiles <= sms && n > 32 && !readback) w.columns = 32;
  if (major != 2) return w;
  // Sums over a batch are cut into the number of parts that takes least, in blocks' times (0.27 us with planes of bf16
  // alone): the rounds of all workers, six blocks for each tile's setting up and end, and each part's writing and reading.
  double best = 0;
  for (int64_t parts = 1; parts <= most_parts(kb, tiles, most); ++parts) {
    const double rounds = (double)ceil_div(tiles * parts, most);
    const double time = rounds * (planes * (planes == 3 ? 2 : 1) * (double)ceil_div(kb, parts) + 6) +
                        (parts > 1 ? (double)(tiles * parts) * (pair ? 0.28 : 0.14) + 8 : 0);
    if (parts == 1 || time < best) {
      best = time;
      w.share = parts > 1 ? ceil_div(kb, parts) : 0;
      w.parts = parts > 1 ? ceil_div(kb, w.share) : 1;
    }
  }
  return w;
}

size_t mm_room(int64_t m, int64_t n, int64_t r) {
  const int64_t kb = ceil_div(r, kBlock);
  int64_t most = 0;
  for (const bool pair : {false, true}) {
    // which of them a call takes depends on r
    if (pair && (m <= 128 || n <= 128)) continue;
    const int64_t side = pair ? 256 : 128, tiles = ceil_div(m, side) * ceil_div(n, side);
    const int64_t parts = most_parts(kb, tiles, mm_workers(pair));
    if (parts > 1) most = imax64(most, tiles * parts * side * side * 4);
  }
  return (size_t)most;
}

int mm_run(const MmCall& c, float* part, cudaStream_t s) {
  const MmPlan plan = mm_plan(c.major, c.planes, c.m, c.n, c.r);
  const int st = c.major == 0   ? launch_dm<0>(c, plan, part, s)
                 : c.major == 1 ? launch_dm<1>(c, plan, part, s)
                                : launch_dm<2>(c, plan, part, s);
  if (st != CTR_OK || !plan.share) return st;
  const int64_t blocks = ceil_div(c.m * ceil_div(c.n, 4), kJoinThreads);
  if (blocks > INT32_MAX) return CTR_ERR_UNSUPPORTED;
  const int eb = c.out_f32 ? 4 : 2;
  const int vec = ((uintptr_t)c.out % (4 * eb)) == 0 && c.ldo % 4 == 0;
  const DmArgs p = dm_args(c, plan);
  const dim3 grid((unsigned)blocks);
  const cudaError_t e =
      c.out_f32 ? launch_after(join_parts_kernel<float>, grid, kJoinThreads, 0, s, 1, p, (const float*)part, plan.side(),
                               (float*)c.out, c.ldo, vec)
                : launch_after(join_parts_kernel<__nv_bfloat16>, grid, kJoinThreads, 0, s, 1, p, (const float*)part,
                               plan.side(), (__nv_bfloat16*)c.out, c.ldo, vec);
  return e == cudaSuccess ? launch_status() : CTR_ERR_CUDA;
}

}  // namespace ctr
