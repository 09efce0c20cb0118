// b3. Products of e4m3 codes with a scale per block of 128, on the tensor cores.
//
//   out[r, i] = sum over blocks kb of  sa[r, kb] * sb[i / 128, kb] * S(r, i, kb),
//   S(r, i, kb) = sum over the block's 128 columns of a[r, c] * b[i, c]
//
// S is four tcgen05.mma (kind::f8f6f4, K = 32 each) into a fresh fp32 TMEM
// accumulator; the scaled sum over kb lives in registers.  Scales are arbitrary
// fp32 numbers, so they cannot ride in the instruction (which takes powers of
// two); what it costs is reading every block's accumulator back once: 128 x 256
// values at 128 lanes a clock, half the time that the block's products take, and
// hidden behind them.
//
// Roles (persistent CTAs, one per SM): warp 0 loads the 128-byte-wide operand
// tiles by TMA (128-byte swizzle, a ring of stages), warp 1 owns TMEM and issues
// the MMAs into two accumulators in turn, warps 2..9 scale and add: a thread
// owns one row (TMEM lane) and half of the tile's columns, so a row scale is one
// register and a block scale is uniform, and one packed multiply-add covers two
// values.  A tile's rows never leave their group: rows past it belong to the
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

constexpr int kMmThreads = 320;      // producer, issuer, 8 scaling warps
constexpr int kScaleWarps = 8;
constexpr int kBM = 128;             // rows of a tile
constexpr uint32_t kABytes = kBM * 128;
constexpr int kSuper = 8;            // row tiles that take the column tiles together
constexpr uint32_t kStageRow = 17;   // words of a staged row (16 data words), odd: no bank conflicts
constexpr uint32_t kStagingBytes = 32 * kStageRow * 4;

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
  int32_t out_f32, wide_rows;  // wide_rows: output rows start 32-byte aligned
};

// kind::f8f6f4 instruction descriptor: e4m3 x e4m3 -> fp32, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_e4m3(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// acc += f * v for 16 values, two at a time.  volatile: stays after the wait for the load of v.
__device__ __forceinline__ void scale_add16(uint64_t* acc, const uint32_t (&v)[16], uint64_t f2) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    asm volatile(
        "{\n\t.reg .b64 t;\n\t"
        "mov.b64 t, {%1, %2};\n\t"
        "fma.rn.f32x2 %0, t, %3, %0;\n\t}"
        : "+l"(acc[i])
        : "r"(v[2 * i]), "r"(v[2 * i + 1]), "l"(f2));
}

__device__ __forceinline__ void st_global_v8(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *(const uint32_t*)&h;
}

struct Tile {
  int32_t nkb;        // blocks to sum
  int32_t rows;       // rows of the tile inside the group
  int64_t a_row;      // first row of the left operand
  int64_t b_row;      // first row of the right operand
  int64_t k0;         // first block along the summed axis
  int64_t sb0;        // row of the block scales for the tile's first 128 columns
  int64_t out_row;    // first output row
  int32_t col;        // first column of the result
};

template <bool WGRAD>
__device__ __forceinline__ Tile locate(const MmArgs& p, const int32_t* start, int64_t t, int bn) {
  Tile x;
  int g, mi, ni;
  if constexpr (WGRAD) {
    const int64_t per = (int64_t)p.mt * p.nt;
    g = (int)(t / per);
    const int l = (int)(t - g * per);
    ni = l / p.mt;
    mi = l - ni * p.mt;
    x.nkb = start[g + 1] - start[g];
    x.k0 = start[g];
    x.rows = min(kBM, p.m - mi * kBM);
    x.a_row = (int64_t)mi * kBM;
    x.b_row = (int64_t)ni * bn;
    x.sb0 = (int64_t)ni * (bn / 128);
    x.out_row = (int64_t)g * p.m + mi * kBM;
  } else {
    const int64_t u = t / p.nt;
    int lo = 0, hi = p.groups - 1;  // the group whose row tiles [start[g], start[g+1]) hold u
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (start[mid] <= u) lo = mid;
      else hi = mid - 1;
    }
    g = lo;
    const int64_t l = t - (int64_t)start[g] * p.nt;
    const int mts = start[g + 1] - start[g];
    const int64_t per = (int64_t)kSuper * p.nt;
    const int sg = (int)(l / per);
    const int rem = (int)(l - sg * per);
    const int mm = min(kSuper, mts - sg * kSuper);
    ni = rem / mm;
    mi = sg * kSuper + rem - ni * mm;
    const int64_t r0 = p.offsets ? __ldg(p.offsets + g) : 0;
    const int64_t r1 = p.offsets ? __ldg(p.offsets + g + 1) : p.rows;
    x.nkb = p.kb;
    x.k0 = 0;
    x.rows = (int)imin64(kBM, r1 - r0 - (int64_t)mi * kBM);
    x.a_row = r0 + (int64_t)mi * kBM;
    x.b_row = (int64_t)g * p.n + (int64_t)ni * bn;
    x.sb0 = (int64_t)g * ((p.n + 127) / 128) + (int64_t)ni * (bn / 128);
    x.out_row = x.a_row;
  }
  x.col = ni * bn;
  return x;
}

// 128-row tiles before each group (start[groups] = all), by one warp.  Bad offsets: all zero and flagged.
__device__ __forceinline__ void group_starts(const MmArgs& p, int32_t* start) {
  const int lane = threadIdx.x & 31;
  if (!p.offsets) {
    if (lane == 0) {
      start[0] = 0;
      start[1] = (int32_t)((p.rows + 127) / 128);
    }
    return;
  }
  int seen = 0;
  bool ok = __ldg(p.offsets) == 0;
  for (int g0 = 0; g0 < p.groups; g0 += 32) {
    const int g = g0 + lane;
    int lo = 0, hi = 0;
    if (g < p.groups) {
      lo = __ldg(p.offsets + g);
      hi = __ldg(p.offsets + g + 1);
      ok = ok && lo >= 0 && hi >= lo && hi <= p.rows;
    }
    int incl = ok ? (hi - lo + 127) / 128 : 0;
    const int mine = incl;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += y;
    }
    if (g < p.groups) start[g] = seen + incl - mine;
    seen += __shfl_sync(kFull, incl, 31);
  }
  if (lane == 0) start[p.groups] = seen;
  const bool good = __all_sync(kFull, ok);
  __syncwarp();
  if (!good) {
    if (lane == 0) set_error(p.err, CTR_ERR_BAD_OFFSETS);
    for (int g = lane; g <= p.groups; g += 32) start[g] = 0;
  }
}

template <int BN, bool WGRAD>
__global__ void __launch_bounds__(kMmThreads, 1) fp8_matmul_kernel(const MmArgs p,
                                                                   const __grid_constant__ CUtensorMap amap,
                                                                   const __grid_constant__ CUtensorMap bmap) {
  constexpr uint32_t kStageBytes = kABytes + BN * 128u;
  constexpr int kStages = (192 * 1024) / kStageBytes;
  constexpr int kHalf = BN / 2;  // columns of a scaling thread
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[2 * kStages + 4];
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag;
  __shared__ int32_t start[CTR_MAX_EXPERTS + 1];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // swizzled tiles need 1024-byte alignment
  const uint32_t full0 = smem_u32(&bars[0]);
  const uint32_t empty0 = smem_u32(&bars[kStages]);
  const uint32_t tfull0 = smem_u32(&bars[2 * kStages]);
  const uint32_t tempty0 = smem_u32(&bars[2 * kStages + 2]);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, kScaleWarps);
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_slot)),
                 "r"(2 * BN)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 2) group_starts(p, start);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_base_slot;
  const int64_t ntiles = WGRAD ? (int64_t)p.groups * p.mt * p.nt : (int64_t)start[p.groups] * p.nt;

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (lane == 0) {
      int64_t it = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < ntiles; t += gridDim.x) {
        const Tile x = locate<WGRAD>(p, start, t, BN);
        for (int j = 0; j < x.nkb; ++j, ++it) {
          const int s = (int)(it % kStages);
          const uint32_t ph = (uint32_t)((it / kStages) & 1);
          if (!mbar_wait(empty0 + 8 * s, ph ^ 1)) {
            set_error(p.err, CTR_ERR_TIMEOUT);
            atomicExch(&abort_flag, 1);
          }
          if (*(volatile int*)&abort_flag) {
            ok = false;
            break;
          }
          mbar_expect_tx(full0 + 8 * s, kStageBytes);
          const uint32_t dst = base + (uint32_t)s * kStageBytes;
          const int32_t k = (int32_t)((x.k0 + j) * 128);
          tma_load_2d(dst, &amap, k, (int32_t)x.a_row, full0 + 8 * s);
          tma_load_2d(dst + kABytes, &bmap, k, (int32_t)x.b_row, full0 + 8 * s);
        }
      }
      // drain: every issued load must have landed before the CTA can exit
      for (int s = 0; s < kStages && s < it; ++s) {
        const int64_t last = it - 1 - ((it - 1 - s) % kStages);  // last iteration using stage s
        if (!mbar_wait(full0 + 8 * s, (uint32_t)((last / kStages) & 1))) set_error(p.err, CTR_ERR_TIMEOUT);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3(kBM, BN);
      int64_t it = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < ntiles; t += gridDim.x) {
        const int nkb = WGRAD ? locate<WGRAD>(p, start, t, BN).nkb : p.kb;
        for (int j = 0; j < nkb; ++j, ++it) {
          const int s = (int)(it % kStages);
          const uint32_t ph = (uint32_t)((it / kStages) & 1);
          const int b = (int)(it & 1);
          if (!mbar_wait(tempty0 + 8 * b, (uint32_t)((it >> 1) & 1) ^ 1) || !mbar_wait(full0 + 8 * s, ph)) {
            set_error(p.err, CTR_ERR_TIMEOUT);
            atomicExch(&abort_flag, 1);
          }
          if (*(volatile int*)&abort_flag) {
            ok = false;
            break;
          }
          fence_after();
          const uint32_t a0 = base + (uint32_t)s * kStageBytes;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_e4m3(tmem + (uint32_t)(b * BN), smem_desc_sw128(a0 + k * 32u), smem_desc_sw128(a0 + kABytes + k * 32u),
                     idesc, k != 0);
          mma_commit(empty0 + 8 * s);
          mma_commit(tfull0 + 8 * b);
        }
      }
      // drain: the last commits must have arrived before TMEM is freed
      for (int b = 0; b < 2 && b < it; ++b) {
        const int64_t last = it - 1 - ((it - 1 - b) % 2);
        if (!mbar_wait(tfull0 + 8 * b, (uint32_t)((last >> 1) & 1))) set_error(p.err, CTR_ERR_TIMEOUT);
      }
    }
  } else {
    // ---------------- scaling warps ----------------
    const int q = warp & 3;             // TMEM lane quarter this warp may read
    const int half = (warp - 2) >> 2;   // which half of the columns
    const int row = q * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(half * kHalf);
    uint32_t* staging = (uint32_t*)(smem_raw + (base - raw) + (size_t)kStages * kStageBytes) +
                        (size_t)(warp - 2) * (kStagingBytes / 4);
    int64_t it = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; ok && t < ntiles; t += gridDim.x) {
      const Tile x = locate<WGRAD>(p, start, t, BN);
      uint64_t acc[kHalf / 2];
#pragma unroll
      for (int i = 0; i < kHalf / 2; ++i) acc[i] = 0;
      const bool live = row < x.rows;
      const int c0 = x.col + half * kHalf;  // this warp's first column
      const float* sa = p.sa + x.k0 * p.ld_sa + x.a_row + row;
      const float* sb = p.sb + (x.sb0 + (half * kHalf) / 128) * p.ld_sb + x.k0;
      const bool cols = c0 < p.n;  // else the whole half lies past the result
      float s_next = live && cols && x.nkb > 0 ? __ldg(sa) * __ldg(sb) : 0.f;
      for (int j = 0; j < x.nkb; ++j, ++it) {
        const int b = (int)(it & 1);
        const float f = s_next;
        if (live && cols && j + 1 < x.nkb) s_next = __ldg(sa + (int64_t)(j + 1) * p.ld_sa) * __ldg(sb + j + 1);
        bool fail = !mbar_wait(tfull0 + 8 * b, (uint32_t)((it >> 1) & 1));
        fail = fail || *(volatile int*)&abort_flag != 0;
        if (__any_sync(kFull, fail)) {
          if (lane == 0 && !*(volatile int*)&abort_flag) {
            set_error(p.err, CTR_ERR_TIMEOUT);
            atomicExch(&abort_flag, 1);
          }
          ok = false;
          break;
        }
        fence_after();
        uint64_t f2;
        asm("mov.b64 %0, {%1, %1};" : "=l"(f2) : "r"(__float_as_uint(f)));
        const uint32_t tb = lane_base + (uint32_t)(b * BN);
        uint32_t v0[16], v1[16];
        tmem_ld16_async(tb, v0);
#pragma unroll
        for (int c = 0; c < kHalf / 32; ++c) {
          tmem_wait_ld();
          tmem_ld16_async(tb + c * 32 + 16, v1);
          scale_add16(acc + c * 16, v0, f2);
          tmem_wait_ld();
          if (c + 1 < kHalf / 32) tmem_ld16_async(tb + c * 32 + 32, v0);
          scale_add16(acc + c * 16 + 8, v1, f2);
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty0 + 8 * b);
      }
      if (!ok) break;
      // ---- the tile's rows leave: straight from registers where every row starts 32-byte aligned,
      // else through shared memory, so that a store covers consecutive columns of a row
      const int64_t orow = x.out_row + row;
#pragma unroll
      for (int c = 0; c < kHalf; c += 32) {
        if (c0 + c >= p.n) break;
        float f[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          uint32_t lo, hi;
          asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(acc[c / 2 + i]));
          f[2 * i] = __uint_as_float(lo);
          f[2 * i + 1] = __uint_as_float(hi);
        }
        const bool whole = c0 + c + 32 <= p.n;
        if (p.out_f32) {
          if (p.wide_rows && whole) {
            if (live) {
              float* dst = (float*)p.out + orow * p.ldo + c0 + c;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(f[8 * i + e]);
                st_global_v8(dst + 8 * i, w);
              }
            }
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 16; ++i) staging[lane * kStageRow + i] = __float_as_uint(f[16 * h + i]);
              __syncwarp();
              const int cc = lane & 15, col = c0 + c + 16 * h + cc;
#pragma unroll 4
              for (int r = lane >> 4; r < 32; r += 2)
                if (q * 32 + r < x.rows && col < p.n)
                  ((float*)p.out)[(x.out_row + q * 32 + r) * p.ldo + col] =
                      __uint_as_float(staging[r * kStageRow + cc]);
            }
          }
        } else {
          if (p.wide_rows && whole) {
            if (live) {
              __nv_bfloat16* dst = (__nv_bfloat16*)p.out + orow * p.ldo + c0 + c;
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = bf16_pair(f[16 * i + 2 * e], f[16 * i + 2 * e + 1]);
                st_global_v8(dst + 16 * i, w);
              }
            }
          } else {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16; ++i) staging[lane * kStageRow + i] = bf16_pair(f[2 * i], f[2 * i + 1]);
            __syncwarp();
            const int col = c0 + c + lane;
#pragma unroll 4
            for (int r = 0; r < 32; ++r)
              if (q * 32 + r < x.rows && col < p.n)
                ((uint16_t*)p.out)[(x.out_row + q * 32 + r) * p.ldo + col] =
                    ((const uint16_t*)(staging + r * kStageRow))[lane];
          }
        }
      }
    }
    if (!WGRAD && p.offsets) {
      // rows past the last group: zeros
      const int64_t used = start[p.groups] > 0 ? __ldg(p.offsets + p.groups) : 0;
      const int64_t stride = (int64_t)gridDim.x * kScaleWarps;
      for (int64_t r = used + (int64_t)blockIdx.x * kScaleWarps + (warp - 2); r < p.rows; r += stride)
        for (int c = lane; c < p.n; c += 32) {
          if (p.out_f32) ((float*)p.out)[r * p.ldo + c] = 0.f;
          else ((uint16_t*)p.out)[r * p.ldo + c] = 0;
        }
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * BN) : "memory");
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

template <int BN, bool WGRAD>
int launch_mm(MmArgs& p, const uint8_t* a, int64_t a_rows, const uint8_t* b, int64_t b_rows, int64_t row_bytes,
              int64_t tiles_m, cudaStream_t s) {
  CUtensorMap amap, bmap;
  if (!code_map(&amap, a, a_rows, row_bytes, kBM) || !code_map(&bmap, b, b_rows, row_bytes, BN)) return CTR_ERR_CUDA;
  p.nt = (int32_t)ceil_div(p.n, BN);
  constexpr uint32_t stage = kABytes + BN * 128u;
  const int smem = (int)(1024 + (192 * 1024) / stage * stage + kScaleWarps * kStagingBytes);
  auto k = fp8_matmul_kernel<BN, WGRAD>;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return CTR_ERR_CUDA;
  const int64_t tiles = tiles_m * p.nt;
  const int grid = (int)imax64(1, imin64(tiles, num_sms()));
  k<<<grid, kMmThreads, smem, s>>>(p, amap, bmap);
  count_launch();
  return launch_status();
}

// 256 columns a tile halve the reads of the left operand and use the tensor cores best; 128 where
// that would leave SMs without a tile, or half a tile empty.
bool tile_256(int64_t tiles_m, int64_t n) { return n > 128 && tiles_m * ceil_div(n, 256) >= num_sms(); }

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
  return kWsHeader;
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
  p.wide_rows = ((uintptr_t)out % 32) == 0 && (ldo * eb) % 32 == 0;
  const int64_t tiles_m = offsets ? ctr_fp8_padded_rows(rows, groups) / 128 : ceil_div(rows, 128);
  cudaStream_t s = (cudaStream_t)stream;
  const int64_t row_bytes = (int64_t)p.kb * 128;
  if (tile_256(tiles_m, n)) return launch_mm<256, false>(p, a, rows, b, groups * n, row_bytes, tiles_m, s);
  return launch_mm<128, false>(p, a, rows, b, groups * n, row_bytes, tiles_m, s);
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
  p.mt = (int32_t)ceil_div(n, kBM);
  p.out_f32 = out_dtype == CTR_F32;
  const int eb = dtype_bytes(out_dtype);
  p.wide_rows = ((uintptr_t)out % 32) == 0 && (k * eb) % 32 == 0;
  const int64_t tiles_m = (int64_t)groups * p.mt;
  cudaStream_t s = (cudaStream_t)stream;
  if (tile_256(tiles_m, k)) return launch_mm<256, true>(p, d, n, x, k, padded, tiles_m, s);
  return launch_mm<128, true>(p, d, n, x, k, padded, tiles_m, s);
}
