// Products of microscaled 4-bit operands on the tensor cores: D[i][j] =
// sum_k A[i][k] B[j][k] (+ D), tcgen05.mma kind::mxf4 (GM_MX4) or kind::mxf4nvf4
// (GM_NV4) on packed e2m1 codes with the block scales in tensor memory, sums in
// fp32, one rounding to D's type.
//
// One kernel, two shapes:
//   CG = 2: a pair of CTAs per 256 x 256 tile (M = 256, N = 256, K = 64 per
//     instruction), persistent over the tiles. Each CTA loads its 128 rows of A and
//     128 of the 256 rows of B. 8192 x 18944 x 3584 into bf16: 237 us (GM_MX4, 4.7
//     PFLOP/s), 227 us (GM_NV4) at 1.6 GHz; without its stores 174 us,
//     with a quarter of its MMAs 196 us, with neither 124 us (36 KB a stage and SM, 68
//     bytes a clock, is what L2 delivers). So loads, MMAs and stores share the memory
//     path of an SM: 64 bytes a clock of copies into shared memory, as many of operand
//     reads at the tensor pipe's full rate, and D's lines going out. Stores through
//     shared memory (250 us) or of whole lines exchanged among lanes (242 us), a fifth
//     stage, other orders of the tiles and scales fetched a stage ahead gained nothing.
//   CG = 1, for products of few tiles, which B's bytes (a weight's) bound: operands
//     change places, so that a tile is 128 rows of B (the instruction's M) by up to 256
//     rows of A (its N, no more than there are, to 16). One CTA per tile, or a cluster of
//     up to 8 that split K stage by stage and join their fp32 parts through distributed
//     shared memory in the order of the ranks (so equal operands give equal bits). A lane
//     holds a column of D, and its stores are contiguous for any N. 1 x 3584 x 18944: 13.6
//     us. In a cold launch with timers in it (14.9 us) the first stage is there after 4.1
//     us, the last 8 us later (36 MB, 4.5 TB/s); the join and its barriers end 2.8 us on.
// Roles of a CTA's warps:
//   warp 0: TMA of A's codes and scales      warp 2: TMA of B's
//   warp 1: tensor memory; copies a stage's scales to tensor memory (tcgen05.cp) and
//           issues its MMAs, one lane issuing under a predicate
//   warps 4..19: epilogue. A warp takes 32 rows and 64 columns into registers at
//           once, so that the accumulator is free for the next tile before the
//           results are written.
// A stage holds 256 columns of K: 128-byte rows of codes in the 128-byte swizzle, and
// the scale atoms as they lie in memory (512 bytes: 128 rows x 4 blocks), each of
// which one tcgen05.cp (32 lanes x 128 bits, repeated over the four lane quarters)
// turns into four columns of tensor memory. The scales of a stage have their own
// columns, so the copies for a stage never touch what an earlier stage's MMAs read.
// Every wait is bounded; a timeout is recorded in the device's error word.

#include <cudaTypedefs.h>
#include <string.h>

#include "gm_common.cuh"
#include "gm_internal.h"
#include "gm_mx4.cuh"
#include "gm_tcgen05.cuh"

namespace gm {
namespace {

constexpr int kBN = 256;                  // columns of a tile
constexpr int kStageK = 256;              // columns of K per stage
constexpr int kStages = 4;                // of CG = 2; CG = 1: as many as fit, at most kMaxStages
constexpr int kMaxStages = 8;
constexpr int kEpiWarp0 = 4, kEpiWarps = 16;
constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
constexpr int kWarpCols = kBN / (kEpiWarps / 4);   // 64 columns of an epilogue warp
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr int kMaxSplit = 8;              // portable cluster size

constexpr uint32_t kABytes = 128 * (kStageK / 2);
constexpr uint32_t sf_bytes(int fmt) { return kStageK / (4 * mx4_block(fmt)) * 512; }   // of 128 rows
// A stage of a CTA: 128 rows of the first operand, `rows` of the second, the scales of
// 128 and of `tiles` times 128 rows.
__host__ __device__ constexpr uint32_t stage_bytes(int fmt, int rows, int tiles) {
  return kABytes + rows * (kStageK / 2) + (1 + tiles) * sf_bytes(fmt);
}
constexpr int kPitch = 17;                // staging of ragged stores: 32 rows x 16 columns a warp
constexpr uint32_t kStageOut = kEpiWarps * 32 * kPitch * 4;
constexpr uint32_t ring_bytes(int cg, int fmt) {
  return kStages * stage_bytes(fmt, cg == 2 ? 128 : kBN, 2);
}
constexpr uint32_t smem_bytes(int cg, int fmt) {
  return ring_bytes(cg, fmt) + (cg == 2 ? kStageOut : 0) + 1024 /* barriers */ + 1024 /* align */;
}
static_assert(smem_bytes(1, GM_NV4) <= 227 * 1024 && smem_bytes(2, GM_NV4) <= 227 * 1024, "shared memory");
static_assert(kBN * 128 * 4 <= ring_bytes(1, GM_MX4), "a part of a split tile fits the idle ring");

// Tensor memory columns: the accumulator, then per stage the scales of the first and of
// the second operand (4 columns per atom of 128 rows).
constexpr uint32_t kTmemCols = 512;
__host__ __device__ constexpr uint32_t sf_cols(int fmt) { return sf_bytes(fmt) / 128; }   // of 128 rows, one stage
static_assert(kBN + kStages * 3 * sf_cols(GM_NV4) <= kTmemCols && kBN + kMaxStages * 2 * sf_cols(GM_NV4) <= kTmemCols,
              "tensor memory");

struct ProductParams {
  int M, N, K;
  int batch, tiles_m, tiles_n;
  int bn;                  // columns of a tile's accumulator (CG = 1: 16 .. 256, CG = 2: 256)
  int sf_tiles;            // 128-row tiles of the second operand's scales in a stage
  int stages;
  int split;               // CTAs that share a tile's K (CG = 1)
  void* D;
  int ddt, accumulate;
  int vec;                 // D's rows start on 32 bytes
  const float *ag, *bg;    // GM_NV4
  int32_t* err;
};

// ------------------------------------------------------------ PTX wrappers
template <int CG>
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar),
        "r"(x), "r"(y), "r"(z)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar),
        "r"(x), "r"(y), "r"(z)
        : "memory");
}
template <int CG>
__device__ __forceinline__ void load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                        int w) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar),
        "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar),
        "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}
// One scale atom (512 bytes, rows of 16) to four columns of tensor memory, in both
// CTAs of a pair.
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t one, uint32_t tmem, uint32_t smem) {
  // no swizzle; 128 bytes from one group of eight 16-byte rows to the next
  const uint64_t d = (uint64_t)((smem >> 4) & 0x3FFF) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
  if constexpr (CG == 2)
    asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %2, 0;\n\t"
                 "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}\n" ::"r"(tmem), "l"(d), "r"(one)
                 : "memory");
  else
    asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %2, 0;\n\t"
                 "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}\n" ::"r"(tmem), "l"(d), "r"(one)
                 : "memory");
}
// Instruction descriptor of the block-scaled 4-bit kinds: e2m1 operands, K-major, K =
// 64; `sf` selects the scale bytes of a 32-bit word to begin with.
template <int CG, int FMT>
__host__ __device__ constexpr uint32_t idesc_mx4(uint32_t sf, int n) {
  return (sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) |
         ((FMT == GM_MX4 ? 1u : 0u) << 23) | ((uint32_t)(128 * CG >> 7) << 27) | (sf << 29);
}
template <int CG, int FMT>
__device__ __forceinline__ void umma_mx4(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
#define GM_UMMA_MX4(GROUP, KIND)                                                                   \
  asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 e, %7, 0;\n\t"        \
               "@e tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d), \
               "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(one)           \
               : "memory")
  if constexpr (CG == 2 && FMT == GM_MX4) GM_UMMA_MX4("2", "mxf4.block_scale.scale_vec::2X");
  if constexpr (CG == 2 && FMT == GM_NV4) GM_UMMA_MX4("2", "mxf4nvf4.block_scale.scale_vec::4X");
  if constexpr (CG == 1 && FMT == GM_MX4) GM_UMMA_MX4("1", "mxf4.block_scale.scale_vec::2X");
  if constexpr (CG == 1 && FMT == GM_NV4) GM_UMMA_MX4("1", "mxf4nvf4.block_scale.scale_vec::4X");
#undef GM_UMMA_MX4
}
// Arrive on the barrier (of both CTAs of a pair) once the MMAs issued so far are done.
template <int CG>
__device__ __forceinline__ void commit(uint32_t one, uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %2, 0;\n\t"
                 "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
                 " [%0], %1;\n\t}\n" ::"r"(bar), "h"((uint16_t)3), "r"(one)
                 : "memory");
  else
    asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar),
                 "r"(one)
                 : "memory");
}
// One lane of a converged warp. The instructions below are issued by it under a
// predicate, the warp staying together: their operands then live in uniform
// registers (under a branch each tcgen05 instruction took about 55 ns to issue).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}\n" : "=r"(r));
  return r;
}
// 64 columns of 32 lanes of tensor memory.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&v)[64]) {
  uint32_t r[64];
#pragma unroll
  for (int h = 0; h < 4; ++h)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[16 * h]), "=r"(r[16 * h + 1]), "=r"(r[16 * h + 2]), "=r"(r[16 * h + 3]), "=r"(r[16 * h + 4]),
          "=r"(r[16 * h + 5]), "=r"(r[16 * h + 6]), "=r"(r[16 * h + 7]), "=r"(r[16 * h + 8]), "=r"(r[16 * h + 9]),
          "=r"(r[16 * h + 10]), "=r"(r[16 * h + 11]), "=r"(r[16 * h + 12]), "=r"(r[16 * h + 13]),
          "=r"(r[16 * h + 14]), "=r"(r[16 * h + 15])
        : "r"(taddr + 16 * h));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}

// ------------------------------------------------------------------ epilogue
// 32 bytes of a row: 8 fp32 or 16 16-bit values.
__device__ __forceinline__ void ld32(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void st32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// GM_NV4: the product of both matrix scales as a * b. b is 1 unless the product leaves
// fp32's normal range, where a sum times it may well lie inside: then a has the product's
// bits and half of its exponent, b the other half.
struct Alpha {
  float a, b;
};
__device__ __forceinline__ double two_to(int e) { return __hiloint2double((e + 1023) << 20, 0); }
template <int FMT>
__device__ __forceinline__ Alpha alpha_of(const ProductParams& p, int bz) {
  if constexpr (FMT == GM_MX4) return {1.f, 1.f};
  const double d = (double)p.ag[bz] * (double)p.bg[bz];   // exact
  if (!(d > 0.0) || d > 1e80 || (d >= 1.1754943508222875e-38 && d <= 3.4028234663852886e38)) return {(float)d, 1.f};
  const int e = (__double2hiint(d) >> 20) - 1023, h = e / 2;   // -298 .. 255
  return {(float)(d * two_to(-e)) * (float)two_to(h), (float)two_to(e - h)};
}

// One warp's 32 rows (a lane each) x 64 columns from column c: whole 32-byte sectors
// per lane when D's rows are aligned to them, else through shared memory, 16 columns
// at a time, so that neighbouring lanes write neighbouring elements.
__device__ __forceinline__ void store_warp(const ProductParams& p, float (&v)[64], int bz, int row0, int c,
                                           int lane, float* stg) {
  const long long base = (long long)bz * p.M * p.N;
  const bool f16 = p.ddt == GM_F16;
  if (p.vec) {
    const int r = row0 + lane;
    if (r >= p.M) return;
    const long long at = base + (long long)r * p.N + c;
    if (p.ddt == GM_F32) {
      float* d = static_cast<float*>(p.D) + at;
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        if (c + g * 8 >= p.N) return;
        uint32_t w[8];
        if (p.accumulate) {
          ld32(d + g * 8, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[g * 8 + e] += __uint_as_float(w[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(v[g * 8 + e]);
        st32(d + g * 8, w);
      }
    } else {
      uint16_t* d = static_cast<uint16_t*>(p.D) + at;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if (c + g * 16 >= p.N) return;
        uint32_t w[8];
        if (p.accumulate) {
          ld32(d + g * 16, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[g * 16 + 2 * e] += h16_to_float((uint16_t)(w[e] & 0xFFFFu), f16);
            v[g * 16 + 2 * e + 1] += h16_to_float((uint16_t)(w[e] >> 16), f16);
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[e] = (uint32_t)float_to_h16(v[g * 16 + 2 * e], f16) |
                 ((uint32_t)float_to_h16(v[g * 16 + 2 * e + 1], f16) << 16);
        st32(d + g * 16, w);
      }
    }
    return;
  }
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 16; ++e) stg[lane * kPitch + e] = v[g * 16 + e];
    __syncwarp();
    const int col = c + g * 16 + (lane & 15);
    if (col < p.N) {
#pragma unroll 4
      for (int rr = lane >> 4; rr < 32; rr += 2) {
        const int r = row0 + rr;
        if (r >= p.M) break;
        const long long at = base + (long long)r * p.N + col;
        float d = stg[rr * kPitch + (lane & 15)];
        if (p.accumulate) d += load_as_float(p.D, at, p.ddt);
        store_from_float(p.D, at, p.ddt, d);
      }
    }
  }
}

// ------------------------------------------------------------------ kernel
template <int CG, int FMT>
__global__ void __launch_bounds__(kThreads, 1)
    k_mx4_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
               const ProductParams p) {
  constexpr uint32_t kSf = sf_bytes(FMT);
  constexpr int kAtoms = kSf / 512;
  // constants for CG = 2
  const int bn = CG == 2 ? kBN : p.bn, sft = CG == 2 ? 2 : p.sf_tiles;
  const uint32_t stages = CG == 2 ? kStages : (uint32_t)p.stages;
  const uint32_t b_size = (uint32_t)(bn / CG) * (kStageK / 2), stage = stage_bytes(FMT, bn / CG, sft);
  extern __shared__ __align__(1024) uint8_t dsm[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm) + 1023) & ~uintptr_t(1023));
  uint8_t* after = ring + ring_bytes(CG, FMT);
  float* stage_out = reinterpret_cast<float*>(after);            // CG = 2
  uint64_t* full = reinterpret_cast<uint64_t*>(after + (CG == 2 ? kStageOut : 0));
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* drain = acc_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* flags = reinterpret_cast<int*>(tmem_slot + 1);
  volatile int* abort_flag = flags;
  int* consumed = flags + 1;
  int* issued = flags + 2;

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int group = CG == 2 ? 2 : p.split;                  // CTAs of a cluster
  const bool leader = CG == 1 || rank == 0;                 // issues MMAs
  const int cid = blockIdx.x / group, ncl = gridDim.x / group;
  const int tiles = p.tiles_m * p.tiles_n, total = p.batch * tiles;
  const int k64 = (int)(mx4_padded(p.K) / 64);              // instructions along K
  const int nst = cdiv(k64, kStageK / 64);
  // CG = 1: the ranks of a cluster take turns, so that together they read a row's bytes
  // in order
  const int st0 = CG == 1 ? (int)rank : 0, st_step = CG == 1 ? p.split : 1;
  const uint32_t stage_tx = CG * stage;

  if (threadIdx.x == 0) {
    for (int s = 0; s < (int)stages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(acc_full), 1);
    mbar_init(smem_u32(acc_empty), CG * kEpiWarps);
    mbar_init(smem_u32(drain), 1);
    flags[0] = flags[1] = flags[2] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    prefetch_map(&tmA);
    prefetch_map(&tmB);
    prefetch_map(&tmSA);
    prefetch_map(&tmSB);
  }
  if (warp == 1) {
    if constexpr (CG == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                   "r"(kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                   "r"(kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  tc_fence_before();
  __syncthreads();
  if (group > 1) cluster_sync_all();   // barriers initialised before any signal from another CTA
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  // Launched as a programmatic dependent: the set-up above runs under the kernel before
  // (often the quantisation of an operand), whose results are visible from here on.
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // First row of this CTA's part of a tile in the instruction's first operand (CG = 2: A,
  // CG = 1: B) and in its second.
  auto origin = [&](int T, int& bz, int& r0, int& c0) {
    bz = T / tiles;
    const int x = T - bz * tiles;
    if constexpr (CG == 2) {
      r0 = x % p.tiles_m * 256 + (int)rank * 128;
      c0 = x / p.tiles_m * kBN;
    } else {
      r0 = x % p.tiles_n * 128;
      c0 = x / p.tiles_n * bn;
    }
  };
  auto slot = [&](uint32_t g, uint32_t& s, uint32_t& ph) {
    s = g % stages;
    ph = (g / stages) & 1u;
  };

  if (warp == 0 || warp == 2) {
    if (lane == 0) {
      // ---------------- TMA producers
      const bool isA = warp == 0;
      uint32_t g = 0;
      bool ok = true;
      for (int T = cid; T < total && ok; T += ncl) {
        int bz, r0, c0;
        origin(T, bz, r0, c0);
        for (int st = st0; st < nst; st += st_step, ++g) {
          uint32_t s, ph;
          slot(g, s, ph);
          if (!mbar_wait(smem_u32(&empty[s]), ph ^ 1u, p.err, abort_flag, kWaitLimitNs)) { ok = false; break; }
          const uint32_t bar = CG == 2 ? map_to_rank(smem_u32(&full[s]), 0) : smem_u32(&full[s]);
          const uint32_t a = smem_u32(ring + s * stage), b = a + kABytes, sa = b + b_size, sb = sa + kSf;
          if (isA) {
            if (leader) mbar_expect_tx(smem_u32(&full[s]), stage_tx);
            load_3d<CG>(a, &tmA, bar, st * (kStageK / 2), r0, bz);
            load_4d<CG>(sa, &tmSA, bar, 0, st * kAtoms, r0 / 128, bz);
          } else {
            load_3d<CG>(b, &tmB, bar, st * (kStageK / 2), c0 + (CG == 2 ? (int)rank * 128 : 0), bz);
            load_4d<CG>(sb, &tmSB, bar, 0, st * kAtoms, c0 / 128, bz);
          }
        }
      }
      atomicMax(issued, (int)g);
    }
  } else if (warp == 1) {
    if (leader) {
      // ---------------- MMA issuer: the whole warp, instructions from one lane
      const uint32_t one = elect_one();
      uint32_t g = 0;
      bool ok = true;
      int it = 0;
      for (int T = cid; T < total && ok; T += ncl, ++it) {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(acc_empty), ((uint32_t)it & 1u) ^ 1u, p.err, abort_flag, kWaitLimitNs));
        if (!ok) break;
        tc_fence_after();
        for (int st = st0; st < nst; st += st_step, ++g) {
          uint32_t s, ph;
          slot(g, s, ph);
          ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&full[s]), ph, p.err, abort_flag, kWaitLimitNs));
          if (!ok) break;
          tc_fence_after();
          const uint32_t a = smem_u32(ring + s * stage), b = a + kABytes, sa = b + b_size, sb = sa + kSf;
          const uint32_t ta = tmem + kBN + s * (uint32_t)(1 + sft) * sf_cols(FMT), tb = ta + sf_cols(FMT);
#pragma unroll
          for (int j = 0; j < kAtoms; ++j) {
            copy_scales<CG>(one, ta + j * 4, sa + j * 512);
            // second operand: [128-row tile][atom] in shared memory, [atom][tile] in tensor memory
            copy_scales<CG>(one, tb + j * 4 * sft, sb + j * 512);
            if (sft == 2) copy_scales<CG>(one, tb + j * 8 + 4, sb + kSf + j * 512);
          }
#pragma unroll
          for (int kk = 0; kk < kStageK / 64; ++kk) {
            const int k = st * (kStageK / 64) + kk;
            if (k >= k64) break;
            const int j = kk * kAtoms / (kStageK / 64);          // the atom that holds this k
            const uint32_t sf = FMT == GM_MX4 ? (kk & 1) * 2 : 0;
            umma_mx4<CG, FMT>(one, tmem, sdesc(a + kk * 32, 16, 1024), sdesc(b + kk * 32, 16, 1024),
                              idesc_mx4<CG, FMT>(sf, bn), ta + j * 4, tb + j * 4 * sft, (st > st0 || kk) ? 1u : 0u);
          }
          commit<CG>(one, smem_u32(&empty[s]));
        }
        if (!ok) break;
        commit<CG>(one, smem_u32(acc_full));
      }
      if (lane == 0) {
        *consumed = (int)g;
        if (!ok) *abort_flag = 1;
      }
      commit<CG>(one, smem_u32(drain));       // fires once every MMA issued above has completed
      mbar_wait(smem_u32(drain), 0, p.err, nullptr, kWaitLimitNs);
    }
  } else if (warp >= kEpiWarp0) {
    // ---------------- epilogue
    const int q = warp & 3, part = (warp - kEpiWarp0) >> 2;     // lane quarter, column part
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    if constexpr (CG == 2) {
      const uint32_t bar = map_to_rank(smem_u32(acc_empty), 0);
      int it = 0;
      for (int T = cid; T < total; T += ncl, ++it) {
        int bz, r0, c0;
        origin(T, bz, r0, c0);
        const Alpha alpha = alpha_of<FMT>(p, bz);
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(acc_full), (uint32_t)it & 1u, p.err, abort_flag, kWaitLimitNs))) break;
        tc_fence_after();
        float v[64];
        tmem_ld64(lanes + (uint32_t)(part * kWarpCols), v);
        tc_fence_before();
        __syncwarp();
        if (lane == 0)
          asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
        const int c = c0 + part * kWarpCols;
        if (FMT == GM_NV4) {
#pragma unroll
          for (int e = 0; e < 64; ++e) v[e] *= alpha.a;
          if (alpha.b != 1.f) {   // (without this branch 8192 x 18944 x 3584 takes 231 us, not 227)
#pragma unroll
            for (int e = 0; e < 64; ++e) v[e] *= alpha.b;
          }
        }
        if (c < p.N) store_warp(p, v, bz, r0 + q * 32, c, lane, stage_out + (warp - kEpiWarp0) * 32 * kPitch);
      }
    } else {
      int bz, r0, c0;
      origin(cid, bz, r0, c0);
      const Alpha alpha = alpha_of<FMT>(p, bz);
      const int n = r0 + q * 32 + lane;                         // this lane's column of D
      if (__all_sync(0xffffffffu, mbar_wait(smem_u32(acc_full), 0, p.err, abort_flag, kWaitLimitNs))) {
        tc_fence_after();
#pragma unroll 1
        for (int ch = part; ch * 16 < bn && c0 + ch * 16 < p.M; ch += kEpiWarps / 4) {
          float v[16];
          tmem_ld16(lanes + (uint32_t)(ch * 16), v);
          const int rows = p.M - (c0 + ch * 16);
          if (group > 1) {
            // this rank's fp32 part of the tile, [row of D][128 columns], in the idle ring
            float* to = reinterpret_cast<float*>(ring) + ch * 16 * 128 + q * 32 + lane;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (e < rows) to[e * 128] = v[e];
          } else if (n < p.N) {
            const long long at = ((long long)bz * p.M + c0 + ch * 16) * p.N + n;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              if (e >= rows) break;
              float d = FMT == GM_NV4 ? v[e] * alpha.a * alpha.b : v[e];
              if (p.accumulate) d += load_as_float(p.D, at + (long long)e * p.N, p.ddt);
              store_from_float(p.D, at + (long long)e * p.N, p.ddt, d);
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && leader) {
    // after an abort, let the copies still in flight land
    for (int g = *consumed; g < *issued; ++g) {
      uint32_t s, ph;
      slot((uint32_t)g, s, ph);
      mbar_wait(smem_u32(&full[s]), ph, p.err, nullptr, kWaitLimitNs);
    }
  }
  if (group > 1) cluster_sync_all();
  if (CG == 1 && group > 1) {
    // join the parts: rank r takes every group-th run of four columns
    int bz, r0, c0;
    origin(cid, bz, r0, c0);
    const Alpha alpha = alpha_of<FMT>(p, bz);
    const int rows = min(bn, p.M - c0);
    const uint32_t mine = smem_u32(ring);
    uint32_t remote[kMaxSplit];
#pragma unroll
    for (int r = 0; r < kMaxSplit; ++r) remote[r] = r < group ? map_to_rank(mine, r) : 0u;
    for (int i = threadIdx.x * group + (int)rank; i < rows * 32; i += kThreads * group) {
      const int r = i / 32, n = r0 + i % 32 * 4;
      if (n >= p.N) continue;
      float4 x[kMaxSplit];   // all loads first: each takes most of a microsecond
#pragma unroll
      for (int s = 0; s < kMaxSplit; ++s) {
        x[s] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s < group)
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(x[s].x), "=f"(x[s].y), "=f"(x[s].z), "=f"(x[s].w)
                       : "r"(remote[s] + (uint32_t)i * 16)
                       : "memory");
      }
      float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < kMaxSplit; ++s) {
        o[0] += x[s].x; o[1] += x[s].y; o[2] += x[s].z; o[3] += x[s].w;
      }
      const long long at = ((long long)bz * p.M + c0 + r) * p.N + n;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (FMT == GM_NV4) o[e] = o[e] * alpha.a * alpha.b;
        if (p.accumulate && n + e < p.N) o[e] += load_as_float(p.D, at + e, p.ddt);
      }
      if (p.N % 4 == 0) {
        store4_from_float(p.D, at, p.ddt, make_float4(o[0], o[1], o[2], o[3]));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < p.N) store_from_float(p.D, at + e, p.ddt, o[e]);
      }
    }
    cluster_sync_all();   // no CTA leaves while another still reads its part
  }
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CG == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// ------------------------------------------------------------------ host side
bool encode(CUtensorMap* map, CUtensorMapDataType type, const void* base, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, type, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Codes [batch][rows][Kp / 2] with 128-byte x box_rows boxes; rows and columns
// behind the end read as zero.
bool map_codes(CUtensorMap* m, const uint8_t* base, int batch, int rows, int K, int box_rows) {
  const cuuint64_t row = (cuuint64_t)mx4_padded(K) / 2;
  const cuuint64_t dims[3] = {row, (cuuint64_t)rows, (cuuint64_t)batch};
  const cuuint64_t strides[2] = {row, row * (cuuint64_t)rows};
  const cuuint32_t box[3] = {kStageK / 2, (cuuint32_t)box_rows, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
// Scales [batch][row tile][atom][128 words]: one stage's atoms of `tiles` row tiles.
bool map_scales(CUtensorMap* m, const uint8_t* base, int batch, int rows, int K, int fmt, int tiles) {
  const cuuint64_t atoms = (cuuint64_t)mx4_atoms(K, fmt), rt = (cuuint64_t)cdiv(rows, 128);
  const cuuint64_t dims[4] = {128, atoms, rt, (cuuint64_t)batch};
  const cuuint64_t strides[3] = {512, atoms * 512, atoms * 512 * rt};
  const cuuint32_t box[4] = {128, sf_bytes(fmt) / 512, (cuuint32_t)tiles, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, base, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

struct Maps {
  CUtensorMap A, B, SA, SB;
};

template <int CG, int FMT>
cudaError_t launch_t(const Maps& m, const ProductParams& p, cudaStream_t s) {
  static DeviceOnce once;
  const cudaError_t e = smem_attr_once(once, k_mx4_gemm<CG, FMT>, smem_bytes(CG, FMT));
  if (e != cudaSuccess) return e;
  const int total = p.tiles_m * p.tiles_n * p.batch;
  const int group = CG == 2 ? 2 : p.split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(CG == 2 ? 2 * (total < sm_count() / 2 ? total : sm_count() / 2) : total * group));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes(CG, FMT);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)group;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_mx4_gemm<CG, FMT>, m.A, m.B, m.SA, m.SB, p);
}

}  // namespace

cudaError_t launch_mx4_matmul(int B, int M, int N, int K, int fmt, const uint8_t* a, const uint8_t* as,
                              const float* ag, const uint8_t* b, const uint8_t* bs, const float* bg,
                              void* D, int ddt, int accumulate, cudaStream_t s) {
  ProductParams p{};
  p.M = M; p.N = N; p.K = K;
  p.batch = B;
  p.D = D; p.ddt = ddt; p.accumulate = accumulate;
  const int per = ddt == GM_F32 ? 8 : 16;   // elements of 32 bytes
  p.vec = N % per == 0 && reinterpret_cast<uintptr_t>(D) % 32 == 0;
  p.ag = ag; p.bg = bg;
  p.err = device_error_word();
  if (!p.err) return cudaErrorUnknown;
  // Pairs from a quarter of the SMs' worth of tiles on; up to 128 rows a tile of one CTA
  // reads the weight as fast (16 x 18944 x 3584: 12.6 us, 15.5 as pairs). Around the limit
  // K decides more than the tiles do: short sums are faster alone (by a quarter at most),
  // long ones as pairs (by a fifth). As pairs / alone, us:
  //   tiles       K = 512     2048         4096          16384
  //   36 (NV4)   7.4 / 6.3   9.5 / 9.2    12.3 / 13.4   30.0 / 28.8   (MX4: 11.2 / 8.4, 31.1 / 26.3)
  //   40 (NV4)   7.7 / 6.3   9.7 / 9.2    12.5 / 13.4   30.8 / 37.3
  //   48 (NV4)   7.7 / 6.3   9.7 / 9.4    12.5 / 13.5   30.9 / 37.9   (MX4: 11.4 / 8.4, 31.8 / 33.2)
  //   64 (NV4)   7.7 / 6.5  10.0 / 9.6    12.9 / 13.8   32.0 / 38.7   (MX4: 11.6 / 8.7, 32.9 / 34.2)
  // (1536 x 1536, 1280 x 2048, 1536 x 2048, 2048 x 2048; a choice by K too is not made.)
  const bool pair = M > 128 && (long long)cdiv(M, 256) * cdiv(N, kBN) * B >= sm_count() / 4;
  p.split = 1;
  Maps m;
  bool ok;
  if (pair) {
    p.tiles_m = cdiv(M, 256);
    p.tiles_n = cdiv(N, kBN);
    ok = map_codes(&m.A, a, B, M, K, 128) && map_codes(&m.B, b, B, N, K, 128) &&
         map_scales(&m.SA, as, B, M, K, fmt, 1) && map_scales(&m.SB, bs, B, N, K, fmt, 2);
  } else {
    p.bn = M < kBN ? cdiv(M, 16) * 16 : kBN;
    p.sf_tiles = cdiv(p.bn, 128);
    const uint32_t fit = ring_bytes(1, fmt) / stage_bytes(fmt, p.bn, p.sf_tiles);
    p.stages = p.sf_tiles == 2 ? kStages : (int)(fit < kMaxStages ? fit : kMaxStages);
    p.tiles_m = cdiv(M, p.bn);
    p.tiles_n = cdiv(N, 128);
    const long long tiles = (long long)p.tiles_m * p.tiles_n * B;
    const int nst = cdiv((int)(mx4_padded(K) / 64), kStageK / 64);
    // A join costs about 2 us and a quarter of a stage's time per eight rows; a split
    // halves the stages (1001 x 2053 x 771, four stages: 15.9 us split in two, 8.7 whole;
    // 1 x 3584 x 18944, 74 stages: 13.6 us split in four).
    while (p.split < kMaxSplit && tiles * p.split * 2 <= sm_count() && nst >= (8 + p.bn / 8) * p.split) p.split *= 2;
    ok = map_codes(&m.A, b, B, N, K, 128) && map_codes(&m.B, a, B, M, K, p.bn) &&
         map_scales(&m.SA, bs, B, N, K, fmt, 1) && map_scales(&m.SB, as, B, M, K, fmt, p.sf_tiles);
  }
  if (!ok) return cudaErrorInvalidValue;
  if (fmt == GM_MX4) return pair ? launch_t<2, GM_MX4>(m, p, s) : launch_t<1, GM_MX4>(m, p, s);
  return pair ? launch_t<2, GM_NV4>(m, p, s) : launch_t<1, GM_NV4>(m, p, s);
}

}  // namespace gm
