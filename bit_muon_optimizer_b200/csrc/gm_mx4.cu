// Quantisation to microscaled 4-bit values and back: along the rows of a matrix,
// along its columns (the transpose's rows), or both in one pass over it.
//
// GM_MX4 (blocks of 32): b = max(floor(log2 max|x|) + 127 - 2, 0), scale 2^(b-127),
//   codes e2m1(x 2^(127-b)): every step is exact but the rounding to e2m1.
// GM_NV4 (blocks of 16): gs = fp32(max|X| / 2688), sb = e4m3(max|x| / (6 gs)), codes
//   e2m1(x / (sb gs)). 2688 = 6 * 448, so the largest block scale is e4m3's largest.
//   Codes and scales are those of the exact quotients: fp32 decides unless the value
//   lies so close to a border that fp32's error could cross it, then the product of
//   border and scales is compared with the value exactly.
//
// HBM moves x once (2 or 4 B) and 0.53 or 0.56 B per orientation; GM_NV4 reads x before
// that for the matrix scale. What bounds the kernels is issue: 8192 x 8192 bf16 both
// ways take 18 instructions an element (GM_MX4, 54 us, 3.8 TB/s) or 32 (GM_NV4, 92 us:
// twice the products and conversions, for each element is coded a little below and a
// little above its quotient to see whether fp32 decides). 16384 x 8192 bf16: rows
// 65 us (GM_MX4, 5.2 TB/s) or 107 us and 41 us for the matrix scale (GM_NV4, 3.2 and 6.5
// TB/s), both ways 96 us (GM_MX4); 18944 x 3584 fp32, GM_NV4, both: 150 us with its
// matrix scale (two such matrices: 79 us of 290, 6.9 TB/s).

#include <math.h>

#include "gm_common.cuh"
#include "gm_internal.h"
#include "gm_mx4.cuh"

namespace gm {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;
constexpr int kRowSpan = 1024;   // elements of a row that a warp takes at a time

// ------------------------------------------------------------------- elements
// Eight consecutive elements of a row as they lie in memory.
template <int DT>
struct Eight {
  uint32_t w[DT == GM_F32 ? 8 : 4];
};
// From column c of a row of n (zeros behind its end).
template <int DT>
__device__ __forceinline__ void load8(const void* row, int c, int n, bool vec, Eight<DT>& x) {
  if (vec && c + 8 <= n) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + (size_t)c * (DT == GM_F32 ? 4 : 2));
    const uint4 a = p[0];
    x.w[0] = a.x; x.w[1] = a.y; x.w[2] = a.z; x.w[3] = a.w;
    if constexpr (DT == GM_F32) {
      const uint4 b = p[1];
      x.w[4] = b.x; x.w[5] = b.y; x.w[6] = b.z; x.w[7] = b.w;
    }
  } else if constexpr (DT == GM_F32) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x.w[e] = c + e < n ? static_cast<const uint32_t*>(row)[c + e] : 0u;
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(row);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      x.w[j] = (c + 2 * j < n ? (uint32_t)p[c + 2 * j] : 0u) | (c + 2 * j + 1 < n ? (uint32_t)p[c + 2 * j + 1] << 16 : 0u);
  }
}
template <int DT>
__device__ __forceinline__ float lo_half(uint32_t w) {
  return DT == GM_BF16 ? __uint_as_float(w << 16) : __half2float(__ushort_as_half((uint16_t)(w & 0xFFFFu)));
}
template <int DT>
__device__ __forceinline__ float hi_half(uint32_t w) {
  return DT == GM_BF16 ? __uint_as_float(w & 0xFFFF0000u) : __half2float(__ushort_as_half((uint16_t)(w >> 16)));
}
template <int DT>
__device__ __forceinline__ void to_floats(const Eight<DT>& x, float (&o)[8]) {
  if constexpr (DT == GM_F32) {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = __uint_as_float(x.w[e]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[2 * j] = lo_half<DT>(x.w[j]);
      o[2 * j + 1] = hi_half<DT>(x.w[j]);
    }
  }
}
// Magnitudes are compared as unsigned bits, two 16-bit ones at a time: ordered like
// the values, a NaN above all of them.
template <int DT>
__device__ __forceinline__ uint32_t max_magnitude(uint32_t t, uint32_t w) {
  if constexpr (DT == GM_F32) return max(t, w & 0x7FFFFFFFu);
  else return __vmaxu2(t, w & 0x7FFF7FFFu);
}
// fp32 bits of the largest magnitude of eight.
template <int DT>
__device__ __forceinline__ uint32_t top8(const Eight<DT>& x) {
  uint32_t t = 0;
#pragma unroll
  for (int j = 0; j < (DT == GM_F32 ? 8 : 4); ++j) t = max_magnitude<DT>(t, x.w[j]);
  if constexpr (DT == GM_F32) return t;
  else return __float_as_uint(lo_half<DT>(max(t & 0xFFFFu, t >> 16)));
}

// --------------------------------------------------------------------- encoding
// Codes of eight values, element 0 in the lowest nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float (&y)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return w;
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

constexpr float kBelow = 1.0f - 9.5367431640625e-7f, kAbove = 1.0f + 9.5367431640625e-7f;   // 1 -+ 2^-20

// Matrix-wide constants of GM_NV4; for GM_MX4 unused.
struct MatrixScale {
  float gs;
  float inv6;      // 1 / (6 gs)
  bool exact;      // fp32 quotients would leave its normal range: decide in fp64
};
template <int FMT>
__device__ __forceinline__ MatrixScale matrix_scale(const float* gscale, int b) {
  MatrixScale g{1.f, 0.f, false};
  if constexpr (FMT == GM_NV4) {
    g.gs = gscale[b];
    g.exact = !(g.gs >= 1e-28f && g.gs <= 1e28f);
    g.inv6 = __fdiv_rn(1.0f, 6.0f * g.gs);
  }
  return g;
}

// |a| against border * gs, exactly, for gs well inside fp32's range: the border has at
// most 7 bits; its product with gs is h + l with h rounded, l the exact rest, and an
// fp32 a other than h lies on h's side of the sum. Does `a` round up (a tie: to even)?
__device__ __forceinline__ bool rounds_up(float a, float border, float gs, bool even_is_up) {
  const float h = border * gs, l = fmaf(border, gs, -h);
  return a != h ? a > h : l != 0.f ? l < 0.f : even_is_up;
}
// e4m3 nearest to top / (6 gs), in fp64: for gs near either end of fp32.
__device__ __noinline__ uint32_t exact_scale(float top, float gs) {
  // 3 fraction bits, exponents from -6, at most 448
  const double t = (double)top / (6.0 * (double)gs);
  const int e = max((__double2hiint(t) >> 20) - 1023, -6);
  const int k = (int)rint(fmin(t, 449.0) * __hiloint2double((3 - e + 1023) << 20, 0));
  return min((uint32_t)(((e + 6) << 3) + k), 126u);
}

// The scale byte of a block whose largest magnitude is `top` (a NaN's bits lie
// above every number's), and what its elements are multiplied by.
template <int FMT>
__device__ __forceinline__ uint32_t block_scale(float top, const MatrixScale& g, float& mul) {
  if constexpr (FMT == GM_MX4) {
    const uint32_t e = __float_as_uint(top) >> 23;   // top >= 0
    if (e == 255u) {
      mul = 0.f;
      return 255u;
    }
    const uint32_t b = e > 2u ? e - 2u : 0u;
    mul = __uint_as_float((254u - b) << 23);
    return b;
  } else {
    mul = 0.f;
    if (!(g.gs > 0.f && g.gs <= 3.402823466e38f)) return 0u;   // a zero matrix, or one that is NaN
    const float t = top * g.inv6;
    const uint32_t q = e4m3x2(t * kBelow, t * kAbove);
    uint32_t b = q & 255u;
    if (b != q >> 8)
      b += rounds_up(top, 3.f * (e4m3_value(b) + e4m3_value(b + 1)), g.gs, (b & 1) != 0) ? 1u : 0u;
    if (g.exact) b = exact_scale(top, g.gs);
    // within 2^-22 of 1 / (sb gs); where it leaves fp32's range the codes are exact_codes'
    if (b) mul = __fdividef(1.0f, e4m3_value(b) * g.gs);
    return b;
  }
}

// Codes of eight elements of a GM_NV4 block in fp64, where sb gs times a border (31 bits
// at most) is exact: for gs near either end of fp32.
struct Values {
  float x[8];
};
__device__ __noinline__ uint32_t exact_codes(Values v, float sb, float gs) {
  const double s = (double)sb * (double)gs;
  uint32_t w = 0;
#pragma unroll 1
  for (int e = 0; e < 8; ++e) {
    const double a = fabs((double)v.x[e]);
    const uint32_t c = (a > 0.25 * s) + (a >= 0.75 * s) + (a > 1.25 * s) + (a >= 1.75 * s) + (a > 2.5 * s) +
                       (a >= 3.5 * s) + (a > 5.0 * s);
    w |= (c | (v.x[e] < 0.f ? 8u : 0u)) << (4 * e);
  }
  return w;
}

// Codes of eight elements of one block; at(e) reads element e again.
template <int FMT, typename At>
__device__ __forceinline__ uint32_t codes8(const float (&x)[8], uint32_t b, float mul, const MatrixScale& g, At&& at) {
  float y[8];
  if constexpr (FMT == GM_MX4) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = x[e] * mul;
    return b == 255u ? 0u : e2m1x8(y);
  } else {
    float z[8];
    const float below = mul * kBelow, above = mul * kAbove;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = x[e] * below;
      z[e] = x[e] * above;
    }
    uint32_t w = e2m1x8(y), d = w ^ e2m1x8(z);
    if (b == 0u) return 0u;
    if (g.exact) return exact_codes(Values{x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]}, e4m3_value(b), g.gs);
    // One call in fifty with bf16 inputs (gs = max|X| / 2688 puts the borders of some
    // block scales on multiples of max|X|): one element at a time, read again, for an
    // index that varies would move all of them to local memory.
    while (d) {
      const int i = (__ffs(d) - 1) & ~3;             // the element's nibble
      d &= ~(15u << i);
      const uint32_t c = w >> i & 7u;                // one step below the other; the border between:
      const float border = __uint_as_float((2 * c + 1) << 21) * 8.507059173023462e37f;   // as e2m1_value
      if (rounds_up(fabsf(at(i >> 2)), border * e4m3_value(b), g.gs, (c & 1) != 0)) w += 1u << i;
    }
    return w;
  }
}

struct QuantParams {
  int m, n;
  const void* X;
  long long ldx, xbs;      // elements
  int vec;                 // rows start on 16 bytes
  float* gscale;           // [B], GM_NV4
  uint8_t *codes, *scales;       // along rows
  uint8_t *codesT, *scalesT;     // along columns
  long long tiles_m, tiles_n;
};

__device__ __forceinline__ const uint8_t* row_ptr(const QuantParams& p, int b, long long r, int es) {
  return static_cast<const uint8_t*>(p.X) + (b * p.xbs + r * p.ldx) * es;
}
template <int DT>
constexpr int kElem = DT == GM_F32 ? 4 : 2;

// The kernel that finds GM_NV4's matrix scale, the one that quantises and the product
// that takes the codes are launched as programmatic dependents: the next may start (its
// set-up, and loads that the one before does not write) once every CTA of the one before
// has, and waits for its results where it needs them.
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ------------------------------------------------------------- the matrix scale
// gscale[b] = max over elements of fp32(|x| / 2688) by atomicMax on its bits (the
// order does not matter; division is monotone, so this is the quotient of the
// maximum); an infinity or a NaN leaves a NaN.
template <int DT>
__global__ void __launch_bounds__(kThreads) k_mx4_top(const QuantParams p) {
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  next_may_start();
  uint32_t top = 0;
  // a warp takes pieces of 1024 elements of a row
  const long long spans = cdivll(p.n, kRowSpan), items = spans * p.m;
  for (long long i = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < items;
       i += (long long)gridDim.x * (kThreads / 32)) {
    long long r;
    if (items < (1LL << 31)) r = (uint32_t)i / (uint32_t)spans;   // a 64-bit division costs more than the loads
    else r = i / spans;
    const int c0 = (int)(i - r * spans) * kRowSpan;
    const void* row = row_ptr(p, b, r, kElem<DT>);
    Eight<DT> x[kRowSpan / 256];
#pragma unroll
    for (int u = 0; u < kRowSpan / 256; ++u) load8<DT>(row, c0 + u * 256 + lane * 8, p.n, p.vec != 0, x[u]);
#pragma unroll
    for (int u = 0; u < kRowSpan / 256; ++u) top = max(top, top8(x[u]));
  }
  top = __reduce_max_sync(0xffffffffu, top);
  __shared__ uint32_t part[kThreads / 32];
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / 32; ++w) top = max(top, part[w]);
    const float t = __uint_as_float(top);
    const float gs = t <= 3.402823466e38f ? __fdiv_rn(t, 2688.0f) : __int_as_float(0x7fffffff);
    atomicMax(reinterpret_cast<unsigned*>(p.gscale + b), __float_as_uint(gs));
  }
}

// -------------------------------------------------------------------- rows only
// A warp takes 256 elements of a row per trip: lane l the eight from 8 l; the
// block's maximum is shared by 4 (GM_MX4) or 2 lanes, a word of four scale bytes
// gathered from 16 or 8. A CTA takes 8 rows and kRowSpan columns. Rows of the last
// 128-row tile behind m get zero scales.
template <int DT, int FMT>
__global__ void __launch_bounds__(kThreads) k_mx4_rows(const QuantParams p, long long spans) {
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const long long r = blockIdx.x / (uint32_t)spans * 8 + (threadIdx.x >> 5);
  const int c0 = (int)(blockIdx.x % (uint32_t)spans) * kRowSpan;
  const int np = (int)mx4_padded(p.n);
  const long long atoms = mx4_atoms(p.n, FMT);
  constexpr int L = mx4_block(FMT) / 8;     // lanes of a block
  uint8_t* sc = p.scales + ((b * p.tiles_m + r / 128) * atoms) * 512 + mx4_atom_byte((int)(r % 128), 0);
  const bool live = r < p.m;
  next_may_start();
  const void* row = row_ptr(p, b, live ? r : 0, kElem<DT>);
  const int n = live ? p.n : 0;
  uint8_t* codes = p.codes + (b * (long long)p.m + r) * (np / 2);
  Eight<DT> x[kRowSpan / 256];
#pragma unroll
  for (int u = 0; u < kRowSpan / 256; ++u)
    load8<DT>(row, c0 + u * 256 + lane * 8, n, p.vec != 0, x[u]);
  if constexpr (FMT == GM_NV4) wait_for_previous();
  const MatrixScale g = matrix_scale<FMT>(p.gscale, b);
#pragma unroll
  for (int u = 0; u < kRowSpan / 256; ++u) {
    const int c = c0 + u * 256 + lane * 8;
    uint32_t top = top8(x[u]);
#pragma unroll
    for (int o = 1; o < L; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    float mul;
    const uint32_t s = block_scale<FMT>(__uint_as_float(top), g, mul);
    if (live && c < np) {
      float v[8];
      to_floats<DT>(x[u], v);
      *reinterpret_cast<uint32_t*>(codes + c / 2) =
          codes8<FMT>(v, s, mul, g, [&](int e) { return load_as_float(row, c + e, DT); });
    }
    // lane 4 L i gathers the bytes of lanes 4 L i, + L, + 2 L, + 3 L
    uint32_t w = s;
    w |= __shfl_down_sync(0xffffffffu, s, L) << 8;
    w |= __shfl_down_sync(0xffffffffu, s, 2 * L) << 16;
    w |= __shfl_down_sync(0xffffffffu, s, 3 * L) << 24;
    if (lane % (4 * L) == 0 && c < np)
      *reinterpret_cast<uint32_t*>(sc + c / (4 * mx4_block(FMT)) * 512) = live ? w : 0u;
  }
}

// ----------------------------------------------------------------- both or columns
// A CTA takes a 128 x 128 tile. Each thread loads eight elements of a row at a time,
// quantises them along the row, and leaves them in shared memory as they are; then it
// takes two neighbouring columns of 32 rows. Scale bytes of both
// orientations are gathered in shared memory and leave as whole atoms.
template <int DT, int FMT>
__global__ void __launch_bounds__(kThreads) k_mx4_tile(const QuantParams p) {
  constexpr int BL = mx4_block(FMT), L = BL / 8, NA = kTile / (4 * BL);   // atoms of a tile: 1 or 2
  constexpr int W = DT == GM_F32 ? 8 : 4;                                 // words of eight elements
  extern __shared__ __align__(16) uint32_t tile[];                        // [kTile][kTile elements]
  __shared__ __align__(16) uint8_t sR[NA * 512], sC[NA * 512];
  const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long tm = blockIdx.x / (uint32_t)p.tiles_n, tn = blockIdx.x % (uint32_t)p.tiles_n;
  const long long r0 = tm * kTile, c0 = tn * kTile;
  const long long np = p.tiles_n * kTile, mp = p.tiles_m * kTile;
  const bool rows = p.codes != nullptr;
  next_may_start();
  MatrixScale g;

  // 16 lanes a row, 16 rows a trip; the loads of kAhead trips together
  const int cl = (lane & 15) * 8, rl0 = warp * 2 + (lane >> 4);
  auto element = [&](int r, int c) {   // of the tile
    if constexpr (DT == GM_F32) return __uint_as_float(tile[r * kTile + c]);
    else return h16_to_float(reinterpret_cast<const uint16_t*>(tile)[r * kTile + c], DT == GM_F16);
  };
  constexpr int kAhead = DT == GM_F32 ? 4 : 8;
  // what is left of the matrix in this tile, and this thread's first row: the loops
  // below count in 32 bits
  const int mrem = (int)min((long long)kTile, p.m - r0), nrem = (int)min((long long)kTile, p.n - c0);
  const uint8_t* src = row_ptr(p, b, r0, kElem<DT>) + (c0 + (long long)rl0 * p.ldx) * kElem<DT>;
  const long long src_step = 16 * p.ldx * kElem<DT>;
  const uint32_t row_bytes = (uint32_t)(np / 2);
  uint8_t* dst = p.codes + ((b * (long long)p.m + r0 + rl0) * np + c0 + cl) / 2;
#pragma unroll 1
  for (int it0 = 0; it0 < kTile / 16; it0 += kAhead) {
    Eight<DT> x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      load8<DT>(src, cl, (it0 + i) * 16 + rl0 < mrem ? nrem : 0, p.vec != 0, x[i]);
      src += src_step;
    }
    if (it0 == 0) {
      if constexpr (FMT == GM_NV4) wait_for_previous();
      g = matrix_scale<FMT>(p.gscale, b);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int rl = (it0 + i) * 16 + rl0;
#pragma unroll
      for (int q = 0; q < W / 4; ++q)
        reinterpret_cast<uint4*>(tile + (rl * kTile + cl) / 8 * W)[q] =
            make_uint4(x[i].w[4 * q], x[i].w[4 * q + 1], x[i].w[4 * q + 2], x[i].w[4 * q + 3]);
      if (rows) {
        uint32_t top = top8<DT>(x[i]);
#pragma unroll
        for (int o = 1; o < L; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        float mul;
        const uint32_t s = block_scale<FMT>(__uint_as_float(top), g, mul);
        const int j = cl / BL;
        if (cl % BL == 0) sR[j / 4 * 512 + mx4_atom_byte(rl, j % 4)] = (uint8_t)(rl < mrem ? s : 0u);
        if (rl < mrem) {
          float v[8];
          to_floats<DT>(x[i], v);
          *reinterpret_cast<uint32_t*>(dst) = codes8<FMT>(v, s, mul, g, [&](int e) { return element(rl, cl + e); });
        }
        dst += 16 * (size_t)row_bytes;
      }
    }
  }
  __syncthreads();

  // Two neighbouring columns cc, cc + 1 (one word of 16-bit elements) of 32 rows a thread.
  const int cc = (warp & 1) * 64 + lane * 2, rb = (warp >> 1) * 32;
  uint32_t w[2][4];
#pragma unroll
  for (int k = 0; k < 32 / BL; ++k) {
    uint32_t v[BL][DT == GM_F32 ? 2 : 1], t[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < BL; ++i) {
      const int at = (rb + k * BL + i) * kTile + cc;
      if constexpr (DT == GM_F32) {
        const uint2 u = *reinterpret_cast<const uint2*>(tile + at);
        v[i][0] = u.x;
        v[i][1] = u.y;
        t[0] = max_magnitude<DT>(t[0], u.x);
        t[1] = max_magnitude<DT>(t[1], u.y);
      } else {
        v[i][0] = tile[at / 2];
        t[0] = max_magnitude<DT>(t[0], v[i][0]);
      }
    }
    if constexpr (DT != GM_F32) {
      const uint32_t u = t[0];
      t[0] = __float_as_uint(lo_half<DT>(u));
      t[1] = __float_as_uint(hi_half<DT>(u));
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float mul;
      const uint32_t s = block_scale<FMT>(__uint_as_float(t[h]), g, mul);
      const int j = rb / BL + k;
      sC[j / 4 * 512 + mx4_atom_byte(cc + h, j % 4)] = (uint8_t)(cc + h < nrem ? s : 0u);
#pragma unroll
      for (int q = 0; q < BL / 8; ++q) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if constexpr (DT == GM_F32) y[e] = __uint_as_float(v[q * 8 + e][h]);
          else y[e] = h ? hi_half<DT>(v[q * 8 + e][0]) : lo_half<DT>(v[q * 8 + e][0]);
        }
        w[h][k * (BL / 8) + q] =
            codes8<FMT>(y, s, mul, g, [&](int e) { return element(rb + k * BL + q * 8 + e, cc + h); });
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (cc + h < nrem)
      *reinterpret_cast<uint4*>(p.codesT + ((b * (long long)p.n + c0 + cc + h) * mp + r0 + rb) / 2) =
          make_uint4(w[h][0], w[h][1], w[h][2], w[h][3]);
  __syncthreads();
  // atoms [row tile][along the row]: NA per tile
  for (int i = threadIdx.x; i < NA * 128; i += kThreads) {
    if (rows)
      reinterpret_cast<uint32_t*>(p.scales + ((b * p.tiles_m + tm) * p.tiles_n + tn) * NA * 512)[i] =
          reinterpret_cast<const uint32_t*>(sR)[i];
    reinterpret_cast<uint32_t*>(p.scalesT + ((b * p.tiles_n + tn) * p.tiles_m + tm) * NA * 512)[i] =
        reinterpret_cast<const uint32_t*>(sC)[i];
  }
}

// ---------------------------------------------------------------------- decoding
template <int FMT>
__global__ void __launch_bounds__(kThreads) k_mx4_dequant(int m, int n, long long tiles_m,
                                                          const uint8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales,
                                                          const float* __restrict__ gscale, void* out,
                                                          int odt, int vec, long long spans) {
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const long long r = blockIdx.x / (uint32_t)spans * 8 + (threadIdx.x >> 5);
  if (r >= m) return;
  const int c0 = (int)(blockIdx.x % (uint32_t)spans) * kRowSpan;
  const long long np = mx4_padded(n), atoms = mx4_atoms(n, FMT);
  const uint8_t* sc = scales + ((b * tiles_m + r / 128) * atoms) * 512 + mx4_atom_byte((int)(r % 128), 0);
  const float gs = FMT == GM_NV4 ? gscale[b] : 1.f;
  const uint8_t* row = codes + (b * (long long)m + r) * (np / 2);
  const long long at = (b * (long long)m + r) * n;
  auto factor = [&](int c) {
    const int j = c / mx4_block(FMT);
    const uint32_t sb = sc[j / 4 * 512 + j % 4];
    return FMT == GM_MX4 ? e8m0_value(sb) : e4m3_value(sb);
  };
  auto value = [&](uint32_t code, float f) {
    const float v = __fmul_rn(e2m1_value(code), f);
    return FMT == GM_NV4 ? __fmul_rn(v, gs) : v;
  };
  if (vec == 8) {
    // 32 bytes a lane (fp32 rows of a multiple of 8)
#pragma unroll
    for (int u = 0; u < kRowSpan / 256; ++u) {
      const int c = c0 + u * 256 + lane * 8;
      if (c >= n) continue;
      const uint32_t w = *reinterpret_cast<const uint32_t*>(row + c / 2);
      const float f = factor(c);
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = value(w >> (4 * e) & 15u, f);
      asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(static_cast<float*>(out) + at + c),
                   "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                   : "memory");
    }
  } else if (vec) {
    // neighbouring lanes write neighbouring groups of four (n is a multiple of 4)
#pragma unroll
    for (int u = 0; u < kRowSpan / 128; ++u) {
      const int c = c0 + u * 128 + lane * 4;
      if (c >= n) continue;
      const uint32_t w = *reinterpret_cast<const uint16_t*>(row + c / 2);
      const float f = factor(c);
      store4_from_float(out, at + c, odt, make_float4(value(w & 15u, f), value(w >> 4 & 15u, f),
                                                      value(w >> 8 & 15u, f), value(w >> 12, f)));
    }
  } else {
    // rows off alignment: eight elements a lane, turned in shared memory so that
    // neighbouring lanes write neighbouring elements
    __shared__ float turn[kThreads / 32][256];
    float* t = turn[threadIdx.x >> 5];
#pragma unroll 1
    for (int u = 0; u < kRowSpan / 256; ++u) {
      const int c = c0 + u * 256;
      if (c >= n) break;
      if (c + lane * 8 < n) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(row + c / 2 + lane * 4);
        const float f = factor(c + lane * 8);
#pragma unroll
        for (int e = 0; e < 8; ++e) t[lane * 8 + e] = value(w >> (4 * e) & 15u, f);
      }
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e * 32 + lane < n) store_from_float(out, at + c + e * 32 + lane, odt, t[e * 32 + lane]);
      __syncwarp();
    }
  }
}

// `dependent`: after k_mx4_top, whose result the kernel waits for.
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, size_t smem, bool dependent, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int DT, int FMT>
cudaError_t quant_t(int B, const QuantParams& p, cudaStream_t s) {
  if constexpr (FMT == GM_NV4) {
    cudaError_t e = cudaMemsetAsync(p.gscale, 0, (size_t)B * 4, s);
    if (e != cudaSuccess) return e;
    const long long blocks = cdivll(cdivll(p.n, kRowSpan) * p.m, kThreads / 32);
    const long long want = cdivll(6LL * sm_count(), B);
    const int gx = (int)(blocks < want ? blocks : want);
    k_mx4_top<DT><<<dim3(gx, B), kThreads, 0, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (p.codesT) {
    constexpr size_t bytes = (size_t)kTile * kTile * kElem<DT>;
    if constexpr (DT == GM_F32) {
      static DeviceOnce once;
      const cudaError_t e = smem_attr_once(once, k_mx4_tile<DT, FMT>, bytes);
      if (e != cudaSuccess) return e;
    }
    return launch(k_mx4_tile<DT, FMT>, dim3((unsigned)(p.tiles_m * p.tiles_n), B), bytes, FMT == GM_NV4, s, p);
  }
  const long long spans = cdivll(mx4_padded(p.n), kRowSpan);
  return launch(k_mx4_rows<DT, FMT>, dim3((unsigned)(p.tiles_m * 16 * spans), B), 0, FMT == GM_NV4, s, p, spans);
}

}  // namespace

cudaError_t launch_mx4_quant(int B, int m, int n, const void* X, int xdt, long long ldx, long long xbs,
                             int fmt, float* gscale, uint8_t* codes, uint8_t* scales, uint8_t* codesT,
                             uint8_t* scalesT, cudaStream_t s) {
  const int es = xdt == GM_F32 ? 4 : 2;
  QuantParams p{};
  p.m = m; p.n = n;
  p.X = X; p.ldx = ldx; p.xbs = xbs;
  p.vec = reinterpret_cast<uintptr_t>(X) % 16 == 0 && ldx * es % 16 == 0 && (B == 1 || xbs * es % 16 == 0);
  p.gscale = gscale;
  p.codes = codes; p.scales = scales; p.codesT = codesT; p.scalesT = scalesT;
  p.tiles_m = cdivll(m, kTile);
  p.tiles_n = cdivll(n, kTile);
  switch (xdt * 2 + fmt) {
    case GM_F32 * 2 + GM_MX4: return quant_t<GM_F32, GM_MX4>(B, p, s);
    case GM_F32 * 2 + GM_NV4: return quant_t<GM_F32, GM_NV4>(B, p, s);
    case GM_BF16 * 2 + GM_MX4: return quant_t<GM_BF16, GM_MX4>(B, p, s);
    case GM_BF16 * 2 + GM_NV4: return quant_t<GM_BF16, GM_NV4>(B, p, s);
    case GM_F16 * 2 + GM_MX4: return quant_t<GM_F16, GM_MX4>(B, p, s);
    case GM_F16 * 2 + GM_NV4: return quant_t<GM_F16, GM_NV4>(B, p, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_mx4_dequant(int B, int m, int n, int fmt, const uint8_t* codes, const uint8_t* scales,
                               const float* gscale, void* out, int odt, cudaStream_t s) {
  const long long spans = cdivll(n, kRowSpan), tiles_m = cdivll(m, kTile);
  const dim3 grid((unsigned)(cdivll(m, 8) * spans), B);
  const int vec = odt == GM_F32 && n % 8 == 0 && reinterpret_cast<uintptr_t>(out) % 32 == 0 ? 8 : n % 4 == 0 ? 4 : 0;
  if (fmt == GM_MX4)
    k_mx4_dequant<GM_MX4><<<grid, kThreads, 0, s>>>(m, n, tiles_m, codes, scales, gscale, out, odt, vec, spans);
  else
    k_mx4_dequant<GM_NV4><<<grid, kThreads, 0, s>>>(m, n, tiles_m, codes, scales, gscale, out, odt, vec, spans);
  return cudaGetLastError();
}

}  // namespace gm
