// Microscaled 4-bit operands: layout and element formats shared by the codec
// (gm_mx4.cu) and the product (gm_mx4_gemm.cu).
#pragma once

#include "gm_common.cuh"

namespace gm {

// Elements are e2m1 (sign, 2 exponent bits, 1 mantissa bit): 0, .5, 1, 1.5, 2, 3,
// 4, 6. Blocks of 32 along a row with a power-of-two scale (GM_MX4), or of 16 with
// an e4m3 scale under one fp32 scale of the matrix (GM_NV4).
__host__ __device__ constexpr int mx4_block(int fmt) { return fmt == GM_MX4 ? 32 : 16; }

// Rows are padded to a multiple of 128 elements with zeros: 64-byte rows of codes,
// and whole scale atoms. An atom is 512 bytes: the scales of 128 rows and 4
// consecutive blocks, byte (r % 32) * 16 + (r / 32) * 4 + j, which is the order in
// which the tensor cores read scales from tensor memory.
__host__ __device__ constexpr long long mx4_padded(long long cols) { return (cols + 127) / 128 * 128; }
__host__ __device__ constexpr long long mx4_atoms(long long cols, int fmt) {   // along a row
  return mx4_padded(cols) / (4 * mx4_block(fmt));
}
__host__ __device__ constexpr int mx4_atom_byte(int r, int j) {   // r < 128, j < 4
  return (r & 31) * 16 + (r >> 5) * 4 + j;
}

// ------------------------------------------------------------------- decoding
__device__ __forceinline__ float e2m1_value(uint32_t code) {
  // the code's exponent and mantissa sit at fp32's lowest exponents, 126 too low
  return __uint_as_float(((code & 7u) << 22) | ((code & 8u) << 28)) * 8.507059173023462e37f;   // 2^126
}
__device__ __forceinline__ float e8m0_value(uint32_t b) {   // 2^(b - 127); 255: NaN
  return b == 255u ? __int_as_float(0x7fffffff) : __uint_as_float(b ? b << 23 : 0x00400000u);
}
__device__ __forceinline__ float e4m3_value(uint32_t b) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)b));
  return __half2float(__ushort_as_half((uint16_t)(d & 0xFFFFu)));
}

}  // namespace gm
