// Products of microscaled 4-bit operands: D[i][j] = sum_k A[i][k] B[j][k] (+ D), the
// sum in fp32, rounded once to D's type.

#include "gm_common.cuh"
#include "gm_internal.h"
#include "gm_mx4.cuh"

namespace gm {
namespace {

struct ProductParams {
  int M, N, K;
  const uint8_t *a, *as;
  const float* ag;
  const uint8_t *b, *bs;
  const float* bg;
  void* D;
  int ddt, accumulate;
};

// A 64 x 64 tile of D per CTA, operands decoded into shared memory 64 columns at a
// time, 4 x 4 outputs a thread.
template <int FMT>
__global__ void __launch_bounds__(256) k_mx4_matmul(const ProductParams p) {
  __shared__ float sA[64][65], sB[64][65];
  const int bz = blockIdx.z, i0 = blockIdx.x * 64, j0 = blockIdx.y * 64;
  const long long kp = mx4_padded(p.K), atoms = mx4_atoms(p.K, FMT);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  auto fill = [&](float (&s)[64][65], const uint8_t* codes, const uint8_t* scales, int rows, int r0, long long k0) {
    for (int i = threadIdx.x; i < 64 * 8; i += 256) {
      const int r = r0 + i / 8;
      const long long c = k0 + (i % 8) * 8;
      uint32_t w = 0, sb = 0;
      if (r < rows) {
        w = *reinterpret_cast<const uint32_t*>(codes + (((long long)bz * rows + r) * kp + c) / 2);
        const long long j = c / mx4_block(FMT);
        sb = scales[((long long)bz * cdiv(rows, 128) + r / 128) * atoms * 512 + j / 4 * 512 +
                    mx4_atom_byte(r % 128, (int)(j % 4))];
      }
      const float f = r < rows ? (FMT == GM_MX4 ? e8m0_value(sb) : e4m3_value(sb)) : 0.f;
      for (int e = 0; e < 8; ++e) s[i / 8][(i % 8) * 8 + e] = e2m1_value((w >> (4 * e)) & 15u) * f;
    }
  };
  for (long long k0 = 0; k0 < kp; k0 += 64) {
    fill(sA, p.a, p.as, p.M, i0, k0);
    fill(sB, p.b, p.bs, p.N, j0, k0);
    __syncthreads();
    for (int k = 0; k < 64; ++k)
      for (int u = 0; u < 4; ++u)
        for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(sA[ty + 16 * u][k], sB[tx + 16 * v][k], acc[u][v]);
    __syncthreads();
  }
  const float alpha = FMT == GM_NV4 ? p.ag[bz] * p.bg[bz] : 1.f;
  for (int u = 0; u < 4; ++u)
    for (int v = 0; v < 4; ++v) {
      const int i = i0 + ty + 16 * u, j = j0 + tx + 16 * v;
      if (i >= p.M || j >= p.N) continue;
      const long long at = ((long long)bz * p.M + i) * p.N + j;
      float d = acc[u][v] * alpha;
      if (p.accumulate) d += load_as_float(p.D, at, p.ddt);
      store_from_float(p.D, at, p.ddt, d);
    }
}

}  // namespace

size_t mx4_matmul_ws_bytes(int, int, int, int) { return 0; }

cudaError_t launch_mx4_matmul(int B, int M, int N, int K, int fmt, const uint8_t* a, const uint8_t* as,
                              const float* ag, const uint8_t* b, const uint8_t* bs, const float* bg,
                              void* D, int ddt, int accumulate, void*, cudaStream_t s) {
  const ProductParams p{M, N, K, a, as, ag, b, bs, bg, D, ddt, accumulate};
  const dim3 grid(cdiv(M, 64), cdiv(N, 64), B);
  if (fmt == GM_MX4) k_mx4_matmul<GM_MX4><<<grid, 256, 0, s>>>(p);
  else k_mx4_matmul<GM_NV4><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace gm
