// AdamW over many tensors in one launch, its states in 32 or in 8 bits, and the
// global gradient norm with the clip factor: the step of the parameters that
// Muon does not take (embeddings, heads, norms, biases).
//
// Per element, with t the completed steps plus one and c the clip factor:
//   g <- c g,  m <- b1 m + (1 - b1) g,  v <- b2 v + (1 - b2) g^2,
//   p <- (1 - lr wd) p - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps).
//
// HBM moves 28 B per element with fp32 states and an fp32 gradient, 14.1 B with 8-bit
// states and a 16-bit gradient; one pass moves each byte once. The tensor table travels
// in the kernel's parameters, so a list of any addresses needs no copy to the device
// and can be captured into a graph. Measured on 1e8 elements with a bf16 gradient and a
// bf16 copy: 32-bit states 412 us (6.8 TB/s: HBM); 8-bit states 374 us (4.3 TB/s),
// bound by issue: 88 instructions an element, 64 % of the issue slots (scales rounded
// from fp64, without which the states would drift from their definition, cost 51 us).

#include <math.h>

#include "gm_common.cuh"
#include "gm_internal.h"

namespace gm {
namespace {

constexpr int kGroup8 = 128;      // elements per scale of an 8-bit state
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// ------------------------------------------------------------ work distribution
// The list is cut into chunks of kChunk elements of one tensor; first[i] is the
// first chunk of tensor i. A CTA walks chunks blockIdx.x, + gridDim.x, ...
template <int N>
struct ChunkMap {
  int count;
  int first[N + 1];
  __device__ __forceinline__ int total() const { return first[count]; }
  // The tensor of a chunk at or after tensor i's first chunk.
  __device__ __forceinline__ int find(int chunk, int i) const {
    if (chunk < first[i + 1]) return i;
    int lo = i + 1, hi = count - 1;   // first[lo] <= chunk < first[hi + 1]
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= chunk) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  }
};

// ------------------------------------------------------------------ load / store
// Eight consecutive elements from i on, `n` of them inside the tensor (n <= 0:
// none). WHOLE: all of them, and the array is aligned to eight elements.
template <int DT>
__device__ __forceinline__ float one(const void* p, long long i) {
  if constexpr (DT == GM_F32) return static_cast<const float*>(p)[i];
  else return h16_to_float(static_cast<const uint16_t*>(p)[i], DT == GM_F16);
}
template <int DT, bool WHOLE>
__device__ __forceinline__ void load8(const void* p, long long i, long long n, float (&o)[8]) {
  if constexpr (!WHOLE) {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = e < n ? one<DT>(p, i + e) : 0.f;
  } else if constexpr (DT == GM_F32) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(o[0]), "=f"(o[1]), "=f"(o[2]), "=f"(o[3]), "=f"(o[4]), "=f"(o[5]), "=f"(o[6]), "=f"(o[7])
                 : "l"(static_cast<const float*>(p) + i)
                 : "memory");
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[2 * j] = h16_to_float((uint16_t)(w[j] & 0xFFFFu), DT == GM_F16);
      o[2 * j + 1] = h16_to_float((uint16_t)(w[j] >> 16), DT == GM_F16);
    }
  }
}
template <bool WHOLE>
__device__ __forceinline__ void store8(void* p, long long i, long long n, int dt, const float (&v)[8]) {
  if constexpr (!WHOLE) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) store_from_float(p, i + e, dt, v[e]);
  } else if (dt == GM_F32) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(static_cast<float*>(p) + i),
                 "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = (uint32_t)float_to_h16(v[2 * j], dt == GM_F16) | ((uint32_t)float_to_h16(v[2 * j + 1], dt == GM_F16) << 16);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
template <bool WHOLE>
__device__ __forceinline__ uint2 load8_codes(const uint8_t* p, long long i, long long n) {
  if constexpr (WHOLE) return *reinterpret_cast<const uint2*>(p + i);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) w[e >> 2] |= (uint32_t)p[i + e] << (8 * (e & 3));
  return make_uint2(w[0], w[1]);
}
template <bool WHOLE>
__device__ __forceinline__ void store8_codes(uint8_t* p, long long i, long long n, uint2 w) {
  if constexpr (WHOLE) {
    *reinterpret_cast<uint2*>(p + i) = w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) p[i + e] = (uint8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3)));
  }
}

// ------------------------------------------------------------------ 8-bit states
// m: e4m3 codes under sm = max(max|m| / 448, 2^-126). v: its root r under
// sv = max(max r / 1.9375, 2^-126), as a float of four exponent and four mantissa
// bits without a sign (2^-18 to 1.9375; r spans v's range at half its exponents,
// and half a step is 3 % of r). A v that fp32 holds as non-zero keeps code 1 at
// least, so that no denominator falls to eps while m lives. The floor 2^-126
// keeps 1 / scale finite.
constexpr float kScaleFloor = 1.17549435e-38f;   // 2^-126
constexpr float kTopM = 448.0f, kTopR = 1.9375f;

__device__ __forceinline__ float scale_of(float top, float inv_max) {
  // an infinity or a NaN stays: it decides what the whole group stands for
  return top <= 3.402823466e38f ? fmaxf(__fmul_rn(top, inv_max), kScaleFloor) : top;
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ void e4m3x4_to_float(uint32_t w, float (&o)[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)(w >> (16 * h))));
    o[2 * h] = __half2float(__ushort_as_half((uint16_t)(d & 0xFFFFu)));
    o[2 * h + 1] = __half2float(__ushort_as_half((uint16_t)(d >> 16)));
  }
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)code));
  return __half2float(__ushort_as_half((uint16_t)(d & 0xFFFFu)));
}
// Exponents 0..15 of the 4 + 4 bit float are fp32's own lowest ones (a value x is
// kept as the fp32 number x 2^-112): code << 19 are that number's bits, subnormals
// included, and rounding is on the bits.
__device__ __forceinline__ float root_value(uint32_t code) {
  return __fmul_rn(__uint_as_float(code << 19), 5.192296858534828e33f);   // 2^112
}
__device__ __forceinline__ float approx_sqrt(float x) {   // 2^-22; x from 2^-126 on
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float approx_rcp(float x) {    // 2^-23
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float max_nan(float a, float b) {   // a NaN where either is one
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Both codes from fp64 values (round to nearest, ties to even).
__device__ __forceinline__ double pow2d(int e) { return __hiloint2double((e + 1023) << 20, 0); }
__device__ __forceinline__ uint32_t e4m3_from_double(double y) {
  const double a = fmin(fabs(y), 448.0);
  const int e = max((__double2hiint(a) >> 20) - 1023, -6);
  const int k = (int)rint(a * pow2d(3 - e));
  return (uint32_t)(((e + 6) << 3) + k) | (y < 0.0 ? 0x80u : 0u);
}
__device__ __forceinline__ uint32_t root_from_double(double y, double v) {
  const int e = max((__double2hiint(y) >> 20) - 1023, -14);
  const int k = (int)rint(fmin(y, 2.0) * pow2d(4 - e));
  const uint32_t c = min((uint32_t)(((e + 14) << 4) + k), 255u);
  return (float)v > 0.f ? max(c, 1u) : c;
}

// Maxima over the 16 lanes that hold a group.
__device__ __forceinline__ double group_max(double x) {
#pragma unroll
  for (int o = 8; o; o >>= 1) x = fmax(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ uint32_t group_max(uint32_t x) {
#pragma unroll
  for (int o = 8; o; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// --------------------------------------------------------------------- the step
// What every chunk of a step needs, computed once per step by k_adamw_begin.
struct Coef {
  double c;          // clip factor (1 without) over c1
  float c32;
  float c1;          // 1, or a power of two that gradients take first (see k_adamw_begin)
  float decay;       // 1 - lr wd
  float scale;       // lr / (1 - b1^t)
  float root;        // 1 / sqrt(1 - b2^t)
  float root8, eps8; // root / scale, eps / scale: the update is m / (r root8 + eps8)
  int skip;
};
static_assert(sizeof(Coef) <= GM_ADAMW_SCRATCH_BYTES, "the step's scratch holds the coefficients");

__global__ void k_adamw_begin(double lr, double b1, double b2, double eps, double wd,
                              const double* clip, const float* lr_dev, const int32_t* skip, int64_t* step, Coef* out) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (skip && *skip) {
    out->skip = 1;
    return;
  }
  const long long t = *step + 1;
  *step = t;
  const double l = lr_dev ? (double)*lr_dev : lr;
  // A clip factor that, alone or times 1 - b1 or the root of 1 - b2, is no normal fp32
  // number (a norm near fp32's end gives one): gradients take a power of two first, which
  // leaves a factor that is. It is exact but for products that fp32 cannot hold either.
  const double c = clip ? *clip : 1.0, a = fabs(c);
  const bool low = c != 0.0 && a * fmin(1.0 - b1, sqrt(1.0 - b2)) < pow2d(-126);
  const double c1 = a > pow2d(127) ? pow2d(126) : low ? pow2d(a < pow2d(-150) ? -126 : -64) : 1.0;
  out->c = c / c1;
  out->c32 = (float)(c / c1);
  out->c1 = (float)c1;
  out->decay = (float)(1.0 - l * wd);
  const double s = l / (1.0 - pow(b1, (double)t)), r = 1.0 / sqrt(1.0 - pow(b2, (double)t));
  out->scale = (float)s;
  out->root = (float)r;
  // a rate of zero: a denominator whose reciprocal is zero
  out->root8 = fabs(s) > 1e-20 ? (float)(r / s) : 0.f;
  out->eps8 = fabs(s) > 1e-20 ? (float)(eps / s) : 3e38f;
  out->skip = 0;
}

struct Entry {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* mscale;
  float* vscale;
  void* copy;
  long long numel;
};
// Tensors per launch: a table of 30.4 KB of the 32 KB of parameters, or, for short
// lists, one of 2.2 KB (the call takes 9 us less of the host's time).
constexpr int kMaxTensors = 440, kFewTensors = 32;
template <int N>
struct Table {
  ChunkMap<N> map;
  uint8_t vec[N];
  Entry e[N];
};
struct Consts {
  float b1, ob1, b2, ob2, eps;   // ob = 1 - b, rounded once from fp64
  float rb2, rob2;               // roots of b2 and ob2
  double db1, dob1, db2, dob2;
  int cdt;
};

constexpr int kPart = 256;                  // elements of a warp at a time: two groups, eight a lane
constexpr int kChunk = kWarps * kPart;

// The codes and scales of two groups in fp64, eight elements a lane (kept out of
// line: one part in thirty comes here).
struct Codes8 {
  uint2 m, v;
  float sm, sv;
};
struct Eight {
  float x[8];
};
__device__ __noinline__ Codes8 exact_codes(const Consts k, double c, Eight g, uint2 mc, uint2 vc, float ms, float vs) {
  float mo[8], ml[4], mh[4];
  e4m3x4_to_float(mc.x, ml);
  e4m3x4_to_float(mc.y, mh);
#pragma unroll
  for (int e = 0; e < 8; ++e) mo[e] = e < 4 ? ml[e & 3] : mh[e & 3];
  double dm[8], dv[8], xm = 0.0, xv = 0.0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const double gd = __dmul_rn((double)g.x[e], c);
    const double rd = (double)root_value((e < 4 ? vc.x : vc.y) >> (8 * (e & 3)) & 255u) * (double)vs;
    const double md = (double)mo[e] * (double)ms;
    dm[e] = __dadd_rn(__dmul_rn(k.db1, md), __dmul_rn(k.dob1, gd));
    dv[e] = __dadd_rn(__dmul_rn(k.db2, __dmul_rn(rd, rd)), __dmul_rn(k.dob2, __dmul_rn(gd, gd)));
    xm = fmax(xm, fabs(dm[e]));
    xv = fmax(xv, dv[e]);
  }
  const double dsm = fmax(__dmul_rn(group_max(xm), 1.0 / 448.0), pow2d(-126));
  const double dsv = fmax(__dmul_rn(sqrt(group_max(xv)), 1.0 / 1.9375), pow2d(-126));
  Codes8 o{make_uint2(0, 0), make_uint2(0, 0), (float)dsm, (float)dsv};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t a = e4m3_from_double(dm[e] / dsm) << (8 * (e & 3));
    const uint32_t b = root_from_double(sqrt(dv[e]) / dsv, dv[e]) << (8 * (e & 3));
    if (e < 4) {
      o.m.x |= a;
      o.v.x |= b;
    } else {
      o.m.y |= a;
      o.v.y |= b;
    }
  }
  return o;
}

__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Eight elements a lane, element i the first. WHOLE: the warp's part lies inside the
// tensor, whose arrays are aligned to eight elements.
template <int PDT, int GDT, int BITS, bool WHOLE>
__device__ __forceinline__ void step_part(const Entry& E, const Consts& k, const Coef* coef, const Coef& f,
                                          long long i, int lane) {
  const long long n = E.numel - i;
  float p[8], g[8];
  load8<PDT, WHOLE>(E.p, i, n, p);
  load8<GDT, WHOLE>(E.g, i, n, g);
  if (f.c1 != 1.f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] *= f.c1;
  }
  if constexpr (BITS == 32) {
    float m[8], v[8];
    load8<GM_F32, WHOLE>(E.m, i, n, m);
    load8<GM_F32, WHOLE>(E.v, i, n, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float gc = g[e] * f.c32;
      m[e] = fmaf(k.b1, m[e], k.ob1 * gc);
      // in this order: g^2 alone leaves fp32's range before (1 - b2) g^2 does
      v[e] = fmaf(k.ob2 * gc, gc, k.b2 * v[e]);
      const float u = __fdiv_rn(m[e], fmaf(__fsqrt_rn(v[e]), f.root, k.eps));
      p[e] = fmaf(p[e], f.decay, -u * f.scale);
    }
    store8<WHOLE>(E.m, i, n, GM_F32, m);
    store8<WHOLE>(E.v, i, n, GM_F32, v);
    store8<WHOLE>(E.p, i, n, PDT, p);
    if (E.copy) store8<WHOLE>(E.copy, i, n, k.cdt, p);
  } else {
    const long long grp = i / kGroup8;
    const bool in = WHOLE || n + (lane & 15) * 8 > 0;     // the group begins inside the tensor
    const uint2 mc = load8_codes<WHOLE>(static_cast<const uint8_t*>(E.m), i, n);
    const uint2 vc = load8_codes<WHOLE>(static_cast<const uint8_t*>(E.v), i, n);
    const float ms = in ? E.mscale[grp] : 0.f, vs = in ? E.vscale[grp] : 0.f;
    // b1 sm and the roots of b2 and 1 - b2 go into the group's factors:
    // m' = code (b1 sm) + g (1 - b1) c, v' = (root sv sqrt(b2))^2 + (g c sqrt(1 - b2))^2
    const float ma = k.b1 * ms, va = k.rb2 * vs;
    const float cm = k.ob1 * f.c32, cv = k.rob2 * f.c32;
    float m[8], size[8], r[8];
    uint32_t vb[8];
    {
      float ml[4], mh[4];
      e4m3x4_to_float(mc.x, ml);
      e4m3x4_to_float(mc.y, mh);
#pragma unroll
      for (int e = 0; e < 8; ++e) m[e] = e < 4 ? ml[e & 3] : mh[e & 3];
    }
    float tm = 0.f, ts = 0.f;
    uint32_t tvb = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = m[e] * ma, b = g[e] * cm;
      const float r0 = root_value((e < 4 ? vc.x : vc.y) >> (8 * (e & 3)) & 255u) * va, g0 = g[e] * cv;
      size[e] = fabsf(a) + fabsf(b);
      m[e] = a + b;
      float v = fmaf(r0, r0, g0 * g0);
      if constexpr (!WHOLE) {
        // behind the tensor's end: nothing, whatever the group's scales are (0 under an
        // infinite scale would be a NaN)
        if (e >= n) m[e] = size[e] = v = 0.f;
      }
      // Approximations (2^-21 of an update) and factors taken out of the loop keep this
      // kernel off its issue rate. A v below 2^-126 has a root below 1.1e-19, taken as
      // zero: nothing beside an eps of 1e-12, the least that is accepted.
      r[e] = approx_sqrt(v);
      p[e] = fmaf(p[e], f.decay, -m[e] * approx_rcp(fmaf(r[e], f.root8, f.eps8)));
      vb[e] = __float_as_uint(v);     // never negative: ordered like the values, a NaN above
      tm = max_nan(tm, fabsf(m[e]));
      tvb = max(tvb, vb[e]);
      ts = fmaxf(ts, size[e]);
    }
    store8<WHOLE>(E.p, i, n, PDT, p);
    if (E.copy) store8<WHOLE>(E.copy, i, n, k.cdt, p);
    const uint32_t tmb = __float_as_uint(tm), gm = group_max(tmb), gv = group_max(tvb);
    tm = __uint_as_float(gm);
    const float tv = __uint_as_float(gv);
    const float sm = scale_of(tm, 1.0f / kTopM), sv = scale_of(approx_sqrt(tv), 1.0f / kTopR);
    // The stored codes are those of m and r in fp64 (each product and sum rounded
    // singly, 1 / 448 and 1 / 1.9375 being constants: true ties occur, for m and r
    // are made of short numbers, and the roundings decide them). fp32 decides a code
    // unless its value lies so close to a border that its error could cross it;
    // then the groups are redone in fp64. Errors, u = 2^-24: m is off by 5 u size at
    // most (two products of three roundings, one sum), and m / sm by that, by 6 u, and
    // by sm's relative error, 5 u size / tm of the top element: size up to 3 tm is
    // allowed for (26 u size in all), a group with more is redone. r / sv is off by 23 u.
    // Near fp32's subnormals these bounds do not hold: 2^-90 and 2^-80 keep the
    // smallest element that gets a code (2^-18 of the top) and its square above them,
    // and 2^14 keeps 1 / sv 2^112 below.
    bool near = f.c1 != 1.f || ts > 3.f * tm;   // (the scales below read gradients again)
    if (tm < 8.1e-28f || tv < 8.3e-25f || sv > 16384.f) near |= ts > 0.f || tvb > 0;
    const float im = approx_rcp(sm), iv = approx_rcp(sv) * 1.925929944387236e-34f;   // 2^-112
    const float w = im * 1.66893005e-6f;   // 28 u
    float lo[8], hi[8];
    uint32_t cr[8], gap = ~0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float y = m[e] * im;
      lo[e] = fmaf(size[e], -w, y);
      hi[e] = fmaf(size[e], w, y);
      // a border is at a set bit 18 with zeros below; +-24 (24 to 48 u) around it
      const uint32_t bits = __float_as_uint(r[e] * iv) + 0x40000u + 24u;
      gap = min(gap, bits & 0x7FFFFu);
      cr[e] = max(bits >> 19, min(vb[e], 1u));
    }
    uint2 wm = make_uint2(e4m3x2(lo[0], lo[1]) | (e4m3x2(lo[2], lo[3]) << 16),
                          e4m3x2(lo[4], lo[5]) | (e4m3x2(lo[6], lo[7]) << 16));
    near |= gap <= 48u || wm.x != (e4m3x2(hi[0], hi[1]) | (e4m3x2(hi[2], hi[3]) << 16)) ||
            wm.y != (e4m3x2(hi[4], hi[5]) | (e4m3x2(hi[6], hi[7]) << 16));
    uint2 wv = make_uint2(bytes4(cr[0], cr[1], cr[2], cr[3]), bytes4(cr[4], cr[5], cr[6], cr[7]));
    // each moment by itself: a v that passes fp32's range leaves m as it is defined
    const bool finite_m = tm <= 3.402823466e38f, finite_v = tv <= 3.402823466e38f;
    if (!finite_v) {
      // codes 1 for what is not zero: infinite (or NaN) under this scale
#pragma unroll
      for (int e = 0; e < 8; ++e) cr[e] = min(vb[e], 1u);
      wv = make_uint2(bytes4(cr[0], cr[1], cr[2], cr[3]), bytes4(cr[4], cr[5], cr[6], cr[7]));
    }
    if (__any_sync(0xffffffffu, near)) {
      const Codes8 o = exact_codes(k, coef->c, Eight{g[0], g[1], g[2], g[3], g[4], g[5], g[6], g[7]}, mc, vc, ms, vs);
      if (finite_m) wm = o.m;
      if (finite_v) wv = o.v;
      if ((lane & 15) == 0 && in) {
        E.mscale[grp] = finite_m ? o.sm : sm;
        E.vscale[grp] = finite_v ? o.sv : sv;
      }
    } else {
      // The scales are rounded from fp64 too: a last place of fp32 in a scale would move
      // the next step's codes. The group's fp64 maximum is in a lane whose fp32 maximum
      // comes within kTie places of the group's: of two elements each m is off by 15 u of
      // the top (5 u size, see above), each v by 10 u of itself (its factors, counted
      // twice by the squares, and two roundings), and a place is u or more. The eight
      // elements of such a lane are computed again, one a lane, m by the first eight lanes
      // of the group's sixteen and v by the others; nearly always there is one such lane.
      constexpr uint32_t kTie = 32;
      const int first = lane & 16;
      const uint32_t om = __ballot_sync(0xffffffffu, gm ? tmb + kTie >= gm : lane == first);
      const uint32_t ov = __ballot_sync(0xffffffffu, gv ? tvb + kTie >= gv : lane == first);
      const bool of_v = (lane & 8) != 0;
      const double scale = (double)(of_v ? vs : ms);
      uint32_t todo = (of_v ? ov : om) >> first & 0xFFFFu;
      const long long group0 = i - (lane & 15) * 8 + (lane & 7);
      double d = 0.0;
      do {
        const long long at = group0 + (__ffs(todo) - 1) * 8;
        const int src = first + max(__ffs(todo) - 1, 0);
        const uint32_t mx = __shfl_sync(0xffffffffu, mc.x, src), my = __shfl_sync(0xffffffffu, mc.y, src);
        const uint32_t vx = __shfl_sync(0xffffffffu, vc.x, src), vy = __shfl_sync(0xffffffffu, vc.y, src);
        if (todo && (WHOLE || at < E.numel)) {
          const uint32_t code = (of_v ? (lane & 4 ? vy : vx) : (lane & 4 ? my : mx)) >> (8 * (lane & 3)) & 255u;
          double x = (double)(of_v ? root_value(code) : e4m3_value(code)) * scale;
          double y = __dmul_rn((double)one<GDT>(E.g, at), coef->c);
          if (of_v) {
            x = __dmul_rn(x, x);
            y = __dmul_rn(y, y);
          }
          d = fmax(d, fabs(__dadd_rn(__dmul_rn(of_v ? k.db2 : k.db1, x), __dmul_rn(of_v ? k.dob2 : k.dob1, y))));
        }
        todo &= todo - 1;
      } while (__any_sync(0xffffffffu, todo));
#pragma unroll
      for (int o = 4; o; o >>= 1) d = fmax(d, __shfl_xor_sync(0xffffffffu, d, o));
      if (of_v) {
        // the root by two of Newton's steps from fp32's (2^-21, 2^-42, fp64's last place)
        const double r0 = (double)approx_sqrt(tv), h = (double)(0.5f * approx_rcp(fmaxf((float)r0, kScaleFloor)));
        const double r1 = fma(fma(-r0, r0, d), h, r0);
        d = fma(fma(-r1, r1, d), h, r1);
      }
      if (in && (lane & 7) == 0) {
        const float f = (float)fmax(__dmul_rn(d, of_v ? 1.0 / 1.9375 : 1.0 / 448.0), pow2d(-126));
        if (of_v) E.vscale[grp] = finite_v ? f : sv;
        else E.mscale[grp] = finite_m ? f : sm;
      }
    }
    store8_codes<WHOLE>(static_cast<uint8_t*>(E.m), i, n, wm);
    store8_codes<WHOLE>(static_cast<uint8_t*>(E.v), i, n, wv);
  }
}

// 32-bit states: 64 registers, for a fourth CTA on each SM (LLaMA-1.1B set 3680 us, 3825
// with three).
template <int PDT, int GDT, int BITS, int N>
__global__ void __launch_bounds__(kThreads, BITS == 32 ? 4 : 3)
    k_adamw(const __grid_constant__ Table<N> t, const Consts k, const Coef* coef) {
  // k_adamw_begin may still be writing *coef until here: no __restrict__, which would
  // promise that nothing writes it while this kernel lives
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Coef f = *coef;
  if (f.skip) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int ti = 0;
  for (int chunk = blockIdx.x; chunk < t.map.total(); chunk += gridDim.x) {
    ti = t.map.find(chunk, ti);
    const Entry& E = t.e[ti];
    const long long base = (long long)(chunk - t.map.first[ti]) * kChunk + warp * kPart;
    if (t.vec[ti] && base + kPart <= E.numel)
      step_part<PDT, GDT, BITS, true>(E, k, coef, f, base + lane * 8, lane);
    else if (base < E.numel)
      step_part<PDT, GDT, BITS, false>(E, k, coef, f, base + lane * 8, lane);
  }
}

// ------------------------------------------------------ 8-bit states to fp32
struct UnpackEntry {
  const uint8_t* m;
  const uint8_t* v;
  const float* mscale;
  const float* vscale;
  float* m_out;
  float* v_out;
  long long numel;
};
constexpr int kMaxUnpack = 480;
template <int N>
struct UnpackTable {
  ChunkMap<N> map;
  uint8_t vec[N];
  UnpackEntry e[N];
};

template <bool WHOLE>
__device__ __forceinline__ void unpack_part(const UnpackEntry& E, long long i) {
  const long long n = E.numel - i;
  const uint2 mc = load8_codes<WHOLE>(E.m, i, n), vc = load8_codes<WHOLE>(E.v, i, n);
  const float ms = E.mscale[i / kGroup8], vs = E.vscale[i / kGroup8];
  float ml[4], mh[4], m[8], v[8];
  e4m3x4_to_float(mc.x, ml);
  e4m3x4_to_float(mc.y, mh);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    m[e] = __fmul_rn(e < 4 ? ml[e & 3] : mh[e & 3], ms);
    const float r = __fmul_rn(root_value((e < 4 ? vc.x : vc.y) >> (8 * (e & 3)) & 255u), vs);
    v[e] = __fmul_rn(r, r);
  }
  store8<WHOLE>(E.m_out, i, n, GM_F32, m);
  store8<WHOLE>(E.v_out, i, n, GM_F32, v);
}

template <int N>
__global__ void __launch_bounds__(kThreads) k_adamw_unpack8(const __grid_constant__ UnpackTable<N> t) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int ti = 0;
  for (int chunk = blockIdx.x; chunk < t.map.total(); chunk += gridDim.x) {
    ti = t.map.find(chunk, ti);
    const UnpackEntry& E = t.e[ti];
    const long long base = (long long)(chunk - t.map.first[ti]) * kChunk + warp * kPart;
    if (t.vec[ti] && base + kPart <= E.numel) unpack_part<true>(E, base + lane * 8);
    else if (base + lane * 8 < E.numel) unpack_part<false>(E, base + lane * 8);
  }
}

// ---------------------------------------------------------------- gradient norm
// Sum of squares in fp64, exact to its roundings: a bf16, fp16 or fp32 magnitude
// becomes a double by moving its bits (no conversion instruction, whose rate would
// bound a 16-bit gradient). Its exponent is then short by 896, which one product by
// 2^896 mends, subnormals included; an infinity or a NaN reads as 2^128 or more, so
// a sum of 2^256 or more, which no fp32 norm could hold either, marks them.
struct GradEntry {
  const void* g;
  long long numel;
};
constexpr int kMaxGrads = 1024, kFewGrads = 64;
// Elements of a chunk, and CTAs (and partial sums) of a launch: 4e8 bf16 elements take
// 126 us (6.4 TB/s), 143 us with half the chunk and two thirds of the CTAs. A constant,
// six for each of a B200's SMs: the workspace's size and the order of the sums do not
// change with the device that is current.
constexpr int kNormChunk = 32768;
constexpr int kNormBlocks = 6 * 148;
template <int N>
struct GradTable {
  ChunkMap<N> map;
  uint8_t kind[N];                          // dtype, plus 4 when 16-byte loads are aligned
  GradEntry e[N];
};

__device__ __forceinline__ double widen(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
  return __hiloint2double((int)(b >> 3), (int)(b << 29)) * pow2d(896);
}
__device__ __forceinline__ void add_square(double& acc, float x) {
  const double d = widen(x);
  acc = fma(d, d, acc);
}

template <int DT>
__device__ __forceinline__ void norm_chunk(const void* g, long long base, long long numel, bool vec,
                                           double (&acc)[2]) {
  constexpr int W = DT == GM_F32 ? 4 : 8;   // elements of 16 bytes
  const long long end = min(numel, base + kNormChunk);
  if (!vec) {
    for (long long i = base + threadIdx.x; i < end; i += kThreads) add_square(acc[0], one<DT>(g, i));
    return;
  }
  const long long full = base + (end - base) / W * W;
#pragma unroll 8
  for (long long i = base + (long long)threadIdx.x * W; i < full; i += kThreads * W) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(g) + i * (16 / W));
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (DT == GM_F32) {
        add_square(acc[j & 1], __uint_as_float(x[j]));
      } else {
        add_square(acc[0], h16_to_float((uint16_t)(x[j] & 0xFFFFu), DT == GM_F16));
        add_square(acc[1], h16_to_float((uint16_t)(x[j] >> 16), DT == GM_F16));
      }
    }
  }
  for (long long i = full + threadIdx.x; i < end; i += kThreads) add_square(acc[0], one<DT>(g, i));
}

__device__ __forceinline__ double block_sum(double x) {
  __shared__ double part[kWarps];
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += part[w];
  return s;
}

template <int N>
__global__ void __launch_bounds__(kThreads) k_grad_norm(const __grid_constant__ GradTable<N> t,
                                                        double* __restrict__ part) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  double acc[2] = {0.0, 0.0};
  int ti = 0;
  for (int chunk = blockIdx.x; chunk < t.map.total(); chunk += gridDim.x) {
    ti = t.map.find(chunk, ti);
    const long long base = (long long)(chunk - t.map.first[ti]) * kNormChunk;
    const bool vec = (t.kind[ti] & 4) != 0;
    switch (t.kind[ti] & 3) {
      case GM_F32: norm_chunk<GM_F32>(t.e[ti].g, base, t.e[ti].numel, vec, acc); break;
      case GM_BF16: norm_chunk<GM_BF16>(t.e[ti].g, base, t.e[ti].numel, vec, acc); break;
      default: norm_chunk<GM_F16>(t.e[ti].g, base, t.e[ti].numel, vec, acc); break;
    }
  }
  const double s = block_sum(acc[0] + acc[1]);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The partial sums in a fixed order, so that equal gradients give equal bits.
__global__ void __launch_bounds__(kThreads) k_grad_norm_join(int n, const double* part, double max_norm,
                                                             float* norm, double* scale,
                                                             int32_t* status) {
  // (no __restrict__: part is written until the wait ends)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  double acc = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) acc += part[i];
  const double s = block_sum(acc);
  if (threadIdx.x) return;
  const double r = sqrt(s);
  const bool ok = s < pow2d(256) && (float)r <= 3.402823466e38f;
  *norm = ok ? (float)r : __int_as_float(0x7f800000);
  *scale = ok ? fmin(1.0, max_norm / (r + 1e-6)) : 0.0;
  *status = ok ? GM_OK : GM_E_NONFINITE;
}

template <typename M>
cudaError_t build_map(M& map, int count, const int64_t* numel_at, size_t stride, int chunk) {
  long long at = 0;
  map.count = count;
  for (int i = 0; i < count; ++i) {
    map.first[i] = (int)at;
    const int64_t n = *reinterpret_cast<const int64_t*>(reinterpret_cast<const uint8_t*>(numel_at) + i * stride);
    at += cdivll(n, chunk);
    if (at > 0x7fffffffLL) return cudaErrorInvalidValue;
  }
  map.first[count] = (int)at;
  return cudaSuccess;
}

bool aligned_to(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
int width(int dt) { return dt == GM_F32 ? 4 : 2; }

template <typename... KArgs, typename... Args>
cudaError_t launch_after(void (*kernel)(KArgs...), int grid, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int N>
using AdamWKernel = void (*)(Table<N>, Consts, const Coef*);
template <int BITS, int N>
AdamWKernel<N> pick(int pdt, int gdt) {
  static const AdamWKernel<N> k[3][3] = {
      {k_adamw<GM_F32, GM_F32, BITS, N>, k_adamw<GM_F32, GM_BF16, BITS, N>, k_adamw<GM_F32, GM_F16, BITS, N>},
      {k_adamw<GM_BF16, GM_F32, BITS, N>, k_adamw<GM_BF16, GM_BF16, BITS, N>, k_adamw<GM_BF16, GM_F16, BITS, N>},
      {k_adamw<GM_F16, GM_F32, BITS, N>, k_adamw<GM_F16, GM_BF16, BITS, N>, k_adamw<GM_F16, GM_F16, BITS, N>}};
  return k[pdt][gdt];
}

// One launch for the first n (<= N) tensors.
template <int N>
cudaError_t adamw_list(int n, const gm_adamw_tensor* tensors, int pdt, int gdt, const Consts& k, int bits,
                       const void* scratch, cudaStream_t s) {
  const int state = bits == 32 ? 32 : 8;   // bytes of eight elements
  Table<N> t;
  const cudaError_t e = build_map(t.map, n, &tensors[0].numel, sizeof(gm_adamw_tensor), kChunk);
  if (e != cudaSuccess) return e;
  for (int i = 0; i < n; ++i) {
    const gm_adamw_tensor& x = tensors[i];
    t.e[i] = {x.p, x.g, x.m, x.v, x.mscale, x.vscale, x.copy, x.numel};
    t.vec[i] = aligned_to(x.p, 8 * width(pdt)) && aligned_to(x.g, 8 * width(gdt)) &&
               aligned_to(x.m, state) && aligned_to(x.v, state) && aligned_to(x.copy, 8 * width(k.cdt));
  }
  const int total = t.map.first[n];
  // 32-bit states: a chunk per CTA, whose launch order walks the arrays front to
  // back (1e8 elements 412 us, 478 us with resident CTAs that stride); 8-bit states:
  // resident CTAs, which save a CTA's start per chunk (374 us, 405 us).
  const int resident = 3 * sm_count();
  const int grid = bits == 32 || total < resident ? total : resident;
  return launch_after(bits == 32 ? pick<32, N>(pdt, gdt) : pick<8, N>(pdt, gdt), grid, s, t, k,
                      static_cast<const Coef*>(scratch));
}

template <int N>
cudaError_t unpack_list(int n, const gm_adamw_state8* tensors, cudaStream_t s) {
  UnpackTable<N> t;
  const cudaError_t e = build_map(t.map, n, &tensors[0].numel, sizeof(gm_adamw_state8), kChunk);
  if (e != cudaSuccess) return e;
  for (int i = 0; i < n; ++i) {
    const gm_adamw_state8& x = tensors[i];
    t.e[i] = {x.m, x.v, x.mscale, x.vscale, x.m_out, x.v_out, x.numel};
    t.vec[i] = aligned_to(x.m, 8) && aligned_to(x.v, 8) && aligned_to(x.m_out, 32) && aligned_to(x.v_out, 32);
  }
  k_adamw_unpack8<N><<<t.map.first[n], kThreads, 0, s>>>(t);
  return cudaGetLastError();
}

// The first n (<= N) gradients; *blocks: the partial sums it writes.
template <int N>
cudaError_t norm_list(int n, const gm_grad* grads, double* part, int* blocks, cudaStream_t s) {
  GradTable<N> t;
  const cudaError_t e = build_map(t.map, n, &grads[0].numel, sizeof(gm_grad), kNormChunk);
  if (e != cudaSuccess) return e;
  for (int i = 0; i < n; ++i) {
    t.e[i] = {grads[i].g, grads[i].numel};
    t.kind[i] = (uint8_t)(grads[i].dtype | (aligned_to(grads[i].g, 16) ? 4 : 0));
  }
  *blocks = t.map.first[n] < kNormBlocks ? t.map.first[n] : kNormBlocks;
  k_grad_norm<N><<<*blocks, kThreads, 0, s>>>(t, part);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_adamw_begin(const gm_adamw_params& prm, int64_t* step, const int32_t* skip,
                               void* scratch, cudaStream_t s) {
  k_adamw_begin<<<1, 1, 0, s>>>(prm.lr, prm.beta1, prm.beta2, prm.eps, prm.wd, prm.clip, prm.lr_dev, skip, step,
                                static_cast<Coef*>(scratch));
  return cudaGetLastError();
}

cudaError_t launch_adamw(int count, const gm_adamw_tensor* tensors, int pdt, int gdt, int cdt,
                         const gm_adamw_params& prm, const void* scratch, cudaStream_t s) {
  const Consts k{(float)prm.beta1, (float)(1.0 - prm.beta1), (float)prm.beta2,
                 (float)(1.0 - prm.beta2), (float)prm.eps, (float)sqrt(prm.beta2),
                 (float)sqrt(1.0 - prm.beta2), prm.beta1, 1.0 - prm.beta1, prm.beta2,
                 1.0 - prm.beta2, cdt};
  for (int at = 0; at < count; at += kMaxTensors) {
    const int n = count - at < kMaxTensors ? count - at : kMaxTensors;
    const cudaError_t e =
        n <= kFewTensors ? adamw_list<kFewTensors>(n, tensors + at, pdt, gdt, k, prm.bits, scratch, s)
                         : adamw_list<kMaxTensors>(n, tensors + at, pdt, gdt, k, prm.bits, scratch, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_adamw_unpack8(int count, const gm_adamw_state8* tensors, cudaStream_t s) {
  for (int at = 0; at < count; at += kMaxUnpack) {
    const int n = count - at < kMaxUnpack ? count - at : kMaxUnpack;
    const cudaError_t e = n <= kFewTensors ? unpack_list<kFewTensors>(n, tensors + at, s)
                                           : unpack_list<kMaxUnpack>(n, tensors + at, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

int grad_norm_partials(int count) { return cdiv(count, kMaxGrads) * kNormBlocks; }

cudaError_t launch_grad_norm(int count, const gm_grad* grads, double max_norm, float* norm,
                             double* scale, int32_t* status, double* part, cudaStream_t s) {
  int used = 0;
  for (int at = 0; at < count; at += kMaxGrads) {
    const int n = count - at < kMaxGrads ? count - at : kMaxGrads;
    int blocks = 0;
    const cudaError_t e = n <= kFewGrads ? norm_list<kFewGrads>(n, grads + at, part + used, &blocks, s)
                                         : norm_list<kMaxGrads>(n, grads + at, part + used, &blocks, s);
    if (e != cudaSuccess) return e;
    used += blocks;
  }
  return launch_after(k_grad_norm_join, 1, s, used, (const double*)part, max_norm, norm, scale, status);
}

}  // namespace gm
