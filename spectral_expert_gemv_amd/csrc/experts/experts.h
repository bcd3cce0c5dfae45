// Shared pieces of the expert-layer kernels (routing, products by expert,
// activation, combine, 4-bit products): element types, 8-wide loads, the
// lookup of a row tile in the experts' bounds, host-side checks.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "bitsmoe.h"
#include "common.h"

namespace bitsmoe {
namespace experts {

typedef _Float16 f16;
typedef __bf16 bf16;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(16))) float f32x16;

template <class T>
struct Vec8;
template <>
struct Vec8<f16> {
  typedef __attribute__((ext_vector_type(8))) _Float16 type;
};
template <>
struct Vec8<bf16> {
  typedef __attribute__((ext_vector_type(8))) __bf16 type;
};

__device__ inline f32x4 mfma16(Vec8<f16>::type a, Vec8<f16>::type b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ inline f32x4 mfma16(Vec8<bf16>::type a, Vec8<bf16>::type b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

template <class T>
__device__ inline float to_f32(T v) {
  return (float)v;
}
template <class T>
__device__ inline T from_f32(float v) {
  // round to nearest even, of the float32 value: the empty statement keeps
  // the product before it from being folded into the conversion, which
  // would round once where the 8-wide stores round twice
  asm("" : "+v"(v));
  return (T)v;
}

// 8 consecutive elements as float: one 16-byte load (two for float32).
__device__ inline void load8(const f16* p, float (&v)[8]) {
  const Vec8<f16>::type t = *reinterpret_cast<const Vec8<f16>::type*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (float)t[i];
}
__device__ inline void load8(const bf16* p, float (&v)[8]) {
  const uint4 t = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ inline void load8(const float* p, float (&v)[8]) {
  const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
}
template <class T>
__device__ inline void store8(T* p, const float (&v)[8]) {
  typename Vec8<T>::type t;
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = (T)v[i];
  *reinterpret_cast<typename Vec8<T>::type*>(p) = t;
}
__device__ inline void store8(float* p, const float (&v)[8]) {
  f32x4 a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = v[i], b[i] = v[4 + i];
  reinterpret_cast<f32x4*>(p)[0] = a;
  reinterpret_cast<f32x4*>(p)[1] = b;
}

// 1 / (1 + exp(-g)).  exp2 of the product with log2(e), whose rounding error
// and low part are put back by one multiplication, and the hardware's
// reciprocal: each within a step of float32, a third of the instructions of
// an exact exp and division (products with the activation, 24576 rows of 64
// experts: 361 -> 351 us).
// Below g = -87.3, where it would be subnormal, it is 0: a SiLU of up to
// 1.1e-36 there is lost.
// (The low part is under 1e-5 wherever the exp is neither 0 nor inf.  Where the
// product overflows it is infinite or NaN: the median of it, -1 and 1 is a
// factor that leaves them 0 and inf.)
__device__ inline float sigmoid(float g) {
#pragma clang fp contract(off)
  constexpr float kHi = -1.44269502162933349609375f, kLo = -1.92596299112661746887e-8f;
  const float t = g * kHi;
  const float lo = __builtin_amdgcn_fmed3f(fmaf(g, kLo, fmaf(g, kHi, -t)), -1.0f, 1.0f);
  const float e = __builtin_amdgcn_exp2f(t) * fmaf(lo, 0.693147182464599609375f, 1.0f);
  return __builtin_amdgcn_rcpf(1.0f + e);
}

// SiLU(g) * u, and its derivative with respect to g and u times dh.  No
// contraction, so that the bits do not depend on which kernel (by alignment)
// evaluates them.
__device__ inline float gated(float g, float u) {
#pragma clang fp contract(off)
  return g * sigmoid(g) * u;
}
__device__ inline void gated_grad(float g, float u, float dh, float& dg, float& du) {
#pragma clang fp contract(off)
  const float s = sigmoid(g);
  // 1 + g (1 - s) as written loses nothing: both terms are of order 1 where it matters
  dg = dh * u * (s * (1.0f + g * (1.0f - s)));
  du = dh * (g * s);
}

// One row tile of the ragged layout: rows [row0, row0 + n) of expert e.
struct Tile {
  int e, row0, n;
};

// Rows [lo, hi) of expert e, clamped into [0, R]: whatever `bounds` holds, no
// row outside the buffers is touched.
__device__ inline void expert_rows(const int32_t* __restrict__ bounds, int e, int R, int& lo,
                                   int& hi) {
  lo = min(max(bounds[e], 0), R);
  hi = max(min(max(bounds[e + 1], 0), R), lo);
}

// The `tile`-th tile of up to BM rows, experts ascending, none for experts
// without rows; n = 0 past the last tile.  Whole waves call it: the lanes
// count the tiles of 64 experts at a time.
__device__ inline Tile find_tile(const int32_t* __restrict__ bounds, int E, int R, int tile,
                                 int BM) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    int lo = 0, hi = 0;
    if (e0 + lane < E) expert_rows(bounds, e0 + lane, R, lo, hi);
    const int n = (hi - lo + BM - 1) / BM;
    int inc = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int t = __shfl_up(inc, d, 64);
      if (lane >= d) inc += t;
    }
    const uint64_t past = __ballot(base + inc > tile);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      const int first = base + __shfl(inc - n, l, 64);
      const int a = __shfl(lo, l, 64) + (tile - first) * BM, b = __shfl(hi, l, 64);
      return Tile{__builtin_amdgcn_readfirstlane(e0 + l), __builtin_amdgcn_readfirstlane(a),
                  __builtin_amdgcn_readfirstlane(min(BM, b - a))};
    }
    base += __shfl(inc, 63, 64);
  }
  return Tile{0, 0, 0};
}

// Tiles of up to BM rows of all experts (whole waves call it).
__device__ inline int count_tiles(const int32_t* __restrict__ bounds, int E, int R, int BM) {
  int n = 0;
  for (int e = threadIdx.x & 63; e < E; e += 64) {
    int lo, hi;
    expert_rows(bounds, e, R, lo, hi);
    n += (hi - lo + BM - 1) / BM;
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) n += __shfl_xor(n, d, 64);
  return __builtin_amdgcn_readfirstlane(n);
}

// The most tiles of BM rows that R rows of E experts can make.
inline long long max_tiles(long long R, long long E, long long BM) {
  return R / BM + (R < E ? R : E);
}

// Whether counts of tiles stay within 32 bits whatever the bounds hold (each
// expert's rows are clamped to R, but wrong bounds may give every expert R).
inline bool countable(long long R, long long E, long long BM) {
  return E * ((R + BM - 1) / BM) < 0x40000000ll;
}

inline bool is_half(int dtype) { return dtype == BITSMOE_F16 || dtype == BITSMOE_BF16; }

inline int launched(const char* what) {
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return fail(BITSMOE_EHIP, "%s launch: %s", what, hipGetErrorString(err));
  return BITSMOE_OK;
}

}  // namespace experts
}  // namespace bitsmoe
