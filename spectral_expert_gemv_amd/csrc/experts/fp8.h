// 8-bit floating point values (OCP e4m3) with a float32 scale per group of
// 128: what the quantizers and the products that quantize on their way share.
//
// With a the largest finite magnitude of a group, in IEEE float32 steps:
//   s = a / 448, r = 448 / a      (both 1 where a < 2^-80: codes of 0)
//   code = e4m3(v r), to nearest even; NaN where v is not finite
// 448 is e4m3's largest value.  v r is at most 448 (1 + 2^-23), which rounds to
// it.  Multiplying by r instead of dividing by s moves v r by at most 2^-23 of
// itself: under 2^-18 of the half step that the code's rounding may add.
#pragma once
#include "experts.h"

namespace bitsmoe {
namespace experts {

constexpr int kGroup = 128;       // elements with one scale
constexpr int kE4M3 = BITSMOE_E4M3;

inline int64_t groups_of(int64_t n) { return (n + kGroup - 1) / kGroup; }

struct Factors {
  float s, r;
};
// a_bits: of a finite magnitude a.  a / 448 from the rounded reciprocal and one
// correction by the remainder, which is exact: the rounded quotient for every
// mantissa.
__device__ __forceinline__ Factors factors8(uint32_t a_bits) {
  const float a = __uint_as_float(a_bits);
  Factors f{1.0f, 1.0f};
  if (a >= 0x1p-80f) {
    constexpr float kInv = 1.0f / 448.0f;
    const float q = a * kInv;
    f.s = fmaf(fmaf(-448.0f, q, a), kInv, q);
    f.r = 448.0f / a;
  }
  return f;
}

constexpr uint32_t kInfBits = 0x7F800000u;
// The largest magnitude's bits (ordered as the magnitudes, infinities and NaN
// above all finite ones), or `finite`: of the finite ones.
template <bool finite, int N>
__device__ __forceinline__ uint32_t amax_bits(const float (&v)[N]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t u = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    if (finite) u = u < kInfBits ? u : 0u;
    m = m > u ? m : u;
  }
  return m;
}

// 4 codes of v r
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float r) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * r, b * r, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c * r, d * r, w, true);
}

// maximum over the 16 lanes of a DPP row, in every lane
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, false);
  return v > o ? v : o;
}
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = dpp_max<0xB1>(v);   // quad_perm [1,0,3,2]
  v = dpp_max<0x4E>(v);   // quad_perm [2,3,0,1]
  v = dpp_max<0x141>(v);  // row_half_mirror
  return dpp_max<0x140>(v);  // row_mirror
}

// 8 elements of a row from any element's alignment (the hardware takes it), 0
// from the `left`-th on
template <class T>
__device__ __forceinline__ void load8_any(const T* p, int left, float (&v)[8]) {
  if (left >= 8) {
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    typedef u4 loose __attribute__((aligned(2)));
    if constexpr (sizeof(T) == 4) {
      const u4 a = reinterpret_cast<const loose*>(p)[0], b = reinterpret_cast<const loose*>(p)[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(a[i]), v[4 + i] = __uint_as_float(b[i]);
    } else {
      const u4 a = *reinterpret_cast<const loose*>(p);
      const typename Vec8<T>::type t = __builtin_bit_cast(typename Vec8<T>::type, a);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (float)t[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? to_f32(p[i]) : 0.0f;
  }
}

// Rows gathered on their way: row r is row rows[r] / div of x, which has x_rows
// rows; an index outside them gives NaN scales.
struct Gather {
  const int32_t* rows;
  int div, x_rows;
};

// Quantizes rows on `st` (what bitsmoe_fp8_rows launches); sizes are checked.
int run_fp8_rows(int dtype, const void* x, int64_t ldx, Gather from, int act,
                 const int32_t* bounds, int R, int E, int K, void* codes, int64_t ldc,
                 float* scales, int64_t lds, hipStream_t st);

}  // namespace experts
}  // namespace bitsmoe
