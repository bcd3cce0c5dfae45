// Products with 4-bit weights: W[n, c] = m[n, c / G] + s[n, c / G] q[n, c]
// with codes q of 0..15 (two per byte, the lower half first), float16 steps s
// and minima m per group of G inputs; dense or grouped by expert, optionally
// SiLU(gate) * up of the two halves of the rows.  Per group
//   sum_c W x = s (sum_c q x) + m (sum_c x),
// so the codes enter the products as small whole numbers, exactly.
#include "experts.h"

namespace bitsmoe {
namespace experts {
namespace {

struct W4Args {
  const void* x;
  int64_t ldx;
  const int32_t* rows;
  int div, x_rows;
  const uint8_t* codes;   // E x rows x K/2
  const f16* scales;      // E x rows x K/G
  const f16* mins;        // E x rows x K/G, or null: -8 s
  const int32_t* bounds;  // null: one expert with all R rows
  int R, E, N, K, G;
  void* y;
  int64_t ldy;
  int act;
};

__device__ inline int w4_row(const W4Args& s, int i) {
  if (!s.rows) return i;
  const int p = s.rows[i];
  const int r = p < 0 ? -1 : p / s.div;
  return r < s.x_rows ? r : -1;
}

// A wave per (row, output): lanes along the inputs, 8 codes at a time.
template <class T, class O>
__global__ __launch_bounds__(256) void k_w4_any(W4Args s) {
  const int lane = threadIdx.x & 63;
  const int n = blockIdx.x * 4 + (threadIdx.x >> 6);
  int e = 0, i = blockIdx.y;
  if (s.bounds) {
    const Tile t = find_tile(s.bounds, s.E, s.R, blockIdx.y, 1);
    if (t.n == 0) return;
    e = t.e, i = t.row0;
  }
  if (n >= s.N) return;
  const int xr = w4_row(s, i);
  const int groups = s.K / s.G;
  float y[2] = {0.f, 0.f};
  for (int h = 0; h < (s.act ? 2 : 1); ++h) {
    const size_t row = (size_t)e * (s.act ? 2 : 1) * s.N + (size_t)h * s.N + n;
    const T* x = (const T*)s.x + (int64_t)max(xr, 0) * s.ldx;
    float acc = 0.f;
    for (int c = lane * 8; c < s.K; c += 64 * 8) {
      const uint8_t* q = s.codes + row * (s.K / 2) + c / 2;
      const float st = (float)s.scales[row * groups + c / s.G];
      const float mn = s.mins ? (float)s.mins[row * groups + c / s.G] : -8.f * st;
      for (int j = 0; j < 8; ++j) {
        const int code = (q[j >> 1] >> (4 * (j & 1))) & 15;
        acc = fmaf(fmaf(st, (float)code, mn), to_f32(x[c + j]), acc);
      }
    }
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) acc += __shfl_xor(acc, m, 64);
    y[h] = acc;
  }
  if (lane == 0) {
    float o = s.act ? gated(y[0], y[1]) : y[0];
    if (xr < 0) o = __builtin_nanf("");
    ((O*)s.y)[(int64_t)i * s.ldy + n] = from_f32<O>(o);
  }
}

}  // namespace
}  // namespace experts
}  // namespace bitsmoe

using namespace bitsmoe;
using namespace bitsmoe::experts;

extern "C" {

int bitsmoe_w4_matmul(int dtype, const void* x, int64_t ldx, int x_rows, const int32_t* rows,
                      int div, const void* codes, const void* scales, const void* mins, int G,
                      const int32_t* bounds, int R, int E, int N, int K, int act, void* y,
                      int y_dtype, int64_t ldy, bitsmoe_stream_t stream) {
  if (!is_half(dtype)) return fail(BITSMOE_EINVAL, "dtype=%d (float16 or bfloat16)", dtype);
  if (y_dtype != dtype && y_dtype != BITSMOE_F32)
    return fail(BITSMOE_EINVAL, "output dtype=%d (that of x or float32)", y_dtype);
  if (R < 0 || R > (1 << 24) || E < 1 || E > 65535 || N < 1 || K < 1 || N > (1 << 20) ||
      K > (1 << 20))
    return fail(BITSMOE_ESHAPE, "R=%d E=%d N=%d K=%d", R, E, N, K);
  if (G != 32 && G != 64 && G != 128) return fail(BITSMOE_ESHAPE, "G=%d (32, 64 or 128)", G);
  if (K % G) return fail(BITSMOE_ESHAPE, "K=%d is not a multiple of G=%d", K, G);
  if (!bounds && E != 1) return fail(BITSMOE_EINVAL, "E=%d without bounds", E);
  if (act != BITSMOE_ACT_NONE && act != BITSMOE_ACT_SILU_MUL)
    return fail(BITSMOE_EINVAL, "act=%d", act);
  if (rows ? (div < 1 || x_rows < 0) : x_rows < R)
    return fail(BITSMOE_ESHAPE, "div=%d, %d rows of x for R=%d", div, x_rows, R);
  if (ldx < K || ldy < N) return fail(BITSMOE_ESHAPE, "a row stride is too small");
  if (R == 0) return BITSMOE_OK;
  if (!codes || !scales || !y || (x_rows && !x)) return fail(BITSMOE_EINVAL, "null pointer argument");
  if (((uintptr_t)codes & 15u) || ((uintptr_t)scales & 3u) || ((uintptr_t)mins & 3u))
    return fail(BITSMOE_EINVAL, "codes must be 16-byte aligned, scales and mins 4-byte aligned");
  W4Args s{x, ldx, rows, div, x_rows, (const uint8_t*)codes, (const f16*)scales, (const f16*)mins,
           bounds, R, E, N, K, G, y, ldy, act};
  const dim3 grid((unsigned)((N + 3) / 4), (unsigned)R);
  if (R > 65535) return fail(BITSMOE_ESHAPE, "R=%d", R);
  auto go = [&](auto t, auto o) {
    hipLaunchKernelGGL((k_w4_any<decltype(t), decltype(o)>), grid, dim3(256), 0,
                       (hipStream_t)stream, s);
  };
  if (dtype == BITSMOE_F16) {
    if (y_dtype == BITSMOE_F32)
      go(f16{}, float{});
    else
      go(f16{}, f16{});
  } else {
    if (y_dtype == BITSMOE_F32)
      go(bf16{}, float{});
    else
      go(bf16{}, bf16{});
  }
  return launched("w4_matmul");
}

}  // extern "C"
