// Products grouped by expert, rows ragged: with rows i in [bounds[e],
// bounds[e + 1]) belonging to expert e,
//   forward  y_i  = W_e x_i          (optionally SiLU(gate) * up of it)
//   dx       dx_i = W_e^T dy_i
//   dw       dW_e = sum_i dy_i x_i^T
// fp16 or bf16 operands, float32 accumulators, one rounding at the end.
#include "experts.h"

namespace bitsmoe {
namespace experts {
namespace {

enum { kFwd = 0, kDx = 1, kDw = 2 };

struct MmArgs {
  const void* a;   // forward: x; dx, dw: dy
  int64_t lda;
  const void* b;   // forward, dx: w; dw: x
  int64_t ldb;     // dw: row stride of x
  const int32_t* rows;  // forward, dw: x row of sorted row i is rows[i] / div
  int div, x_rows;
  const int32_t* bounds;
  int R, E, N, K;  // W_e is (act ? 2 N : N) x K
  void* y;
  int64_t ldy;
  int act;
};

// The row of x behind sorted row i; -1: an index outside x, whose products
// are NaN.
__device__ inline int x_row(const MmArgs& s, int i) {
  if (!s.rows) return i;
  const int p = s.rows[i];
  const int r = p < 0 ? -1 : p / s.div;
  return r < s.x_rows ? r : -1;
}

// ------------------------------------------------------------ any layout
// 64 x 64 tiles, 4 waves of 32 x 32, 32 of the contraction per step.  Both
// operands are staged element by element with every index checked, so any
// size, stride and alignment is served; shapes with 16-byte rows take the
// kernels below.
constexpr int kAnyTile = 64, kAnyStep = 32, kAnyLd = kAnyStep + 8;

template <class T, class O, int MODE>
__global__ __launch_bounds__(256) void k_mm_any(MmArgs s) {
  __shared__ T la[kAnyTile][kAnyLd], lb[kAnyTile][kAnyLd];
  __shared__ int lrow[kAnyTile];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const T* A = (const T*)s.a;
  const T* B = (const T*)s.b;
  const T nan = (T)__builtin_nanf("");
  // m, n: output row and column, c: contraction
  int m0, mn, n0, nn, c0, cn, e;
  if (MODE == kDw) {
    e = blockIdx.z;
    int lo, hi;
    expert_rows(s.bounds, e, s.R, lo, hi);
    m0 = blockIdx.y * kAnyTile, mn = min(kAnyTile, s.N - m0);
    n0 = blockIdx.x * kAnyTile, nn = min(kAnyTile, s.K - n0);
    c0 = lo, cn = hi - lo;
  } else {
    const Tile t = find_tile(s.bounds, s.E, s.R, blockIdx.y, kAnyTile);
    if (t.n == 0) return;
    e = t.e;
    m0 = t.row0, mn = t.n;
    const int per = MODE == kFwd && s.act ? kAnyTile / 2 : kAnyTile;
    const int cols = MODE == kFwd ? s.N : s.K;
    n0 = blockIdx.x * per, nn = min(per, cols - n0);
    c0 = 0, cn = MODE == kFwd ? s.K : s.N;
    if (tid < kAnyTile) lrow[tid] = tid < mn ? (MODE == kFwd ? x_row(s, m0 + tid) : m0 + tid) : 0;
  }
  const T* W = MODE == kDw ? nullptr : B + (size_t)e * (s.act ? 2 : 1) * s.N * s.K;
  f32x4 acc[2][2] = {};
  __syncthreads();
  for (int c = 0; c < cn; c += kAnyStep) {
    if (MODE == kDw) {
      if (tid < kAnyStep) lrow[tid] = c + tid < cn ? x_row(s, c0 + c + tid) : 0;
      __syncthreads();
    }
    for (int i = tid; i < kAnyTile * kAnyStep; i += 256) {
      // the inner index runs along the operand's contiguous axis
      const int ci = MODE == kDw ? i / kAnyTile : i % kAnyStep;
      const int mi = MODE == kDw ? i % kAnyTile : i / kAnyStep;
      T v = (T)0.f;
      if (mi < mn && c + ci < cn) {
        if (MODE == kDw)
          v = A[(int64_t)(c0 + c + ci) * s.lda + m0 + mi];
        else
          v = lrow[mi] < 0 ? nan : A[(int64_t)lrow[mi] * s.lda + c + ci];
      }
      la[mi][ci] = v;
    }
    for (int i = tid; i < kAnyTile * kAnyStep; i += 256) {
      const int ci = MODE == kFwd ? i % kAnyStep : i / kAnyTile;
      const int ni = MODE == kFwd ? i / kAnyStep : i % kAnyTile;
      T v = (T)0.f;
      if (c + ci < cn) {
        if (MODE == kFwd) {
          // with the activation, blocks of 16 columns alternate gate and up
          const int col = s.act ? (ni >> 5) * 16 + (ni & 15) : ni;
          const int up = s.act ? (ni >> 4) & 1 : 0;
          if (col < nn) v = W[((int64_t)up * s.N + n0 + col) * s.K + c + ci];
        } else if (ni < nn) {
          if (MODE == kDx)
            v = W[(int64_t)(c + ci) * s.K + n0 + ni];
          else
            v = lrow[ci] < 0 ? nan : B[(int64_t)lrow[ci] * s.ldb + n0 + ni];
        }
      }
      lb[ni][ci] = v;
    }
    __syncthreads();
    const int r = lane & 15, q = (lane >> 4) * 8;
    typename Vec8<T>::type fa[2], fb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fa[i] = *reinterpret_cast<const typename Vec8<T>::type*>(&la[(wv >> 1) * 32 + i * 16 + r][q]);
      fb[i] = *reinterpret_cast<const typename Vec8<T>::type*>(&lb[(wv & 1) * 32 + i * 16 + r][q]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mfma16(fa[i], fb[j], acc[i][j]);
    __syncthreads();
  }
  // D: column lane % 16, rows 4 (lane / 16) + v
  O* Y = (O*)s.y;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int mi = (wv >> 1) * 32 + i * 16 + (lane >> 4) * 4 + v;
        int ni = (wv & 1) * 32 + j * 16 + (lane & 15);
        float o = acc[i][j][v];
        if (MODE == kFwd && s.act) {
          if (j) continue;
          ni = (wv & 1) * 16 + (lane & 15);
          o = gated(acc[i][0][v], acc[i][1][v]);
        }
        if (mi >= mn || ni >= nn) continue;
        if (MODE == kDw)
          Y[((int64_t)e * s.N + m0 + mi) * s.K + n0 + ni] = from_f32<O>(o);
        else
          Y[(int64_t)(m0 + mi) * s.ldy + n0 + ni] = from_f32<O>(o);
      }
}

template <class F>
void with_types(int dtype, int o_dtype, F f) {
  if (dtype == BITSMOE_F16) {
    if (o_dtype == BITSMOE_F32)
      f(f16{}, float{});
    else
      f(f16{}, f16{});
  } else {
    if (o_dtype == BITSMOE_F32)
      f(bf16{}, float{});
    else
      f(bf16{}, bf16{});
  }
}

int mm_check(int dtype, int o_dtype, int R, int E, int N, int K, const int32_t* bounds) {
  if (!is_half(dtype)) return fail(BITSMOE_EINVAL, "dtype=%d (float16 or bfloat16)", dtype);
  if (o_dtype != dtype && o_dtype != BITSMOE_F32)
    return fail(BITSMOE_EINVAL, "output dtype=%d (the operands' or float32)", o_dtype);
  if (R < 0 || R > (1 << 26) || E < 1 || E > 65535 || N < 1 || K < 1 || N > (1 << 20) ||
      K > (1 << 20))
    return fail(BITSMOE_ESHAPE, "R=%d E=%d N=%d K=%d", R, E, N, K);
  if (!bounds) return fail(BITSMOE_EINVAL, "bounds is null");
  return BITSMOE_OK;
}

int rows_check(const int32_t* rows, int div, int x_rows, int R) {
  if (rows ? (div < 1 || x_rows < 0) : x_rows < R)
    return fail(BITSMOE_ESHAPE, "div=%d, %d rows of x for R=%d", div, x_rows, R);
  return BITSMOE_OK;
}

int row_grid(int R, int E, int tile, unsigned* out) {
  const long long n = max_tiles(R, E, tile);
  if (n > 65535 * 16ll) return fail(BITSMOE_ESHAPE, "R=%d E=%d make too many row tiles", R, E);
  *out = (unsigned)n;
  return BITSMOE_OK;
}

template <int MODE>
int launch_any(const MmArgs& s, int dtype, int o_dtype, hipStream_t st) {
  dim3 grid;
  if (MODE == kDw) {
    grid = dim3((unsigned)((s.K + kAnyTile - 1) / kAnyTile),
                (unsigned)((s.N + kAnyTile - 1) / kAnyTile), (unsigned)s.E);
  } else {
    const int per = MODE == kFwd && s.act ? kAnyTile / 2 : kAnyTile;
    const int cols = MODE == kFwd ? s.N : s.K;
    const long long tiles = max_tiles(s.R, s.E, kAnyTile);
    if (tiles > 65535) return fail(BITSMOE_ESHAPE, "R=%d E=%d make too many row tiles", s.R, s.E);
    grid = dim3((unsigned)((cols + per - 1) / per), (unsigned)tiles);
  }
  with_types(dtype, o_dtype, [&](auto t, auto o) {
    hipLaunchKernelGGL((k_mm_any<decltype(t), decltype(o), MODE>), grid, dim3(256), 0, st, s);
  });
  return launched("grouped_matmul");
}

}  // namespace
}  // namespace experts
}  // namespace bitsmoe

using namespace bitsmoe;
using namespace bitsmoe::experts;

extern "C" {

int bitsmoe_grouped_matmul(int dtype, const void* x, int64_t ldx, int x_rows, const int32_t* rows,
                           int div, const void* w, const int32_t* bounds, int R, int E, int N,
                           int K, int act, void* y, int y_dtype, int64_t ldy,
                           bitsmoe_stream_t stream) {
  int st = mm_check(dtype, y_dtype, R, E, N, K, bounds);
  if (st || (st = rows_check(rows, div, x_rows, R))) return st;
  if (act != BITSMOE_ACT_NONE && act != BITSMOE_ACT_SILU_MUL)
    return fail(BITSMOE_EINVAL, "act=%d", act);
  if (ldx < K || ldy < N) return fail(BITSMOE_ESHAPE, "a row stride is too small");
  if (R == 0) return BITSMOE_OK;
  if (!w || !y || (x_rows && !x)) return fail(BITSMOE_EINVAL, "null pointer argument");
  MmArgs s{x, ldx, w, 0, rows, div, x_rows, bounds, R, E, N, K, y, ldy, act};
  return launch_any<kFwd>(s, dtype, y_dtype, (hipStream_t)stream);
}

int bitsmoe_grouped_matmul_dx(int dtype, const void* dy, int64_t lddy, const void* w,
                              const int32_t* bounds, int R, int E, int N, int K, void* dx,
                              int dx_dtype, int64_t lddx, bitsmoe_stream_t stream) {
  const int st = mm_check(dtype, dx_dtype, R, E, N, K, bounds);
  if (st) return st;
  if (lddy < N || lddx < K) return fail(BITSMOE_ESHAPE, "a row stride is too small");
  if (R == 0) return BITSMOE_OK;
  if (!dy || !w || !dx) return fail(BITSMOE_EINVAL, "null pointer argument");
  MmArgs s{dy, lddy, w, 0, nullptr, 1, R, bounds, R, E, N, K, dx, lddx, 0};
  return launch_any<kDx>(s, dtype, dx_dtype, (hipStream_t)stream);
}

int bitsmoe_grouped_matmul_dw(int dtype, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                              int x_rows, const int32_t* rows, int div, const int32_t* bounds,
                              int R, int E, int N, int K, void* dw, int dw_dtype,
                              bitsmoe_stream_t stream) {
  int st = mm_check(dtype, dw_dtype, R, E, N, K, bounds);
  if (st || (st = rows_check(rows, div, x_rows, R))) return st;
  if (lddy < N || ldx < K) return fail(BITSMOE_ESHAPE, "a row stride is too small");
  if (!dw || (R && (!dy || (x_rows && !x)))) return fail(BITSMOE_EINVAL, "null pointer argument");
  MmArgs s{dy, lddy, x, ldx, rows, div, x_rows, bounds, R, E, N, K, dw, 0, 0};
  return launch_any<kDw>(s, dtype, dw_dtype, (hipStream_t)stream);
}

}  // extern "C"
