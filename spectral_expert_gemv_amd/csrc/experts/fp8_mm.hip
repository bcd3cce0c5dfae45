// Products grouped by expert of 8-bit floating point operands: rows with a
// scale per 128 inputs, weights with a scale per block of 128 x 128,
//   y[i, n] = sum_g sx[i, g] sw[e, n / 128, g] sum_{c in group g} qx[i, c] qw[e, n, c]
// (optionally SiLU(gate) * up of it).  The inner sums are the matrix cores', the
// outer one float32; each output is rounded once.  Rows may also come as fp16
// or bf16: they are then quantized on the way, to the same codes as by
// bitsmoe_fp8_rows.
#include <type_traits>

#include "fp8.h"

namespace bitsmoe {
namespace experts {
namespace {

typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((ext_vector_type(4))) int i32x4;

// 32 codes of a lane as fp16, which holds every e4m3 number
struct Halves {
  Vec8<f16>::type v[4];
};
__device__ __forceinline__ Halves halves(i32x8 q) {
  Halves h;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f16x2 a = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(q[2 * j + i], 1.0f, false));
      const f16x2 b = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(q[2 * j + i], 1.0f, true));
      h.v[j][4 * i] = a[0], h.v[j][4 * i + 1] = a[1], h.v[j][4 * i + 2] = b[0], h.v[j][4 * i + 3] = b[1];
    }
  }
  return h;
}
// a group's sums, in float32: four fp16 instructions.  (The 8-bit instruction
// aligns eight products at a time to their largest and drops what lies more
// than 13 bits below its first one: 1.4e-5 to 5e-5 of the result where this is
// 1e-7.)
__device__ __forceinline__ f32x4 group_sums(const Halves& a, const Halves& b) {
  f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 4; ++j) p = mfma16(a.v[j], b.v[j], p);
  return p;
}

struct E4M3 {};  // rows that are codes already

struct Mm8Args {
  const void* x;
  int64_t ldx;
  const float* xs;      // scales of codes
  int64_t ldxs;
  const int32_t* rows;  // sorted row i reads row rows[i] / div of x
  int div, x_rows;
  const uint8_t* w;     // E x (act ? 2 N : N) x kg * 128
  const float* ws;      // E x (act ? 2 nb : nb) x kg
  const int32_t* bounds;
  int R, E, N, K, kg, nb;
  void* y;
  int64_t ldy;
  int y16;              // rows of y are whole 16-byte pieces
};

__device__ __forceinline__ int x_row8(const Mm8Args& s, int i) {
  if (!s.rows) return i;
  const int p = s.rows[i];
  const int r = p < 0 ? -1 : p / s.div;
  return r < s.x_rows ? r : -1;
}

// ------------------------------------------------- few rows per expert
// A work-group takes up to 64 sorted rows of one expert and 32 rows of its
// weights (with the activation 16 of the gate and the same 16 of the up half);
// its four waves split the inputs in turns of 128, one group and a whole line
// of each weight row, and add up their sums through LDS.  Weights go straight
// into registers, once; they are the products' first operand, so a lane holds 4
// outputs of one row of x, whose scale it needs once.  Which of a group's 128
// elements lie in which lane does not matter as long as both operands agree:
// lane (r, q) holds bytes 16 q .. and 64 + 16 q .. of row r, so that a load
// covers 64 bytes of 16 rows.
constexpr int kFewRows = 64, kFewCols = 32, kFewWaves = 4;

// 16 + 16 bytes of a row of codes at group start p (+ 16 q)
__device__ __forceinline__ i32x8 load_codes(const uint8_t* p) {
  const i32x4 a = *reinterpret_cast<const i32x4*>(p), b = *reinterpret_cast<const i32x4*>(p + 64);
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// One row operand of a group: codes as they are, or 16 + 16 elements on their
// way to codes.
template <class X>
struct RowPiece {
  float v[4][8];
  __device__ __forceinline__ void load(const X* p, int left) {  // left: elements of the row from p on
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int at = (h >> 1) * 64 + (h & 1) * 8;
      load8_any(p + at, left - at, v[h]);
    }
  }
  __device__ __forceinline__ i32x8 codes(float& s) const {
    auto over_lanes = [](uint32_t m) {  // the four lanes of the row
#pragma unroll
      for (int d = 16; d < 64; d <<= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)m, d, 64);
        m = m > o ? m : o;
      }
      return m;
    };
    uint32_t a = 0;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const uint32_t m = amax_bits<false>(v[h]);
      a = a > m ? a : m;
    }
    a = over_lanes(a);
    if (__any(a >= kInfBits)) {
      a = 0;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const uint32_t m = amax_bits<true>(v[h]);
        a = a > m ? a : m;
      }
      a = over_lanes(a);
    }
    const Factors f = factors8(a);
    s = f.s;
    i32x8 q;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      q[2 * h] = (int)codes4(v[h][0], v[h][1], v[h][2], v[h][3], f.r);
      q[2 * h + 1] = (int)codes4(v[h][4], v[h][5], v[h][6], v[h][7], f.r);
    }
    return q;
  }
};

template <class X, class O, bool ACT, int MB>
__device__ __forceinline__ void few8_rows(const Mm8Args& s, const Tile& t, float* lds) {
  constexpr bool kCodes = std::is_same<X, E4M3>::value;
  constexpr int U = MB == 1 ? 4 : MB == 2 ? 2 : 1;  // turns whose loads are in flight together
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * (ACT ? kFewCols / 2 : kFewCols);
  const int64_t kp = (int64_t)s.kg * kGroup;
  const uint8_t* w[2];
  const float* ws[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int n = n0 + (ACT ? 0 : 16 * b);
    const int64_t row = (int64_t)(ACT ? b : 0) * s.N + min(n + r, s.N - 1);
    w[b] = s.w + ((int64_t)t.e * (ACT ? 2 : 1) * s.N + row) * kp + 16 * q;
    // (32 and 16 divide 128: a work-group's rows share a block)
    ws[b] = s.ws + ((int64_t)t.e * (ACT ? 2 : 1) * s.nb + (ACT ? b : 0) * s.nb + n0 / kGroup) * s.kg;
  }
  int64_t x[MB];
  bool bad[MB];
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const int xr = x_row8(s, t.row0 + min(16 * m + r, t.n - 1));
    bad[m] = xr < 0;
    x[m] = max(xr, 0);
  }
  f32x4 acc[MB][2] = {};
  auto turn = [&](int g0, auto whole_) {  // group g0 and every kFewWaves on, U times
    constexpr bool whole = decltype(whole_)::value;
    i32x8 vw[U][2];
    float sw[U][2];
    // (rows of two bytes an element stay as loaded until their turn)
    typename std::conditional<kCodes, i32x8, RowPiece<typename std::conditional<kCodes, f16, X>::type>>::type vx[U][MB];
    float sx[U][MB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = whole ? g0 + u * kFewWaves : min(g0 + u * kFewWaves, s.kg - 1);
#pragma unroll
      for (int b = 0; b < 2; ++b) vw[u][b] = load_codes(w[b] + (int64_t)g * kGroup), sw[u][b] = ws[b][g];
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        if constexpr (kCodes) {
          vx[u][m] = load_codes((const uint8_t*)s.x + x[m] * s.ldx + 16 * q + g * kGroup);
          sx[u][m] = s.xs[x[m] * s.ldxs + g];
        } else {
          vx[u][m].load((const X*)s.x + x[m] * s.ldx + 16 * q + g * kGroup,
                        s.K - (16 * q + g * kGroup));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!whole && g0 + u * kFewWaves >= s.kg) break;
      const Halves hw[2] = {halves(vw[u][0]), halves(vw[u][1])};
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        Halves hx;
        if constexpr (kCodes)
          hx = halves(vx[u][m]);
        else
          hx = halves(vx[u][m].codes(sx[u][m]));
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const f32x4 p = group_sums(hw[b], hx);
          const float f = sx[u][m] * sw[u][b];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[m][b][j] = fmaf(p[j], f, acc[m][b][j]);
        }
      }
    }
  };
  constexpr int kTurn = U * kFewWaves;
  int g = wv;
  for (; g + kTurn - kFewWaves < s.kg; g += kTurn) turn(g, std::true_type{});
  if (g < s.kg) turn(g, std::false_type{});

  // sums of the four waves: [wave][tile of 16 x 16][lane]
  f32x4* part = (f32x4*)lds;
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int b = 0; b < 2; ++b) part[(wv * MB * 2 + m * 2 + b) * 64 + lane] = acc[m][b];
  __syncthreads();
  O* Y = (O*)s.y;
  for (int i = wv; i < (ACT ? MB : MB * 2); i += kFewWaves) {
    const int m = ACT ? i : i >> 1;
    f32x4 v[2];
#pragma unroll
    for (int b = 0; b < (ACT ? 2 : 1); ++b) {
      const int at = ACT ? m * 2 + b : i;
      v[b] = part[at * 64 + lane];
#pragma unroll
      for (int o = 1; o < kFewWaves; ++o) {
        const f32x4 p = part[(o * MB * 2 + at) * 64 + lane];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[b][j] += p[j];
      }
    }
    const int n = n0 + (ACT ? 0 : 16 * (i & 1)) + 4 * q;
    bool nan = false;
#pragma unroll
    for (int u = 0; u < MB; ++u) nan = u == m ? bad[u] : nan;
    if (16 * m + r >= t.n) continue;
    typedef __attribute__((ext_vector_type(4))) O O4;
    O4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float f = ACT ? gated(v[0][j], v[1][j]) : v[0][j];
      o[j] = (O)(nan ? __builtin_nanf("") : f);
    }
    O* y = Y + (int64_t)(t.row0 + 16 * m + r) * s.ldy + n;
    if (s.y16 && n + 4 <= s.N) {
      *reinterpret_cast<O4*>(y) = o;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < s.N) y[j] = o[j];
    }
  }
}

template <class X, class O, bool ACT>
__global__ __launch_bounds__(64 * kFewWaves) void k_mm8_few(Mm8Args s) {
  __shared__ float lds[kFewWaves * 8 * 64 * 4];
  Tile t{0, 0, 0};
  if (s.bounds) {
    t = find_tile(s.bounds, s.E, s.R, blockIdx.y, kFewRows);
  } else {
    t.row0 = (int)blockIdx.y * kFewRows;
    t.n = min(kFewRows, s.R - t.row0);
  }
  if (t.n <= 0) return;
  if (t.n <= 16)
    few8_rows<X, O, ACT, 1>(s, t, lds);
  else if (t.n <= 32)
    few8_rows<X, O, ACT, 2>(s, t, lds);
  else
    few8_rows<X, O, ACT, 4>(s, t, lds);
}

template <class F>
void with_out(int o_dtype, F f) {
  if (o_dtype == BITSMOE_F32)
    f(float{});
  else if (o_dtype == BITSMOE_F16)
    f(f16{});
  else
    f(bf16{});
}

size_t rows_ws(int x_dtype, int64_t x_rows, int K) {
  (void)x_dtype, (void)x_rows, (void)K;
  return 0;
}

bool rows16(const void* p, int64_t ld, int size) {
  return (((uintptr_t)p | (uintptr_t)(ld * size)) & 15u) == 0;
}

int sizes8(int x_dtype, int x_rows, int R, int E, int N, int K, int act) {
  if (x_dtype != kE4M3 && !is_half(x_dtype))
    return fail(BITSMOE_EINVAL, "x dtype=%d (float16, bfloat16 or e4m3)", x_dtype);
  if (act != BITSMOE_ACT_NONE && act != BITSMOE_ACT_SILU_MUL)
    return fail(BITSMOE_EINVAL, "act=%d", act);
  if (R < 0 || R > (1 << 26) || x_rows < 0 || E < 1 || E > 65535 || N < 1 || K < 1 ||
      N > (1 << 20) || K > (1 << 20))
    return fail(BITSMOE_ESHAPE, "R=%d x_rows=%d E=%d N=%d K=%d", R, x_rows, E, N, K);
  if (!countable(R, E, kFewRows)) return fail(BITSMOE_ESHAPE, "R=%d with E=%d", R, E);
  return BITSMOE_OK;
}

}  // namespace
}  // namespace experts
}  // namespace bitsmoe

using namespace bitsmoe;
using namespace bitsmoe::experts;

extern "C" {

int bitsmoe_fp8_matmul_workspace_size(int x_dtype, int x_rows, int R, int E, int N, int K, int act,
                                      size_t* bytes) {
  if (!bytes) return fail(BITSMOE_EINVAL, "bytes is null");
  const int st = sizes8(x_dtype, x_rows, R, E, N, K, act);
  if (st) return st;
  *bytes = rows_ws(x_dtype, x_rows, K);
  return BITSMOE_OK;
}

int bitsmoe_fp8_matmul(int x_dtype, const void* x, int64_t ldx, const float* x_scales, int64_t ldxs,
                       int x_rows, const int32_t* rows, int div, const void* codes,
                       const float* scales, const int32_t* bounds, int R, int E, int N, int K,
                       int act, void* y, int y_dtype, int64_t ldy, void* ws, size_t ws_bytes,
                       bitsmoe_stream_t stream) {
  const int st = sizes8(x_dtype, x_rows, R, E, N, K, act);
  if (st) return st;
  const bool given = x_dtype == kE4M3;
  if (y_dtype != BITSMOE_F32 && !(given ? is_half(y_dtype) : y_dtype == x_dtype))
    return fail(BITSMOE_EINVAL, "y dtype=%d with x dtype=%d", y_dtype, x_dtype);
  if (!bounds && E != 1) return fail(BITSMOE_EINVAL, "bounds is null with E=%d", E);
  // (with rows: a row of x that a wrong index may be clamped to)
  if (rows ? (div < 1 || x_rows < (R > 0)) : x_rows < R)
    return fail(BITSMOE_ESHAPE, "div=%d, %d rows of x for R=%d", div, x_rows, R);
  const int64_t kg = groups_of(K), nb = groups_of(N);
  if (ldx < (given ? kg * kGroup : K) || (given && ldxs < kg) || ldy < N)
    return fail(BITSMOE_ESHAPE, "a row stride is too small");
  if (R == 0) return BITSMOE_OK;
  if (!x || !codes || !scales || !y || (given && !x_scales))
    return fail(BITSMOE_EINVAL, "null pointer argument");
  if (((uintptr_t)codes & 15u) || (given && !rows16(x, ldx, 1)))
    return fail(BITSMOE_EINVAL, "codes must be 16-byte aligned");
  const size_t need = rows_ws(x_dtype, x_rows, K);
  if (need > ws_bytes || (need && !ws))
    return fail(BITSMOE_ENOSPC, "ws_bytes=%zu < %zu", ws_bytes, need);
  if (need && ((uintptr_t)ws & 255u))
    return fail(BITSMOE_EINVAL, "misaligned workspace (256 bytes)");
  Mm8Args s{x, ldx, x_scales, ldxs, rows, div, x_rows, (const uint8_t*)codes, scales, bounds, R, E,
            N, K, (int)kg, (int)nb, y, ldy, 0};
  s.y16 = rows16(y, ldy, y_dtype == BITSMOE_F32 ? 4 : 2);
  const int fp = act ? kFewCols / 2 : kFewCols;
  const dim3 grid((unsigned)((N + fp - 1) / fp),
                  (unsigned)(bounds ? max_tiles(R, E, kFewRows) : (R + kFewRows - 1) / kFewRows));
  if (grid.y > 65535) return fail(BITSMOE_ESHAPE, "R=%d with E=%d: too many row tiles", R, E);
  with_out(y_dtype, [&](auto o) {
    using O = decltype(o);
    auto go = [&](auto tag) {
      using X = decltype(tag);
      if (act)
        hipLaunchKernelGGL((k_mm8_few<X, O, true>), grid, dim3(64 * kFewWaves), 0,
                           (hipStream_t)stream, s);
      else
        hipLaunchKernelGGL((k_mm8_few<X, O, false>), grid, dim3(64 * kFewWaves), 0,
                           (hipStream_t)stream, s);
    };
    if (given)
      go(E4M3{});
    else if constexpr (std::is_same<O, f16>::value)
      go(f16{});
    else if constexpr (std::is_same<O, bf16>::value)
      go(bf16{});
    else if (x_dtype == BITSMOE_F16)
      go(f16{});
    else
      go(bf16{});
  });
  return launched("fp8_matmul");
}

}  // extern "C"
