// Products grouped by expert of 8-bit floating point operands: rows with a
// scale per 128 inputs, weights with a scale per block of 128 x 128,
//   y[i, n] = sum_g sx[i, g] sw[e, n / 128, g] sum_{c in group g} qx[i, c] qw[e, n, c]
// (optionally SiLU(gate) * up of it).  The inner sums are the matrix cores', the
// outer one float32; each output is rounded once.  Rows may also come as fp16
// or bf16: they are then quantized on the way, to the same codes as by
// bitsmoe_fp8_rows.
#include <type_traits>

#include "fp8.h"
#include "tiles.h"

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
// A group's sums.  The 8-bit instruction aligns eight products at a time to their
// largest and drops what lies more than 13 bits below its first bit: an error of
// 1.4e-5 to 5e-5 of a result, where rounding it to fp16 adds up to 4.9e-4, to
// bf16 3.9e-3.  So 16-bit outputs come from it, and float32 ones (EXACT) from
// codes turned to fp16, four instructions in float32 (1e-7 of a result) at under
// half the rate, and a slow conversion of every two codes.
__device__ __forceinline__ f32x4 group_sums(const Halves& a, const Halves& b) {
  f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 4; ++j) p = mfma16(a.v[j], b.v[j], p);
  return p;
}

// (scale operands of 0: none of its own)
__device__ __forceinline__ f32x4 group_sums(const i32x8& a, const i32x8& b) {
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}

template <bool EXACT>
struct Operands {
  typedef i32x8 type;
  static __device__ __forceinline__ i32x8 of(const i32x8& q) { return q; }
};
template <>
struct Operands<true> {
  typedef Halves type;
  static __device__ __forceinline__ Halves of(const i32x8& q) { return halves(q); }
};

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

__device__ const float g_nan = __builtin_nanf("");

__device__ __forceinline__ int x_row8(const Mm8Args& s, int i) {
  if (!s.rows) return i;
  const int p = s.rows[i];
  const int r = p < 0 ? -1 : p / s.div;
  return r < s.x_rows ? r : -1;
}

// ------------------------------------------------- few rows per expert
// A work-group takes up to 32 sorted rows of one expert and 32 rows of its
// weights (with the activation 16 of the gate and the same 16 of the up half);
// its four waves split the groups, a whole line of each weight row each, and
// add up their sums through LDS (eight waves: a pair takes 16 of the weight
// rows each, so that the sums keep their order).  Weights go straight into
// registers, once; they are the products' first operand, so a lane holds 4
// outputs of one row of x, whose scale it needs once.  Which of a group's 128
// elements lie in which lane does not matter as long as both operands agree:
// lane (r, q) holds bytes 16 q .. and 64 + 16 q .. of row r, so that a load
// covers 64 bytes of 16 rows.
//
// Rows that are not codes yet are quantized by the work-group, a turn's groups
// at a time, into LDS, while its weights are on their way.
//
// Bound by the weights' bytes: two rows of each of 128 experts of 1536 x 2048
// (403 MB) 68 us from codes, 5.9 TB/s; 32 tokens of them, Zipf, 45 us (5.2 TB/s
// over the experts reached); the 8 of one token (25 MB) 8.2 us, a chain of
// latencies: bounds, row, its codes, weights, sums of the waves.  With more rows
// (up to 64 a work-group) 64 rows of 4096 x 4096 19 us instead of 13; with the
// last turn always whole, where half its groups do not exist, 64 experts of 512 x
// 1024, 8 rows each, 14.6 instead of 9.7.
constexpr int kFewRows = 32, kFewCols = 32;
// Most sorted rows of a call that quantizes them on the way: every wave holds
// the indexes of all of them, one a lane.
constexpr int kWayRows = 32;
static_assert(kWayRows <= 64, "a shuffle finds a row's index");

// 16 + 16 bytes of a row of codes at group start p (+ 16 q)
__device__ __forceinline__ i32x8 load_codes(const uint8_t* p) {
  const i32x4 a = *reinterpret_cast<const i32x4*>(p), b = *reinterpret_cast<const i32x4*>(p + 64);
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

template <int W>
struct FewLds {
  static constexpr int kTurn = 4 * W;  // groups of 16 rows (half as many of 32) in a turn
  // rows of a turn's codes, 16 bytes apart from a multiple of 256 so that the
  // reads of 16 rows spread over the banks; later the waves' sums
  union {
    uint8_t codes[16 * (kTurn * kGroup) + 32 * 16];
    f32x4 part[4 * 4 * 64];
  };
  float scales[16 * kTurn];
};

// (at: for rows that are not codes, the index of row `lane` of all R <= kWayRows rows)
template <class X, class O, bool ACT, int MB, int W>
__device__ __forceinline__ void few8_rows(const Mm8Args& s, const Tile& t, int at, FewLds<W>& lds) {
  constexpr bool kCodes = std::is_same<X, E4M3>::value;
  typedef typename Operands<sizeof(O) == 4>::type Frag;
  constexpr auto operand = Operands<sizeof(O) == 4>::of;
  constexpr int kTurn = FewLds<W>::kTurn / MB;  // groups of a turn
  constexpr int kMine = kTurn / 4;              // of a wave, whose loads are in flight together
  constexpr int NB = 8 / W;                     // its 16 x 16 tiles across, from b0
  constexpr int kRow = kTurn * kGroup + 16;  // bytes of an LDS row
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4, quarter = wv & 3, b0 = wv >> 2;
  const int n0 = blockIdx.x * (ACT ? kFewCols / 2 : kFewCols);
  const int64_t kp = (int64_t)s.kg * kGroup;
  const uint8_t* w[NB];
  const float* ws[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int b = b0 + i;
    const int n = n0 + (ACT ? 0 : 16 * b);
    const int64_t row = (int64_t)(ACT ? b : 0) * s.N + min(n + r, s.N - 1);
    w[i] = s.w + ((int64_t)t.e * (ACT ? 2 : 1) * s.N + row) * kp + 16 * q;
    // (32 and 16 divide 128: a work-group's rows share a block)
    ws[i] = s.ws + ((int64_t)t.e * (ACT ? 2 : 1) * s.nb + (ACT ? b : 0) * s.nb + n0 / kGroup) * s.kg;
  }
  const uint8_t* x[MB];
  const float* xs[MB];
  int xs_step[MB];  // (a row outside x: the same NaN for every group)
  if constexpr (kCodes) {
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const int xr = x_row8(s, t.row0 + min(16 * m + r, t.n - 1));
      x[m] = (const uint8_t*)s.x + (int64_t)max(xr, 0) * s.ldx + 16 * q;
      xs[m] = xr < 0 ? &g_nan : s.xs + (int64_t)xr * s.ldxs;
      xs_step[m] = xr < 0 ? 0 : 1;
    }
  }
  f32x4 acc[MB][NB] = {};
  // groups g0 .., U of each wave
  auto turn = [&](int g0, auto mine) {
    constexpr int U = decltype(mine)::value;
    // (groups past the last are loaded as it and not used)
    i32x8 vw[U][NB], vx[U][MB];
    float sw[U][NB], sx[U][MB];
    // rows on their way to codes: 16 lanes a group, as in k_fp8_rows.  The first
    // ones' loads come before the weights', so that their codes are made while
    // the weights are on their way.
    constexpr int kGroups = U * 4;
    const int groups = t.n * kGroups, l = threadIdx.x & 15;
    auto load_row = [&](int i, float (&v)[8]) {
      const int row = i / kGroups, c = (g0 + i % kGroups) * kGroup + 8 * l;
      int xr = t.row0 + min(row, t.n - 1);
      if (s.rows) {
        const int p = __shfl(at, xr, 64);
        xr = p < 0 || p / s.div >= s.x_rows ? -1 : p / s.div;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
      typedef typename std::conditional<kCodes, f16, X>::type Elem;
      if (i < groups && xr >= 0) load8_any((const Elem*)s.x + (int64_t)xr * s.ldx + c, s.K - c, v);
      return xr;
    };
    float v[8];
    int xr = 0;
    if constexpr (!kCodes) xr = load_row(threadIdx.x >> 4, v);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = min(g0 + u * 4 + quarter, s.kg - 1);
#pragma unroll
      for (int b = 0; b < NB; ++b) vw[u][b] = load_codes(w[b] + (int64_t)g * kGroup), sw[u][b] = ws[b][g];
      if constexpr (kCodes) {
#pragma unroll
        for (int m = 0; m < MB; ++m) {
          vx[u][m] = load_codes(x[m] + (int64_t)g * kGroup);
          sx[u][m] = xs[m][g * xs_step[m]];
        }
      }
    }
    // (all of a turn's loads before the first use)
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (!kCodes) {
      if (g0) __syncthreads();  // (the turn before is read)
      for (int i = threadIdx.x >> 4; i < (groups + 4 * W - 1) / (4 * W) * (4 * W); i += 4 * W) {
        const int row = i / kGroups, g = i % kGroups;
        if (i >= 4 * W) xr = load_row(i, v);
        uint32_t a = row_max(amax_bits<false>(v));
        if (__any(a >= kInfBits)) a = row_max(amax_bits<true>(v));
        const Factors f = factors8(a);
        if (i < groups) {
          uint2 o;
          o.x = codes4(v[0], v[1], v[2], v[3], f.r);
          o.y = codes4(v[4], v[5], v[6], v[7], f.r);
          *reinterpret_cast<uint2*>(lds.codes + row * kRow + g * kGroup + 8 * l) = o;
          if (l == 0) lds.scales[row * kTurn + g] = xr < 0 ? __builtin_nanf("") : f.s;
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int gl = u * 4 + quarter;
      if (g0 + gl >= s.kg) break;
      Frag hw[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) hw[b] = operand(vw[u][b]);
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        if constexpr (!kCodes) {
          const int row = min(16 * m + r, t.n - 1);
          vx[u][m] = load_codes(lds.codes + row * kRow + gl * kGroup + 16 * q);
          sx[u][m] = lds.scales[row * kTurn + gl];
        }
        const Frag hx = operand(vx[u][m]);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const f32x4 p = group_sums(hw[b], hx);
          const float f = sx[u][m] * sw[u][b];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[m][b][j] = fmaf(p[j], f, acc[m][b][j]);
        }
      }
    }
  };
#pragma unroll 1
  for (int g0 = 0; g0 < s.kg; g0 += kTurn) {
    if (s.kg - g0 > kTurn / 2)
      turn(g0, std::integral_constant<int, kMine>{});
    else
      turn(g0, std::integral_constant<int, kMine / 2>{});
  }

  // sums of the waves: [wave][tile of 16 x 16][lane]
  if (!kCodes) __syncthreads();
  f32x4* part = lds.part;
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int b = 0; b < NB; ++b) part[(quarter * MB * 2 + m * 2 + b0 + b) * 64 + lane] = acc[m][b];
  __syncthreads();
  O* Y = (O*)s.y;
  for (int i = wv; i < (ACT ? MB : MB * 2); i += W) {
    const int m = ACT ? i : i >> 1;
    f32x4 v[2];
#pragma unroll
    for (int b = 0; b < (ACT ? 2 : 1); ++b) {
      const int at = ACT ? m * 2 + b : i;
      v[b] = part[at * 64 + lane];
#pragma unroll
      for (int o = 1; o < 4; ++o) {
        const f32x4 p = part[(o * MB * 2 + at) * 64 + lane];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[b][j] += p[j];
      }
    }
    const int n = n0 + (ACT ? 0 : 16 * (i & 1)) + 4 * q;
    if (16 * m + r >= t.n) continue;
    typedef __attribute__((ext_vector_type(4))) O O4;
    O4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = (O)(ACT ? gated(v[0][j], v[1][j]) : v[0][j]);
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

// (16-bit outputs of codes fit four work-groups a compute unit; the others would
// spill, or are too few to need them)
template <class X, class O>
constexpr int kFewOnUnit = sizeof(O) == 2 && std::is_same<X, E4M3>::value ? 4 : 3;

template <class X, class O, bool ACT, int W>
__global__ __launch_bounds__(64 * W, W == 8 ? 2 : (kFewOnUnit<X, O>)) void k_mm8_few(Mm8Args s) {
  __shared__ FewLds<W> lds;
  int at = 0;
  if (!std::is_same<X, E4M3>::value && s.rows) at = s.rows[min((int)threadIdx.x & 63, s.R - 1)];
  Tile t{0, 0, 0};
  if (s.bounds) {
    t = find_tile(s.bounds, s.E, s.R, blockIdx.y, kFewRows);
  } else {
    t.row0 = (int)blockIdx.y * kFewRows;
    t.n = min(kFewRows, s.R - t.row0);
  }
  if (t.n <= 0) return;
  if (t.n <= 16)
    few8_rows<X, O, ACT, 1, W>(s, t, at, lds);
  else
    few8_rows<X, O, ACT, 2, W>(s, t, at, lds);
}

// --------------------------------------------------------------- tiled
// Work-group tile of TM sorted rows x TN weight rows, WM x WN waves, the
// contraction a group of 128 at a time: both operands' tiles are rows of 128
// bytes, copied straight into LDS into one of kBufs buffers, kBufs - 1 groups
// ahead of the products, with the rows' scales and the tile's (at most two)
// weight scales behind them.  16-byte piece p of row r lies at place
// p ^ (r / 2 % 8), so that the 16 rows a matrix-core operand touches spread
// over all 64 banks.
//
// A group's 16 x 16 sums leave the matrix cores unscaled and are added to the
// accumulators times the product of the two scales, 16 rows later in the
// wave's order, while the matrix cores work on: four multiply-adds a lane
// against 32 cycles of the matrix cores.
//
// 8192 rows x 4096 weight rows x 14336 inputs 382 us, 2520 TFLOP/s (the library's
// 8192^3 product with one scale for each operand 2710), with 2048 inputs 69 us,
// 2000; 24576 rows of 64 experts with the activation 198 us, 8 experts of about
// 1024 rows, 4096 x 14336, 468.  The matrix cores are busy 57 % of a busy compute
// unit's time; without the copies the same loop takes 75 % of its time, without
// the scaling 98 %, with operands that stay in L2 93 %.
constexpr int kTile = 256;  // rows and weight rows of a whole tile
constexpr uint32_t kScaleLds = 2048;                              // of one buffer
constexpr uint32_t kLds8 = 3 * ((kTile + kTile / 2) * kGroup + kScaleLds);  // three buffers of a 256 x 128 tile

// As copy16, 4 bytes per lane.
__device__ __forceinline__ void copy4(const void* src, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" : : "v"(src), "{m0}"(lds) : "memory");
}

template <class V>
__device__ __forceinline__ V lds_read(uint32_t at) {
  typedef __attribute__((address_space(3))) const V lds_v;
  return *(lds_v*)(uintptr_t)at;
}

// SiLU(g) u for a 16-bit output: the exponent -g log2(e) keeps its own
// rounding, off by up to 5e-6 of the result (|g| < 87), where the sums' 14 bits
// may be off by more; two thirds of gated()'s time, which is 5 us of a tile's
// 38 with 2048 inputs.
__device__ __forceinline__ float gated16(float g, float u) {
  const float e = __builtin_amdgcn_exp2f(g * -1.44269502162933349609375f);
  return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

// Sorted rows m0 .. m0 + mn, weight rows (of each half) n0 .. n0 + nn of expert e.
template <class O, int TM, int TN, int WM, int WN, int kBufs, bool ACT, bool EXACT>
__device__ __forceinline__ void mm8_tile(const Mm8Args& s, uint32_t base, int e, int m0, int mn,
                                         int n0, int nn) {
  constexpr int NT = 64 * WM * WN;
  constexpr int MI = TM / WM / 16, NI = TN / WN / 16;  // 16 x 16 tiles of a wave
  constexpr int kCa = TM * 8 / NT, kCb = TN * 8 / NT;  // copies of a lane
  constexpr int kPieces = kCa + kCb + 1;
  constexpr uint32_t kBytesA = TM * kGroup, kScales = (TM + TN) * kGroup;
  constexpr uint32_t kBuf = kScales + kScaleLds;
  static_assert(kBufs * kBuf <= kLds8 && kCa * NT == TM * 8 && kCb * NT == TN * 8, "buffers");
  static_assert(NT * 4 <= (int)kScaleLds && TM <= NT - 64, "a wave for the weights' scales");
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = s.kg;

  // addresses of the pieces of group 0
  const uint8_t* pa[kCa];
  const uint8_t* pb[kCb];
  const int64_t kp = (int64_t)kg * kGroup;
#pragma unroll
  for (int i = 0; i < kCa; ++i) {
    const int l = (i * NT + (int)threadIdx.x) >> 3, p = (threadIdx.x & 7) ^ ((l >> 1) & 7);
    const int xr = x_row8(s, m0 + min(l, mn - 1));
    pa[i] = (const uint8_t*)s.x + (int64_t)max(xr, 0) * s.ldx + p * 16;
  }
#pragma unroll
  for (int i = 0; i < kCb; ++i) {
    const int l = (i * NT + (int)threadIdx.x) >> 3, p = (threadIdx.x & 7) ^ ((l >> 1) & 7);
    // with the activation, blocks of 16 tile rows alternate gate and up
    const int col = ACT ? (l >> 5) * 16 + (l & 15) : l;
    const int64_t row = (int64_t)e * (ACT ? 2 : 1) * s.N + n0 + min(col, nn - 1) + (ACT && (l & 16) ? s.N : 0);
    pb[i] = s.w + row * kp + p * 16;
  }
  // scales: TM / 64 waves copy the rows' (NaN for a row outside x), the others
  // the weights', blocks 0 and 1 in turn
  const float* ps;
  int step_s = 1;
  if (wv * 64 < TM) {
    const int xr = x_row8(s, m0 + min(wv * 64 + lane, mn - 1));
    ps = xr < 0 ? &g_nan : s.xs + (int64_t)xr * s.ldxs;
    step_s = xr < 0 ? 0 : 1;
  } else {
    const int which = lane & 1, nb0 = n0 / kGroup;
    const int64_t block = (int64_t)e * (ACT ? 2 : 1) * s.nb + (ACT ? nb0 + which * s.nb : min(nb0 + which, s.nb - 1));
    ps = s.ws + block * kg;
  }
  // Piece i of the copies of group g: rows first, then weights, then scales.
  // (Groups past the last repeat it: nobody reads them.)
  auto stage_piece = [&](int i, int g, uint32_t buf) {
    const int at = min(g, kg - 1);
    if (i < kCa)
      copy16(pa[i] + (int64_t)at * kGroup, buf + (uint32_t)(i * NT + wv * 64) * 16);
    else if (i < kCa + kCb)
      copy16(pb[i - kCa] + (int64_t)at * kGroup, buf + kBytesA + (uint32_t)((i - kCa) * NT + wv * 64) * 16);
    else
      copy4(ps + at * step_s, buf + kScales + (uint32_t)wv * 256);
  };

  static_assert(MI % 2 == 0, "turns of the registers");
  typedef typename Operands<EXACT>::type Frag;
  constexpr auto operand = Operands<EXACT>::of;
  const int wm = (wv / WN) * (TM / WM), wn = (wv % WN) * (TN / WN);
  const int l16 = lane & 15;
  const uint32_t piece = ((lane >> 4) ^ ((l16 >> 1) & 7)) << 4;
  // (buffers start at multiples of 1024 bytes, so adding one keeps the xor)
  const uint32_t off_a = (wm + l16) * kGroup + piece, off_b = kBytesA + (wn + l16) * kGroup + piece;
  const uint32_t off_s = kScales + (wm + l16) * 4, off_w = kScales + TM * 4 + (ACT ? 0 : wn / kGroup * 4);
  auto raw = [&](uint32_t at, int g) {
    const i32x4 a = lds_read<i32x4>(at + g * 16 * kGroup), b = lds_read<i32x4>((at ^ 64) + g * 16 * kGroup);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  f32x4 acc[MI][NI] = {}, part[NI] = {};
  i32x8 fa[2], fb[NI];
  float sa[2], sw[2], f[2] = {0.f, 0.f};
  auto read_a = [&](int g, uint32_t buf) {
    fa[g & 1] = raw(buf + off_a, g);
    sa[g & 1] = lds_read<float>(buf + off_s + g * 64);
  };
  auto read_w = [&](uint32_t buf) {
    sw[0] = lds_read<float>(buf + off_w);
    if (ACT) sw[1] = lds_read<float>(buf + off_w + 4);
  };
  auto add = [&](int g, int j) {  // the sums of the 16 rows before, scaled
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[g][j][q] = fmaf(part[j][q], f[ACT ? j & 1 : 0], acc[g][j][q]);
  };
  uint32_t cur = base;
  auto after = [&](uint32_t b) { return b == base + (kBufs - 1) * kBuf ? base : b + kBuf; };
  // MI turns of 16 rows; the reads of a turn's rows are issued a turn ahead,
  // the weights' of the next group as soon as the last products have theirs.
  // Before the last turn (the border) the wave waits for its copies of the next
  // group and meets the others; then nobody reads this group's buffer any more.
  //
  // With two buffers the copies of a later group would have one group's time,
  // and come all at once: so the waves meet once more, halfway, and what is read
  // by then (the weights, which lie in registers; the first half of the rows) is
  // copied over early (8 experts of about 1024 rows, 4096 x 14336: 529 -> 470
  // us; meeting twice for it 490).
  constexpr bool kEarly = kBufs == 2;
  static_assert(!kEarly || (MI == 8 && kCa == 4 && kCb == 4), "early copies");
  auto stage = [&](int g, int c) {  // in turn g of group c, into its own buffer
    if constexpr (kEarly) {
      if (g == 4 || g == 5) {
        stage_piece(kCa + 2 * (g - 4), c + kBufs, cur);
        stage_piece(kCa + 2 * (g - 4) + 1, c + kBufs, cur);
      }
      if (g == 6) {
        stage_piece(0, c + kBufs, cur);
        stage_piece(2, c + kBufs, cur);
      }
      if (g == 7) {
        stage_piece(1, c + kBufs, cur);
        stage_piece(3, c + kBufs, cur);
        stage_piece(kCa + kCb, c + kBufs, cur);
      }
    } else if (g == MI - 1) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) stage_piece(i, c + kBufs, cur);
    }
  };
  auto meet = [&](int g) {
    if (g == MI - 1) {
      wait_copies<kEarly ? 6 : (kBufs - 2) * kPieces>();
      lds_barrier();
    } else if (kEarly && (g == 4)) {
      lds_barrier();
    }
  };
  auto step = [&](int c, auto last_) {
    constexpr bool kLast = decltype(last_)::value;
    const uint32_t nxt = after(cur);
    Frag b[NI];
#pragma unroll
    for (int j = 0; j < NI; ++j) b[j] = operand(fb[j]);
#pragma unroll
    for (int g = 0; g < MI; ++g) {
      const bool border = g == MI - 1;
      if (!kLast) meet(g);
      const Frag a = operand(fa[g & 1]);
      const float f0 = sa[g & 1] * sw[0], f1 = ACT ? sa[g & 1] * sw[1] : 0.f;
      if (!border) read_a(g + 1, cur);
      if (!kLast && border) {
        read_a(0, nxt);
        read_w(nxt);
      }
      if (!kLast) stage(g, c);
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        add(g == 0 ? MI - 1 : g - 1, j);
        part[j] = group_sums(b[j], a);
        if (!kLast && border) fb[j] = raw(nxt + off_b, j);
      }
      f[0] = f0, f[1] = f1;
      if (!EXACT && !border) {
        __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    cur = nxt;
  };
#pragma unroll 1
  for (int i = 0; i < kBufs; ++i)
#pragma unroll
    for (int j = 0; j < kPieces; ++j) stage_piece(j, i, base + i * kBuf);
  wait_copies<(kBufs - 1) * kPieces>();  // the first group's
  lds_barrier();
  if (wm < mn) {
    read_w(cur);
#pragma unroll
    for (int j = 0; j < NI; ++j) fb[j] = raw(cur + off_b, j);
    read_a(0, cur);
    int c = 0;
#pragma unroll 1
    for (; c + 1 < kg; ++c) step(c, std::false_type{});
    step(c, std::true_type{});
#pragma unroll
    for (int j = 0; j < NI; ++j) add(MI - 1, j);
  } else {  // a wave past the tile's rows only copies
#pragma unroll 1
    for (int c = 0; c + 1 < kg; ++c) {
#pragma unroll
      for (int g = 0; g < MI; ++g) {
        meet(g);
        stage(g, c);
      }
      cur = after(cur);
    }
  }
  wait_copies<0>();  // nothing is written into this work-group's LDS after its end

  // The products were formed transposed: lane % 16 is the output row, and a
  // lane holds 4 consecutive columns 4 (lane / 16) .. of each 16 x 16 tile.
  // 16-bit outputs: two tiles side by side trade their odd and even quarters,
  // which leaves every lane 8 consecutive columns of one of them, so a store
  // writes 16 bytes a lane and 64 a row (a wave with one tile across trades
  // with the next 16 rows: 32 a row); float32 ones do as they are.
  if (wm >= mn) return;
  O* Y = (O*)s.y + (int64_t)m0 * s.ldy + n0;
  constexpr int kPer = 16 / (int)sizeof(O);
  constexpr int kOuts = ACT ? NI / 2 : NI;                             // output tiles of a wave across
  constexpr int kTrade = sizeof(O) == 4 ? 0 : kOuts % 2 == 0 ? 1 : 2;  // with no tile, the next across, the next down
  constexpr int kTiles = kTrade ? 2 : 1;
  const int quarter = lane >> 4;
  typedef __attribute__((ext_vector_type(kPer))) O On;
#pragma unroll
  for (int i = 0; i < MI; i += kTrade == 2 ? 2 : 1) {
#pragma unroll
    for (int j = 0; j < kOuts; j += kTrade == 1 ? 2 : 1) {
      uint32_t w[4];
      int row = wm + 16 * i + l16, col = (ACT ? wn / 2 : wn) + 16 * j + 4 * quarter;
      f32x4 v[kTiles];
#pragma unroll
      for (int u = 0; u < kTiles; ++u) {
        const int ii = i + (kTrade == 2 ? u : 0), jj = j + (kTrade == 1 ? u : 0);
        v[u] = acc[ii][jj * (ACT ? 2 : 1)];
        if constexpr (ACT) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float g = v[u][q], up = acc[ii][jj * 2 + 1][q];
            v[u][q] = EXACT ? gated(g, up) : gated16(g, up);
          }
        }
      }
      if constexpr (kTiles == 2) {
        typedef __attribute__((ext_vector_type(2))) O O2;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const O2 a = {(O)v[0][2 * h], (O)v[0][2 * h + 1]}, b = {(O)v[1][2 * h], (O)v[1][2 * h + 1]};
          const auto t = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a),
                                                          __builtin_bit_cast(uint32_t, b), false, false);
          w[h] = t[0], w[2 + h] = t[1];
        }
        col = (ACT ? wn / 2 : wn) + 16 * (j + (kTrade == 1 ? quarter & 1 : 0)) + 8 * (quarter >> 1);
        if (kTrade == 2) row += 16 * (quarter & 1);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = __float_as_uint(v[0][q]);
      }
      if (row >= mn) continue;
      O* y = Y + (int64_t)row * s.ldy + col;
      const i32x4 o = {(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
      if (s.y16 && col + kPer <= nn) {
        *reinterpret_cast<i32x4*>(y) = o;
      } else {
        const On e = __builtin_bit_cast(On, o);
#pragma unroll
        for (int q = 0; q < kPer; ++q)
          if (col + q < nn) y[q] = e[q];
      }
    }
  }
}

// One work-group per tile: first the whole rounds of the chip's compute units
// with 256 x 256 tiles, then what is left, cut in four 128 x 128 tiles where
// those make one round at most, in two of 256 x 128 where those do, else as it
// is.  float32 outputs: 256 x 128 tiles alone (fp16 operands take twice the
// registers).
template <class O, bool ACT>
__global__ __launch_bounds__(512, 2) void k_mm8_tile(Mm8Args s) {
  __shared__ __align__(1024) uint8_t lds[kLds8];
  constexpr bool kExact = sizeof(O) == 4;
  const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  constexpr int kCols = (kExact ? kTile / 2 : kTile) / (ACT ? 2 : 1);  // output columns per tile
  const int ntn = (s.N + kCols - 1) / kCols;
  const int mt = s.bounds ? count_tiles(s.bounds, s.E, s.R, kTile) : (s.R + kTile - 1) / kTile;
  const uint32_t total = (uint32_t)mt * ntn, left = total % kUnits;
  const uint32_t parts = kExact ? 1 : left <= kUnits / 4 ? 4 : left <= kUnits / 2 ? 2 : 1;
  const uint32_t whole = parts > 1 ? total - left : total;
  // Work-group b runs on XCD b % 8, and every XCD takes 32 consecutive tiles of
  // a round, which share operand rows in its L2.
  uint32_t b = blockIdx.x, id;
  int part = -1;
  const uint32_t rounds = (whole + kUnits - 1) / kUnits;
  if (b < rounds * kUnits) {
    id = b / kUnits * kUnits + (b & 7) * (kUnits / 8) + b % kUnits / 8;
    if (id >= whole) return;
  } else {
    b -= rounds * kUnits;
    const uint32_t cut = (total - whole) * parts, run = (cut + 7) / 8;
    const uint32_t at = (b & 7) * run + (b >> 3);
    if ((b >> 3) >= run || at >= cut) return;
    id = whole + at / parts;
    part = at % parts;
  }
  int mi, ni;
  tile_place(id, mt, ntn, mi, ni);
  Tile t{0, mi * kTile, min(kTile, s.R - mi * kTile)};
  if (s.bounds) t = find_tile(s.bounds, s.E, s.R, mi, kTile);
  if (t.n <= 0) return;
  int n0 = ni * kCols, nn = min(kCols, s.N - n0);
  if constexpr (kExact) {
    mm8_tile<O, kTile, kTile / 2, 2, 4, 3, ACT, true>(s, base, t.e, t.row0, t.n, n0, nn);
  } else if (part < 0) {
    if (t.n <= kTile / 2)
      mm8_tile<O, kTile / 2, kTile, 2, 4, 3, ACT, false>(s, base, t.e, t.row0, t.n, n0, nn);
    else
      mm8_tile<O, kTile, kTile, 2, 4, 2, ACT, false>(s, base, t.e, t.row0, t.n, n0, nn);
  } else if (parts == 4) {
    const int pm = (part & 1) * (kTile / 2), pn = (part >> 1) * (kCols / 2);
    t.n = min(kTile / 2, t.n - pm), nn = min(kCols / 2, nn - pn);
    if (t.n <= 0 || nn <= 0) return;
    mm8_tile<O, kTile / 2, kTile / 2, 2, 4, 4, ACT, false>(s, base, t.e, t.row0 + pm, t.n, n0 + pn, nn);
  } else {
    const int pn = part * (kCols / 2);
    nn = min(kCols / 2, nn - pn);
    if (nn <= 0) return;
    if (t.n <= kTile / 2)
      mm8_tile<O, kTile / 2, kTile / 2, 2, 4, 4, ACT, false>(s, base, t.e, t.row0, t.n, n0 + pn, nn);
    else
      mm8_tile<O, kTile, kTile / 2, 2, 4, 3, ACT, false>(s, base, t.e, t.row0, t.n, n0 + pn, nn);
  }
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

// The few-rows kernel is the faster one up to 8 rows per expert on average, up to
// 16 where it makes at most four work-groups a compute unit, and where it makes
// at most two.  us by it and by the tiled one, from codes, over weights that no
// cache holds: 128 experts of 1536 x 2048 (6144 work-groups), 4 rows 70 and 80,
// 8 rows 76 and 81, 16 rows 92 and 82; 8 experts of 4096 x 4096 (1024), 16 rows
// 34 and 36, 32 rows 43 and 36; 32 of 1536 x 2048 (1536), 16 rows 26 and 25; one
// of 4096 x 4096, 64 rows (256) 13 and 23, 128 rows (512) 21 and 30, 192 rows
// (768) 30 and 27; one of 8192 x 2048, 64 rows (512) 12.7 and 12.6.
constexpr int kFewMean = 8, kFewMean4 = 16;

long long few_parts(int R, int E, int N, int act) {
  const long long mean = ((long long)R + E - 1) / E, wn = act ? 2ll * N : N;
  return (wn + kFewCols - 1) / kFewCols * ((mean + kFewRows - 1) / kFewRows) * E;
}

bool few8(int R, int E, int N, int act) {
  const long long mean = ((long long)R + E - 1) / E, parts = few_parts(R, E, N, act);
  return max_tiles(R, E, kFewRows) <= 65535 &&
         (mean <= kFewMean || (mean <= kFewMean4 && parts <= 4 * kUnits) || parts <= 2 * kUnits);
}

// Rows quantized by the work-groups that use them: eight waves where there is at
// most one work-group a compute unit (4 rows of 4096 x 4096 9.3 us instead of
// 12.1; 8 experts of 1536 x 2048, 384 work-groups, 10.8 instead of 8.9) and at
// least a turn of 16 groups (one row of 2048 x 512 4.4 instead of 3.4).
bool few_more(int R, int E, int N, int K, int act) {
  return few_parts(R, E, N, act) <= kUnits && K >= 16 * kGroup;
}

// Few rows are quantized by the work-groups that use them, without a launch of
// their own: each work-group of an expert does it again, which takes four waves
// 1.2 us per 4096 elements.  us by it and by two launches: one row of 8 experts
// of 1536 x 2048 8.9 and 12.2, of 32 experts 21 and 24; of 8 experts of 4096 x
// 4096, one row 31 and 33, four rows 37 and 34; of one such projection, one row
// 7.6 and 11.3, 4 rows 9.3 and 12.0, 6 rows 10.9 and 12.2, 8 rows 12.5 and 12.5;
// 16 rows of 4096 x 2048 10.7 and 9.5.
// At most kWayRows rows, which one expert may have all.
bool on_the_way(int R, int E, int N, int K, int act) {
  const long long mean = ((long long)R + E - 1) / E;
  const long long most = mean <= 8 && few_more(R, E, N, K, act) ? 32768 : few_parts(R, E, N, act) <= 2 * kUnits ? 16384 : 8192;
  return R <= kWayRows && mean * K <= most;
}

// The workspace of rows that are quantized before the products: codes, then
// scales.
struct RowsWs {
  size_t codes, scales;
};
RowsWs rows_ws(int x_dtype, int64_t rows, int R, int E, int N, int K, int act) {
  if (x_dtype == kE4M3 || (few8(R, E, N, act) && on_the_way(R, E, N, K, act))) return RowsWs{0, 0};
  auto al = [](size_t x) { return (x + 255) / 256 * 256; };
  return RowsWs{al((size_t)rows * groups_of(K) * kGroup), al((size_t)rows * groups_of(K) * 4)};
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
  const RowsWs w = rows_ws(x_dtype, x_rows < R ? x_rows : R, R, E, N, K, act);
  *bytes = w.codes + w.scales;
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
  // Each row of x once, or each sorted row where those are fewer (without
  // indexes only the first R rows of x are read).
  const bool sorted = !rows || R < x_rows;
  const int live = sorted ? R : x_rows;
  const RowsWs w = rows_ws(x_dtype, live, R, E, N, K, act);
  const size_t need = w.codes + w.scales;
  if (need > ws_bytes || (need && !ws))
    return fail(BITSMOE_ENOSPC, "ws_bytes=%zu < %zu", ws_bytes, need);
  if (need && ((uintptr_t)ws & 255u))
    return fail(BITSMOE_EINVAL, "misaligned workspace (256 bytes)");
  Mm8Args s{x, ldx, x_scales, ldxs, rows, div, x_rows, (const uint8_t*)codes, scales, bounds, R, E,
            N, K, (int)kg, (int)nb, y, ldy, 0};
  s.y16 = rows16(y, ldy, y_dtype == BITSMOE_F32 ? 4 : 2);
  const bool few = few8(R, E, N, act);
  const int fp = act ? kFewCols / 2 : kFewCols;
  const dim3 grid((unsigned)((N + fp - 1) / fp),
                  (unsigned)(bounds ? max_tiles(R, E, kFewRows) : (R + kFewRows - 1) / kFewRows));
  const int per = (y_dtype == BITSMOE_F32 ? kTile / 2 : kTile) / (act ? 2 : 1);
  const long long ntn = (N + per - 1) / per;
  const long long mt = bounds ? max_tiles(R, E, kTile) : (R + kTile - 1) / kTile;
  // enough for any split of at most mt * ntn tiles into whole rounds and cut tiles
  const long long groups = (mt * ntn + kUnits - 1) / kUnits * kUnits + kUnits + 8;
  if (!few && groups * 512 > 0xFFFFFFFFll)  // (a grid's work-items)
    return fail(BITSMOE_ESHAPE, "R=%d E=%d N=%d K=%d make too many tiles", R, E, N, K);
  if (need) {
    s.x = ws, s.ldx = kg * kGroup;
    s.xs = (const float*)((uint8_t*)ws + w.codes), s.ldxs = kg;
    if (sorted) s.rows = nullptr, s.div = 1, s.x_rows = R;
    const int rc = run_fp8_rows(x_dtype, x, ldx, Gather{sorted ? rows : nullptr, div, x_rows},
                                BITSMOE_ACT_NONE, sorted ? bounds : nullptr, live, E, K, ws, s.ldx,
                                (float*)s.xs, kg, (hipStream_t)stream);
    if (rc) return rc;
  }
  with_out(y_dtype, [&](auto o) {
    using O = decltype(o);
    if (!few) {
      if (act)
        hipLaunchKernelGGL((k_mm8_tile<O, true>), dim3((unsigned)groups), dim3(512), 0,
                           (hipStream_t)stream, s);
      else
        hipLaunchKernelGGL((k_mm8_tile<O, false>), dim3((unsigned)groups), dim3(512), 0,
                           (hipStream_t)stream, s);
      return;
    }
    auto go = [&](auto tag) {
      using X = decltype(tag);
      constexpr int W = std::is_same<X, E4M3>::value ? 4 : 8;  // (codes: four waves always)
      const bool more = W == 8 && few_more(R, E, N, K, act);
      void (*kernel)(Mm8Args) = act ? k_mm8_few<X, O, true, 4> : k_mm8_few<X, O, false, 4>;
      if (more) kernel = act ? k_mm8_few<X, O, true, W> : k_mm8_few<X, O, false, W>;
      hipLaunchKernelGGL(kernel, grid, dim3(more ? 512 : 256), 0, (hipStream_t)stream, s);
    };
    if (given || need)
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
