// Products with 4-bit weights: W[n, c] = m[n, c / G] + s[n, c / G] q[n, c]
// with codes q of 0..15 (two per byte, the lower half first), float16 steps s
// and minima m per group of G inputs; dense or grouped by expert, optionally
// SiLU(gate) * up of the two halves of the rows.  Per group
//   sum_c W x = s (sum_c q x) + m (sum_c x),
// so the codes enter the products as the whole numbers 0..15, exactly.
#include <type_traits>

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

// 8 elements of x from an address of any element's alignment: the hardware
// takes 16 bytes at once all the same, so rows of any stride and offset run
// the same kernel, with the same bits.
template <class T>
__device__ __forceinline__ uint4 load_x8(const T* p) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  typedef u4 loose __attribute__((aligned(2)));
  return __builtin_bit_cast(uint4, (u4)*reinterpret_cast<const loose*>(p));
}

// One output, one input after another: sum_c (m + s q) x.  With an infinity or
// values near float32's largest in x the two sums of a group may be infinite
// where W x is not, or cancel to NaN where it is infinite, so the kernels below
// take every output that is not finite from here: slow (8 rows of each of 128
// experts with an infinity in each: 3.0 ms for 0.1), but what the product is, whichever
// kernel runs.
template <class T>
__device__ __forceinline__ float w4_one(const W4Args& s, int64_t row, const T* x) {
  const uint8_t* codes = s.codes + row * (s.K / 2);
  const int groups = s.K / s.G;
  float acc = 0.f;
#pragma unroll 1
  for (int c = 0; c < s.K && acc == acc; c += 8) {  // (a NaN stays one)
    const int64_t g = row * groups + c / s.G;
    const float sc = (float)s.scales[g], mn = s.mins ? (float)s.mins[g] : -8.f * sc;
    const uint32_t q = *reinterpret_cast<const uint32_t*>(codes + c / 2);
    const auto v = __builtin_bit_cast(typename Vec8<T>::type, load_x8(x + c));
#pragma unroll
    for (int j = 0; j < 8; ++j)
      acc = fmaf(fmaf(sc, (float)(q >> (4 * j) & 15), mn), to_f32<T>(v[j]), acc);
  }
  return acc;
}
// Output n of sorted row i of expert e from its sums g (and u, of the up half).
template <class T, class O, bool ACT>
__device__ __forceinline__ void w4_store(const W4Args& s, int e, int i, int n, float g, float u) {
  const int xr = w4_row(s, i);
  if (xr >= 0 && !(isfinite(g) && (!ACT || isfinite(u)))) {
    const T* x = (const T*)s.x + (int64_t)xr * s.ldx;
    const int64_t row = (int64_t)e * (ACT ? 2 : 1) * s.N + n;
    g = w4_one(s, row, x);
    if (ACT) u = w4_one(s, row + s.N, x);
  }
  float o = ACT ? gated(g, u) : g;
  if (xr < 0) o = __builtin_nanf("");
  ((O*)s.y)[(int64_t)i * s.ldy + n] = from_f32<O>(o);
}

// ------------------------------------------------------- three rows and more
// A work-group takes up to 32 rows of one expert and a block of 32 rows of its
// weights (with the activation 16 of the gate and the same 16 of the up
// half), whose inputs its four waves split in turns of 128, adding up through
// LDS.  Every code is read once per tile of rows, 16 bytes (32 inputs of one
// row) a lane, a stage of turns ahead of its use.
//
// In a turn lane (r, q) loads the codes of row r, inputs 32 q .. 32 q + 31.
// One matrix-core step takes 32 inputs, 8 a lane, that have to lie in one
// group: a 4 x 4 transpose of the words between the four lanes of a row (two
// row swaps each way) gives lane (r, q) the inputs 32 s + 8 q .. of step s.
// A word's eight codes become eight fp16 (bf16) values q, exactly: a byte q of
// 0..15 is the e4m3 number q 2^-9 (a subnormal up to 7, then 2^-6 (1 + (q - 8) / 8)),
// which the hardware converts two at a time, times 512.  Seven instructions,
// in the order 0 2 4 6 1 3 5 7; x is put into that order.  Per group
//   y += s (sum q x) + m (sum x),
// where sum x comes from one more matrix-core step with ones.  (The values 16 + q, q
// in the mantissa of 16.0, cost eight instructions and the difference of two
// sums as large as 16 s sum |x| where s q and m may be small.)  x is the first
// operand, so a lane's sums all belong to its own row of weights, whose s and
// m it holds.  All sums are float32.  Bound by vector instructions (about 170 a
// turn and wave, a third of them decode): 8 rows of each of 128 experts of
// 1536 x 2048, groups of 128, weights that no cache holds: 102 us.
constexpr int kRows = 32, kCols = 32, kWaves = 4, kTurn = 128;

// two ones
template <class T>
constexpr uint32_t kOnes = 0x3C003C00u;
template <>
constexpr uint32_t kOnes<bf16> = 0x3F803F80u;

// the e4m3 numbers of the lower (upper) two bytes times 512
template <bool kHigh>
__device__ __forceinline__ uint32_t codes2(uint32_t w, f16) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 512.0f, kHigh));
}
template <bool kHigh>
__device__ __forceinline__ uint32_t codes2(uint32_t w, bf16) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 512.0f, kHigh));
}

// 8 codes of a word, order 0 2 4 6 1 3 5 7
template <class T>
__device__ __forceinline__ typename Vec8<T>::type codes8(uint32_t w) {
  const uint32_t even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
  const uint4 o = {codes2<false>(even, T{}), codes2<true>(even, T{}), codes2<false>(odd, T{}),
                   codes2<true>(odd, T{})};
  return __builtin_bit_cast(typename Vec8<T>::type, o);
}

// x in the same order
template <class T>
__device__ __forceinline__ typename Vec8<T>::type order8(uint4 v) {
  uint4 o;
  o.x = __builtin_amdgcn_perm(v.y, v.x, 0x05040100u);
  o.y = __builtin_amdgcn_perm(v.w, v.z, 0x05040100u);
  o.z = __builtin_amdgcn_perm(v.y, v.x, 0x07060302u);
  o.w = __builtin_amdgcn_perm(v.w, v.z, 0x07060302u);
  return __builtin_bit_cast(typename Vec8<T>::type, o);
}

// d[j] of lane row q <- d[q] of lane row j
__device__ __forceinline__ void transpose4(uint32_t (&d)[4]) {
  typedef __attribute__((ext_vector_type(2))) uint32_t u2;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const u2 t = __builtin_bit_cast(u2, __builtin_amdgcn_permlane32_swap(d[j], d[j + 2], false, false));
    d[j] = t[0], d[j + 2] = t[1];
  }
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    const u2 t = __builtin_bit_cast(u2, __builtin_amdgcn_permlane16_swap(d[j], d[j + 1], false, false));
    d[j] = t[0], d[j + 1] = t[1];
  }
}

// the 128 / G float16 values of a turn's groups, from an address that is only
// 2-byte aligned
template <int N>
struct Halves {
  typedef _Float16 type __attribute__((ext_vector_type(N)));
  typedef type loose __attribute__((aligned(2)));
};
template <int N>
__device__ __forceinline__ typename Halves<N>::type load_halves(const f16* p) {
  return *reinterpret_cast<const typename Halves<N>::loose*>(p);
}

// U: turns of a stage; the loads of one are in flight during the products of
// the one before
template <class T, class O, int G, bool ACT, int MB, int U>
__device__ __forceinline__ void w4_rows(const W4Args& s, const Tile& t, float* lds) {
  constexpr int NG = kTurn / G;  // groups of a turn
  constexpr int kPer = ACT ? kCols / 2 : kCols;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int groups = s.K / G;
  const int n0 = blockIdx.x * kPer;
  const int stages = (s.K + kTurn * kWaves * U - 1) / (kTurn * kWaves * U);
  const T* x[MB];
#pragma unroll
  for (int m = 0; m < MB; ++m)
    x[m] = (const T*)s.x + (int64_t)max(w4_row(s, t.row0 + min(16 * m + r, t.n - 1)), 0) * s.ldx + 8 * q;
  const uint4 ones = {kOnes<T>, kOnes<T>, kOnes<T>, kOnes<T>};
  const typename Vec8<T>::type one8 = __builtin_bit_cast(typename Vec8<T>::type, ones);

  struct Stage {
    uint4 c[U][2], x[U][MB][4];
    typename Halves<NG>::type s[U][2], m[U][2];
  };
  const uint8_t* codes[2];
  const f16 *scales[2], *mins[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int64_t row =
        (int64_t)t.e * (ACT ? 2 : 1) * s.N +
        (ACT ? (int64_t)b * s.N + min(n0 + r, s.N - 1) : min(n0 + 16 * b + r, s.N - 1));
    codes[b] = s.codes + row * (s.K / 2);
    scales[b] = s.scales + row * groups;
    mins[b] = s.mins + row * groups;
  }
  // Turn u of stage st starts at input ((st U + u) kWaves + wave) kTurn.  Past
  // the end x is 0, and codes and groups are the row's last ones.
  auto load = [&](int st, Stage& v) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = ((st * U + u) * kWaves + wv) * kTurn;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        v.c[u][b] = *reinterpret_cast<const uint4*>(codes[b] + min(k + 32 * q, s.K - 32) / 2);
        if (k + kTurn <= s.K) {
          v.s[u][b] = load_halves<NG>(scales[b] + k / G);
          if (s.mins) v.m[u][b] = load_halves<NG>(mins[b] + k / G);
        } else {
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const int at = min(k / G + g, groups - 1);
            v.s[u][b][g] = scales[b][at];
            if (s.mins) v.m[u][b][g] = mins[b][at];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in = k + 32 * i < s.K;
#pragma unroll
        for (int m = 0; m < MB; ++m) {
          v.x[u][m][i] = uint4{0, 0, 0, 0};
          if (in) v.x[u][m][i] = load_x8(x[m] + k + 32 * i);
        }
      }
    }
  };
  f32x4 acc[MB][2] = {};
  auto add = [&](const Stage& v) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t d[2][4];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        d[b][0] = v.c[u][b].x, d[b][1] = v.c[u][b].y, d[b][2] = v.c[u][b].z, d[b][3] = v.c[u][b].w;
        transpose4(d[b]);
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        f32x4 sum[MB][2] = {}, sx[MB] = {};
#pragma unroll
        for (int i = 0; i < 4 / NG; ++i) {
          const int st = g * (4 / NG) + i;
          typename Vec8<T>::type w[2];
#pragma unroll
          for (int b = 0; b < 2; ++b) w[b] = codes8<T>(d[b][st]);
#pragma unroll
          for (int m = 0; m < MB; ++m) {
            const typename Vec8<T>::type xv = order8<T>(v.x[u][m][st]);
            sx[m] = mfma16(xv, one8, sx[m]);
#pragma unroll
            for (int b = 0; b < 2; ++b) sum[m][b] = mfma16(xv, w[b], sum[m][b]);
          }
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const float sc = (float)v.s[u][b][g];
          const float mn = s.mins ? (float)v.m[u][b][g] : -8.f * sc;
#pragma unroll
          for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[m][b][j] = fmaf(sc, sum[m][b][j], fmaf(mn, sx[m][j], acc[m][b][j]));
        }
      }
    }
  };
  Stage va, vb;
  load(0, va);
  for (int i = 0; i < stages; i += 2) {
    if (i + 1 < stages) load(i + 1, vb);
    add(va);
    if (i + 1 == stages) break;
    if (i + 2 < stages) load(i + 2, va);
    add(vb);
  }

  // tile i of the MB x 2 (with the activation: of the MB pairs)
  auto put = [&](int m, int b, const f32x4& g, const f32x4& u) {
    const int n = n0 + (ACT ? 0 : 16 * b) + r;
    if (n >= s.N) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = 16 * m + 4 * q + j;
      if (row < t.n) w4_store<T, O, ACT>(s, t.e, t.row0 + row, n, g[j], u[j]);
    }
  };
  // the four waves' sums, [wave][tile of 16 x 16][lane]
  f32x4* sums = (f32x4*)lds;
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int b = 0; b < 2; ++b) sums[(wv * MB * 2 + m * 2 + b) * 64 + lane] = acc[m][b];
  __syncthreads();
  for (int i = wv; i < (ACT ? MB : MB * 2); i += kWaves) {
    f32x4 v[2];
#pragma unroll
    for (int b = 0; b < (ACT ? 2 : 1); ++b) {
      const int at = ACT ? i * 2 + b : i;
      v[b] = sums[at * 64 + lane];
#pragma unroll
      for (int o = 1; o < kWaves; ++o) {
        const f32x4 p = sums[(o * MB * 2 + at) * 64 + lane];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[b][j] += p[j];
      }
    }
    put(ACT ? i : i >> 1, i & 1, v[0], v[1]);
  }
}

// The row tiles are the grid's y, in layers of kTilesY (what a grid takes).
constexpr int kTilesY = 65535;
__device__ __forceinline__ Tile w4_tile(const W4Args& s, int rows) {
  const int tile = blockIdx.z * kTilesY + blockIdx.y;
  if (s.bounds) return find_tile(s.bounds, s.E, s.R, tile, rows);
  const int row0 = tile * rows;
  return Tile{0, row0, min(rows, s.R - row0)};
}

template <class T, class O, int G, bool ACT>
__global__ __launch_bounds__(64 * kWaves, 2) void k_w4_mm(W4Args s) {
  __shared__ __align__(16) float lds[kWaves * 4 * 64 * 4];
  const Tile t = w4_tile(s, kRows);
  if (t.n <= 0) return;
  if (t.n <= 16)
    w4_rows<T, O, G, ACT, 1, 2>(s, t, lds);
  else
    w4_rows<T, O, G, ACT, 2, 1>(s, t, lds);
}

// ---------------------------------------------------------- one or two rows
// A wave takes 8 rows of the weights (with the activation 4 of the gate and
// the same 4 of the up half) and all their inputs: 32 inputs of one row per
// lane and 16-byte load, `lanes` lanes per row (64 from 1024 inputs on), so
// that 64 / lanes rows are read by one load; four loads' codes are in use
// while the next four are in flight.  x lies in LDS, in the codes' order and
// so that a read is contiguous over the lanes, with its sums per 32 inputs
// (which lie in one group), and two products are added per v_dot2.  The
// decode of 8 codes is 7 instructions however few rows there are, and here
// nothing but one sum per row is exchanged between lanes.  One row of each of
// 128 experts (1536 x 2048, groups of 128): 58 us, 3.7 TB/s over weights that
// no cache holds, 52 us over the same ones at each call; one row of 4096 x
// 2048: 5.4 us, a chain of latencies.  (On the matrix cores the latter took
// 1.4 us more.)
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c, f16) {
  typedef __attribute__((ext_vector_type(2))) _Float16 h2;
  return __builtin_amdgcn_fdot2(__builtin_bit_cast(h2, a), __builtin_bit_cast(h2, b), c, false);
}
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c, bf16) {
  typedef __attribute__((ext_vector_type(2))) __bf16 h2;
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(h2, a), __builtin_bit_cast(h2, b), c, false);
}

template <int kCtrl>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                           0, __builtin_bit_cast(int, v), kCtrl, 0xF, 0xF, false));
}
// sum over runs of `lanes` lanes (8, 16, 32 or 64), in every lane
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  typedef __attribute__((ext_vector_type(2))) uint32_t u2;
  v = dpp_add<0xB1>(v);   // quad_perm [1,0,3,2]
  v = dpp_add<0x4E>(v);   // quad_perm [2,3,0,1]
  v = dpp_add<0x141>(v);  // row_half_mirror
  if (lanes >= 16) v = dpp_add<0x140>(v);  // row_mirror
  if (lanes >= 32) {
    const uint32_t u = __float_as_uint(v);
    const u2 t = __builtin_bit_cast(u2, __builtin_amdgcn_permlane16_swap(u, u, false, false));
    v = __uint_as_float(t[0]) + __uint_as_float(t[1]);
  }
  if (lanes >= 64) {
    const uint32_t u = __float_as_uint(v);
    const u2 t = __builtin_bit_cast(u2, __builtin_amdgcn_permlane32_swap(u, u, false, false));
    v = __uint_as_float(t[0]) + __uint_as_float(t[1]);
  }
  return v;
}

constexpr int kVecRows = 2;  // rows of x the vector path takes
constexpr int kOuts = 8;     // rows of the weights per wave
constexpr int kBatch = 4;    // loads whose rows are summed together
constexpr int kVecInputs = 16384;  // rows x inputs of x that the LDS holds
constexpr int kVecLds = kVecInputs * 2 + kVecInputs / 32 * 4 + kWaves * kOuts * kVecRows * 4;

template <class T, class O, bool ACT, int M, bool kWide>
__device__ __forceinline__ void w4_vec(const W4Args& s, const Tile& t, uint8_t* lds) {
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int log_lanes = kWide ? 6 : s.K <= 256 ? 3 : s.K <= 512 ? 4 : 5;
  const int lanes = 1 << log_lanes, sub = 64 >> log_lanes;  // lanes per row, rows per load
  // (kWide: a load's row is the wave's, and its address a scalar)
  const int at = kWide ? lane : lane & (lanes - 1), which = kWide ? 0 : lane >> log_lanes;
  const int chunks = (s.K + 32 * lanes - 1) >> (5 + log_lanes);
  constexpr int kN = ACT ? kOuts / 2 : kOuts;
  const int n0 = (blockIdx.x * kWaves + wv) * kN;
  const int groups = s.K / s.G;
  uint4* xs = (uint4*)lds;                                   // [m][chunk][piece][lane]
  float* sums = (float*)(lds + kVecInputs * 2);              // [m][chunk][lane]
  float* mine = (float*)(lds + kVecInputs * 2 + kVecInputs / 32 * 4) + wv * kOuts * M;

  // the wave's rows, clamped to the last one
  const int64_t first = (int64_t)t.e * (ACT ? 2 : 1) * s.N + min(n0, s.N - 1);
  const int most = max(s.N - 1 - n0, 0);
  const uint8_t* codes = s.codes + first * (s.K / 2);
  const uint8_t* codes_up = codes + (int64_t)s.N * (s.K / 2);
  const f16* scales = s.scales + first * groups;
  const f16* scales_up = scales + (int64_t)s.N * groups;
  const f16* mins = s.mins + first * groups;
  const f16* mins_up = mins + (int64_t)s.N * groups;
  const int log_g = s.G == 32 ? 5 : s.G == 64 ? 6 : 7;
  struct Loads {
    uint4 c[kBatch];
    f16 s[kBatch], m[kBatch];
  };
  auto load = [&](int batch, int chunk, Loads& l) {
    const int k = 32 * ((chunk << log_lanes) + at);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int j = (batch * kBatch + i) * sub + which;
      l.c[i] = uint4{0, 0, 0, 0};
      l.s[i] = l.m[i] = (f16)0.f;
      if (j < kOuts && k < s.K) {
        // (the rows of a wave lie within 2^22 bytes and 2^18 groups)
        const int wr = min(ACT ? j & 3 : j, most);
        const bool up = ACT && (j & 4);
        const int g = wr * groups + (k >> log_g);
        l.c[i] = *reinterpret_cast<const uint4*>((up ? codes_up : codes) + wr * (s.K / 2) + k / 2);
        l.s[i] = (up ? scales_up : scales)[g];
        if (s.mins) l.m[i] = (up ? mins_up : mins)[g];
      }
    }
  };
  Loads now, next;
  load(0, 0, now);

  // x into LDS, 0 past its end; 8 inputs a thread, a lane's 32 in 4 neighbours
  const int pieces = chunks << (log_lanes + 2);
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const T* x = (const T*)s.x + (int64_t)max(w4_row(s, t.row0 + min(m, t.n - 1)), 0) * s.ldx;
    for (int p = tid; p < pieces; p += 64 * kWaves) {
      uint4 v = uint4{0, 0, 0, 0};
      if (8 * p < s.K) v = load_x8(x + 8 * p);
      const uint4 o = __builtin_bit_cast(uint4, order8<T>(v));
      const int a = (p >> 2) & (lanes - 1), c = p >> (log_lanes + 2);
      xs[(((m * chunks + c) * 4 + (p & 3)) << log_lanes) + a] = o;
      float f = dot2(o.x, kOnes<T>, 0.f, T{});
      f = dot2(o.y, kOnes<T>, f, T{});
      f = dot2(o.z, kOnes<T>, f, T{});
      f = dot2(o.w, kOnes<T>, f, T{});
      f = dpp_add<0x4E>(dpp_add<0xB1>(f));  // the four neighbours' sum
      if ((p & 3) == 0) sums[((m * chunks + c) << log_lanes) + a] = f;
    }
  }
  __syncthreads();

  const int batches = (kOuts + sub * kBatch - 1) / (sub * kBatch);
  float acc[kBatch][M];
  for (int batch = 0, chunk = 0; batch < batches;) {
    const bool last = chunk + 1 == chunks;
    const int nb = last ? batch + 1 : batch, nc = last ? 0 : chunk + 1;
    if (nb < batches) load(nb, nc, next);
    if (chunk == 0) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
#pragma unroll
        for (int m = 0; m < M; ++m) acc[i][m] = 0.f;
    }
    float d[kBatch][M] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint4 v[M];
#pragma unroll
      for (int m = 0; m < M; ++m) v[m] = xs[(((m * chunks + chunk) * 4 + j) << log_lanes) + at];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const uint32_t w = j == 0 ? now.c[i].x : j == 1 ? now.c[i].y : j == 2 ? now.c[i].z : now.c[i].w;
        const uint4 c = __builtin_bit_cast(uint4, codes8<T>(w));
#pragma unroll
        for (int m = 0; m < M; ++m) {
          d[i][m] = dot2(c.x, v[m].x, d[i][m], T{});
          d[i][m] = dot2(c.y, v[m].y, d[i][m], T{});
          d[i][m] = dot2(c.z, v[m].z, d[i][m], T{});
          d[i][m] = dot2(c.w, v[m].w, d[i][m], T{});
        }
      }
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const float sx = sums[((m * chunks + chunk) << log_lanes) + at];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float sc = (float)now.s[i];
        const float mn = s.mins ? (float)now.m[i] : -8.f * sc;
        acc[i][m] = fmaf(sc, d[i][m], fmaf(mn, sx, acc[i][m]));
      }
    }
    if (last) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int j = (batch * kBatch + i) * sub + which;
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const float v = lanes_sum(acc[i][m], lanes);
          if (at == 0 && j < kOuts) mine[j * M + m] = v;
        }
      }
    }
    now = next;
    batch = nb, chunk = nc;
  }
  __syncthreads();
  static_assert(kOuts * kVecRows <= 64, "an output per lane");
  if (lane < kN * M) {
    const int j = lane / M, m = lane % M;
    if (m < t.n && n0 + j < s.N)
      w4_store<T, O, ACT>(s, t.e, t.row0 + m, n0 + j, mine[j * M + m],
                          ACT ? mine[(j + kN) * M + m] : 0.f);
  }
}

// Up to 16 rows of an expert: by v_dot2 or on the matrix cores.
constexpr int kFewRows = 16;
template <class T, class O, int G, bool ACT>
__global__ __launch_bounds__(64 * kWaves, 3) void k_w4_few(W4Args s) {
  __shared__ __align__(16) uint8_t lds[kVecLds];
  static_assert(kVecLds >= kWaves * 2 * 64 * 16, "sums of the waves");
  const Tile t = w4_tile(s, kFewRows);
  if (t.n <= 0) return;
  // (x of the tile in LDS, in whole turns of 64 lanes x 32 inputs)
  const bool vec = t.n <= kVecRows && t.n * ((s.K + 2047) & ~2047) <= kVecInputs;
  const bool wide = s.K > 1024;
  if (vec && t.n == 1 && wide)
    w4_vec<T, O, ACT, 1, true>(s, t, lds);
  else if (vec && t.n == 1)
    w4_vec<T, O, ACT, 1, false>(s, t, lds);
  else if (vec && wide)
    w4_vec<T, O, ACT, 2, true>(s, t, lds);
  else if (vec)
    w4_vec<T, O, ACT, 2, false>(s, t, lds);
  else
    w4_rows<T, O, G, ACT, 1, 1>(s, t, (float*)lds);
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
  if (rows ? (div < 1 || x_rows < (R > 0)) : x_rows < R)
    return fail(BITSMOE_ESHAPE, "div=%d, %d rows of x for R=%d", div, x_rows, R);
  if (ldx < K || ldy < N) return fail(BITSMOE_ESHAPE, "a row stride is too small");
  if (R == 0) return BITSMOE_OK;
  if (!codes || !scales || !y || (x_rows && !x)) return fail(BITSMOE_EINVAL, "null pointer argument");
  if (((uintptr_t)codes & 15u) || ((uintptr_t)scales & 3u) || ((uintptr_t)mins & 3u))
    return fail(BITSMOE_EINVAL, "codes must be 16-byte aligned, scales and mins 4-byte aligned");
  W4Args s{x, ldx, rows, div, x_rows, (const uint8_t*)codes, (const f16*)scales, (const f16*)mins,
           bounds, R, E, N, K, G, y, ldy, act};
  const hipStream_t st = (hipStream_t)stream;
  const bool few = R <= (long long)kFewRows * E;
  const int rows_tile = few ? kFewRows : kRows;
  if (!countable(R, E, rows_tile)) return fail(BITSMOE_ESHAPE, "R=%d with E=%d", R, E);
  const long long tiles =
      bounds ? max_tiles(R, E, rows_tile) : ((long long)R + rows_tile - 1) / rows_tile;
  const int per = act ? kCols / 2 : kCols;
  const dim3 grid((unsigned)((N + per - 1) / per), (unsigned)(tiles < kTilesY ? tiles : kTilesY),
                  (unsigned)((tiles + kTilesY - 1) / kTilesY));
  auto go = [&](auto t, auto o) {
    using T = decltype(t);
    using O = decltype(o);
    const dim3 block(64 * kWaves);
    auto rows_of = [&](auto g) {
      constexpr int kG = decltype(g)::value;
      if (few && act)
        hipLaunchKernelGGL((k_w4_few<T, O, kG, true>), grid, block, 0, st, s);
      else if (few)
        hipLaunchKernelGGL((k_w4_few<T, O, kG, false>), grid, block, 0, st, s);
      else if (act)
        hipLaunchKernelGGL((k_w4_mm<T, O, kG, true>), grid, block, 0, st, s);
      else
        hipLaunchKernelGGL((k_w4_mm<T, O, kG, false>), grid, block, 0, st, s);
    };
    if (G == 32)
      rows_of(std::integral_constant<int, 32>{});
    else if (G == 64)
      rows_of(std::integral_constant<int, 64>{});
    else
      rows_of(std::integral_constant<int, 128>{});
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
