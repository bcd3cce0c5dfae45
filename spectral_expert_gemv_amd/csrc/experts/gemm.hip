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

// -------------------------------------------------------- tiled, 16-byte rows
// Work-group tile of TM output rows x TN output columns, WM x WN waves, the
// contraction in steps of 64.  Every step's two operand tiles are copied
// straight into LDS by 16-byte loads (no registers in between) into one of
// two buffers, a step ahead of the products.
//
// An operand whose rows run along the contraction lies in LDS as
// [row][64 elements]: 16-byte piece p of row r at place p ^ (r / 2 % 8), so
// that the 16 rows a matrix-core read touches spread over all 64 banks.  The
// others (the weights of dx, both operands of dw) lie as
// [contraction][columns] and are read with the transposing LDS load, which
// hands lane i of 16 column i of a 4 x 16 block: 32-byte unit u of line c at
// place u ^ key(c), with the eight lines that 32 lanes read at different
// places.

// 16 bytes past the ends of an operand: 0, or NaN for a row outside x
__device__ __align__(16) const uint32_t g_pad[8] = {0,           0,           0,           0,
                                                    0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu};

// Copies 16 bytes per lane from `src` to LDS at lds + 16 lane.  (The
// compiler would wait for all such copies before any LDS read, so the copy is
// an opaque statement without register outputs; the loop below waits for its
// copies by count.)
__device__ __forceinline__ void copy16(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :
               : "v"(src), "s"(lds)
               : "memory");
}
__device__ __forceinline__ void wait_copies() { __builtin_amdgcn_s_waitcnt(0x0F70); }  // vmcnt(0)
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

constexpr int kStep = 64;  // contraction elements per step

typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(8))) short s16x8;

// One operand's tile: B rows (or columns) of 64 elements of the contraction.
// kTr: the contraction is the slow axis.  The lanes of NT threads hold the
// global addresses of the pieces they copy each step.
template <int B, bool kTr, int NT>
struct Operand {
  static constexpr int kCopies = B * kStep * 2 / 16 / NT;
  static constexpr int kBytes = B * kStep * 2;
  const uint8_t* ptr[kCopies];
  int step[kCopies];  // bytes per step (kTr: unused)

  // place of a lane's piece in copy i: line of the tile, and the 16-byte
  // piece of that line it has to fetch
  static __device__ __forceinline__ int line(int i) {
    const int at = i * NT + threadIdx.x;
    return kTr ? at / (B / 8) : at / 8;
  }
  static __device__ __forceinline__ int key(int l) {
    return kTr ? (l & 3) | ((l >> 1) & 4) : (l >> 1) & 7;
  }
  static __device__ __forceinline__ int piece(int i) {
    const int at = i * NT + threadIdx.x;
    if (kTr) {
      const int p = at % (B / 8), l = at / (B / 8);
      return (((p >> 1) ^ key(l)) << 1) | (p & 1);
    }
    return (at % 8) ^ key(at / 8);
  }
  // LDS byte offset of the wave's piece run of copy i
  static __device__ __forceinline__ uint32_t dest(uint32_t base, int i) {
    return base + (uint32_t)__builtin_amdgcn_readfirstlane((i * NT + (threadIdx.x & ~63)) * 16);
  }

  // 8 consecutive contraction elements (32 s + 8 (lane / 16) ..) of row or
  // column r + lane % 16
  template <class T>
  static __device__ __forceinline__ typename Vec8<T>::type frag(uint32_t base, int r, int s) {
    const int lane = threadIdx.x & 63;
    if constexpr (kTr) {
      typedef __attribute__((address_space(3))) s16x4 lds_s4;
      const int g = lane >> 4, i = lane & 15;
      s16x8 v;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = 32 * s + 8 * g + 4 * h + (i >> 2);
        const int unit = (r >> 4) ^ key(c);
        const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s4*)(uintptr_t)(base + c * (B * 2) + unit * 32 + (i & 3) * 8));
        v[4 * h] = t[0], v[4 * h + 1] = t[1], v[4 * h + 2] = t[2], v[4 * h + 3] = t[3];
      }
      return __builtin_bit_cast(typename Vec8<T>::type, v);
    } else {
      const int row = r + (lane & 15), p = 4 * s + (lane >> 4);
      typedef __attribute__((address_space(3))) const s16x8 lds_s8;
      return __builtin_bit_cast(typename Vec8<T>::type,
                                *(lds_s8*)(uintptr_t)(base + row * (kStep * 2) +
                                                      ((p ^ key(row)) << 4)));
    }
  }
};

template <class T, class O, int MODE, int TM, int TN, int WM, int WN, bool ACT>
__global__ __launch_bounds__(64 * WM* WN) void k_mm_tile(MmArgs s, int mtiles_cap) {
  constexpr int NT = 64 * WM * WN;
  constexpr int MI = TM / WM / 16, NI = TN / WN / 16;  // 16 x 16 tiles of a wave
  constexpr bool kTrA = MODE == kDw, kTrB = MODE != kFwd;
  typedef Operand<TM, kTrA, NT> OpA;
  typedef Operand<TN, kTrB, NT> OpB;
  constexpr uint32_t kBuf = OpA::kBytes + OpB::kBytes;
  __shared__ __align__(128) uint8_t lds[2 * kBuf];
  const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;

  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int cols = MODE == kFwd ? s.N : s.K;  // output columns
  constexpr int kCols = ACT ? TN / 2 : TN;    // of them per tile
  const int ntn = (cols + kCols - 1) / kCols;
  int e, m0, mn, c0, cn, nt;
  if (MODE == kDw) {
    const int ntm = (s.N + TM - 1) / TM;
    const int per = ntm * ntn;
    int b = blockIdx.x;
    e = b / per;
    b -= e * per;
    m0 = (b / ntn) * TM, mn = min(TM, s.N - m0), nt = b % ntn;
    int hi;
    expert_rows(s.bounds, e, s.R, c0, hi);
    cn = hi - c0;
  } else {
    const Tile t = find_tile(s.bounds, s.E, s.R, blockIdx.x % mtiles_cap, TM);
    if (t.n == 0) return;
    nt = blockIdx.x / mtiles_cap;
    e = t.e, m0 = t.row0, mn = t.n;
    c0 = 0, cn = MODE == kFwd ? s.K : s.N;
  }
  const int n0 = nt * kCols, nn = min(kCols, cols - n0);

  // addresses of the pieces of step 0
  OpA a;
  OpB b;
  const uint8_t* A = (const uint8_t*)s.a;
  const uint8_t* Bp = (const uint8_t*)s.b;
  if (MODE != kDw) Bp += (size_t)e * (ACT ? 2 : 1) * s.N * s.K * 2;
  const int64_t lda = s.lda * 2, ldb = MODE == kDw ? s.ldb * 2 : (int64_t)s.K * 2;
#pragma unroll
  for (int i = 0; i < OpA::kCopies; ++i) {
    const int l = OpA::line(i), p = OpA::piece(i);
    a.step[i] = kStep * 2;
    if (kTrA) {
      a.ptr[i] = A + (int64_t)(c0 + l) * lda + (int64_t)(m0 + min(8 * p, mn - 8)) * 2;
    } else {
      const int row = m0 + min(l, mn - 1);
      const int xr = MODE == kFwd ? x_row(s, row) : row;
      a.ptr[i] = A + (int64_t)xr * lda + p * 16;
      if (xr < 0) a.ptr[i] = (const uint8_t*)(g_pad + 4), a.step[i] = 0;
    }
  }
#pragma unroll
  for (int i = 0; i < OpB::kCopies; ++i) {
    const int l = OpB::line(i), p = OpB::piece(i);
    if (MODE == kFwd) {
      // with the activation, blocks of 16 tile rows alternate gate and up
      const int col = ACT ? (l >> 5) * 16 + (l & 15) : l;
      const int64_t row = n0 + min(col, nn - 1) + (ACT && (l & 16) ? s.N : 0);
      b.ptr[i] = Bp + row * ldb + p * 16;
    } else {
      b.ptr[i] = Bp + (int64_t)(MODE == kDw ? 0 : l) * ldb + (int64_t)(n0 + min(8 * p, nn - 8)) * 2;
    }
  }
  // dw: rows of x of the next step (-1: outside x)
  int xr[MODE == kDw ? OpB::kCopies : 1];
  auto fetch_rows = [&](int c) {
#pragma unroll
    for (int i = 0; i < (MODE == kDw ? OpB::kCopies : 1); ++i)
      xr[i] = c + OpB::line(i) < cn ? x_row(s, c0 + c + OpB::line(i)) : 0;
  };
  if (MODE == kDw) fetch_rows(0);

  // copies of the step at contraction index c into the buffer at `buf`;
  // pieces past the end of the contraction are 0
  auto stage = [&](int c, uint32_t buf) {
    const bool whole = c + kStep <= cn;
#pragma unroll
    for (int i = 0; i < OpA::kCopies; ++i) {
      const uint8_t* p = a.ptr[i];
      if (!whole && c + (kTrA ? OpA::line(i) : 8 * OpA::piece(i)) >= cn) p = (const uint8_t*)g_pad;
      copy16(p, OpA::dest(buf, i));
      a.ptr[i] += kTrA ? (int64_t)kStep * lda : (int64_t)a.step[i];
    }
#pragma unroll
    for (int i = 0; i < OpB::kCopies; ++i) {
      const uint8_t* p = b.ptr[i];
      if (MODE == kDw) {
        p = xr[i] < 0 ? (const uint8_t*)(g_pad + 4) : p + (int64_t)xr[i] * ldb;
      }
      if (!whole && c + (kTrB ? OpB::line(i) : 8 * OpB::piece(i)) >= cn) p = (const uint8_t*)g_pad;
      copy16(p, OpB::dest(buf + OpA::kBytes, i));
      if (MODE == kFwd) b.ptr[i] += kStep * 2;
      if (MODE == kDx) b.ptr[i] += (int64_t)kStep * ldb;
    }
  };

  const int wm = (wv / WN) * (TM / WM), wn = (wv % WN) * (TN / WN);
  f32x4 acc[MI][NI] = {};
  uint32_t cur = base;
  if (cn > 0) stage(0, cur);
  for (int c = 0; c < cn; c += kStep) {
    if (MODE == kDw && c + kStep < cn) fetch_rows(c + kStep);
    wait_copies();
    lds_barrier();  // this step's copies are in, and nobody reads the other buffer any more
    const uint32_t next = base + (cur == base ? kBuf : 0u);
    if (c + kStep < cn) stage(c + kStep, next);
#pragma unroll
    for (int k = 0; k < kStep / 32; ++k) {
      typename Vec8<T>::type fa[MI], fb[NI];
#pragma unroll
      for (int j = 0; j < NI; ++j)
        fb[j] = OpB::template frag<T>(cur + OpA::kBytes, wn + 16 * j, k);
#pragma unroll
      for (int i = 0; i < MI; ++i) fa[i] = OpA::template frag<T>(cur, wm + 16 * i, k);
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = mfma16(fb[j], fa[i], acc[i][j]);
    }
    cur = next;
  }

  // the products were formed transposed: lane % 16 is the output row, and a
  // lane holds 4 consecutive columns 4 (lane / 16) .. of each 16 x 16 tile
  O* Y = (O*)s.y;
  const int64_t ldy = MODE == kDw ? s.K : s.ldy;
  if (MODE == kDw) Y += (size_t)e * s.N * s.K;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int m = wm + 16 * i + (lane & 15);
    if (m >= mn) continue;
    O* row = Y + (int64_t)(m0 + m) * ldy + n0;
#pragma unroll
    for (int j = 0; j < NI; j += ACT ? 2 : 1) {
      const int n = (ACT ? (wn + 16 * j) / 2 : wn + 16 * j) + 4 * (lane >> 4);
      f32x4 v = acc[i][j];
      if constexpr (ACT) {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = gated(v[q], acc[i][j + 1][q]);
      }
      if (n + 4 <= nn) {  // (columns are a multiple of 8, rows 16-byte aligned)
        typedef __attribute__((ext_vector_type(4))) O O4;
        O4 o;
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = (O)v[q];
        *reinterpret_cast<O4*>(row + n) = o;
      }
    }
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

bool rows16(const void* p, int64_t ld) { return ((uintptr_t)p & 15u) == 0 && ld % 8 == 0; }

// The tiled kernel serves rows of whole 16-byte pieces.
bool tiled(const MmArgs& s, int mode, int o_dtype) {
  return s.N % 8 == 0 && s.K % 8 == 0 && rows16(s.a, s.lda) &&
         rows16(s.b, mode == kDw ? s.ldb : s.K) && rows16(s.y, mode == kDw ? s.K : s.ldy);
}

template <int MODE>
int launch_mm(const MmArgs& s, int dtype, int o_dtype, hipStream_t st) {
  if (!tiled(s, MODE, o_dtype)) return launch_any<MODE>(s, dtype, o_dtype, st);
  int rc = BITSMOE_OK;
  with_types(dtype, o_dtype, [&](auto t, auto o) {
    using T = decltype(t);
    using O = decltype(o);
    constexpr int TM = 256, TN = 256, WM = 2, WN = 4;
    const int cols = MODE == kFwd ? s.N : s.K, per = s.act ? TN / 2 : TN;
    const long long ntn = (cols + per - 1) / per;
    const long long mt = MODE == kDw ? (long long)s.E * ((s.N + TM - 1) / TM) : max_tiles(s.R, s.E, TM);
    if (mt * ntn > 0x7FFFFFFFll) {
      rc = fail(BITSMOE_ESHAPE, "R=%d E=%d N=%d K=%d make too many tiles", s.R, s.E, s.N, s.K);
      return;
    }
    const dim3 grid((unsigned)(mt * ntn));
    if (MODE == kFwd && s.act)
      hipLaunchKernelGGL((k_mm_tile<T, O, MODE, TM, TN, WM, WN, MODE == kFwd>), grid,
                         dim3(64 * WM * WN), 0, st, s, (int)mt);
    else
      hipLaunchKernelGGL((k_mm_tile<T, O, MODE, TM, TN, WM, WN, false>), grid, dim3(64 * WM * WN),
                         0, st, s, (int)mt);
    rc = launched("grouped_matmul");
  });
  return rc;
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
  return launch_mm<kFwd>(s, dtype, y_dtype, (hipStream_t)stream);
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
  return launch_mm<kDx>(s, dtype, dx_dtype, (hipStream_t)stream);
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
  return launch_mm<kDw>(s, dtype, dw_dtype, (hipStream_t)stream);
}

}  // extern "C"
