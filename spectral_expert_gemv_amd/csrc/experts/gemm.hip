// Products grouped by expert, rows ragged: with rows i in [bounds[e],
// bounds[e + 1]) belonging to expert e,
//   forward  y_i  = W_e x_i          (optionally SiLU(gate) * up of it)
//   dx       dx_i = W_e^T dy_i
//   dw       dW_e = sum_i dy_i x_i^T
// fp16 or bf16 operands, float32 accumulators, one rounding at the end.
#include <type_traits>

#include "experts.h"

namespace bitsmoe {
namespace experts {
namespace {

enum { kFwd = 0, kDx = 1, kDw = 2 };

struct MmArgs {
  const void* a;   // forward: x; dx, dw: dy
  int64_t lda;
  const void* b;   // forward, dx: w; dw: x
  int64_t ldb;     // their row strides (w: of all experts' rows)
  const int32_t* rows;  // forward, dw: x row of sorted row i is rows[i] / div
  int div, x_rows;
  const int32_t* bounds;
  int R, E, N, K;  // W_e is (act ? 2 N : N) x K
  void* y;
  int64_t ldy;     // dw: K
  int act;
  int y16;         // rows of y are whole 16-byte pieces
};

// The row of x behind sorted row i; -1: an index outside x, whose products
// are NaN.
__device__ inline int x_row(const MmArgs& s, int i) {
  if (!s.rows) return i;
  const int p = s.rows[i];
  const int r = p < 0 ? -1 : p / s.div;
  return r < s.x_rows ? r : -1;
}

// Rows of `cols` elements of 2 bytes, at any stride and alignment, to rows of
// whole 16-byte pieces, 0 past the end: what the tiled kernel wants of an
// operand that is not like that.
__global__ __launch_bounds__(256) void k_mm_pad(const uint16_t* __restrict__ src, int64_t ld,
                                                int64_t rows, int cols, uint4* __restrict__ dst) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  typedef u4 loose __attribute__((aligned(2)));
  const int per = (cols + 7) / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * per;
       i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / per;
    const int c = (int)(i - r * per) * 8;
    const uint16_t* p = src + r * ld + c;
    u4 v = {0, 0, 0, 0};
    if (c + 8 <= cols) {
      v = *reinterpret_cast<const loose*>(p);
    } else {
      uint16_t e[8] = {};
      for (int j = 0; j < 8; ++j)
        if (c + j < cols) e[j] = p[j];
      __builtin_memcpy(&v, e, 16);
    }
    dst[i] = __builtin_bit_cast(uint4, v);
  }
}

// -------------------------------------------------------- tiled, 16-byte rows
// Work-group tile of TM output rows x TN output columns, WM x WN waves, the
// contraction in steps of 64 (whole 128-byte lines of a row).  Every step's two operand tiles are copied
// straight into LDS by 16-byte loads (no registers in between) into one of
// kBufs buffers, kBufs - 1 steps ahead of the products: 2 of the 256 x 256
// tile's 64 KB, 3 of the 256 x 128 tile's 48 KB, 4 of the 128 x 128 tile's
// 32 KB, whose steps are too short to hide one copy's latency.
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
// copies by count.  The LDS address is an operand in m0, so the compiler knows
// what it holds; the copy may not be the instruction after the one that sets it.)
__device__ __forceinline__ void copy16(const void* src, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(src), "{m0}"(lds) : "memory");
}
// all but the last kLeft copies of the wave have landed
template <int kLeft>
__device__ __forceinline__ void wait_copies() {
  static_assert(kLeft < 16, "vmcnt field");
  __builtin_amdgcn_s_waitcnt(0x0F70 | kLeft);
}
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
  static constexpr int kBytes = B * kStep * 2;
  static constexpr int kCopies = kBytes / 16 / NT;
  static_assert(kCopies * NT * 16 == kBytes, "whole copies");
  const uint8_t* ptr[kCopies];

  // place of a lane's piece in copy i: line of the tile, and the 16-byte
  // piece of that line it has to fetch
  static __device__ __forceinline__ int line(int i) {
    const int at = i * NT + threadIdx.x;
    return kTr ? at / (B / 8) : at / (kStep / 8);
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
    return (at % (kStep / 8)) ^ key(at / (kStep / 8));
  }
  // LDS address of the wave's piece run of copy i
  static __device__ __forceinline__ uint32_t dest(uint32_t base, int wv, int i) {
    return base + (uint32_t)(i * NT + wv * 64) * 16;
  }

  // A lane's offset in the tile for the matrix-core piece of rows (columns)
  // r0 .. r0 + 15, r0 a multiple of 16, and the piece itself, 16 g rows on: 8
  // consecutive contraction elements (8 (lane / 16) ..) of row or column
  // r0 + 16 g + lane % 16.  Both layouts' keys depend on the lane alone; in
  // the transposed one the block's index enters by xor.
  static __device__ __forceinline__ uint32_t lane_offset(int r0) {
    const int lane = threadIdx.x & 63;
    if (kTr) {
      const int i = lane & 15, c = 8 * (lane >> 4) + (i >> 2);
      return c * (B * 2) + (((r0 >> 4) ^ key(c)) << 5) + (i & 3) * 8;
    }
    const int l = lane & 15;
    return (r0 + l) * (kStep * 2) + (((lane >> 4) ^ key(l)) << 4);
  }
  // (half: which 32 of the step's contraction)
  template <class T>
  static __device__ __forceinline__ typename Vec8<T>::type frag(uint32_t at, int g, int half) {
    if constexpr (kTr) {
      typedef __attribute__((address_space(3))) s16x4 lds_s4;
      s16x8 v;
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // (contraction + 4 has the same key)
        const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s4*)(uintptr_t)((at ^ (g << 5)) + (h * 4 + half * 32) * (B * 2)));
        v[4 * h] = t[0], v[4 * h + 1] = t[1], v[4 * h + 2] = t[2], v[4 * h + 3] = t[3];
      }
      return __builtin_bit_cast(typename Vec8<T>::type, v);
    } else {
      typedef __attribute__((address_space(3))) const s16x8 lds_s8;
      return __builtin_bit_cast(typename Vec8<T>::type,
                                *(lds_s8*)(uintptr_t)((at ^ (half << 6)) + g * 16 * (kStep * 2)));
    }
  }
};

// Tile `id` of mt x nt in the order that keeps the 32 work-groups of an XCD on
// shared operand rows (in its L2): 4 row tiles by 8 column tiles, then the
// next columns.
__device__ __forceinline__ void tile_place(uint32_t id, int mt, int nt, int& m, int& n) {
  const uint32_t g = id / (4u * nt), r = id - g * (4u * nt);
  const uint32_t gm = min(4, mt - (int)g * 4);
  m = g * 4 + r % gm;
  n = r / gm;
}

constexpr int kTile = 256;                          // rows and columns of a tile
constexpr uint32_t kOutLds = 2 * 2 * kTile * kStep * 2;  // of the output on its way
constexpr uint32_t kLds = 3 * (kTile + kTile / 2) * kStep * 2;  // three buffers of a 256 x 128 tile

// Output rows m0 .. m0 + mn and columns n0 .. n0 + nn of expert e, with the
// contraction c0 .. c0 + cn.
template <class T, class O, int MODE, int TM, int TN, int WM, int WN, int kBufs, bool ACT>
__device__ __forceinline__ void mm_tile(const MmArgs& s, uint32_t base, int e, int m0, int mn,
                                        int n0, int nn, int c0, int cn) {
  constexpr int NT = 64 * WM * WN;
  constexpr int MI = TM / WM / 16, NI = TN / WN / 16;  // 16 x 16 tiles of a wave
  constexpr bool kTrA = MODE == kDw, kTrB = MODE != kFwd;
  typedef Operand<TM, kTrA, NT> OpA;
  typedef Operand<TN, kTrB, NT> OpB;
  constexpr uint32_t kBuf = OpA::kBytes + OpB::kBytes;
  static_assert(kBufs * kBuf <= kLds, "buffers");
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // addresses of the pieces of step 0
  OpA a;
  OpB b;
  const uint8_t* A = (const uint8_t*)s.a;
  const uint8_t* Bp = (const uint8_t*)s.b;
  const int64_t lda = s.lda * 2, ldb = s.ldb * 2;
  if (MODE != kDw) Bp += (int64_t)e * (ACT ? 2 : 1) * s.N * ldb;
  uint32_t nan_rows = 0;  // bit i: copy i's row of A lies outside x
#pragma unroll
  for (int i = 0; i < OpA::kCopies; ++i) {
    const int l = OpA::line(i), p = OpA::piece(i);
    if (kTrA) {
      a.ptr[i] = A + (int64_t)(c0 + l) * lda + (int64_t)(m0 + min(8 * p, ((mn + 7) & ~7) - 8)) * 2;
    } else {
      const int row = m0 + min(l, mn - 1);
      const int xr = MODE == kFwd ? x_row(s, row) : row;
      a.ptr[i] = A + (int64_t)xr * lda + p * 16;
      if (xr < 0) a.ptr[i] = (const uint8_t*)(g_pad + 4), nan_rows |= 1u << i;
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
      b.ptr[i] = Bp + (int64_t)(MODE == kDw ? 0 : l) * ldb + (int64_t)(n0 + min(8 * p, ((nn + 7) & ~7) - 8)) * 2;
    }
  }

  // The row of x in line l (of 64 lanes at most two lines) of a step of dw,
  // read through the scalar cache: a vector load would make its reader wait
  // for the copies in flight.
  auto dw_row = [&](int i, int c) -> int {
    constexpr int kPer = 64 / (TN / 8);  // lines of a wave's copy
    static_assert(MODE != kDw || kPer == 1 || kPer == 2 || kPer == 4, "lines per copy");
    const int l0 = (i * NT + wv * 64) / (TN / 8);
    const int l = OpB::line(i) - l0;
    int r = -1;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int at = c + l0 + u;
      int v = c0 + at;
      if (s.rows) {
        typedef __attribute__((address_space(4))) const int32_t cint;
        v = at < cn ? ((cint*)(uintptr_t)s.rows)[v] : -1;
        v = v < 0 ? -1 : v / s.div;
        v = v < s.x_rows ? v : -1;
      }
      if (l == u) r = v;
    }
    return r;
  };

  // Piece i of the copies of the step at contraction index c into the buffer
  // at `buf` (A's pieces first).  Pieces past the end of the contraction are
  // 0, and so are steps past it.
  auto stage_piece = [&](int i, int c, bool whole, uint32_t buf) {
    if (i < OpA::kCopies) {
      const uint8_t* p = a.ptr[i];
      if (!whole && c + (kTrA ? OpA::line(i) : 8 * OpA::piece(i)) >= cn) p = (const uint8_t*)g_pad;
      // (rows past the tile's need not be copied: nobody uses what lies there;
      // with more than two buffers the copies in flight are counted, though)
      if (kTrA || whole || kBufs > 2 || i * (NT / 8) < mn) copy16(p, OpA::dest(buf, wv, i));
      if (kTrA)
        a.ptr[i] += (int64_t)kStep * lda;
      else
        a.ptr[i] += (nan_rows >> i) & 1 ? 0 : kStep * 2;
    } else {
      i -= OpA::kCopies;
      const uint8_t* p = b.ptr[i];
      if (MODE == kDw) {
        const int r = dw_row(i, c);
        p = r < 0 ? (const uint8_t*)(g_pad + 4) : p + (int64_t)r * ldb;
      }
      if (!whole && c + (kTrB ? OpB::line(i) : 8 * OpB::piece(i)) >= cn) p = (const uint8_t*)g_pad;
      copy16(p, OpB::dest(buf + OpA::kBytes, wv, i));
      if (MODE == kFwd) b.ptr[i] += kStep * 2;
      if (MODE == kDx) b.ptr[i] += (int64_t)kStep * ldb;
    }
  };
  constexpr int kPieces = OpA::kCopies + OpB::kCopies;
  // A step is two halves of MI groups of NI products with one A piece; the LDS reads run
  // kAhead groups before the products, across the steps' border.  There (group
  // kSwitch) the wave waits for its copies of the next step, meets the
  // others, and starts to copy a later step into the buffer that nobody reads
  // any more; the last groups' products run meanwhile.
  constexpr int kAhead = 3, kGroups = kStep / 32 * MI, kSwitch = kGroups - kAhead;
  static_assert(MI % (kAhead + 1) == 0 && kStep == 64, "turns of the registers");
  typedef typename Vec8<T>::type Frag;
  const int wm = (wv / WN) * (TM / WM), wn = (wv % WN) * (TN / WN);
  // (buffers start at multiples of 1024 bytes, so adding one keeps the xor)
  const uint32_t off_a = OpA::lane_offset(wm), off_b = OpA::kBytes + OpB::lane_offset(wn);
  f32x4 acc[MI][NI] = {};
  Frag fa[kAhead + 1], fb[2][NI];
  auto read_a = [&](int g, uint32_t at) {  // (at: the lane's own address)
    fa[g % (kAhead + 1)] = OpA::template frag<T>(at, g % MI, g / MI);
  };
  // B pieces of one half of a step, the first of them or the others
  auto read_b = [&](int half, int part, uint32_t at) {
#pragma unroll
    for (int j = 0; j < NI; ++j)
      if (j * 2 / NI == part) fb[half][j] = OpB::template frag<T>(at, j, half);
  };
  uint32_t cur = base, at_a = base + off_a, at_b = base + off_b;
  auto after = [&](uint32_t b) { return b == base + (kBufs - 1) * kBuf ? base : b + kBuf; };
  // kind 0: the step copied meanwhile is whole; 1: it may not be; 2: there is
  // no next step
  auto step = [&](int c, auto kind_) {
    constexpr int kKind = decltype(kind_)::value;
    constexpr bool kLast = kKind == 2;
    const uint32_t nxt = after(cur);
    uint32_t next_a = nxt + off_a, next_b = nxt + off_b;
    asm("" : "+v"(next_a), "+v"(next_b));  // one register and immediate offsets each
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      if (!kLast && g == kSwitch) {
        wait_copies<(kBufs - 2) * kPieces>();
        lds_barrier();
      }
      if (!kLast || g + kAhead < kGroups) {
        const int ahead = (g + kAhead) % kGroups;
        const bool here = g + kAhead < kGroups;
        if (ahead % MI == 0) read_b(ahead / MI, 0, here ? at_b : next_b);
        read_a(ahead, here ? at_a : next_a);
        if (ahead % MI == 1) read_b(ahead / MI, 1, here ? at_b : next_b);
      }
      if (!kLast && g >= kSwitch) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          if (i * kAhead / kPieces == g - kSwitch)
            stage_piece(i, c + kBufs * kStep, kKind == 0, cur);
      }
#pragma unroll
      for (int j = 0; j < NI; ++j)
        acc[g % MI][j] = mfma16(fb[g / MI][j], fa[g % (kAhead + 1)], acc[g % MI][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
    cur = nxt, at_a = next_a, at_b = next_b;
  };
  if (cn > 0) {
    const bool full = kTrA || mn > TM - NT / 8;  // every copy has rows
#pragma unroll 1
    for (int i = 0; i < kBufs; ++i)
#pragma unroll
      for (int j = 0; j < kPieces; ++j) stage_piece(j, i * kStep, false, base + i * kBuf);
    if (full || kBufs > 2)
      wait_copies<(kBufs - 1) * kPieces>();  // the first step's
    else
      wait_copies<0>();
    lds_barrier();
    int c = 0;
    using std::integral_constant;
    if (wm < mn) {
      read_b(0, 0, at_b);
      read_a(0, at_a);
      read_b(0, 1, at_b);
      read_a(1, at_a);
      read_a(2, at_a);
      if (full)
        for (; c + (kBufs + 1) * kStep <= cn; c += kStep) step(c, integral_constant<int, 0>{});
#pragma unroll 1
      for (; c + kStep < cn; c += kStep) step(c, integral_constant<int, 1>{});
      step(c, integral_constant<int, 2>{});
    } else {  // a wave past the tile's rows only copies
#pragma unroll 1
      for (; c + kStep < cn; c += kStep) {
        wait_copies<(kBufs - 2) * kPieces>();
        lds_barrier();
#pragma unroll
        for (int i = 0; i < kPieces; ++i) stage_piece(i, c + kBufs * kStep, false, cur);
        cur = after(cur);
      }
    }
    wait_copies<0>();  // nothing is written into this work-group's LDS after its end
  }

  // The products were formed transposed: lane % 16 is the output row, and a
  // lane holds 4 consecutive columns 4 (lane / 16) .. of each 16 x 16 tile.
  // Stored like that a store would touch 16 rows with 32 (64) bytes each; so
  // the tile goes through LDS, as far as it fits at a time, and leaves as
  // whole rows, 16 bytes a lane.  16-byte piece p of LDS row r lies at
  // p ^ (r % 16), which spreads 16 rows' writes over the banks.
  constexpr int kOut = ACT ? TN / 2 : TN;                         // columns
  constexpr int kPassRows = kOutLds / (kOut * (int)sizeof(O)) < TM ? kOutLds / (kOut * (int)sizeof(O)) : TM;
  constexpr int kPasses = TM / kPassRows, kI = MI / kPasses;       // 16-row blocks of a wave per pass
  constexpr int kRowPieces = kOut * (int)sizeof(O) / 16;
  constexpr int kKey = kRowPieces < 16 ? kRowPieces - 1 : 15;
  static_assert(kPassRows * kPasses == TM && kI * kPasses == MI, "whole passes");
  O* Y = (O*)s.y;
  const int64_t ldy = s.ldy;
  if (MODE == kDw) Y += (size_t)e * s.N * s.K;
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
    // (nobody reads the operands, or the pass before, any more)
    lds_barrier();
#pragma unroll
    for (int i = 0; i < kI; ++i) {
      const int row = (wv / WN) * (kPassRows / WM) + 16 * i + (lane & 15);
#pragma unroll
      for (int j = 0; j < NI; j += ACT ? 2 : 1) {
        f32x4 v = acc[pass * kI + i][j];
        if constexpr (ACT) {
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = gated(v[q], acc[pass * kI + i][j + 1][q]);
        }
        typedef __attribute__((ext_vector_type(4))) O O4;
        O4 o;
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = (O)v[q];
        const int at = ((ACT ? (wn + 16 * j) / 2 : wn + 16 * j) + 4 * (lane >> 4)) * (int)sizeof(O);
        typedef __attribute__((address_space(3))) O4 lds_o4;
        *(lds_o4*)(uintptr_t)(base + row * (kOut * (int)sizeof(O)) +
                              ((((at >> 4) ^ (row & kKey)) << 4) | (at & 15))) = o;
      }
    }
    lds_barrier();
#pragma unroll 4
    for (int at = threadIdx.x; at < kPassRows * kRowPieces; at += NT) {
      const int row = at / kRowPieces, piece = at % kRowPieces;
      // the output row behind LDS row `row` of this pass
      const int m = row / (kPassRows / WM) * (TM / WM) + pass * (kPassRows / WM) + row % (kPassRows / WM);
      typedef __attribute__((address_space(3))) const s16x8 lds_s8;
      const s16x8 v = *(lds_s8*)(uintptr_t)(base + row * (kOut * (int)sizeof(O)) +
                                            ((piece ^ (row & kKey)) << 4));
      constexpr int kPer = 16 / (int)sizeof(O);
      const int n = piece * kPer;
      O* y = Y + (int64_t)(m0 + m) * ldy + n0 + n;
      if (m < mn && s.y16 && n + kPer <= nn) {
        *reinterpret_cast<s16x8*>(y) = v;
      } else if (m < mn) {
        typedef __attribute__((ext_vector_type(kPer))) O On;
        const On o = __builtin_bit_cast(On, v);
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (n + j < nn) y[j] = o[j];
      }
    }
  }
}

// Bound by the matrix cores and the copies that feed them: 8 experts of
// 4096 x 14336 with 1024 rows each, forward 745 us (1290 TFLOP/s), dx 745, dw
// (1.9 GB of float32 written) 1045.
//
// One work-group per tile: first the whole rounds of the chip's compute units
// with 256 x 256 tiles, then what is left: cut in four 128 x 128 tiles where
// those make one round at most, in two of 256 x 128 where those do (a quarter
// takes about 0.45 of a tile's time, a half 0.65: its copies, not its
// products, take the time), else as it is.
constexpr int kUnits = 256;       // compute units of an MI355X, one work-group each (its LDS)

template <class T, class O, int MODE, bool ACT>
__global__ __launch_bounds__(512, 2) void k_mm_tile(MmArgs s) {
  __shared__ __align__(1024) uint8_t lds[kLds];
  const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const int cols = MODE == kFwd ? s.N : s.K;     // output columns
  constexpr int kCols = ACT ? kTile / 2 : kTile; // of them per tile
  const int ntn = (cols + kCols - 1) / kCols, ntm = (s.N + kTile - 1) / kTile;
  const int mt = MODE == kDw ? s.E * ntm : count_tiles(s.bounds, s.E, s.R, kTile);
  const uint32_t total = (uint32_t)mt * ntn, left = total % kUnits;
  const uint32_t parts = left <= kUnits / 4 ? 4 : left <= kUnits / 2 ? 2 : 1;
  const uint32_t whole = parts > 1 ? total - left : total;
  // Work-group b runs on XCD b % 8, and every XCD takes 32 consecutive tiles of
  // a round, which share operand rows in its L2.  (One long run per XCD would
  // leave those with the small experts' part tiles idle at the end.)
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
  int e, m0, mn, c0, cn, mi, ni;
  tile_place(id, mt, ntn, mi, ni);
  if (MODE == kDw) {
    e = mi / ntm;
    m0 = (mi - e * ntm) * kTile, mn = min(kTile, s.N - m0);
    int hi;
    expert_rows(s.bounds, e, s.R, c0, hi);
    cn = hi - c0;
  } else {
    const Tile t = find_tile(s.bounds, s.E, s.R, mi, kTile);
    if (t.n <= 0) return;
    e = t.e, m0 = t.row0, mn = t.n;
    c0 = 0, cn = MODE == kFwd ? s.K : s.N;
  }
  int n0 = ni * kCols, nn = min(kCols, cols - n0);
  if (part < 0) {
    mm_tile<T, O, MODE, kTile, kTile, 2, 4, 2, ACT>(s, base, e, m0, mn, n0, nn, c0, cn);
  } else if (parts == 4) {
    const int pm = (part & 1) * (kTile / 2), pn = (part >> 1) * (kCols / 2);
    mn = min(kTile / 2, mn - pm), nn = min(kCols / 2, nn - pn);
    if (mn <= 0 || nn <= 0) return;
    mm_tile<T, O, MODE, kTile / 2, kTile / 2, 2, 4, 4, ACT>(s, base, e, m0 + pm, mn, n0 + pn, nn,
                                                            c0, cn);
  } else {
    const int pn = part * (kCols / 2);
    nn = min(kCols / 2, nn - pn);
    if (nn <= 0) return;
    mm_tile<T, O, MODE, kTile, kTile / 2, 2, 4, 3, ACT>(s, base, e, m0, mn, n0 + pn, nn, c0, cn);
  }
}

// ------------------------------------------------- few rows per expert, forward
// Reads every weight once, straight into registers.  A work-group takes up to
// 64 sorted rows of one expert and 32 rows of its weights (with the
// activation 16 of the gate and the same 16 of the up half); its four waves
// split the inputs in turns of 64, a whole 128-byte line of each weight row,
// and add up their sums through LDS.  The weights are the products' first
// operand, so that 16 rows of x fill the other side of one matrix-core
// instruction; rows of x past the tile's repeat the last one.  Bound by the
// weights' bytes: gate/up of 8 experts (50 MB) 12.3 us, of the 70 experts that
// 32 tokens reach (429 MB) 85 us, 5.0 TB/s.
constexpr int kFewRows = 64, kFewCols = 32, kFewWaves = 4;

// 8 elements from an address of any element's alignment (the hardware takes
// it), 0 from the `left`-th on
template <class V, class T>
__device__ __forceinline__ V few_load(const T* p, int left) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  typedef u4 loose __attribute__((aligned(2)));
  u4 v = {0, 0, 0, 0};
  if (left >= 8) {
    v = *reinterpret_cast<const loose*>(p);
  } else if (left > 0) {
    V e = {};
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < left) e[j] = p[j];
    return e;
  }
  return __builtin_bit_cast(V, v);
}

template <class T, class O, bool ACT, int MB>
__device__ __forceinline__ void few_rows(const MmArgs& s, const Tile& t, float* lds) {
  typedef typename Vec8<T>::type V;
  constexpr int U = MB == 1 ? 4 : MB == 2 ? 2 : 1;  // turns whose loads are in flight together
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * (ACT ? kFewCols / 2 : kFewCols);
  const T* w[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int64_t row = ACT ? (int64_t)b * s.N + min(n0 + r, s.N - 1) : min(n0 + 16 * b + r, s.N - 1);
    w[b] = (const T*)s.b + ((int64_t)t.e * (ACT ? 2 : 1) * s.N + row) * s.ldb + 8 * q;
  }
  const T* x[MB];
  bool bad[MB];
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const int xr = x_row(s, t.row0 + min(16 * m + r, t.n - 1));
    bad[m] = xr < 0;
    x[m] = (const T*)s.a + (int64_t)max(xr, 0) * s.lda + 8 * q;
  }
  f32x4 acc[MB][2] = {};
  auto turn = [&](int k0, auto whole_) {  // inputs k0 .. and every kFewWaves * 64 on, U times
    constexpr bool whole = decltype(whole_)::value;
    V vw[U][2][2], vx[U][MB][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = k0 + u * kFewWaves * 64 + 32 * h;
        const int left = whole ? 8 : s.K - (k + 8 * q);  // inputs of this lane
#pragma unroll
        for (int b = 0; b < 2; ++b) vw[u][b][h] = few_load<V>(w[b] + k, left);
#pragma unroll
        for (int m = 0; m < MB; ++m) vx[u][m][h] = few_load<V>(x[m] + k, left);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
          for (int b = 0; b < 2; ++b) acc[m][b] = mfma16(vw[u][b][h], vx[u][m][h], acc[m][b]);
  };
  constexpr int kTurn = U * kFewWaves * 64;
  int k = wv * 64;
  for (; k + kTurn - kFewWaves * 64 + 64 <= s.K; k += kTurn) turn(k, std::true_type{});
  if (k < s.K) turn(k, std::false_type{});

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

template <class T, class O, bool ACT>
__global__ __launch_bounds__(64 * kFewWaves, 4) void k_mm_few(MmArgs s) {
  __shared__ float lds[kFewWaves * 8 * 64 * 4];
  const Tile t = find_tile(s.bounds, s.E, s.R, blockIdx.y, kFewRows);
  if (t.n == 0) return;
  if (t.n <= 16)
    few_rows<T, O, ACT, 1>(s, t, lds);
  else if (t.n <= 32)
    few_rows<T, O, ACT, 2>(s, t, lds);
  else
    few_rows<T, O, ACT, 4>(s, t, lds);
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
  if (!countable(R, E, kFewRows)) return fail(BITSMOE_ESHAPE, "R=%d with E=%d", R, E);
  if (!bounds) return fail(BITSMOE_EINVAL, "bounds is null");
  return BITSMOE_OK;
}

int rows_check(const int32_t* rows, int div, int x_rows, int R) {
  // (with rows: a row of x that a wrong index may be clamped to)
  if (rows ? (div < 1 || x_rows < (R > 0)) : x_rows < R)
    return fail(BITSMOE_ESHAPE, "div=%d, %d rows of x for R=%d", div, x_rows, R);
  return BITSMOE_OK;
}

bool rows16(const void* p, int64_t ld) { return ((uintptr_t)p & 15u) == 0 && ld % 8 == 0; }

// Up to kFewMean rows per expert on average the few-rows kernel is the faster
// one (us by it and by the tiled one: 64 experts of 1536 x 2048, 16 rows 97 and
// 109, 32 rows 112 and 111, 64 rows 149 and 116; 8 experts of 4096 x 4096, 16
// rows 70 and 57), and up to kFewMeanSmall while there are few 256 x 256 tiles
// to spread over the chip (one expert of 4096 x 4096: 32 rows 21 and 27, 64
// rows 32 and 27).
constexpr int kFewMean = 12, kFewMeanSmall = 32, kFewTiles = 32;

bool few(const MmArgs& s) {
  const long long tiles = (long long)((s.N + kTile - 1) / kTile) * s.E * ((s.R / s.E + kTile - 1) / kTile);
  return s.R <= (long long)(tiles <= kFewTiles ? kFewMeanSmall : kFewMean) * s.E &&
         max_tiles(s.R, s.E, kFewRows) <= 65535;
}

// What of the operands the tiled kernel cannot read in place: rows that are
// not whole 16-byte pieces, along the contraction or across it.
struct Pad {
  bool a, b;
  size_t a_bytes, b_bytes;
};
Pad pad_of(const MmArgs& s, int mode, int64_t a_rows) {
  Pad p{};
  if (mode == kFwd && few(s)) return p;
  const int ac = mode == kFwd ? s.K : s.N, bc = s.K;
  const int64_t b_rows = mode == kDw ? s.x_rows : (int64_t)s.E * s.N * (s.act ? 2 : 1);
  p.a = ac % 8 != 0 || !rows16(s.a, s.lda);
  p.b = bc % 8 != 0 || !rows16(s.b, s.ldb);
  auto al = [](size_t x) { return (x + 255) / 256 * 256; };
  p.a_bytes = p.a ? al((size_t)a_rows * ((ac + 7) / 8) * 16) : 0;
  p.b_bytes = p.b ? al((size_t)b_rows * ((bc + 7) / 8) * 16) : 0;
  return p;
}

int pad_rows(const void*& src, int64_t& ld, int64_t rows, int cols, void* dst, hipStream_t st) {
  const int64_t pieces = rows * ((cols + 7) / 8);
  if (pieces) {
    const int64_t blocks = (pieces + 255) / 256;
    hipLaunchKernelGGL(k_mm_pad, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, st,
                       (const uint16_t*)src, ld, rows, cols, (uint4*)dst);
  }
  src = dst;
  ld = (cols + 7) / 8 * 8;
  return launched("grouped_matmul rows");
}

template <int MODE>
int launch_mm(MmArgs s, int dtype, int o_dtype, int64_t a_rows, void* ws, size_t ws_bytes,
              hipStream_t st) {
  s.y16 = rows16(s.y, s.ldy);
  const Pad p = pad_of(s, MODE, a_rows);
  if (p.a_bytes + p.b_bytes > ws_bytes || (p.a_bytes + p.b_bytes && !ws))
    return fail(BITSMOE_ENOSPC, "ws_bytes=%zu < %zu (operands that are not 16-byte rows)", ws_bytes,
                p.a_bytes + p.b_bytes);
  if (p.a_bytes + p.b_bytes && ((uintptr_t)ws & 255u))
    return fail(BITSMOE_EINVAL, "misaligned workspace (256 bytes)");
  const int cols = MODE == kFwd ? s.N : s.K, per = s.act ? kTile / 2 : kTile;
  const long long ntn = (cols + per - 1) / per;
  const long long mt =
      MODE == kDw ? (long long)s.E * ((s.N + kTile - 1) / kTile) : max_tiles(s.R, s.E, kTile);
  // enough for any split of at most mt * ntn tiles into whole rounds and cut tiles
  const long long groups = (mt * ntn + kUnits - 1) / kUnits * kUnits + kUnits + 8;
  if (groups * 512 > 0xFFFFFFFFll)  // (a grid's work-items)
    return fail(BITSMOE_ESHAPE, "R=%d E=%d N=%d K=%d make too many tiles", s.R, s.E, s.N, s.K);
  int rc = BITSMOE_OK;
  if (p.a &&
      (rc = pad_rows(s.a, s.lda, a_rows, MODE == kFwd ? s.K : s.N, ws, st)))
    return rc;
  if (p.b && (rc = pad_rows(s.b, s.ldb,
                            MODE == kDw ? s.x_rows : (int64_t)s.E * s.N * (s.act ? 2 : 1), s.K,
                            (uint8_t*)ws + p.a_bytes, st)))
    return rc;
  with_types(dtype, o_dtype, [&](auto t, auto o) {
    using T = decltype(t);
    using O = decltype(o);
    if constexpr (MODE == kFwd) {
      if (few(s)) {
        const int fp = s.act ? kFewCols / 2 : kFewCols;
        const dim3 grid((unsigned)((s.N + fp - 1) / fp), (unsigned)max_tiles(s.R, s.E, kFewRows));
        if (s.act)
          hipLaunchKernelGGL((k_mm_few<T, O, true>), grid, dim3(64 * kFewWaves), 0, st, s);
        else
          hipLaunchKernelGGL((k_mm_few<T, O, false>), grid, dim3(64 * kFewWaves), 0, st, s);
        return;
      }
    }
    const dim3 grid((unsigned)groups);
    if (MODE == kFwd && s.act)
      hipLaunchKernelGGL((k_mm_tile<T, O, MODE, MODE == kFwd>), grid, dim3(512), 0, st, s);
    else
      hipLaunchKernelGGL((k_mm_tile<T, O, MODE, false>), grid, dim3(512), 0, st, s);
  });
  return launched("grouped_matmul");
}

}  // namespace
}  // namespace experts
}  // namespace bitsmoe

using namespace bitsmoe;
using namespace bitsmoe::experts;

extern "C" {

int bitsmoe_grouped_matmul_workspace_size(int op, const void* a, int64_t lda, int64_t a_rows,
                                          const void* b, int64_t ldb, int64_t b_rows, int R, int E,
                                          int N, int K, int act, size_t* bytes) {
  if (!bytes) return fail(BITSMOE_EINVAL, "bytes is null");
  if (op < BITSMOE_GROUPED_FORWARD || op > BITSMOE_GROUPED_DW) return fail(BITSMOE_EINVAL, "op=%d", op);
  if (R < 0 || E < 1 || N < 1 || K < 1 || a_rows < 0 || b_rows < 0 || b_rows > 0x7FFFFFFFll)
    return fail(BITSMOE_ESHAPE, "R=%d E=%d N=%d K=%d", R, E, N, K);
  MmArgs s{};
  s.a = a, s.lda = lda, s.b = b, s.ldb = op == BITSMOE_GROUPED_DW ? ldb : K;
  s.x_rows = (int)b_rows, s.R = R, s.E = E, s.N = N, s.K = K, s.act = act;
  const Pad p = pad_of(s, op, a_rows);
  *bytes = p.a_bytes + p.b_bytes;
  return BITSMOE_OK;
}

int bitsmoe_grouped_matmul(int dtype, const void* x, int64_t ldx, int x_rows, const int32_t* rows,
                           int div, const void* w, const int32_t* bounds, int R, int E, int N,
                           int K, int act, void* y, int y_dtype, int64_t ldy, void* ws,
                           size_t ws_bytes, bitsmoe_stream_t stream) {
  int st = mm_check(dtype, y_dtype, R, E, N, K, bounds);
  if (st || (st = rows_check(rows, div, x_rows, R))) return st;
  if (act != BITSMOE_ACT_NONE && act != BITSMOE_ACT_SILU_MUL)
    return fail(BITSMOE_EINVAL, "act=%d", act);
  if (ldx < K || ldy < N) return fail(BITSMOE_ESHAPE, "a row stride is too small");
  if (R == 0) return BITSMOE_OK;
  if (!w || !y || (x_rows && !x)) return fail(BITSMOE_EINVAL, "null pointer argument");
  const MmArgs s{x, ldx, w, K, rows, div, x_rows, bounds, R, E, N, K, y, ldy, act, 0};
  return launch_mm<kFwd>(s, dtype, y_dtype, x_rows, ws, ws_bytes, (hipStream_t)stream);
}

int bitsmoe_grouped_matmul_dx(int dtype, const void* dy, int64_t lddy, const void* w,
                              const int32_t* bounds, int R, int E, int N, int K, void* dx,
                              int dx_dtype, int64_t lddx, void* ws, size_t ws_bytes,
                              bitsmoe_stream_t stream) {
  const int st = mm_check(dtype, dx_dtype, R, E, N, K, bounds);
  if (st) return st;
  if (lddy < N || lddx < K) return fail(BITSMOE_ESHAPE, "a row stride is too small");
  if (R == 0) return BITSMOE_OK;
  if (!dy || !w || !dx) return fail(BITSMOE_EINVAL, "null pointer argument");
  const MmArgs s{dy, lddy, w, K, nullptr, 1, R, bounds, R, E, N, K, dx, lddx, 0, 0};
  return launch_mm<kDx>(s, dtype, dx_dtype, R, ws, ws_bytes, (hipStream_t)stream);
}

int bitsmoe_grouped_matmul_dw(int dtype, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                              int x_rows, const int32_t* rows, int div, const int32_t* bounds,
                              int R, int E, int N, int K, void* dw, int dw_dtype, void* ws,
                              size_t ws_bytes, bitsmoe_stream_t stream) {
  int st = mm_check(dtype, dw_dtype, R, E, N, K, bounds);
  if (st || (st = rows_check(rows, div, x_rows, R))) return st;
  if (lddy < N || ldx < K) return fail(BITSMOE_ESHAPE, "a row stride is too small");
  if (!dw || (R && (!dy || (x_rows && !x)))) return fail(BITSMOE_EINVAL, "null pointer argument");
  const MmArgs s{dy, lddy, x, ldx, rows, div, x_rows, bounds, R, E, N, K, dw, K, 0, 0};
  return launch_mm<kDw>(s, dtype, dw_dtype, R, ws, ws_bytes, (hipStream_t)stream);
}

}  // extern "C"
