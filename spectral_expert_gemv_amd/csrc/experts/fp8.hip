// Quantizers to 8-bit floating point with a scale per 128 elements of a row
// (activations, optionally of SiLU(gate) * up) or per block of 128 x 128
// (weights, optionally with a transposed copy for the gradients).
#include "fp8.h"

namespace bitsmoe {
namespace experts {
namespace {

constexpr int kThreads = 256;

// Rows of x (ACT: [gate | up], 2 K wide) to rows of codes, K filled up with 0
// to whole groups.  16 lanes a group, 8 elements a lane: the group's largest
// magnitude is four DPP steps.  Bound by memory, reads and writes mixed: 24576
// rows of the activation of 2 x 1408 36 us (4.8 TB/s), 8192 x 4096 20 us (5.0);
// two groups of a lane in flight 38, stores past the caches 35.
template <class T, bool ACT>
__global__ __launch_bounds__(kThreads) void k_fp8_rows(const T* __restrict__ x, int64_t ldx,
                                                       Gather from,
                                                       const int32_t* __restrict__ bounds, int E,
                                                       int R, int K, int kg,
                                                       uint8_t* __restrict__ codes, int64_t ldc,
                                                       float* __restrict__ scales, int64_t lds) {
  const int n = bounds ? min(max(bounds[E], 0), R) : R;
  const int l = threadIdx.x & 15;
  const int64_t first = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 4;
  const int64_t step = (int64_t)gridDim.x * (kThreads / 16);
  // (row and group of the loop's steps without a division each)
  int64_t r = first / kg;
  int g = (int)(first - r * kg);
  const int64_t dr = step / kg;
  const int dg = (int)(step - dr * kg);
  while (__any(r < n)) {  // whole waves
    const bool live = r < n;
    const int c = g * kGroup + 8 * l;
    float v[8] = {};
    int64_t xr = r;
    if (from.rows) {
      const int p = live ? from.rows[r] : -1;
      xr = p < 0 || p / from.div >= from.x_rows ? -1 : p / from.div;
    }
    if (live && xr >= 0) {
      load8_any(x + xr * ldx + c, K - c, v);
      if constexpr (ACT) {
        float u[8];
        load8_any(x + xr * ldx + K + c, K - c, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = gated(v[i], u[i]);
      }
    }
    uint32_t a = row_max(amax_bits<false>(v));
    if (__any(a >= kInfBits)) a = row_max(amax_bits<true>(v));
    const Factors f = factors8(a);
    if (live) {
      uint2 q;
      q.x = codes4(v[0], v[1], v[2], v[3], f.r);
      q.y = codes4(v[4], v[5], v[6], v[7], f.r);
      *reinterpret_cast<uint2*>(codes + r * ldc + c) = q;
      if (l == 0) scales[r * lds + g] = xr < 0 ? __builtin_nanf("") : f.s;
    }
    r += dr;
    g += dg;
    if (g >= kg) g -= kg, ++r;
  }
}

// One work-group per block of 128 x 128 weights: 16 lanes a row, 8 elements a
// lane, 8 rows a thread, so the block is read once and stays in registers
// between the maximum and the codes.  The transposed copy goes through LDS as
// bytes: a thread reads 4 columns of 16 rows and turns 4 x 4 bytes at a time.
// Bound by memory: 8 x 4096 x 14336 float32 weights with the copy 525 us
// (5.4 TB/s over 1.9 GB read and 0.9 written).
constexpr int kPitch = 33;  // words of an LDS row of 128 codes

template <class T>
__global__ __launch_bounds__(kThreads) void k_fp8_weights(const T* __restrict__ w, int N, int K,
                                                          int nb, int kb,
                                                          uint8_t* __restrict__ codes,
                                                          float* __restrict__ scales,
                                                          uint8_t* __restrict__ codes_t,
                                                          float* __restrict__ scales_t) {
  __shared__ uint32_t tile[kGroup * kPitch];
  __shared__ uint32_t part[2][kThreads / 64];
  const int tid = threadIdx.x, l = tid & 15;
  const int64_t b = blockIdx.x;
  const int ki = (int)(b % kb);
  const int64_t en = b / kb;
  const int ni = (int)(en % nb);
  const int64_t e = en / nb;
  const int64_t kp = (int64_t)kb * kGroup, np = (int64_t)nb * kGroup;
  const int k0 = ki * kGroup + 8 * l, n0 = ni * kGroup + (tid >> 4);
  float v[8][8];
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = n0 + 16 * i;
    load8_any(w + (e * N + (n < N ? n : 0)) * K + k0, n < N ? K - k0 : 0, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t m = amax_bits<false>(v[i]);
    a = a > m ? a : m;
  }
  auto block_max = [&](uint32_t m, int turn) {
    m = row_max(m);
#pragma unroll
    for (int d = 16; d < 64; d <<= 1) {
      const uint32_t o = (uint32_t)__shfl_xor((int)m, d, 64);
      m = m > o ? m : o;
    }
    if ((tid & 63) == 0) part[turn][tid >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) m = m > part[turn][i] ? m : part[turn][i];
    return m;
  };
  a = block_max(a, 0);
  if (a >= kInfBits) {  // (the same in all threads)
    a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t m = amax_bits<true>(v[i]);
      a = a > m ? a : m;
    }
    a = block_max(a, 1);
  }
  const Factors f = factors8(a);
  if (tid == 0) {
    scales[b] = f.s;
    if (codes_t) scales_t[(e * kb + ki) * nb + ni] = f.s;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = n0 + 16 * i;
    uint2 q;
    q.x = codes4(v[i][0], v[i][1], v[i][2], v[i][3], f.r);
    q.y = codes4(v[i][4], v[i][5], v[i][6], v[i][7], f.r);
    if (n < N) *reinterpret_cast<uint2*>(codes + (e * N + n) * kp + k0) = q;
    if (codes_t) {
      uint32_t* t = tile + ((tid >> 4) + 16 * i) * kPitch + 2 * l;
      t[0] = q.x, t[1] = q.y;
    }
  }
  if (!codes_t) return;
  __syncthreads();
  // columns 4 c .. 4 c + 3 of rows 16 h ..: rows past N hold the codes of 0
  const int c = tid >> 3, h = tid & 7;
  uint32_t out[4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t in[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) in[i] = tile[(16 * h + 4 * j + i) * kPitch + c];
    // bytes 0 and 1, 2 and 3 of two rows side by side, then of four
    const uint32_t a0 = __builtin_amdgcn_perm(in[1], in[0], 0x05010400u);
    const uint32_t a1 = __builtin_amdgcn_perm(in[1], in[0], 0x07030602u);
    const uint32_t b0 = __builtin_amdgcn_perm(in[3], in[2], 0x05010400u);
    const uint32_t b1 = __builtin_amdgcn_perm(in[3], in[2], 0x07030602u);
    out[0][j] = __builtin_amdgcn_perm(b0, a0, 0x05040100u);
    out[1][j] = __builtin_amdgcn_perm(b0, a0, 0x07060302u);
    out[2][j] = __builtin_amdgcn_perm(b1, a1, 0x05040100u);
    out[3][j] = __builtin_amdgcn_perm(b1, a1, 0x07060302u);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = ki * kGroup + 4 * c + i;
    if (k < K)
      *reinterpret_cast<uint4*>(codes_t + (e * K + k) * np + ni * kGroup + 16 * h) =
          make_uint4(out[i][0], out[i][1], out[i][2], out[i][3]);
  }
}

bool any_float(int dtype) { return dtype == BITSMOE_F32 || is_half(dtype); }

template <class F>
void with_type(int dtype, F f) {
  if (dtype == BITSMOE_F32)
    f(float{});
  else if (dtype == BITSMOE_F16)
    f(f16{});
  else
    f(bf16{});
}

}  // namespace

int run_fp8_rows(int dtype, const void* x, int64_t ldx, Gather from, int act,
                 const int32_t* bounds, int R, int E, int K, void* codes, int64_t ldc,
                 float* scales, int64_t lds, hipStream_t st) {
  const int kg = (int)groups_of(K);
  // 256 compute units, 8 work-groups each, then a loop over the rest
  const int64_t want = ((int64_t)R * kg + kThreads / 16 - 1) / (kThreads / 16);
  const dim3 grid((unsigned)(want < 2048 ? want : 2048));
  with_type(dtype, [&](auto tag) {
    using T = decltype(tag);
    if (act)
      hipLaunchKernelGGL((k_fp8_rows<T, true>), grid, dim3(kThreads), 0, st, (const T*)x, ldx,
                         from, bounds, E, R, K, kg, (uint8_t*)codes, ldc, scales, lds);
    else
      hipLaunchKernelGGL((k_fp8_rows<T, false>), grid, dim3(kThreads), 0, st, (const T*)x, ldx,
                         from, bounds, E, R, K, kg, (uint8_t*)codes, ldc, scales, lds);
  });
  return launched("fp8_rows");
}

}  // namespace experts
}  // namespace bitsmoe

using namespace bitsmoe;
using namespace bitsmoe::experts;

extern "C" {

int bitsmoe_fp8_rows(int dtype, const void* x, int64_t ldx, int act, const int32_t* bounds, int R,
                     int E, int K, void* codes, int64_t ldc, float* scales, int64_t lds,
                     bitsmoe_stream_t stream) {
  if (!any_float(dtype)) return fail(BITSMOE_EINVAL, "dtype=%d", dtype);
  if (act != BITSMOE_ACT_NONE && act != BITSMOE_ACT_SILU_MUL)
    return fail(BITSMOE_EINVAL, "act=%d", act);
  if (R < 0 || R > (1 << 26) || K < 1 || K > (1 << 20) || E < 0)
    return fail(BITSMOE_ESHAPE, "R=%d K=%d E=%d", R, K, E);
  if (bounds && E < 1) return fail(BITSMOE_ESHAPE, "bounds with E=%d", E);
  if (ldx < (act ? 2 : 1) * (int64_t)K || ldc < groups_of(K) * kGroup || lds < groups_of(K))
    return fail(BITSMOE_ESHAPE, "a row stride is too small");
  if (R == 0) return BITSMOE_OK;
  if (!x || !codes || !scales) return fail(BITSMOE_EINVAL, "null pointer argument");
  if (((uintptr_t)codes | (uintptr_t)ldc) & 15u)
    return fail(BITSMOE_EINVAL, "rows of codes must be 16-byte aligned");
  return run_fp8_rows(dtype, x, ldx, Gather{nullptr, 1, 0}, act, bounds, R, E, K, codes, ldc, scales,
                      lds, (hipStream_t)stream);
}

int bitsmoe_fp8_weights(int dtype, const void* w, int E, int N, int K, void* codes, float* scales,
                        void* codes_t, float* scales_t, bitsmoe_stream_t stream) {
  if (!any_float(dtype)) return fail(BITSMOE_EINVAL, "dtype=%d", dtype);
  if (E < 0 || N < 1 || K < 1 || N > (1 << 21) || K > (1 << 21))
    return fail(BITSMOE_ESHAPE, "E=%d N=%d K=%d", E, N, K);
  if (!codes_t != !scales_t) return fail(BITSMOE_EINVAL, "codes_t and scales_t go together");
  const int64_t nb = groups_of(N), kb = groups_of(K);
  if (E * nb * kb > 0xFFFFFFll)  // (2^32 - 1 work-items a grid)
    return fail(BITSMOE_ESHAPE, "E=%d N=%d K=%d make too many blocks", E, N, K);
  if (E == 0) return BITSMOE_OK;
  if (!w || !codes || !scales) return fail(BITSMOE_EINVAL, "null pointer argument");
  if (((uintptr_t)codes | (uintptr_t)codes_t) & 15u)
    return fail(BITSMOE_EINVAL, "codes must be 16-byte aligned");
  with_type(dtype, [&](auto tag) {
    using T = decltype(tag);
    hipLaunchKernelGGL((k_fp8_weights<T>), dim3((unsigned)(E * nb * kb)), dim3(kThreads), 0,
                       (hipStream_t)stream, (const T*)w, N, K, (int)nb, (int)kb, (uint8_t*)codes,
                       scales, (uint8_t*)codes_t, scales_t);
  });
  return launched("fp8_weights");
}

}  // extern "C"
