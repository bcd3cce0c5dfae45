// The gated activation h = SiLU(gate) * up of rows [gate | up], its gradient,
// and the routing-weighted combine of the experts' rows with its gradient.
// Every kernel here is bound by memory: each input element is read once and
// each output written once, 16 bytes a lane where the rows allow it.  24576 x
// 1408: 33 us and 53 us with the gradient's; combine of 8192 x 6 rows of 2048:
// 53 us, its gradient 73.
#include "experts.h"

namespace bitsmoe {
namespace experts {
namespace {

constexpr int kThreads = 256;

// Rows behind the last expert's are left as they were.
__device__ inline int live_rows(const int32_t* __restrict__ bounds, int E, int R) {
  return bounds ? min(max(bounds[E], 0), R) : R;
}

// h[r, i] = SiLU(a[r, i]) a[r, F + i], V elements a lane (8: F, both strides
// and the pointers are multiples of 8 elements; 1 otherwise).
template <class T, int V>
__global__ __launch_bounds__(kThreads) void k_silu_mul(const T* __restrict__ a, int64_t lda,
                                                       const int32_t* __restrict__ bounds, int E,
                                                       int R, int F, T* __restrict__ h,
                                                       int64_t ldh) {
  const int n = live_rows(bounds, E, R);
  const int per = F / V;
  const int64_t total = (int64_t)n * per;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kThreads) {
    const int64_t r = i / per;
    const int c = (int)(i - r * per) * V;
    if constexpr (V == 8) {
      float g[8], u[8], o[8];
      load8(a + r * lda + c, g);
      load8(a + r * lda + F + c, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = gated(g[j], u[j]);
      store8(h + r * ldh + c, o);
    } else {
      h[r * ldh + c] = from_f32<T>(gated(to_f32(a[r * lda + c]), to_f32(a[r * lda + F + c])));
    }
  }
}

// (da may be a: a lane reads its elements of a before it writes them to da,
// and neither pointer promises that they differ)
template <class T, int V>
__global__ __launch_bounds__(kThreads) void k_silu_mul_grad(
    const T* a, int64_t lda, const T* __restrict__ dh, int64_t lddh,
    const int32_t* __restrict__ bounds, int E, int R, int F, T* da, int64_t ldda) {
  const int n = live_rows(bounds, E, R);
  const int per = F / V;
  const int64_t total = (int64_t)n * per;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kThreads) {
    const int64_t r = i / per;
    const int c = (int)(i - r * per) * V;
    if constexpr (V == 8) {
      float g[8], u[8], d[8], dg[8], du[8];
      load8(a + r * lda + c, g);
      load8(a + r * lda + F + c, u);
      load8(dh + r * lddh + c, d);
#pragma unroll
      for (int j = 0; j < 8; ++j) gated_grad(g[j], u[j], d[j], dg[j], du[j]);
      store8(da + r * ldda + c, dg);
      store8(da + r * ldda + F + c, du);
    } else {
      float dg, du;
      gated_grad(to_f32(a[r * lda + c]), to_f32(a[r * lda + F + c]), to_f32(dh[r * lddh + c]), dg,
                 du);
      da[r * ldda + c] = from_f32<T>(dg);
      da[r * ldda + F + c] = from_f32<T>(du);
    }
  }
}

constexpr int kSlots = 8;  // slots of a token whose rows are in flight together

// out[t] = sum_j g[t, j] y[slot[t, j]] in slot order, float32 sums.  A slot
// outside [0, R) has a row of zeros: the NaN weights of a token that has no
// softmax make its output NaN.  One work-group takes kThreads * V columns of a
// token; the rows of kSlots slots are loaded before the first is used.
template <class T, class O, int V>
__global__ __launch_bounds__(kThreads) void k_combine_rows(const T* __restrict__ y, int64_t ldy,
                                                           int R, const int32_t* __restrict__ slot,
                                                           const float* __restrict__ g, int k,
                                                           int D, O* __restrict__ out,
                                                           int64_t ldo) {
  const int64_t t = blockIdx.x;
  const int c = ((int)blockIdx.y * kThreads + (int)threadIdx.x) * V;
  if (c >= D) return;
  float acc[V] = {};
  for (int j0 = 0; j0 < k; j0 += kSlots) {
    float row[kSlots][V], w[kSlots];
#pragma unroll
    for (int u = 0; u < kSlots; ++u) {
      const int s = j0 + u < k ? slot[t * k + j0 + u] : -1;
      const bool there = s >= 0 && s < R;
      w[u] = j0 + u < k && g ? g[t * k + j0 + u] : 1.f;
#pragma unroll
      for (int i = 0; i < V; ++i) row[u][i] = 0.f;
      if (there) {
        if constexpr (V == 8)
          load8(y + s * ldy + c, row[u]);
        else
          row[u][0] = to_f32(y[s * ldy + c]);
      }
    }
#pragma unroll
    for (int u = 0; u < kSlots; ++u)
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = fmaf(w[u], row[u][i], acc[i]);
  }
  if constexpr (V == 8)
    store8(out + t * ldo + c, acc);
  else
    out[t * ldo + c] = from_f32<O>(acc[0]);
}

// dy[slot[t, j]] = g[t, j] dout[t]; dg[t, j] = <dout[t], y[slot[t, j]]> (0
// where there is no row).  One work-group per token; a slot's dot product is
// summed over a lane's columns, the wave and the waves, always in this order.
template <class T, class O, int V>
__global__ __launch_bounds__(kThreads) void k_combine_grad(
    const O* __restrict__ dout, int64_t ldo, const T* __restrict__ y, int64_t ldy, int R,
    const int32_t* __restrict__ slot, const float* __restrict__ g, int k, int D,
    T* __restrict__ dy, int64_t lddy, float* __restrict__ dg) {
  __shared__ float part[kThreads / 64][kSlots];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  for (int j0 = 0; j0 < k; j0 += kSlots) {
    float acc[kSlots] = {};
    for (int c = (int)threadIdx.x * V; c < D; c += kThreads * V) {
      float d[V];
      if constexpr (V == 8)
        load8(dout + t * ldo + c, d);
      else
        d[0] = to_f32(dout[t * ldo + c]);
#pragma unroll
      for (int u = 0; u < kSlots; ++u) {
        const int s = j0 + u < k ? slot[t * k + j0 + u] : -1;
        if (s < 0 || s >= R) continue;
        const float w = g ? g[t * k + j0 + u] : 1.f;
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = w * d[i];
        if (dg) {
          float row[V];
          if constexpr (V == 8)
            load8(y + s * ldy + c, row);
          else
            row[0] = to_f32(y[s * ldy + c]);
#pragma unroll
          for (int i = 0; i < V; ++i) acc[u] = fmaf(d[i], row[i], acc[u]);
        }
        if constexpr (V == 8)
          store8(dy + s * lddy + c, o);
        else
          dy[s * lddy + c] = from_f32<T>(o[0]);
      }
    }
    if (!dg) continue;
#pragma unroll
    for (int u = 0; u < kSlots; ++u) {
#pragma unroll
      for (int m = 32; m > 0; m >>= 1) acc[u] += __shfl_xor(acc[u], m, 64);
      if (lane == 0) part[wv][u] = acc[u];
    }
    __syncthreads();
    if ((int)threadIdx.x < kSlots && j0 + (int)threadIdx.x < k) {
      float s = 0.f;
      for (int w = 0; w < kThreads / 64; ++w) s += part[w][threadIdx.x];
      dg[t * k + j0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

unsigned elem_grid(int64_t work) {
  // 256 compute units, 16 work-groups each, then a loop over the rest
  const int64_t b = (work + kThreads - 1) / kThreads;
  return (unsigned)(b < 1 ? 1 : b > 4096 ? 4096 : b);
}

bool aligned(const void* p, int64_t ld, int dtype) {
  return ((uintptr_t)p & 15u) == 0 && ld % 8 == 0 && (dtype == BITSMOE_F32 || is_half(dtype));
}

int act_check(int dtype, const void* a, int64_t lda, const int32_t* bounds, int R, int E, int F,
              const void* h, int64_t ldh) {
  if (!is_half(dtype)) return fail(BITSMOE_EINVAL, "dtype=%d (float16 or bfloat16)", dtype);
  if (R < 0 || F < 1 || E < 0) return fail(BITSMOE_ESHAPE, "R=%d F=%d E=%d", R, F, E);
  if (bounds && E < 1) return fail(BITSMOE_ESHAPE, "bounds with E=%d", E);
  if (F > (1 << 28)) return fail(BITSMOE_ESHAPE, "F=%d too large", F);
  if (R && (!a || !h)) return fail(BITSMOE_EINVAL, "null pointer argument");
  if (lda < 2 * (int64_t)F || ldh < F) return fail(BITSMOE_ESHAPE, "a row stride is too small");
  return BITSMOE_OK;
}

int combine_check(int T, int k, int R, int D, int y_dtype, int o_dtype, const void* y,
                  int64_t ldy, const int32_t* slot, const void* out, int64_t ldo) {
  if (T < 0 || k < 1 || R < 0 || D < 1)
    return fail(BITSMOE_ESHAPE, "T=%d k=%d R=%d D=%d", T, k, R, D);
  // (a work-group per token, 2^32 - 1 work-items a grid)
  if (T > ((1 << 30) - 1) / (k < 64 ? 64 : k)) return fail(BITSMOE_ESHAPE, "T=%d k=%d too large", T, k);
  if (D > (1 << 24)) return fail(BITSMOE_ESHAPE, "D=%d too large", D);
  if (!is_half(y_dtype) || (o_dtype != y_dtype && o_dtype != BITSMOE_F32))
    return fail(BITSMOE_EINVAL, "y dtype %d, out dtype %d", y_dtype, o_dtype);
  if (ldy < D || ldo < D) return fail(BITSMOE_ESHAPE, "a row stride is smaller than D=%d", D);
  if (T && (!slot || !out || (R && !y))) return fail(BITSMOE_EINVAL, "null pointer argument");
  return BITSMOE_OK;
}

}  // namespace
}  // namespace experts
}  // namespace bitsmoe

using namespace bitsmoe;
using namespace bitsmoe::experts;

extern "C" {

int bitsmoe_silu_mul(int dtype, const void* a, int64_t lda, const int32_t* bounds, int R, int E,
                     int F, void* h, int64_t ldh, bitsmoe_stream_t stream) {
  const int st = act_check(dtype, a, lda, bounds, R, E, F, h, ldh);
  if (st || R == 0) return st;
  const bool v8 = F % 8 == 0 && aligned(a, lda, dtype) && aligned(h, ldh, dtype);
  const dim3 grid(elem_grid((int64_t)R * F / (v8 ? 8 : 1)));
  auto go = [&](auto tag) {
    using T = decltype(tag);
    if (v8)
      hipLaunchKernelGGL((k_silu_mul<T, 8>), grid, dim3(kThreads), 0, (hipStream_t)stream,
                         (const T*)a, lda, bounds, E, R, F, (T*)h, ldh);
    else
      hipLaunchKernelGGL((k_silu_mul<T, 1>), grid, dim3(kThreads), 0, (hipStream_t)stream,
                         (const T*)a, lda, bounds, E, R, F, (T*)h, ldh);
  };
  if (dtype == BITSMOE_F16)
    go(f16{});
  else
    go(bf16{});
  return launched("silu_mul");
}

int bitsmoe_silu_mul_grad(int dtype, const void* a, int64_t lda, const void* dh, int64_t lddh,
                          const int32_t* bounds, int R, int E, int F, void* da, int64_t ldda,
                          bitsmoe_stream_t stream) {
  const int st = act_check(dtype, a, lda, bounds, R, E, F, dh, lddh);
  if (st || R == 0) return st;
  if (!da) return fail(BITSMOE_EINVAL, "da is null");
  if (ldda < 2 * (int64_t)F) return fail(BITSMOE_ESHAPE, "a row stride is too small");
  const bool v8 = F % 8 == 0 && aligned(a, lda, dtype) && aligned(dh, lddh, dtype) &&
                  aligned(da, ldda, dtype);
  const dim3 grid(elem_grid((int64_t)R * F / (v8 ? 8 : 1)));
  auto go = [&](auto tag) {
    using T = decltype(tag);
    if (v8)
      hipLaunchKernelGGL((k_silu_mul_grad<T, 8>), grid, dim3(kThreads), 0, (hipStream_t)stream,
                         (const T*)a, lda, (const T*)dh, lddh, bounds, E, R, F, (T*)da, ldda);
    else
      hipLaunchKernelGGL((k_silu_mul_grad<T, 1>), grid, dim3(kThreads), 0, (hipStream_t)stream,
                         (const T*)a, lda, (const T*)dh, lddh, bounds, E, R, F, (T*)da, ldda);
  };
  if (dtype == BITSMOE_F16)
    go(f16{});
  else
    go(bf16{});
  return launched("silu_mul_grad");
}

int bitsmoe_moe_combine(int y_dtype, const void* y, int64_t ldy, int R, const int32_t* slot,
                        const float* g, int T, int k, int D, void* out, int out_dtype,
                        int64_t ldo, bitsmoe_stream_t stream) {
  const int st = combine_check(T, k, R, D, y_dtype, out_dtype, y, ldy, slot, out, ldo);
  if (st || T == 0) return st;
  const bool v8 = D % 8 == 0 && aligned(y, ldy, y_dtype) && aligned(out, ldo, out_dtype);
  const int per = kThreads * (v8 ? 8 : 1);
  const dim3 grid((unsigned)T, (unsigned)((D + per - 1) / per));
  if (grid.y > 65535) return fail(BITSMOE_ESHAPE, "D=%d too large for rows that are not 16-byte aligned", D);
  auto go = [&](auto ty, auto to) {
    using TY = decltype(ty);
    using TO = decltype(to);
    if (v8)
      hipLaunchKernelGGL((k_combine_rows<TY, TO, 8>), grid, dim3(kThreads), 0,
                         (hipStream_t)stream, (const TY*)y, ldy, R, slot, g, k, D, (TO*)out, ldo);
    else
      hipLaunchKernelGGL((k_combine_rows<TY, TO, 1>), grid, dim3(kThreads), 0,
                         (hipStream_t)stream, (const TY*)y, ldy, R, slot, g, k, D, (TO*)out, ldo);
  };
  if (y_dtype == BITSMOE_F16) {
    if (out_dtype == BITSMOE_F32)
      go(f16{}, float{});
    else
      go(f16{}, f16{});
  } else {
    if (out_dtype == BITSMOE_F32)
      go(bf16{}, float{});
    else
      go(bf16{}, bf16{});
  }
  return launched("moe_combine");
}

int bitsmoe_moe_combine_grad(const void* dout, int out_dtype, int64_t ldo, int y_dtype,
                             const void* y, int64_t ldy, int R, const int32_t* slot,
                             const float* g, int T, int k, int D, void* dy, int64_t lddy,
                             float* dg, bitsmoe_stream_t stream) {
  // without dg the rows themselves are not read
  const int st = combine_check(T, k, R, D, y_dtype, out_dtype, dg ? y : dy, dg ? ldy : lddy, slot,
                               dout, ldo);
  if (st || T == 0) return st;
  if (R && !dy) return fail(BITSMOE_EINVAL, "dy is null");
  if (lddy < D) return fail(BITSMOE_ESHAPE, "a row stride is smaller than D=%d", D);
  const bool v8 = D % 8 == 0 && aligned(dout, ldo, out_dtype) && aligned(dy, lddy, y_dtype) &&
                  (!dg || aligned(y, ldy, y_dtype));
  auto go = [&](auto ty, auto to) {
    using TY = decltype(ty);
    using TO = decltype(to);
    if (v8)
      hipLaunchKernelGGL((k_combine_grad<TY, TO, 8>), dim3((unsigned)T), dim3(kThreads), 0,
                         (hipStream_t)stream, (const TO*)dout, ldo, (const TY*)y, ldy, R, slot, g,
                         k, D, (TY*)dy, lddy, dg);
    else
      hipLaunchKernelGGL((k_combine_grad<TY, TO, 1>), dim3((unsigned)T), dim3(kThreads), 0,
                         (hipStream_t)stream, (const TO*)dout, ldo, (const TY*)y, ldy, R, slot, g,
                         k, D, (TY*)dy, lddy, dg);
  };
  if (y_dtype == BITSMOE_F16) {
    if (out_dtype == BITSMOE_F32)
      go(f16{}, float{});
    else
      go(f16{}, f16{});
  } else {
    if (out_dtype == BITSMOE_F32)
      go(bf16{}, float{});
    else
      go(bf16{}, bf16{});
  }
  return launched("moe_combine_grad");
}

}  // extern "C"
