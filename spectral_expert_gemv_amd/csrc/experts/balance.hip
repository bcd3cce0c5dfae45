// The router's balance: per-expert counts of every sequence's tokens, the
// balance loss and the z loss, and the gradient of both with respect to the
// logits.
//
// A token takes part if one of its ids lies in [0, E) and one of its logits is
// above -inf.  Over the n tokens of a sequence that do, with p = softmax(l):
//   f_e = E / (k n) #{(t, j): id_tj = e},   P_e = 1/n sum_t p_te
//   loss = sum_e f_e P_e,   z = 1/n sum_t lse_t^2,   lse = log sum_e exp(l_te)
//   dl_te = p_te (dloss / n (f_e - sum_m p_tm f_m) + 2 dz / n lse_t)
// (f does not depend on the logits as far as a gradient goes).  softmax and
// each work-group's sums are float32; the sums over work-groups and the losses
// are float64.  No sum depends on the order of atomics.
#include <type_traits>

#include "experts.h"

namespace bitsmoe {
namespace experts {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxSlots = 64, kMaxExperts = 2048;

template <int kCtrl>
__device__ inline float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, 0xF, 0xF, false));
}
// over the L lanes of a token (16: one DPP row; 64: the wave), in every lane
template <int L, class F>
__device__ inline float reduce(float v, F f) {
  v = f(v, dpp<0xB1>(v));   // quad_perm [1,0,3,2]
  v = f(v, dpp<0x4E>(v));   // quad_perm [2,3,0,1]
  v = f(v, dpp<0x141>(v));  // row_half_mirror
  v = f(v, dpp<0x140>(v));  // row_mirror
  if constexpr (L == 64) {
    v = f(v, __shfl_xor(v, 16, 64));
    v = f(v, __shfl_xor(v, 32, 64));
  }
  return v;
}
template <int L>
__device__ inline float reduce_sum(float v) {
  return reduce<L>(v, [](float a, float b) { return a + b; });
}

// The softmax of one token over the L lanes that hold it, expert v L + l in
// value v of lane l.
template <int V>
struct Soft {
  float p[V];   // probabilities; NaN everywhere for a NaN or +inf among the logits
  float lse;
  bool part;    // whether the token takes part
};

template <class T, int L, int V>
__device__ __forceinline__ Soft<V> soft(const T* __restrict__ logits, const int32_t* __restrict__ ids,
                                        int E, int k, bool live) {
  const int l = threadIdx.x & (L - 1);
  Soft<V> o;
  float m = -INFINITY;
  bool bad = false, any = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * L + l;
    o.p[v] = live && e < E ? to_f32(logits[e]) : -INFINITY;
    bad |= !(o.p[v] < INFINITY);
    m = fmaxf(m, o.p[v]);
  }
  for (int j = l; j < k; j += L) any |= live && ids[j] >= 0 && ids[j] < E;
  m = reduce<L>(m, [](float a, float b) { return fmaxf(a, b); });
  // bit 0: an id of the experts', bit 1: a NaN or +inf
  float flags = (any ? 1.f : 0.f) + (bad ? 256.f : 0.f);
  flags = reduce_sum<L>(flags);  // (at most 64 of each: exact)
  bad = flags >= 256.f;
  any = flags != (bad ? floorf(flags * (1.f / 256.f)) * 256.f : 0.f);
  o.part = any && (bad || m > -INFINITY);
  const float top = m > -INFINITY ? m : 0.f;
  float total = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    o.p[v] = expf(o.p[v] - top);
    total += o.p[v];
  }
  total = reduce_sum<L>(total);
  const float inv = bad ? __builtin_nanf("") : 1.0f / total;
#pragma unroll
  for (int v = 0; v < V; ++v) o.p[v] *= inv;
  o.lse = bad ? __builtin_nanf("") : top + logf(total);
  return o;
}

// Rows of one work-group: a chunk of one sequence's tokens.
__device__ __forceinline__ Tile chunk_of(const int32_t* __restrict__ seqs, int S, int T, int at,
                                         int per) {
  if (seqs) return find_tile(seqs, S, T, at, per);
  return Tile{0, at * per, min(per, T - at * per)};
}

struct Part {  // of a chunk, after E probabilities' sums and E counts
  float z;
  int32_t n;
};

// Sums of one chunk: [E] float probabilities, [E] counts, z, n.
template <class T, int L, int V>
__global__ __launch_bounds__(kThreads) void k_balance_part(
    const T* __restrict__ logits, int64_t ld, const int32_t* __restrict__ ids,
    const int32_t* __restrict__ seqs, int S, int T_, int E, int k, int per,
    uint32_t* __restrict__ parts) {
  constexpr int G = kThreads / L;  // tokens at a time
  extern __shared__ uint32_t lds[];
  float* sums = (float*)lds;       // [G][E]
  int32_t* count = (int32_t*)(lds + G * E);
  float* zs = (float*)(count + E);
  int32_t* ns = (int32_t*)(zs + G);
  const Tile c = chunk_of(seqs, S, T_, blockIdx.x, per);
  if (c.n <= 0) return;
  const int tid = threadIdx.x, l = tid & (L - 1), group = tid / L;
  for (int e = tid; e < E; e += kThreads) count[e] = 0;
  __syncthreads();
  float sum[V] = {}, z = 0.f;
  int n = 0;
  for (int i0 = 0; i0 < c.n; i0 += G) {
    const int64_t t = c.row0 + i0 + group;
    const bool live = i0 + group < c.n;
    const Soft<V> s = soft<T, L, V>(logits + (live ? t : 0) * ld, ids + (live ? t : 0) * k, E, k, live);
    if (s.part) {
#pragma unroll
      for (int v = 0; v < V; ++v) sum[v] += s.p[v];
      z += s.lse * s.lse;
      ++n;
      for (int j = l; j < k; j += L) {
        const int id = ids[t * k + j];
        if (id >= 0 && id < E) atomicAdd(&count[id], 1);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (v * L + l < E) sums[group * E + v * L + l] = sum[v];
  if (l == 0) zs[group] = z, ns[group] = n;
  __syncthreads();
  uint32_t* out = parts + (size_t)blockIdx.x * (2 * E + 2);
  for (int e = tid; e < E; e += kThreads) {
    float p = 0.f;
#pragma unroll 4
    for (int g = 0; g < G; ++g) p += sums[g * E + e];
    out[e] = __float_as_uint(p);
    out[E + e] = (uint32_t)count[e];
  }
  if (tid == 0) {
    float p = 0.f;
    int32_t m = 0;
    for (int g = 0; g < G; ++g) p += zs[g], m += ns[g];
    out[2 * E] = __float_as_uint(p);
    out[2 * E + 1] = (uint32_t)m;
  }
}

__device__ __forceinline__ double block_sum(double v, double* buf) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
  for (int w = 0; w < (int)blockDim.x / 64; ++w) v += buf[w];
  return v;
}

// One work-group per sequence: its chunks' sums in chunk order, then the
// losses.  `split` threads share an expert's chunks.
constexpr int kJoin = 1024;
__global__ __launch_bounds__(kJoin) void k_balance_join(
    const uint32_t* __restrict__ parts, const int32_t* __restrict__ seqs, int S, int T_, int E,
    int k, int per, int chunks, float* __restrict__ loss, float* __restrict__ z,
    int32_t* __restrict__ counts, int32_t* __restrict__ tokens) {
  extern __shared__ double dlds[];
  double* buf = dlds;                // [16]
  double* ps = dlds + 16;            // [split][E]
  const int s = blockIdx.x, tid = threadIdx.x;
  int first = 0, last = chunks;
  if (seqs) {  // chunks of the sequences before this one
    int lo, hi;
    first = count_tiles(seqs, s, T_, per);
    expert_rows(seqs, s, T_, lo, hi);
    last = min(chunks, first + (hi - lo + per - 1) / per);
  }
  const size_t len = 2 * (size_t)E + 2;
  const int split = kJoin / E < 1 ? 1 : kJoin / E;
  int32_t* cs = (int32_t*)(ps + (size_t)split * E);  // [split][E]
  for (int i = tid; i < split * E; i += kJoin) {
    const int e = i % E, q = i / E;
    double p = 0.0;
    int32_t c = 0;
#pragma unroll 4
    for (int b = first + q; b < last; b += split) {
      p += (double)__uint_as_float(parts[b * len + e]);
      c += (int32_t)parts[b * len + E + e];
    }
    ps[i] = p, cs[i] = c;
  }
  double zz = 0.0, nn = 0.0;
  for (int b = first + tid; b < last; b += kJoin) {
    zz += (double)__uint_as_float(parts[b * len + 2 * E]);
    nn += (double)(int32_t)parts[b * len + 2 * E + 1];
  }
  zz = block_sum(zz, buf);
  nn = block_sum(nn, buf);
  const double inv = nn > 0.0 ? 1.0 / nn : 0.0;
  double part = 0.0;
  for (int e = tid; e < E; e += kJoin) {
    double p = 0.0;
    int32_t c = 0;
    for (int q = 0; q < split; ++q) p += ps[q * E + e], c += cs[q * E + e];
    counts[(size_t)s * E + e] = c;
    part += (double)c * inv * p * inv;
  }
  part = block_sum(part, buf);
  if (tid == 0) {
    loss[s] = (float)(part * ((double)E / k));
    z[s] = (float)(zz * inv);
    tokens[s] = (int32_t)nn;
  }
}

template <class T, int L, int V, bool ADD>
__global__ __launch_bounds__(kThreads) void k_balance_grad(
    const T* __restrict__ logits, int64_t ld, const int32_t* __restrict__ ids,
    const int32_t* __restrict__ seqs, int S, int T_, int E, int k, int per,
    const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens,
    const float* __restrict__ dloss, const float* __restrict__ dz, T* __restrict__ dl,
    int64_t ldd) {
  constexpr int G = kThreads / L;
  const Tile c = chunk_of(seqs, S, T_, blockIdx.x, per);
  if (c.n <= 0) return;
  const int tid = threadIdx.x, l = tid & (L - 1), group = tid / L;
  const int n = tokens[c.e];
  const float inv = n > 0 ? 1.0f / (float)n : 0.f;
  const float a = dloss ? dloss[c.e] * inv : 0.f, b = dz ? 2.0f * dz[c.e] * inv : 0.f;
  float f[V];
  const float unit = (float)E / (float)k * inv;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * L + l;
    f[v] = e < E ? (float)counts[(size_t)c.e * E + e] * unit : 0.f;
  }
  for (int i0 = 0; i0 < c.n; i0 += G) {
    const int64_t t = c.row0 + i0 + group;
    const bool live = i0 + group < c.n;
    const Soft<V> s = soft<T, L, V>(logits + (live ? t : 0) * ld, ids + (live ? t : 0) * k, E, k, live);
    float mean = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) mean += s.p[v] * f[v];
    mean = reduce_sum<L>(mean);
    if (!live || (ADD && !s.part)) continue;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * L + l;
      if (e >= E) continue;
      float d = s.part ? s.p[v] * (a * (f[v] - mean) + b * s.lse) : 0.f;
      if (ADD) d += to_f32(dl[t * ldd + e]);
      dl[t * ldd + e] = from_f32<T>(d);
    }
  }
}

// As in the router: a row of 16 lanes up to 256 experts, a wave beyond.
template <class F>
void with_shape(int E, F f) {
  using std::integral_constant;
  if (E <= 16)
    f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (E <= 64)
    f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  else if (E <= 128)
    f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
  else if (E <= 256)
    f(integral_constant<int, 16>{}, integral_constant<int, 16>{});
  else if (E <= 512)
    f(integral_constant<int, 64>{}, integral_constant<int, 8>{});
  else if (E <= 1024)
    f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
  else
    f(integral_constant<int, 64>{}, integral_constant<int, 32>{});
}
template <class F>
void with_type(int dtype, F f) {
  if (dtype == BITSMOE_F32)
    f(float{});
  else if (dtype == BITSMOE_F16)
    f(f16{});
  else
    f(bf16{});
}

// Tokens of a chunk: four turns of 16 tokens at a time, more where that would
// make over 512 chunks of a sequence.
int chunk_tokens(int T) {
  const int per = (T + 511) / 512;
  return per < 64 ? 64 : (per + 15) / 16 * 16;
}
int max_chunks(int T, int S) {
  const int per = chunk_tokens(T);
  return T / per + (S < T ? S : T);
}
size_t parts_bytes(int T, int S, int E) { return (size_t)max_chunks(T, S) * (2 * (size_t)E + 2) * 4; }

int sizes(int dtype, int T, int E, int k, int S) {
  if (dtype != BITSMOE_F32 && !is_half(dtype)) return fail(BITSMOE_EINVAL, "dtype=%d", dtype);
  if (E < 1 || E > kMaxExperts) return fail(BITSMOE_ESHAPE, "E=%d (1..%d)", E, kMaxExperts);
  if (k < 1 || k > kMaxSlots) return fail(BITSMOE_EINVAL, "k=%d (1..%d)", k, kMaxSlots);
  if (T < 0 || T > (1 << 30) / kMaxSlots) return fail(BITSMOE_ESHAPE, "T=%d", T);
  if (S < 1 || S > 65535) return fail(BITSMOE_ESHAPE, "S=%d sequences (1..65535)", S);
  return BITSMOE_OK;
}

}  // namespace
}  // namespace experts
}  // namespace bitsmoe

using namespace bitsmoe;
using namespace bitsmoe::experts;

extern "C" {

int bitsmoe_moe_balance_workspace_size(int T, int E, int S, size_t* bytes) {
  if (!bytes) return fail(BITSMOE_EINVAL, "bytes is null");
  const int st = sizes(BITSMOE_F32, T, E, 1, S);
  if (st) return st;
  *bytes = parts_bytes(T, S, E);
  return BITSMOE_OK;
}

int bitsmoe_moe_balance(int dtype, const void* logits, int64_t ld, const int32_t* ids,
                        const int32_t* seqs, int S, int T, int E, int k, float* loss, float* z,
                        int32_t* counts, int32_t* tokens, void* ws, size_t ws_bytes,
                        bitsmoe_stream_t stream) {
  const int st = sizes(dtype, T, E, k, S);
  if (st) return st;
  if (!seqs && S != 1) return fail(BITSMOE_EINVAL, "seqs is null with S=%d", S);
  if (ld < E) return fail(BITSMOE_ESHAPE, "a row stride is smaller than E=%d", E);
  if (!loss || !z || !counts || !tokens || (T && (!logits || !ids)))
    return fail(BITSMOE_EINVAL, "null pointer argument");
  if (parts_bytes(T, S, E) > ws_bytes || (T && !ws))
    return fail(BITSMOE_ENOSPC, "ws_bytes=%zu < %zu", ws_bytes, parts_bytes(T, S, E));
  if ((uintptr_t)ws & 3u) return fail(BITSMOE_EINVAL, "misaligned workspace");
  const int per = chunk_tokens(T), chunks = seqs ? max_chunks(T, S) : (T + per - 1) / per;
  hipStream_t q = (hipStream_t)stream;
  if (T) {
    with_type(dtype, [&](auto tag) {
      using X = decltype(tag);
      with_shape(E, [&](auto l, auto v) {
        constexpr int L = decltype(l)::value, V = decltype(v)::value, G = kThreads / L;
        const size_t lds = ((size_t)G * E + E + 2 * G) * 4;
        hipLaunchKernelGGL((k_balance_part<X, L, V>), dim3((unsigned)chunks), dim3(kThreads), lds,
                           q, (const X*)logits, ld, ids, seqs, S, T, E, k, per, (uint32_t*)ws);
      });
    });
    const int rc = launched("moe_balance sums");
    if (rc) return rc;
  }
  const int split = kJoin / E < 1 ? 1 : kJoin / E;
  const size_t lds = 16 * 8 + (size_t)split * E * 12;
  hipLaunchKernelGGL(k_balance_join, dim3((unsigned)S), dim3(kJoin), lds, q, (const uint32_t*)ws,
                     seqs, S, T, E, k, per, chunks, loss, z, counts, tokens);
  return launched("moe_balance");
}

int bitsmoe_moe_balance_grad(int dtype, const void* logits, int64_t ld, const int32_t* ids,
                             const int32_t* seqs, int S, int T, int E, int k,
                             const int32_t* counts, const int32_t* tokens, const float* dloss,
                             const float* dz, int add, void* dlogits, int64_t ldd,
                             bitsmoe_stream_t stream) {
  const int st = sizes(dtype, T, E, k, S);
  if (st) return st;
  if (!seqs && S != 1) return fail(BITSMOE_EINVAL, "seqs is null with S=%d", S);
  if (ld < E || ldd < E) return fail(BITSMOE_ESHAPE, "a row stride is smaller than E=%d", E);
  if (T == 0) return BITSMOE_OK;
  if (!logits || !ids || !counts || !tokens || !dlogits)
    return fail(BITSMOE_EINVAL, "null pointer argument");
  const int per = chunk_tokens(T), chunks = seqs ? max_chunks(T, S) : (T + per - 1) / per;
  with_type(dtype, [&](auto tag) {
    using X = decltype(tag);
    with_shape(E, [&](auto l, auto v) {
      constexpr int L = decltype(l)::value, V = decltype(v)::value;
      auto go = [&](auto more) {
        hipLaunchKernelGGL((k_balance_grad<X, L, V, decltype(more)::value>), dim3((unsigned)chunks),
                           dim3(kThreads), 0, (hipStream_t)stream, (const X*)logits, ld, ids, seqs,
                           S, T, E, k, per, counts, tokens, dloss, dz, (X*)dlogits, ldd);
      };
      if (add)
        go(std::true_type{});
      else
        go(std::false_type{});
    });
  });
  return launched("moe_balance_grad");
}

}  // extern "C"
