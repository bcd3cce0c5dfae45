// The router's balance: per-expert counts of every sequence's tokens, the
// balance loss and the z loss, and the gradient of both with respect to the
// logits.
//
// A token takes part if one of its ids lies in [0, E) and one of its logits is
// above -inf.  Over the n tokens of a sequence that do, with p = softmax(l):
//   f_e = E / (k n) #{(t, j): id_tj = e},   P_e = 1/n sum_t p_te
//   loss = sum_e f_e P_e,   z = 1/n sum_t lse_t^2,   lse = log sum_e exp(l_te)
//   dl_te = p_te (dloss / n (f_e - sum_m p_tm f_m) + 2 dz / n lse_t)
// (f does not depend on the logits as far as a gradient goes).  softmax is
// float32, and so are the sums of a run of up to 32 tokens of a lane and of the
// work-group's lanes: at most 42 additions between a token's term and the sums of
// runs and work-groups and the losses, which are float64.  (A work-group's share
// of the tokens grows with them: in float32 to its end, z of 2^24 tokens of 257
// experts was off by 5e-5, their loss by 1.5e-5.)  No sum depends on the order of
// atomics.
#include <type_traits>

#include "experts.h"

namespace bitsmoe {
namespace experts {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxSlots = 64, kMaxExperts = 2048;
constexpr int kRunTurns = 32;    // tokens that a lane adds up in float32
constexpr int kOneMost = 1024;   // tokens of a call in one launch (one_chunk)

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

// exp(x), x <= 0: exp2 of the product with log2(e), whose rounding error and low
// part are put back by one multiplication (each within a float32 step; for -inf
// the median keeps the factor finite).
__device__ __forceinline__ float exp_below(float x) {
#pragma clang fp contract(off)
  constexpr float kHi = 1.44269502162933349609375f, kLo = 1.92596299112661746887e-8f;
  const float t = x * kHi;
  const float lo = __builtin_amdgcn_fmed3f(fmaf(x, kLo, fmaf(x, kHi, -t)), -1.0f, 1.0f);
  return __builtin_amdgcn_exp2f(t) * fmaf(lo, 0.693147182464599609375f, 1.0f);
}

// Experts l V .. l V + V - 1 of a token in lane l of its L: V consecutive
// elements from any element's alignment (the hardware takes it).
template <class T, int V>
struct Run {
  T v[V];
};
template <class T, int V>
__device__ __forceinline__ Run<T, V> load_run(const T* p, int left) {  // -inf from the left-th on
  Run<T, V> r;
  if (left >= V) {
    __builtin_memcpy(&r, p, sizeof(r));
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) r.v[v] = v < left ? p[v] : (T)-INFINITY;
  }
  return r;
}
template <class T, int V>
__device__ __forceinline__ void store_run(T* p, const Run<T, V>& r, int left) {
  if (left >= V) {
    __builtin_memcpy(p, &r, sizeof(r));
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v < left) p[v] = r.v[v];
  }
}

// What a lane reads of a token: its experts' logits, and whether one of its ids
// (every L-th) is one of the experts'.
template <class T, int L, int V>
struct Token {
  Run<T, V> x;
  int32_t id;  // the lane's first id, -1 past the k-th
  __device__ __forceinline__ void load(const T* logits, const int32_t* ids, int E, int k, bool live) {
    const int l = threadIdx.x & (L - 1);
    x = load_run<T, V>(logits + l * V, live ? E - l * V : 0);
    id = live && l < k ? ids[l] : -1;
  }
};

// The softmax of one token over its L lanes.
template <int V>
struct Soft {
  float p[V];   // probabilities; NaN everywhere for a NaN or +inf among the logits
  float lse;
  bool part;    // whether the token takes part
};

template <class T, int L, int V>
__device__ __forceinline__ Soft<V> soft(const Token<T, L, V>& in, const int32_t* ids, int E, int k,
                                        bool live) {
  const int l = threadIdx.x & (L - 1);
  Soft<V> o;
  float m = -INFINITY;
  bool bad = false, any = in.id >= 0 && in.id < E;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    o.p[v] = to_f32(in.x.v[v]);
    bad |= !(o.p[v] < INFINITY);
    m = fmaxf(m, o.p[v]);
  }
  for (int j = l + L; j < k; j += L) any |= live && ids[j] >= 0 && ids[j] < E;
  m = reduce<L>(m, [](float a, float b) { return fmaxf(a, b); });
  // (whole waves; the flags of a token's lanes are a run of the ballots)
  const int lane = threadIdx.x & 63;
  const uint64_t mine = L == 64 ? ~0ull : 0xFFFFull << (lane & 48);
  any = (__ballot(any) & mine) != 0;
  bad = (__ballot(bad) & mine) != 0;
  o.part = any && (bad || m > -INFINITY);
  const float top = m > -INFINITY ? m : 0.f;
  float total = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    o.p[v] = exp_below(o.p[v] - top);
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

// Calls f for the chunk's tokens, NT / L at a time, kFlight tokens' loads in
// flight together.
template <class T, int L, int V, int NT, class F>
__device__ __forceinline__ void each_token(const Tile& c, const T* __restrict__ logits, int64_t ld,
                                           const int32_t* __restrict__ ids, int E, int k, F f) {
  constexpr int G = NT / L;
  constexpr int kFlight = V <= 16 ? 2 : 1;
  const int group = threadIdx.x / L;
  for (int i0 = 0; i0 < c.n; i0 += G * kFlight) {
    Token<T, L, V> in[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const bool live = i0 + u * G + group < c.n;
      const int64_t t = c.row0 + (live ? i0 + u * G + group : 0);
      in[u].load(logits + t * ld, ids + t * k, E, k, live);
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      if (i0 + u * G >= c.n) break;
      const bool live = i0 + u * G + group < c.n;
      const int64_t t = c.row0 + (live ? i0 + u * G + group : 0);
      f(t, live, in[u], soft<T, L, V>(in[u], ids + t * k, E, k, live));
    }
  }
}

// Sum over a work-group of W waves, in lane 0 of wave 0 (buf: W doubles, not
// read or written by others before the next barrier).
template <int W>
__device__ __forceinline__ double block_sum(double v, double* buf) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  if (lane == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lane < W ? buf[lane] : 0.0;
#pragma unroll
  for (int d = 1; d < W; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// Words of a chunk's record: E probabilities' sums (float), E counts, z, n.
__host__ __device__ inline size_t record(int E) { return (2 * (size_t)E + 2 + 3) / 4 * 4; }

struct Outs {
  float *loss, *z;
  int32_t *counts, *tokens;
};

// Sums of one chunk, a run of tokens at a time, into its record; ONE: of a whole
// sequence, one run, whose losses it writes.  Bound by latencies and the exp
// (16384 tokens of 128 experts, 8.4 MB: 6 us; 67 tokens of 8 experts with the
// losses 4.1).
template <class T, int L, int V, int NT, bool ONE>
__global__ __launch_bounds__(NT) void k_balance_part(
    const T* __restrict__ logits, int64_t ld, const int32_t* __restrict__ ids,
    const int32_t* __restrict__ seqs, int S, int T_, int E, int k, int per,
    uint32_t* __restrict__ parts, Outs o) {
  constexpr int W = NT / 64;
  extern __shared__ double dlds[];
  double* buf = dlds;              // [W]
  float* sums = (float*)(dlds + W);  // [W][E]
  float* zs = sums + (size_t)W * E;
  int32_t* ns = (int32_t*)(zs + W);
  int32_t* count = ns + W;         // [E]
  Tile c{(int)blockIdx.x, 0, T_};
  if (!ONE) {
    c = chunk_of(seqs, S, T_, blockIdx.x, per);
    if (c.n <= 0) return;
  } else if (seqs) {
    int hi;
    expert_rows(seqs, c.e, T_, c.row0, hi);
    c.n = hi - c.row0;
  }
  const int tid = threadIdx.x, l = tid & (L - 1), wv = tid >> 6;
  for (int e = tid; e < E; e += NT) count[e] = 0;
  __syncthreads();
  constexpr int kRun = kRunTurns * (NT / L);  // tokens
  static_assert(!ONE || kOneMost <= kRun, "one run");
  constexpr int kOwn = (L * V + NT - 1) / NT;  // experts tid, tid + NT, .. of a thread
  double own[kOwn] = {}, zz = 0.0;
  int nn = 0, at = 0;
  do {
    const Tile run{c.e, c.row0 + at, ONE ? c.n : min(kRun, c.n - at)};
    float sum[V] = {}, z = 0.f;
    int n = 0;
    each_token<T, L, V, NT>(run, logits, ld, ids, E, k, [&](int64_t t, bool, const Token<T, L, V>& in, const Soft<V>& s) {
      if (s.part) {
#pragma unroll
        for (int v = 0; v < V; ++v) sum[v] += s.p[v];
        z += s.lse * s.lse;
        ++n;
        if (in.id >= 0 && in.id < E) atomicAdd(&count[in.id], 1);
        for (int j = l + L; j < k; j += L) {
          const int id = ids[t * k + j];
          if (id >= 0 && id < E) atomicAdd(&count[id], 1);
        }
      }
    });
#pragma unroll
    for (int d = L; d < 64; d <<= 1) {  // the wave's tokens
#pragma unroll
      for (int v = 0; v < V; ++v) sum[v] += __shfl_xor(sum[v], d, 64);
      z += __shfl_xor(z, d, 64);
      n += __shfl_xor(n, d, 64);
    }
    if (!ONE && at) __syncthreads();  // (the run before is read)
    if ((tid & 63) < L) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (l * V + v < E) sums[wv * E + l * V + v] = sum[v];
      if (l == 0) zs[wv] = z, ns[wv] = n;
    }
    __syncthreads();
    z = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) z += zs[w], nn += ns[w];
    zz += (double)z;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int e = tid + i * NT;
      float p = 0.f;
      if (e < E) {
#pragma unroll
        for (int w = 0; w < W; ++w) p += sums[w * E + e];
      }
      own[i] += (double)p;
    }
    at += kRun;
  } while (!ONE && at < c.n);
  double part = 0.0;
  uint32_t* out = ONE ? nullptr : parts + (size_t)blockIdx.x * record(E);
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int e = tid + i * NT;
    if (e >= E) break;
    if (ONE) {
      o.counts[(size_t)c.e * E + e] = count[e];
      part += (double)count[e] * own[i];
    } else {
      out[e] = __float_as_uint((float)own[i]);
      out[E + e] = (uint32_t)count[e];
    }
  }
  if (ONE) {
    part = block_sum<W>(part, buf);
    const double inv = nn > 0 ? 1.0 / nn : 0.0;
    if (tid == 0) {
      o.loss[c.e] = (float)(part * inv * inv * ((double)E / k));
      o.z[c.e] = (float)(zz * inv);
      o.tokens[c.e] = nn;
    }
  } else if (tid == 0) {
    out[2 * E] = __float_as_uint((float)zz);
    out[2 * E + 1] = (uint32_t)nn;
  }
}

// One work-group per sequence: its chunks' records in chunk order, then the
// losses.  A thread takes W words of a record (4, 16 bytes, where E allows it)
// of every `split`-th chunk, up to 16 of them in flight.  Bound by what one
// compute unit reads (256 records of 128 experts, 262 KB: 6.4 us).
constexpr int kJoin = 1024;
__host__ __device__ inline int join_split(int E, int W) {
  const int n = kJoin / (2 * E / W);
  return n < 1 ? 1 : n > 16 ? 16 : n;
}
template <int W>
__global__ __launch_bounds__(kJoin) void k_balance_join(
    const uint32_t* __restrict__ parts, const int32_t* __restrict__ seqs, int S, int T_, int E,
    int k, int per, int chunks, Outs o) {
  extern __shared__ double dlds[];
  const int split = join_split(E, W), q2 = 2 * E / W;  // words / W of a record's sums
  double* ps = dlds;                              // [split][E]
  int32_t* cs = (int32_t*)(ps + (size_t)split * E);  // [split][E]
  const int s = blockIdx.x, tid = threadIdx.x;
  int first = 0, last = chunks;
  if (seqs) {  // chunks of the sequences before this one
    int lo, hi;
    first = count_tiles(seqs, s, T_, per);
    expert_rows(seqs, s, T_, lo, hi);
    last = min(chunks, first + (hi - lo + per - 1) / per);
  }
  const size_t len = record(E);
  struct Words {
    uint32_t w[W];
  };
  double zz = 0.0, nn = 0.0;
  if (tid < 64)
    for (int b = first + tid; b < last; b += 64) {
      zz += (double)__uint_as_float(parts[b * len + 2 * E]);
      nn += (double)(int32_t)parts[b * len + 2 * E + 1];
    }
  for (int i = tid; i < split * q2; i += kJoin) {
    const int q = i / q2, j = (i - q * q2) * W;
    const bool whole = j >= E;  // counts
    double p[W] = {};
    int32_t c[W] = {};
    constexpr int kFlight = 16;
    const uint32_t* at = parts + (size_t)(first + q) * len + j;
    for (int b0 = first + q; b0 < last; b0 += split * kFlight) {
      Words x[kFlight];
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        x[u] = Words{};
        if (b0 + u * split < last) __builtin_memcpy(&x[u], __builtin_assume_aligned(at, 4 * W), sizeof(Words));
        at += split * len;
      }
#pragma unroll
      for (int u = 0; u < kFlight; ++u)
#pragma unroll
        for (int v = 0; v < W; ++v) {
          if (whole)
            c[v] += (int32_t)x[u].w[v];
          else
            p[v] += (double)__uint_as_float(x[u].w[v]);
        }
    }
#pragma unroll
    for (int v = 0; v < W; ++v) {
      if (whole)
        cs[q * E + j - E + v] = c[v];
      else
        ps[q * E + j + v] = p[v];
    }
  }
  __syncthreads();
  if (tid >= 64) return;
  double part = 0.0;
  for (int e = tid; e < E; e += 64) {
    double p = 0.0;
    int32_t c = 0;
#pragma unroll 8
    for (int q = 0; q < split; ++q) p += ps[q * E + e], c += cs[q * E + e];
    o.counts[(size_t)s * E + e] = c;
    part += (double)c * p;
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const double a = __shfl_xor(part, d, 64), b = __shfl_xor(zz, d, 64), n = __shfl_xor(nn, d, 64);
    part += a, zz += b, nn += n;
  }
  if (tid == 0) {
    const double inv = nn > 0.0 ? 1.0 / nn : 0.0;
    o.loss[s] = (float)(part * inv * inv * ((double)E / k));
    o.z[s] = (float)(zz * inv);
    o.tokens[s] = (int32_t)nn;
  }
}

// Two tokens a lane: 16384 tokens of 128 experts, 16.8 MB, 9 us (four tokens 9,
// and 4096 of 64 experts 6.4 instead of 5.2; one 10).
template <class T, int L, int V, bool ADD>
__global__ __launch_bounds__(kThreads) void k_balance_grad(
    const T* __restrict__ logits, int64_t ld, const int32_t* __restrict__ ids,
    const int32_t* __restrict__ seqs, int S, int T_, int E, int k, int per,
    const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens,
    const float* __restrict__ dloss, const float* __restrict__ dz, T* __restrict__ dl,
    int64_t ldd) {
  const Tile c = chunk_of(seqs, S, T_, blockIdx.x, per);
  if (c.n <= 0) return;
  const int l = threadIdx.x & (L - 1);
  const int n = tokens[c.e];
  const float inv = n > 0 ? 1.0f / (float)n : 0.f;
  const float a = dloss ? dloss[c.e] * inv : 0.f, b = dz ? 2.0f * dz[c.e] * inv : 0.f;
  float f[V];
  const float unit = (float)E / (float)k * inv;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = l * V + v;
    f[v] = e < E ? (float)counts[(size_t)c.e * E + e] * unit : 0.f;
  }
  each_token<T, L, V, kThreads>(c, logits, ld, ids, E, k, [&](int64_t t, bool live, const Token<T, L, V>&, const Soft<V>& s) {
    float mean = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) mean += s.p[v] * f[v];
    mean = reduce_sum<L>(mean);
    if (!live || (ADD && !s.part)) return;
    T* to = dl + t * ldd + l * V;
    Run<T, V> d;
    if (ADD) d = load_run<T, V>(to, E - l * V);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float g = s.part ? s.p[v] * (a * (f[v] - mean) + b * s.lse) : 0.f;
      if (ADD) g += to_f32(d.v[v]);
      d.v[v] = from_f32<T>(g);
    }
    store_run<T, V>(to, d, E - l * V);
  });
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

// Tokens of a chunk: two turns of 32 tokens at a time, more where that would
// make over 512 chunks of a sequence.
int chunk_tokens(int T) {
  const int per = (T + 511) / 512;
  return per < 64 ? 64 : (per + 31) / 32 * 32;
}
// A work-group of 1024 lanes per sequence, one launch: for few tokens, and a few
// more of sequences that are short on average.  (us by it and by two launches,
// which also take the host 4 us longer: 67 tokens 4.2 and 8, 256 of 128 experts
// 8.9 and 8, 512 14 and 8, whatever sequence has them.)
constexpr int kOneTokens = 256, kOneMean = 128;
bool one_chunk(int T, int E, int S) {
  return T >= 1 && E <= 256 && (T <= kOneTokens || (T <= kOneMost && T <= (long long)kOneMean * S));
}
constexpr int kGradTokens = 32;  // of a work-group of the gradient: two turns
int max_chunks(int T, int S) {
  const int per = chunk_tokens(T);
  return T / per + (S < T ? S : T);
}
size_t parts_bytes(int T, int S, int E) {
  return one_chunk(T, E, S) ? 0 : (size_t)max_chunks(T, S) * record(E) * 4;
}

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
  if (parts_bytes(T, S, E) > ws_bytes || (parts_bytes(T, S, E) && !ws))
    return fail(BITSMOE_ENOSPC, "ws_bytes=%zu < %zu", ws_bytes, parts_bytes(T, S, E));
  if ((uintptr_t)ws & 3u) return fail(BITSMOE_EINVAL, "misaligned workspace");
  const int per = chunk_tokens(T), chunks = seqs ? max_chunks(T, S) : (T + per - 1) / per;
  const Outs o{loss, z, counts, tokens};
  hipStream_t q = (hipStream_t)stream;
  const bool one = one_chunk(T, E, S);
  if (T) {
    with_type(dtype, [&](auto tag) {
      using X = decltype(tag);
      with_shape(E, [&](auto l, auto v) {
        constexpr int L = decltype(l)::value, V = decltype(v)::value;
        auto go = [&](auto threads, auto one_) {
          constexpr int NT = decltype(threads)::value, W = NT / 64;
          constexpr bool ONE = decltype(one_)::value;
          const size_t lds = W * 8 + ((size_t)W * E + 2 * W + E) * 4;
          hipLaunchKernelGGL((k_balance_part<X, L, V, NT, ONE>), dim3((unsigned)(ONE ? S : chunks)),
                             dim3(NT), lds, q, (const X*)logits, ld, ids, seqs, S, T, E, k,
                             per, (uint32_t*)ws, o);
        };
        using std::integral_constant;
        if constexpr (L == 16) {
          if (one)
            go(integral_constant<int, 1024>{}, std::true_type{});
          else
            go(integral_constant<int, 512>{}, std::false_type{});
        } else {
          go(integral_constant<int, 256>{}, std::false_type{});
        }
      });
    });
    const int rc = launched("moe_balance sums");
    if (rc || one) return rc;
  }
  auto join = [&](auto w) {
    constexpr int W = decltype(w)::value;
    const size_t lds = (size_t)join_split(E, W) * E * 12;
    hipLaunchKernelGGL((k_balance_join<W>), dim3((unsigned)S), dim3(kJoin), lds, q,
                       (const uint32_t*)ws, seqs, S, T, E, k, per, chunks, o);
  };
  if (E % 4 == 0 && ((uintptr_t)ws & 15u) == 0)
    join(std::integral_constant<int, 4>{});
  else
    join(std::integral_constant<int, 1>{});
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
  constexpr int per = kGradTokens;
  const unsigned chunks = (unsigned)(seqs ? T / per + (S < T ? S : T) : (T + per - 1) / per);
  with_type(dtype, [&](auto tag) {
    using X = decltype(tag);
    with_shape(E, [&](auto l, auto v) {
      constexpr int L = decltype(l)::value, V = decltype(v)::value;
      auto go = [&](auto more) {
        hipLaunchKernelGGL((k_balance_grad<X, L, V, decltype(more)::value>), dim3(chunks),
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
