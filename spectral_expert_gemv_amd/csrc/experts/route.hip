// The router: the k largest logits of every token with their softmax weights,
// the gradient of the logits, and the stable grouping of the (token, slot)
// pairs by expert.
//
// p = softmax(l) over all E experts; the chosen ids are the k largest logits
// in falling order, equal logits by rising index; g_j = scale p_{id_j}, or
// scale p_{id_j} / sum_i p_{id_i} with `renorm`.  All of it in float32.
// An expert whose logit is -inf is never chosen; slots left over get id -1
// and weight 0.  A row with a NaN or a +inf has no softmax: ids -1, g NaN.
#include <type_traits>

#include "experts.h"

namespace bitsmoe {
namespace experts {
namespace {

constexpr int kMaxSlots = 64;
constexpr int kMaxExperts = 2048;
constexpr uint32_t kKeyMinusInf = 0x007FFFFFu;  // order_key(-inf); 0 is below it

// Unsigned key in the order of the floats (-0 made +0, so the two tie).
__device__ inline uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ inline float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// Reductions over groups of L lanes (16: one DPP row, whose mirrors leave the
// result in every lane; 64: the rows' results joined by two shuffles).
template <int kCtrl>
__device__ inline uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, false);
}
template <int L, class F>
__device__ inline uint32_t reduce(uint32_t v, F f) {
  v = f(v, dpp<0xB1>(v));   // quad_perm [1,0,3,2]
  v = f(v, dpp<0x4E>(v));   // quad_perm [2,3,0,1]
  v = f(v, dpp<0x141>(v));  // row_half_mirror
  v = f(v, dpp<0x140>(v));  // row_mirror
  if constexpr (L == 64) {
    v = f(v, (uint32_t)__shfl_xor((int)v, 16, 64));
    v = f(v, (uint32_t)__shfl_xor((int)v, 32, 64));
  }
  return v;
}
template <int L>
__device__ inline uint32_t reduce_max(uint32_t v) {
  return reduce<L>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int L>
__device__ inline uint32_t reduce_min(uint32_t v) {
  return reduce<L>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
template <int L>
__device__ inline float reduce_sum(float v) {
  return __uint_as_float(reduce<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// L lanes per token, V logits a lane: expert v L + lane in value v, so a
// load of all lanes is contiguous.  A choice is the largest key of the lanes'
// own largest ones, then the lowest expert that has it: about 45 instructions
// for 16 lanes (16384 tokens, 128 experts, 8 of them: 8 us for 8.4 MB).
template <class T, int L, int V>
__device__ __forceinline__ int32_t route_token(const T* __restrict__ logits, int64_t ld, int64_t t0,
                                            int T_, int E, int k, int renorm, float scale,
                                            int32_t* __restrict__ ids, float* __restrict__ g) {
  const int l = threadIdx.x & (L - 1);
  const bool live = t0 < T_;
  const int64_t t = live ? t0 : T_ - 1;  // (whole waves stay in the reductions)
  uint32_t key[V];
  uint32_t bad = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * L + l;
    key[v] = 0;
    if (e < E) {
      const float x = to_f32(logits[t * ld + e]);
      key[v] = order_key(x);
      bad |= !(x < INFINITY);
    }
  }
  bad = reduce_max<L>(bad);
  float top = 0.f, total = 0.f;
  int32_t my_id = -1;
  float my_e = 0.f;
  for (int j = 0; j < k; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = m > key[v] ? m : key[v];
    m = reduce_max<L>(m);
    uint32_t at = 0xFFFFFFFFu;
#pragma unroll
    for (int v = V - 1; v >= 0; --v) at = key[v] == m ? (uint32_t)(v * L + l) : at;
    at = reduce_min<L>(at);
    const bool there = m > kKeyMinusInf;
    if (j == 0) {
      top = there ? key_value(m) : 0.f;
      if (!renorm) {
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (key[v] > kKeyMinusInf) total += expf(key_value(key[v]) - top);
        total = reduce_sum<L>(total);
      }
    }
    if (l == j) {
      my_id = there ? (int32_t)at : -1;
      my_e = there ? expf(key_value(m) - top) : 0.f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = at == (uint32_t)(v * L + l) ? 0u : key[v];
  }
  if (renorm) total = reduce_sum<L>(my_e);
  if (live && l < k) {
    ids[t * k + l] = bad ? -1 : my_id;
    g[t * k + l] = bad ? __builtin_nanf("") : my_id >= 0 ? scale * (my_e / total) : 0.f;
  }
  return bad ? -1 : my_id;  // the l-th choice
}

template <class T, int L, int V>
__global__ __launch_bounds__(256) void k_route(const T* __restrict__ logits, int64_t ld, int T_,
                                               int E, int k, int renorm, float scale,
                                               int32_t* __restrict__ ids, float* __restrict__ g) {
  route_token<T, L, V>(logits, ld, ((int64_t)blockIdx.x * 256 + threadIdx.x) / L, T_, E, k, renorm,
                       scale, ids, g);
}

// With w = softmax over all experts and q_i = scale dg_j at i = id_j (0
// elsewhere): dl_i = w_i (q_i - sum_m w_m q_m).  With renorm w is the softmax
// over the chosen experts alone (0 at the others), as c_i exp(l_i) / sum with
// c_i how often i is among the ids.  Ids outside [0, E) take no part.
template <class T, int L, int V>
__global__ __launch_bounds__(256) void k_route_grad(const T* __restrict__ logits, int64_t ld,
                                                    const int32_t* __restrict__ ids,
                                                    const float* __restrict__ dg, int T_, int E,
                                                    int k, int renorm, float scale,
                                                    T* __restrict__ dl, int64_t ldd) {
  const int l = threadIdx.x & (L - 1);
  const int64_t t0 = ((int64_t)blockIdx.x * 256 + threadIdx.x) / L;
  const bool live = t0 < T_;
  const int64_t t = live ? t0 : T_ - 1;
  float x[V], q[V], c[V];
  uint32_t bad = 0, m = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * L + l;
    x[v] = e < E ? to_f32(logits[t * ld + e]) : -INFINITY;
    bad |= e < E && !(x[v] < INFINITY);
    q[v] = c[v] = 0.f;
  }
  for (int j = 0; j < k; ++j) {
    const int id = ids[t * k + j];
    const float d = dg[t * k + j];
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (id == v * L + l && id < E) q[v] += scale * d, c[v] += 1.f;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (!renorm) c[v] = 1.f;
    const uint32_t key = order_key(x[v]);
    if (c[v] > 0.f && key > m) m = key;
  }
  bad = reduce_max<L>(bad);
  m = reduce_max<L>(m);
  const float top = m > kKeyMinusInf ? key_value(m) : 0.f;
  float total = 0.f, mean = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    // (with repeated ids q_i already holds their sum, so the mean below
    // weighs q once and the own term c times)
    x[v] = x[v] > -INFINITY && c[v] > 0.f ? expf(x[v] - top) : 0.f;
    total += c[v] * x[v];
    mean += q[v] * x[v];
  }
  total = reduce_sum<L>(total);
  mean = reduce_sum<L>(mean);
  const float inv = total > 0.f ? 1.0f / total : 0.f;
  mean *= inv;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * L + l;
    if (live && e < E)
      dl[t * ldd + e] =
          from_f32<T>(bad ? __builtin_nanf("") : x[v] * inv * (q[v] - c[v] * mean));
  }
}

// ---------------------------------------------------------------- grouping
// Stable counting sort of P ids: pairs of expert 0 first, in pair order,
// pairs whose id lies outside [0, E) last.  A wave takes a run of consecutive
// pairs, 64 at a time: a pair's rank among the wave's 64 is the number of
// lower lanes with the same id, found by one ballot per id bit; the wave's
// counter of that id gives the place of the first.  No result depends on the
// order of atomics.  131072 pairs of 128 experts: 3 us to count, 9 to place.
__device__ inline uint64_t same_id(int id, int bits) {
  uint64_t m = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const bool s = (id >> b) & 1;
    const uint64_t v = __ballot(s);
    m &= s ? v : ~v;
  }
  return m;
}

constexpr int kIdBatch = 8;  // turns of 64 ids loaded before the first is used

// counts of one wave's run [p0, p1) into cnt[E + 1] (LDS, zeroed)
__device__ inline void count_run(const int32_t* __restrict__ ids, int p0, int p1, int E,
                                 uint32_t* cnt) {
  for (int b = p0 + (int)(threadIdx.x & 63); b < p1; b += 64 * kIdBatch) {
    int id[kIdBatch];
#pragma unroll
    for (int u = 0; u < kIdBatch; ++u) id[u] = b + 64 * u < p1 ? ids[b + 64 * u] : 0;
#pragma unroll
    for (int u = 0; u < kIdBatch; ++u)
      if (b + 64 * u < p1) atomicAdd(&cnt[id[u] >= 0 && id[u] < E ? id[u] : E], 1u);
  }
}

// scatters the run with cur[] = next place per id (LDS, this wave's own)
__device__ inline void place_run(const int32_t* __restrict__ ids, int p0, int p1, int E, int bits,
                                 uint32_t* cur, int32_t* __restrict__ order,
                                 int32_t* __restrict__ slot) {
  const int lane = threadIdx.x & 63;
  for (int b = p0; b < p1; b += 64 * kIdBatch) {
    int ids_[kIdBatch];
#pragma unroll
    for (int u = 0; u < kIdBatch; ++u) ids_[u] = b + 64 * u + lane < p1 ? ids[b + 64 * u + lane] : -1;
#pragma unroll
    for (int u = 0; u < kIdBatch; ++u) {
      const int p = b + 64 * u + lane;
      const int id = ids_[u] >= 0 && ids_[u] < E ? ids_[u] : E;
      const bool live = p < p1;
      const uint64_t m = same_id(id, bits) & __ballot(live);
      if (live) {
        const uint32_t rank = (uint32_t)__popcll(m & ((1ull << lane) - 1));
        const uint32_t base = cur[id];
        order[base + rank] = id < E ? p : -1;
        slot[p] = id < E ? (int32_t)(base + rank) : -1;
        if (rank + 1 == (uint32_t)__popcll(m)) cur[id] = base + rank + 1;
      }
      // (LDS operations of one wave complete in order: the reads of `cur`
      // above are done before the next 64 pairs' reads)
      __builtin_amdgcn_wave_barrier();
    }
  }
}

// Exclusive scan over one work-group of NW waves (NW <= 16), any NT values.
__device__ inline uint32_t block_scan(uint32_t v, uint32_t* buf, int nw) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  uint32_t inc = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t t = (uint32_t)__shfl_up((int)inc, d, 64);
    if (lane >= d) inc += t;
  }
  if (lane == 63) buf[wv] = inc;
  __syncthreads();
  uint32_t off = 0;
  for (int w = 0; w < wv && w < nw; ++w) off += buf[w];
  __syncthreads();
  return off + inc - v;
}

// All pairs in one work-group of 16 waves: dynamic LDS 16 (E + 1) words of
// counters, then 16 of scan totals.
constexpr int kOneWaves = 16;
__device__ __forceinline__ void group_one(const int32_t* __restrict__ ids, int P, int E, int bits,
                                          int32_t* __restrict__ bounds,
                                          int32_t* __restrict__ order,
                                          int32_t* __restrict__ slot) {
  extern __shared__ uint32_t lds[];
  uint32_t* buf = lds + kOneWaves * (E + 1);
  const int tid = threadIdx.x, wv = tid >> 6, n = 64 * kOneWaves;
  for (int i = tid; i < kOneWaves * (E + 1); i += n) lds[i] = 0;
  __syncthreads();
  const int per = (P + n - 1) / n * 64;  // pairs a wave, whole groups of 64
  const int p0 = min(P, wv * per), p1 = min(P, p0 + per);
  uint32_t* mine = lds + wv * (E + 1);
  count_run(ids, p0, p1, E, mine);
  __syncthreads();
  // experts in runs of n: totals scanned, then each wave's first place
  uint32_t before = 0;
  for (int e0 = 0; e0 <= E; e0 += n) {
    const int e = e0 + tid;
    uint32_t sum = 0;
    if (e <= E)
      for (int w = 0; w < kOneWaves; ++w) sum += lds[w * (E + 1) + e];
    const uint32_t ex = before + block_scan(sum, buf, kOneWaves);
    if (e <= E) {
      bounds[e] = (int32_t)ex;  // (entry E: where the pairs without expert start)
      uint32_t at = ex;
      for (int w = 0; w < kOneWaves; ++w) {
        const uint32_t c = lds[w * (E + 1) + e];
        lds[w * (E + 1) + e] = at;
        at += c;
      }
    }
    if (tid == n - 1) buf[kOneWaves] = ex + sum;
    __syncthreads();
    before = buf[kOneWaves];
    __syncthreads();
  }
  place_run(ids, p0, p1, E, bits, mine, order, slot);
}

__global__ __launch_bounds__(64 * kOneWaves) void k_group_one(const int32_t* __restrict__ ids,
                                                              int P, int E, int bits,
                                                              int32_t* __restrict__ bounds,
                                                              int32_t* __restrict__ order,
                                                              int32_t* __restrict__ slot) {
  group_one(ids, P, E, bits, bounds, order, slot);
}

// No pairs: bounds of 0, however many experts.
__global__ __launch_bounds__(256) void k_group_none(int E, int32_t* __restrict__ bounds) {
  const int e = blockIdx.x * 256 + threadIdx.x;
  if (e <= E) bounds[e] = 0;
}

// Up to 4 tokens and 64 pairs: one wave, nothing but registers.  Lane p holds
// pair p's id; a place is the number of pairs with a lower id, or the same
// and a lower index.
template <class T, int V>
__global__ __launch_bounds__(64) void k_route_group_wave(
    const T* __restrict__ logits, int64_t ld, int T_, int E, int k, int renorm, float scale,
    int32_t* __restrict__ ids, float* __restrict__ g, int32_t* __restrict__ bounds,
    int32_t* __restrict__ order, int32_t* __restrict__ slot) {
  const int lane = threadIdx.x, P = T_ * k;
  int id = route_token<T, 16, V>(logits, ld, lane / 16, T_, E, k, renorm, scale, ids, g);
  id = __shfl(id, min(lane / k * 16 + lane % k, 63), 64);
  id = id >= 0 ? id : E;
  int at = 0;
  for (int p = 0; p < P; ++p) {
    const int o = __builtin_amdgcn_readlane(id, p);
    at += o < id || (o == id && p < lane);
  }
  if (lane < P) {
    order[at] = id < E ? lane : -1;
    slot[lane] = id < E ? at : -1;
  }
  for (int e0 = 0; e0 <= E; e0 += 64) {
    int n = 0;
    for (int p = 0; p < P; ++p) n += __builtin_amdgcn_readlane(id, p) < e0 + lane;
    if (e0 + lane <= E) bounds[e0 + lane] = n;
  }
}

// Few tokens (at most kOneTokens): routing and grouping in one work-group, 64
// tokens at a time, which saves a launch.
constexpr int kOneTokens = 128;
template <class T, int V>
__global__ __launch_bounds__(64 * kOneWaves) void k_route_group_one(
    const T* __restrict__ logits, int64_t ld, int T_, int E, int k, int renorm, float scale,
    int32_t* ids, float* __restrict__ g, int bits, int32_t* __restrict__ bounds,
    int32_t* __restrict__ order, int32_t* __restrict__ slot) {
  for (int t0 = 0; t0 < T_; t0 += 64 * kOneWaves / 16)
    route_token<T, 16, V>(logits, ld, t0 + (int)threadIdx.x / 16, T_, E, k, renorm, scale, ids, g);
  __threadfence_block();  // (group_one starts with a barrier)
  group_one(ids, T_ * k, E, bits, bounds, order, slot);
}

// Many pairs: every wave of the grid counts its run into runs[unit][E + 1],
// the work-group's sums go to blocks[block][E + 1] ...
__global__ __launch_bounds__(512) void k_group_count(const int32_t* __restrict__ ids, int P, int E,
                                                     int per, uint32_t* __restrict__ runs,
                                                     uint32_t* __restrict__ blocks) {
  extern __shared__ uint32_t lds[];
  const int wv = threadIdx.x >> 6, lane = threadIdx.x & 63, nw = blockDim.x >> 6;
  const int unit = blockIdx.x * nw + wv;
  uint32_t* mine = lds + wv * (E + 1);
  for (int i = lane; i <= E; i += 64) mine[i] = 0;
  __syncthreads();
  const int p0 = (int)min((int64_t)P, (int64_t)unit * per), p1 = (int)min((int64_t)P, (int64_t)p0 + per);
  count_run(ids, p0, p1, E, mine);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += blockDim.x) {
    uint32_t sum = 0;
    for (int w = 0; w < nw; ++w) {
      const uint32_t c = lds[w * (E + 1) + e];
      runs[(size_t)(blockIdx.x * nw + w) * (E + 1) + e] = c;
      sum += c;
    }
    blocks[(size_t)blockIdx.x * (E + 1) + e] = sum;
  }
}

// ... and places it after the pairs of lower experts, of earlier work-groups,
// whose sums every work-group adds up for itself, 16 in flight, and of the
// earlier waves of its own.
__global__ __launch_bounds__(512) void k_group_place(
    const int32_t* __restrict__ ids, int P, int E, int bits, int per,
    const uint32_t* __restrict__ runs, const uint32_t* __restrict__ blocks,
    int32_t* __restrict__ bounds, int32_t* __restrict__ order, int32_t* __restrict__ slot) {
  extern __shared__ uint32_t lds[];
  const int tid = threadIdx.x, wv = tid >> 6, n = blockDim.x, nw = n >> 6;
  const int nb = gridDim.x, b0 = blockIdx.x;
  uint32_t* buf = lds + nw * (E + 1);
  uint32_t before = 0;
  for (int e0 = 0; e0 <= E; e0 += n) {
    const int e = e0 + tid;
    uint32_t sum = 0, earlier = 0, c[16], own[8];
    if (e <= E) {
#pragma unroll
      for (int w = 0; w < 8; ++w) own[w] = w < nw ? runs[(size_t)(b0 * nw + w) * (E + 1) + e] : 0;
      for (int u = 0; u < nb; u += 16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) c[i] = u + i < nb ? blocks[(size_t)(u + i) * (E + 1) + e] : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          earlier += u + i < b0 ? c[i] : 0;
          sum += c[i];
        }
      }
    }
    const uint32_t ex = before + block_scan(sum, buf, nw);
    if (e <= E) {
      if (b0 == 0) bounds[e] = (int32_t)ex;
      uint32_t at = ex + earlier;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        if (w < nw) lds[w * (E + 1) + e] = at;
        at += own[w];
      }
    }
    if (tid == n - 1) buf[nw] = ex + sum;
    __syncthreads();
    before = buf[nw];
    __syncthreads();
  }
  const int unit = b0 * nw + wv;
  const int p0 = (int)min((int64_t)P, (int64_t)unit * per), p1 = (int)min((int64_t)P, (int64_t)p0 + per);
  place_run(ids, p0, p1, E, bits, lds + wv * (E + 1), order, slot);
}

int id_bits(int E) {
  int b = 1;
  while ((E >> b) != 0) ++b;  // ids 0 .. E
  return b;
}

// One work-group takes up to 4096 pairs (4 turns a wave); its counters fit
// the LDS up to 512 experts (33 KB).
bool group_in_one(int P, int E) { return P <= 4096 && E <= 512; }

// Waves per work-group of the grid: their counters take at most 33 KB.
int grid_waves(int E) { return E <= 1024 ? 8 : 4; }
// Pairs a wave of the grid: whole groups of 64, at least 256, and at most
// about 64 work-groups, whose sums every work-group reads.
int group_per(int P, int E) {
  const long long most = 64 * grid_waves(E);
  long long per = (P + most - 1) / most;
  per = (per + 63) / 64 * 64;
  return (int)(per < 256 ? 256 : per);
}
int group_blocks(int P, int E) {
  const long long run = (long long)group_per(P, E) * grid_waves(E);
  return (int)((P + run - 1) / run);
}

int group_check(int P, int E) {
  if (P < 0 || P > (1 << 30)) return fail(BITSMOE_ESHAPE, "P=%d pairs", P);
  if (E < 1 || E > kMaxExperts) return fail(BITSMOE_ESHAPE, "E=%d (1..%d)", E, kMaxExperts);
  return BITSMOE_OK;
}

size_t group_ws(int P, int E) {
  return P == 0 || group_in_one(P, E) ? 0 : (size_t)group_blocks(P, E) * (grid_waves(E) + 1) * (E + 1) * 4;
}

int run_group(const int32_t* ids, int P, int E, int32_t* bounds, int32_t* order, int32_t* slot,
              void* ws, hipStream_t st) {
  if (P == 0) {  // (the grids below would have no work-group)
    hipLaunchKernelGGL(k_group_none, dim3((unsigned)(E / 256 + 1)), dim3(256), 0, st, E, bounds);
    return launched("moe_group");
  }
  const int bits = id_bits(E);
  if (group_in_one(P, E)) {
    const size_t lds = ((size_t)kOneWaves * (E + 1) + kOneWaves + 1) * 4;
    hipLaunchKernelGGL(k_group_one, dim3(1), dim3(64 * kOneWaves), lds, st, ids, P, E, bits, bounds,
                       order, slot);
    return launched("moe_group");
  }
  const int per = group_per(P, E), nb = group_blocks(P, E), nw = grid_waves(E);
  const size_t lds = ((size_t)nw * (E + 1) + nw + 1) * 4;
  uint32_t* runs = (uint32_t*)ws;
  uint32_t* blocks = runs + (size_t)nb * nw * (E + 1);
  hipLaunchKernelGGL(k_group_count, dim3(nb), dim3(64 * nw), lds, st, ids, P, E, per, runs, blocks);
  int rc = launched("moe_group count");
  if (rc) return rc;
  hipLaunchKernelGGL(k_group_place, dim3(nb), dim3(64 * nw), lds, st, ids, P, E, bits, per,
                     (const uint32_t*)runs, (const uint32_t*)blocks, bounds, order, slot);
  return launched("moe_group place");
}

int route_check(int dtype, int64_t ld, int T, int E, int k) {
  if (dtype != BITSMOE_F32 && !is_half(dtype)) return fail(BITSMOE_EINVAL, "dtype=%d", dtype);
  if (E < 1 || E > kMaxExperts) return fail(BITSMOE_ESHAPE, "E=%d (1..%d)", E, kMaxExperts);
  if (k < 1 || k > E || k > kMaxSlots)
    return fail(BITSMOE_EINVAL, "k=%d (1..min(E, %d)), E=%d", k, kMaxSlots, E);
  if (T < 0 || T > (1 << 30) / kMaxSlots) return fail(BITSMOE_ESHAPE, "T=%d", T);
  if (ld < E) return fail(BITSMOE_ESHAPE, "a row stride is smaller than E=%d", E);
  return BITSMOE_OK;
}

// Calls f(lanes, values) with the constants for E experts and k slots: a row
// of 16 lanes up to 256 experts and 16 slots, a wave beyond.
template <class F>
void with_shape(int E, int k, F f) {
  using std::integral_constant;
  if (E <= 256 && k <= 16) {
    if (E <= 16)
      f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
    else if (E <= 64)
      f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
    else if (E <= 128)
      f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
    else
      f(integral_constant<int, 16>{}, integral_constant<int, 16>{});
  } else if (E <= 512) {
    f(integral_constant<int, 64>{}, integral_constant<int, 8>{});
  } else if (E <= 1024) {
    f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
  } else {
    f(integral_constant<int, 64>{}, integral_constant<int, 32>{});
  }
}

}  // namespace
}  // namespace experts
}  // namespace bitsmoe

using namespace bitsmoe;
using namespace bitsmoe::experts;

extern "C" {

int bitsmoe_moe_group_workspace_size(int P, int E, size_t* bytes) {
  if (!bytes) return fail(BITSMOE_EINVAL, "bytes is null");
  const int st = group_check(P, E);
  if (st) return st;
  *bytes = group_ws(P, E);
  return BITSMOE_OK;
}

int bitsmoe_moe_group(const int32_t* ids, int P, int E, int32_t* bounds, int32_t* order,
                      int32_t* slot, void* ws, size_t ws_bytes, bitsmoe_stream_t stream) {
  const int st = group_check(P, E);
  if (st) return st;
  if (!bounds || (P && (!ids || !order || !slot))) return fail(BITSMOE_EINVAL, "null pointer argument");
  if (ws_bytes < group_ws(P, E) || (group_ws(P, E) && !ws))
    return fail(BITSMOE_ENOSPC, "ws_bytes=%zu < %zu", ws_bytes, group_ws(P, E));
  if ((uintptr_t)ws & 3u) return fail(BITSMOE_EINVAL, "misaligned workspace");
  return run_group(ids, P, E, bounds, order, slot, ws, (hipStream_t)stream);
}

int bitsmoe_moe_route(int dtype, const void* logits, int64_t ld, int T, int E, int k, int renorm,
                      float scale, int32_t* ids, float* g, int32_t* bounds, int32_t* order,
                      int32_t* slot, void* ws, size_t ws_bytes, bitsmoe_stream_t stream) {
  int st = route_check(dtype, ld, T, E, k);
  if (st) return st;
  if (T && (!logits || !ids || !g)) return fail(BITSMOE_EINVAL, "null pointer argument");
  const bool grouped = bounds || order || slot;
  if (grouped) {
    if (!bounds || (T && (!order || !slot)))
      return fail(BITSMOE_EINVAL, "bounds, order and slot go together");
    if ((st = group_check(T * k, E))) return st;
    if (ws_bytes < group_ws(T * k, E) || (group_ws(T * k, E) && !ws))
      return fail(BITSMOE_ENOSPC, "ws_bytes=%zu < %zu", ws_bytes, group_ws(T * k, E));
    if ((uintptr_t)ws & 3u) return fail(BITSMOE_EINVAL, "misaligned workspace");
  }
  // few tokens: one launch for both
  const bool one = grouped && T && T <= kOneTokens && E <= 256 && k <= 16 && group_in_one(T * k, E);
  if (T) {
    auto go = [&](auto tag) {
      using X = decltype(tag);
      with_shape(E, k, [&](auto l, auto v) {
        constexpr int L = decltype(l)::value, V = decltype(v)::value;
        if constexpr (L == 16) {
          if (one && T <= 4 && T * k <= 64) {
            hipLaunchKernelGGL((k_route_group_wave<X, V>), dim3(1), dim3(64), 0,
                               (hipStream_t)stream, (const X*)logits, ld, T, E, k, renorm, scale,
                               ids, g, bounds, order, slot);
            return;
          }
          if (one) {
            const size_t lds = ((size_t)kOneWaves * (E + 1) + kOneWaves + 1) * 4;
            hipLaunchKernelGGL((k_route_group_one<X, V>), dim3(1), dim3(64 * kOneWaves), lds,
                               (hipStream_t)stream, (const X*)logits, ld, T, E, k, renorm, scale,
                               ids, g, id_bits(E), bounds, order, slot);
            return;
          }
        }
        hipLaunchKernelGGL((k_route<X, L, V>), dim3((unsigned)(((int64_t)T * L + 255) / 256)),
                           dim3(256), 0, (hipStream_t)stream, (const X*)logits, ld, T, E, k,
                           renorm, scale, ids, g);
      });
    };
    if (dtype == BITSMOE_F32)
      go(float{});
    else if (dtype == BITSMOE_F16)
      go(f16{});
    else
      go(bf16{});
    if ((st = launched("moe_route"))) return st;
  }
  if (grouped && !one) return run_group(ids, T * k, E, bounds, order, slot, ws, (hipStream_t)stream);
  return BITSMOE_OK;
}

int bitsmoe_moe_route_grad(int dtype, const void* logits, int64_t ld, const int32_t* ids,
                           const float* dg, int T, int E, int k, int renorm, float scale,
                           void* dlogits, int64_t ldd, bitsmoe_stream_t stream) {
  const int st = route_check(dtype, ld < ldd ? ld : ldd, T, E, k);
  if (st || T == 0) return st;
  if (!logits || !ids || !dg || !dlogits) return fail(BITSMOE_EINVAL, "null pointer argument");
  auto go = [&](auto tag) {
    using X = decltype(tag);
    with_shape(E, k, [&](auto l, auto v) {
      constexpr int L = decltype(l)::value, V = decltype(v)::value;
      hipLaunchKernelGGL((k_route_grad<X, L, V>), dim3((unsigned)(((int64_t)T * L + 255) / 256)),
                         dim3(256), 0, (hipStream_t)stream, (const X*)logits, ld, ids, dg, T, E, k,
                         renorm, scale, (X*)dlogits, ldd);
    });
  };
  if (dtype == BITSMOE_F32)
    go(float{});
  else if (dtype == BITSMOE_F16)
    go(f16{});
  else
    go(bf16{});
  return launched("moe_route_grad");
}

}  // extern "C"
