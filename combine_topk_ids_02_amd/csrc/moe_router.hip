// The router of an expert-parallel layer and the loss that balances it: HIP
// kernels for CDNA4 (gfx950, wave64) behind include/moe_dispatch.h.
//
// Pages cited (title, section):
//  [A2A]  "A2A backends" page, vincentzed.com/writing/a2a-backends
//  [EP]   "Beyond One GPU: Tensor, Pipeline and Expert Parallelism, and Split
//         Prefill and Decode"
//
// Kernels
//  route_tokens    one wave per token: its logits in registers, k rounds of a
//                  wave maximum for the choice, the weights ([A2A] sec 1.1:
//                  the router picks k of the E experts and a weight for each)
//  route_gradient  one wave per token: the gradient of its logits from the
//                  weights' gradient and from the balance loss's
//  balance_tiles   one workgroup per tile of tokens: the sums of the scores
//                  and the pairs of each expert, sequence by sequence
//  balance_join    one workgroup per sequence: joins the tiles' sums, the loss
//                  ([EP]: the busiest GPU's experts set the time of a layer)
// All of them read the logits once and are bound by that (and by the launch,
// for a decode batch). Nothing depends on the order in which waves run.

#include "moe_common.h"

namespace {

using namespace moe;

constexpr int kBlock = 256;
constexpr int kWavesPerBlock = kBlock / kWave;
constexpr int kMaxSequences = 1 << 16;

// Expert e = 64 * i + lane lies in register i of lane e % 64; V registers.
template <typename Tz, int V>
__device__ __forceinline__ void load_logits(const Tz* row, int E, float (&z)[V]) {
  const int lane = lane_id();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * kWave + lane;
    z[i] = e < E ? float(row[e]) : -INFINITY;
  }
}

// 1 / (1 + e^-z) rounded to float from 64 bits: a choice by scores compares
// values whose last bit decides, so it is the nearest float, not one of two.
__device__ __forceinline__ float sigmoid_nearest(float z) {
  return float(1.0 / (1.0 + exp(-double(z))));
}

struct RouteArgs {
  const void* logits;
  const float* bias;
  const uint8_t* mask;
  int32_t* ids;
  float* weights;
  int32_t* err;
  int T, E, k;
  int renorm;
  float scale;
  int groups, top_groups;
};

// Keeps the experts of the best groups. Lanes [g * L, g * L + L) find the two
// best keys of group g (L = 64 / groups rounded down to a power of two), the
// group's score is their sum; a group is kept when fewer than top_groups are
// better (a lower index wins a tie).
template <int V>
__device__ __forceinline__ void keep_groups(float (&key)[V], float* lds, int E, int groups,
                                            int top_groups) {
  const int lane = lane_id();
  const int per = E / groups;
  int L = kWave;
  while (L * groups > kWave) L >>= 1;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i * kWave + lane < E) lds[i * kWave + lane] = key[i];
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  const int g = lane / L, sub = lane % L;
  float a = -INFINITY, b = -INFINITY;  // the two best
  if (g < groups)
    for (int e = sub; e < per; e += L) {
      const float v = lds[g * per + e];
      b = fmaxf(b, fminf(a, v));
      a = fmaxf(a, v);
    }
  for (int s = 1; s < L; s <<= 1) {
    const float a2 = __shfl_xor(a, s), b2 = __shfl_xor(b, s);
    b = fmaxf(fminf(a, a2), fmaxf(b, b2));
    a = fmaxf(a, a2);
  }
  const float score = b > -INFINITY ? a + b : a;
  int better = 0;
  for (int o = 0; o < groups; ++o) {
    const float so = read_lane(score, o * L);
    better += (so > score || (so == score && o < g)) ? 1 : 0;
  }
  const uint64_t kept = __ballot(g < groups && better < top_groups);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * kWave + lane;
    if (e < E && !((kept >> (e / per * L)) & 1)) key[i] = -INFINITY;
  }
  __builtin_amdgcn_wave_barrier();
}

// One wave per token. Each of k rounds takes the wave's maximum (a lane's own
// over its V registers, then 6 steps across lanes), finds its holders with a
// ballot per register (the first set bit of the first register that has one is
// the lowest expert id among equal keys) and strikes that one out.
template <typename Tz, int V, bool kSigmoid, bool kKeyed>
__global__ __launch_bounds__(kBlock) void route_tokens(RouteArgs a) {
  extern __shared__ float lds_all[];
  const int lane = lane_id();
  const int wave = wave_in_block();
  const int64_t t = (int64_t)blockIdx.x * kWavesPerBlock + wave;
  if (t >= a.T) return;
  const int E = a.E, k = a.k;
  bool routed = !a.mask || a.mask[t];
  float z[V], key[V];
  int chosen = 0;      // experts found
  int id = -1;         // lane j: the expert of slot j
  float picked = 0.0f; // lane j: its key
  const Tz* row = static_cast<const Tz*>(a.logits) + t * E;
  if (routed) {
    load_logits<Tz, V>(row, E, z);
    bool bad = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = z[i];
      if (kKeyed) {
        const int e = i * kWave + lane;
        const float s = sigmoid_nearest(z[i]) + (a.bias && e < E ? a.bias[e] : 0.0f);
        key[i] = z[i] == -INFINITY ? -INFINITY : s;
      }
      bad |= !(z[i] < INFINITY) || !(key[i] < INFINITY);
    }
    if (__ballot(bad)) {
      if (lane == 0) flag_error(a.err, MOE_ERRBIT_BAD_LOGIT);
      routed = false;
    }
  }
  if (routed) {
    if (kKeyed && a.groups > 1)
      keep_groups<V>(key, lds_all + wave * E, E, a.groups, a.top_groups);
    float total = 0.0f;
    float top = 0.0f;
    for (int j = 0; j < k; ++j) {
      float m = key[0];
#pragma unroll
      for (int i = 1; i < V; ++i) m = fmaxf(m, key[i]);
      m = wave_max(m);
      if (m == -INFINITY) break;
      int at = -1;
      uint64_t hit = 0;
#pragma unroll
      for (int i = V - 1; i >= 0; --i) {
        const uint64_t b = __ballot(key[i] == m);
        if (b) {
          at = i;
          hit = b;
        }
      }
      const int win = __ffsll((unsigned long long)hit) - 1;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == at && lane == win) key[i] = -INFINITY;
      if (lane == j) {
        id = at * kWave + win;
        picked = m;
      }
      if (j == 0) top = m;
      ++chosen;
    }
    const bool mine = lane < chosen;
    float w = 0.0f;
    if (kSigmoid) {
      // the scores times e^-m, m = min(0, largest chosen logit): no chosen
      // score underflows against another
      const float zj = kKeyed ? (mine ? float(row[id]) : -INFINITY) : (mine ? picked : -INFINITY);
      const float m = a.renorm ? fminf(0.0f, row_max(zj)) : 0.0f;
      if (mine) {
        const float en = expf(-fabsf(zj));
        w = zj >= 0.0f ? 1.0f / (1.0f + en) : expf(zj - m) / (1.0f + en);
      }
    } else {
      if (mine) w = expf(picked - top);
      if (!a.renorm) {
#pragma unroll
        for (int i = 0; i < V; ++i) total += expf(z[i] - top);
        total = wave_sum(total);
      }
    }
    if (a.renorm) total = row_sum(w);
    if (kSigmoid && !a.renorm) total = 1.0f;
    picked = mine ? w / total * a.scale : 0.0f;
  }
  if (lane < k) {
    const bool mine = lane < chosen;
    a.ids[t * k + lane] = mine ? id : -1;
    a.weights[t * k + lane] = mine ? picked : 0.0f;
  }
}

// ---------------------------------------------------------------------------
// Balance loss

// The sequence of token t: the first s with offsets[s + 1] > t (S when none),
// by bisection; whatever the offsets hold, the answer is in [0, S].
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int S, int64_t t) {
  int lo = 0, hi = S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (offsets[mid + 1] > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

struct BalanceArgs {
  const void* logits;
  const int32_t* ids;
  const int32_t* offsets;  // NULL: one sequence of all tokens
  float* sums;             // [(tiles + S) * E] sums of the scores
  int32_t* pairs;          // [(tiles + S) * E] pairs
  int32_t* used;           // [tiles + S] tokens with an expert
  float* loss;
  int32_t* counts;
  int32_t* tokens;
  float* mean;
  int32_t* err;
  int T, E, k, S, tile;
};

// A token's scores scaled to a sum of one: softmax, or sigmoid over the sum
// of sigmoids (times e^-m as in route_tokens). Experts past E give 0.
template <int V, bool kSigmoid>
__device__ __forceinline__ void shares(const float (&z)[V], float (&p)[V]) {
  float m = z[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = fmaxf(m, z[i]);
  m = wave_max(m);
  if (kSigmoid) m = fminf(m, 0.0f);
  if (m == -INFINITY) m = 0.0f;  // no expert has a score: all shares are 0
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (kSigmoid) {
      const float en = expf(-fabsf(z[i]));
      p[i] = (z[i] >= 0.0f ? 1.0f : expf(z[i] - m)) / (1.0f + en);
    } else {
      p[i] = expf(z[i] - m);
    }
    sum += p[i];
  }
  sum = wave_sum(sum);
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) p[i] *= inv;
}

constexpr int kTileThreads = 1024;
constexpr int kTileWaves = kTileThreads / kWave;

// Whether a wave's token has an expert; counts its pairs in LDS.
__device__ __forceinline__ bool token_used(const BalanceArgs& a, int64_t t, int* pairs) {
  const int lane = lane_id();
  const int id = lane < a.k ? a.ids[t * a.k + lane] : -1;
  const bool ok = id >= 0 && id < a.E;
  if (__ballot(id < -1 || id >= a.E) && lane == 0) flag_error(a.err, MOE_ERRBIT_BAD_ID);
  if (ok) atomicAdd(pairs + id, 1);  // integers: any order gives the same count
  return __ballot(ok) != 0;
}

// One workgroup per tile of tokens, one wave per token in turn; the scores are
// summed per lane in registers. Where a sequence ends within the tile, the
// sums so far go to the slot tile + sequence (increasing along the tokens, so
// no two pairs of them share one) and start anew.
template <typename Tz, int V, bool kSigmoid>
__global__ __launch_bounds__(kTileThreads) void balance_tiles(BalanceArgs a) {
  extern __shared__ float lds_all[];
  const int E = a.E;
  int* pairs = reinterpret_cast<int*>(lds_all);  // [E]
  int* used = pairs + E;                         // [1]
  float* part = lds_all + E + 1;                 // [waves / 2 * E]
  const int wave = wave_in_block(), lane = lane_id();
  const int64_t begin = (int64_t)blockIdx.x * a.tile;
  const int64_t end = min(begin + a.tile, (int64_t)a.T);
  int s = a.offsets ? sequence_of(a.offsets, a.S, begin) : 0;
  for (; s < a.S; ++s) {
    const int64_t first = a.offsets ? max((int64_t)a.offsets[s], begin) : begin;
    const int64_t last = a.offsets ? min((int64_t)a.offsets[s + 1], end) : end;
    if (first >= end) break;
    if (first >= last) continue;
    for (int e = threadIdx.x; e <= E; e += kTileThreads) pairs[e] = 0;
    __syncthreads();
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = 0.0f;
    int n = 0;
    for (int64_t t = first + wave; t < last; t += kTileWaves) {
      if (!token_used(a, t, pairs)) continue;
      ++n;
      float z[V], p[V];
      load_logits<Tz, V>(static_cast<const Tz*>(a.logits) + t * E, E, z);
      shares<V, kSigmoid>(z, p);
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] += p[i];
    }
    if (lane == 0 && n) atomicAdd(used, n);
    // the upper half of the waves hands its sums to the lower half, whose
    // are then added up in wave order (half the LDS of all of them at once)
    constexpr int kHalf = kTileWaves / 2;
    if (wave >= kHalf) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i * kWave + lane < E) part[(wave - kHalf) * E + i * kWave + lane] = sum[i];
    }
    __syncthreads();
    if (wave < kHalf) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i * kWave + lane < E) part[wave * E + i * kWave + lane] += sum[i];
    }
    __syncthreads();
    const int64_t slot = (int64_t)blockIdx.x + s;
    for (int e = threadIdx.x; e < E; e += kTileThreads) {
      float total = 0.0f;
      for (int w = 0; w < kHalf; ++w) total += part[w * E + e];
      a.sums[slot * E + e] = total;
      a.pairs[slot * E + e] = pairs[e];
    }
    if (threadIdx.x == 0) a.used[slot] = *used;
    __syncthreads();
  }
}

// One workgroup per sequence. The tiles' sums of a column are added in tile
// order, in 64 bits, by as many threads as there are columns times slices.
__global__ __launch_bounds__(kTileThreads) void balance_join(BalanceArgs a) {
  __shared__ double lds_sum[kTileThreads];
  __shared__ int lds_pairs[kTileThreads];
  __shared__ int lds_used;
  const int E = a.E, s = blockIdx.x, tid = threadIdx.x;
  int64_t first = a.offsets ? a.offsets[s] : 0, last = a.offsets ? a.offsets[s + 1] : a.T;
  if (first < 0 || last > a.T || first > last) {
    if (tid == 0) flag_error(a.err, MOE_ERRBIT_BAD_SEQ);
    first = last = 0;
  }
  const int64_t w0 = first / a.tile;
  const int64_t w1 = last > first ? (last - 1) / a.tile + 1 : w0;
  if (tid == 0) lds_used = 0;
  __syncthreads();
  for (int64_t w = w0 + tid; w < w1; w += kTileThreads) atomicAdd(&lds_used, a.used[w + s]);
  const int slices = kTileThreads / E;  // E <= 1024
  const int e = tid % E, slice = tid / E;
  double sum = 0.0;
  int pairs = 0;
  if (slice < slices)
    for (int64_t w = w0 + slice; w < w1; w += slices) {
      sum += a.sums[(w + s) * E + e];
      pairs += a.pairs[(w + s) * E + e];
    }
  lds_sum[tid] = sum;
  lds_pairs[tid] = pairs;
  __syncthreads();
  const int n = lds_used;
  double term = 0.0;
  if (tid < E) {
    for (int q = 1; q < slices; ++q) {
      sum += lds_sum[q * E + e];
      pairs += lds_pairs[q * E + e];
    }
    const double mean = n > 0 ? sum / n : 0.0;
    a.counts[(int64_t)s * E + e] = pairs;
    a.mean[(int64_t)s * E + e] = float(mean);
    term = mean * pairs;
  }
  __syncthreads();
  lds_sum[tid] = term;
  __syncthreads();
  for (int h = kTileThreads / 2; h > 0; h >>= 1) {
    if (tid < h) lds_sum[tid] += lds_sum[tid + h];
    __syncthreads();
  }
  if (tid == 0) {
    a.tokens[s] = n;
    a.loss[s] = n > 0 ? float(lds_sum[0] * E / (double(a.k) * n)) : 0.0f;
  }
}

// ---------------------------------------------------------------------------
// Gradient

struct GradArgs {
  const void* logits;
  const int32_t* ids;
  const float* d_weights;  // NULL: no gradient of the weights
  const float* d_loss;     // [S], NULL: no balance loss
  const int32_t* counts;   // [S * E]
  const int32_t* tokens;   // [S]
  const int32_t* offsets;  // NULL: one sequence of all tokens
  void* d_logits;
  int32_t* err;
  int T, E, k, S;
  int renorm;
  float scale;
};

// With s the scores, inner = 1 for softmax and 1 - s for sigmoid:
//  renormalised weights  q_j = s_j / sum s:  dz_(e_j) += inner q_j (g_j - sum q g)
//  raw sigmoid           dz_(e_j) += inner s_j g_j
//  raw softmax, balance  dz_e += inner p_e (u_e - sum p u), p the scores scaled
//                        to a sum of one, u_e the gradient of p_e
// For the balance loss u_e = d E n_e / (k T'^2). One number taken off every u
// changes nothing in u_e - sum p u, so k T' / E is taken off n_e first: what
// is left to cancel is the imbalance, not the counts.
template <typename Tz, int V, bool kSigmoid>
__global__ __launch_bounds__(kBlock) void route_gradient(GradArgs a) {
  const int lane = lane_id();
  const int64_t t = (int64_t)blockIdx.x * kWavesPerBlock + wave_in_block();
  if (t >= a.T) return;
  const int E = a.E, k = a.k;
  const Tz* row = static_cast<const Tz*>(a.logits) + t * E;
  Tz* out = static_cast<Tz*>(a.d_logits) + t * E;
  const int id = lane < k ? a.ids[t * k + lane] : -1;
  const bool ok = id >= 0 && id < E;
  if (__ballot(id < -1 || id >= E) && lane == 0) flag_error(a.err, MOE_ERRBIT_BAD_ID);
  const bool used = __ballot(ok) != 0;
  float d[V];
#pragma unroll
  for (int i = 0; i < V; ++i) d[i] = 0.0f;
  int s = 0;
  bool inside = used && a.d_loss;
  if (inside && a.offsets) {
    s = sequence_of(a.offsets, a.S, t);
    inside = s < a.S && a.offsets[s] <= t;
  }
  if (used) {
    float z[V];
    load_logits<Tz, V>(row, E, z);
    const float g = ok && a.d_weights ? a.d_weights[t * k + lane] * a.scale : 0.0f;
    const bool dense = !kSigmoid && !a.renorm && a.d_weights;
    float part = 0.0f;  // lane j: what slot j adds to its expert
    if (a.d_weights) {
      const float zj = ok ? float(row[id]) : -INFINITY;
      float q = 0.0f;
      if (kSigmoid) {
        const float m = a.renorm ? fminf(0.0f, row_max(zj)) : 0.0f;
        const float en = expf(-fabsf(zj));
        if (zj > -INFINITY) q = (zj >= 0.0f ? 1.0f : expf(zj - m)) / (1.0f + en);
        if (a.renorm) {
          const float sum = row_sum(q);
          q = sum > 0.0f ? q / sum : 0.0f;
        }
        const float inner = (zj >= 0.0f ? en : 1.0f) / (1.0f + en);
        part = inner * q * (g - (a.renorm ? row_sum(q * g) : 0.0f));
      } else if (a.renorm) {
        const float m = row_max(zj);
        if (ok && m > -INFINITY) q = expf(zj - m);
        const float sum = row_sum(q);
        q = sum > 0.0f ? q / sum : 0.0f;
        part = q * (g - row_sum(q * g));
      } else {
        part = g;
      }
      if (!ok) part = 0.0f;
    }
    float u[V];
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] = 0.0f;
    if (a.d_weights) {
      for (int j = 0; j < k; ++j) {
        const int e = read_lane(id, j);
        const float v = read_lane(part, j);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i * kWave + lane == e) u[i] += v;
      }
    }
    if (!dense) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        d[i] = u[i];
        u[i] = 0.0f;
      }
    }
    if (inside) {
      const int n = a.tokens[s];
      const float rate =
          n > 0 ? float(double(a.d_loss[s]) * E / (double(k) * double(n) * double(n))) : 0.0f;
      const float off = float(double(k) * n / E);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = i * kWave + lane;
        if (e < E) u[i] += rate * (float(a.counts[(int64_t)s * E + e]) - off);
      }
    }
    if (dense || inside) {
      float p[V];
      shares<V, kSigmoid>(z, p);
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) dot += p[i] * u[i];
      dot = wave_sum(dot);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float v = p[i] * (u[i] - dot);
        if (kSigmoid) v *= 1.0f / (1.0f + expf(z[i]));
        d[i] += v;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * kWave + lane;
    if (e < E) out[e] = Tz(d[i]);
  }
}

// ---------------------------------------------------------------------------
// Host side

size_t type_size(int type) { return type == MOE_TYPE_F32 ? 4 : 2; }

bool router_ok(const moe_shape_t* sh, const moe_router_t* r, int type) {
  if (!shape_ok(sh) || !r) return false;
  if (type != MOE_TYPE_F32 && type != MOE_TYPE_BF16 && type != MOE_TYPE_F16) return false;
  if (r->scoring != MOE_SCORE_SOFTMAX && r->scoring != MOE_SCORE_SIGMOID) return false;
  if (r->renorm != 0 && r->renorm != 1) return false;
  if (!(r->scale - r->scale == 0.0f)) return false;  // finite
  if (r->groups < 1 || r->groups > kWave || sh->E % r->groups != 0) return false;
  if (r->top_groups < 1 || r->top_groups > r->groups) return false;
  if (r->scoring == MOE_SCORE_SOFTMAX && r->groups > 1) return false;
  return true;
}

// Calls fn<Tz, V>: V registers of 64 experts each.
template <template <typename, int> class F, typename Tz, typename... Args>
void by_experts(int E, Args&&... args) {
  const int v = (E + kWave - 1) / kWave;
  if (v <= 1) return F<Tz, 1>::go(args...);
  if (v <= 2) return F<Tz, 2>::go(args...);
  if (v <= 4) return F<Tz, 4>::go(args...);
  if (v <= 6) return F<Tz, 6>::go(args...);
  if (v <= 8) return F<Tz, 8>::go(args...);
  return F<Tz, 16>::go(args...);
}

template <template <typename, int> class F, typename... Args>
void by_type(int type, int E, Args&&... args) {
  if (type == MOE_TYPE_F32) return by_experts<F, float>(E, args...);
  if (type == MOE_TYPE_BF16) return by_experts<F, __bf16>(E, args...);
  return by_experts<F, _Float16>(E, args...);
}

int token_blocks(int T) { return (T + kWavesPerBlock - 1) / kWavesPerBlock; }

template <typename Tz, int V>
struct RouteLaunch {
  static void go(hipStream_t st, const RouteArgs& a, int scoring) {
    const dim3 grid(token_blocks(a.T));
    const bool keyed = scoring == MOE_SCORE_SIGMOID && (a.bias || a.groups > 1);
    const size_t lds = a.groups > 1 ? size_t(kWavesPerBlock) * a.E * 4 : 0;
    if (keyed)
      route_tokens<Tz, V, true, true><<<grid, kBlock, lds, st>>>(a);
    else if (scoring == MOE_SCORE_SIGMOID)
      route_tokens<Tz, V, true, false><<<grid, kBlock, 0, st>>>(a);
    else
      route_tokens<Tz, V, false, false><<<grid, kBlock, 0, st>>>(a);
  }
};

template <typename Tz, int V>
struct GradLaunch {
  static void go(hipStream_t st, const GradArgs& a, int scoring) {
    const dim3 grid(token_blocks(a.T));
    if (scoring == MOE_SCORE_SIGMOID)
      route_gradient<Tz, V, true><<<grid, kBlock, 0, st>>>(a);
    else
      route_gradient<Tz, V, false><<<grid, kBlock, 0, st>>>(a);
  }
};

template <typename Tz, int V>
struct BalanceLaunch {
  static void go(hipStream_t st, const BalanceArgs& a, int scoring, int tiles) {
    const size_t lds = (size_t(a.E) * (kTileWaves / 2 + 1) + 1) * 4;
    if (scoring == MOE_SCORE_SIGMOID)
      balance_tiles<Tz, V, true><<<tiles, kTileThreads, lds, st>>>(a);
    else
      balance_tiles<Tz, V, false><<<tiles, kTileThreads, lds, st>>>(a);
  }
};

// Tiles of the balance loss: at most 128 of them, of 32 tokens or more.
constexpr int kMaxTiles = 128;
int balance_tile(int T) {
  const int least = (T + kMaxTiles - 1) / kMaxTiles;
  return std::max(32, (least + kTileWaves - 1) / kTileWaves * kTileWaves);
}
int balance_tile_count(int T) {
  const int tile = balance_tile(T);
  return (T + tile - 1) / tile;
}

}  // namespace

extern "C" {

int moe_route(const moe_shape_t* shape, const moe_router_t* router, int logits_type,
              const void* logits, const float* bias, const uint8_t* token_mask, int32_t* topk_ids,
              float* topk_weights, int32_t* err_word, void* stream) {
  if (!router_ok(shape, router, logits_type)) return MOE_ERR_ARG;
  if (bias && router->scoring == MOE_SCORE_SOFTMAX) return MOE_ERR_ARG;
  if (shape->T == 0) return MOE_OK;
  if (!logits || !topk_ids || !topk_weights) return MOE_ERR_ARG;
  if (!aligned(logits, type_size(logits_type)) || !aligned(bias, 4) || !aligned(topk_ids, 4) ||
      !aligned(topk_weights, 4))
    return MOE_ERR_ARG;
  const RouteArgs a{logits, bias, token_mask, topk_ids, topk_weights, err_word, shape->T,
                    shape->E, shape->k, router->renorm, router->scale, router->groups,
                    router->top_groups};
  by_type<RouteLaunch>(logits_type, shape->E, static_cast<hipStream_t>(stream), a,
                       router->scoring);
  return launch_status();
}

int moe_route_backward(const moe_shape_t* shape, const moe_router_t* router, int logits_type,
                       const void* logits, const int32_t* topk_ids, const float* d_weights,
                       const float* d_loss, const int32_t* expert_counts,
                       const int32_t* token_counts, const int32_t* seq_offsets, int sequences,
                       void* d_logits, int32_t* err_word, void* stream) {
  if (!router_ok(shape, router, logits_type)) return MOE_ERR_ARG;
  if (d_loss) {
    if (sequences < 1 || sequences > kMaxSequences) return MOE_ERR_ARG;
    if (!expert_counts || !token_counts) return MOE_ERR_ARG;
    if (!seq_offsets && sequences != 1) return MOE_ERR_ARG;
  }
  if (shape->T == 0) return MOE_OK;
  if (!d_weights && !d_loss) return MOE_ERR_ARG;
  if (!logits || !topk_ids || !d_logits) return MOE_ERR_ARG;
  const size_t size = type_size(logits_type);
  if (!aligned(logits, size) || !aligned(d_logits, size) || !aligned(topk_ids, 4) ||
      !aligned(d_weights, 4) || !aligned(d_loss, 4) || !aligned(expert_counts, 4) ||
      !aligned(token_counts, 4) || !aligned(seq_offsets, 4))
    return MOE_ERR_ARG;
  const GradArgs a{logits, topk_ids, d_weights, d_loss, expert_counts, token_counts, seq_offsets,
                   d_logits, err_word, shape->T, shape->E, shape->k, sequences, router->renorm,
                   router->scale};
  by_type<GradLaunch>(logits_type, shape->E, static_cast<hipStream_t>(stream), a,
                      router->scoring);
  return launch_status();
}

size_t moe_balance_workspace_bytes(const moe_shape_t* shape, int sequences) {
  if (!shape_ok(shape) || sequences < 1 || sequences > kMaxSequences) return 0;
  const size_t slots = size_t(balance_tile_count(shape->T)) + sequences;
  return slots * (size_t(shape->E) * 8 + 4);
}

int moe_balance_loss(const moe_shape_t* shape, const moe_router_t* router, int logits_type,
                     const void* logits, const int32_t* topk_ids, const int32_t* seq_offsets,
                     int sequences, float* loss, int32_t* expert_counts, int32_t* token_counts,
                     float* score_mean, void* workspace, size_t workspace_bytes,
                     int32_t* err_word, void* stream) {
  if (!router_ok(shape, router, logits_type)) return MOE_ERR_ARG;
  if (sequences < 1 || sequences > kMaxSequences) return MOE_ERR_ARG;
  if (!seq_offsets && sequences != 1) return MOE_ERR_ARG;
  if (!loss || !expert_counts || !token_counts || !score_mean || !workspace) return MOE_ERR_ARG;
  if (shape->T > 0 && (!logits || !topk_ids)) return MOE_ERR_ARG;
  if (workspace_bytes < moe_balance_workspace_bytes(shape, sequences)) return MOE_ERR_ARG;
  if (!aligned(logits, type_size(logits_type)) || !aligned(topk_ids, 4) ||
      !aligned(seq_offsets, 4) || !aligned(loss, 4) || !aligned(expert_counts, 4) ||
      !aligned(token_counts, 4) || !aligned(score_mean, 4) || !aligned(workspace, 16))
    return MOE_ERR_ARG;
  const int tiles = balance_tile_count(shape->T);
  const size_t slots = size_t(tiles) + sequences;
  float* sums = static_cast<float*>(workspace);
  int32_t* pairs = reinterpret_cast<int32_t*>(sums + slots * shape->E);
  const BalanceArgs a{logits, topk_ids, seq_offsets, sums, pairs, pairs + slots * shape->E, loss,
                      expert_counts, token_counts, score_mean, err_word, shape->T, shape->E,
                      shape->k, sequences, balance_tile(shape->T)};
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (tiles > 0) by_type<BalanceLaunch>(logits_type, shape->E, st, a, router->scoring, tiles);
  balance_join<<<sequences, kTileThreads, 0, st>>>(a);
  return launch_status();
}

}  // extern "C"
