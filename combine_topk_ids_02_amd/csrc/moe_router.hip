// The router of an expert-parallel layer and the loss that balances it: HIP
// kernels for CDNA4 (gfx950, wave64) behind include/moe_dispatch.h.
//
// Pages cited (title, section):
//  [A2A]  "A2A backends" page, vincentzed.com/writing/a2a-backends
//  [EP]   "Beyond One GPU: Tensor, Pipeline and Expert Parallelism, and Split
//         Prefill and Decode"
//
// Kernels
//  route_tokens    four tokens per wave, 16 lanes each: the choice and the
//                  weights ([A2A] sec 1.1: the router picks k of the E experts
//                  and a weight for each); route_wide: one wave per token
//  route_gradient  the gradient of the logits from the weights' gradient and
//                  from the balance loss's
//  balance_tiles   one workgroup per tile of tokens: the sums of the scores
//                  and the pairs of each expert, sequence by sequence
//  balance_join    one workgroup per sequence: joins the tiles' sums, the loss
//                  ([EP]: the busiest GPU's experts set the time of a layer)
// All of them read the logits once. No result depends on the order in which
// waves run.

#include "moe_common.h"

namespace {

using namespace moe;

constexpr int kBlock = 256;
constexpr int kWavesPerBlock = kBlock / kWave;
constexpr int kMaxSequences = 1 << 16;
constexpr int kMaxTokens = 1 << 25;  // a launch has fewer than 2^32 threads, 64 a token

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

// The weights from the chosen logits: lane j of a row of 16 holds slot j's
// (`mine`: it has an expert); `top` is the softmax's largest logit and `all` its
// sum over all experts, used where the weights are not renormalised.
// Sigmoids are taken times e^-m, m = min(0, largest chosen logit): none
// underflows against another.
template <bool kSigmoid>
__device__ __forceinline__ float weight_of(const RouteArgs& a, bool mine, float zj, float top,
                                           float all) {
  float w = 0.0f, total = 1.0f;
  if (kSigmoid) {
    const float m = a.renorm ? fminf(0.0f, row_max(mine ? zj : -INFINITY)) : 0.0f;
    if (mine) {
      const float en = expf(-fabsf(zj));
      w = zj >= 0.0f ? 1.0f / (1.0f + en) : expf(zj - m) / (1.0f + en);
    }
  } else {
    if (mine) w = expf(zj - top);
    total = all;
  }
  if (a.renorm) total = row_sum(w);
  return mine ? w / total * a.scale : 0.0f;
}

// One wave for token t, every comparison exact. Each of k rounds takes the
// wave's maximum (a lane's own over its V registers, then 6 steps across
// lanes), finds its holders with a ballot per register (the first set bit of
// the first register that has one is the lowest expert id among equal keys) and
// strikes that one out.
template <typename Tz, int V, bool kSigmoid, bool kKeyed>
__device__ __forceinline__ void route_exactly(const RouteArgs& a, int64_t t, float* lds) {
  const int lane = lane_id();
  const int E = a.E, k = a.k;
  bool routed = !a.mask || a.mask[t];
  float z[V], key[V];
  int chosen = 0;       // experts found
  int id = -1;          // lane j: the expert of slot j
  float weight = 0.0f;  // and its weight
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
    if (kKeyed && a.groups > 1) keep_groups<V>(key, lds, E, a.groups, a.top_groups);
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
      if (lane == j) id = at * kWave + win;
      ++chosen;
    }
    const bool mine = lane < chosen;
    const float zj = mine ? float(row[id]) : -INFINITY;
    float top = 0.0f, all = 1.0f;
    if (!kSigmoid) {
      top = read_lane(row_max(zj), 0);
      if (!a.renorm) {
        all = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) all += expf(z[i] - top);
        all = wave_sum(all);
      }
    }
    weight = weight_of<kSigmoid>(a, mine, zj, top, all);
  }
  if (lane < k) {
    a.ids[t * k + lane] = lane < chosen ? id : -1;
    a.weights[t * k + lane] = lane < chosen ? weight : 0.0f;
  }
}

// ---------------------------------------------------------------------------
// Four tokens at a time

// Whether a predicate holds in any lane of this lane's row of 16.
__device__ __forceinline__ bool row_any(bool p) {
  return ((__ballot(p) >> (lane_id() & 48)) & 0xFFFF) != 0;
}

// Rotations within a row (every lane has a source).
template <int kCtrl>
__device__ __forceinline__ int rotated(int v) {
  return __builtin_amdgcn_mov_dpp(v, kCtrl, 0xF, 0xF, true);
}

__device__ __forceinline__ int row_max_int(int v) {
  v = max(v, rotated<kRowRor + 8>(v));
  v = max(v, rotated<kRowRor + 4>(v));
  v = max(v, rotated<kRowRor + 2>(v));
  return max(v, rotated<kRowRor + 1>(v));
}

// Of the lanes where p holds, the first of every row (p holds in each).
__device__ __forceinline__ uint64_t first_of_rows(bool p) {
  const uint64_t b = __ballot(p);
  return b & ~(b - 0x0001000100010001ull);
}

// The two largest of a row, x >= y, from every lane's two.
template <int kCtrl>
__device__ __forceinline__ void merge_two(int& x, int& y) {
  const int x2 = rotated<kCtrl>(x), y2 = rotated<kCtrl>(y);
  y = max(min(x, x2), max(y, y2));
  x = max(x, x2);
}

// Floats as integers of the same order (-0 as +0). Below kLeast lie -infinity
// (kNone) and kAbsent: no key.
constexpr int kAbsent = INT32_MIN;
constexpr int kNone = int(0x807FFFFFu);
constexpr int kLeast = int(0x80800000u);  // the lowest finite float
__device__ __forceinline__ int ordered(float v) {
  const int b = __float_as_int(v + 0.0f);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float unordered(int b) {
  return __int_as_float(b ^ ((b >> 31) & 0x7FFFFFFF));
}

// Descending sort of n = 1, 2, 4, 8 or 16 integers in registers (Batcher's
// odd-even merge sort).
template <int N, int kLo, int kN>
__device__ __forceinline__ void sort_run(int (&v)[N]) {
  if constexpr (kN > 1) {
    sort_run<N, kLo, kN / 2>(v);
    sort_run<N, kLo + kN / 2, kN / 2>(v);
#pragma unroll
    for (int p = kN / 2; p >= 1; p /= 2) {
      // p = kN / 2: halves against each other; then the inner pairs
#pragma unroll
      for (int i = 0; i < kN - p; ++i) {
        const bool pair = p == kN / 2 ? i < p : i >= p && (i - p) % (2 * p) < p;
        if (pair) {
          const int x = v[kLo + i], y = v[kLo + i + p];
          v[kLo + i] = max(x, y);
          v[kLo + i + p] = min(x, y);
        }
      }
    }
  }
}

// A bitonic run of kN sorted, descending.
template <int N, int kN>
__device__ __forceinline__ void sort_bitonic(int (&v)[N]) {
#pragma unroll
  for (int p = kN / 2; p >= 1; p /= 2)
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if ((i & p) == 0) {
        const int x = v[i], y = v[i + p];
        v[i] = max(x, y);
        v[i + p] = min(x, y);
      }
}

// The L largest of V integers, descending, in v[0 .. L-1] (V a multiple of L):
// runs of L sorted, then each merged into the first (the larger of the one and
// the reverse of the other is bitonic and holds the L largest).
template <int V, int L>
__device__ __forceinline__ void largest(int (&v)[V]) {
  sort_run<V, 0, L>(v);
  if constexpr (V > L) {
#pragma unroll
    for (int r = L; r < V; r += L) {
      int w[L];
#pragma unroll
      for (int i = 0; i < L; ++i) w[i] = v[r + i];
      sort_run<L, 0, L>(w);
#pragma unroll
      for (int i = 0; i < L; ++i) v[i] = max(v[i], w[L - 1 - i]);
      sort_bitonic<V, L>(v);
    }
  }
}

// Four tokens per wave, a row of 16 lanes each: expert e = 16 * i + l in
// register i of the row's lane l. A key becomes an integer of the same order
// whose kBits lowest bits hold V - 1 - i (of equal keys the lower register is
// the larger integer); a lane keeps its L largest sorted, and each of k rounds
// takes the row's largest head (4 steps within the row, for four tokens at
// once), its first holder, and pops that lane's list. What the low bits have
// hidden, and what a sigmoid in 32 bits may be off, can turn a choice only
// where two keys next to each other in it (or a kept and a dropped group) are
// that close. Then the candidates' exact keys (or the two groups') decide; what
// even that leaves open (three as close) is chosen again by route_exactly.
// Every vector step serves four tokens; with a wave per token the same work
// took 28.2 us at T = 16384, E = 256, k = 8 with bias and 8 groups (float32
// logits, 16.8 MB), this takes 14.0 us (16.6 with every close token chosen again).
template <typename Tz, int V, int L, bool kSigmoid, bool kKeyed>
__global__ __launch_bounds__(kBlock) void route_tokens(RouteArgs a) {
  constexpr int kBits = V <= 2 ? 1 : V <= 4 ? 2 : V <= 8 ? 3 : V <= 16 ? 4 : 5;
  constexpr int kLow = (1 << kBits) - 1;
  constexpr bool kHidden = kKeyed || sizeof(Tz) == 4;  // low bits of a key can be lost
  extern __shared__ float lds_all[];
  const int lane = lane_id(), l = lane & 15;
  const int wave = wave_in_block();
  const int64_t first = ((int64_t)blockIdx.x * kWavesPerBlock + wave) * 4;
  if (first >= a.T) return;
  const int64_t t = first + (lane >> 4);
  const int E = a.E, k = a.k;
  bool routed = t < a.T && (!a.mask || a.mask[t]);
  // loads of clamped places, all at once; what they hold past E or T or for a
  // masked token is not used
  const Tz* row = static_cast<const Tz*>(a.logits) + min(t, (int64_t)a.T - 1) * E;
  Tz raw[V];
  float bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i) raw[i] = row[min(i * 16 + l, E - 1)];
  if (kKeyed && a.bias) {
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = a.bias[min(i * 16 + l, E - 1)];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = 0.0f;
  }
  float z[V];
  int key[V];  // in the order of the keys
  bool bad = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    z[i] = routed && i * 16 + l < E ? float(raw[i]) : -INFINITY;
    float v = z[i];
    if (kKeyed) {
      v = __builtin_amdgcn_rcpf(1.0f + __expf(-z[i])) + bias[i];
      v = z[i] == -INFINITY ? -INFINITY : v;
      bad |= !(v < INFINITY);
    }
    bad |= !(z[i] < INFINITY);
    key[i] = ordered(v);
  }
  bool unsure = false;
  if (row_any(bad)) {
    if (l == 0) flag_error(a.err, MOE_ERRBIT_BAD_LOGIT);
    routed = false;
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = kAbsent;
  }

  if (kKeyed && a.groups > 1) {
    // Group g is the registers [g * per, (g + 1) * per): the two largest keys of
    // every group, in the end in lane g of the row.
    const int per = E / a.groups / 16;
    int first_key = kAbsent, second_key = kAbsent;  // lane g: those of group g
    int x = kAbsent, y = kAbsent;    // the two largest so far
    int g = 0, left = per;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      y = max(y, min(x, key[i]));
      x = max(x, key[i]);
      if (--left == 0) {  // uniform
        merge_two<kRowRor + 8>(x, y);
        merge_two<kRowRor + 4>(x, y);
        merge_two<kRowRor + 2>(x, y);
        merge_two<kRowRor + 1>(x, y);
        if (l == g) {
          first_key = x;
          second_key = y;
        }
        x = y = kAbsent;
        ++g;
        left = per;
      }
    }
    // A sigmoid here is off by at most 2^-22 (4 roundings), a key by that and two
    // roundings of its size, a score by both keys' and two of its own: 4.8e-7 and
    // 2^-22 of the keys' sizes, which their sum says nothing of where they cancel.
    // `off` is twice that (products first: it cannot overflow).
    const float one = unordered(first_key);
    const float two = second_key >= kLeast ? unordered(second_key) : 0.0f;
    const float score = one + two;
    const float off = first_key >= kLeast ? 1e-6f + (fabsf(one) * 0x1p-21f + fabsf(two) * 0x1p-21f)
                                          : 0.0f;
    // The score as a key. Two keys may sum to -infinity, which is the score of a
    // group without any too: it takes part all the same.
    int head = first_key >= kLeast ? ordered(score) : kNone;
    if (l >= a.groups) head = kAbsent;
    // the best top_groups of them, the first of equal ones: lane g learns
    // whether its group is kept
    bool kept = false;
    for (int r = 0; r < a.top_groups; ++r) {
      const int worst = row_max_int(head);
      const uint64_t at_worst = first_of_rows(head == worst);
      if ((at_worst >> lane) & 1) {  // a group's: there are top_groups of them
        kept = true;
        head = kAbsent;
      }
    }
    // A kept group can be exactly below one that is not only where the least it
    // may score is not above the most the other may. (Scores past 2^127 count as
    // that, which leaves room for `off`.)
    const float score_at = fminf(fmaxf(score, -0x1p127f), 0x1p127f);
    const float least = score_at - off;
    const float most = off > 0.0f ? score_at + off : -INFINITY;
    const float worst = -row_max(kept ? -least : -INFINITY);
    const float next = row_max(kept ? -INFINITY : most);
    const bool close = worst <= next;
    if (__ballot(close && routed)) {
      // exact scores decide between one such kept group and one such other; more
      // of either go the long way
      const uint32_t doubted = uint32_t(__ballot(kept && least <= next) >> (lane & 48)) & 0xFFFF;
      const uint32_t hopeful = uint32_t(__ballot(!kept && most >= worst) >> (lane & 48)) & 0xFFFF;
      unsure |= close && (__popc(doubted) != 1 || __popc(hopeful) != 1);
      const int group_a = max(__ffs(int(doubted)) - 1, 0);
      const int group_b = max(__ffs(int(hopeful)) - 1, 0);
      float exact[2];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        int x2 = kNone, y2 = kNone;
        for (int i = 0; i < per; ++i) {
          const int e = min((w ? group_b : group_a) * per * 16 + i * 16 + l, E - 1);
          const float ze = float(row[e]);
          const float ke = sigmoid_nearest(ze) + (a.bias ? a.bias[e] : 0.0f);
          const int o = ze == -INFINITY ? kNone : ordered(ke);
          y2 = max(y2, min(x2, o));
          x2 = max(x2, o);
        }
        merge_two<kRowRor + 8>(x2, y2);
        merge_two<kRowRor + 4>(x2, y2);
        merge_two<kRowRor + 2>(x2, y2);
        merge_two<kRowRor + 1>(x2, y2);
        exact[w] = y2 >= kLeast ? unordered(x2) + unordered(y2) : unordered(x2);
      }
      const bool swap = exact[1] > exact[0] || (exact[1] == exact[0] && group_b < group_a);
      if (close && swap) kept = l == group_b || (kept && l != group_a);
    }
    const uint32_t keep = uint32_t(__ballot(kept) >> (lane & 48));
    uint32_t bit = 1;
    left = per;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = keep & bit ? key[i] : kAbsent;
      if (--left == 0) {
        bit <<= 1;
        left = per;
      }
    }
  }

  int list[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
    list[i] = (key[i] & ~kLow) | (V - 1 - i);
  largest<V, L>(list);
  const bool full = V > L && list[L - 1] >= kLeast;
  // One candidate more than slots (where the row has a lane for it): the choice
  // is put right among them below.
  const int taken = kHidden ? min(k + 1, 16) : k;
  int found = kAbsent;          // lane j: candidate j's key
  uint32_t low0 = 0, low1 = 0;  // and the lanes its round took it from
  for (int j = 0; j < taken; ++j) {
    const int m = row_max_int(list[0]);
    const uint64_t low = first_of_rows(list[0] == m);
    if (l == j) {
      found = m;
      low0 = uint32_t(low);
      low1 = uint32_t(low >> 32);
    }
    if ((low >> lane) & 1) {
#pragma unroll
      for (int i = 0; i + 1 < L; ++i) list[i] = list[i + 1];
      list[L - 1] = kAbsent;
    }
  }
  const bool candidate = l < taken && found >= kLeast;
  const uint32_t field = (lane & 32 ? low1 : low0) >> (lane & 16) & 0xFFFF;
  const int id = candidate ? (V - 1 - (found & kLow)) * 16 + __ffs(int(field)) - 1 : -1;
  float zj = candidate ? float(row[id]) : -INFINITY;
  int slot = l;
  if (kHidden) {
    // Whether a candidate may come before one whose key is `after` at most.
    auto close = [&](int after) {
      if (after < kLeast) return false;
      if (!kKeyed) return (found | kLow) == (after | kLow);
      const float v = unordered(found | kLow);
      return v - unordered(after & ~kLow) < 1e-6f + fabsf(v) * (0x1p-22f + 0x1p-22f * kLow);
    };
    const int rest = row_max_int(list[0]);
    const int shifted = __builtin_amdgcn_update_dpp(kAbsent, found, 0x101, 0xF, 0xF, false);
    const bool near = candidate && l < k && close(l == taken - 1 ? rest : shifted);
    // what is not among the candidates may be the last slot's, or be hidden
    // behind a list that has run out: the long way
    unsure |= candidate && l == k - 1 && close(rest);
    unsure |= full && list[0] < kLeast;
    if (__ballot(near && routed)) {
      // the candidates' exact keys, and each one's place by them
      float exact = zj;
      if (kKeyed && candidate) exact = sigmoid_nearest(zj) + (a.bias ? a.bias[id] : 0.0f);
      if (!candidate) exact = -INFINITY;
      slot = 0;
#pragma unroll
      for (int r = 1; r < 16; ++r) {
        // the candidate r lanes on
        const int from = (lane & 48) | ((l + r) & 15);
        const float other = __shfl(exact, from);
        const int other_id = __shfl(id, from);
        slot += other > exact || (other == exact && other_id >= 0 && other_id < id) ? 1 : 0;
      }
      if (!candidate) slot = 16;
    }
  }
  const bool mine = candidate && slot < k;
  if (!mine) zj = -INFINITY;

  float top = 0.0f, all = 1.0f;
  if (!kSigmoid) {
    top = row_max(zj);
    if (!a.renorm) {
      all = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) all += expf(z[i] - top);
      all = row_sum(all);
    }
  }
  const float weight = weight_of<kSigmoid>(a, mine, zj, top, all);
  const uint64_t again = kHidden ? __ballot(unsure && routed) : 0;
  if (t < a.T && !((again >> (lane & 48)) & 0xFFFF)) {
    // slots that no candidate takes are the last ones
    const int count = __popc(uint32_t(__ballot(mine) >> (lane & 48)) & 0xFFFF);
    const int to = mine ? slot : l;
    if (mine || (l >= count && l < k)) {
      a.ids[t * k + to] = mine ? id : -1;
      a.weights[t * k + to] = weight;
    }
  }
  if (kHidden) {
    if (again) {
      constexpr int V64 = (V + 3) / 4;
#pragma unroll 1
      for (int r = 0; r < 4; ++r)
        if ((again >> (16 * r)) & 0xFFFF)
          route_exactly<Tz, V64, kSigmoid, kKeyed>(a, first + r, lds_all + wave * E);
    }
  }
}

// One wave per token, for what route_tokens does not take: more than 512
// experts, or groups that do not fill rows of 16 experts.
template <typename Tz, int V, bool kSigmoid, bool kKeyed>
__global__ __launch_bounds__(kBlock) void route_wide(RouteArgs a) {
  extern __shared__ float lds_all[];
  const int wave = wave_in_block();
  const int64_t t = (int64_t)blockIdx.x * kWavesPerBlock + wave;
  if (t < a.T) route_exactly<Tz, V, kSigmoid, kKeyed>(a, t, lds_all + wave * a.E);
}

// ---------------------------------------------------------------------------
// Scores of whole tokens (the balance loss, the gradient)

// LT lanes per token: 16 (four tokens a wave) up to 512 experts, 64 above.
// Expert e = LT * i + l lies in register i of the token's lane l.
template <int LT>
__device__ __forceinline__ float token_sum(float v) {
  return LT == 16 ? row_sum(v) : wave_sum(v);
}
template <int LT>
__device__ __forceinline__ float token_max(float v) {
  return LT == 16 ? row_max(v) : wave_max(v);
}
template <int LT>
__device__ __forceinline__ bool token_any(bool p) {
  return LT == 16 ? row_any(p) : __ballot(p) != 0;
}

// A token's scores scaled to a sum of one (p), and for sigmoid 1 - s of each
// (inner). Masked experts, and those past E, have -infinity and get 0.
// e^x is 2^(x log2 e) with the product in 32 bits: off by |x| 2^-24 and the
// instruction's own rounding, which is least where the shares are large (the
// gradient at T = 16384, E = 256 is 9e-8 off the 64-bit formula, 1e-7 with a
// full-length exponential, which takes five steps more per expert).
template <int LT, int V, bool kSigmoid>
__device__ __forceinline__ void shares(const float (&z)[V], float (&p)[V], float (&inner)[V]) {
  constexpr float kLog2e = 1.44269504089f;
  float m = z[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = fmaxf(m, z[i]);
  m = token_max<LT>(m);
  if (m == -INFINITY) m = 0.0f;  // no expert has a score: all shares are 0
  const float top = -m * kLog2e;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (kSigmoid) {
      const float en = __builtin_amdgcn_exp2f(z[i] * -kLog2e);
      p[i] = __builtin_amdgcn_rcpf(1.0f + en);
      inner[i] = fminf(en, 1e38f) * p[i];
    } else {
      p[i] = __builtin_amdgcn_exp2f(fmaf(z[i], kLog2e, top));
    }
  }
  if (kSigmoid && __ballot(m < -40.0f)) {
    // all sigmoids of some token are tiny: there they are taken times e^-m
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (m < -40.0f) {
        p[i] = __builtin_amdgcn_exp2f(fmaf(z[i], kLog2e, top));  // 1 + e^z is 1
        inner[i] = 1.0f;
      }
  }
  if (__ballot(fabsf(m) > 0x1p20f)) {
    // The rounding of `top` is a factor on all of a token's exponentials, from
    // here on no longer near 1: it passes float32's range at |m| = 2^32, as m
    // log2 e does at the end of it. There the difference comes first, which
    // costs it a rounding (and sigmoids of logits above are ones as they stand).
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (fabsf(m) > 0x1p20f && !(kSigmoid && m > 0.0f))
        p[i] = __builtin_amdgcn_exp2f((z[i] - m) * kLog2e);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) sum += p[i];
  sum = token_sum<LT>(sum);
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) p[i] *= inv;
}

// The logits of a token with E experts, all loads at once (kFull: E is V * LT;
// else of clamped places); as floats, -infinity past E or where the token takes
// no part.
template <typename Tz, int LT, int V, bool kFull>
__device__ __forceinline__ void load_token(const Tz* row, int l, int E, Tz (&raw)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) raw[i] = row[kFull ? i * LT + l : min(i * LT + l, E - 1)];
}
template <typename Tz, int LT, int V, bool kFull>
__device__ __forceinline__ void to_floats(const Tz (&raw)[V], int l, int E, bool used,
                                          float (&z)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i)
    z[i] = used && (kFull || i * LT + l < E) ? float(raw[i]) : -INFINITY;
}

// ---------------------------------------------------------------------------
// Balance loss

// The sequence of the token t that LT lanes share: the first s with
// offsets[s + 1] > t (S when none). The lanes look at LT places at a time, so
// that up to LT sequences take one load's time; whatever the offsets hold, the
// answer is in [0, S].
template <int LT>
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int S, int64_t t) {
  const int lane = lane_id(), l = lane % LT;
  int lo = 0;
  for (int n = S; n > 0;) {  // it is one of lo .. lo + n
    const int step = (n + LT - 1) / LT;
    const int behind = (l + 1) * step - 1;
    const bool below = behind < n && lo + behind < S && offsets[lo + behind + 1] <= t;
    const uint64_t b = __ballot(below) >> (LT == 16 ? lane & 48 : 0);
    lo += (LT == 16 ? __popc(uint32_t(b) & 0xFFFF) : __popcll(b)) * step;
    n = step - 1;
  }
  return min(lo, S);
}

struct BalanceArgs {
  const void* logits;
  const int32_t* ids;
  const int32_t* offsets;  // NULL: one sequence of all tokens
  float* sums;             // [slots * stride] sums of the scores, slots = tiles + S
  int32_t* pairs;          // [slots * stride] pairs
  int32_t* used;           // [slots] tokens with an expert
  float* loss;
  int32_t* counts;
  int32_t* tokens;
  float* mean;
  int32_t* err;
  int T, E, k, S, tile;
  int stride;              // E rounded up to a multiple of 4
};

constexpr int kTileThreads = 512;
constexpr int kTileWaves = kTileThreads / kWave;

// One workgroup per tile of tokens, each wave 64 / LT tokens at a time (the
// next ones' logits on their way); the scores are summed per lane in
// registers. Where a sequence ends within the tile, the sums so far go to the
// slot tile + sequence (increasing along the tokens, so no two pairs of them
// share one) and start anew. Bound by latency: T = 16384, E = 256 with
// sigmoids of bfloat16 logits (8.4 MB) takes 9.6 us (23.7 us with a wave per
// token), T = 4096, E = 384 in float32 6.8 us. A lane's float sum has a token a
// pass: one or two up to T = 16384, T / 8192 past that (16 lanes a token; 4 times
// as many with 64); the waves' 8 sums are joined in floats, tiles in 64 bits.
template <typename Tz, int LT, int V, bool kSigmoid, bool kFull>
__global__ __launch_bounds__(kTileThreads) void balance_tiles(BalanceArgs a) {
  extern __shared__ float lds_all[];
  const int E = a.E;
  int* pairs = reinterpret_cast<int*>(lds_all);  // [E]
  int* used = pairs + E;                         // [1]
  float* part = lds_all + E + 1;                 // [waves * E]
  constexpr int kTokens = kWave / LT;
  constexpr int kPass = kTileWaves * kTokens;
  const int wave = wave_in_block(), lane = lane_id(), l = lane % LT;
  const int64_t begin = (int64_t)blockIdx.x * a.tile;
  const int64_t end = min(begin + a.tile, (int64_t)a.T);
  int s = a.offsets ? sequence_of<kWave>(a.offsets, a.S, begin) : 0;
  for (; s < a.S; ++s) {
    const int64_t first = a.offsets ? max((int64_t)a.offsets[s], begin) : begin;
    const int64_t last = a.offsets ? min((int64_t)a.offsets[s + 1], end) : end;
    if (first >= end) break;
    if (first >= last) continue;
    const int64_t mine = first + wave * kTokens + lane / LT;
    Tz raw[V];
    int id = -1;
    auto load = [&](int64_t t) {  // past the last token: the last one's, not used
      const int64_t at = min(t, last - 1);
      load_token<Tz, LT, V, kFull>(static_cast<const Tz*>(a.logits) + at * E, l, E, raw);
      id = t < last && l < a.k ? a.ids[at * a.k + l] : -1;
    };
    load(mine);
    for (int e = threadIdx.x; e <= E; e += kTileThreads) pairs[e] = 0;
    __syncthreads();
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = 0.0f;
    for (int64_t t = mine; t - lane / LT < last; t += kPass) {
      float z[V], p[V], inner[V];
      const bool ok = id >= 0 && id < E;
      if (__ballot(id < -1 || id >= E) && lane == 0) flag_error(a.err, MOE_ERRBIT_BAD_ID);
      if (ok) atomicAdd(pairs + id, 1);  // integers: any order gives the same count
      const bool counted = token_any<LT>(ok);
      if (counted && l == 0) atomicAdd(used, 1);
      to_floats<Tz, LT, V, kFull>(raw, l, E, counted, z);
      if (t - lane / LT + kPass < last) load(t + kPass);
      shares<LT, V, kSigmoid>(z, p, inner);
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] += p[i];
    }
    // the wave's tokens together, then the waves in order
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (LT == 16) {
        sum[i] += __shfl_xor(sum[i], 16);
        sum[i] += __shfl_xor(sum[i], 32);
      }
      if (lane < LT && (kFull || i * LT + l < E)) part[wave * E + i * LT + l] = sum[i];
    }
    __syncthreads();
    const int64_t slot = (int64_t)blockIdx.x + s;
    for (int e = threadIdx.x; e < E; e += kTileThreads) {
      float total = 0.0f;
#pragma unroll
      for (int w = 0; w < kTileWaves; ++w) total += part[w * E + e];
      a.sums[slot * a.stride + e] = total;
      a.pairs[slot * a.stride + e] = pairs[e];
    }
    if (threadIdx.x == 0) a.used[slot] = *used;
    __syncthreads();
  }
}

// One workgroup per sequence: a thread adds up four experts' sums of every
// slices-th tile, then the slices are joined, all in an order that the sizes
// alone fix and in 64 bits. (A workgroup per 64 experts, the last of them
// adding up the loss, took 7.3 us for 13 sequences of 16384 tokens where this
// takes 5.7, and with 128 tiles 7.5 against 7.8 us for one of 4096, which takes
// 5.7 with 64: the fence and the count between workgroups cost what reading from
// more of them gave.)
constexpr int kJoinThreads = 1024;
constexpr int kJoinSlices = 32;  // at most
__global__ __launch_bounds__(kJoinThreads) void balance_join(BalanceArgs a) {
  typedef float float4v __attribute__((ext_vector_type(4)));
  typedef int int4v __attribute__((ext_vector_type(4)));
  __shared__ double lds_sum[kJoinThreads * 4];
  __shared__ int lds_pairs[kJoinThreads * 4];
  __shared__ double lds_term[kJoinThreads / kWave];
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
  int n = 0;
  for (int64_t w = w0 + tid; w < w1; w += kJoinThreads) n += a.used[w + s];
  if (n) atomicAdd(&lds_used, n);
  const int quads = a.stride / 4;  // at most 256
  const int slices = min(kJoinSlices, kJoinThreads / quads);
  const int quad = tid % quads, slice = tid / quads;
  double sum[4] = {0, 0, 0, 0};
  int pairs[4] = {0, 0, 0, 0};
  if (slice < slices) {
    constexpr int kAtOnce = 8;  // loads of either kind on their way
    for (int64_t w = w0 + slice; w < w1; w += slices * kAtOnce) {
      float4v x[kAtOnce];
      int4v c[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int64_t at = (min(w + i * slices, w1 - 1) + s) * a.stride + quad * 4;
        x[i] = *reinterpret_cast<const float4v*>(a.sums + at);
        c[i] = *reinterpret_cast<const int4v*>(a.pairs + at);
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (w + i * slices < w1)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            sum[q] += x[i][q];
            pairs[q] += c[i][q];
          }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      lds_sum[slice * a.stride + quad * 4 + q] = sum[q];
      lds_pairs[slice * a.stride + quad * 4 + q] = pairs[q];
    }
  }
  __syncthreads();
  n = lds_used;
  double term = 0.0;
  if (tid < E) {
    double total = 0.0;
    int count = 0;
    for (int q = 0; q < slices; ++q) {
      total += lds_sum[q * a.stride + tid];
      count += lds_pairs[q * a.stride + tid];
    }
    const double mean = n > 0 ? total / n : 0.0;
    a.counts[(int64_t)s * E + tid] = count;
    a.mean[(int64_t)s * E + tid] = float(mean);
    term = mean * count;
  }
  for (int h = kWave / 2; h > 0; h >>= 1) term += __shfl_xor(term, h);
  if (lane_id() == 0) lds_term[wave_in_block()] = term;
  __syncthreads();
  if (tid == 0) {
    double total = 0.0;
    for (int w = 0; w < kJoinThreads / kWave; ++w) total += lds_term[w];
    a.tokens[s] = n;
    a.loss[s] = n > 0 ? float(total * E / (double(a.k) * n)) : 0.0f;
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
// The slots' parts reach their experts' lanes through LDS. Bound by the bytes:
// T = 16384, E = 256 in float32 (33.6 MB both ways) takes 9.9 us, 13.8 us
// with a wave per token; T = 8192 in bfloat16 with both gradients 6.2 us.
template <typename Tz, int LT, int V, bool kSigmoid, bool kFull>
__global__ __launch_bounds__(kBlock) void route_gradient(GradArgs a) {
  constexpr int kTokens = kWave / LT;
  extern __shared__ float lds_all[];
  const int lane = lane_id(), l = lane % LT, wave = wave_in_block();
  const int64_t t0 = ((int64_t)blockIdx.x * kWavesPerBlock + wave) * kTokens;
  if (t0 >= a.T) return;
  const int E = a.E, k = a.k;
  float* spread = lds_all + (wave * kTokens + lane / LT) * E;  // this token's experts
  const int64_t t = t0 + lane / LT;
  const bool here = t < a.T;
  const int64_t at = min(t, (int64_t)a.T - 1);
  const Tz* row = static_cast<const Tz*>(a.logits) + at * E;
  Tz raw[V];
  load_token<Tz, LT, V, kFull>(row, l, E, raw);
  const int id = here && l < k ? a.ids[at * k + l] : -1;
  const bool ok = id >= 0 && id < E;
  if (__ballot(id < -1 || id >= E) && lane == 0) flag_error(a.err, MOE_ERRBIT_BAD_ID);
  const bool used = token_any<LT>(ok);
  int s = 0;
  bool inside = used && a.d_loss;
  if (a.d_loss && a.offsets) {
    s = sequence_of<LT>(a.offsets, a.S, at);
    inside = inside && s < a.S && a.offsets[min(s, a.S - 1)] <= t;
    s = min(s, a.S - 1);
  }
  float z[V], d[V], u[V];
  to_floats<Tz, LT, V, kFull>(raw, l, E, used, z);
#pragma unroll
  for (int i = 0; i < V; ++i) d[i] = u[i] = 0.0f;
  const bool dense = !kSigmoid && !a.renorm && a.d_weights;

  if (a.d_weights) {
    const float g = ok ? a.d_weights[at * k + l] * a.scale : 0.0f;
    const float zj = ok ? float(row[id]) : -INFINITY;
    float q = 0.0f, part = g;  // part: what slot l adds to its expert
    if (kSigmoid) {
      const float m = a.renorm ? fminf(0.0f, row_max(zj)) : 0.0f;
      const float en = expf(-fabsf(zj));
      if (zj > -INFINITY) q = (zj >= 0.0f ? 1.0f : expf(zj - m)) / (1.0f + en);
      if (a.renorm) {
        const float sum = row_sum(q);
        q = sum > 0.0f ? q / sum : 0.0f;
      }
      const float away = (zj >= 0.0f ? en : 1.0f) / (1.0f + en);
      part = away * q * (g - (a.renorm ? row_sum(q * g) : 0.0f));
    } else if (a.renorm) {
      const float m = row_max(zj);
      if (ok && m > -INFINITY) q = expf(zj - m);
      const float sum = row_sum(q);
      q = sum > 0.0f ? q / sum : 0.0f;
      part = q * (g - row_sum(q * g));
    }
    // To the experts' lanes. The slot that finds another's number in its
    // expert's place shares it: then the slots add one after the other.
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (kFull || i * LT + l < E) spread[i * LT + l] = 0.0f;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (ok) spread[id] = float(l);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const bool shared = ok && spread[id] != float(l);
    const bool again = __ballot(shared) != 0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (!again) {
      if (ok) spread[id] = part;
    } else {
      if (ok) spread[id] = 0.0f;
      for (int j = 0; j < k; ++j) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (ok && l == j) spread[id] += part;
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float v = kFull || i * LT + l < E ? spread[i * LT + l] : 0.0f;
      if (dense)
        u[i] = v;
      else
        d[i] = v;
    }
  }

  if (a.d_loss) {
    const int n = a.tokens[s];
    const float rate = inside && n > 0 ? float(double(a.d_loss[s]) * E /
                                               (double(k) * double(n) * double(n)))
                                       : 0.0f;
    const float off = -rate * float(double(k) * n / E);
    int count[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
      count[i] = a.counts[(int64_t)s * E + (kFull ? i * LT + l : min(i * LT + l, E - 1))];
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] += fmaf(rate, float(count[i]), off);
  }
  if (dense || a.d_loss) {
    float p[V], inner[V];
    shares<LT, V, kSigmoid>(z, p, inner);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) dot += p[i] * u[i];
    dot = token_sum<LT>(dot);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float v = kSigmoid ? p[i] * inner[i] : p[i];
      d[i] = fmaf(v, u[i] - dot, d[i]);
    }
  }
  if (!here) return;
  Tz* out = static_cast<Tz*>(a.d_logits) + t * E;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (kFull || i * LT + l < E) out[i * LT + l] = Tz(d[i]);
}

// ---------------------------------------------------------------------------
// Host side

size_t type_size(int type) { return type == MOE_TYPE_F32 ? 4 : 2; }

bool router_ok(const moe_shape_t* sh, const moe_router_t* r, int type) {
  if (!shape_ok(sh) || !r || sh->T > kMaxTokens) return false;
  if (type != MOE_TYPE_F32 && type != MOE_TYPE_BF16 && type != MOE_TYPE_F16) return false;
  if (r->scoring != MOE_SCORE_SOFTMAX && r->scoring != MOE_SCORE_SIGMOID) return false;
  if (r->renorm != 0 && r->renorm != 1) return false;
  if (!(r->scale - r->scale == 0.0f)) return false;  // finite
  if (r->groups < 1 || r->groups > kWave || sh->E % r->groups != 0) return false;
  if (r->top_groups < 1 || r->top_groups > r->groups) return false;
  if (r->scoring == MOE_SCORE_SOFTMAX && r->groups > 1) return false;
  return true;
}

// Calls F<Tz, V>::go: V registers of 64 experts each.
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

bool keyed(const RouteArgs& a, int scoring) {
  return scoring == MOE_SCORE_SIGMOID && (a.bias || a.groups > 1);
}

// LDS of the exact choice: its groups' keys.
size_t route_lds(const RouteArgs& a) {
  return a.groups > 1 ? size_t(kWavesPerBlock) * a.E * 4 : 0;
}

template <typename Tz, int V>
struct RouteWideLaunch {
  static void go(hipStream_t st, const RouteArgs& a, int scoring) {
    const dim3 grid(token_blocks(a.T));
    if (keyed(a, scoring))
      route_wide<Tz, V, true, true><<<grid, kBlock, route_lds(a), st>>>(a);
    else if (scoring == MOE_SCORE_SIGMOID)
      route_wide<Tz, V, true, false><<<grid, kBlock, 0, st>>>(a);
    else
      route_wide<Tz, V, false, false><<<grid, kBlock, 0, st>>>(a);
  }
};

template <typename Tz, int V, int L>
void launch_route(hipStream_t st, const RouteArgs& a, int scoring) {
  const dim3 grid((token_blocks(a.T) + 3) / 4);
  if (keyed(a, scoring))
    route_tokens<Tz, V, L, true, true><<<grid, kBlock, route_lds(a), st>>>(a);
  else if (scoring == MOE_SCORE_SIGMOID)
    route_tokens<Tz, V, L, true, false><<<grid, kBlock, 0, st>>>(a);
  else
    route_tokens<Tz, V, L, false, false><<<grid, kBlock, 0, st>>>(a);
}

template <typename Tz>
struct RouteLaunch {
  static void go(hipStream_t st, const RouteArgs& a, int scoring) {
    const int v = (a.E + 15) / 16;
    if (v <= 4) return launch_route<Tz, 4, 4>(st, a, scoring);
    if (a.k <= 8) {
      if (v <= 8) return launch_route<Tz, 8, 8>(st, a, scoring);
      if (v <= 16) return launch_route<Tz, 16, 8>(st, a, scoring);
      if (v <= 24) return launch_route<Tz, 24, 8>(st, a, scoring);
      return launch_route<Tz, 32, 8>(st, a, scoring);
    }
    if (v <= 8) return launch_route<Tz, 8, 8>(st, a, scoring);
    if (v <= 16) return launch_route<Tz, 16, 16>(st, a, scoring);
    return launch_route<Tz, 32, 16>(st, a, scoring);
  }
};

template <typename Tz, int LT, int V>
struct GradLaunch {
  static void go(hipStream_t st, const GradArgs& a, int scoring) {
    constexpr int kTokens = kWavesPerBlock * kWave / LT;
    const dim3 grid((a.T + kTokens - 1) / kTokens);
    const size_t lds = a.d_weights ? size_t(kTokens) * a.E * 4 : 0;
    const bool full = a.E == V * LT;
    auto go = full ? scoring == MOE_SCORE_SIGMOID ? route_gradient<Tz, LT, V, true, true>
                                                  : route_gradient<Tz, LT, V, false, true>
                   : scoring == MOE_SCORE_SIGMOID ? route_gradient<Tz, LT, V, true, false>
                                                  : route_gradient<Tz, LT, V, false, false>;
    go<<<grid, kBlock, lds, st>>>(a);
  }
};

template <typename Tz, int LT, int V>
struct BalanceLaunch {
  static void go(hipStream_t st, const BalanceArgs& a, int scoring, int tiles) {
    const size_t lds = (size_t(a.E) * (kTileWaves + 1) + 1) * 4;
    const bool full = a.E == V * LT;
    auto go = full ? scoring == MOE_SCORE_SIGMOID ? balance_tiles<Tz, LT, V, true, true>
                                                  : balance_tiles<Tz, LT, V, false, true>
                   : scoring == MOE_SCORE_SIGMOID ? balance_tiles<Tz, LT, V, true, false>
                                                  : balance_tiles<Tz, LT, V, false, false>;
    go<<<tiles, kTileThreads, lds, st>>>(a);
  }
};

// Calls F<Tz, LT, V>::go for the lanes per token and registers that E takes.
template <template <typename, int, int> class F, typename Tz, typename... Args>
void by_tokens(int E, Args&&... args) {
  const int v = (E + 15) / 16;
  if (v <= 4) return F<Tz, 16, 4>::go(args...);
  if (v <= 8) return F<Tz, 16, 8>::go(args...);
  if (v <= 16) return F<Tz, 16, 16>::go(args...);
  if (v <= 24) return F<Tz, 16, 24>::go(args...);
  if (v <= 32) return F<Tz, 16, 32>::go(args...);
  return F<Tz, 64, 16>::go(args...);
}

template <template <typename, int, int> class F, typename... Args>
void by_type_tokens(int type, int E, Args&&... args) {
  if (type == MOE_TYPE_F32) return by_tokens<F, float>(E, args...);
  if (type == MOE_TYPE_BF16) return by_tokens<F, __bf16>(E, args...);
  return by_tokens<F, _Float16>(E, args...);
}

// Tiles of the balance loss: a multiple of 32 tokens (a workgroup's pass), at
// most 256 of them; two passes where one would make more than 64 tiles, for the join
// reads every tile of a sequence (T = 4096, E = 384: 64 tiles 6.8 + 5.6 us, 128 tiles
// 5.8 + 7.8 us, 32 tiles 10.1 + 5.1 us), and more only past 16384 tokens.
constexpr int kMaxTiles = 256;
constexpr int kOnePassTiles = 64;
constexpr int kPass = kTileWaves * 4;
int balance_tile(int T) {
  const int least = (T + kMaxTiles - 1) / kMaxTiles;
  return std::max(T > kOnePassTiles * kPass ? 2 : 1, (least + kPass - 1) / kPass) * kPass;
}
int balance_tile_count(int T) {
  const int tile = balance_tile(T);
  return (T + tile - 1) / tile;
}

// The most tiles that any batch of up to T tokens has (a longer tile makes
// fewer: 2048 tokens have 64, 2049 have 33, so a workspace for the second alone
// would not do for the first).
int balance_tile_bound(int T) {
  return std::max(std::min((T + kPass - 1) / kPass, kOnePassTiles),
                  std::min((T + 2 * kPass - 1) / (2 * kPass), kMaxTiles));
}

// The workspace: sums and pairs [slots * stride], used [slots], a slot for
// every tile and sequence.
int balance_stride(const moe_shape_t& sh) { return (sh.E + 3) / 4 * 4; }
size_t balance_bytes(const moe_shape_t& sh, int tiles, int sequences) {
  return (size_t(tiles) + sequences) * (size_t(balance_stride(sh)) * 8 + 4);
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
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool rows = shape->E <= 512 &&
                    (a.groups == 1 || (a.groups <= 16 && shape->E / a.groups % 16 == 0));
  if (!rows)
    by_type<RouteWideLaunch>(logits_type, shape->E, st, a, router->scoring);
  else if (logits_type == MOE_TYPE_F32)
    RouteLaunch<float>::go(st, a, router->scoring);
  else if (logits_type == MOE_TYPE_BF16)
    RouteLaunch<__bf16>::go(st, a, router->scoring);
  else
    RouteLaunch<_Float16>::go(st, a, router->scoring);
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
  by_type_tokens<GradLaunch>(logits_type, shape->E, static_cast<hipStream_t>(stream), a,
                             router->scoring);
  return launch_status();
}

size_t moe_balance_workspace_bytes(const moe_shape_t* shape, int sequences) {
  if (!shape_ok(shape) || sequences < 1 || sequences > kMaxSequences) return 0;
  return balance_bytes(*shape, balance_tile_bound(shape->T), sequences);
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
  const int tiles = balance_tile_count(shape->T), stride = balance_stride(*shape);
  if (workspace_bytes < balance_bytes(*shape, tiles, sequences)) return MOE_ERR_ARG;
  if (!aligned(logits, type_size(logits_type)) || !aligned(topk_ids, 4) ||
      !aligned(seq_offsets, 4) || !aligned(loss, 4) || !aligned(expert_counts, 4) ||
      !aligned(token_counts, 4) || !aligned(score_mean, 4) || !aligned(workspace, 16))
    return MOE_ERR_ARG;
  const size_t slots = size_t(tiles) + sequences;
  float* sums = static_cast<float*>(workspace);
  int32_t* pairs = reinterpret_cast<int32_t*>(sums + slots * stride);
  const BalanceArgs a{logits, topk_ids, seq_offsets, sums, pairs, pairs + slots * stride, loss,
                      expert_counts, token_counts, score_mean, err_word, shape->T, shape->E,
                      shape->k, sequences, balance_tile(shape->T), stride};
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (tiles > 0) by_type_tokens<BalanceLaunch>(logits_type, shape->E, st, a, router->scoring, tiles);
  balance_join<<<sequences, kJoinThreads, 0, st>>>(a);
  return launch_status();
}

}  // extern "C"
