// The norm before a layer, its gradient, and rows to 8-bit integers: HIP
// kernels for CDNA4 (gfx950, wave64) behind include/moe_dispatch.h.
//
// All three are one pass over their rows: a row lies in the registers of W
// waves (pieces of 4 or 8 values, NC of them a lane), is read once in loads that are
// all on their way before the first is used, and its sum or maximum is joined
// through DPP and, with W > 1, a value of each wave in LDS. What bounds them is the
// memory: few operations a value. Measured (median kernel time of a trace, two sets of
// buffers in turn):
//  - norm, 4,093 x 5,120 in bf16 to bf16 and MXFP8 (189 MB, in part from the cache of
//    256 MB) 28.3 us, 6.7 TB/s; 8,192 x 7,168 with a float32 stream (705 MB) 126 us, 5.6
//    TB/s; one row of 5,120 2.6 us;
//  - its gradient, 8,192 x 7,168 with a float32 stream (940 MB) 170 us and 5 for the
//    weight's sums, 5.4 TB/s (512 workgroups of 14 waves. Calls in a graph: 179 us, with
//    256 workgroups 173, but 8,192 x 5,120 in bf16 82 instead of 70; a row's loads
//    before the row ahead is done: 185);
//  - rows to int8, 24,576 of 2,048 (151 MB) 25.7 us, 5.9 TB/s.
// A copy of 1 GiB on this card takes its bytes at 5.1 TB/s, a large read at 6.4.

#include "moe_common.h"

namespace {

using namespace moe;

typedef uint32_t vec2 __attribute__((ext_vector_type(2)));
typedef uint32_t vec4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short short2v __attribute__((ext_vector_type(2)));

// Values of a row that a lane takes at once: 16 bytes of the stream, so that an
// instruction reads and writes whole cache lines (8 values of float32, two pieces of
// 16 bytes, made half lines of each: 8,192 x 7,168 130 us, with 4 123).
template <bool kF32>
constexpr int kPieceOf = kF32 ? 4 : 8;
constexpr int kMostRow = 1 << 16;   // values of a row of the quantiser
constexpr int kMostNorm = 1 << 15;  // and of the norm and its gradient
constexpr int kMostWaves = 16;      // waves of a workgroup
constexpr int kMostGroups = 1 << 21;

// N values of a row: what a lane takes at once.
template <int N>
struct Row {
  float v[N];
};

template <int N>
struct Bf16;
template <>
struct Bf16<4> {
  typedef bf16x4 type;
};
template <>
struct Bf16<8> {
  typedef bf16x8 type;
};

template <int N>
__device__ __forceinline__ Row<N> widen(typename Bf16<N>::type p) {
  Row<N> r;
#pragma unroll
  for (int i = 0; i < N; ++i) r.v[i] = float(p[i]);
  return r;
}

template <int N>
__device__ __forceinline__ typename Bf16<N>::type narrow(const Row<N>& r) {
  typename Bf16<N>::type p;
#pragma unroll
  for (int i = 0; i < N; ++i) p[i] = __bf16(r.v[i]);
  return p;
}

// Piece `at` (of N values each) of a tensor of bf16 or of float32.
template <bool kF32, int N>
struct Piece;
template <int N>
struct Piece<false, N> {
  typename Bf16<N>::type p;
  __device__ __forceinline__ void load(const void* t, int64_t at) {
    p = static_cast<const typename Bf16<N>::type*>(t)[at];
  }
  __device__ __forceinline__ Row<N> get() const { return widen<N>(p); }
};
template <int N>
struct Piece<true, N> {
  f32x4 p[N / 4];
  __device__ __forceinline__ void load(const void* t, int64_t at) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) p[i] = static_cast<const f32x4*>(t)[N / 4 * at + i];
  }
  __device__ __forceinline__ Row<N> get() const {
    Row<N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.v[i] = p[i / 4][i % 4];
    return r;
  }
};

template <typename V, bool kStream>
__device__ __forceinline__ void store(void* t, int64_t at, const V& v) {
  if (kStream)
    __builtin_nontemporal_store(v, static_cast<V*>(t) + at);
  else
    static_cast<V*>(t)[at] = v;
}

// kStream: nontemporal, for what this kernel does not read again (4,093 x 5,120 in
// bf16 with MXFP8 codes 37 us without, 29 us with).
template <bool kF32, bool kStream, int N>
__device__ __forceinline__ void store_piece(void* t, int64_t at, const Row<N>& r) {
  if (kF32) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      store<f32x4, kStream>(t, N / 4 * at + i,
                            f32x4{r.v[4 * i], r.v[4 * i + 1], r.v[4 * i + 2], r.v[4 * i + 3]});
  } else {
    store<typename Bf16<N>::type, kStream>(t, at, narrow<N>(r));
  }
}

// Codes of N values, a byte each.
template <int N>
struct Codes {
  uint32_t w[N / 4];
};

__device__ __forceinline__ void store_codes(void* t, int64_t at, const Codes<8>& c) {
  store<vec2, true>(t, at, vec2{c.w[0], c.w[1]});
}
__device__ __forceinline__ void store_codes(void* t, int64_t at, const Codes<4>& c) {
  store<uint32_t, true>(t, at, c.w[0]);
}

// A value's magnitude as bits, which order as the magnitudes do, an infinity
// above the finite ones and a NaN above all.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

template <int kCtrl, int kRowMask = 0xF>
__device__ __forceinline__ uint32_t dpp_bits(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(int(v), int(v), kCtrl, kRowMask, 0xF, false));
}

__device__ __forceinline__ uint32_t wave_max_bits(uint32_t v) {
  v = max(v, dpp_bits<kRowShr + 1>(v));
  v = max(v, dpp_bits<kRowShr + 2>(v));
  v = max(v, dpp_bits<kRowShr + 4>(v));
  v = max(v, dpp_bits<kRowShr + 8>(v));
  v = max(v, dpp_bits<kRowBcast15, 0xA>(v));
  v = max(v, dpp_bits<kRowBcast31, 0xC>(v));
  return uint32_t(read_lane(int(v), 63));
}

// Of all waves of the workgroup, in wave order: the same in every wave. `at`:
// LDS that the last join does not use (one barrier a join).
__device__ __forceinline__ float join_sum(float v, float* at, int wave, int waves) {
  v = wave_sum(v);
  if (waves == 1) return v;
  if (lane_id() == 0) at[wave] = v;
  __syncthreads();
  float total = 0.0f;
  for (int w = 0; w < waves; ++w) total += at[w];
  return total;
}

__device__ __forceinline__ uint32_t join_max(uint32_t v, uint32_t* at, int wave, int waves) {
  v = wave_max_bits(v);
  if (waves == 1) return v;
  if (lane_id() == 0) at[wave] = v;
  __syncthreads();
  uint32_t total = 0;
  for (int w = 0; w < waves; ++w) total = max(total, at[w]);
  return total;
}

// A row's values in 127ths of the largest magnitude `top` (its bits). The scale
// is top / 127 and the factor 127 * (1 / top), rounded at each step; a code is the
// nearest whole number to the float32 product v * factor, so that only a quotient
// next to the middle between two codes may go to either. Tops whose reciprocal
// would come near the ends of float32's range are moved by 2^64 first, with the
// values.
struct Int8Scale {
  float scale, factor;  // factor 0: all codes are 0 (a row of zeros, or not finite)
  float move;
  __device__ __forceinline__ explicit Int8Scale(uint32_t top) {
    const float t = __uint_as_float(top);
    const bool finite = top < 0x7F800000u;
    move = t < 0x1p-64f ? 0x1p64f : t > 0x1p64f ? 0x1p-64f : 1.0f;
    scale = finite ? t / 127.0f : __uint_as_float(0x7FC00000u);
    factor = finite && top > 0 ? 127.0f * (1.0f / (t * move)) : 0.0f;
  }
  template <int N>
  __device__ __forceinline__ Codes<N> codes(Row<N> r) const {
    Codes<N> q = {};
    if (factor == 0.0f) return q;  // uniform, as `move` is
    if (move != 1.0f) {
#pragma unroll
      for (int i = 0; i < N; ++i) r.v[i] *= move;
    }
    // The product plus 1.5 * 2^23 has the nearest whole number in its low bits (as
    // ties to even; the two must not become one fma), the code in its low byte.
    uint32_t b[N];
    {
#pragma clang fp contract(off)
#pragma unroll
      for (int i = 0; i < N; ++i) b[i] = __float_as_uint(r.v[i] * factor + 0x1.8p23f);
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint32_t* p = b + 4 * i;
      const uint32_t lo = __builtin_amdgcn_perm(p[1], p[0], 0x0C0C0400u);
      const uint32_t hi = __builtin_amdgcn_perm(p[3], p[2], 0x0C0C0400u);
      q.w[i] = lo | hi << 16;
    }
    return q;
  }
};

// Four float32 divided by a power of two and rounded to e4m3 by the scaled
// conversion (nearest, ties to even). It turns a magnitude that rounds past 448
// into NaN (0x7F with the sign); among finite values that can only be such an
// overflow, so those bytes are lowered by one, to +-448.
__device__ __forceinline__ uint32_t e4m3x4(const float* v, float scale) {
  short2v r = {0, 0};
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, v[0], v[1], scale, false);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, v[2], v[3], scale, true);
  const uint32_t x = __builtin_bit_cast(uint32_t, r);
  const uint32_t nan_bytes = ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  return x - (nan_bytes >> 7);
}

// MXFP8 codes of a lane's piece and the scale byte of its block of 32 values,
// which 32 / N neighbouring lanes hold (all of a block, or none).
template <int N>
__device__ __forceinline__ Codes<N> mxfp8_codes(const Row<N>& r, uint32_t* scale_byte) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) top = max(top, magnitude(r.v[i]));
  top = max(top, dpp_bits<0xB1>(top));  // lanes 1 0 3 2 of each four
  top = max(top, dpp_bits<0x4E>(top));  // lanes 2 3 0 1
  if (N == 4) top = max(top, dpp_bits<0x141>(top));  // each eight lanes in reverse
  Codes<N> q = {};
  if (top >= 0x7F800000u) {  // NaN codes with the value's sign
    *scale_byte = 0xFF;
#pragma unroll
    for (int i = 0; i < N; ++i)
      q.w[i / 4] |= ((__float_as_uint(r.v[i]) >> 24 & 0x80u) | 0x7Fu) << (i % 4 * 8);
    return q;
  }
  // floor(log2(top)) - 8, at least -127: a subnormal top is below that anyway
  const int e = max(-127, int(top >> 23) - 127 - 8);
  *scale_byte = uint32_t(e + 127);
  const float scale = __uint_as_float(uint32_t(e + 127) << 23);  // E8M0 byte as an exponent
#pragma unroll
  for (int i = 0; i < N / 4; ++i) q.w[i] = e4m3x4(r.v + 4 * i, scale);
  return q;
}

// ---------------------------------------------------------------------------
// The norm

enum : int { kNone = 0, kInt8 = 1, kMxfp8 = 2 };

struct NormArgs {
  const void *x, *residual, *weight;
  void* sum;
  uint16_t* out;
  void *q, *q_scale;
  float* inv;
  float eps;
  int T, H;
};

// One row per workgroup at a time. The sum is rounded to the stream's type
// before anything else is made of it: the norm is of what the next layer, and
// the gradient, read. The squares are added in 32 bits, each lane's own first,
// then over the wave and the waves; the row is divided by a root that is
// correctly rounded.
template <bool kF32, bool kWeightF32, int kFmt, int NC>
__global__ __launch_bounds__(kMostWaves * kWave) void norm_rows(NormArgs a) {
  __shared__ float part[2][kMostWaves];
  __shared__ uint32_t tops[2][kMostWaves];
  const int waves = blockDim.x / kWave, wave = wave_in_block();
  constexpr int N = kPieceOf<kF32>;
  const int pieces = a.H / N;
  int turn = 0;
  for (int row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
    const int64_t at0 = int64_t(row) * pieces;
    Piece<false, N> x[NC];
    Piece<kF32, N> res[NC];
    Piece<kWeightF32, N> w[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int p = i * blockDim.x + threadIdx.x;
      if (p < pieces) {
        x[i].load(a.x, at0 + p);
        if (a.residual) res[i].load(a.residual, at0 + p);
        w[i].load(a.weight, p);
      }
    }
    Row<N> h[NC];
    float squares = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int p = i * blockDim.x + threadIdx.x;
      if (p < pieces) {
        h[i] = x[i].get();
        if (a.residual) {
          const Row<N> r = res[i].get();
#pragma unroll
          for (int j = 0; j < N; ++j) h[i].v[j] += r.v[j];
          if (!kF32) h[i] = widen<N>(narrow<N>(h[i]));
          store_piece<kF32, true>(a.sum, at0 + p, h[i]);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) squares = fmaf(h[i].v[j], h[i].v[j], squares);
      }
    }
    const float total = join_sum(squares, part[turn], wave, waves);
    const float inv = 1.0f / sqrtf(total / float(a.H) + a.eps);
    if (a.inv && threadIdx.x == 0) a.inv[row] = inv;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int p = i * blockDim.x + threadIdx.x;
      if (p < pieces) {
        const Row<N> g = w[i].get();
#pragma unroll
        for (int j = 0; j < N; ++j) {
          h[i].v[j] = h[i].v[j] * inv * g.v[j];
          if (kFmt == kInt8) top = max(top, magnitude(h[i].v[j]));
        }
        if (a.out) store_piece<false, true>(a.out, at0 + p, h[i]);
        if (kFmt == kMxfp8) {
          uint32_t byte;
          store_codes(a.q, at0 + p, mxfp8_codes(h[i], &byte));
          if (p % (32 / N) == 0)
            static_cast<uint8_t*>(a.q_scale)[(at0 + p) / (32 / N)] = uint8_t(byte);
        }
      }
    }
    if (kFmt == kInt8) {
      const Int8Scale s(join_max(top, tops[turn], wave, waves));
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int p = i * blockDim.x + threadIdx.x;
        if (p < pieces) store_codes(a.q, at0 + p, s.codes(h[i]));
      }
      if (threadIdx.x == 0) static_cast<float*>(a.q_scale)[row] = s.scale;
    }
  }
}

// ---------------------------------------------------------------------------
// Its gradient

struct NormGradArgs {
  const uint16_t* d_out;
  const void *h, *weight, *d_sum;
  const float* inv;
  uint16_t* d_x;
  void* d_res;
  float* part;  // [gridDim.x][H]: each workgroup's share of the weight's gradient, or NULL
  int T, H;
  int waves, at_once;  // waves a row, rows a workgroup
};

// Rows that a thread adds up in one float32 value, at most.
constexpr int kShortSum = 16;

// With g = d_out * w and unit = h * inv: d_h = inv * (g - unit * mean(g * unit))
// + d_sum. A workgroup takes `at_once` rows at a time, W waves each, and keeps the
// sums of d_out * unit in registers; at the end its rows' meet in LDS, one after
// the other, and norm_grad_join adds up the workgroups' in a fixed order.
//
// kLong: a thread adds up more than kShortSum rows, and one float32 sum's error would
// grow with them (2^23 rows of 8 equal values, 1,024 a thread: 1e-5 of the sum). So
// after every kShortSum rows the sums in registers are added to two float32 values each,
// what the addition to the one rounds off going to the other. These lie in LDS as long
// as two workgroups of a CU have room for both (up to 8 sums a thread); else the first
// has the workgroup's row of `part`. It costs 1% up to 8,192 values a row and 2 to 8%
// beyond (16,384 rows of 10,240 in bf16 256 us, one sum 247; with the second values
// brought up to date at every row, in LDS, 310). With 16 sums a thread in bf16 the
// registers are held to 80, as without kLong: two workgroups of up to 12 waves a CU
// (82 registers: 292 us).
template <bool kF32, bool kWeightF32, int NC, bool kLong>
__global__ __launch_bounds__(kMostWaves * kWave)
__attribute__((amdgpu_waves_per_eu(kLong && !kF32 && NC == 2 ? 6 : 4))) void norm_grad(
    NormGradArgs a) {
  constexpr int N = kPieceOf<kF32>;
  constexpr int kSums = NC * kMostWaves * kWave * N;  // of a workgroup
  constexpr bool kFirstInLds = NC * N <= 8;
  __shared__ float part[2][kMostWaves];
  __shared__ __align__(16) float joined[kLong ? (kFirstInLds ? 2 : 1) * kSums : kSums / 2];
  const int W = a.waves, threads = W * kWave;
  const int mine = wave_in_block() / W, wave = wave_in_block() % W;  // its row of those at once
  const int thread = wave * kWave + lane_id();
  const int pieces = a.H / N;
  Row<N> w[NC], dw[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int p = i * threads + thread;
    Piece<kWeightF32, N> piece;
    if (p < pieces) {
      piece.load(a.weight, p);
      w[i] = piece.get();
    }
#pragma unroll
    for (int j = 0; j < N; ++j) dw[i].v[j] = 0.0f;
  }
  // Adds the sums to their two parts, which are 0 before the `begin`ning, or at the
  // `end` makes them of both. In LDS 4 neighbouring sums of all threads lie next to each
  // other; in `part` (at_once is 1 then) the sums lie as they do at the end.
  int rows = 0;
  auto empty = [&](bool begin, bool end) {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));  // no addresses of this kept in registers over the rows
    f32x4* low = reinterpret_cast<f32x4*>(joined) + t;
    f32x4* first = low + kSums / 4;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int p = i * threads + (kFirstInLds ? thread : t);
      if (p < pieces) {
        if (!kFirstInLds)
          first = reinterpret_cast<f32x4*>(a.part) + (int64_t(blockIdx.x) * pieces + p) * (N / 4);
#pragma unroll
        for (int k = 0; k < N / 4; ++k) {
          f32x4& one_at = first[kFirstInLds ? (i * (N / 4) + k) * blockDim.x : k];
          f32x4& two_at = low[(i * (N / 4) + k) * blockDim.x];
          f32x4 one = {0, 0, 0, 0}, two = {0, 0, 0, 0};
          if (!begin) one = one_at, two = two_at;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float& sum = dw[i].v[4 * k + j];
            const float add = end && rows % kShortSum == 0 ? 0.0f : sum;
            const float now = one[j] + add, step = now - one[j];
            two[j] += (one[j] - (now - step)) + (add - step);
            one[j] = now;
            const float both = now + two[j];  // (none where a sum is not finite)
            if (end) sum = fabsf(both) < __builtin_inff() ? both : now;
          }
          if (!end) one_at = one, two_at = two;
        }
      }
    }
  };
  int turn = 0;
  for (int row0 = blockIdx.x * a.at_once; row0 < a.T; row0 += gridDim.x * a.at_once, turn ^= 1) {
    const int row = row0 + mine;
    const bool live = row < a.T;
    const int64_t at0 = int64_t(row) * pieces;
    if (kLong) {  // (not where they are added to their parts: it took 3 more registers)
      const bool anew = rows % kShortSum == 0;
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) dw[i].v[j] = anew ? 0.0f : dw[i].v[j];
    }
    Piece<false, N> d[NC];
    Piece<kF32, N> h[NC], through[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int p = i * threads + thread;
      if (live && p < pieces) {
        d[i].load(a.d_out, at0 + p);
        h[i].load(a.h, at0 + p);
        if (a.d_sum) through[i].load(a.d_sum, at0 + p);
      }
    }
    const float inv = live ? a.inv[row] : 0.0f;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int p = i * threads + thread;
      if (live && p < pieces) {
        const Row<N> dd = d[i].get(), hh = h[i].get();
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float unit = hh.v[j] * inv;
          dw[i].v[j] = fmaf(dd.v[j], unit, dw[i].v[j]);
          dot = fmaf(dd.v[j] * w[i].v[j], unit, dot);
        }
      }
    }
    const float mean = join_sum(dot, part[turn] + mine * W, wave, W) / float(a.H);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int p = i * threads + thread;
      if (live && p < pieces) {
        const Row<N> dd = d[i].get(), hh = h[i].get();
        Row<N> r;
#pragma unroll
        for (int j = 0; j < N; ++j)
          r.v[j] = inv * (dd.v[j] * w[i].v[j] - hh.v[j] * inv * mean);
        if (a.d_sum) {
          const Row<N> t = through[i].get();
#pragma unroll
          for (int j = 0; j < N; ++j) r.v[j] += t.v[j];
        }
        if (a.d_res) store_piece<kF32, kF32>(a.d_res, at0 + p, r);
        if (a.d_x) store_piece<false, true>(a.d_x, at0 + p, r);
      }
    }
    if (kLong && ++rows % kShortSum == 0) empty(rows == kShortSum, false);
  }
  if (!a.part) return;
  if (kLong) {
    empty(rows < kShortSum, true);
    __syncthreads();  // the parts make room for the rows' sums
  }
  for (int r = 1; r < a.at_once; ++r) {  // (at_once > 1: at most half the waves a row)
    if (mine == r) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int p = i * threads + thread;
        if (p < pieces) {
          if (r > 1) {
#pragma unroll
            for (int j = 0; j < N; ++j) dw[i].v[j] += joined[p * N + j];
          }
#pragma unroll
          for (int j = 0; j < N; ++j) joined[p * N + j] = dw[i].v[j];
        }
      }
    }
    __syncthreads();
  }
  if (mine == 0) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int p = i * threads + thread;
      if (p < pieces) {
        if (a.at_once > 1) {
#pragma unroll
          for (int j = 0; j < N; ++j) dw[i].v[j] += joined[p * N + j];
        }
        store_piece<true, false>(a.part, int64_t(blockIdx.x) * pieces + p, dw[i]);
      }
    }
  }
}

// d_weight[c] = the sum of part[.][c]: 32 columns a workgroup, each half wave
// every 32nd row, joined in 64 bits in their order.
constexpr int kJoinCols = kWave / 2;
__global__ __launch_bounds__(kMostWaves * kWave) void norm_grad_join(const float* part, int groups,
                                                                     int H, float* d_weight) {
  __shared__ double sums[2 * kMostWaves][kJoinCols];
  const int at = threadIdx.x / kJoinCols, col = threadIdx.x % kJoinCols;
  const int c = blockIdx.x * kJoinCols + col;
  double total = 0.0;
  if (c < H) {
#pragma unroll 8
    for (int g = at; g < groups; g += 2 * kMostWaves) total += double(part[int64_t(g) * H + c]);
  }
  sums[at][col] = total;
  __syncthreads();
  if (at == 0 && c < H) {
    for (int o = 1; o < 2 * kMostWaves; ++o) total += sums[o][col];
    d_weight[c] = float(total);
  }
}

// ---------------------------------------------------------------------------
// Rows to 8-bit integers

struct QuantArgs {
  const uint16_t* rows;
  const int32_t* pair_row;
  int8_t* q;
  float* scale;
  int32_t* err;
  int64_t cap, count;
  int H;
};

// kWide: a row per workgroup; else a row per wave.
template <bool kWide, int NC>
__global__ __launch_bounds__(kMostWaves * kWave) void quantise_rows(QuantArgs a) {
  __shared__ uint32_t tops[2][kMostWaves];
  const int waves = kWide ? blockDim.x / kWave : 1, wave = kWide ? wave_in_block() : 0;
  const int thread = kWide ? threadIdx.x : lane_id(), threads = kWide ? blockDim.x : kWave;
  constexpr int N = kPieceOf<false>;
  const int pieces = a.H / N;
  const int64_t stride = kWide ? gridDim.x : int64_t(gridDim.x) * (blockDim.x / kWave);
  int64_t i = kWide ? blockIdx.x : int64_t(blockIdx.x) * (blockDim.x / kWave) + wave_in_block();
  for (int turn = 0; i < a.count; i += stride) {
    int64_t row = i;
    if (a.pair_row) row = __builtin_amdgcn_readfirstlane(a.pair_row[i]);
    if (row >= a.cap && thread == 0) flag_error(a.err, MOE_ERRBIT_EXPERT_CAP);
    if (row < 0 || row >= a.cap) continue;  // the same for all that share the row
    const int64_t at0 = row * pieces;
    Piece<false, N> x[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int p = c * threads + thread;
      if (p < pieces) x[c].load(a.rows, at0 + p);
    }
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int p = c * threads + thread;
      if (p < pieces) {
        const Row<N> r = x[c].get();
#pragma unroll
        for (int j = 0; j < N; ++j) top = max(top, magnitude(r.v[j]));
      }
    }
    const Int8Scale s(join_max(top, tops[turn], wave, waves));
    turn ^= 1;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int p = c * threads + thread;
      if (p < pieces) store_codes(a.q, at0 + p, s.codes(x[c].get()));
    }
    if (thread == 0) a.scale[row] = s.scale;
  }
}

// ---------------------------------------------------------------------------
// Launches

int waves_for(int pieces, int each) {
  return std::max(1, (pieces + each * kWave - 1) / (each * kWave));
}

// Pieces a lane: as few as 16 waves allow.
int pieces_a_lane(int pieces) {
  for (int each = 1;; each *= 2)
    if (waves_for(pieces, each) <= kMostWaves) return each;
}

template <bool kF32, bool kWeightF32, int kFmt>
void launch_norm(int each, dim3 grid, int threads, hipStream_t st, const NormArgs& a) {
  switch (each) {
    case 1: norm_rows<kF32, kWeightF32, kFmt, 1><<<grid, threads, 0, st>>>(a); break;
    case 2: norm_rows<kF32, kWeightF32, kFmt, 2><<<grid, threads, 0, st>>>(a); break;
    case 4: norm_rows<kF32, kWeightF32, kFmt, 4><<<grid, threads, 0, st>>>(a); break;
    default:  // only a float32 stream has as many pieces
      norm_rows<kF32, kWeightF32, kFmt, kF32 ? 8 : 4><<<grid, threads, 0, st>>>(a);
  }
}

template <bool kF32, bool kWeightF32>
void launch_norm(int fmt, int each, dim3 grid, int threads, hipStream_t st, const NormArgs& a) {
  if (fmt == kInt8)
    launch_norm<kF32, kWeightF32, kInt8>(each, grid, threads, st, a);
  else if (fmt == kMxfp8)
    launch_norm<kF32, kWeightF32, kMxfp8>(each, grid, threads, st, a);
  else
    launch_norm<kF32, kWeightF32, kNone>(each, grid, threads, st, a);
}

template <bool kF32, bool kWeightF32, bool kLong>
void launch_grad(int each, dim3 grid, int threads, hipStream_t st, const NormGradArgs& a) {
  switch (each) {
    case 1: norm_grad<kF32, kWeightF32, 1, kLong><<<grid, threads, 0, st>>>(a); break;
    case 2: norm_grad<kF32, kWeightF32, 2, kLong><<<grid, threads, 0, st>>>(a); break;
    case 4: norm_grad<kF32, kWeightF32, 4, kLong><<<grid, threads, 0, st>>>(a); break;
    default:  // only a float32 stream has as many pieces
      norm_grad<kF32, kWeightF32, kF32 ? 8 : 4, kLong><<<grid, threads, 0, st>>>(a);
  }
}

template <bool kF32, bool kWeightF32>
void launch_grad(bool is_long, int each, dim3 grid, int threads, hipStream_t st,
                 const NormGradArgs& a) {
  if (is_long)
    launch_grad<kF32, kWeightF32, true>(each, grid, threads, st, a);
  else
    launch_grad<kF32, kWeightF32, false>(each, grid, threads, st, a);
}

template <bool kWide>
void launch_quant(int each, dim3 grid, int threads, hipStream_t st, const QuantArgs& a) {
  if constexpr (kWide) {
    if (each == 4)
      quantise_rows<true, 4><<<grid, threads, 0, st>>>(a);
    else
      quantise_rows<true, 8><<<grid, threads, 0, st>>>(a);
  } else {
    switch (each) {
      case 1: quantise_rows<false, 1><<<grid, threads, 0, st>>>(a); break;
      case 2: quantise_rows<false, 2><<<grid, threads, 0, st>>>(a); break;
      default: quantise_rows<false, 4><<<grid, threads, 0, st>>>(a);
    }
  }
}

bool norm_shape_ok(const moe_shape_t* s, int stream_type, int weight_type) {
  return shape_ok(s) && s->H <= kMostNorm &&
         (stream_type == MOE_TYPE_F32 || stream_type == MOE_TYPE_BF16) &&
         (weight_type == MOE_TYPE_F32 || weight_type == MOE_TYPE_BF16);
}

// Workgroups of the gradient, at most: two for each CU. All are resident at once where a
// row has at most 8,192 values; the registers of longer ones leave a CU 24 waves (16 sums a
// thread in bf16), 20 or 16 (in float32) or 16 (32 sums), so that of workgroups of up to 16
// waves it may hold only one at a time.
constexpr int kGradGroups = 512;

}  // namespace

extern "C" {

int moe_norm(const moe_shape_t* shape, int stream_type, const uint16_t* x, const void* residual,
             void* sum, int weight_type, const void* weight, float eps, uint16_t* out, int format,
             void* q, void* q_scale, float* inv_rms, void* stream) {
  if (!norm_shape_ok(shape, stream_type, weight_type)) return MOE_ERR_ARG;
  if (!(eps > 0.0f) || !(eps < __builtin_inff())) return MOE_ERR_ARG;
  if (format != 0 && format != MOE_ROWS_INT8 && format != MOE_WIRE_MXFP8) return MOE_ERR_ARG;
  if (format == MOE_WIRE_MXFP8 && shape->H % 32 != 0) return MOE_ERR_ARG;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(sum, 16) || !aligned(weight, 16) ||
      !aligned(out, 16) || !aligned(q, 16) || !aligned(q_scale, 4) || !aligned(inv_rms, 4))
    return MOE_ERR_ARG;
  if (shape->T == 0) return MOE_OK;  // empty tensors have no address
  if (!x || !weight || (!out && !q)) return MOE_ERR_ARG;
  if ((residual == nullptr) != (sum == nullptr)) return MOE_ERR_ARG;
  if ((format != 0) != (q != nullptr) || (format != 0) != (q_scale != nullptr)) return MOE_ERR_ARG;
  const NormArgs a{x, residual, weight, sum, out, q, q_scale, inv_rms, eps, shape->T, shape->H};
  const bool f32 = stream_type == MOE_TYPE_F32;
  const int pieces = shape->H / (f32 ? kPieceOf<true> : kPieceOf<false>);
  // The maximum of 8-bit rows is a second wait for the whole row: two pieces a lane,
  // and more rows at once on a CU (4,093 x 7,168 39 us against 49, 64 x 5,120 4.4 against 4.1).
  const int each = std::max(format == MOE_ROWS_INT8 && shape->T > 256 ? 2 : 1,
                            pieces_a_lane(pieces));
  const int threads = waves_for(pieces, each) * kWave;
  const dim3 grid(std::min(shape->T, kMostGroups));
  const int fmt = format == 0 ? kNone : format == MOE_ROWS_INT8 ? kInt8 : kMxfp8;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (f32) {
    if (weight_type == MOE_TYPE_F32)
      launch_norm<true, true>(fmt, each, grid, threads, st, a);
    else
      launch_norm<true, false>(fmt, each, grid, threads, st, a);
  } else {
    if (weight_type == MOE_TYPE_F32)
      launch_norm<false, true>(fmt, each, grid, threads, st, a);
    else
      launch_norm<false, false>(fmt, each, grid, threads, st, a);
  }
  return launch_status();
}

size_t moe_norm_workspace_bytes(const moe_shape_t* shape) {
  if (!norm_shape_ok(shape, MOE_TYPE_F32, MOE_TYPE_F32)) return 0;
  return size_t(std::min(shape->T, kGradGroups)) * shape->H * sizeof(float);
}

int moe_norm_backward(const moe_shape_t* shape, int stream_type, const uint16_t* d_out,
                      const void* sum, const float* inv_rms, int weight_type, const void* weight,
                      const void* d_sum, uint16_t* d_x, void* d_residual, float* d_weight,
                      void* workspace, size_t workspace_bytes, void* stream) {
  if (!norm_shape_ok(shape, stream_type, weight_type)) return MOE_ERR_ARG;
  if (!aligned(d_out, 16) || !aligned(sum, 16) || !aligned(inv_rms, 4) || !aligned(weight, 16) ||
      !aligned(d_sum, 16) || !aligned(d_x, 16) || !aligned(d_residual, 16) ||
      !aligned(d_weight, 4) || !aligned(workspace, 16))
    return MOE_ERR_ARG;
  const bool rows = shape->T > 0;
  if (rows && (!d_out || !sum || !inv_rms || !weight)) return MOE_ERR_ARG;
  if (rows && d_weight && (!workspace || workspace_bytes < moe_norm_workspace_bytes(shape)))
    return MOE_ERR_ARG;
  if (!rows && !d_weight) return MOE_OK;
  if (!d_x && !d_residual && !d_weight) return MOE_ERR_ARG;
  hipStream_t st = static_cast<hipStream_t>(stream);
  float* part = d_weight ? static_cast<float*>(workspace) : nullptr;
  int groups = 0;
  if (rows) {
    const bool f32 = stream_type == MOE_TYPE_F32;
    const int pieces = shape->H / (f32 ? kPieceOf<true> : kPieceOf<false>);
    // Two pieces a lane halve the waves a row, so that twice as many rows meet before
    // they reach memory: where every workgroup has one row, 509 x 5,120 in bf16 11.3
    // us against 13.6, 512 x 7,168 in float32 17.7 against 19.2; with 1,024 rows 17.8
    // against 16.0, with 64 7.9 against 6.8.
    const int each = std::max(shape->T > 128 && shape->T <= kGradGroups ? (f32 ? 4 : 2) : 1,
                              pieces_a_lane(pieces));
    const int waves = waves_for(pieces, each), at_once = kMostWaves / waves;
    const int threads = waves * at_once * kWave;
    groups = std::min((shape->T + at_once - 1) / at_once, kGradGroups);
    const NormGradArgs a{d_out,      sum,  weight,   d_sum,    inv_rms, d_x,
                         d_residual, part, shape->T, shape->H, waves,   at_once};
    const dim3 grid(groups);
    // (at_once is 1 then where a lane has more than 8 sums: rows of 9 waves and more)
    const bool is_long = d_weight && shape->T > int64_t(kShortSum) * groups * at_once;
    if (f32) {
      if (weight_type == MOE_TYPE_F32)
        launch_grad<true, true>(is_long, each, grid, threads, st, a);
      else
        launch_grad<true, false>(is_long, each, grid, threads, st, a);
    } else {
      if (weight_type == MOE_TYPE_F32)
        launch_grad<false, true>(is_long, each, grid, threads, st, a);
      else
        launch_grad<false, false>(is_long, each, grid, threads, st, a);
    }
    const int status = launch_status();
    if (status != MOE_OK || !d_weight) return status;
  }
  norm_grad_join<<<(shape->H + kJoinCols - 1) / kJoinCols, kMostWaves * kWave, 0, st>>>(
      part, groups, shape->H, d_weight);
  return launch_status();
}

int moe_quantise_rows(const moe_shape_t* shape, const uint16_t* rows, const int32_t* pair_row,
                      int64_t cap_expert, int8_t* q, float* scale, int32_t* err_word,
                      void* stream) {
  if (!shape_ok(shape) || shape->H > kMostRow || cap_expert < 0) return MOE_ERR_ARG;
  const int64_t count = int64_t(shape->T) * shape->k;
  if (!pair_row && count > cap_expert) return MOE_ERR_ARG;
  if (!aligned(rows, 16) || !aligned(pair_row, 4) || !aligned(q, 16) || !aligned(scale, 4))
    return MOE_ERR_ARG;
  if (count == 0) return MOE_OK;
  if (cap_expert > 0 && (!rows || !q || !scale)) return MOE_ERR_ARG;
  const QuantArgs a{rows, pair_row, q, scale, err_word, cap_expert, count, shape->H};
  const int pieces = shape->H / kPieceOf<false>;
  hipStream_t st = static_cast<hipStream_t>(stream);
  // A wave takes rows of up to 2,048 values alone; longer ones four pieces a lane,
  // few waves that wait for each other (16,384 rows of 5,120: one piece a lane 84
  // us, two 58, four 50, eight 52).
  if (pieces <= 4 * kWave) {
    const int64_t groups = (count + 3) / 4;
    const int each = pieces <= kWave ? 1 : pieces <= 2 * kWave ? 2 : 4;
    launch_quant<false>(each, dim3(uint32_t(std::min<int64_t>(groups, kMostGroups))), 4 * kWave, st,
                        a);
  } else {
    const int each = std::max(4, pieces_a_lane(pieces));
    launch_quant<true>(each, dim3(uint32_t(std::min<int64_t>(count, kMostGroups))),
                       waves_for(pieces, each) * kWave, st, a);
  }
  return launch_status();
}

}  // extern "C"
