// The norm before a layer, its gradient, and rows to 8-bit integers: HIP
// kernels for CDNA4 (gfx950, wave64) behind include/moe_dispatch.h.
//
// All three are one pass over their rows: a row lies in the registers of W
// waves (pieces of 8 values, NC of them a lane), is read once in 16-byte loads
// that are all on their way before the first is used, and its sum or maximum
// is joined through DPP and, with W > 1, 64 bytes of LDS. What bounds them is
// the memory: few bytes a value are computed on.

#include "moe_common.h"

namespace {

using namespace moe;

typedef uint32_t vec2 __attribute__((ext_vector_type(2)));
typedef uint32_t vec4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short short2v __attribute__((ext_vector_type(2)));

constexpr int kPiece = 8;           // values of a row that a lane takes at once
constexpr int kMostRow = 1 << 16;   // values of a row of the quantiser
constexpr int kMostNorm = 1 << 15;  // and of the norm and its gradient
constexpr int kMostWaves = 16;      // waves of a workgroup
constexpr int kMostGroups = 1 << 21;

struct Row8 {
  float v[kPiece];
};

__device__ __forceinline__ Row8 widen(bf16x8 p) {
  Row8 r;
#pragma unroll
  for (int i = 0; i < kPiece; ++i) r.v[i] = float(p[i]);
  return r;
}

__device__ __forceinline__ bf16x8 narrow(const Row8& r) {
  bf16x8 p;
#pragma unroll
  for (int i = 0; i < kPiece; ++i) p[i] = __bf16(r.v[i]);
  return p;
}

// Piece `at` (in pieces) of a tensor of bf16 or of float32.
template <bool kF32>
struct Piece;
template <>
struct Piece<false> {
  bf16x8 p;
  __device__ __forceinline__ void load(const void* t, int64_t at) {
    p = static_cast<const bf16x8*>(t)[at];
  }
  __device__ __forceinline__ Row8 get() const { return widen(p); }
};
template <>
struct Piece<true> {
  f32x4 p[2];
  __device__ __forceinline__ void load(const void* t, int64_t at) {
    p[0] = static_cast<const f32x4*>(t)[2 * at];
    p[1] = static_cast<const f32x4*>(t)[2 * at + 1];
  }
  __device__ __forceinline__ Row8 get() const {
    Row8 r;
#pragma unroll
    for (int i = 0; i < kPiece; ++i) r.v[i] = p[i / 4][i % 4];
    return r;
  }
};

template <bool kF32>
__device__ __forceinline__ void store_piece(void* t, int64_t at, const Row8& r) {
  if (kF32) {
    f32x4* to = static_cast<f32x4*>(t) + 2 * at;
    to[0] = f32x4{r.v[0], r.v[1], r.v[2], r.v[3]};
    to[1] = f32x4{r.v[4], r.v[5], r.v[6], r.v[7]};
  } else {
    static_cast<bf16x8*>(t)[at] = narrow(r);
  }
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
  __device__ __forceinline__ vec2 codes(Row8 r) const {
    vec2 q = {0, 0};
    if (factor == 0.0f) return q;  // uniform, as `move` is
    if (move != 1.0f) {
#pragma unroll
      for (int i = 0; i < kPiece; ++i) r.v[i] *= move;
    }
#pragma unroll
    for (int i = 0; i < kPiece; ++i)
      q[i / 4] |= uint32_t(int(__builtin_rintf(r.v[i] * factor)) & 0xFF) << (i % 4 * 8);
    return q;
  }
};

// Eight float32 divided by a power of two and rounded to e4m3 by the scaled
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
// which four neighbouring lanes hold (a block has all four or none).
__device__ __forceinline__ vec2 mxfp8_codes(const Row8& r, uint32_t* scale_byte) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kPiece; ++i) top = max(top, magnitude(r.v[i]));
  top = max(top, dpp_bits<0xB1>(top));  // lanes 1 0 3 2 of each four
  top = max(top, dpp_bits<0x4E>(top));  // lanes 2 3 0 1
  vec2 q;
  if (top >= 0x7F800000u) {  // NaN codes with the value's sign
    *scale_byte = 0xFF;
    q = vec2{0, 0};
#pragma unroll
    for (int i = 0; i < kPiece; ++i)
      q[i / 4] |= ((__float_as_uint(r.v[i]) >> 24 & 0x80u) | 0x7Fu) << (i % 4 * 8);
    return q;
  }
  // floor(log2(top)) - 8, at least -127: a subnormal top is below that anyway
  const int e = max(-127, int(top >> 23) - 127 - 8);
  *scale_byte = uint32_t(e + 127);
  const float scale = __uint_as_float(uint32_t(e + 127) << 23);  // E8M0 byte as an exponent
  q[0] = e4m3x4(r.v, scale);
  q[1] = e4m3x4(r.v + 4, scale);
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
  const int pieces = a.H / kPiece;
  int turn = 0;
  for (int row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
    const int64_t at0 = int64_t(row) * pieces;
    Piece<false> x[NC];
    Piece<kF32> res[NC];
    Piece<kWeightF32> w[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int p = i * blockDim.x + threadIdx.x;
      if (p < pieces) {
        x[i].load(a.x, at0 + p);
        if (a.residual) res[i].load(a.residual, at0 + p);
        w[i].load(a.weight, p);
      }
    }
    Row8 h[NC];
    float squares = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int p = i * blockDim.x + threadIdx.x;
      if (p < pieces) {
        h[i] = x[i].get();
        if (a.residual) {
          const Row8 r = res[i].get();
#pragma unroll
          for (int j = 0; j < kPiece; ++j) h[i].v[j] += r.v[j];
          if (!kF32) h[i] = widen(narrow(h[i]));
          store_piece<kF32>(a.sum, at0 + p, h[i]);
        }
#pragma unroll
        for (int j = 0; j < kPiece; ++j) squares = fmaf(h[i].v[j], h[i].v[j], squares);
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
        const Row8 g = w[i].get();
#pragma unroll
        for (int j = 0; j < kPiece; ++j) {
          h[i].v[j] = h[i].v[j] * inv * g.v[j];
          if (kFmt == kInt8) top = max(top, magnitude(h[i].v[j]));
        }
        if (a.out) store_piece<false>(a.out, at0 + p, h[i]);
        if (kFmt == kMxfp8) {
          uint32_t byte;
          static_cast<vec2*>(a.q)[at0 + p] = mxfp8_codes(h[i], &byte);
          if (p % 4 == 0) static_cast<uint8_t*>(a.q_scale)[(at0 + p) / 4] = uint8_t(byte);
        }
      }
    }
    if (kFmt == kInt8) {
      const Int8Scale s(join_max(top, tops[turn], wave, waves));
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int p = i * blockDim.x + threadIdx.x;
        if (p < pieces) static_cast<vec2*>(a.q)[at0 + p] = s.codes(h[i]);
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
};

// With g = d_out * w and unit = h * inv: d_h = inv * (g - unit * mean(g * unit))
// + d_sum. A workgroup takes every gridDim.x-th row and keeps the sum of d_out *
// unit over them in registers; norm_grad_join adds up the workgroups' in a fixed
// order.
template <bool kF32, bool kWeightF32, int NC>
__global__ __launch_bounds__(kMostWaves * kWave) void norm_grad(NormGradArgs a) {
  __shared__ float part[2][kMostWaves];
  const int waves = blockDim.x / kWave, wave = wave_in_block();
  const int pieces = a.H / kPiece;
  Row8 w[NC], dw[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int p = i * blockDim.x + threadIdx.x;
    Piece<kWeightF32> piece;
    if (p < pieces) {
      piece.load(a.weight, p);
      w[i] = piece.get();
    }
#pragma unroll
    for (int j = 0; j < kPiece; ++j) dw[i].v[j] = 0.0f;
  }
  int turn = 0;
  for (int row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
    const int64_t at0 = int64_t(row) * pieces;
    Piece<false> d[NC];
    Piece<kF32> h[NC], through[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int p = i * blockDim.x + threadIdx.x;
      if (p < pieces) {
        d[i].load(a.d_out, at0 + p);
        h[i].load(a.h, at0 + p);
        if (a.d_sum) through[i].load(a.d_sum, at0 + p);
      }
    }
    const float inv = a.inv[row];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int p = i * blockDim.x + threadIdx.x;
      if (p < pieces) {
        const Row8 dd = d[i].get(), hh = h[i].get();
#pragma unroll
        for (int j = 0; j < kPiece; ++j) {
          const float unit = hh.v[j] * inv;
          dw[i].v[j] = fmaf(dd.v[j], unit, dw[i].v[j]);
          dot = fmaf(dd.v[j] * w[i].v[j], unit, dot);
        }
      }
    }
    const float mean = join_sum(dot, part[turn], wave, waves) / float(a.H);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int p = i * blockDim.x + threadIdx.x;
      if (p < pieces) {
        const Row8 dd = d[i].get(), hh = h[i].get();
        Row8 r;
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
          r.v[j] = inv * (dd.v[j] * w[i].v[j] - hh.v[j] * inv * mean);
        if (a.d_sum) {
          const Row8 t = through[i].get();
#pragma unroll
          for (int j = 0; j < kPiece; ++j) r.v[j] += t.v[j];
        }
        if (a.d_res) store_piece<kF32>(a.d_res, at0 + p, r);
        if (a.d_x) store_piece<false>(a.d_x, at0 + p, r);
      }
    }
  }
  if (a.part) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int p = i * blockDim.x + threadIdx.x;
      if (p < pieces) store_piece<true>(a.part, int64_t(blockIdx.x) * pieces + p, dw[i]);
    }
  }
}

// d_weight[c] = the sum of part[.][c]: 64 columns a workgroup, each wave a
// sixteenth of the rows, joined in wave order in 64 bits.
__global__ __launch_bounds__(kMostWaves * kWave) void norm_grad_join(const float* part, int groups,
                                                                     int H, float* d_weight) {
  __shared__ double sums[kMostWaves][kWave];
  const int lane = lane_id(), wave = wave_in_block();
  const int c = blockIdx.x * kWave + lane;
  double total = 0.0;
  if (c < H) {
#pragma unroll 8
    for (int g = wave; g < groups; g += kMostWaves) total += double(part[int64_t(g) * H + c]);
  }
  sums[wave][lane] = total;
  __syncthreads();
  if (wave == 0 && c < H) {
    for (int w = 1; w < kMostWaves; ++w) total += sums[w][lane];
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
  const int pieces = a.H / kPiece;
  const int64_t stride = kWide ? gridDim.x : int64_t(gridDim.x) * (blockDim.x / kWave);
  int64_t i = kWide ? blockIdx.x : int64_t(blockIdx.x) * (blockDim.x / kWave) + wave_in_block();
  for (int turn = 0; i < a.count; i += stride) {
    int64_t row = i;
    if (a.pair_row) row = __builtin_amdgcn_readfirstlane(a.pair_row[i]);
    if (row >= a.cap && thread == 0) flag_error(a.err, MOE_ERRBIT_EXPERT_CAP);
    if (row < 0 || row >= a.cap) continue;  // the same for all that share the row
    const int64_t at0 = row * pieces;
    Piece<false> x[NC];
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
        const Row8 r = x[c].get();
#pragma unroll
        for (int j = 0; j < kPiece; ++j) top = max(top, magnitude(r.v[j]));
      }
    }
    const Int8Scale s(join_max(top, tops[turn], wave, waves));
    turn ^= 1;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int p = c * threads + thread;
      if (p < pieces) reinterpret_cast<vec2*>(a.q)[at0 + p] = s.codes(x[c].get());
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
    default: norm_rows<kF32, kWeightF32, kFmt, 4><<<grid, threads, 0, st>>>(a);
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

template <bool kF32, bool kWeightF32>
void launch_grad(int each, dim3 grid, int threads, hipStream_t st, const NormGradArgs& a) {
  switch (each) {
    case 1: norm_grad<kF32, kWeightF32, 1><<<grid, threads, 0, st>>>(a); break;
    case 2: norm_grad<kF32, kWeightF32, 2><<<grid, threads, 0, st>>>(a); break;
    default: norm_grad<kF32, kWeightF32, 4><<<grid, threads, 0, st>>>(a);
  }
}

template <bool kWide>
void launch_quant(int each, dim3 grid, int threads, hipStream_t st, const QuantArgs& a) {
  switch (each) {
    case 1: quantise_rows<kWide, 1><<<grid, threads, 0, st>>>(a); break;
    case 2: quantise_rows<kWide, 2><<<grid, threads, 0, st>>>(a); break;
    case 4: quantise_rows<kWide, 4><<<grid, threads, 0, st>>>(a); break;
    default: quantise_rows<kWide, 8><<<grid, threads, 0, st>>>(a);
  }
}

bool norm_shape_ok(const moe_shape_t* s, int stream_type, int weight_type) {
  return shape_ok(s) && s->H <= kMostNorm &&
         (stream_type == MOE_TYPE_F32 || stream_type == MOE_TYPE_BF16) &&
         (weight_type == MOE_TYPE_F32 || weight_type == MOE_TYPE_BF16);
}

// Workgroups of the gradient: as many as are resident at once (two of each CU),
// each with a row at least.
int grad_groups(int T) { return std::min(T, 512); }

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
  const int pieces = shape->H / kPiece;
  const int each = pieces_a_lane(pieces), threads = waves_for(pieces, each) * kWave;
  const dim3 grid(std::min(shape->T, kMostGroups));
  const int fmt = format == 0 ? kNone : format == MOE_ROWS_INT8 ? kInt8 : kMxfp8;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (stream_type == MOE_TYPE_F32) {
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
  return size_t(grad_groups(shape->T)) * shape->H * sizeof(float);
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
  const int groups = grad_groups(shape->T);
  float* part = d_weight ? static_cast<float*>(workspace) : nullptr;
  if (rows) {
    const NormGradArgs a{d_out, sum,        weight, d_sum,    inv_rms,
                         d_x,   d_residual, part,   shape->T, shape->H};
    const int pieces = shape->H / kPiece;
    const int each = pieces_a_lane(pieces), threads = waves_for(pieces, each) * kWave;
    const dim3 grid(groups);
    if (stream_type == MOE_TYPE_F32) {
      if (weight_type == MOE_TYPE_F32)
        launch_grad<true, true>(each, grid, threads, st, a);
      else
        launch_grad<true, false>(each, grid, threads, st, a);
    } else {
      if (weight_type == MOE_TYPE_F32)
        launch_grad<false, true>(each, grid, threads, st, a);
      else
        launch_grad<false, false>(each, grid, threads, st, a);
    }
    const int status = launch_status();
    if (status != MOE_OK || !d_weight) return status;
  }
  norm_grad_join<<<(shape->H + kWave - 1) / kWave, kMostWaves * kWave, 0, st>>>(part, groups,
                                                                                shape->H, d_weight);
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
  const int pieces = shape->H / kPiece;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (pieces <= 4 * kWave) {
    const int64_t groups = (count + 3) / 4;
    launch_quant<false>(pieces <= kWave ? 1 : pieces <= 2 * kWave ? 2 : 4,
                        dim3(uint32_t(std::min<int64_t>(groups, kMostGroups))), 4 * kWave, st, a);
  } else {
    const int each = pieces_a_lane(pieces);
    launch_quant<true>(each, dim3(uint32_t(std::min<int64_t>(count, kMostGroups))),
                       waves_for(pieces, each) * kWave, st, a);
  }
  return launch_status();
}

}  // extern "C"
