// Expert products with 4-bit weights: HIP kernels for CDNA4 (gfx950, wave64)
// behind include/moe_dispatch.h.
//
// Kernels
//  product_rows   one workgroup per (up to 16 * MT rows of one expert, 32 rows
//                 of its weights): the four waves split H, each expands its
//                 codes to bf16 in registers and feeds them to MFMA

#include "moe_common.h"

namespace {

using namespace moe;

typedef uint32_t vec4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kBlock = 256;
constexpr int kWaves = kBlock / kWave;
constexpr int kTile = 16;    // an MFMA tile: 16 weight rows, 16 buffer rows
constexpr int kChunk = 32;   // values of H in 16 bytes of codes

struct ProductArgs {
  const uint16_t* rows;
  const int32_t* counts;
  const int32_t* offsets;
  const uint8_t* w_q;
  const uint8_t* w_scale;
  const float* factor;
  uint16_t* out;
  int32_t* err;
  int64_t cap;
  int E, K, N, wide;  // wide: columns of out
  int tiles, slots;   // column tiles, row chunks in the grid
};

// Eight codes (a word) times a power of two, as bf16: exact, e2m1 has two
// significant bits.
__device__ __forceinline__ bf16x8 expand_e8m0(uint32_t w, float scale) {
  union {
    bf16x2 p[4];
    bf16x8 v;
  } r;
  r.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
  r.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
  r.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
  r.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  return r.v;
}

// Eight codes times an E4M3 scale, as bf16: exact too (2 + 4 significant bits).
// The conversion takes powers of two only, so the scale is multiplied in floats.
__device__ __forceinline__ bf16x8 expand_e4m3(uint32_t w, float scale) {
  bf16x8 r;
  f32x2 p[4];
  p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
  p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
  p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[2 * i] = __bf16(p[i][0] * scale);
    r[2 * i + 1] = __bf16(p[i][1] * scale);
  }
  return r;
}

// The first rows of expert e in the buffer and how many are in use; rows the
// buffer does not hold are left out.
__device__ __forceinline__ int run_of(const ProductArgs& a, int e, int64_t* first) {
  const int64_t begin = a.offsets[e];
  int64_t n = min((int64_t)a.counts[e], (int64_t)a.offsets[e + 1] - begin);
  if (begin < 0) n = 0;
  if (n > 0 && begin + n > a.cap) {
    flag_error(a.err, MOE_ERRBIT_EXPERT_CAP);
    n = a.cap - begin;
  }
  *first = begin;
  return n > 0 ? int(n) : 0;
}

template <bool kE4M3, bool kSwiglu, int MT>
__global__ __launch_bounds__(kBlock) void product_rows(ProductArgs a) {
  constexpr int kRows = kTile * MT;
  constexpr int kPer = kMaxExperts / kBlock;  // experts a thread looks at
  __shared__ float part[kWaves][2 * MT * 4][kWave];
  __shared__ int wave_total[kWaves];
  __shared__ int found[4];
  const int tid = threadIdx.x, lane = lane_id(), wave = wave_in_block();
  const int tile = blockIdx.x % a.tiles;
  int chunk = blockIdx.x / a.tiles;

  // Row chunks of the experts in order: those of experts [kPer * tid, ..) are
  // numbered from `base`.
  int chunks[kPer], mine = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int e = kPer * tid + q;
    int64_t first;
    chunks[q] = e < a.E ? (run_of(a, e, &first) + kRows - 1) / kRows : 0;
    mine += chunks[q];
  }
  int base = mine;
  for (int s = 1; s < kWave; s <<= 1) {
    const int up = __shfl_up(base, s);
    if (lane >= s) base += up;
  }
  if (lane == kWave - 1) wave_total[wave] = base;
  __syncthreads();
  base -= mine;
  int total = 0;
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) base += wave_total[w];
    total += wave_total[w];
  }

  for (; chunk < total; chunk += a.slots) {
    if (chunk >= base && chunk < base + mine) {
      int c = chunk - base;
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        if (c >= 0 && c < chunks[q]) {
          found[0] = kPer * tid + q;
          found[1] = c;
        }
        c -= chunks[q];
      }
    }
    __syncthreads();
    const int e = __builtin_amdgcn_readfirstlane(found[0]);
    int64_t first;
    const int run = run_of(a, e, &first);
    const int r0 = __builtin_amdgcn_readfirstlane(found[1]) * kRows;
    const int nr = min(kRows, run - r0);
    first += r0;

    const int m = lane & 15, kq = lane >> 4;
    const int n0 = tile * (kSwiglu ? kTile : 2 * kTile);
    const int half = a.N / 2;
    int wrow[2];  // the weight rows of this lane, clamped
    wrow[0] = kSwiglu ? min(n0 + m, half - 1) : min(n0 + m, a.N - 1);
    wrow[1] = kSwiglu ? half + min(n0 + m, half - 1) : min(n0 + kTile + m, a.N - 1);
    const int nchunks = a.K / kChunk;
    const uint8_t* wq[2];
    const uint8_t* ws[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t r = (int64_t)e * a.N + wrow[h];
      wq[h] = a.w_q + r * (a.K / 2);
      ws[h] = a.w_scale + r * (kE4M3 ? a.K / 16 : a.K / 32);
    }
    const uint16_t* x[MT];
#pragma unroll
    for (int q = 0; q < MT; ++q)
      x[q] = a.rows + (first + min(q * kTile + m, nr - 1)) * a.K;

    f32x4 acc[2][MT];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < MT; ++q) acc[h][q] = f32x4{0, 0, 0, 0};

    for (int c0 = wave * 8; c0 < nchunks; c0 += kWaves * 8) {
      vec4 code[2][2];
      uint32_t sc[2][2];
      vec4 xv[2][MT][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int c = c0 + 4 * u + kq;
        const bool in = c < nchunks;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          code[u][h] = vec4{0, 0, 0, 0};
          sc[u][h] = 0;
          if (in) {
            code[u][h] = *reinterpret_cast<const vec4*>(wq[h] + (int64_t)c * 16);
            sc[u][h] = kE4M3 ? *reinterpret_cast<const uint16_t*>(ws[h] + 2 * c) : ws[h][c];
          }
        }
#pragma unroll
        for (int q = 0; q < MT; ++q)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            xv[u][q][j] = vec4{0, 0, 0, 0};
            if (in) xv[u][q][j] = *reinterpret_cast<const vec4*>(x[q] + c * kChunk + 8 * j);
          }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            bf16x8 w;
            if (kE4M3) {
              const float s = j < 2 ? __builtin_amdgcn_cvt_f32_fp8(sc[u][h], 0)
                                    : __builtin_amdgcn_cvt_f32_fp8(sc[u][h], 1);
              w = expand_e4m3(code[u][h][j], s);
            } else {
              w = expand_e8m0(code[u][h][j], __uint_as_float(sc[u][h] << 23));
            }
#pragma unroll
            for (int q = 0; q < MT; ++q)
              acc[h][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  w, __builtin_bit_cast(bf16x8, xv[u][q][j]), acc[h][q], 0, 0, 0);
          }
        }
    }

    // join the waves' parts: thread (wave i, lane) adds up element i of every
    // fragment of that lane, in wave order
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < MT; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[wave][(h * MT + q) * 4 + i][lane] = acc[h][q][i];
    __syncthreads();
    const float factor = a.factor ? a.factor[e] : 1.0f;
#pragma unroll
    for (int q = 0; q < MT; ++q) {
      float y[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        y[h] = 0.0f;
        for (int w = 0; w < kWaves; ++w) y[h] += part[w][(h * MT + q) * 4 + wave][lane];
        y[h] *= factor;
      }
      const int r = q * kTile + m;
      const int n = n0 + 4 * kq + wave;
      if (r < nr) {
        __bf16* out = reinterpret_cast<__bf16*>(a.out) + (first + r) * a.wide;
        if (kSwiglu) {
          if (n < half) out[n] = __bf16(y[0] / (1.0f + expf(-y[0])) * y[1]);
        } else {
          if (n < a.N) out[n] = __bf16(y[0]);
          if (n + kTile < a.N) out[n + kTile] = __bf16(y[1]);
        }
      }
    }
    __syncthreads();
  }
}

template <bool kE4M3, bool kSwiglu>
void launch_product(int mt, dim3 grid, hipStream_t st, const ProductArgs& a) {
  if (mt == 1)
    product_rows<kE4M3, kSwiglu, 1><<<grid, kBlock, 0, st>>>(a);
  else if (mt == 2)
    product_rows<kE4M3, kSwiglu, 2><<<grid, kBlock, 0, st>>>(a);
  else
    product_rows<kE4M3, kSwiglu, 4><<<grid, kBlock, 0, st>>>(a);
}

}  // namespace

extern "C" {

int moe_expert_product(const moe_shape_t* shape, int N, int format, int act,
                       const uint16_t* rows, const int32_t* expert_counts,
                       const int32_t* expert_offsets, int64_t cap_expert, const uint8_t* w_q,
                       const uint8_t* w_scale, const float* factor, uint16_t* out,
                       int32_t* err_word, void* stream) {
  if (!shape_ok(shape) || shape->H % kChunk != 0) return MOE_ERR_ARG;
  if (format != MOE_WIRE_MXFP4 && format != MOE_WIRE_NVFP4) return MOE_ERR_ARG;
  if (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU) return MOE_ERR_ARG;
  if (N < 1 || N > (1 << 24) || (act == MOE_ACT_SWIGLU && N % 2 != 0)) return MOE_ERR_ARG;
  if (cap_expert < 0) return MOE_ERR_ARG;
  const int64_t pairs = int64_t(shape->T) * shape->k;
  if (pairs == 0) return MOE_OK;
  if (!expert_counts || !expert_offsets || !w_q || !w_scale) return MOE_ERR_ARG;
  if (cap_expert > 0 && (!rows || !out)) return MOE_ERR_ARG;
  if (!aligned(rows, 16) || !aligned(out, 16) || !aligned(w_q, 16) || !aligned(w_scale, 16) ||
      !aligned(factor, 4) || !aligned(expert_counts, 4) || !aligned(expert_offsets, 4))
    return MOE_ERR_ARG;
  const bool swiglu = act == MOE_ACT_SWIGLU;
  const int wide = swiglu ? N / 2 : N;
  const int cols = swiglu ? kTile : 2 * kTile;
  const int tiles = (wide + cols - 1) / cols;
  const int64_t active = std::min<int64_t>(shape->E, pairs);
  const int64_t per = (pairs + active - 1) / active;
  const int mt = per <= 12 ? 1 : per <= 28 ? 2 : 4;
  // every expert starts a chunk of rows of its own
  const int64_t slots =
      std::min<int64_t>(active + pairs / (kTile * mt), int64_t(INT32_MAX) / tiles);
  const ProductArgs a{rows, expert_counts, expert_offsets, w_q, w_scale, factor, out, err_word,
                      cap_expert, shape->E, shape->H, N, wide, tiles, int(slots)};
  const dim3 grid(uint32_t(slots * tiles));
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (format == MOE_WIRE_NVFP4) {
    if (swiglu)
      launch_product<true, true>(mt, grid, st, a);
    else
      launch_product<true, false>(mt, grid, st, a);
  } else {
    if (swiglu)
      launch_product<false, true>(mt, grid, st, a);
    else
      launch_product<false, false>(mt, grid, st, a);
  }
  return launch_status();
}

}  // extern "C"
