// Expert products with 4-bit weights: HIP kernels for CDNA4 (gfx950, wave64)
// behind include/moe_dispatch.h.
//
// Kernel
//  product_rows   one workgroup per (expert, column tile): reads the tile's
//                 codes once for up to 32 rows of the buffer, expands them to
//                 bf16 in registers and feeds them to MFMA

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
constexpr int kNT = 2;       // tiles of weight rows per wave
constexpr int kDepth = 2;    // granules of H that a wave has on their way
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

// The first row of expert e in the buffer and how many are in use; rows the
// buffer does not hold are left out.
__device__ __forceinline__ int run_of(const ProductArgs& a, int e, int64_t* first) {
  const int64_t begin = a.offsets[e], end = a.offsets[e + 1];
  const int64_t n = min((int64_t)a.counts[e], end - begin);
  *first = begin;
  return ((begin < 0) | (n <= 0)) ? 0 : int(n);
}

// The expert of a slot: with as many slots as experts the slot itself, else
// the slot-th expert that has rows (-1 when there are fewer); one wave looks
// at 64 experts at a time.
__device__ __forceinline__ int expert_of_slot(const ProductArgs& a, int slot) {
  if (a.slots == a.E) return slot < a.E ? slot : -1;
  const int lane = lane_id();
  for (int e0 = 0; e0 < a.E; e0 += kWave) {
    const int e = min(e0 + lane, a.E - 1);
    int64_t first;
    const uint64_t live = __ballot(run_of(a, e, &first) > 0 && e0 + lane < a.E);
    const int n = __popcll(live);
    if (slot < n) {
      const bool at = ((live >> lane) & 1) && __popcll(live & ((uint64_t(1) << lane) - 1)) == slot;
      return e0 + __ffsll((unsigned long long)__ballot(at)) - 1;
    }
    slot -= n;
  }
  return -1;
}

typedef __amdgpu_buffer_rsrc_t buffer;

// A buffer of `bytes` from p; a load past its end gives 0 and touches nothing.
// (The same for the whole wave; the reads of the first lane say so.)
__device__ __forceinline__ buffer make_buffer(const void* p, int bytes) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(uint32_t(v >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(uint64_t(hi) << 32 | lo), 0,
                                           __builtin_amdgcn_readfirstlane(bytes), 0x00027000);
}

// `off` where `in`, else past the end (opaque: the compiler would make two
// loads and a branch of it).
__device__ __forceinline__ int offset_if(bool in, int off) {
  int r = in ? off : 0x7FFFFF00;
  asm("" : "+v"(r));
  return r;
}

// What a wave takes of one granule of H (256 values): two loads of codes per
// tile of 16 weight rows (lane (m, kq): row m, chunks kq and 4 + kq) and its
// part of the granule of the buffer's rows.
template <int NX>
struct Stage {
  vec4 code[2][kNT];
  vec4 x[NX];
};

// Scales: 128 bytes of each of the wave's 32 weight rows at a time, a cache
// line's worth, into the wave's LDS (rows 144 bytes apart: 16 rows' same bytes
// in different banks).
constexpr int kScaleRow = 144;
constexpr int kScaleBytes = kNT * kTile * kScaleRow;

// The rows of the weights, of a granule of the buffer rows in LDS, and their
// products.
template <bool kE4M3, bool kSwiglu, int WK, int MT>
__global__ __launch_bounds__(kBlock, MT == 1 ? 3 : 2) void product_rows(ProductArgs a) {
  constexpr int kRows = WK == 1 ? kTile * MT : 4;        // buffer rows at a time
  constexpr int kSharers = WK == 1 ? kBlock : kWave;     // threads that stage them
  constexpr int NX = kRows * 32 / kSharers;              // 16-byte pieces per thread
  constexpr int kSlot = kRows * 512;                     // bytes of a granule of them
  constexpr int kSlots = 2 * (WK == 1 ? 1 : kWaves);
  static_assert(WK == 1 || (WK == kWaves && MT == 1), "waves split N, or all of them H");
  __shared__ __align__(16) char staged[kSlots * kSlot];
  __shared__ __align__(16) uint8_t scales[kWaves][kScaleBytes];
  __shared__ float part[WK == 1 ? 1 : kWaves][kNT * 4][kWave];
  const int lane = lane_id(), wave = wave_in_block();
  const int m = lane & 15, kq = lane >> 4;
  const int tile = blockIdx.x % a.tiles;
  const int nchunks = a.K / kChunk;
  const int stages = ((nchunks + 7) / 8 + WK - 1) / WK;  // granules per wave
  const int half = a.N / 2;
  const int limit = kSwiglu ? half : a.N;                // columns of y (of each factor)
  const int srow = kE4M3 ? a.K / 16 : a.K / 32;          // scale bytes per weight row
  const int wn = WK == 1 ? wave : 0, wk = WK == 1 ? 0 : wave;
  constexpr int kPerGranule = kE4M3 ? 16 : 8;  // scale bytes of a row
  constexpr int kSuper = 128 / kPerGranule;    // granules whose scales are in LDS
  static_assert(kSuper % kDepth == 0, "scales are renewed between rounds of the ring");
  const int g0 = wk * stages;                  // the wave's first granule,
  const int end = min(nchunks, 8 * (g0 + stages));  // and the end of its chunks
  uint8_t* sc = scales[wave];
  const int64_t scale_bytes = (int64_t)a.E * a.N * srow;
  char* lds = staged + (WK == 1 ? 0 : wave * 2 * kSlot);
  const int n0 = (tile * (kWaves / WK) + wn) * kTile * (kSwiglu ? 1 : kNT);

  for (int slot = blockIdx.x / a.tiles;; slot += a.slots) {
    const int e = __builtin_amdgcn_readfirstlane(expert_of_slot(a, slot));
    if (e < 0) return;
    int64_t first;
    int run = run_of(a, e, &first);
    if (run > 0 && first + run > a.cap) {
      if (threadIdx.x == 0) flag_error(a.err, MOE_ERRBIT_EXPERT_CAP);
      run = first < a.cap ? int(a.cap - first) : 0;
    }
    run = __builtin_amdgcn_readfirstlane(run);

    buffer wq[kNT];  // this wave's tiles of the weights, and their scales
    int64_t ws[kNT];
#pragma unroll
    for (int h = 0; h < kNT; ++h) {
      const int n = n0 + (kSwiglu ? 0 : h * kTile);
      const int64_t r = (int64_t)e * a.N + n + (kSwiglu ? h * half : 0);
      const int rows = max(0, min(kTile, limit - n));
      wq[h] = make_buffer(a.w_q + r * (a.K / 2), rows * (a.K / 2));
      ws[h] = r * srow;
    }

    for (int r0 = 0; r0 < run; r0 += kRows) {
      const int nr = min(kRows, run - r0);
      const int64_t row0 = __builtin_amdgcn_readfirstlane((int)first) + (int64_t)r0;
      const buffer xb = make_buffer(a.rows + row0 * a.K, nr * a.K * 2);
      const int sharer = WK == 1 ? threadIdx.x : lane;

      // The loads of a stage stay together and in the order of the stages: a
      // wait for one stage then leaves the later ones on their way.
      auto load = [&](Stage<NX>& f, int s) {
        __builtin_amdgcn_sched_barrier(0);
        const int g = g0 + s;
#pragma unroll
        for (int i = 0; i < NX; ++i) {
          const int r = (sharer + i * kSharers) >> 5, p = 32 * g + (sharer & 31);
          const int off = offset_if(p < 4 * end, r * (a.K * 2) + p * 16);
          f.x[i] = __builtin_bit_cast(vec4, __builtin_amdgcn_raw_buffer_load_b128(xb, off, 0, 0));
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int c = 8 * g + 4 * u + kq;
          const int off = offset_if(c < end, m * (a.K / 2) + c * 16);
#pragma unroll
          for (int h = 0; h < kNT; ++h)
            f.code[u][h] =
                __builtin_bit_cast(vec4, __builtin_amdgcn_raw_buffer_load_b128(wq[h], off, 0, 0));
        }
        __builtin_amdgcn_sched_barrier(0);
      };

      // The scales of granules [g0 + s, g0 + s + kSuper) to LDS: 8 lanes a row,
      // 16 bytes from any address each, held within the scales of all experts
      // (what a row's end or a row past N leaves there is not used). A piece
      // that the end of the scales cuts off is read again byte by byte.
      auto load_scales = [&](int s) {
        vec4 v[kNT * kTile / 8];
        bool cut = false;
        auto place = [&](int i) {
          const int h = i / 2, r = 8 * (i % 2) + (lane >> 3);
          return (h ? ws[1] : ws[0]) + r * srow + (g0 + s) * kPerGranule + 16 * (lane & 7);
        };
#pragma unroll
        for (int i = 0; i < kNT * kTile / 8; ++i) {
          const int64_t at = place(i);
          cut |= at < scale_bytes && at > scale_bytes - 16;
          v[i] = vec4{0, 0, 0, 0};
          if (scale_bytes >= 16)  // uniform
            __builtin_memcpy(&v[i], a.w_scale + min(at, scale_bytes - 16), 16);
        }
        uint8_t* to = sc + (lane >> 3) * kScaleRow + 16 * (lane & 7);
#pragma unroll
        for (int i = 0; i < kNT * kTile / 8; ++i)
          *reinterpret_cast<vec4*>(to + i * 8 * kScaleRow) = v[i];
        if (__ballot(cut)) {
#pragma unroll 1
          for (int i = 0; i < kNT * kTile / 8; ++i)
#pragma unroll 1
            for (int q = 0; q < 16; ++q) {
              const int64_t at = place(i) + q;
              if (at < scale_bytes) to[i * 8 * kScaleRow + q] = a.w_scale[at];
            }
        }
        __builtin_amdgcn_wave_barrier();
      };

      f32x4 acc[kNT][MT];
#pragma unroll
      for (int h = 0; h < kNT; ++h)
#pragma unroll
        for (int q = 0; q < MT; ++q) acc[h][q] = f32x4{0, 0, 0, 0};

      // kDepth granules are on their way at any time. One past the last reads
      // nothing and adds 0.
      Stage<NX> f[kDepth];
#pragma unroll
      for (int d = 0; d < kDepth; ++d) load(f[d], d);
      for (int s0 = 0; s0 < stages; s0 += kDepth) {
        if (s0 % kSuper == 0) load_scales(s0);
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
          const int s = s0 + d;
          // The granule's rows to LDS, two slots in turn: the one written here
          // was last read before the barrier of the granule before. Piece p of
          // row r lies at place p ^ r, so that the rows' same pieces are in
          // different banks.
          char* at = lds + (s & 1) * kSlot;
#pragma unroll
          for (int i = 0; i < NX; ++i) {
            const int r = (sharer + i * kSharers) >> 5, p = sharer & 31;
            *reinterpret_cast<vec4*>(at + r * 512 + ((p ^ (r & 15)) * 16)) = f[d].x[i];
          }
          if (WK == 1)
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
          else
            __builtin_amdgcn_wave_barrier();
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            // this lane's chunk: its scale, 0 past H (a code there is 0, but
            // 0 times a NaN scale would not be)
            const bool in = 8 * (g0 + s) + 4 * u + kq < end;
            uint32_t b[kNT];
#pragma unroll
            for (int h = 0; h < kNT; ++h) {
              const uint8_t* p = sc + (h * kTile + m) * kScaleRow + (s % kSuper) * kPerGranule;
              const uint32_t v = kE4M3 ? *reinterpret_cast<const uint16_t*>(p + 8 * u + 2 * kq)
                                       : p[4 * u + kq];
              b[h] = in ? v : 0;
            }
            bf16x8 x[MT][4];
#pragma unroll
            for (int q = 0; q < MT; ++q) {
              if (q > 0 && nr <= q * kTile) break;  // uniform: no rows there
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int r = WK == 1 ? q * kTile + m : m & 3, p = 16 * u + 4 * kq + j;
                x[q][j] = *reinterpret_cast<const bf16x8*>(at + r * 512 + (p ^ (r & 15)) * 16);
              }
            }
#pragma unroll
            for (int h = 0; h < kNT; ++h)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t code = f[d].code[u][h][j];
                bf16x8 w;
                if (kE4M3)
                  w = expand_e4m3(code, j < 2 ? __builtin_amdgcn_cvt_f32_fp8(b[h], 0)
                                              : __builtin_amdgcn_cvt_f32_fp8(b[h], 1));
                else
                  w = expand_e8m0(code, __uint_as_float(b[h] << 23));
#pragma unroll
                for (int q = 0; q < MT; ++q) {
                  if (q > 0 && nr <= q * kTile) break;
                  acc[h][q] =
                      __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x[q][j], acc[h][q], 0, 0, 0);
                }
              }
          }
          load(f[d], s + kDepth);
        }
      }

      const float factor = a.factor ? a.factor[e] : 1.0f;
      __bf16* out = reinterpret_cast<__bf16*>(a.out) + row0 * a.wide;
      if (WK == 1) {
#pragma unroll
        for (int q = 0; q < MT; ++q) {
          const int r = q * kTile + m;
          if (r >= nr) continue;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int n = n0 + 4 * kq + i;
            const float y0 = acc[0][q][i] * factor, y1 = acc[1][q][i] * factor;
            if (kSwiglu) {
              if (n < half) out[(int64_t)r * a.wide + n] = __bf16(y0 / (1.0f + expf(-y0)) * y1);
            } else {
              if (n < a.N) out[(int64_t)r * a.wide + n] = __bf16(y0);
              if (n + kTile < a.N) out[(int64_t)r * a.wide + n + kTile] = __bf16(y1);
            }
          }
        }
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      } else {
        // join the waves' parts: thread (wave i, lane) adds up element i of
        // every fragment of that lane, in wave order
#pragma unroll
        for (int h = 0; h < kNT; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) part[wave][h * 4 + i][lane] = acc[h][0][i];
        __syncthreads();
        float y[kNT];
#pragma unroll
        for (int h = 0; h < kNT; ++h) {
          y[h] = 0.0f;
#pragma unroll
          for (int w = 0; w < (WK == 1 ? 1 : kWaves); ++w) y[h] += part[w][h * 4 + wave][lane];
          y[h] *= factor;
        }
        const int n = n0 + 4 * kq + wave;
        if (m < nr) {
          if (kSwiglu) {
            if (n < half) out[(int64_t)m * a.wide + n] = __bf16(y[0] / (1.0f + expf(-y[0])) * y[1]);
          } else {
            if (n < a.N) out[(int64_t)m * a.wide + n] = __bf16(y[0]);
            if (n + kTile < a.N) out[(int64_t)m * a.wide + n + kTile] = __bf16(y[1]);
          }
        }
        __syncthreads();
      }
    }
  }
}

template <bool kE4M3, bool kSwiglu>
void launch_product(int wk, int mt, dim3 grid, hipStream_t st, const ProductArgs& a) {
  if (wk == kWaves)
    product_rows<kE4M3, kSwiglu, kWaves, 1><<<grid, kBlock, 0, st>>>(a);
  else if (mt == 1)
    product_rows<kE4M3, kSwiglu, 1, 1><<<grid, kBlock, 0, st>>>(a);
  else
    product_rows<kE4M3, kSwiglu, 1, 2><<<grid, kBlock, 0, st>>>(a);
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
  const int64_t active = std::min<int64_t>(shape->E, pairs);
  const int64_t per = (pairs + active - 1) / active;
  const int wk = per <= 2 ? kWaves : 1;
  const int mt = per <= 6 ? 1 : 2;
  const int cols = kTile * (swiglu ? 1 : kNT) * (kWaves / wk);
  const int tiles = (wide + cols - 1) / cols;
  const int64_t slots = std::min<int64_t>(active, int64_t(INT32_MAX) / tiles);
  const ProductArgs a{rows, expert_counts, expert_offsets, w_q, w_scale, factor, out, err_word,
                      cap_expert, shape->E, shape->H, N, wide, tiles, int(slots)};
  const dim3 grid(uint32_t(slots * tiles));
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (format == MOE_WIRE_NVFP4) {
    if (swiglu)
      launch_product<true, true>(wk, mt, grid, st, a);
    else
      launch_product<true, false>(wk, mt, grid, st, a);
  } else {
    if (swiglu)
      launch_product<false, true>(wk, mt, grid, st, a);
    else
      launch_product<false, false>(wk, mt, grid, st, a);
  }
  return launch_status();
}

}  // extern "C"
