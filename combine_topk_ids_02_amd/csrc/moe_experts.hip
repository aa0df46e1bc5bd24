// Expert products with 4-bit weights: HIP kernels for CDNA4 (gfx950, wave64)
// behind include/moe_dispatch.h.
//
// product_rows: out = W_e x for the rows x of the expert-grouped buffer. The
// time of a decode batch is the weights' bytes, so everything goes by reading
// each of them once, in whole cache lines, with the next ones on their way:
//  - a workgroup takes a chunk of one expert's rows (4, 16, 32 or 64) and 32
//    weight rows per wave; along H it goes in granules of 256 values, of which
//    a wave has two on their way;
//  - codes: a lane loads 16 bytes, 32 values of one weight row, so that a
//    wave's two loads cover 128 bytes of each of 16 rows. Which values of H
//    meet in one MFMA does not matter as long as both operands agree, so a
//    lane's own 32 values are its part of four 16x16x32 MFMAs;
//  - a word of 8 codes becomes 8 bf16 (exact: a code has 2 significant bits,
//    an E4M3 scale 4) as MFMA's first operand: the weights are its rows, the
//    buffer's rows its columns, of which a decode batch fills few;
//  - scales come to LDS 128 bytes of a row at a time: read where they are
//    used, a few bytes per row and granule, they cost 45 of 164 us at the
//    decode size (their lines are gone from the cache before the next use);
//  - the buffer's rows go through LDS, shared by the workgroup's waves. Read
//    straight into registers they took 64 cache accesses an instruction (one
//    per lane) and bounded the kernel: 190 us at that size.
// Measured (kernel time; E = 48): one token's 6 experts, H = 5120, N = 4096,
// SwiGLU, MXFP4 (67 MB) 15 us; 64 tokens in NVFP4 (566 MB) 127 us, 4.5 TB/s; H =
// 2048, N = 5120 in MXFP4 (267 MB) 63 us, 4.2 TB/s; 256 tokens top-8 of E = 32, H =
// 7168, N = 4096 in MXFP4 (499 MB, 64 rows an expert) 185 us, 203 as the median of 15
// calls and 242 of 30, where the clock falls. A kernel that only reads the codes in this
// pattern takes 86 us and 47 us at the second and third size (5.9 and 5.3 TB/s).

#include "moe_common.h"

namespace {

using namespace moe;

typedef uint32_t vec4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kTile = 16;    // an MFMA tile: 16 weight rows, 16 buffer rows
constexpr int NT = 2;        // tiles of weight rows per wave
constexpr int kDepth = 2;    // granules of H that a wave has on their way
constexpr int kChunk = 32;   // values of H in 16 bytes of codes
constexpr int kMostGroups = 1 << 22;

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
  int tiles;            // column tiles
  int firsts, beyonds;  // slots of the grid for experts' first chunks, and for others
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

// The first row of expert e in the buffer and how many are in use, without the
// rows that the buffer does not hold (`over`: there are such).
__device__ __forceinline__ int run_of(const ProductArgs& a, int e, int64_t* first, bool* over) {
  const int64_t begin = a.offsets[e], end = a.offsets[e + 1];
  const int64_t n = min((int64_t)a.counts[e], end - begin), held = min(n, a.cap - begin);
  *first = begin;
  *over = (begin >= 0) & (held < n) & (n > 0);
  return ((begin < 0) | (held <= 0)) ? 0 : int(held);
}

// Chunks of an expert; one (without rows) where the buffer holds none of its
// rows, for the workgroup that takes it to say so.
template <int kRows>
__device__ __forceinline__ int chunks_of(int run, bool over) {
  return run / kRows + (run % kRows > 0 || (run == 0 && over) ? 1 : 0);
}

// The chunk of at most kRows rows that an index stands for, found by a wave
// looking at 64 experts at a time: an expert's first chunk (`beyond` false), or
// one of those it has beyond its first. False when there are no more.
template <int kRows>
__device__ __forceinline__ bool chunk_of(const ProductArgs& a, bool beyond, int at, int* expert,
                                         int* chunk) {
  const int lane = lane_id();
  *chunk = 0;
  if (!beyond && a.firsts == a.E) {  // a slot for each expert: no need to look
    *expert = at;
    return at < a.E;
  }
  for (int e0 = 0; e0 < a.E; e0 += kWave) {
    int64_t first;
    bool over;
    const int run = run_of(a, min(e0 + lane, a.E - 1), &first, &over);
    int n = chunks_of<kRows>(run, over);
    n = e0 + lane >= a.E ? 0 : beyond ? max(0, n - 1) : min(1, n);
    int before = n;  // becomes the sum over the lanes up to this one
    for (int s = 1; s < kWave; s <<= 1) {
      const int up = __shfl_up(before, s);
      if (lane >= s) before += up;
    }
    const int total = read_lane(before, kWave - 1);
    before -= n;
    if (at < total) {
      const uint64_t hit = __ballot(at >= before && at < before + n);
      if (!hit) return false;  // counts of no layout, whose sum has overflowed
      const int l = __ffsll((unsigned long long)hit) - 1;
      *expert = e0 + l;
      if (beyond) *chunk = 1 + at - read_lane(before, l);
      return true;
    }
    at -= total;
  }
  return false;
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

// What a wave takes of one granule of H (256 values) from the codes: two loads
// per tile of 16 weight rows (lane (m, kq): row m, chunks kq and 4 + kq).
struct Codes {
  vec4 code[2][NT];
};

// Scales: 128 bytes of each of the wave's weight rows at a time, a cache
// line's worth, into the wave's LDS (rows 144 bytes apart: 16 rows' same bytes
// in different banks).
constexpr int kScaleRow = 144;

// Where 16-byte piece p (0..31) of row r of a granule lies in LDS. A 16-byte
// read is served for 16 lanes at a time, taken from two neighbouring groups of
// 16: (m, kq) with kq = 0 for half of the m and kq = 1 for the other half. With
// kq in the low bits of the place and the row folded in, these 16 lie in
// different banks.
__device__ __forceinline__ int piece_at(int r, int p) {
  const int place = (p & 16) | (p & 3) << 2 | (p >> 2 & 3);
  return r * 512 + (place ^ (r & 15)) * 16;
}

// W waves per workgroup. WK = 1: they share kRows rows of the buffer and take
// NT tiles of weight rows each. WK = W: they take a part of H each, of the same
// NT tiles.
template <bool kE4M3, bool kSwiglu, int W, int WK, int MT>
__global__ __launch_bounds__(W * kWave, MT == 1 ? 3 : 2) void product_rows(ProductArgs a) {
  static_assert(WK == 1 || (WK == W && MT == 1 && W == 4), "waves split N, or all of them H");
  constexpr int kThreads = W * kWave;
  constexpr int kRows = WK == 1 ? kTile * MT : 4;        // buffer rows at a time
  constexpr int kSharers = WK == 1 ? kThreads : kWave;   // threads that stage them
  constexpr int NX = kRows * 32 / kSharers;              // 16-byte pieces per thread
  constexpr int kSlot = kRows * 512;                     // bytes of a granule of them
  constexpr int kCols = kTile * (kSwiglu ? NT / 2 : NT); // columns of out per wave
  constexpr int kPerGranule = kE4M3 ? 16 : 8;            // scale bytes of a weight row
  constexpr int kSuper = 128 / kPerGranule;              // granules whose scales are in LDS
  constexpr int NS = NT * kTile / 8;                     // 16-byte loads of them per lane
  static_assert(kSuper % kDepth == 0, "scales are renewed between rounds of the ring");
  static_assert(kDepth == 2, "a granule of the ring has a slot of the two");
  // Rows come to LDS in the middle of the granule before: with many of them the
  // MFMAs hide the write and the wait for it (E = 48, H = 5120, N = 4096 in
  // MXFP4, 16 rows an expert 148 -> 138 us, 64 rows 252 -> 226 us; H = 2048, N = 5120
  // in NVFP4 103 -> 97 and 176 -> 169 us), with few the rows' loads would have
  // too little time (8 rows 130 -> 143 us and, in MXFP4, 64 -> 80 us).
  constexpr bool kHalfway = MT >= 2;
  __shared__ __align__(16) char staged[2 * (WK == 1 ? 1 : W) * kSlot];
  __shared__ __align__(16) uint8_t scales[W][NT * kTile * kScaleRow];
  __shared__ float part[WK == 1 ? 1 : W][NT * 4][WK == 1 ? 1 : kWave];
  const int lane = lane_id(), wave = wave_in_block();
  const int m = lane & 15, kq = lane >> 4;
  const int nchunks = a.K / kChunk;
  const int stages = ((nchunks + 7) / 8 + WK - 1) / WK;  // granules of a wave
  const int half = a.N / 2;
  const int limit = kSwiglu ? half : a.N;                // columns of y (of each factor)
  const int srow = kE4M3 ? a.K / 16 : a.K / 32;          // scale bytes per weight row
  const int g0 = WK == 1 ? 0 : wave * stages;            // the wave's first granule,
  const int end = min(nchunks, 8 * (g0 + stages));       // and the end of its chunks
  uint8_t* sc = scales[wave];
  const int64_t scale_bytes = (int64_t)a.E * a.N * srow;
  char* lds = staged + (WK == 1 ? 0 : wave * 2 * kSlot);
  const int sharer = WK == 1 ? threadIdx.x : lane;

  // The first weight row of tile h of this wave, and how many rows it has
  // (none past the last column).
  const int n0 = (blockIdx.x % a.tiles * (W / WK) + (WK == 1 ? wave : 0)) * kCols;
  auto row_of = [&](int h) {
    return kSwiglu ? n0 + h / 2 * kTile + h % 2 * half : n0 + h * kTile;
  };

  // The last `beyonds` slots take what experts have beyond a first chunk.
  const int slot = blockIdx.x / a.tiles;
  const bool beyond = slot >= a.firsts;
  for (int index = beyond ? slot - a.firsts : slot;; index += beyond ? a.beyonds : a.firsts) {
    int e, chunk;
    if (!chunk_of<kRows>(a, beyond, index, &e, &chunk)) return;
    e = __builtin_amdgcn_readfirstlane(e);
    chunk = __builtin_amdgcn_readfirstlane(chunk);
    int64_t first;
    bool over;
    const int run = __builtin_amdgcn_readfirstlane(run_of(a, e, &first, &over));
    if (over && threadIdx.x == 0) flag_error(a.err, MOE_ERRBIT_EXPERT_CAP);
    first = (int64_t)__builtin_amdgcn_readfirstlane((int)first);  // offsets are int32

    buffer wq[NT];  // this wave's weight rows
#pragma unroll
    for (int h = 0; h < NT; ++h) {
      const int n = n0 + (kSwiglu ? h / 2 : h) * kTile;
      wq[h] = make_buffer(a.w_q + ((int64_t)e * a.N + row_of(h)) * (a.K / 2),
                          max(0, min(kTile, limit - n)) * (a.K / 2));
    }

    // one chunk; all of them where the grid has no slots for the others
    for (int r0 = chunk * kRows; r0 < run; r0 += a.beyonds > 0 ? run : kRows) {
      const int nr = min(kRows, run - r0);
      const int64_t row0 = first + r0;
      const buffer xb = make_buffer(a.rows + row0 * a.K, nr * a.K * 2);

      // Loads stay together and in the order of the granules: a wait for one
      // then leaves the later ones on their way.
      auto load_rows = [&](vec4 (&xr)[NX], int s) {
        __builtin_amdgcn_sched_barrier(0);
        const int g = g0 + s;
#pragma unroll
        for (int i = 0; i < NX; ++i) {
          const int r = (sharer + i * kSharers) >> 5, p = 32 * g + (sharer & 31);
          const int off = offset_if(p < 4 * end, r * (a.K * 2) + p * 16);
          xr[i] = __builtin_bit_cast(vec4, __builtin_amdgcn_raw_buffer_load_b128(xb, off, 0, 0));
        }
        __builtin_amdgcn_sched_barrier(0);
      };
      auto store_rows = [&](const vec4 (&xr)[NX], char* at) {
#pragma unroll
        for (int i = 0; i < NX; ++i) {
          const int r = (sharer + i * kSharers) >> 5, p = sharer & 31;
          *reinterpret_cast<vec4*>(at + piece_at(r, p)) = xr[i];
        }
      };
      auto load_codes = [&](Codes& f, int s) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int c = 8 * (g0 + s) + 4 * u + kq;
          const int off = offset_if(c < end, m * (a.K / 2) + c * 16);
#pragma unroll
          for (int h = 0; h < NT; ++h)
            f.code[u][h] =
                __builtin_bit_cast(vec4, __builtin_amdgcn_raw_buffer_load_b128(wq[h], off, 0, 0));
        }
        __builtin_amdgcn_sched_barrier(0);
      };
      // The scales of granules [g0 + s, g0 + s + kSuper): 8 lanes a row, 16
      // bytes from any address each, held within the scales of all experts
      // (what a row's end or a row past N leaves there is not used).
      vec4 sv[NS];
      auto scale_place = [&](int s, int i) {
        return ((int64_t)e * a.N + row_of(i / 2) + 8 * (i % 2) + (lane >> 3)) * srow +
               (g0 + s) * kPerGranule + 16 * (lane & 7);
      };
      auto load_scales = [&](int s) {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          sv[i] = vec4{0, 0, 0, 0};
          if (scale_bytes >= 16)  // uniform
            __builtin_memcpy(&sv[i], a.w_scale + min(scale_place(s, i), scale_bytes - 16), 16);
        }
      };
      // Into LDS; a piece that the end of the scales cuts off is read again
      // byte by byte.
      auto store_scales = [&](int s) {
        uint8_t* to = sc + (lane >> 3) * kScaleRow + 16 * (lane & 7);
        bool cut = false;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          *reinterpret_cast<vec4*>(to + i * 8 * kScaleRow) = sv[i];
          const int64_t at = scale_place(s, i);
          cut |= at < scale_bytes && at > scale_bytes - 16;
        }
        if (__ballot(cut)) {
#pragma unroll 1
          for (int i = 0; i < NS; ++i)
#pragma unroll 1
            for (int q = 0; q < 16; ++q) {
              const int64_t at = scale_place(s, i) + q;
              if (at < scale_bytes) to[i * 8 * kScaleRow + q] = a.w_scale[at];
            }
        }
        __builtin_amdgcn_wave_barrier();
      };

      // The scales of this lane's chunk 4 u + kq of a granule, 0 past H (a code
      // there is 0, but 0 times a NaN scale would not be).
      auto read_scales = [&](uint32_t (&v)[NT], int s, int u) {
#pragma unroll
        for (int h = 0; h < NT; ++h) {
          const uint8_t* p = sc + (h * kTile + m) * kScaleRow + (s % kSuper) * kPerGranule;
          const uint32_t byte = kE4M3 ? *reinterpret_cast<const uint16_t*>(p + 8 * u + 2 * kq)
                                      : p[4 * u + kq];
          v[h] = 8 * (g0 + s) + 4 * u + kq < end ? byte : 0;
        }
      };
      auto wait_for_all = [&]() {
        if (WK == 1)
          asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        else
          __builtin_amdgcn_wave_barrier();
      };

      // kDepth granules are on their way at any time. One past the last reads
      // nothing and adds 0. The rows of a granule come to LDS as it begins, or
      // (kHalfway) in the middle of the one before, into the slot that was last
      // read before that one's barrier, and its scales to registers.
      Codes f[kDepth];
      vec4 xr[kHalfway ? 1 : kDepth][NX];  // this thread's parts of granules of the rows
      uint32_t b[2][NT], next[2][NT];
      load_scales(0);
      load_rows(xr[0], 0);
      load_codes(f[0], 0);
      if (kHalfway) {
        store_scales(0);
        read_scales(b[0], 0, 0);
        read_scales(b[1], 0, 1);
        store_rows(xr[0], lds);
      }
      load_rows(xr[kHalfway ? 0 : 1], 1);
      load_codes(f[1], 1);
      f32x4 acc[NT][MT];
#pragma unroll
      for (int h = 0; h < NT; ++h)
#pragma unroll
        for (int q = 0; q < MT; ++q) acc[h][q] = f32x4{0, 0, 0, 0};
      if (kHalfway) wait_for_all();
      for (int s0 = 0; s0 < stages; s0 += kDepth) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
          const int s = s0 + d;
          char* at = lds + d % 2 * kSlot;
          if (!kHalfway) {
            if (d == 0 && s % kSuper == 0) store_scales(s);
            if (d == 0 && (s + kDepth) % kSuper == 0) load_scales(s + kDepth);
            store_rows(xr[d], at);
            wait_for_all();
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (!kHalfway) read_scales(b[u], s, u);
            if (kHalfway && u == 1) {
              store_rows(xr[0], lds + (d + 1) % 2 * kSlot);
              if (d == 1 && (s + 1) % kSuper == 0) store_scales(s + 1);
              if (d == 0 && (s + 2) % kSuper == 0) load_scales(s + 2);
              load_rows(xr[0], s + 2);
              read_scales(next[0], s + 1, 0);
              read_scales(next[1], s + 1, 1);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              bf16x8 x[MT];
#pragma unroll
              for (int q = 0; q < MT; ++q) {
                const int r = WK == 1 ? q * kTile + m : m & 3, p = 16 * u + 4 * kq + j;
                x[q] = *reinterpret_cast<const bf16x8*>(at + piece_at(r, p));
              }
#pragma unroll
              for (int h = 0; h < NT; ++h) {
                const uint32_t code = f[d].code[u][h][j];
                bf16x8 w;
                if (kE4M3)
                  w = expand_e4m3(code, j < 2 ? __builtin_amdgcn_cvt_f32_fp8(b[u][h], 0)
                                              : __builtin_amdgcn_cvt_f32_fp8(b[u][h], 1));
                else
                  w = expand_e8m0(code, __uint_as_float(b[u][h] << 23));
#pragma unroll
                for (int q = 0; q < MT; ++q) {
                  acc[h][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x[q], acc[h][q], 0, 0, 0);
                }
              }
            }
          }
          if (!kHalfway) load_rows(xr[d], s + kDepth);
          load_codes(f[d], s + kDepth);
          if (kHalfway) {
            wait_for_all();
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int h = 0; h < NT; ++h) b[u][h] = next[u][h];
          }
        }
      }

      // y to out: lane (m, kq) holds rows 16 q + m, columns 4 kq .. 4 kq + 3 of
      // each tile
      const float factor = a.factor ? a.factor[e] : 1.0f;
      auto put = [&](int r, int h, int i, float y, float up) {
        const int n = n0 + (kSwiglu ? h / 2 : h) * kTile + 4 * kq + i;
        if (r >= nr || n >= limit) return;
        if (kSwiglu) y = y / (1.0f + expf(-y)) * up;
        reinterpret_cast<__bf16*>(a.out)[(row0 + r) * a.wide + n] = __bf16(y);
      };
      if (WK == 1) {
#pragma unroll
        for (int q = 0; q < MT; ++q)
#pragma unroll
          for (int h = 0; h < NT; h += kSwiglu ? 2 : 1)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              put(q * kTile + m, h, i, acc[h][q][i] * factor, acc[(h + 1) % NT][q][i] * factor);
        // LDS is written anew when every wave is done with it
        if (!kHalfway) wait_for_all();
      } else {
        // join the waves' parts: thread (wave i, lane) adds up element i of
        // every fragment of that lane, in wave order
#pragma unroll
        for (int h = 0; h < NT; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            part[WK == 1 ? 0 : wave][h * 4 + i][WK == 1 ? 0 : lane] = acc[h][0][i];
        __syncthreads();
        float y[NT];
#pragma unroll
        for (int h = 0; h < NT; ++h) {
          y[h] = 0.0f;
#pragma unroll
          for (int w = 0; w < (WK == 1 ? 1 : W); ++w)
            y[h] += part[w][h * 4 + (wave & 3)][WK == 1 ? 0 : lane];
          y[h] *= factor;
        }
#pragma unroll
        for (int h = 0; h < NT; h += kSwiglu ? 2 : 1) put(m, h, wave, y[h], y[(h + 1) % NT]);
        __syncthreads();
      }
    }
  }
}

// Forms of the kernel: waves, waves over H, tiles of buffer rows.
struct Form {
  int waves, over_h, rows;  // rows: of the buffer at a time
};
constexpr Form kForms[] = {{4, 4, 4}, {4, 1, 16}, {8, 1, 32}, {8, 1, 64}};

template <bool kE4M3, bool kSwiglu>
void launch_product(int form, dim3 grid, hipStream_t st, const ProductArgs& a) {
  const int threads = kForms[form].waves * kWave;
  switch (form) {
    case 0: product_rows<kE4M3, kSwiglu, 4, 4, 1><<<grid, threads, 0, st>>>(a); break;
    case 1: product_rows<kE4M3, kSwiglu, 4, 1, 1><<<grid, threads, 0, st>>>(a); break;
    case 2: product_rows<kE4M3, kSwiglu, 8, 1, 2><<<grid, threads, 0, st>>>(a); break;
    default: product_rows<kE4M3, kSwiglu, 8, 1, 4><<<grid, threads, 0, st>>>(a);
  }
}

int column_tiles(int form, bool swiglu, int wide) {
  const int cols = kTile * (swiglu ? NT / 2 : NT) * kForms[form].waves / kForms[form].over_h;
  return (wide + cols - 1) / cols;
}

// By the mean number of rows of an expert that has any (uniform routing at
// worst): as many rows at a time as that takes, since every chunk of rows
// reads the codes again. Measured at E = 48, H = 5120, N = 4096 with SwiGLU in
// MXFP4, mean rows 2 / 8 / 12 / 16 / 20 / 24 / 32: 16 rows 75 / 113 / 130 / 158 / 175 /
// 193 / 236 us, 32 rows 90 / 107 / 128 / 138 / 142 / 149 / 177 us, 64 rows 100 / 121 / 123 /
// 140 / 149 / 142 / 160 us; H = 2048, N = 5120 in NVFP4: 55 / 76 / 86 / 102 / 113 / 123 / 152,
// 69 / 82 / 82 / 97 / 101 / 107 / 130 and 77 / 91 / 93 / 97 / 100 / 103 / 122 us.
// Few workgroups with long rows split H over the waves instead of columns:
// 16.3 against 18.6 us for one token's 6 experts there (192 workgroups), 27
// against 30 us for two tokens', but 49.1 against 49.2 us for four (768), and
// at H = 2048 14.8 against 14.3 us for one. 48 experts with N = 4096 and more fill
// the chip in every form; fewer or narrower ones were not measured. A mean of 8
// would be 5% faster with 32 rows in MXFP4 and is 8% slower with them in NVFP4:
// one rule for both. The mean is of T * k rows over all E experts, so it is
// right for a slice of a layout's experts where T is their share: 192 rows of 48 of
// 384 experts take 98 us then (MXFP4, H = 5120), 146 us with the layout's T = 256.
// (The form of 16 rows without an activation keeps 2 registers in scratch in MXFP4
// and 4 in NVFP4, for three waves a SIMD.)
int form_of(const moe_shape_t& sh, bool swiglu, int wide, int64_t pairs, int64_t active) {
  const int64_t mean = (pairs + active - 1) / active;
  if (mean > 20) return 3;
  if (mean > 10) return 2;
  const bool few = active * column_tiles(1, swiglu, wide) < 512;
  return mean <= 2 && few && sh.H >= 4096 ? 0 : 1;
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
  if (shape->H > (1 << 20) || N < 1 || N > (1 << 24) || (act == MOE_ACT_SWIGLU && N % 2 != 0)) return MOE_ERR_ARG;
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
  const int form = form_of(*shape, swiglu, wide, pairs, active);
  const int tiles = column_tiles(form, swiglu, wide);
  // A launch has fewer than 2^32 threads: fewer slots than chunks, and a
  // workgroup takes several, where N is very large.
  const int64_t most = std::max(1, kMostGroups / 2 / tiles);
  const int firsts = int(std::min(active, most));
  const int beyonds = int(std::min((pairs - 1) / kForms[form].rows, most));
  const ProductArgs a{rows, expert_counts, expert_offsets, w_q, w_scale, factor, out, err_word,
                      cap_expert, shape->E, shape->H, N, wide, tiles, firsts, beyonds};
  const dim3 grid(uint32_t(firsts + beyonds) * tiles);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (format == MOE_WIRE_NVFP4) {
    if (swiglu)
      launch_product<true, true>(form, grid, st, a);
    else
      launch_product<true, false>(form, grid, st, a);
  } else {
    if (swiglu)
      launch_product<false, true>(form, grid, st, a);
    else
      launch_product<false, false>(form, grid, st, a);
  }
  return launch_status();
}

}  // extern "C"
