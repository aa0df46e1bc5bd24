// Products in 8-bit integers with a scale for each row and each weight row: HIP
// kernels for CDNA4 (gfx950, wave64) behind include/moe_dispatch.h.
//
// out = rows times weights, both int8 with K values a row, summed exactly in
// int32 (K < 2^17), then scaled and activated in float32. Because the sums are
// exact, H may be cut and joined in any order. Two kernels:
//  - product_few, for few rows: the weights' bytes are the time. A workgroup takes
//    at most 64 rows and 32 weight rows, each wave a part of K: both
//    operands go straight into MFMA registers, whole cache lines of each row,
//    several granules ahead, and the waves' sums meet in LDS;
//  - product_tile, for many: tiles of both come to LDS without passing through
//    registers while the tile before is multiplied.

#include "moe_common.h"

namespace {

using namespace moe;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int kMostRow = 1 << 16;  // values of a row
constexpr int kGranule = 128;      // bytes of each row that are taken at a time
constexpr int kMostGroups = 1 << 22;

struct Int8Args {
  const int8_t* rows;
  const float* row_scale;
  const int32_t* counts;   // NULL: one expert, `dense` rows
  const int32_t* offsets;
  const int8_t* w;
  const float* w_scale;
  uint16_t* out;
  int32_t* err;
  int64_t cap;
  int dense;
  int E, K, N, wide;  // wide: columns of out
  int tiles;          // column tiles
};

// The chunks of at most BM rows that the experts' runs are cut into, numbered
// in the order of the experts; found by a wave together, each lane counting
// for its share of the experts.
template <int BM>
struct Chunks {
  const Int8Args& a;
  int per, before, mine, total;

  __device__ __forceinline__ int count(int e, bool flag) const {
    int64_t first;
    bool over;
    const int run = run_of(a.counts, a.offsets, a.cap, e, &first, &over);
    if (flag && over) flag_error(a.err, MOE_ERRBIT_EXPERT_CAP);
    return run / BM + (run % BM > 0 ? 1 : 0);
  }

  // `flag`: this wave says which experts' rows the buffer does not hold.
  __device__ __forceinline__ Chunks(const Int8Args& args, bool flag) : a(args) {
    if (!a.counts) {
      total = (a.dense + BM - 1) / BM;
      return;
    }
    const int lane = lane_id();
    per = (a.E + kWave - 1) / kWave;
    mine = 0;
    for (int j = 0; j < per; ++j)
      if (lane * per + j < a.E) mine += count(lane * per + j, flag);
    int upto = mine;
    for (int s = 1; s < kWave; s <<= 1) {
      const int up = __shfl_up(upto, s);
      if (lane >= s) upto += up;
    }
    before = upto - mine;
    total = read_lane(upto, kWave - 1);
  }

  // Chunk `at` of them: its expert, first row and number of rows. False where
  // there is none (counts of no layout, whose sum has overflowed).
  __device__ __forceinline__ bool get(int at, int* expert, int64_t* row0, int* rows) const {
    if (!a.counts) {
      *expert = 0;
      *row0 = int64_t(at) * BM;
      *rows = min(BM, a.dense - at * BM);
      return true;
    }
    const uint64_t hit = __ballot(at >= before && at < before + mine);
    if (!hit) return false;
    const int l = __ffsll((unsigned long long)hit) - 1;
    at -= read_lane(before, l);
    for (int j = 0; j < per; ++j) {
      const int e = l * per + j;
      if (e >= a.E) return false;
      int64_t first;
      bool over;
      const int run =
          __builtin_amdgcn_readfirstlane(run_of(a.counts, a.offsets, a.cap, e, &first, &over));
      const int n = run / BM + (run % BM > 0 ? 1 : 0);
      if (at < n) {
        *expert = e;
        *row0 = __builtin_amdgcn_readfirstlane(int(first)) + int64_t(at) * BM;  // int32 offsets
        *rows = min(BM, run - at * BM);
        return true;
      }
      at -= n;
    }
    return false;
  }
};

// Tile `i` of `total` chunks times `tiles` columns. Workgroups go round the 8
// XCDs one by one, so each XCD is given a contiguous eighth of the order, and
// the order goes through the columns of 8 chunks at a time: what an XCD works on
// at one time shares rows and weights in its L2.
__device__ __forceinline__ void place_of(int64_t i, int total, int tiles, int* chunk, int* col) {
  const int64_t all = int64_t(total) * tiles, each = all / 8, more = all % 8;
  const int64_t x = i % 8, at = x * each + min(x, more) + i / 8;
  const int64_t per = int64_t(8) * tiles;
  const int64_t g = at / per, rest = at - g * per;
  const int held = min(8, total - int(g) * 8);
  *chunk = int(g) * 8 + int(rest % held);
  *col = int(rest / held);
}

__device__ __forceinline__ float swiglu(float gate, float up) {
  return gate / (1.0f + expf(-gate)) * up;
}

// ---------------------------------------------------------------------------

// W waves, each a part of K, of 16 * MT rows and 16 * NT weight rows.
template <bool kSwiglu, int MT, int NT, int W, int D>
__global__ __launch_bounds__(W * kWave) void product_few(Int8Args a) {
  static_assert(!kSwiglu || NT == 2, "a tile of gates and one of the other factors");
  constexpr int BM = 16 * MT;
  constexpr int kCols = 16 * (kSwiglu ? NT / 2 : NT);
  __shared__ int part[W][NT * MT * 4][kWave];
  const int lane = lane_id(), wave = wave_in_block();
  const int m = lane & 15, kq = lane >> 4;
  const int half = a.N / 2, limit = kSwiglu ? half : a.N;
  const int granules = (a.K + kGranule - 1) / kGranule;
  const int each = (granules + W - 1) / W;
  const int g0 = wave * each, steps = max(0, min(each, granules - g0));
  const Chunks<BM> chunks(a, blockIdx.x == 0 && wave == 0);
  const int64_t all = int64_t(chunks.total) * a.tiles;
  for (int64_t i = blockIdx.x; i < all; i += gridDim.x) {
    int chunk, col, e, nr;
    int64_t row0;
    place_of(i, chunks.total, a.tiles, &chunk, &col);
    if (!chunks.get(chunk, &e, &row0, &nr)) return;
    const int n0 = col * kCols;
    buffer wb[NT];
#pragma unroll
    for (int h = 0; h < NT; ++h) {
      const int n = kSwiglu ? n0 : n0 + 16 * h;
      wb[h] = make_buffer(a.w + (int64_t(e) * a.N + n + (kSwiglu ? h * half : 0)) * a.K,
                          max(0, min(16, limit - n)) * a.K);
    }
    const buffer xb = make_buffer(a.rows + row0 * a.K, nr * a.K);
    i32x4 w[D][2][NT], x[D][2][MT];
    auto load = [&](int d, int s) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int k = (g0 + s) * kGranule + (4 * u + kq) * 16;
        const int off = offset_if(s < steps && k < a.K, m * a.K + k);
#pragma unroll
        for (int h = 0; h < NT; ++h)
          w[d][u][h] =
              __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(wb[h], off, 0, 0));
#pragma unroll
        for (int q = 0; q < MT; ++q)
          x[d][u][q] = __builtin_bit_cast(
              i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                         xb, off == 0x7FFFFF00 ? off : off + q * 16 * a.K, 0, 0));
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    i32x4 acc[NT][MT];
#pragma unroll
    for (int h = 0; h < NT; ++h)
#pragma unroll
      for (int q = 0; q < MT; ++q) acc[h][q] = i32x4{0, 0, 0, 0};
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, d);
    for (int s0 = 0; s0 < steps; s0 += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int h = 0; h < NT; ++h)
#pragma unroll
            for (int q = 0; q < MT; ++q)
              acc[h][q] =
                  __builtin_amdgcn_mfma_i32_16x16x64_i8(w[d][u][h], x[d][u][q], acc[h][q], 0, 0, 0);
        load(d, s0 + d + D);
      }
    }
#pragma unroll
    for (int h = 0; h < NT; ++h)
#pragma unroll
      for (int q = 0; q < MT; ++q)
#pragma unroll
        for (int r = 0; r < 4; ++r) part[wave][(h * MT + q) * 4 + r][lane] = acc[h][q][r];
    __syncthreads();
    // a wave adds up the elements `at` of every fragment: lane (m, kq) holds row
    // 16 q + m and column 4 kq + r
    for (int at = wave; at < MT * 4; at += W) {
      const int q = at / 4, r = at % 4;
      const int row = 16 * q + m;
      const float xs = row < nr ? a.row_scale[row0 + row] : 0.0f;
      float y[NT];
#pragma unroll
      for (int h = 0; h < NT; ++h) {
        int sum = 0;
#pragma unroll
        for (int v = 0; v < W; ++v) sum += part[v][(h * MT + q) * 4 + r][lane];
        const int n = (kSwiglu ? n0 : n0 + 16 * h) + 4 * kq + r;
        const float ws =
            n < limit ? a.w_scale[int64_t(e) * a.N + n + (kSwiglu ? h * half : 0)] : 0.0f;
        y[h] = float(sum) * xs * ws;
      }
      if (row < nr) {
        __bf16* to = reinterpret_cast<__bf16*>(a.out) + (row0 + row) * a.wide;
        if (kSwiglu) {
          if (n0 + 4 * kq + r < limit) to[n0 + 4 * kq + r] = __bf16(swiglu(y[0], y[NT - 1]));
        } else {
#pragma unroll
          for (int h = 0; h < NT; ++h)
            if (n0 + 16 * h + 4 * kq + r < limit) to[n0 + 16 * h + 4 * kq + r] = __bf16(y[h]);
        }
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------

// BM rows and BN weight rows, by WM x WN waves, in 32x32x32 MFMAs; with SwiGLU
// tiles of 32 gates alternate with the 32 other factors that they meet.
template <bool kSwiglu, int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__(WM * WN * kWave) void product_tile(Int8Args a) {
  constexpr int W = WM * WN;
  constexpr int MT = BM / WM / 32, NT = BN / WN / 32;
  static_assert(BM == WM * MT * 32 && BN == WN * NT * 32 && (!kSwiglu || NT % 2 == 0), "tiles");
  static_assert(W % 2 == 0 && BM % (8 * W) == 0 && BN % (8 * W) == 0, "8 rows a load of a wave");
  constexpr int LW = BN / (8 * W), LX = BM / (8 * W), L = LW + LX;  // loads of a wave
  constexpr int kStage = (BM + BN) * kGranule;
  constexpr int kCols = kSwiglu ? BN / 2 : BN;
  __shared__ __align__(16) char lds[S * kStage];
  const int lane = lane_id(), wave = wave_in_block();
  const int wm = wave / WN, wn = wave % WN;
  const int half = a.N / 2, limit = kSwiglu ? half : a.N;
  const int steps = (a.K + kGranule - 1) / kGranule;
  const Chunks<BM> chunks(a, blockIdx.x == 0 && wave == 0);
  const int64_t all = int64_t(chunks.total) * a.tiles;
  for (int64_t i = blockIdx.x; i < all; i += gridDim.x) {
    int chunk, col, e, nr;
    int64_t row0;
    place_of(i, chunks.total, a.tiles, &chunk, &col);
    if (!chunks.get(chunk, &e, &row0, &nr)) return;
    const int n0 = col * kCols, held = min(kCols, limit - n0);
    const int8_t* w0 = a.w + (int64_t(e) * a.N + n0) * a.K;
    const buffer wg = make_buffer(w0, held * a.K);
    const buffer wu = make_buffer(w0 + int64_t(kSwiglu ? half : 0) * a.K, held * a.K);
    const buffer xb = make_buffer(a.rows + row0 * a.K, nr * a.K);

    // Load j of this wave fills rows 8 (j W + wave) .. + 7 of a stage, a lane 16
    // bytes: lane l the slot l % 8 of row l / 8. Slot s of row r holds piece s ^
    // (r / 2) % 8, so that 16 rows' same piece lies in different banks.
    const int piece = (lane & 7) ^ ((wave & 1) * 4 + (lane >> 4));
    int from[L];
#pragma unroll
    for (int j = 0; j < L; ++j) {
      const int r = 8 * ((j < LW ? j : j - LW) * W + wave) + (lane >> 3);
      const int c = j >= LW ? r : kSwiglu ? r / 64 * 32 + r % 32 : r;
      from[j] = offset_if(c < (j < LW ? held : nr), c * a.K + piece * 16);
    }
    auto load = [&](int s, int slot) {
#pragma unroll
      for (int j = 0; j < L; ++j) {
        const int tile = 8 * (j * W + wave);  // the first row it fills
        const buffer& b = j >= LW ? xb : kSwiglu && tile / 32 % 2 == 1 ? wu : wg;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            b, (__attribute__((address_space(3))) void*)(lds + slot * kStage + tile * kGranule), 16,
            int(uint32_t(from[j]) + uint32_t(s * kGranule)), 0, 0, 0);
      }
    };

    i32x16 acc[NT][MT];
#pragma unroll
    for (int h = 0; h < NT; ++h)
#pragma unroll
      for (int q = 0; q < MT; ++q)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[h][q][r] = 0;

    const int swz = (lane >> 1) & 7, hi = lane >> 5;
    const int wrow = (wn * NT * 32 + (lane & 31)) * kGranule;
    const int xrow = (BN + wm * MT * 32 + (lane & 31)) * kGranule;
    // kEnd: the last step where K ends inside it; what lies behind is masked in
    // one of the operands.
    auto multiply = [&](int s, int slot, bool end) {
      const char* at = lds + slot * kStage;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const int place = ((2 * kk + hi) ^ swz) * 16;
        i32x4 w[NT], x[MT];
#pragma unroll
        for (int h = 0; h < NT; ++h)
          w[h] = *reinterpret_cast<const i32x4*>(at + wrow + h * 32 * kGranule + place);
#pragma unroll
        for (int q = 0; q < MT; ++q)
          x[q] = *reinterpret_cast<const i32x4*>(at + xrow + q * 32 * kGranule + place);
        if (end) {
          const bool in = s * kGranule + (2 * kk + hi) * 16 < a.K;
#pragma unroll
          for (int q = 0; q < MT; ++q)
#pragma unroll
            for (int r = 0; r < 4; ++r) x[q][r] = in ? x[q][r] : 0;
        }
#pragma unroll
        for (int h = 0; h < NT; ++h)
#pragma unroll
          for (int q = 0; q < MT; ++q)
            acc[h][q] = __builtin_amdgcn_mfma_i32_32x32x32_i8(w[h], x[q], acc[h][q], 0, 0, 0);
      }
    };

#pragma unroll
    for (int s = 0; s < S - 1; ++s)
      if (s < steps) load(s, s);
    int slot = 0;
    for (int s = 0; s < steps; ++s) {
      // the loads of this step have come when at most those of the later ones
      // are on their way
      if (S > 2 && s + S - 2 < steps)
        asm volatile("s_waitcnt vmcnt(%0)" ::"i"((S - 2) * L) : "memory");
      else
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      const int next = slot == 0 ? S - 1 : slot - 1;
      if (s + S - 1 < steps) load(s + S - 1, next);
      multiply(s, slot, s == steps - 1 && a.K % kGranule != 0);
      slot = slot == S - 1 ? 0 : slot + 1;
    }

    // lane: row lane % 32, columns 8 (r / 4) + 4 (lane / 32) + r % 4 of each tile
#pragma unroll
    for (int q = 0; q < MT; ++q) {
      const int row = (wm * MT + q) * 32 + (lane & 31);
      if (row < nr) {
        const float xs = a.row_scale[row0 + row];
        __bf16* to = reinterpret_cast<__bf16*>(a.out) + (row0 + row) * a.wide;
#pragma unroll
        for (int h = 0; h < NT; h += kSwiglu ? 2 : 1) {
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int n = n0 + (wn * NT + h) / (kSwiglu ? 2 : 1) * 32 + 8 * (r / 4) + 4 * hi + r % 4;
            if (n < limit) {
              const float* ws = a.w_scale + int64_t(e) * a.N + n;
              float y = float(acc[h][q][r]) * xs * ws[0];
              if (kSwiglu) y = swiglu(y, float(acc[(h + 1) % NT][q][r]) * xs * ws[half]);
              to[n] = __bf16(y);
            }
          }
        }
      }
    }
    __syncthreads();  // LDS is written anew when every wave is done with it
  }
}

// ---------------------------------------------------------------------------

// Forms: rows and columns of weights (with SwiGLU two weight rows a column)
// that a workgroup takes, its waves.
struct Form {
  int rows, weights, waves;
};
constexpr Form kForms[] = {{16, 32, 8}, {32, 32, 8}, {64, 32, 8}, {128, 128, 4}, {256, 256, 8}};

template <bool kSwiglu>
void launch(int form, dim3 grid, hipStream_t st, const Int8Args& a) {
  const int threads = kForms[form].waves * kWave;
  switch (form) {
    case 0: product_few<kSwiglu, 1, 2, 8, 4><<<grid, threads, 0, st>>>(a); break;
    case 1: product_few<kSwiglu, 2, 2, 8, 3><<<grid, threads, 0, st>>>(a); break;
    case 2: product_few<kSwiglu, 4, 2, 8, 2><<<grid, threads, 0, st>>>(a); break;
    case 3: product_tile<kSwiglu, 128, 128, 2, 2, 2><<<grid, threads, 0, st>>>(a); break;
    default: product_tile<kSwiglu, 256, 256, 2, 4, 2><<<grid, threads, 0, st>>>(a);
  }
}

// By the mean number of rows of an expert that has any (uniform routing at worst).
int form_of(int64_t mean, int64_t tiles256) {
  if (mean <= 16) return 0;
  if (mean <= 32) return 1;
  if (mean <= 64) return 2;
  return tiles256 < 200 ? 3 : 4;
}

}  // namespace

extern "C" {

int moe_int8_product(const moe_shape_t* shape, int N, int act, const int8_t* rows,
                     const float* row_scale, const int32_t* expert_counts,
                     const int32_t* expert_offsets, int64_t cap_expert, const int8_t* w_q,
                     const float* w_scale, uint16_t* out, int32_t* err_word, void* stream) {
  if (!shape_ok(shape) || shape->H % 16 != 0 || shape->H > kMostRow) return MOE_ERR_ARG;
  if (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU) return MOE_ERR_ARG;
  if (N < 1 || N > (1 << 24) || (act == MOE_ACT_SWIGLU && N % 2 != 0)) return MOE_ERR_ARG;
  if (cap_expert < 0) return MOE_ERR_ARG;
  const int64_t pairs = int64_t(shape->T) * shape->k;
  if (pairs == 0) return MOE_OK;
  if (!expert_counts != !expert_offsets) return MOE_ERR_ARG;
  if (!expert_counts && (shape->E != 1 || pairs > cap_expert)) return MOE_ERR_ARG;
  if (!w_q || !w_scale) return MOE_ERR_ARG;
  if (cap_expert > 0 && (!rows || !row_scale || !out)) return MOE_ERR_ARG;
  if (!aligned(rows, 16) || !aligned(out, 16) || !aligned(w_q, 16) || !aligned(w_scale, 4) ||
      !aligned(row_scale, 4) || !aligned(expert_counts, 4) || !aligned(expert_offsets, 4))
    return MOE_ERR_ARG;
  const bool swiglu = act == MOE_ACT_SWIGLU;
  const int64_t active = std::min<int64_t>(shape->E, pairs), mean = (pairs + active - 1) / active;
  auto most = [&](const Form& f) {  // chunks, at most, and column tiles
    const int64_t chunks = active + (pairs - active) / f.rows;
    return std::pair<int64_t, int64_t>(chunks, (N + f.weights - 1) / f.weights);
  };
  const auto big = most(kForms[4]);
  const int form = form_of(mean, (pairs + 255) / 256 * big.second);
  const auto [chunks, tiles] = most(kForms[form]);
  const Int8Args a{rows, row_scale, expert_counts, expert_offsets, w_q, w_scale, out, err_word,
                   cap_expert, int(pairs), shape->E, shape->H, N, swiglu ? N / 2 : N, int(tiles)};
  const dim3 grid(uint32_t(std::min<int64_t>(chunks * tiles, kMostGroups)));
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (swiglu)
    launch<true>(form, grid, st, a);
  else
    launch<false>(form, grid, st, a);
  return launch_status();
}

}  // extern "C"
