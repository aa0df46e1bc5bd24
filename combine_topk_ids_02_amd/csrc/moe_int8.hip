// Products in 8-bit integers with a scale for each row and each weight row: HIP
// kernels for CDNA4 (gfx950, wave64) behind include/moe_dispatch.h.
//
// out = rows times weights, both int8 with K values a row, summed exactly in
// int32 (K < 2^17), then scaled and activated in float32. Because the sums are
// exact, K may be cut and joined in any order.
//
// Two kernels, which bring 128 bytes of each of their rows and weight rows at a time to
// LDS by loads that pass through no register, several such steps ahead:
//  - product_few, for few rows, cuts K over the waves of a workgroup, so that few
//    weight rows make many workgroups; their sums meet in LDS at the end. No wave
//    waits for another before that;
//  - product_tile, for many, has the waves share a tile of 64 to 256 rows.
// (Straight into MFMA's registers, 16 rows' 64 bytes an instruction, one token's
// product with K = 5,120, N = 4,096 took 9.4 us, where it takes 6.1 now, and 384 rows of
// 48 experts 317 us, where they take 166: 6.1 TB/s of the weights.)

#include "moe_common.h"

namespace {

using namespace moe;

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef bf16x8 bf16x8_any __attribute__((aligned(2)));  // at any address of a value
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef const __attribute__((address_space(4))) int32_t* scalar_ints;
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
  int run0, first0;  // of this lane's first expert

  __device__ __forceinline__ static int chunks_of(int run) {
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
    mine = run0 = first0 = 0;
    for (int j = 0; j < per && lane * per + j < a.E; ++j) {
      int64_t first;
      bool over;
      const int run = run_of(a.counts, a.offsets, a.cap, lane * per + j, &first, &over);
      if (flag && over) flag_error(a.err, MOE_ERRBIT_EXPERT_CAP);
      mine += chunks_of(run);
      if (j == 0) run0 = run, first0 = int(first);  // offsets are int32
    }
    int upto = mine;
    for (int s = 1; s < kWave; s <<= 1) {
      const int up = __shfl_up(upto, s);
      if (lane >= s) upto += up;
    }
    before = upto - mine;
    total = read_lane(upto, kWave - 1);
  }

  // Tiles, with those of the columns. Weights and rows of out that this card's memory
  // holds make fewer than 2^31; counts of no layout may not: they get none.
  __device__ __forceinline__ uint32_t all() const {
    const int64_t n = int64_t(total) * a.tiles;
    return n > 0 && n < int64_t(1) << 31 ? uint32_t(n) : 0;
  }

  // Tile i of the total * tiles that the chunks make with the column tiles: its
  // expert, column tile, first row and number of rows. Workgroups go round the 8 XCDs
  // one by one, so each XCD is given a contiguous eighth of an order that goes through
  // the columns of up to 8 chunks of one expert at a time: what an XCD works on at one
  // time shares rows and weights in its L2, and weights are wanted only once. (With
  // 8 chunks of whatever experts at a time 8,192 rows of 32 experts, K = 2,048, N = 7,168,
  // read 690 MB for 490 and took 205 us instead of 196; 1,536 rows of 48, 110 and 106.)
  // False where there is no such tile (counts of no layout, whose sum has overflowed).
  __device__ __forceinline__ bool tile(uint32_t i, int* expert, int* col, int64_t* row0,
                                       int* rows) const {
    const uint32_t tiles = a.tiles, all = this->all(), x = i % 8;
    uint32_t at = x * (all / 8) + min(x, all % 8) + i / 8;
    int e = 0, run = a.dense, n = total;
    int64_t first = 0;
    if (a.counts) {
      const int v = int(at / tiles);
      const uint64_t hit = __ballot(v >= before && v < before + mine);
      if (!hit) return false;
      const int l = __ffsll((unsigned long long)hit) - 1;
      at -= uint32_t(read_lane(before, l)) * tiles;
      e = l * per;
      run = read_lane(run0, l);
      first = read_lane(first0, l);
      n = chunks_of(run);
      for (int j = 1; at >= n * tiles; ++j) {
        at -= n * tiles;
        if (j == per || ++e == a.E) return false;
        bool over;  // scalar loads: the kernel does not write what they read
        run = run_of(scalar_ints(uint64_t(a.counts)), scalar_ints(uint64_t(a.offsets)), a.cap, e,
                     &first, &over);
        n = chunks_of(run);
      }
    }
    const uint32_t g = at / (8 * tiles), rest = at - g * 8 * tiles;
    const uint32_t held = min(8u, n - g * 8);
    const int chunk = g * 8 + rest % held;
    *expert = e;
    *col = int(rest / held);
    *row0 = first + int64_t(chunk) * BM;
    *rows = min(BM, run - chunk * BM);
    return true;
  }
};

// 16 bytes a lane from a buffer to LDS, lane l's to at + 16 l (`at` the same for
// the whole wave), without a register in between; counted as a vector load.
__device__ __forceinline__ void load_to_lds(const buffer& b, char* at, int off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      b, (__attribute__((address_space(3))) void*)at, 16, off, 0, 0, 0);
}

__device__ __forceinline__ float swiglu(float gate, float up) {
  return gate / (1.0f + expf(-gate)) * up;
}

// ---------------------------------------------------------------------------

// W waves, each a part of K, of 16 * MT rows and 16 * NT weight rows. A wave has
// S granules in its own part of LDS, S - 1 of them on their way.
template <bool kSwiglu, int MT, int NT, int W, int S>
__global__ __launch_bounds__(W * kWave) void product_few(Int8Args a) {
  static_assert(NT <= 2, "with SwiGLU half a tile, or a tile, of gates and of the other factors");
  static_assert(S >= 2 && S <= 4, "waits are written for these");
  constexpr bool kMixed = kSwiglu && NT == 1;  // 8 gates and the 8 factors that they meet
  constexpr int BM = 16 * MT;
  constexpr int kCols = kSwiglu ? 8 * NT : 16 * NT;
  constexpr int L = 2 * (NT + MT);         // loads of a granule, 8 rows each
  constexpr int kStage = L * 8 * kGranule;
  constexpr int kJoin = W * NT * MT * 4 * kWave * 4;
  constexpr int kRoom = W * S * kStage > kJoin ? W * S * kStage : kJoin;
  // One array for all of LDS: with two the compiler waits for every load that is on
  // its way to LDS before each read of it.
  __shared__ __align__(16) char lds[kRoom + (16 * NT + BM) * 4];
  float* scales = reinterpret_cast<float*>(lds + kRoom);  // of the weight rows, then the rows
  int(*part)[NT * MT * 4][kWave] = reinterpret_cast<int(*)[NT * MT * 4][kWave]>(lds);
  const int lane = lane_id(), wave = wave_in_block();
  const int m = lane & 15, kq = lane >> 4;
  char* mine = lds + wave * S * kStage;
  const int half = a.N / 2, limit = kSwiglu ? half : a.N;
  const int granules = (a.K + kGranule - 1) / kGranule;
  const int each = (granules + W - 1) / W;
  const int g0 = wave * each, steps = max(0, min(each, granules - g0));
  const Chunks<BM> chunks(a, blockIdx.x == 0 && wave == 0);
  const uint32_t all = chunks.all();
  for (uint32_t i = blockIdx.x; i < all; i += gridDim.x) {
    int col, e, nr;
    int64_t row0;
    if (!chunks.tile(i, &e, &col, &row0, &nr)) return;
    const int n0 = col * kCols;
    const int8_t* w0 = a.w + (int64_t(e) * a.N + n0) * a.K;
    buffer wb[NT];
#pragma unroll
    for (int h = 0; h < NT; ++h) {
      if (kMixed)
        wb[h] = make_buffer(w0, (half + min(8, limit - n0)) * a.K);
      else
        wb[h] = make_buffer(w0 + int64_t(kSwiglu ? h * half : 16 * h) * a.K,
                            max(0, min(16, limit - (kSwiglu ? n0 : n0 + 16 * h))) * a.K);
    }
    const buffer xb = make_buffer(a.rows + row0 * a.K, nr * a.K);
    // The scales come first, so that no one waits for them at the end.
    float scale = 0.0f;
    if (threadIdx.x < 16 * NT + BM) {
      const int r = threadIdx.x, c = kMixed ? r % 8 : kSwiglu ? r % 16 : r;
      if (r >= 16 * NT)
        scale = r - 16 * NT < nr ? a.row_scale[row0 + r - 16 * NT] : 0.0f;
      else if (n0 + c < limit)
        scale = a.w_scale[int64_t(e) * a.N + n0 + c + (r == c ? 0 : half)];
    }

    // Load j fills rows 8 j .. 8 j + 7 of a granule: the weights' tiles, then the
    // rows'; a lane 16 bytes, lane l the slot l % 8 of row l / 8. Slot s of row r
    // holds piece s ^ (r / 2) % 8: 16 rows' same piece lies in different banks.
    int from[L];
#pragma unroll
    for (int j = 0; j < L; ++j) {
      const int r = 8 * j + (lane >> 3), piece = (lane & 7) ^ (r / 2 & 7);
      const int row = j >= 2 * NT ? r - 16 * NT : kMixed && j == 1 ? r - 8 + half : r % 16;
      from[j] = row * a.K + g0 * kGranule + piece * 16;
    }
    auto load = [&](int s, int slot) {
#pragma unroll
      for (int j = 0; j < L; ++j) {
        const buffer& b = j < 2 * NT ? wb[j / 2 % NT] : xb;
        load_to_lds(b, mine + slot * kStage + j * 8 * kGranule, from[j] + s * kGranule);
      }
    };
    i32x4 acc[NT][MT];
#pragma unroll
    for (int h = 0; h < NT; ++h)
#pragma unroll
      for (int q = 0; q < MT; ++q) acc[h][q] = i32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < S - 1; ++s)
      if (s < steps) load(s, s);
    if (threadIdx.x < 16 * NT + BM) scales[threadIdx.x] = scale;
    int slot = 0;
    for (int s = 0; s < steps; ++s) {
      // this granule has come when at most the later ones are on their way, and
      // the reads of the slot that is filled next are done
      const int later = min(S - 2, steps - 1 - s);
      if (S > 3 && later == 2)
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"(2 * L) : "memory");
      else if (S > 2 && later == 1)
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"(L) : "memory");
      else
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      if (s + S - 1 < steps) load(s + S - 1, slot == 0 ? S - 1 : slot - 1);
      if ((g0 + s + 1) * kGranule > a.K) {
        // what the weights have behind the end of K becomes 0
#pragma unroll
        for (int j = 0; j < 2 * NT; ++j) {
          const int piece = (lane & 7) ^ ((8 * j + (lane >> 3)) / 2 & 7);
          if ((g0 + s) * kGranule + piece * 16 >= a.K)
            *reinterpret_cast<i32x4*>(mine + slot * kStage + j * 8 * kGranule + lane * 16) =
                i32x4{0, 0, 0, 0};
        }
      }
      const char* at = mine + slot * kStage + m * kGranule;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int place = ((4 * u + kq) ^ (m >> 1)) * 16;
        i32x4 w[NT];
#pragma unroll
        for (int h = 0; h < NT; ++h)
          w[h] = *reinterpret_cast<const i32x4*>(at + h * 16 * kGranule + place);
#pragma unroll
        for (int q = 0; q < MT; ++q) {
          const i32x4 x =
              *reinterpret_cast<const i32x4*>(at + (NT + q) * 16 * kGranule + place);
#pragma unroll
          for (int h = 0; h < NT; ++h)
            acc[h][q] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[h], x, acc[h][q], 0, 0, 0);
        }
      }
      slot = slot == S - 1 ? 0 : slot + 1;
    }
    __syncthreads();  // every wave is done with its granules
#pragma unroll
    for (int h = 0; h < NT; ++h)
#pragma unroll
      for (int q = 0; q < MT; ++q)
#pragma unroll
        for (int r = 0; r < 4; ++r) part[wave][(h * MT + q) * 4 + r][lane] = acc[h][q][r];
    __syncthreads();
    // a wave adds up the elements `at` of every fragment: lane (m, kq) holds row
    // 16 q + m and weight row 4 kq + r of each tile
    for (int at = wave; at < MT * 4; at += W) {
      const int q = at / 4, r = at % 4;
      const int row = 16 * q + m;
      auto sum = [&](int h, int l) {
        int v = 0;
#pragma unroll
        for (int o = 0; o < W; ++o) v += part[o][(h * MT + q) * 4 + r][l];
        return float(v);
      };
      const float xs = scales[16 * NT + row];
      __bf16* to = reinterpret_cast<__bf16*>(a.out) + (row0 + row) * a.wide;
#pragma unroll
      for (int h = 0; h < (kSwiglu ? 1 : NT); ++h) {
        const int n = n0 + 16 * h + 4 * kq + r;
        if (row >= nr || n >= limit || (kMixed && kq >= 2)) continue;
        const float* ws = scales + 16 * h + 4 * kq + r;
        float y = sum(h, lane) * xs * ws[0];
        if (kSwiglu)
          y = swiglu(y, sum(NT - 1, kMixed ? lane + 32 : lane) * xs * ws[kMixed ? 8 : 16]);
        to[n] = __bf16(y);
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------

// BM rows and BN weight rows, by WM x WN waves, in 32x32x32 MFMAs; with SwiGLU
// tiles of 32 gates alternate with the 32 other factors that they meet.
template <bool kSwiglu, int BM, int BN, int WM, int WN, int S, int P>
__global__ __launch_bounds__(WM * WN * kWave) void product_tile(Int8Args a) {
  constexpr int W = WM * WN;
  constexpr int MT = BM / WM / 32, NT = BN / WN / 32;
  static_assert(BM == WM * MT * 32 && BN == WN * NT * 32 && (!kSwiglu || NT % 2 == 0), "tiles");
  static_assert(W % 2 == 0 && BM % (8 * W) == 0 && BN % (8 * W) == 0, "8 rows a load of a wave");
  constexpr int LW = BN / (8 * W), LX = BM / (8 * W), L = LW + LX;  // loads of a wave
  static_assert(L <= 4 * NT * MT, "a load an MFMA");
  constexpr int kStage = (BM + BN) * kGranule;
  constexpr int kCols = kSwiglu ? BN / 2 : BN;
  // a row of results is 16 bytes longer than it needs to be: 32 rows' same columns
  // then lie in different banks
  constexpr int kPitch = kCols * 2 + 16;
  constexpr int kRoom = S * kStage > BM * kPitch ? S * kStage : BM * kPitch;
  // One array for all of LDS: with two the compiler waits for every load that is on
  // its way to LDS before each read of it (512 rows, K = 5,120, N = 4,096: 33 us, not 20).
  __shared__ __align__(16) char lds[kRoom + (BN + BM) * 4];
  float* scales = reinterpret_cast<float*>(lds + kRoom);  // of the weight rows, then the rows
  const int lane = lane_id(), wave = wave_in_block();
  const int wm = wave / WN, wn = wave % WN;
  const int half = a.N / 2, limit = kSwiglu ? half : a.N;
  const int steps = (a.K + kGranule - 1) / kGranule;
  const Chunks<BM> chunks(a, blockIdx.x == 0 && wave == 0);
  const uint32_t all = chunks.all();
  for (uint32_t i = blockIdx.x; i < all; i += gridDim.x) {
    int col, e, nr;
    int64_t row0;
    if (!chunks.tile(i, &e, &col, &row0, &nr)) return;
    const int n0 = col * kCols, held = min(kCols, limit - n0);
    const int8_t* w0 = a.w + (int64_t(e) * a.N + n0) * a.K;
    const buffer wg = make_buffer(w0, held * a.K);
    const buffer wu = make_buffer(w0 + int64_t(kSwiglu ? half : 0) * a.K, held * a.K);
    const buffer xb = make_buffer(a.rows + row0 * a.K, nr * a.K);

    // The scales come first, so that no one waits for them at the end: one of each
    // thread, or two.
    constexpr int kScales = (BN + BM + W * kWave - 1) / (W * kWave);
    float scale[kScales];
#pragma unroll
    for (int k = 0; k < kScales; ++k) {
      const int r = k * W * kWave + threadIdx.x, c = kSwiglu ? r / 64 * 32 + r % 32 : r;
      scale[k] = 0.0f;
      if (r < BN) {
        if (c < held)
          scale[k] = a.w_scale[int64_t(e) * a.N + n0 + c + (kSwiglu && r / 32 % 2 ? half : 0)];
      } else if (r - BN < nr) {
        scale[k] = a.row_scale[row0 + r - BN];
      }
    }

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
    // Load j of step s; past the last step one that reads nothing, so that every
    // step has as many on their way.
    auto load = [&](int j, int s, int slot) {
      const int tile = 8 * (j * W + wave);  // the first row it fills
      const buffer& b = j >= LW ? xb : kSwiglu && tile / 32 % 2 == 1 ? wu : wg;
      const uint32_t at = s < steps ? s * kGranule : 0x70000000u;
      load_to_lds(b, lds + slot * kStage + tile * kGranule, int(uint32_t(from[j]) + at));
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
    // The operands of one MFMA step (32 values of K) of a slot.
    i32x4 w[4][NT], x[4][MT];
    auto read = [&](int slot, int kk) {
      const char* at = lds + slot * kStage + ((2 * kk + hi) ^ swz) * 16;
#pragma unroll
      for (int h = 0; h < NT; ++h)
        w[kk][h] = *reinterpret_cast<const i32x4*>(at + wrow + h * 32 * kGranule);
#pragma unroll
      for (int q = 0; q < MT; ++q)
        x[kk][q] = *reinterpret_cast<const i32x4*>(at + xrow + q * 32 * kGranule);
    };

#pragma unroll
    for (int s = 0; s < S - 1; ++s)
#pragma unroll
      for (int j = 0; j < L; ++j) load(j, s, s);
#pragma unroll
    for (int k = 0; k < kScales; ++k)
      if (k * W * kWave + threadIdx.x < BN + BM) scales[k * W * kWave + threadIdx.x] = scale[k];
    // One step's end of the waiting: its loads have come when only those of the
    // later steps are on their way, and the reads of the slot that is filled next
    // are done.
    auto arrive = [&](int s, int slot) {
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"((S - 2) * L) : "memory");
      if (s == steps - 1 && a.K % kGranule != 0) {
        // what the rows have behind the end of K becomes 0, each piece by the
        // lane that has loaded it
        if (s * kGranule + piece * 16 >= a.K) {
#pragma unroll
          for (int j = LW; j < L; ++j)
            *reinterpret_cast<i32x4*>(lds + slot * kStage + 8 * (j * W + wave) * kGranule +
                                      lane * 16) = i32x4{0, 0, 0, 0};
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      }
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    };
    int slot = 0;
    if (wm * MT * 32 >= nr) {
      // waves whose rows are all behind the chunk's only load. (A loop of their own:
      // a branch around the MFMAs moved the accumulators at every step, 1,320
      // cycles a step of the form of 64 rows and 128 weight rows instead of 1,000.)
      for (int s = 0; s < steps; ++s) {
        arrive(s, slot);
#pragma unroll
        for (int j = 0; j < L; ++j) load(j, s + S - 1, slot == 0 ? S - 1 : slot - 1);
        slot = slot == S - 1 ? 0 : slot + 1;
      }
    } else {
      for (int s = 0; s < steps; ++s) {
        arrive(s, slot);
        const int next = slot == 0 ? S - 1 : slot - 1;
        // The operands of the MFMAs are read P steps ahead of them, and the loads
        // are issued between MFMAs: all at once they hold the wave up.
#pragma unroll
        for (int kk = 0; kk < P; ++kk) read(slot, kk);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (kk + P < 4) read(slot, kk + P);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int h = 0; h < NT; ++h)
#pragma unroll
            for (int q = 0; q < MT; ++q) {
              acc[h][q] =
                  __builtin_amdgcn_mfma_i32_32x32x32_i8(w[kk][h], x[kk][q], acc[h][q], 0, 0, 0);
              // one load behind each MFMA till all are issued
              const int j = (kk * NT + h) * MT + q;
              if (j < L) {
                __builtin_amdgcn_sched_barrier(0);
                load(j, s + S - 1, next);
                __builtin_amdgcn_sched_barrier(0);
              }
            }
        }
        slot = slot == S - 1 ? 0 : slot + 1;
      }
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");

    // The results leave through LDS, so that rows are stored whole: written as
    // they lie in the accumulators they were 16 bytes of 32 rows an instruction (4,093
    // rows, K = 2,048, N = 7,168 130 us, not 66; nontemporal 64).
    // Lane: row lane % 32, columns 8 (r / 4) + 4 (lane / 32) + r % 4 of each tile.
    __syncthreads();
#pragma unroll
    for (int h = 0; h < NT; h += kSwiglu ? 2 : 1) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int c = (wn * NT + h) / (kSwiglu ? 2 : 1) * 32 + 8 * g + 4 * hi;
        const int at = (wn * NT + h) * 32 + 8 * g + 4 * hi;  // weight row of the tile
        const f32x4 ws = *reinterpret_cast<const f32x4*>(scales + at);
        const f32x4 us = *reinterpret_cast<const f32x4*>(scales + (kSwiglu ? at + 32 : at));
#pragma unroll
        for (int q = 0; q < MT; ++q) {
          const int row = (wm * MT + q) * 32 + (lane & 31);
          const float xs = scales[BN + row];
          bf16x4 y;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float v = float(acc[h][q][4 * g + r]) * xs * ws[r];
            if (kSwiglu) v = swiglu(v, float(acc[(h + 1) % NT][q][4 * g + r]) * xs * us[r]);
            y[r] = __bf16(v);
          }
          *reinterpret_cast<bf16x4*>(lds + row * kPitch + c * 2) = y;
        }
      }
    }
    __syncthreads();
    __bf16* to = reinterpret_cast<__bf16*>(a.out) + row0 * a.wide + n0;
    constexpr int kPieces = kCols / 8;  // of 16 bytes, a row
    for (int at = threadIdx.x; at < nr * kPieces; at += W * kWave) {
      const int row = at / kPieces, c = at % kPieces * 8;
      const bf16x8 y = *reinterpret_cast<const bf16x8*>(lds + row * kPitch + c * 2);
      __bf16* p = to + int64_t(row) * a.wide + c;
      if (c + 8 <= held) {
        // whole pieces also where rows of out begin at odd addresses, which this memory
        // takes (3,088 rows, K = 1,920, N = 5,322 57 us, value by value 71; N = 5,376 56)
        __builtin_nontemporal_store(y, reinterpret_cast<bf16x8_any*>(p));
      } else {
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (c + r < held) p[r] = y[r];
      }
    }
    __syncthreads();  // LDS is written anew when every wave is done with it
  }
}

// ---------------------------------------------------------------------------

// Forms of the two kernels, and what each takes. A launch's time goes in rounds:
// every CU takes per_cu workgroups at a time, and a round with at most one for
// each CU, or else with two, takes fixed + step * (steps of 128 values) ns.
struct Form {
  int rows, weights;  // of a workgroup (with SwiGLU two weight rows make a column)
  int waves, over_k;  // its waves, and how many parts they cut K into
  int per_cu;
  int fixed1, step1, fixed2, step2;
};

// The times are fitted to 790 measured ones: rows from 1 to 16,384, plain and of 2 to
// 48 experts, K and N from 1,024 to 7,168. Chosen by them, a launch takes 0.6% more than
// in the form that was the fastest there, 31% at most (20 rows each of 2 experts). Every
// form is the best of some sizes (K = 5,120, N = 4,096 with SwiGLU, kernel us, the forms
// next to it in brackets): 32 rows 7.1 in form 0 (8.4); 64 rows 8.2 in form 1 (11.2, 11.2);
// 128 rows 11.1 in form 2 (13.6, 14.7); 256 rows 15.1 in form 3 (19.2, 18.9); 512 rows 19.5
// in form 4 (21.0, 32.7); 1,300 rows 38.9 in form 5 (45.0, 59.9); 4,093 rows 78.9 in form 6
// (87.5). Tiles of 128 x 128 by 4 waves were 3% better than form 5 at 2,048 rows of K =
// 2,048 and 10% worse for experts: there is no form of them.
constexpr Form kForms[] = {
    {32, 16, 8, 8, 1, 1770, 490, 0, 0},       {32, 32, 4, 4, 1, 1900, 386, 0, 0},
    {64, 32, 4, 4, 1, 2510, 564, 0, 0},       {64, 64, 2, 1, 2, 3520, 223, 2970, 435},
    {64, 128, 4, 1, 2, 2300, 330, 3410, 690}, {128, 256, 8, 1, 1, 5770, 782, 0, 0},
    {256, 256, 8, 1, 1, 9700, 1296, 0, 0},
};
constexpr int kFormCount = sizeof(kForms) / sizeof(kForms[0]);

template <bool kSwiglu>
void launch(int form, dim3 grid, hipStream_t st, const Int8Args& a) {
  const int threads = kForms[form].waves * kWave;
  switch (form) {
    case 0: product_few<kSwiglu, 2, 1, 8, 3><<<grid, threads, 0, st>>>(a); break;
    case 1: product_few<kSwiglu, 2, 2, 4, 3><<<grid, threads, 0, st>>>(a); break;
    case 2: product_few<kSwiglu, 4, 2, 4, 3><<<grid, threads, 0, st>>>(a); break;
    case 3: product_tile<kSwiglu, 64, 64, 2, 1, 4, 2><<<grid, threads, 0, st>>>(a); break;
    case 4: product_tile<kSwiglu, 64, 128, 2, 2, 3, 2><<<grid, threads, 0, st>>>(a); break;
    case 5: product_tile<kSwiglu, 128, 256, 2, 4, 3, 1><<<grid, threads, 0, st>>>(a); break;
    default: product_tile<kSwiglu, 256, 256, 2, 4, 2, 1><<<grid, threads, 0, st>>>(a);
  }
}

int64_t column_tiles(const Form& f, int N) { return (N + f.weights - 1) / f.weights; }

// The time of a form in ns, for `pairs` rows of `active` experts; an expert's last
// chunk is half full on average.
double time_of(const Form& f, int64_t pairs, int64_t active, int N, int K) {
  const int64_t chunks = active == 1 ? (pairs + f.rows - 1) / f.rows
                                     : std::max(active, pairs / f.rows + active / 2);
  const int64_t granules = (K + kGranule - 1) / kGranule;
  const int64_t steps = (granules + f.over_k - 1) / f.over_k;
  const int64_t tiles = chunks * column_tiles(f, N), round = int64_t(256) * f.per_cu;
  const int64_t full = tiles / round, rest = tiles % round;
  const double one = f.fixed1 + f.step1 * double(steps), two = f.fixed2 + f.step2 * double(steps);
  if (f.per_cu == 1) return double(full + (rest > 0)) * one;
  return double(full) * two + (rest > 256 ? two : rest > 0 ? one : 0.0);
}

int form_of(int64_t pairs, int64_t active, int N, int K) {
  int best = 1;
  for (int f = 0; f < kFormCount; ++f) {
    // form 0 reaches from a gate to its other factor by a 32-bit offset
    if (f == 0 && int64_t(N) * K >= int64_t(1) << 31) continue;
    if (time_of(kForms[f], pairs, active, N, K) < time_of(kForms[best], pairs, active, N, K))
      best = f;
  }
  return best;
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
  const int64_t active = std::min<int64_t>(shape->E, pairs);
  const int form = form_of(pairs, active, N, shape->H);
  // chunks of the experts' rows, at most, and tiles of the weights' columns
  const int64_t chunks = active + (pairs - active) / kForms[form].rows;
  const int64_t tiles = column_tiles(kForms[form], N);
  const Int8Args a{rows, row_scale, expert_counts, expert_offsets, w_q, w_scale, out, err_word,
                   cap_expert, int(pairs), shape->E, shape->H, N, swiglu ? N / 2 : N, int(tiles)};
  // The two large tiles go round the workgroups that the CUs hold at once, which find
  // the experts' chunks only once (8,192 rows of 32 experts, K = 2,048, N = 7,168 185 us
  // against 197); smaller ones are taken as CUs come free (384 rows of 48 experts, K =
  // 5,120, N = 4,096 169 us against 171).
  const bool large = kForms[form].waves == 8 && kForms[form].over_k == 1;
  const dim3 grid(uint32_t(std::min<int64_t>(chunks * tiles, large ? 256 : kMostGroups)));
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (swiglu)
    launch<true>(form, grid, st, a);
  else
    launch<false>(form, grid, st, a);
  return launch_status();
}

}  // extern "C"
