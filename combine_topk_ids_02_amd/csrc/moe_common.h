// What the router's and the expert products' kernels share: the wave's
// helpers, the limits of a shape and the host's checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "moe_dispatch.h"

namespace moe {

constexpr int kWave = 64;
constexpr int kMaxExperts = 1024;
constexpr int kMaxRanks = 64;
constexpr int kMaxK = 16;

__device__ __forceinline__ int lane_id() { return __lane_id(); }

// The wave's index in its workgroup, in a scalar register (the compiler does
// not know that threadIdx.x / 64 is the same in every lane of a wave).
__device__ __forceinline__ int wave_in_block() {
  return __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
}

__device__ __forceinline__ int read_lane(int v, int lane) {
  return __builtin_amdgcn_readlane(v, lane);
}

__device__ __forceinline__ float read_lane(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

__device__ __forceinline__ void flag_error(int32_t* err_word, int bit) {
  if (err_word) atomicOr(err_word, bit);
}

// A lane's value from another lane of its row of 16, or from an earlier row
// (data-parallel primitives, no LDS); a lane without a source keeps `old`.
template <int kCtrl, int kRowMask = 0xF>
__device__ __forceinline__ float dpp(float old, float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(v), kCtrl,
                                                    kRowMask, 0xF, false));
}

constexpr int kRowShr = 0x110;     // + n: from n lanes below within the row
constexpr int kRowRor = 0x120;     // + n: rotated within the row
constexpr int kRowBcast15 = 0x142; // row r from lane 15 of row r-1
constexpr int kRowBcast31 = 0x143; // rows 2, 3 from lane 31

// Sum of the 16 lanes of a row, in every lane of it.
__device__ __forceinline__ float row_sum(float v) {
  v += dpp<kRowRor + 8>(0.0f, v);
  v += dpp<kRowRor + 4>(0.0f, v);
  v += dpp<kRowRor + 2>(0.0f, v);
  v += dpp<kRowRor + 1>(0.0f, v);
  return v;
}

__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, dpp<kRowRor + 8>(v, v));
  v = fmaxf(v, dpp<kRowRor + 4>(v, v));
  v = fmaxf(v, dpp<kRowRor + 2>(v, v));
  v = fmaxf(v, dpp<kRowRor + 1>(v, v));
  return v;
}

// Maximum / sum over the wave, uniform.
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp<kRowShr + 1>(v, v));
  v = fmaxf(v, dpp<kRowShr + 2>(v, v));
  v = fmaxf(v, dpp<kRowShr + 4>(v, v));
  v = fmaxf(v, dpp<kRowShr + 8>(v, v));
  v = fmaxf(v, dpp<kRowBcast15, 0xA>(v, v));
  v = fmaxf(v, dpp<kRowBcast31, 0xC>(v, v));
  return read_lane(v, 63);
}

__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<kRowShr + 1>(0.0f, v);
  v += dpp<kRowShr + 2>(0.0f, v);
  v += dpp<kRowShr + 4>(0.0f, v);
  v += dpp<kRowShr + 8>(0.0f, v);
  v += dpp<kRowBcast15, 0xA>(0.0f, v);
  v += dpp<kRowBcast31, 0xC>(0.0f, v);
  return read_lane(v, 63);
}

// The limits of moe_dispatch.h's "Common conventions" that concern T, H, E, R,
// k, align and block.
inline bool shape_ok(const moe_shape_t* s) {
  if (!s) return false;
  if (s->T < 0 || s->H <= 0 || s->H % 8 != 0) return false;
  if (s->R < 1 || s->R > kMaxRanks || s->E < 1 || s->E > kMaxExperts || s->E % s->R != 0)
    return false;
  if (s->k < 1 || s->k > kMaxK) return false;
  if (s->align < 1 || s->align > (1 << 16) || s->block < 0) return false;
  if (s->block > 0 && s->align != 1) return false;
  if (int64_t(s->E) * s->block + int64_t(s->T) * s->k >= (int64_t(1) << 31)) return false;
  if (int64_t(s->T) * s->k + int64_t(s->E) * (s->align - 1) >= (int64_t(1) << 31)) return false;
  if (int64_t(s->T) * s->k >= (int64_t(1) << 30)) return false;
  if (int64_t(s->T) * s->R >= (int64_t(1) << 31)) return false;
  return true;
}

inline bool aligned(const void* p, size_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

inline int launch_status() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

}  // namespace moe
