// Inclusive scans over the 64 lanes of a wavefront inside the vector unit (fixed
// order: 1, 2, 4 and 8 lanes within each row of 16, then the rows).
#pragma once

#include "moe_common.h"

namespace bitffn {

// v of the lane that the DPP control names, `none` where there is no such lane or
// the row is not in ROWS.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_or(int v, int none) {
  return __builtin_amdgcn_update_dpp(none, v, CTRL, ROWS, 0xF, false);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_or_zero(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = dpp_or<CTRL, ROWS>(static_cast<int>(u), 0);
  const uint32_t hi = dpp_or<CTRL, ROWS>(static_cast<int>(u >> 32), 0);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

constexpr int kRowShr1 = 0x111, kRowShr2 = 0x112, kRowShr4 = 0x114, kRowShr8 = 0x118;
constexpr int kRowBcast15 = 0x142;   // lane 15 of a row to the next row
constexpr int kRowBcast31 = 0x143;   // lane 31 to the upper half

__device__ __forceinline__ int wave_scan_add(int v) {
  v += dpp_or<kRowShr1, 0xF>(v, 0);
  v += dpp_or<kRowShr2, 0xF>(v, 0);
  v += dpp_or<kRowShr4, 0xF>(v, 0);
  v += dpp_or<kRowShr8, 0xF>(v, 0);
  v += dpp_or<kRowBcast15, 0xA>(v, 0);
  return v + dpp_or<kRowBcast31, 0xC>(v, 0);
}

// v >= 0
__device__ __forceinline__ int wave_scan_max(int v) {
  v = max(v, dpp_or<kRowShr1, 0xF>(v, 0));
  v = max(v, dpp_or<kRowShr2, 0xF>(v, 0));
  v = max(v, dpp_or<kRowShr4, 0xF>(v, 0));
  v = max(v, dpp_or<kRowShr8, 0xF>(v, 0));
  v = max(v, dpp_or<kRowBcast15, 0xA>(v, 0));
  return max(v, dpp_or<kRowBcast31, 0xC>(v, 0));
}

__device__ __forceinline__ double wave_scan_add(double v) {
  v += dpp_or_zero<kRowShr1, 0xF>(v);
  v += dpp_or_zero<kRowShr2, 0xF>(v);
  v += dpp_or_zero<kRowShr4, 0xF>(v);
  v += dpp_or_zero<kRowShr8, 0xF>(v);
  v += dpp_or_zero<kRowBcast15, 0xA>(v);
  return v + dpp_or_zero<kRowBcast31, 0xC>(v);
}

// The value of one lane, the same for all.
__device__ __forceinline__ int lane_value(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = lane_value(static_cast<int>(u), lane);
  const uint32_t hi = lane_value(static_cast<int>(u >> 32), lane);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// The value of the lane before, 0 in lane 0.
template <typename T>
__device__ __forceinline__ T lane_before(T v) {
  const T up = __shfl_up(v, 1);
  return (threadIdx.x & 63) == 0 ? T(0) : up;
}

}  // namespace bitffn
