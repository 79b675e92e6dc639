// Reductions over the 64 lanes of a wave; every lane gets the result.  Rotations
// inside rows of 16 lanes (DPP), then the swap instructions for rows and halves:
// register to register, a few cycles a step, where shuffles go through LDS.
// Rotations add in another order in every lane, so lane 0's result is handed
// to all.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace swm {

template <int n>
__device__ __forceinline__ uint32_t rotate_row(uint32_t v) {
  return uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0x120 | n, 0xf, 0xf, true));
}

// v combined over the wave by op, on 32-bit words.
template <typename Op>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, Op op) {
  v = op(v, rotate_row<1>(v));
  v = op(v, rotate_row<2>(v));
  v = op(v, rotate_row<4>(v));
  v = op(v, rotate_row<8>(v));
  // the same value twice: odd and even rows (halves) exchanged, the two results
  // hold both partners' values
  const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = op(r[0], r[1]);
  const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return uint32_t(__builtin_amdgcn_readfirstlane(int(op(h[0], h[1]))));
}

__device__ __forceinline__ float wave_max(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
__device__ __forceinline__ float wave_sum(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
__device__ __forceinline__ uint32_t wave_sum(uint32_t v) {
  return wave_reduce(v, [](uint32_t a, uint32_t b) { return a + b; });
}
__device__ __forceinline__ uint32_t wave_min(uint32_t v) {
  return wave_reduce(v, [](uint32_t a, uint32_t b) { return min(a, b); });
}
__device__ __forceinline__ int wave_max(int v) {
  return int(wave_reduce(uint32_t(v), [](uint32_t a, uint32_t b) { return uint32_t(max(int(a), int(b))); }));
}

// Sums of the lanes up to and including this one: shifts inside rows of 16
// lanes, then the last lane of a row to the next row, of a half to the other
// (lanes without a source add zero).
template <int ctrl, int rows>
__device__ __forceinline__ uint32_t add_from(uint32_t v) {
  return v + uint32_t(__builtin_amdgcn_update_dpp(0, int(v), ctrl, rows, 0xf, false));
}
__device__ __forceinline__ uint32_t scan_wave(uint32_t v) {
  v = add_from<0x111, 0xf>(v);  // row_shr 1, 2, 4, 8
  v = add_from<0x112, 0xf>(v);
  v = add_from<0x114, 0xf>(v);
  v = add_from<0x118, 0xf>(v);
  v = add_from<0x142, 0xa>(v);  // row_bcast 15 into rows 1 and 3
  return add_from<0x143, 0xc>(v);  // row_bcast 31 into rows 2 and 3
}

}  // namespace swm
