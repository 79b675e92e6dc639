// Division by the page size as one multiplication: t / S = (t m) >> p for
// 0 <= t < 2^31.  With 2^l >= S the shift is p = 31 + l and m = floor(2^p / S)
// + 1 < 2^32 + 1; m S exceeds 2^p by e <= S <= 2^l, so the quotient is off by
// t e / (S 2^p) < 1 / S, too little to reach the next whole number.  (S a power
// of two: 2^31 2^l / S + 1 still fits 32 bits, and the same bound holds.)
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace swm {

struct PageDiv {
  uint32_t m = 0;
  int32_t p = 31;
};

inline PageDiv page_div(int64_t S) {
  int l = 0;
  while ((int64_t(1) << l) < S) ++l;
  PageDiv d;
  d.p = 31 + l;
  d.m = uint32_t((uint64_t(1) << d.p) / uint64_t(S) + 1);
  return d;
}

__device__ __forceinline__ int page_index(const PageDiv& d, int t) { return int((uint64_t(uint32_t(t)) * d.m) >> d.p); }

}  // namespace swm
