// What a product's epilogue does to an fp32 sum before its one rounding:
// act(sum + bias[m]) + residual[n][m].
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "kernels.h"

namespace swm {

// GELU by the error function, v Phi(v) = max(v, 0) - u Phi(-u) with u = |v|.
// Phi(-u) = t P(t) e^(-u^2 / 2), t = 1 / (1 + 0.27 u), with P fitted to a
// relative error of 1.2e-6 over u = 0..13: relative, so that the small results
// of large negative v keep their bits where 1 + erf would cancel.  Beyond u =
// 16 the tail is below fp32, and the clamp keeps inf * 0 out.  Written as the
// sum 0.5 (v + |v|) a NaN stays one (and -inf gives NaN, as its formula does).
// About 15 instructions and two transcendentals, on up to 128 outputs a lane
// after the last product: 11008 x 4096 at 2048 tokens in one round and a third
// of blocks takes 223 us with bias alone, 227 with SiLU, 238 with GELU.
__device__ __forceinline__ float gelu(float v) {
  const float u = fminf(fabsf(v), 16.f);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.27f, u, 1.f));
  float p = -0.0605442076f;
  p = __builtin_fmaf(p, t, 0.157403131f);
  p = __builtin_fmaf(p, t, -0.022568841f);
  p = __builtin_fmaf(p, t, 0.116333763f);
  p = __builtin_fmaf(p, t, 0.093338313f);
  p = __builtin_fmaf(p, t, 0.108341907f);
  p = __builtin_fmaf(p, t, 0.107695361f);
  const float s = u * 0.84932180028801904272f;  // sqrt(log2(e) / 2)
  const float q = t * p * __builtin_amdgcn_exp2f(-(s * s));
  return __builtin_fmaf(0.5f, v + fabsf(v), -(u * q));
}

// The epilogues a product kernel is built with: none, the gated FFN step's,
// `Epilogue`, or none yet: the fp32 sums of one split of K.  Kernels without
// one keep their own instances: the epilogue's operands and code would cost
// some of them registers and occupancy.
enum { kPlain, kGated, kFused, kPartial };

template <int kAct>
__device__ __forceinline__ float activate(float v) {
  if constexpr (kAct == 1) return v < 0.f ? 0.f : v;
  if constexpr (kAct == 2)
    return v * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v * -1.44269504088896340736f));
  if constexpr (kAct == 3) return gelu(v);
  return v;
}

// f(std::integral_constant<int, act>), for loops over many outputs: one
// branch for all of them.
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case 1: f(std::integral_constant<int, 1>{}); break;
    case 2: f(std::integral_constant<int, 2>{}); break;
    case 3: f(std::integral_constant<int, 3>{}); break;
    default: f(std::integral_constant<int, 0>{}); break;
  }
}

__device__ __forceinline__ float half_at(const uint16_t* p) { return float(__builtin_bit_cast(_Float16, *p)); }

// The matrix products' outputs.  A wave holds kI x kJ accumulators of 32 x 32:
// element v of lane l of accumulator (i, j) is row 32 i + 8 (v/4) + 4 (l/32) +
// v%4 and token 32 j + l%32, from row m0 and token n0 on.
typedef float epi_f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t epi_u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t epi_u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) epi_u32x2 epi_lds_u32x2;
typedef __attribute__((address_space(3))) uint16_t epi_lds_u16;

// Four consecutive halves from p[at]; those from p[end] on read p[end - 1].
__device__ __forceinline__ epi_u32x2 halves4(const uint16_t* p, int at, int end, bool aligned8) {
  if (aligned8 && at + 4 <= end) return *reinterpret_cast<const epi_u32x2*>(p + at);
  uint32_t h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = p[min(at + e, end - 1)];
  return epi_u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
}
__device__ __forceinline__ float half_of(const epi_u32x2& w, int e) {
  return float(__builtin_bit_cast(_Float16, uint16_t(w[e / 2] >> (16 * (e % 2)))));
}
__device__ __forceinline__ bool aligned(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// The bias of a lane's rows, all requested at once.
template <int kI>
__device__ __forceinline__ void load_bias(const Epilogue& e, int m0, int M, int lane, epi_u32x2 (&bias)[kI][4]) {
  const bool vec = aligned(e.bias, 8);  // m0 and the lane's rows are multiples of 4
#pragma unroll
  for (int i = 0; i < kI; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      bias[i][q] = e.bias ? halves4(e.bias, m0 + i * 32 + q * 8 + (lane >> 5) * 4, M, vec) : epi_u32x2{0, 0};
}

// One lane's four outputs of accumulator (i, j), rounded and packed.
template <int kAct>
__device__ __forceinline__ epi_u32x2 fuse4(const epi_f32x16& acc, int q, const epi_u32x2& bias,
                                           const epi_u32x2& res) {
  uint32_t h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    h[e] = __builtin_bit_cast(
        uint16_t, _Float16(activate<kAct>(acc[q * 4 + e] + half_of(bias, e)) + half_of(res, e)));
  return epi_u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
}

// Outputs into the wave's LDS region, a row of `stride` bytes per token, from
// where the kernel stores them.  The residual comes in by the same way: whole
// rows, 16 bytes a lane, and every lane finds the values of its outputs in
// their places; read directly, a load would take 8 bytes from 32 rows.  Rows
// that are not aligned for 16 bytes come in by halves, consecutive ones of a row
// in consecutive lanes (with eight loads of a half a lane 885 x 72 at 174 tokens
// took 20.6 us, 17.0 so).  The barriers keep the scheduler from starting every output at once, which would
// spill the accumulators.
template <int kI, int kJ>
__device__ __forceinline__ void fuse_to_lds(const Epilogue& e, const epi_f32x16 (&acc)[kI][kJ], uint32_t reg,
                                            int stride, int m0, int n0, int M, int N, int lane) {
  constexpr int kTM = 32 * kI, kTN = 32 * kJ, kLPR = kTM / 8, kRPI = 64 / kLPR;
  constexpr int kU = kTN / kRPI < 4 ? kTN / kRPI : 4;  // rounds of rows at a time
  static_assert(kTN % (kU * kRPI) == 0, "");
  epi_u32x2 bias[kI][4];
  load_bias(e, m0, M, lane, bias);
  if (e.residual) {
    const int gm = m0 + (lane % kLPR) * 8;
    const bool rows = e.ldr % 8 == 0 && aligned(e.residual, 16), vec = gm + 8 <= M;
    for (int i0 = 0; !rows && i0 < kTM * kTN / 64; i0 += 8) {
      uint16_t v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int at = (i0 + u) * 64 + lane;
        v[u] = e.residual[int64_t(min(n0 + at / kTM, N - 1)) * e.ldr + min(m0 + at % kTM, M - 1)];
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int at = (i0 + u) * 64 + lane;
        *reinterpret_cast<epi_lds_u16*>(static_cast<uintptr_t>(reg + at / kTM * stride + at % kTM * 2)) = v[u];
      }
    }
    for (int r = 0; rows && r < kTN; r += kU * kRPI) {
      epi_u32x4 v[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint16_t* src = e.residual + int64_t(min(n0 + r + u * kRPI + lane / kLPR, N - 1)) * e.ldr;
        if (vec) {
          v[u] = *reinterpret_cast<const epi_u32x4*>(src + gm);
        } else {
          const epi_u32x2 lo = halves4(src, gm, M, false), hi = halves4(src, gm + 4, M, false);
          v[u] = epi_u32x4{lo[0], lo[1], hi[0], hi[1]};
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint32_t at = reg + (r + u * kRPI + lane / kLPR) * stride + (lane % kLPR) * 16;  // a multiple of 8
        *reinterpret_cast<epi_lds_u32x2*>(static_cast<uintptr_t>(at)) = epi_u32x2{v[u][0], v[u][1]};
        *reinterpret_cast<epi_lds_u32x2*>(static_cast<uintptr_t>(at + 8)) = epi_u32x2{v[u][2], v[u][3]};
      }
    }
  }
  with_act(e.act, [&](auto act) {
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const uint32_t at = reg + (j * 32 + (lane & 31)) * stride + 2 * (i * 32 + (lane >> 5) * 4);
        epi_u32x2 res[4] = {};
        if (e.residual) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            res[q] = *reinterpret_cast<const epi_lds_u32x2*>(static_cast<uintptr_t>(at + 16 * q));
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<epi_lds_u32x2*>(static_cast<uintptr_t>(at + 16 * q)) =
              fuse4<act>(acc[i][j], q, bias[i][q], res[q]);
        __builtin_amdgcn_sched_barrier(0);
      }
  });
}

// Outputs through the wave's LDS region to Y, 16 bytes of a token's row a lane.
// Straight from the accumulators a store would take 8 bytes, or 2 where rows are
// not aligned, of 32 rows (2001 x 480 at 300 tokens, residual and SiLU 18.1 us so,
// 16.8 this way; rows of 2000 16.7 and 16.0).
template <int kI, int kJ>
__device__ __forceinline__ void fuse_and_store_rows(const Epilogue& e, const epi_f32x16 (&acc)[kI][kJ], uint32_t reg,
                                                    int m0, int n0, int M, int N, uint16_t* Y, int64_t ldy,
                                                    int lane) {
  constexpr int kTM = 32 * kI, kTN = 32 * kJ, kLPR = kTM / 8, kRPI = 64 / kLPR, kStride = 2 * kTM + 8;
  fuse_to_lds(e, acc, reg, kStride, m0, n0, M, N, lane);
  if (ldy % 8 != 0 || !aligned(Y, 16)) {  // by halves, as above
#pragma unroll 8
    for (int i = 0; i < kTM * kTN / 64; ++i) {
      const int at = i * 64 + lane, n = n0 + at / kTM, m = m0 + at % kTM;
      const uint16_t v = *reinterpret_cast<const epi_lds_u16*>(static_cast<uintptr_t>(reg + at / kTM * kStride + at % kTM * 2));
      if (n < N && m < M) Y[int64_t(n) * ldy + m] = v;
    }
    return;
  }
  const int gm = m0 + (lane % kLPR) * 8;
  const bool vec = gm + 8 <= M;
#pragma unroll 4
  for (int r = 0; r < kTN; r += kRPI) {
    const int nl = r + lane / kLPR, n = n0 + nl;
    const uint32_t at = reg + nl * kStride + (lane % kLPR) * 16;
    const epi_u32x2 lo = *reinterpret_cast<const epi_lds_u32x2*>(static_cast<uintptr_t>(at));
    const epi_u32x2 hi = *reinterpret_cast<const epi_lds_u32x2*>(static_cast<uintptr_t>(at + 8));
    const epi_u32x4 v = {lo[0], lo[1], hi[0], hi[1]};
    if (n >= N) continue;
    uint16_t* dst = Y + int64_t(n) * ldy + gm;
    if (vec) {
      *reinterpret_cast<epi_u32x4*>(dst) = v;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (gm + k < M) dst[k] = uint16_t(v[k / 2] >> (16 * (k % 2)));
    }
  }
}

// Outputs straight to Y, four rows of a token at a time.
template <int kI, int kJ>
__device__ __forceinline__ void fuse_and_store(const Epilogue& e, const epi_f32x16 (&acc)[kI][kJ], int m0, int n0,
                                               int M, int N, uint16_t* Y, int64_t ldy, int lane) {
  const bool rvec = e.ldr % 4 == 0 && aligned(e.residual, 8);
  const bool yvec = ldy % 4 == 0 && aligned(Y, 8);
  const bool bvec = aligned(e.bias, 8);
  with_act(e.act, [&](auto act) {
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const int n = n0 + j * 32 + (lane & 31);
        const uint16_t* src = e.residual + int64_t(min(n, N - 1)) * e.ldr;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int m = m0 + i * 32 + q * 8 + (lane >> 5) * 4;
          const epi_u32x2 bias = e.bias ? halves4(e.bias, m, M, bvec) : epi_u32x2{0, 0};
          const epi_u32x2 res = e.residual ? halves4(src, m, M, rvec) : epi_u32x2{0, 0};
          const epi_u32x2 w = fuse4<act>(acc[i][j], q, bias, res);
          uint16_t* dst = Y + int64_t(n) * ldy + m;
          if (n < N && m + 4 <= M && yvec) {
            *reinterpret_cast<epi_u32x2*>(dst) = w;
          } else if (n < N) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (m + k < M) dst[k] = uint16_t(w[k / 2] >> (16 * (k % 2)));
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
  });
}

}  // namespace swm
