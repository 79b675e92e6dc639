// Log probabilities of given tokens, entropies and most likely tokens from
// rows of logits.
//
//   log p_t = x_t - log Z,  Z = sum_i e^x_i,  H = log Z - sum_i p_i x_i
//
// One workgroup per row and one pass over it: every thread keeps a running
// maximum m, l = sum e^(x - m) and s = sum e^(x - m) (x - m), all in fp32;
// a larger maximum m' rescales them by r = e^(m - m') to l r and
// (s + l (m - m')) r.  The parts are merged by the same rule.  With the row's
// maximum taken off everywhere, log p_t = (x_t - m) - log l and
// H = log l - s / l lose nothing to large logits.  Exponents are in base 2:
// x - m becomes one fused multiply-add with log2(e), exact up to its one
// rounding and that of the base m log2(e), which is the same for every logit of
// a part and is taken off again in the end.
//
// That rounding grows with m, and fp32 logits reach 3.4e38 (a usual mask).  So
// the running maximum starts at -2^24 instead of -inf: logits far below that add
// zeros as long as anything in the row is larger.  A row whose own maximum is
// beyond 2^24 either way is summed once more with the maximum known and
// subtracted first, which is exact there.  Subtracting first everywhere is one
// instruction more per logit: 300 x 50021 fp32, 20 top tokens 22.2 us so, 19.6
// this way.
//
// The top tokens need no second pass over the row.  The k-th largest of the
// maxima of 64 or 128 groups of threads is a lower bound of the k-th largest
// logit, and only the logits of threads whose own maximum reaches it are looked
// at again (a few more than k of them pass).  The candidates are ranked by
// counting; a token's rank is the number of candidates with a larger logit, or
// an equal one at a lower index.  Rows with so many equal logits that the list
// overflows (a constant row) take the larger ones first and then the equal
// ones in index order, and stop at k; if even the larger ones overflow, k
// rounds of a maximum over the row.  NaN stand before all numbers in this order,
// in the threads' maxima as among the candidates: were a bound taken without
// them, a row of NaN would have no logit at its bound.
//
// Bound: with many rows the read of the logits (2 or 4 bytes each), the
// exponentials (one per logit, at a quarter of the vector rate) and the five
// other vector instructions close behind: 4096 x 32000 fp16 44 us in the
// kernel, 262 MB at 5.9 TB/s.  With few rows the chain of one load, two
// reductions and the choice of the top tokens: 1 x 32000 fp16 with 5 of them
// 7.5 us in the kernel (4.6 with none), 61 x 50021 fp32 with 20 11.4 (7.4).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kernels.h"
#include "wave.h"

// A part's base m log2(e) is one rounded number wherever it is used: fusing
// its product into a subtraction would give parts of different bases.  Other
// multiply-adds that are meant to be fused are written out.
#pragma clang fp contract(off)

namespace swm {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kMaxGroups = 128;  // groups whose maxima bound the top tokens from below

struct LogprobArgs {
  const void* x;
  const void* targets;
  float *logp, *entropy, *top_logp;
  int64_t* top_ids;
  int64_t ld;
  int32_t V, top, wide;  // wide: 64-bit targets
};

template <typename T>
struct Row;
template <>
struct Row<_Float16> {
  static constexpr int kVec = 8;
  static constexpr uint32_t kNone = 0xfc00fc00u;  // -inf
  static __device__ __forceinline__ void unpack(const u32x4& w, float* f) {
    typedef _Float16 half8 __attribute__((ext_vector_type(8)));
    const half8 h = __builtin_bit_cast(half8, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = float(h[e]);
  }
};
template <>
struct Row<float> {
  static constexpr int kVec = 4;
  static constexpr uint32_t kNone = 0xff800000u;
  static __device__ __forceinline__ void unpack(const u32x4& w, float* f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(w[e]);
  }
};

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// Logits by size as whole numbers, -0 like +0, NaN before all; 0 is below all.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  if ((b & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

constexpr float kFar = 16777216.f;  // 2^24

// A part of a row: its maximum, or -kFar if that is larger, and the sums
// relative to it.
struct Part {
  float m = -kFar, l = 0.f, s = 0.f;
};

__device__ __forceinline__ void rebase(Part& p, float m) {
  const float d = p.m * kLog2e - m * kLog2e;
  const float r = __builtin_amdgcn_exp2f(d);
  p.s = (p.s + p.l * d) * r;
  p.l *= r;
  p.m = m;
}
// The term of exponent d; one of -inf is 0 times a finite number.
__device__ __forceinline__ void add(Part& p, float d) {
  const float q = __builtin_amdgcn_exp2f(d);
  p.l += q;
  p.s = __builtin_fmaf(q, fmaxf(d, -150.f), p.s);
}
// own: the largest logit so far.
template <int n>
__device__ __forceinline__ void take(Part& p, float& own, const float* f) {
#pragma unroll
  for (int e = 0; e < n; ++e) own = fmaxf(own, f[e]);
  if (__builtin_amdgcn_ballot_w64(own > p.m)) rebase(p, fmaxf(p.m, own));
  const float b = p.m * kLog2e;
#pragma unroll
  for (int e = 0; e < n; ++e) add(p, __builtin_fmaf(f[e], kLog2e, -b));
}

// kR > 0: a thread's vectors, kR at most, stay in registers and the top tokens
// are found there; kR = 0: the row is streamed.
template <typename T, int kThreads, int kR, bool kTop>
__global__ __launch_bounds__(kThreads) void logprobs_kernel(LogprobArgs a) {
  constexpr int kVec = Row<T>::kVec;
  constexpr int kWaves = kThreads / 64;
  __shared__ float red[kWaves][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t n = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + n * a.ld;
  // logits before the first 16-byte boundary, whole vectors, the rest
  const int lead = min(int((16 - (reinterpret_cast<uintptr_t>(x) & 15)) % 16 / sizeof(T)), a.V);
  const int vecs = (a.V - lead) / kVec;
  const int rest = lead + vecs * kVec;
  const u32x4* xv = reinterpret_cast<const u32x4*>(x + lead);
  const bool head = tid < lead, tail = rest + tid < a.V;  // a logit of either end

  Part p;
  float own = neg_inf();  // the largest logit of this thread
  u32x4 keep[kR > 0 ? kR : 1];
  if constexpr (kR > 0) {
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      constexpr uint32_t z = Row<T>::kNone;
      keep[r] = tid + r * kThreads < vecs ? xv[tid + r * kThreads] : u32x4{z, z, z, z};
    }
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      if (r * kThreads < vecs) {  // the same for every thread
        float f[kVec];
        Row<T>::unpack(keep[r], f);
        take<kVec>(p, own, f);
      }
    }
  } else {
    constexpr int kUnroll = 4;
    int i = tid;
    for (; i + (kUnroll - 1) * kThreads < vecs; i += kUnroll * kThreads) {
      u32x4 w[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) w[u] = xv[i + u * kThreads];
      __builtin_amdgcn_sched_barrier(0);  // all requested before the first is waited for
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        float f[kVec];
        Row<T>::unpack(w[u], f);
        take<kVec>(p, own, f);
      }
    }
    for (; i < vecs; i += kThreads) {
      float f[kVec];
      Row<T>::unpack(xv[i], f);
      take<kVec>(p, own, f);
    }
  }
  const float xh = head ? float(x[tid]) : neg_inf(), xt = tail ? float(x[rest + tid]) : neg_inf();
  int64_t target = -1;
  float at_target = 0.f;
  if (a.targets && tid == 0) {
    target = a.wide ? static_cast<const int64_t*>(a.targets)[n] : int64_t(static_cast<const int32_t*>(a.targets)[n]);
    at_target = float(x[target >= 0 && target < a.V ? target : 0]);
  }
  if (lead > 0) take<1>(p, own, &xh);
  if (rest < a.V) take<1>(p, own, &xt);

  // A thread without logits has the key 0, below that of -inf.
  constexpr int kGroups = kThreads < kMaxGroups ? kThreads : kMaxGroups;
  __shared__ alignas(16) uint32_t group[kTop ? kGroups : 1];  // maxima of kThreads / kGroups threads
  __shared__ uint32_t bound, count, passed;
  const bool has = tid < vecs || head || tail;
  uint32_t mine = has ? key_of(own) : 0u;
  if constexpr (kTop) {
    // The maximum leaves NaN out, the candidates' order puts them first: a thread
    // whose sum tells of a NaN (or +inf) looks at its logits by that order.
    if (p.l != p.l) {
      mine = max(head ? key_of(xh) : 0u, tail ? key_of(xt) : 0u);
      for (int i = tid; i < vecs; i += kThreads) {
        float f[kVec];
        Row<T>::unpack(xv[i], f);
#pragma unroll
        for (int e = 0; e < kVec; ++e) mine = max(mine, key_of(f[e]));
      }
    }
    constexpr int kPer = kThreads / kGroups;
    uint32_t g = mine;
    if (kPer > 1) g = max(g, rotate_row<1>(g));  // 2 or 8 consecutive lanes of a row: maxima of the last kPer
    if (kPer > 2) g = max(g, rotate_row<2>(g));
    if (kPer > 4) g = max(g, rotate_row<4>(g));
    if (tid % kPer == kPer - 1) group[tid / kPer] = g;
    if (tid == 0) {
      count = passed = 0;
      bound = 0xffffffffu;
    }
  }

  // Maximum first, then every part moves to it once and the sums are added.
  rebase(p, wave_max(p.m));
  p.l = wave_sum(p.l);
  p.s = wave_sum(p.s);
  if constexpr (kWaves > 1) {
    if (lane == 0) {
      red[wave][0] = p.m;
      red[wave][1] = p.l;
      red[wave][2] = p.s;
    }
    __syncthreads();
    p = Part{};
    if (lane < kWaves) p = Part{red[lane][0], red[lane][1], red[lane][2]};
    rebase(p, wave_max(p.m));
    p.l = wave_sum(p.l);
    p.s = wave_sum(p.s);
  }
  // what the base's rounding has added to every exponent
  float off = __builtin_fmaf(p.m, kLog2e, -(p.m * kLog2e));
  if (sizeof(T) == 4 && !(p.m > -kFar && p.m <= kFar)) {  // the same for every thread: a row of -inf or far from zero
    red[wave][3] = wave_max(own);
    __syncthreads();
    const float m = wave_max(red[min(lane, kWaves - 1)][3]);
    if (m > neg_inf()) {
      p = Part{m, 0.f, 0.f};
      off = 0.f;
#pragma unroll 1
      for (int i = tid; i < vecs; i += kThreads) {
        float f[kVec];
        Row<T>::unpack(xv[i], f);
#pragma unroll
        for (int e = 0; e < kVec; ++e) add(p, (f[e] - m) * kLog2e);
      }
      add(p, (xh - m) * kLog2e);
      add(p, (xt - m) * kLog2e);
      p.l = wave_sum(p.l);
      p.s = wave_sum(p.s);
      if (lane == 0) {
        red[wave][1] = p.l;
        red[wave][2] = p.s;
      }
      __syncthreads();
      p.l = wave_sum(lane < kWaves ? red[lane][1] : 0.f);
      p.s = wave_sum(lane < kWaves ? red[lane][2] : 0.f);
    }
  }
  const bool none = p.l == 0.f;  // every logit is -inf: log probabilities of -inf, entropy 0
  const float log2l = none ? 0.f : __builtin_log2f(p.l);
  const float logl = (log2l - off) * kLn2;
  auto logp_of = [&](float v) { return (v - p.m) - logl; };

  if (tid == 0) {
    if (a.targets) a.logp[n] = target < 0 ? 0.f : target < a.V ? logp_of(at_target) : __builtin_nanf("");
    if (a.entropy) a.entropy[n] = none ? 0.f : (log2l - p.s / p.l) * kLn2;
  }
  if constexpr (kTop) {
  constexpr int kList = kThreads < 256 ? 512 : 1024;  // candidates ranked by counting
  __shared__ uint64_t list[kList];
  __shared__ uint16_t who[kThreads];  // threads whose maximum reaches the bound
  const int k = min(a.top, a.V);
  if (kWaves == 1) __syncthreads();
  // The k-th largest of the groups' maxima is the least of those that fewer than
  // k exceed.
  if (tid < kGroups) {
    const uint32_t v = group[tid];
    int above = 0;
#pragma unroll 8
    for (int j = 0; j < kGroups; j += 4) {
      const u32x4 o = *reinterpret_cast<const u32x4*>(&group[j]);
#pragma unroll
      for (int e = 0; e < 4; ++e) above += o[e] > v;
    }
    const uint32_t least = wave_min(above < k ? v : 0xffffffffu);
    if (lane == 0) atomicMin(&bound, least);
  }
  __syncthreads();
  const uint32_t low = bound;

  // Appends the logits with keys of at least `least`; the count keeps growing
  // past the end of the list.  The threads whose maximum reaches it are listed
  // first, and their vectors are dealt to all threads: a few hundred loads at
  // once, in a loop of few instructions.  (Every thread searching its own
  // registers was a long unrolled code that each wave met cold: 300 x 50021 fp32,
  // 20 top tokens 43 us so, 24 this way.)
  auto collect = [&](uint32_t least) {
    auto push = [&](float f, int at) {
      const uint32_t key = key_of(f);
      if (key < least) return;
      const uint32_t c = atomicAdd(&count, 1u);
      if (c < kList) list[c] = uint64_t(key) << 32 | (0xffffffffu - uint32_t(at));
    };
    const bool pass = has && mine >= least;
    if (pass && tid < vecs) who[atomicAdd(&passed, 1u)] = uint16_t(tid);
    if (pass && head) push(xh, tid);
    if (pass && tail) push(xt, rest + tid);
    __syncthreads();
    const uint32_t n_pass = passed, rounds = uint32_t(vecs + kThreads - 1) / kThreads;
    for (uint32_t i = tid; i < n_pass * rounds; i += kThreads) {
      if (*const_cast<volatile uint32_t*>(&count) > kList) break;  // this list is not used
      const uint32_t r = i / n_pass, v = who[i - r * n_pass] + r * kThreads;
      if (v >= uint32_t(vecs)) continue;
      float f[kVec];
      Row<T>::unpack(xv[v], f);
#pragma unroll
      for (int e = 0; e < kVec; ++e) push(f[e], lead + int(v) * kVec + e);
    }
    __syncthreads();
  };
  collect(low);
  int found = int(count);
  int64_t* ids = a.top_ids + n * a.top;
  float* lps = a.top_logp + n * a.top;
  // More than the bound lets through by chance: equal logits, which are faster
  // taken in index order than ranked (2032 x 387, 32 top, a row of nothing but
  // -inf among them: 40 us ranked, 11 so).
  if (found > min(max(6 * k, 128), kList)) {
    __syncthreads();
    if (tid == 0) count = passed = 0;
    __syncthreads();
    if (low != 0xffffffffu) collect(low + 1);
    found = int(count);
    if (found <= kList - 64) {
      // the lowest indices with the bound's own key fill up the k; the row's end
      // is a second limit, so that the loop ends whatever the row holds
      for (int j0 = 0; found < k && j0 < a.V; j0 += kThreads) {
        const int j = j0 + tid;
        __syncthreads();
        const bool on = j < a.V && key_of(float(x[j])) == low;
        const uint64_t b = __builtin_amdgcn_ballot_w64(on);
        if (lane == 0) group[wave] = __popcll(b);
        __syncthreads();
        int at = found + __builtin_amdgcn_mbcnt_hi(uint32_t(b >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(b), 0u));
        for (int w = 0; w < kWaves; ++w) {
          at += w < wave ? group[w] : 0;
          found += group[w];
        }
        if (on && at < k) list[at] = uint64_t(low) << 32 | (0xffffffffu - uint32_t(j));
      }
      found = min(found, max(k, int(count)));
      __syncthreads();
    } else {
      // k rounds: the best logit after the last one's place in the order
      uint64_t last = ~0ull;
      for (int r = 0; r < k; ++r) {
        uint64_t best = 0;
        for (int j = tid; j < a.V; j += kThreads) {
          const uint64_t c = uint64_t(key_of(float(x[j]))) << 32 | (0xffffffffu - uint32_t(j));
          if ((r == 0 || c < last) && c > best) best = c;  // a NaN at index 0 has the largest number there is
        }
#pragma unroll
        for (int s = 1; s < 64; s *= 2) best = max(best, uint64_t(__shfl_xor((unsigned long long)best, s)));
        __syncthreads();
        if (lane == 0) list[wave] = best;
        __syncthreads();
        for (int w = 0; w < kWaves; ++w) best = max(best, list[w]);
        last = best;
        if (tid == 0) {
          ids[r] = int64_t(0xffffffffu - uint32_t(best));
          lps[r] = logp_of(value_of(uint32_t(best >> 32)));
        }
      }
      found = 0;
    }
  }
  for (int c = tid; c < found; c += kThreads) {
    const uint64_t v = list[c];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < found; ++j) rank += list[j] > v;
    if (rank < k) {
      ids[rank] = int64_t(0xffffffffu - uint32_t(v));
      lps[rank] = logp_of(value_of(uint32_t(v >> 32)));
    }
  }
  for (int r = k + tid; r < a.top; r += kThreads) {  // more asked for than there are tokens
    ids[r] = -1;
    lps[r] = neg_inf();
  }
  }
}

template <typename T, int kThreads, int kR>
hipError_t launch(const LogprobArgs& a, int64_t N, hipStream_t s) {
  const dim3 grid = dim3(uint32_t(N));
  if (a.top > 0)
    logprobs_kernel<T, kThreads, kR, true><<<grid, kThreads, 0, s>>>(a);
  else
    logprobs_kernel<T, kThreads, kR, false><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

// Threads of a row: more where the rows do not fill the chip, and no more than
// the row has work for.  Rows whose vectors fit in the registers of their
// threads (8 a thread; 16 of 1024 threads) stay there.  Measured, us:
//   below one row per CU    255 x 50021 fp32, 20 top tokens: 1024 threads 14,
//                           256 threads 19; 1 x 128000 fp16, 20: 15 and 21
//   from one row per CU on  300 x 50021 fp32, 20: 256 threads 20, 1024 23, 64
//                           76; 1500 x 32000 fp16: 20, 28, 25
//   from eight, no top      4096 x 32000 fp16: 64 threads 42, 256 44, 1024 67
//   tokens                  (with 20 of fp32: 64 threads 171, 256 117: a wave
//                           alone looks at its candidates in many rounds)
template <typename T>
hipError_t launch_rows(const LogprobArgs& a, int64_t N, int num_cus, hipStream_t s) {
  constexpr int kR = 8, kWide = 16;
  const int64_t vecs = a.V / Row<T>::kVec + 1;
  const int by_rows = N >= 8 * num_cus && a.top == 0 ? 64 : N >= num_cus ? 256 : 1024;
  // many top tokens of a short row are most of the row to rank: 1000 x 300, 64:
  // 27 us by 64 threads, 18 by 256
  const int by_row = vecs <= 256 && a.top <= 32 ? 64 : vecs <= 2048 ? 256 : 1024;
  switch (std::min(by_rows, by_row)) {
    case 64:
      if (vecs <= 64 * kR) return launch<T, 64, kR>(a, N, s);
      logprobs_kernel<T, 64, 0, false><<<uint32_t(N), 64, 0, s>>>(a);  // by its rows, so no top tokens
      return hipGetLastError();
    case 256: return vecs <= 256 * kR ? launch<T, 256, kR>(a, N, s) : launch<T, 256, 0>(a, N, s);
    default: return vecs <= 1024 * kWide ? launch<T, 1024, kWide>(a, N, s) : launch<T, 1024, 0>(a, N, s);
  }
}

}  // namespace

hipError_t launch_logprobs(const LogprobCall& r, int num_cus, hipStream_t s) {
  LogprobArgs a{};
  a.x = r.logits;
  a.targets = r.targets;
  a.logp = r.logp;
  a.entropy = r.entropy;
  a.top_logp = r.top_logp;
  a.top_ids = r.top_ids;
  a.ld = r.ld;
  a.V = int(r.V);
  a.top = r.top;
  a.wide = r.wide;
  return r.fp32 ? launch_rows<float>(a, r.N, num_cus, s) : launch_rows<_Float16>(a, r.N, num_cus, s);
}

}  // namespace swm
