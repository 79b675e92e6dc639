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
// rounding.
//
// The top tokens need no second pass over the row.  The k-th largest of the
// maxima of 256 groups of threads is a lower bound of the k-th largest logit,
// and only the threads whose own maximum reaches it look at their logits
// again (a few more than k logits pass).  The candidates are ranked by
// counting; a token's rank is the number of candidates with a larger logit, or
// an equal one at a lower index.  Rows with so many equal logits that the list
// overflows (a constant row) take the larger ones first and then the equal
// ones in index order, and stop at k; if even the larger ones overflow, k
// rounds of a maximum over the row.
//
// Bound: the read of the logits (2 or 4 bytes each); with fp16 logits the
// exponentials (one per logit, at a quarter of the vector rate) and the five
// other vector instructions come close to it.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kernels.h"

// A part's base m log2(e) is one rounded number wherever it is used: fusing
// its product into a subtraction would give parts of different bases.  The
// multiply-adds that are meant to be fused are written out.
#pragma clang fp contract(off)

namespace swm {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kGroups = 256;   // groups whose maxima bound the top tokens from below
constexpr int kList = 1024;    // candidates ranked by counting

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

// A part of a row: its maximum, and the sums relative to it.  A part without
// finite logits has the base 0 (its sums are zero, or NaN).
struct Part {
  float m, l, s;
};
__device__ __forceinline__ float base_of(float m) { return m == neg_inf() ? 0.f : m * kLog2e; }

__device__ __forceinline__ void rebase(Part& p, float m) {
  const bool none = p.m == neg_inf();
  const float d = none ? 0.f : base_of(p.m) - base_of(m);
  const float r = __builtin_amdgcn_exp2f(d);
  p.s = (p.s + p.l * d) * r;
  p.l *= r;
  p.m = m;
}
__device__ __forceinline__ void merge(Part& p, Part o) {
  const float m = fmaxf(p.m, o.m);
  rebase(p, m);
  rebase(o, m);
  p.l += o.l;
  p.s += o.s;
}

template <int n>
__device__ __forceinline__ void take(Part& p, const float* f) {
  float top = f[0];
#pragma unroll
  for (int e = 1; e < n; ++e) top = fmaxf(top, f[e]);
  if (__builtin_amdgcn_ballot_w64(top > p.m)) rebase(p, fmaxf(p.m, top));
  const float b = base_of(p.m);
#pragma unroll
  for (int e = 0; e < n; ++e) {
    const float d = __builtin_fmaf(f[e], kLog2e, -b);
    const float q = __builtin_amdgcn_exp2f(d);
    p.l += q;
    p.s = __builtin_fmaf(q, fmaxf(d, -150.f), p.s);  // a logit of -inf: 0 times a finite number
  }
}

template <typename T, int kThreads, bool kTop>
__global__ __launch_bounds__(kThreads) void logprobs_kernel(LogprobArgs a) {
  constexpr int kVec = Row<T>::kVec;
  constexpr int kWaves = kThreads / 64;
  __shared__ float red[kWaves][3];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t n = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + n * a.ld;
  // logits before the first 16-byte boundary, whole vectors, the rest
  const int lead = min(int((16 - (reinterpret_cast<uintptr_t>(x) & 15)) % 16 / sizeof(T)), a.V);
  const int vecs = (a.V - lead) / kVec;
  const int rest = lead + vecs * kVec;
  const u32x4* xv = reinterpret_cast<const u32x4*>(x + lead);

  Part p{neg_inf(), 0.f, 0.f};
  constexpr int kUnroll = 4;
  int i = tid;
  for (; i + (kUnroll - 1) * kThreads < vecs; i += kUnroll * kThreads) {
    u32x4 w[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) w[u] = xv[i + u * kThreads];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float f[kVec];
      Row<T>::unpack(w[u], f);
      take<kVec>(p, f);
    }
  }
  for (; i < vecs; i += kThreads) {
    float f[kVec];
    Row<T>::unpack(xv[i], f);
    take<kVec>(p, f);
  }
  if (tid < lead) {
    const float f = float(x[tid]);
    take<1>(p, &f);
  }
  if (rest + tid < a.V) {
    const float f = float(x[rest + tid]);
    take<1>(p, &f);
  }
  const float own = p.m;  // the largest logit of this thread

#pragma unroll
  for (int s = 1; s < 64; s *= 2) {
    Part o{__shfl_xor(p.m, s), __shfl_xor(p.l, s), __shfl_xor(p.s, s)};
    merge(p, o);
  }
  if (lane == 0) {
    red[wave][0] = p.m;
    red[wave][1] = p.l;
    red[wave][2] = p.s;
  }
  __syncthreads();
  p = Part{red[0][0], red[0][1], red[0][2]};
#pragma unroll
  for (int w = 1; w < kWaves; ++w) merge(p, Part{red[w][0], red[w][1], red[w][2]});
  const bool none = p.l == 0.f;  // every logit is -inf: log probabilities of -inf, entropy 0
  const float log2l = none ? 0.f : __builtin_log2f(p.l);
  const float base = base_of(p.m);
  // log p of a logit
  auto logp_of = [&](float v) { return (__builtin_fmaf(v, kLog2e, -base) - log2l) * kLn2; };

  if (tid == 0) {
    if (a.targets) {
      const int64_t t = a.wide ? static_cast<const int64_t*>(a.targets)[n] : static_cast<const int32_t*>(a.targets)[n];
      a.logp[n] = t < 0 ? 0.f : t < a.V ? logp_of(float(x[t])) : __builtin_nanf("");
    }
    if (a.entropy) a.entropy[n] = none ? 0.f : (log2l - p.s / p.l) * kLn2;
  }
  if (!kTop) return;

  __shared__ uint32_t group[kGroups];
  __shared__ uint64_t list[kList];
  __shared__ uint32_t bound, count;
  const int k = min(a.top, a.V);
  // a thread without logits has the key 0, below that of -inf
  const bool has = tid < vecs || tid < lead || rest + tid < a.V;
  const uint32_t mine = has ? key_of(own) : 0u;
  constexpr int kPer = kThreads / kGroups;
  uint32_t g = mine;
#pragma unroll
  for (int s = 1; s < kPer; s *= 2) g = max(g, uint32_t(__shfl_xor(int(g), s)));
  if (tid % kPer == 0) group[tid / kPer] = g;
  if (tid == 0) count = 0;
  __syncthreads();
  if (tid < kGroups) {
    const uint32_t v = group[tid];
    int rank = 0;
    for (int j = 0; j < kGroups; j += 4) {
      const u32x4 o = *reinterpret_cast<const u32x4*>(&group[j]);
#pragma unroll
      for (int e = 0; e < 4; ++e) rank += o[e] > v || (o[e] == v && j + e < tid);
    }
    if (rank == k - 1) bound = v;
  }
  __syncthreads();
  const uint32_t low = bound;

  // Appends the thread's logits with keys of at least `least`; the count keeps
  // growing past the end of the list.
  auto collect = [&](uint32_t least) {
    auto push = [&](float f, int at) {
      const uint32_t key = key_of(f);
      if (key < least) return;
      const uint32_t c = atomicAdd(&count, 1u);
      if (c < kList) list[c] = uint64_t(key) << 32 | (0xffffffffu - uint32_t(at));
    };
    if (has && mine >= least) {
      for (int j = tid; j < vecs; j += kThreads) {
        float f[kVec];
        Row<T>::unpack(xv[j], f);
#pragma unroll
        for (int e = 0; e < kVec; ++e) push(f[e], lead + j * kVec + e);
      }
      if (tid < lead) push(float(x[tid]), tid);
      if (rest + tid < a.V) push(float(x[rest + tid]), rest + tid);
    }
    __syncthreads();
  };
  collect(low);
  int found = int(count);
  int64_t* ids = a.top_ids + n * a.top;
  float* lps = a.top_logp + n * a.top;
  if (found > kList) {
    __syncthreads();
    if (tid == 0) count = 0;
    __syncthreads();
    if (low != 0xffffffffu) collect(low + 1);
    found = int(count);
    if (found <= kList - 64) {
      // the lowest indices with the bound's own key fill up the k
      for (int j = tid; found < k; j += kThreads) {
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
          if (c < last && c > best) best = c;
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

template <typename T, int kThreads>
hipError_t launch(const LogprobArgs& a, int64_t N, hipStream_t s) {
  const dim3 grid = dim3(uint32_t(N));
  if (a.top > 0)
    logprobs_kernel<T, kThreads, true><<<grid, kThreads, 0, s>>>(a);
  else
    logprobs_kernel<T, kThreads, false><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_logprobs(const LogprobCall& r, hipStream_t s) {
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
  return r.fp32 ? launch<float, 1024>(a, r.N, s) : launch<_Float16, 1024>(a, r.N, s);
}

}  // namespace swm
