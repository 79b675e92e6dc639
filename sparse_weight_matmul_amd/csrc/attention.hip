// Attention of one new token per sequence over a paged key-value cache, the
// length split over workgroups and joined.
//
//   x_t = scale * q . k_t ;  p_t = e^(x_t - m) / sum_u e^(x_u - m), m = max x
//   o   = sum_t p_t v_t   ;  weight_t += sum over the query heads of a group p_t
//
// over the live tokens t of a sequence (below its length, on a page of the
// pool, not masked).  Every key and value row is used once per group of query
// heads, so the bound is the read of the live rows (4 D bytes per token and
// key-value head); the arithmetic of up to 16 query heads fits beside it on
// the matrix cores.
//
// One pass with a running maximum and sum.  A wave takes 32 tokens at a time
// and keeps everything in registers: there is no LDS in the loop, no barrier
// and no transpose.
//  - Scores: two v_mfma_f32_16x16x32_f16 chains with a key tile as A (rows =
//    tokens) and the query heads as B (columns).  Lane l of the result holds
//    rows 4(l/16)..+3 of head l%16.  The tokens of the two tiles are dealt so
//    that row 4q + r of tile i is token 8q + 4i + r: lane group q = l/16 then
//    owns tokens 8q..8q+7 of head l%16, in order.
//  - That is the B operand of the second product (k = 8(l/16) + e, column
//    l%16) as it stands, so the weights never leave their lanes.
//  - Values: lane (q, c = l%16) loads 16 bytes (dimensions 8c..8c+7) of the
//    eight tokens 8q..8q+7.  Instruction j takes dimension 8c + j of every c
//    as its 16 rows, i.e. the j-th half of each of the lane's eight loads:
//    four byte permutes per instruction instead of a transpose through LDS.
//  - Row maxima and the running rescale are per head, so per lane; only the
//    maximum over the four lane groups crosses lanes.
// The weights e^(x - m) go into the second product as two fp16 parts (value
// and remainder): one part alone would put its rounding (2^-12 relative) on
// every weight, which is as large as the output's own rounding; the matrix
// cores are idle anyway.  Scores, maxima, sums and outputs are fp32, and the
// output is rounded once.
//
// Values of tokens that are not live are replaced by zeros before the second
// product (their weight is zero, but a stale row may hold an infinity or a
// NaN), and their scores by -inf.  All row addresses are clamped into the
// pool, so a page table entry outside it reads nothing out of range: its
// tokens just are not live.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kernels.h"

namespace swm {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kTile = 32;   // tokens a wave takes at a time
constexpr int kWaves = 4;   // waves of a workgroup; they take tiles in turn
constexpr int kHeads = 16;  // query heads of a workgroup (columns of the matrix instruction)

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

struct AttnArgs {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  const int32_t *table, *lengths;
  const uint8_t* mask;
  float* weights;
  float* ml;      // [B][Hq][splits][2] maximum (in units of log2) and sum
  float* part;    // [B][Hq][splits][D] unnormalised outputs
  float* logits;  // [B][Hq][cap] scores in units of log2
  int64_t q_b, q_h, o_b, o_h;
  int64_t k_p, k_s, k_h, v_p, v_s, v_h;
  int64_t table_b, mask_b, w_p, w_h;
  int32_t B, Hq, Hkv, G, D, S, pages, cap, per_seq;
  int32_t splits, split_len;
  float scale;  // softmax scale * log2(e)
  double inv_s;  // 1 / S
};

// Page and slot of token t (t < 2^31): t / S by one fp64 product; the half
// keeps the quotient clear of rounding at whole numbers.
__device__ __forceinline__ void page_of(const AttnArgs& a, int t, int* index, int* slot) {
  const int i = int((double(t) + 0.5) * a.inv_s);
  *index = i;
  *slot = t - i * a.S;
}

// Where a token's rows are: its page, clamped into the pool, and whether the
// table names a page of the pool for it.
struct Place {
  int page, slot;
  bool ok;
};

__device__ __forceinline__ Place place(const AttnArgs& a, const int32_t* row, int t) {
  Place p;
  int i;
  page_of(a, t, &i, &p.slot);
  const int id = row[min(i, a.per_seq - 1)];
  p.ok = i < a.per_seq && id >= 0 && id < a.pages;
  p.page = p.ok ? id : 0;
  return p;
}

// Keys and values of one tile in registers.
template <int DP>
struct Tile {
  u32x4 k[2][DP / 32];
  u32x4 v[8][DP / 128 ? DP / 128 : 1];  // DP = 64: the first two words of each
};

// kSame8: a page holds a multiple of eight tokens, so eight aligned tokens
// share one.
template <int DP, bool kFull, bool kSame8>
__device__ __forceinline__ void load_tile(const AttnArgs& a, const int32_t* row, const uint16_t* kh,
                                          const uint16_t* vh, int t0, int lane, const Place& pk, const Place& pv,
                                          Tile<DP>& t) {
  const int g = lane >> 4, c = lane & 15;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int off = 4 * i + (c & 3);
    const Place p = kSame8 ? pk : place(a, row, t0 + 8 * (c >> 2) + off);
    const uint16_t* src = kh + int64_t(p.page) * a.k_p + int64_t(p.slot + (kSame8 ? off : 0)) * a.k_s;
#pragma unroll
    for (int s = 0; s < DP / 32; ++s) {
      const int d = 32 * s + 8 * g;
      t.k[i][s] = *reinterpret_cast<const u32x4*>(src + (kFull || d < a.D ? d : 0));
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const Place p = kSame8 ? pv : place(a, row, t0 + 8 * g + e);
    const uint16_t* src = vh + int64_t(p.page) * a.v_p + int64_t(p.slot + (kSame8 ? e : 0)) * a.v_s;
    if (DP == 64) {
      const int d = 4 * c;
      const u32x2 w = *reinterpret_cast<const u32x2*>(src + (kFull || d < a.D ? d : 0));
      t.v[e][0][0] = w[0];
      t.v[e][0][1] = w[1];
    } else {
#pragma unroll
      for (int u = 0; u < DP / 128; ++u) {
        const int d = 128 * u + 8 * c;
        t.v[e][u] = *reinterpret_cast<const u32x4*>(src + (kFull || d < a.D ? d : 0));
      }
    }
  }
}

// Live tokens of the lane's group: bit e for token t0 + 8 (lane/16) + e.
template <bool kSame8>
__device__ __forceinline__ uint32_t live_bits(const AttnArgs& a, const int32_t* row, const uint8_t* mask, int t,
                                              int end, const Place& pv) {
  uint32_t bits = 0;
  if (kSame8) {
    bits = pv.ok ? 0xffu : 0u;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) bits |= place(a, row, t + e).ok ? 1u << e : 0u;
  }
  const int left = end - t;
  bits &= left >= 8 ? 0xffu : left > 0 ? (1u << left) - 1 : 0u;
  if (mask) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (mask[min(t + e, a.cap - 1)] == 0) bits &= ~(1u << e);
  }
  return bits;
}

__device__ __forceinline__ float max_groups(float v) {  // over the four lane groups
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float sum_groups(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// One workgroup: one split of one sequence, up to 16 query heads of one
// key-value head.
template <int DP, bool kFull, bool kSame8>
__global__ __launch_bounds__(64 * kWaves) void attn_kernel(AttnArgs a) {
  constexpr int kJ = DP == 64 ? 4 : 8;             // halves of a value chunk
  constexpr int kU = DP / 128 ? DP / 128 : 1;      // value chunks of a lane
  extern __shared__ float smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.x, b = blockIdx.z;
  const int tiles_h = (a.G + kHeads - 1) / kHeads;
  const int hkv = blockIdx.y / tiles_h, ht = blockIdx.y % tiles_h;
  const int gn = min(kHeads, a.G - ht * kHeads);  // query heads here
  const int h0 = hkv * a.G + ht * kHeads;
  const int n = min(max(a.lengths[b], 0), a.cap);
  const int begin = split * a.split_len, end = min(begin + a.split_len, n);
  if (begin >= end && a.splits > 1) return;  // the join does not read splits past the length

  const int32_t* row = a.table + int64_t(b) * a.table_b;
  const uint8_t* mask = a.mask ? a.mask + int64_t(b) * a.mask_b : nullptr;
  const uint16_t* kh = a.k + int64_t(hkv) * a.k_h;
  const uint16_t* vh = a.v + int64_t(hkv) * a.v_h;
  const int g = lane >> 4, c = lane & 15;

  half8 q[DP / 32];
  {
    const uint16_t* src = a.q + int64_t(b) * a.q_b + int64_t(h0 + min(c, gn - 1)) * a.q_h;
#pragma unroll
    for (int s = 0; s < DP / 32; ++s) {
      const int d = 32 * s + 8 * g;
      u32x4 w = *reinterpret_cast<const u32x4*>(src + (kFull || d < a.D ? d : 0));
      if (c >= gn || (!kFull && d >= a.D)) w = u32x4{0, 0, 0, 0};
      q[s] = __builtin_bit_cast(half8, w);
    }
  }

  f32x4 o[kU][kJ];
#pragma unroll
  for (int u = 0; u < kU; ++u)
#pragma unroll
    for (int j = 0; j < kJ; ++j) o[u][j] = f32x4{0, 0, 0, 0};
  float m = neg_inf(), l = 0.f;

  float* logits = a.logits ? a.logits + (int64_t(b) * a.Hq + h0 + min(c, gn - 1)) * a.cap : nullptr;

  constexpr int kStep = kTile * kWaves;
  const int first = begin + kTile * wave;
  Tile<DP> cur;
  Place pk{}, pv{}, pk2{}, pv2{};
  uint32_t live = 0;
  if (first < end) {
    if (kSame8) {
      pk = place(a, row, first + 8 * (c >> 2));
      pv = place(a, row, first + 8 * g);
      pk2 = place(a, row, first + kStep + 8 * (c >> 2));
      pv2 = place(a, row, first + kStep + 8 * g);
    }
    load_tile<DP, kFull, kSame8>(a, row, kh, vh, first, lane, pk, pv, cur);
    live = live_bits<kSame8>(a, row, mask, first + 8 * g, end, pv);
  }
  for (int t0 = first; t0 < end; t0 += kStep) {
    // request the next tile (its pages were looked up a tile ago) and look up
    // the pages of the one after it
    Tile<DP> nxt;
    uint32_t live_n = 0;
    const bool more = t0 + kStep < end;
    if (more) {
      Place pk3{}, pv3{};
      if (kSame8) {
        pk3 = place(a, row, t0 + 2 * kStep + 8 * (c >> 2));
        pv3 = place(a, row, t0 + 2 * kStep + 8 * g);
      }
      load_tile<DP, kFull, kSame8>(a, row, kh, vh, t0 + kStep, lane, pk2, pv2, nxt);
      live_n = live_bits<kSame8>(a, row, mask, t0 + kStep + 8 * g, end, pv2);
      pk2 = pk3;
      pv2 = pv3;
    }

    f32x4 s2[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
    for (int s = 0; s < DP / 32; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        u32x4 w = cur.k[i][s];
        if (!kFull && 32 * s + 8 * g >= a.D) w = u32x4{0, 0, 0, 0};
        s2[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, w), q[s], s2[i], 0, 0, 0);
      }
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = s2[e >> 2][e & 3] * a.scale;
    if (__builtin_amdgcn_ballot_w64(live != 0xffu)) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool on = (live >> e) & 1;
        x[e] = on ? x[e] : neg_inf();
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (!on) cur.v[e][u] = u32x4{0, 0, 0, 0};
      }
    }
    if (logits && c < gn) {
      const int t = t0 + 8 * g;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (t + e < end) logits[t + e] = x[e];
    }
    float mx = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) mx = fmaxf(mx, x[e]);
    mx = fmaxf(m, max_groups(mx));
    const float base = mx == neg_inf() ? 0.f : mx;  // nothing live so far: weights of 2^-inf
    if (__builtin_amdgcn_ballot_w64(mx != m)) {
      const float r = __builtin_amdgcn_exp2f(m - base);
      l *= r;
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int j = 0; j < kJ; ++j) o[u][j] *= r;
      m = mx;
    }
    half8 hi, lo;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float p = __builtin_amdgcn_exp2f(x[e] - base);
      l += p;
      hi[e] = _Float16(p);
      lo[e] = _Float16(p - float(hi[e]));
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = __builtin_amdgcn_perm(cur.v[2 * e + 1][u][j / 2], cur.v[2 * e][u][j / 2],
                                       j & 1 ? 0x07060302u : 0x05040100u);
        const half8 vt = __builtin_bit_cast(half8, w);
        o[u][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vt, hi, o[u][j], 0, 0, 0);
        o[u][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vt, lo, o[u][j], 0, 0, 0);
      }
    cur = nxt;
    live = live_n;
  }
  l = sum_groups(l);

  // Join the waves: maxima and sums, then the outputs (dimension 8(4g + r) + j
  // of head c is element r of o[..][j]).
  float* sm_m = smem;
  float* sm_l = smem + kWaves * kHeads;
  float* sm_o = smem + 2 * kWaves * kHeads;
  if (g == 0) {
    sm_m[wave * kHeads + c] = m;
    sm_l[wave * kHeads + c] = l;
  }
  if (c < gn) {
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          sm_o[(wave * gn + c) * DP + 128 * u + kJ * (4 * g + r) + j] = o[u][j][r];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < gn * DP; i += 64 * kWaves) {
    const int h = i / DP, d = i % DP;
    float mm = neg_inf();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, sm_m[w * kHeads + h]);
    const float base = mm == neg_inf() ? 0.f : mm;
    float sum = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float r = __builtin_amdgcn_exp2f(sm_m[w * kHeads + h] - base);
      sum += r * sm_l[w * kHeads + h];
      acc += r * sm_o[(w * gn + h) * DP + d];
    }
    const int64_t bh = int64_t(b) * a.Hq + h0 + h;
    if (d == 0 && a.ml) {
      a.ml[(bh * a.splits + split) * 2] = mm;
      a.ml[(bh * a.splits + split) * 2 + 1] = sum;
    }
    if (d >= a.D) continue;
    if (a.splits > 1)
      a.part[(bh * a.splits + split) * a.D + d] = acc;
    else
      a.out[int64_t(b) * a.o_b + int64_t(h0 + h) * a.o_h + d] =
          __builtin_bit_cast(uint16_t, _Float16(sum == 0.f ? 0.f : acc / sum));
  }
}

constexpr int kJoinThreads = 256;
constexpr int kWeightTokens = 1024;  // tokens whose weights one workgroup adds
constexpr int kMaxSplits = 1024;

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int s = 1; s < 64; s *= 2) v = fmaxf(v, __shfl_xor(v, s));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int s = 1; s < 64; s *= 2) v += __shfl_xor(v, s);
  return v;
}

// Maximum and sum of one head over its splits (the whole wave gets both).
__device__ __forceinline__ void head_ml(const float* ml, int valid, int lane, float* m, float* l) {
  float mm = neg_inf();
  for (int s = lane; s < valid; s += 64) mm = fmaxf(mm, ml[2 * s]);
  mm = wave_max(mm);
  const float base = mm == neg_inf() ? 0.f : mm;
  float ll = 0.f;
  for (int s = lane; s < valid; s += 64) ll += __builtin_amdgcn_exp2f(ml[2 * s] - base) * ml[2 * s + 1];
  *m = mm;
  *l = wave_sum(ll);
}

// After the splits: the first `joins` workgroups add up the splits of one
// query head each; the others add the attention weights of kWeightTokens
// tokens of a sequence and key-value head to the accumulator.  The adds are
// atomic because sequences may share a page.
__global__ __launch_bounds__(kJoinThreads) void attn_join_kernel(AttnArgs a, int joins) {
  __shared__ float sc[kMaxSplits];
  __shared__ float red[kJoinThreads];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (int(blockIdx.x) < joins) {
    const int b = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq;
    const int n = min(max(a.lengths[b], 0), a.cap);
    const int valid = (n + a.split_len - 1) / a.split_len;
    const int64_t bh = int64_t(b) * a.Hq + h;
    const float* ml = a.ml + bh * a.splits * 2;
    float m, l;
    head_ml(ml, valid, lane, &m, &l);
    const float base = m == neg_inf() ? 0.f : m;
    for (int s = threadIdx.x; s < valid; s += kJoinThreads) sc[s] = __builtin_amdgcn_exp2f(ml[2 * s] - base);
    __syncthreads();
    // a power of two of threads per split row, the rest in parts over the splits
    int dp = 64;
    while (dp < a.D) dp *= 2;
    const int parts = kJoinThreads / dp, part = threadIdx.x / dp, d = threadIdx.x % dp;
    float acc = 0.f;
    if (d < a.D) {
      const float* src = a.part + bh * a.splits * a.D + d;
      for (int s = part; s < valid; s += parts) acc += sc[s] * src[int64_t(s) * a.D];
    }
    red[threadIdx.x] = acc;
    __syncthreads();
    if (part == 0 && d < a.D) {
      for (int p = 1; p < parts; ++p) acc += red[p * dp + d];
      a.out[int64_t(b) * a.o_b + int64_t(h) * a.o_h + d] =
          __builtin_bit_cast(uint16_t, _Float16(l == 0.f ? 0.f : acc / l));
    }
    return;
  }
  const int chunks = (a.cap + kWeightTokens - 1) / kWeightTokens;
  int i = blockIdx.x - joins;
  const int chunk = i % chunks;
  i /= chunks;
  const int hkv = i % a.Hkv, b = i / a.Hkv;
  const int n = min(max(a.lengths[b], 0), a.cap);
  const int t0 = chunk * kWeightTokens, t1 = min(t0 + kWeightTokens, n);
  if (t0 >= t1) return;
  const int valid = (n + a.split_len - 1) / a.split_len;
  float w[kWeightTokens / kJoinThreads] = {};
  // kMaxSplits / 2 heads' maxima and reciprocal sums at a time
  for (int g0 = 0; g0 < a.G; g0 += kMaxSplits / 2) {
    const int gn = min(a.G - g0, kMaxSplits / 2);
    for (int g = wave; g < gn; g += kJoinThreads / 64) {
      const int64_t bh = int64_t(b) * a.Hq + hkv * a.G + g0 + g;
      float m, l;
      head_ml(a.ml + bh * a.splits * 2, valid, lane, &m, &l);
      if (lane == 0) {
        sc[2 * g] = m == neg_inf() ? 0.f : m;
        sc[2 * g + 1] = l == 0.f ? 0.f : 1.f / l;
      }
    }
    __syncthreads();
    for (int g = 0; g < gn; ++g) {
      const float* x = a.logits + (int64_t(b) * a.Hq + hkv * a.G + g0 + g) * a.cap;
#pragma unroll
      for (int e = 0; e < kWeightTokens / kJoinThreads; ++e) {
        const int t = t0 + e * kJoinThreads + threadIdx.x;
        if (t < t1) w[e] += __builtin_amdgcn_exp2f(x[t] - sc[2 * g]) * sc[2 * g + 1];
      }
    }
    __syncthreads();
  }
  const int32_t* row = a.table + int64_t(b) * a.table_b;
#pragma unroll
  for (int e = 0; e < kWeightTokens / kJoinThreads; ++e) {
    const int t = t0 + e * kJoinThreads + threadIdx.x;
    if (t >= t1 || w[e] == 0.f) continue;
    const Place p = place(a, row, t);
    if (p.ok) unsafeAtomicAdd(a.weights + int64_t(p.page) * a.w_p + int64_t(hkv) * a.w_h + p.slot, w[e]);
  }
}

template <int DP, bool kFull>
hipError_t launch_main(const AttnArgs& a, bool same8, dim3 grid, size_t lds, hipStream_t s) {
  if (same8)
    attn_kernel<DP, kFull, true><<<grid, 64 * kWaves, lds, s>>>(a);
  else
    attn_kernel<DP, kFull, false><<<grid, 64 * kWaves, lds, s>>>(a);
  return hipGetLastError();
}

template <int DP>
hipError_t launch_dim(const AttnArgs& a, bool same8, dim3 grid, size_t lds, hipStream_t s) {
  return a.D == DP ? launch_main<DP, true>(a, same8, grid, lds, s) : launch_main<DP, false>(a, same8, grid, lds, s);
}

}  // namespace

// The split of the length.  A workgroup's four waves take 128 tokens at a
// time.
AttnPlan plan_attention(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t cap, bool weights, int num_cus) {
  AttnPlan p;
  const int64_t G = Hq / Hkv;
  const int64_t units = B * Hkv * ((G + kHeads - 1) / kHeads);
  const int64_t step = int64_t(kTile) * kWaves;
  const int64_t steps = std::max<int64_t>(1, (cap + step - 1) / step);
  int64_t splits = 1;
  const int64_t want = 4 * int64_t(num_cus);
  if (units < want) splits = std::min<int64_t>({(want + units - 1) / units, (steps + 1) / 2, kMaxSplits});
  splits = std::max<int64_t>(splits, 1);
  const int64_t per = (steps + splits - 1) / splits;
  p.split_len = int(std::min<int64_t>(per * step, (int64_t(1) << 31) - step));
  p.splits = int((cap + p.split_len - 1) / p.split_len);
  if (p.splits < 1) p.splits = 1;
  const size_t rows = size_t(B) * size_t(Hq);
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  p.bytes = 0;
  if (p.splits > 1 || weights) p.bytes += up(rows * p.splits * 2 * 4);
  p.off_part = p.bytes;
  if (p.splits > 1) p.bytes += up(rows * p.splits * size_t(D) * 4);
  p.off_logits = p.bytes;
  if (weights) p.bytes += up(rows * size_t(cap) * 4);
  return p;
}

hipError_t launch_attention(const KvView& c, const AttnCall& r, const AttnPlan& p, void* ws, hipStream_t s) {
  AttnArgs a{};
  a.q = r.q;
  a.out = r.out;
  a.q_b = r.q_b;
  a.q_h = r.q_h;
  a.o_b = r.o_b;
  a.o_h = r.o_h;
  a.k = c.k;
  a.v = c.v;
  a.k_p = c.k_p;
  a.k_s = c.k_s;
  a.k_h = c.k_h;
  a.v_p = c.v_p;
  a.v_s = c.v_s;
  a.v_h = c.v_h;
  a.table = c.table;
  a.table_b = c.table_b;
  a.lengths = c.lengths;
  a.mask = r.mask;
  a.mask_b = r.mask_b;
  a.weights = r.weights;
  a.w_p = r.w_p;
  a.w_h = r.w_h;
  a.B = int(c.B);
  a.Hq = int(r.Hq);
  a.Hkv = int(c.Hkv);
  a.G = int(r.Hq / c.Hkv);
  a.D = int(c.D);
  a.S = int(c.S);
  a.pages = int(c.pages);
  a.per_seq = int(c.per_seq);
  a.cap = int(c.per_seq * c.S);
  a.splits = p.splits;
  a.split_len = p.split_len;
  a.scale = r.scale * 1.44269504088896340736f;
  a.inv_s = 1.0 / double(c.S);
  uint8_t* w = static_cast<uint8_t*>(ws);
  const bool second = p.splits > 1 || r.weights;
  if (second) a.ml = reinterpret_cast<float*>(w);
  if (p.splits > 1) a.part = reinterpret_cast<float*>(w + p.off_part);
  if (r.weights) a.logits = reinterpret_cast<float*>(w + p.off_logits);

  const int tiles_h = (a.G + kHeads - 1) / kHeads, gn = std::min(a.G, kHeads);
  const int dp = a.D <= 64 ? 64 : a.D <= 128 ? 128 : 256;
  const size_t lds = 4 * (2 * kWaves * kHeads + size_t(kWaves) * gn * dp);
  const dim3 grid(a.splits, a.Hkv * tiles_h, a.B);
  const bool same8 = a.S % 8 == 0;
  hipError_t e = dp == 64    ? launch_dim<64>(a, same8, grid, lds, s)
                 : dp == 128 ? launch_dim<128>(a, same8, grid, lds, s)
                             : launch_dim<256>(a, same8, grid, lds, s);
  if (e != hipSuccess || !second) return e;
  const int64_t joins = p.splits > 1 ? int64_t(a.B) * a.Hq : 0;
  const int64_t adds = r.weights ? int64_t(a.B) * a.Hkv * ((a.cap + kWeightTokens - 1) / kWeightTokens) : 0;
  if (joins + adds == 0) return hipSuccess;
  attn_join_kernel<<<dim3(uint32_t(joins + adds)), kJoinThreads, 0, s>>>(a, int(joins));
  return hipGetLastError();
}

}  // namespace swm
