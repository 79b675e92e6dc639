// Attention of one new token per sequence over a paged key-value cache, long
// sequences cut into pieces that a second launch joins.
//
//   x_t = scale * q . k_t ;  p_t = e^(x_t - m) / sum_u e^(x_u - m), m = max x
//   o   = sum_t p_t v_t   ;  weight_t += sum over the query heads of a group p_t
//
// over the live tokens t of a sequence (below its length, on a page of the
// pool, not masked).  Every key and value row is used once per group of query
// heads, so the bound is the read of the live rows (4 D bytes per token and
// key-value head); the arithmetic of up to 16 query heads fits beside it on
// the matrix cores.  Measured: 2 x 131072 tokens, 64 heads on 8: 1.07 GB in 167
// us, 6.4 TB/s; 16 ragged x 4096, 32 heads, weights added: 554 MB in 88 us (6.3
// TB/s) where a part of the cache is in the last-level cache, 99 otherwise.
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
// cores are idle anyway.  They go in times 2^15, the most that fits: the parts
// of a weight are then off by 2^-23 of it down to weights of 2^-17, by 2^-40
// below.  Without the factor that would be 2^-25, and a hundred thousand tokens
// some 17 nats below one of value zero (an attention sink) would lose their
// share of the output while the sum counts it.  The sum adds a tile's weights up
// before it takes them, for the same reason.  Scores, maxima, sums and outputs
// are fp32, and the output is rounded once.
//
// Values of tokens that are not live are replaced by zeros before the second
// product (their weight is zero, but a stale row may hold an infinity or a
// NaN), and their scores by -inf.  All row addresses are clamped into the
// pool, so a page table entry outside it reads nothing out of range: its
// tokens just are not live.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kernels.h"
#include "paging.h"
#include "wave.h"

namespace swm {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kTile = 32;   // tokens a wave takes at a time
constexpr int kWaves = 4;   // waves of a workgroup; they take tiles in turn
constexpr int kMaxSorted = 128;  // sequences whose lengths a wave holds, two a lane
constexpr int kHeads = 16;  // query heads of a workgroup (columns of the matrix instruction)
constexpr float kUp = 32768.f;  // of the weights in the second product

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

struct AttnArgs {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  const int32_t *table, *lengths;
  const uint8_t* mask;
  float* weights;
  int32_t* plan;  // tokens of a piece, then the first piece of each sequence
  float* ml;      // [piece][query head of it][2] maximum (in units of log2) and sum
  float* part;    // [piece][query head of it][D] unnormalised outputs
  float* logits;  // [B][Hq][lrow] scores in units of log2
  int64_t q_b, q_h, o_b, o_h;
  int64_t k_p, k_s, k_h, v_p, v_s, v_h;
  int64_t table_b, mask_b, w_p, w_h;
  int32_t B, Hq, Hkv, G, D, S, pages, cap, per_seq;
  int32_t room;  // pieces of all sequences at most; 0: every sequence is one
  int32_t lrow, order, cus, adds;
  int32_t own_weights;  // a whole sequence's workgroup adds the weights itself, its scores in LDS
  float scale;  // softmax scale * log2(e)
  PageDiv div;    // by S
  PageDiv per_b;  // by the units of a sequence: key-value heads x groups of 16 query heads
  PageDiv per_hq, per_g;  // by the query heads, and those of a key-value head
  int32_t units;  // of all sequences
};

// Where a token's rows are: its page, clamped into the pool, and whether the
// table names a page of the pool for it.
struct Place {
  int page, slot;
  bool ok;
};

__device__ __forceinline__ Place place(const AttnArgs& a, const int32_t* row, int t) {
  Place p;
  const int i = page_index(a.div, t);
  p.slot = t - i * a.S;
  const int id = row[min(i, a.per_seq - 1)];
  p.ok = i < a.per_seq && id >= 0 && id < a.pages;
  p.page = p.ok ? id : 0;
  return p;
}

// The lane's part of a tile's keys: of each of the two key tiles one row, 16
// bytes of every 64.  kSame8: a page holds a multiple of eight tokens, so eight
// aligned tokens share one (16 ragged x 4096, 32 heads, weights 100 us, 136 with
// a page looked up for every token).
template <int DP, bool kFull, bool kSame8>
__device__ __forceinline__ void load_keys(const AttnArgs& a, const int32_t* row, const uint16_t* kh, int t0,
                                          int lane, const Place& pk, u32x4 (&k)[2][DP / 32]) {
  const int g = lane >> 4, c = lane & 15;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int off = 4 * i + (c & 3);
    const Place p = kSame8 ? pk : place(a, row, t0 + 8 * (c >> 2) + off);
    const uint16_t* src = kh + int64_t(p.page) * a.k_p + int64_t(p.slot + (kSame8 ? off : 0)) * a.k_s;
#pragma unroll
    for (int s = 0; s < DP / 32; ++s) {
      const int d = 32 * s + 8 * g;
      k[i][s] = *reinterpret_cast<const u32x4*>(src + (kFull || d < a.D ? d : 0));
    }
  }
}

// The lane's part of a tile's values: its chunk of eight tokens' rows (DP =
// 64: four halves, in the first two words).
template <int DP, bool kFull, bool kSame8>
__device__ __forceinline__ void load_values(const AttnArgs& a, const int32_t* row, const uint16_t* vh, int t0,
                                            int lane, const Place& pv, u32x4 (&v)[8][DP / 128 ? DP / 128 : 1]) {
  const int g = lane >> 4, c = lane & 15;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const Place p = kSame8 ? pv : place(a, row, t0 + 8 * g + e);
    const uint16_t* src = vh + int64_t(p.page) * a.v_p + int64_t(p.slot + (kSame8 ? e : 0)) * a.v_s;
    if (DP == 64) {
      const int d = 4 * c;
      const u32x2 w = *reinterpret_cast<const u32x2*>(src + (kFull || d < a.D ? d : 0));
      v[e][0][0] = w[0];
      v[e][0][1] = w[1];
    } else {
#pragma unroll
      for (int u = 0; u < DP / 128; ++u) {
        const int d = 128 * u + 8 * c;
        v[e][u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(src + (kFull || d < a.D ? d : 0)));
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

// Maximum and sum over the four lane groups.  The swap instructions exchange
// odd and even rows of 16 lanes (halves of 32) of two registers: given the
// same value twice, the two results hold both partners' values.
__device__ __forceinline__ void partners16(float v, float* a, float* b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  *a = __uint_as_float(r[0]);
  *b = __uint_as_float(r[1]);
}
__device__ __forceinline__ void partners32(float v, float* a, float* b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  *a = __uint_as_float(r[0]);
  *b = __uint_as_float(r[1]);
}
__device__ __forceinline__ float max_groups(float v) {
  float a, b;
  partners16(v, &a, &b);
  partners32(fmaxf(a, b), &a, &b);
  return fmaxf(a, b);
}
__device__ __forceinline__ float sum_groups(float v) {
  float a, b;
  partners16(v, &a, &b);
  partners32(a + b, &a, &b);
  return a + b;
}

// Tokens t, t + 64, t + 128 and t + 192: a wave's 64 lanes hold consecutive
// slots, 64 a word.  Their places (of those from n on, the last one's), and the
// adding of their weights to the accumulator, atomic because sequences may share
// a page.
__device__ __forceinline__ void four_places(const AttnArgs& a, const int32_t* row, int t, int n, Place (&p)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) p[e] = place(a, row, min(t + 64 * e, n - 1));
}
__device__ __forceinline__ void add_weights(const AttnArgs& a, const Place (&p)[4], int hkv, int t, int n,
                                            const f32x4& w) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (t + 64 * e < n && w[e] != 0.f && p[e].ok)
      unsafeAtomicAdd(a.weights + int64_t(p[e].page) * a.w_p + int64_t(hkv) * a.w_h + p[e].slot, w[e]);
}

// A head's weight of a token with score x.  A token that is not live has none,
// also where the head's sum is NaN (a live key or the query holds one).
__device__ __forceinline__ float weight_of(float x, float base, float inv) {
  const float p = __builtin_amdgcn_exp2f(x - base) * inv;
  return x == neg_inf() ? 0.f : p;
}

// Lengths of sequences 2 lane and 2 lane + 1 (0 past the batch), in tokens.
__device__ __forceinline__ void two_lengths(const AttnArgs& a, int lane, int* n0, int* n1) {
  const int x0 = a.lengths[min(2 * lane, a.B - 1)], x1 = a.lengths[min(2 * lane + 1, a.B - 1)];
  *n0 = 2 * lane < a.B ? min(max(x0, 0), a.cap) : 0;
  *n1 = 2 * lane + 1 < a.B ? min(max(x1, 0), a.cap) : 0;
}

// The pieces that the sequences of a batch are cut into, by their lengths: `len`
// tokens each, the fewest steps with which they are a.room at most, or every
// sequence whole if that ends no later.  Sequence 2 lane owns pieces first0 ..
// first1 - 1, the next one first1 .. last1 - 1.
struct Plan {
  int n0, n1, len, first0, first1, last1;
};

// s / q rounded up, inv = 1 / q to fp32's precision: the quotient of s < 2^31 is
// off by two at most (a division of whole numbers takes three times as long).
__device__ __forceinline__ uint32_t ceil_div(uint32_t s, uint32_t q, float inv) {
  const uint32_t t = uint32_t(float(s) * inv);
  const int64_t r = int64_t(s) - int64_t(t) * q;
  return t + (r > 0) + (r > q) - (r <= -int64_t(q)) - (r <= -2 * int64_t(q));
}
__device__ __forceinline__ Plan make_plan(const AttnArgs& a, int lane) {
  Plan p;
  two_lengths(a, lane, &p.n0, &p.n1);
  constexpr uint32_t kStep = kTile * kWaves;
  const uint32_t s0 = (uint32_t(p.n0) + kStep - 1) / kStep, s1 = (uint32_t(p.n1) + kStep - 1) / kStep;
  const uint32_t total = wave_sum(s0 + s1), room = a.room;
  uint32_t c0, c1;  // pieces of either sequence
  auto cut = [&](uint32_t q) {
    const float inv = __builtin_amdgcn_rcpf(float(q));
    c0 = ceil_div(s0, q, inv);
    c1 = ceil_div(s1, q, inv);
    return wave_sum(c0 + c1);
  };
  uint32_t q = max((total + room - 1) / room, 2u);
  uint32_t all = cut(q);
  if (all > room) {
    // every sequence rounds up by less than one piece: this many steps fit; the
    // least that do, to a sixteenth
    uint32_t low = q;
    q = (total + room - a.B - 1) / (room - a.B);
    while (q - low > max(low / 16, 1u)) {
      const uint32_t mid = low + (q - low) / 2;
      if (cut(mid) > room)
        low = mid;
      else
        q = mid;
    }
    all = cut(q);
  }
  if (2 * a.units > a.cus) {
    // rounds over the CUs times the steps of one
    const uint32_t most = uint32_t(wave_max(int(max(s0, s1)))), cus = a.cus, rows = uint32_t(a.units) / a.B;
    if ((a.units + cus - 1) / cus * most <= (all * rows + cus - 1) / cus * q) {
      q = max(most, q);
      cut(q);
    }
  }
  const uint32_t upto = scan_wave(c0 + c1);
  p.len = int(q * kStep);
  p.last1 = int(upto);
  p.first1 = int(upto - c1);
  p.first0 = int(upto - c1 - c0);
  return p;
}

// The workgroups in the order of their work, the longest first in the first
// round over the CUs, the shortest first in the second and so on: a CU's
// workgroups then add up to about the same length.  Returns the unit within
// sequence *b.
__device__ __forceinline__ int sorted_unit(const AttnArgs& a, int lane, int per_b, int* b) {
  int n0, n1;
  two_lengths(a, lane, &n0, &n1);
  constexpr uint32_t kStep = kTile * kWaves;
  // unique keys: steps, then the lower sequence; those past the batch have none below them
  auto key = [&](int n, int i) {
    return i < a.B ? (uint32_t(n) + kStep - 1) / kStep << 7 | uint32_t(127 - i) : 0u;
  };
  const uint32_t k0 = key(n0, 2 * lane), k1 = key(n1, 2 * lane + 1);
  int r0 = 0, r1 = 0;
  for (int l = 0; l < (a.B + 1) / 2; ++l) {
    const uint32_t x = __builtin_amdgcn_readlane(k0, l), z = __builtin_amdgcn_readlane(k1, l);
    r0 += int(x > k0) + int(z > k0);
    r1 += int(x > k1) + int(z > k1);
  }
  const int i = blockIdx.x, round = i / a.cus;
  const int s = round & 1 ? round * a.cus + min((round + 1) * a.cus, a.units) - 1 - i : i;
  const int rank = page_index(a.per_b, s);
  const uint64_t in0 = __builtin_amdgcn_ballot_w64(2 * lane < a.B && r0 == rank);
  const uint64_t in1 = __builtin_amdgcn_ballot_w64(2 * lane + 1 < a.B && r1 == rank);
  *b = in0 ? 2 * __builtin_ctzll(in0) : 2 * __builtin_ctzll(in1) + 1;
  return s - rank * per_b;
}

// One workgroup: a sequence or a piece of one, up to 16 query heads of one
// key-value head.
template <int DP, bool kFull, bool kSame8>
__global__ __launch_bounds__(64 * kWaves, DP == 256 ? 1 : 3) void attn_kernel(AttnArgs a) {
  constexpr int kJ = DP == 64 ? 4 : 8;             // halves of a value chunk
  constexpr int kU = DP / 128 ? DP / 128 : 1;      // value chunks of a lane
  extern __shared__ float smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles_h = (a.G + kHeads - 1) / kHeads, per_b = a.Hkv * tiles_h;
  int b, y, n, begin = 0, end;
  int piece = blockIdx.x;  // where its sums go
  if (a.room > 0) {
    const Plan p = make_plan(a, lane);
    if (blockIdx.x == 0 && wave == 0) {
      if (lane == 0) a.plan[0] = p.len;
      if (2 * lane < a.B) a.plan[1 + 2 * lane] = p.first0;
      if (2 * lane + 1 < a.B) a.plan[2 + 2 * lane] = p.first1;
    }
    const int cut = page_index(a.per_b, piece);  // the batch's cut-th piece of a row of units
    y = piece - cut * per_b;
    const uint64_t in = __builtin_amdgcn_ballot_w64(cut >= p.first0 && cut < p.last1);
    if (in == 0) return;  // more workgroups than pieces
    const int l = __builtin_ctzll(in);
    const bool odd = cut >= __builtin_amdgcn_readlane(p.first1, l);
    b = 2 * l + odd;
    n = __builtin_amdgcn_readlane(odd ? p.n1 : p.n0, l);
    begin = (cut - __builtin_amdgcn_readlane(odd ? p.first1 : p.first0, l)) * p.len;
    end = n - begin < p.len ? n : begin + p.len;
  } else {
    const int unit = a.order ? sorted_unit(a, lane, per_b, &b) : piece;
    if (!a.order) b = page_index(a.per_b, unit);
    y = a.order ? unit : unit - b * per_b;
    piece = b * per_b + y;
    n = min(max(a.lengths[b], 0), a.cap);
    end = n;
  }
  b = __builtin_amdgcn_readfirstlane(b);
  y = __builtin_amdgcn_readfirstlane(y);
  begin = __builtin_amdgcn_readfirstlane(begin);
  end = __builtin_amdgcn_readfirstlane(end);
  piece = __builtin_amdgcn_readfirstlane(piece);
  const int hkv = tiles_h == 1 ? y : y / tiles_h, ht = y - hkv * tiles_h;
  const int gn = min(kHeads, a.G - ht * kHeads);  // query heads here
  const int h0 = hkv * a.G + ht * kHeads;
  const int first = begin + kTile * wave;
  const int32_t* row = a.table + int64_t(b) * a.table_b;
  const uint8_t* mask = a.mask ? a.mask + int64_t(b) * a.mask_b : nullptr;
  const uint16_t* kh = a.k + int64_t(hkv) * a.k_h;
  const uint16_t* vh = a.v + int64_t(hkv) * a.v_h;
  const int g = lane >> 4, c = lane & 15;

  // The query and the first pages are requested together, the length too where
  // nothing depends on it: each waited for in turn would add its latency to the
  // shortest calls.
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
  Place pk{}, pv{};
  if (kSame8 && a.per_seq > 0) {
    pk = place(a, row, first + 8 * (c >> 2));
    pv = place(a, row, first + 8 * g);
    asm volatile("" ::"v"(pk.page), "v"(pv.page), "v"(q[0]));  // not moved past the branch
  }

  f32x4 o[kU][kJ];
#pragma unroll
  for (int u = 0; u < kU; ++u)
#pragma unroll
    for (int j = 0; j < kJ; ++j) o[u][j] = f32x4{0, 0, 0, 0};
  float m = neg_inf(), l = 0.f;

  float* sm_x = smem + 2 * kWaves * kHeads + kWaves * gn * (DP + 4);  // own_weights: scores [gn][lrow]
  float* logits = a.logits ? a.logits + (int64_t(b) * a.Hq + h0 + min(c, gn - 1)) * a.lrow : nullptr;

  constexpr int kStep = kTile * kWaves;
  u32x4 k[2][DP / 32], v[8][kU];
  uint32_t live = 0;
  if (first < end) {
    load_keys<DP, kFull, kSame8>(a, row, kh, first, lane, pk, k);
    load_values<DP, kFull, kSame8>(a, row, vh, first, lane, pv, v);
    live = live_bits<kSame8>(a, row, mask, first + 8 * g, end, pv);
    if (kSame8) {
      pk = place(a, row, first + kStep + 8 * (c >> 2));
      pv = place(a, row, first + kStep + 8 * g);
    }
  }
  for (int t0 = first; t0 < end; t0 += kStep) {
    const bool more = t0 + kStep < end;
    f32x4 s2[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
    for (int s = 0; s < DP / 32; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        u32x4 w = k[i][s];
        if (!kFull && 32 * s + 8 * g >= a.D) w = u32x4{0, 0, 0, 0};
        s2[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, w), q[s], s2[i], 0, 0, 0);
      }
    // the keys' registers are free: the next tile's keys
    if (more) load_keys<DP, kFull, kSame8>(a, row, kh, t0 + kStep, lane, pk, k);
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
          if (!on) v[e][u] = u32x4{0, 0, 0, 0};
      }
    }
    if (a.own_weights && c < gn) {
      f32x4* dst = reinterpret_cast<f32x4*>(sm_x + c * a.lrow + t0 + 8 * g);
      dst[0] = f32x4{x[0], x[1], x[2], x[3]};
      dst[1] = f32x4{x[4], x[5], x[6], x[7]};
    } else if (logits && c < gn) {  // rows are padded to whole tiles
      f32x4* dst = reinterpret_cast<f32x4*>(logits + t0 + 8 * g);
      dst[0] = f32x4{x[0], x[1], x[2], x[3]};
      dst[1] = f32x4{x[4], x[5], x[6], x[7]};
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
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float p = __builtin_amdgcn_exp2f(x[e] - base);
      sum += p;
      hi[e] = _Float16(p * kUp);
      lo[e] = _Float16(p * kUp - float(hi[e]));
    }
    l += sum;
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = __builtin_amdgcn_perm(v[2 * e + 1][u][j / 2], v[2 * e][u][j / 2],
                                       j & 1 ? 0x07060302u : 0x05040100u);
        const half8 vt = __builtin_bit_cast(half8, w);
        o[u][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vt, hi, o[u][j], 0, 0, 0);
        o[u][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vt, lo, o[u][j], 0, 0, 0);
      }
    if (more) {  // the next tile's values, and the pages of the tile after it
      const Place now = pv;
      const uint32_t bits = live_bits<kSame8>(a, row, mask, t0 + kStep + 8 * g, end, now);
      if (kSame8) {
        pk = place(a, row, t0 + 2 * kStep + 8 * (c >> 2));
        pv = place(a, row, t0 + 2 * kStep + 8 * g);
      }
      load_values<DP, kFull, kSame8>(a, row, vh, t0 + kStep, lane, now, v);
      live = bits;
    }
  }
  l = sum_groups(l);

  // Join the waves: maxima and sums, then the outputs (dimension 8(4g + r) + j
  // of head c is element r of o[..][j]), four dimensions a thread.
  constexpr int kRow = DP + 4;  // floats per row, off the bank stride
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
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int j = 0; j < kJ; j += 4)
          *reinterpret_cast<f32x4*>(&sm_o[(wave * gn + c) * kRow + 128 * u + kJ * (4 * g + r) + j]) =
              f32x4{o[u][j][r], o[u][j + 1][r], o[u][j + 2][r], o[u][j + 3][r]};
  }
  __syncthreads();
  for (int i = threadIdx.x; i < gn * (DP / 4); i += 64 * kWaves) {
    const int h = i / (DP / 4), d = i % (DP / 4) * 4;
    float mm = neg_inf();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, sm_m[w * kHeads + h]);
    const float base = mm == neg_inf() ? 0.f : mm;
    float sum = 0.f;
    f32x4 acc = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float r = __builtin_amdgcn_exp2f(sm_m[w * kHeads + h] - base);
      sum += r * sm_l[w * kHeads + h];
      acc += r * *reinterpret_cast<const f32x4*>(&sm_o[(w * gn + h) * kRow + d]);
    }
    acc *= 1.f / kUp;
    const int64_t at = int64_t(piece) * min(a.G, kHeads) + h;
    if (d == 0 && a.ml) {
      a.ml[at * 2] = mm;
      a.ml[at * 2 + 1] = sum;
    }
    if (d >= a.D) continue;  // D is a multiple of 8
    if (a.room > 0) {
      *reinterpret_cast<f32x4*>(&a.part[at * a.D + d]) = acc;
    } else {
      uint16_t* dst = a.out + int64_t(b) * a.o_b + int64_t(h0 + h) * a.o_h + d;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        dst[e] = __builtin_bit_cast(uint16_t, _Float16(sum == 0.f ? 0.f : acc[e] / sum));
    }
  }
  if (!a.own_weights) return;
  // Base and reciprocal sum of each head where its first wave's were, then
  // four tokens a thread.
  __syncthreads();
  float base = 0.f, inv = 0.f;
  if (threadIdx.x < gn) {
    float mm = neg_inf(), sum = 0.f;
    for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, sm_m[w * kHeads + threadIdx.x]);
    base = mm == neg_inf() ? 0.f : mm;
    for (int w = 0; w < kWaves; ++w)
      sum += __builtin_amdgcn_exp2f(sm_m[w * kHeads + threadIdx.x] - base) * sm_l[w * kHeads + threadIdx.x];
    inv = sum == 0.f ? 0.f : 1.f / sum;
  }
  __syncthreads();
  if (threadIdx.x < gn) {
    sm_m[threadIdx.x] = base;
    sm_l[threadIdx.x] = inv;
  }
  __syncthreads();
  for (int t = 256 * wave + lane; t < n; t += 256 * kWaves) {
    Place p[4];
    four_places(a, row, t, n, p);
    f32x4 w = {0, 0, 0, 0};
    for (int h = 0; h < gn; ++h) {
      const float* x = sm_x + h * a.lrow;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] += weight_of(x[min(t + 64 * e, n - 1)], sm_m[h], sm_l[h]);
    }
    add_weights(a, p, hkv, t, n, w);
  }
}

// The pieces of a sequence of n tokens: how many, and where the sums of the
// first one are for query head h of the sequence; the next piece's are `step`
// entries on.
struct Pieces {
  int count;
  int64_t at, step;
};
__device__ __forceinline__ Pieces pieces_of(const AttnArgs& a, int b, int n, int h) {
  const int hs = min(a.G, kHeads), tiles_h = (a.G + kHeads - 1) / kHeads, per_b = a.Hkv * tiles_h;
  const int hkv = page_index(a.per_g, h), g = h - hkv * a.G, ht = g / kHeads;
  const int first = a.room > 0 ? a.plan[1 + b] : b;
  Pieces p;
  p.count = a.room > 0 ? int((uint32_t(n) + uint32_t(a.plan[0]) - 1) / uint32_t(a.plan[0])) : n > 0;
  p.step = int64_t(per_b) * hs;
  p.at = (int64_t(first) * per_b + hkv * tiles_h + ht) * hs + g - ht * kHeads;
  return p;
}

constexpr int kJoinThreads = 256;
constexpr int kWeightTokens = 4 * kJoinThreads;  // tokens whose weights one workgroup adds at a time
constexpr int kMaxPieces = 1024;  // of a batch, so of a sequence
constexpr int kStatHeads = 128;  // heads whose maxima and sums a workgroup holds at a time

// Maximum and sum over groups of `width` lanes, a power of two.
__device__ __forceinline__ float max_over(float v, int width) {
  for (int s = 1; s < width; s *= 2) v = fmaxf(v, __shfl_xor(v, s));
  return v;
}
__device__ __forceinline__ float sum_over(float v, int width) {
  for (int s = 1; s < width; s *= 2) v += __shfl_xor(v, s);
  return v;
}

// After the pieces: the first `joins` workgroups add up the pieces of one
// query head each; the others, a.adds to a sequence and key-value head, add the
// attention weights of kWeightTokens tokens at a time to the accumulator.  Both are chains
// of a few memory latencies, so every loop requests several rounds before it
// uses one.
__global__ __launch_bounds__(kJoinThreads) void attn_join_kernel(AttnArgs a, int joins) {
  __shared__ float sc[kMaxPieces];
  __shared__ f32x4 red[kJoinThreads];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (int(blockIdx.x) < joins) {
    const int b = page_index(a.per_hq, blockIdx.x), h = blockIdx.x - b * a.Hq;
    const int n = min(max(a.lengths[b], 0), a.cap);
    const Pieces p = pieces_of(a, b, n, h);
    const int valid = p.count;
    const float* ml = a.ml + p.at * 2;
    const int64_t next = 2 * p.step;
    // every wave finds the maximum and the sum; wave 0 leaves the factors
    float m = neg_inf();
    for (int s = lane; s < valid; s += 64) m = fmaxf(m, ml[next * s]);
    m = max_over(m, 64);
    const float base = m == neg_inf() ? 0.f : m;
    float l = 0.f;
    for (int s = lane; s < valid; s += 64) {
      const float f = __builtin_amdgcn_exp2f(ml[next * s] - base);
      l += f * ml[next * s + 1];
      if (wave == 0) sc[s] = f;
    }
    l = sum_over(l, 64);
    __syncthreads();
    // four dimensions a thread, the pieces dealt over the threads left
    const int per = a.D <= 64 ? 16 : a.D <= 128 ? 32 : 64;
    const int parts = kJoinThreads / per, part = tid / per, d = tid % per * 4;
    f32x4 acc = {0, 0, 0, 0};
    if (d < a.D) {
      const float* src = a.part + p.at * a.D + d;
      const int64_t row = p.step * a.D;
      constexpr int kUnroll = 8;
      for (int s0 = part; s0 < valid; s0 += kUnroll * parts) {
        f32x4 v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          v[u] = *reinterpret_cast<const f32x4*>(src + min(s0 + u * parts, valid - 1) * row);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (s0 + u * parts < valid) acc += sc[s0 + u * parts] * v[u];
      }
    }
    red[tid] = acc;
    __syncthreads();
    if (part == 0 && d < a.D) {
      for (int o = 1; o < parts; ++o) acc += red[o * per + tid];
      uint16_t* dst = a.out + int64_t(b) * a.o_b + int64_t(h) * a.o_h + d;
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[e] = __builtin_bit_cast(uint16_t, _Float16(l == 0.f ? 0.f : acc[e] / l));
    }
    return;
  }
  int i = blockIdx.x - joins;
  const int chunk = i % a.adds;
  i /= a.adds;
  const int hkv = i % a.Hkv, b = i / a.Hkv;
  const int n = min(max(a.lengths[b], 0), a.cap);
  const int64_t t0 = int64_t(chunk) * kWeightTokens, next_t = int64_t(a.adds) * kWeightTokens;
  if (t0 >= n) return;
  // requested before the maxima and sums, whose chain they would lengthen: the
  // places and the scores of the first tokens and heads
  const int32_t* row = a.table + int64_t(b) * a.table_b;
  Place at[4];
  int t = int(t0) + 256 * wave + lane;
  four_places(a, row, t, n, at);
  constexpr int kUnroll = 4;
  const float* x = a.logits + (int64_t(b) * a.Hq + hkv * a.G) * a.lrow;
  auto scores = [&](int g, float (&v)[kUnroll][4]) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[u][e] = x[int64_t(min(g + u, a.G - 1)) * a.lrow + min(t + 64 * e, n - 1)];
  };
  float v[kUnroll][4];
  scores(0, v);
  const int valid = pieces_of(a, b, n, 0).count;
  // lanes per head for its maximum and sum over the pieces
  int width = 1;
  while (width < valid && width < 64) width *= 2;
  for (int g0 = 0; g0 < a.G; g0 += kStatHeads) {
    const int gn = min(a.G - g0, kStatHeads);
    for (int g = tid / width; g < (gn + 63) / 64 * 64; g += kJoinThreads / width) {
      const Pieces p = pieces_of(a, b, n, hkv * a.G + g0 + min(g, gn - 1));
      const float* ml = a.ml + p.at * 2;
      const int64_t next = 2 * p.step;
      const int s0 = tid % width;
      float m = neg_inf(), l = 0.f;
      for (int s = s0; s < valid; s += width) m = fmaxf(m, ml[next * s]);
      m = max_over(m, width);
      const float base = m == neg_inf() ? 0.f : m;
      for (int s = s0; s < valid; s += width) l += __builtin_amdgcn_exp2f(ml[next * s] - base) * ml[next * s + 1];
      l = sum_over(l, width);
      if (s0 == 0 && g < gn) {
        sc[2 * g] = base;
        sc[2 * g + 1] = l == 0.f ? 0.f : 1.f / l;
      }
    }
    __syncthreads();
    for (int64_t c = t0; c < n; c += next_t) {
      if (c != t0 || g0 > 0) {
        t = int(c) + 256 * wave + lane;
        four_places(a, row, t, n, at);
        scores(g0, v);
      }
      f32x4 w = {0, 0, 0, 0};
      for (int g = 0; g < gn; g += kUnroll) {
        if (g > 0) scores(g0 + g, v);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (g + u < gn) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] += weight_of(v[u][e], sc[2 * (g + u)], sc[2 * (g + u) + 1]);
          }
      }
      add_weights(a, at, hkv, t, n, w);
    }
    __syncthreads();
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

// How the work is dealt.  A unit, up to 16 query heads of one key-value head of
// one sequence, is one workgroup, or several pieces along the length: four waves
// take 128 tokens (a step) at a time, at about 1.1 us, and a second launch that
// joins the pieces costs 5 us.  The lengths are in device memory, so the host
// decides by the capacity alone whether there are pieces and how many at most,
// and the kernel sizes them by the lengths.  Measured, us:
//  - Up to half as many units as CUs, more than eight steps: as many pieces as
//    CUs, of two steps or more (1 x 4096 tokens, 32 heads 51 whole / 17; 2 x
//    131072, 8 heads 1567 / 167; 1 x 1000, 32 heads 13 / 13).  Pieces of one
//    size for all sequences, not so many per sequence: 24 ragged sequences of up
//    to 19030, 2 heads of 256 98 / 71, 11 of up to 19823, 4 heads 52 / 37, for
//    0.7 us of planning (1 x 4096 16.4 / 17.1).  One workgroup per CU: a CU with
//    one more than the others ends last (17 x 43648, one head: 60 at 255
//    workgroups, 73 at 272).  Rows of 64 and less need up to four to keep the
//    memory busy and get them where eight steps or more are left to each (7
//    ragged x 103992, 2 heads: 47 with one, 17 with four).
//  - Up to as many units as CUs, 32 steps or more: two pieces per CU (three with
//    rows above 128, of which a CU holds one workgroup at a time), for batches
//    of unlike lengths (20 ragged x 4096, 8 heads 53 whole / 40; 32 x 8192 126 /
//    115; of one length 94 / 103; 12 ragged x 8000, 12 heads of 256 214 / 104).
//    Below 32 steps the join costs as much as it saves.
//  - More units than CUs: whole sequences, dealt by their length (16 ragged x
//    4096, 32 heads 110 in the batch's order / 89; 64 ragged x 2000, 8 heads 58
//    / 49; cut into pieces no faster), unless they are too short for the sorting
//    in every workgroup to pay (64 x 300 of 32 heads: 32 unsorted / 37; 64 x
//    1000 101 / 90).
//
// The weights: one workgroup that sees a whole sequence keeps its scores in
// LDS and adds the weights itself, as long as three such workgroups fit on a
// CU; otherwise the scores go through the workspace to the second launch (16
// ragged x 4096, 32 heads 100 us and 106; 1 x 137 10 and 15).
AttnPlan plan_attention(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t cap, bool weights, int num_cus) {
  AttnPlan p;
  const int64_t G = Hq / Hkv;
  const int64_t units = B * Hkv * ((G + kHeads - 1) / kHeads);
  const int64_t step = int64_t(kTile) * kWaves;
  const int64_t steps = std::max<int64_t>(1, (cap + step - 1) / step);
  if (B >= 1 && B <= kMaxSorted && units <= num_cus && steps > 8) {
    const int64_t rows = units / B;  // units of a sequence
    int64_t k = 0;                   // workgroups per CU
    if (units <= num_cus / 2) {
      k = 1;
      while (D <= 64 && k < 4 && (k + 1) * num_cus / units <= steps / 8) ++k;
    } else if (steps >= 32) {
      k = D <= 128 ? 2 : 3;
    }
    p.room = int(std::min<int64_t>(k * num_cus / rows, kMaxPieces));
    if (p.room < 2 * B) p.room = 0;
  }
  p.order = p.room == 0 && B > 1 && B <= kMaxSorted && units > num_cus && steps > 4 + B / 32;
  p.cus = num_cus;
  p.lrow = int((cap + kTile - 1) / kTile * kTile);
  const int64_t dp = D <= 64 ? 64 : D <= 128 ? 128 : 256;
  const int64_t join = 4 * (2 * kWaves * kHeads + kWaves * std::min<int64_t>(G, kHeads) * (dp + 4));
  p.own_weights = weights && p.room == 0 && G <= kHeads && join + 4 * G * p.lrow <= 52 * 1024;
  p.lds = size_t(join + (p.own_weights ? 4 * G * p.lrow : 0));
  const size_t rows = size_t(B) * size_t(Hq);
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  const bool scores = weights && !p.own_weights;
  // workgroups of a sequence and head that add the weights: one per 1024 tokens
  // of the capacity, but eight per CU in all; the lengths may be far below it
  // (16 ragged x 4096, 32 heads, tables for 131072 tokens: 155 us with one per
  // 1024, 110 so)
  p.adds = int(std::max<int64_t>(1, std::min<int64_t>((cap + kWeightTokens - 1) / kWeightTokens,
                                                      8 * int64_t(num_cus) / (B * Hkv))));
  const int64_t pieces = p.room > 0 ? p.room * (units / B) : units;
  const size_t sums = size_t(pieces) * size_t(std::min<int64_t>(G, kHeads));
  p.grid = pieces;
  if (p.room > 0) p.bytes += up((1 + size_t(B)) * 4);
  p.off_ml = p.bytes;
  if (p.room > 0 || scores) p.bytes += up(sums * 2 * 4);
  p.off_part = p.bytes;
  if (p.room > 0) p.bytes += up(sums * size_t(D) * 4);
  p.off_logits = p.bytes;
  if (scores) p.bytes += up(rows * size_t(p.lrow) * 4);
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
  a.room = p.room;
  a.lrow = p.lrow;
  a.order = p.order;
  a.cus = p.cus;
  a.scale = r.scale * 1.44269504088896340736f;
  a.div = page_div(c.S);
  uint8_t* w = static_cast<uint8_t*>(ws);
  const bool scores = r.weights && !p.own_weights;
  const bool second = p.room > 0 || scores;
  a.own_weights = p.own_weights;
  if (p.room > 0) a.plan = reinterpret_cast<int32_t*>(w);
  if (second) a.ml = reinterpret_cast<float*>(w + p.off_ml);
  if (p.room > 0) a.part = reinterpret_cast<float*>(w + p.off_part);
  if (scores) a.logits = reinterpret_cast<float*>(w + p.off_logits);

  const int tiles_h = (a.G + kHeads - 1) / kHeads;
  const int dp = a.D <= 64 ? 64 : a.D <= 128 ? 128 : 256;
  const size_t lds = p.lds;
  a.units = a.B * a.Hkv * tiles_h;
  a.per_b = page_div(int64_t(a.Hkv) * tiles_h);
  a.per_hq = page_div(a.Hq);
  a.per_g = page_div(a.G);
  const dim3 grid(uint32_t(p.grid));
  const bool same8 = a.S % 8 == 0;
  hipError_t e = dp == 64    ? launch_dim<64>(a, same8, grid, lds, s)
                 : dp == 128 ? launch_dim<128>(a, same8, grid, lds, s)
                             : launch_dim<256>(a, same8, grid, lds, s);
  if (e != hipSuccess || !second) return e;
  const int64_t joins = p.room > 0 ? int64_t(a.B) * a.Hq : 0;
  a.adds = p.adds;
  const int64_t adds = scores ? int64_t(a.B) * a.Hkv * p.adds : 0;
  if (joins + adds == 0) return hipSuccess;
  attn_join_kernel<<<dim3(uint32_t(joins + adds)), kJoinThreads, 0, s>>>(a, int(joins));
  return hipGetLastError();
}

}  // namespace swm
