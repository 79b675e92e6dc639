// Eviction from a paged key-value cache by accumulated attention weight.
//
// For each sequence with more than `budget` tokens and each key-value head,
// the budget tokens with the largest keys stay, ties going to the lower slot:
//   key = "first" where position > newest - recent, or the weight is NaN or
//         +inf; the weight otherwise.
// The tokens that stay above the budget move into the slots that were freed
// below it, the j-th of them into the j-th free slot.  So a row is copied only
// if its slot goes away: an eviction of one token after each step moves one
// row per head, where closing the gap in order would move half the cache.
// Sources (slots >= budget) and destinations (slots < budget) are disjoint, so
// the copies need no order among themselves.
//
// Up to 32768 tokens, one workgroup per (sequence, head) does everything, its
// keys in registers, four consecutive tokens to a thread:
//  1. Weights and positions, 16 bytes a load, all requested at once; the newest
//     position.
//  2. The key of rank `budget` from the top: a histogram of the top 11 bits
//     (LDS atomics), one wave finds the digit where the budget ends.  If few
//     keys share that digit they are ranked against each other by counting;
//     otherwise the next 11 and 10 bits follow, and keys that are equal in all
//     bits are numbered in slot order.  (Counting by ballots two or three bits
//     at a time took longer at every length: 2000 cycles a step, 6 to 16 steps.)
//  3. Ballots and a prefix sum over the chunks of 256 tokens number the movers
//     and the free slots.
//  4. The map, the weights and positions, and the rows: a wave per 64 pairs,
//     eight rows in flight.
// Beyond that, the first launch reads the keys again for every pass and a
// second one copies the rows; the second launch also serves shorter caches
// with too few heads to fill the CUs and many rows to move.
//
// Bound: by its bytes (8 per token and head, and the moved rows) a call takes
// a few us at most; what it takes is the chain of some ten barriers and four
// memory latencies inside a workgroup.  Measured, in the kernel: 1 x 1025 to
// 1024, 32 heads 10.1 us; 16 x 2176 to 2048, 8 heads 15.2 us; 8 ragged
// sequences of up to 4096 to 1024, 32 heads 43 us with another cache in every
// call, 31 of them for 51 MB of rows, read and written (28.6 us, 16 of them,
// where the rows are in the last-level cache from the call before).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kernels.h"
#include "paging.h"
#include "wave.h"

namespace swm {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kFirst = 0xffffffffu;  // key of the tokens that stay before all others
constexpr int kMaxTokens = 32768;         // tokens whose keys one workgroup holds

struct EvictArgs {
  uint16_t *k, *v;
  const int32_t *table, *lengths;
  const float* w;
  const int32_t* pos;
  float* w_out;
  int32_t *pos_out, *lengths_out, *kept;
  int64_t k_p, k_s, k_h, v_p, v_s, v_h, table_b;
  int64_t w_p, w_h, p_p, p_h, wo_p, wo_h, po_p, po_h;
  int32_t B, Hkv, D, S, pages, cap, per_seq, budget, recent;
  int32_t list_len;  // most tokens that can move
  int32_t vec;       // four weights or positions by one 16-byte load
  PageDiv div;  // by S
};

// Page and slot of token t < capacity.  Where the table names no page of the
// pool, ok is false and the page is 0, so that loads need no branch: a branch
// around each would make a chain of their latencies.
struct Place {
  int page, slot;
  bool ok;
};
__device__ __forceinline__ Place place(const EvictArgs& a, const int32_t* row, int t) {
  Place p;
  const int i = page_index(a.div, t);
  p.slot = t - i * a.S;
  p.page = row[min(i, a.per_seq - 1)];
  p.ok = p.page >= 0 && p.page < a.pages;
  p.page = p.ok ? p.page : 0;
  return p;
}

// Weights by size as whole numbers: NaN and +inf before all, -0 like +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t b = __float_as_uint(w + 0.f);
  if ((b & 0x7fffffffu) > 0x7f800000u || b == 0x7f800000u) return kFirst;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Entry of a per-slot array.
template <typename T>
__device__ __forceinline__ T* entry(T* base, int64_t head, int64_t page, int h, const Place& p) {
  return base + int64_t(h) * head + (int64_t(p.page) * page + p.slot);
}
__device__ __forceinline__ float weight_at(const EvictArgs& a, int h, const Place& p) {
  return *entry(a.w, a.w_h, a.w_p, h, p);
}
__device__ __forceinline__ int32_t position_at(const EvictArgs& a, int h, const Place& p) {
  return *entry(a.pos, a.p_h, a.p_p, h, p);
}
__device__ __forceinline__ void put(const EvictArgs& a, int h, const Place& p, float w, int32_t pos) {
  *entry(a.w_out, a.wo_h, a.wo_p, h, p) = w;
  *entry(a.pos_out, a.po_h, a.po_p, h, p) = pos;
}

// Weight and position of the token in slot `from` become those of slot `to`.
__device__ __forceinline__ void carry(const EvictArgs& a, const int32_t* row, int h, int from, int to) {
  if (from == to && a.w_out == a.w && a.pos_out == a.pos) return;
  const Place p0 = place(a, row, from), p1 = place(a, row, to);
  const float w = weight_at(a, h, p0);
  const int32_t pos = position_at(a, h, p0);
  if (p0.ok && p1.ok) put(a, h, p1, w, pos);
}

template <int kThreads>
struct Scan {  // numbering of the set threads of a workgroup, in thread order
  uint32_t count[kThreads / 64];
};

// Set threads before this one, and how many there are in all.
template <int kThreads>
__device__ __forceinline__ int rank_of(Scan<kThreads>& s, bool on, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint64_t b = __builtin_amdgcn_ballot_w64(on);
  __syncthreads();  // the last call's counts have been read
  if (lane == 0) s.count[wave] = __popcll(b);
  __syncthreads();
  int before = __builtin_amdgcn_mbcnt_hi(uint32_t(b >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(b), 0u));
  int all = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) {
    before += i < wave ? s.count[i] : 0;
    all += s.count[i];
  }
  *total = all;
  return before;
}

// Any length: the keys are read again in every pass.  The list of movers is
// kept in the map's own row until the last pass, which runs from the top slot
// down: the i-th free slot j has j >= i, so an entry is read before anything
// overwrites it.
template <int kThreads>
__global__ __launch_bounds__(kThreads) void evict_long_kernel(EvictArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t chosen[2];
  __shared__ int32_t red[kThreads / 64];
  __shared__ Scan<kThreads> scan_a, scan_b;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int h = blockIdx.x, b = blockIdx.y;
  const int n = min(max(a.lengths[b], 0), a.cap);
  const int left = min(n, a.budget);
  if (h == 0 && tid == 0) a.lengths_out[b] = left;
  const int32_t* row = a.table + int64_t(b) * a.table_b;
  int32_t* kept = a.kept + (int64_t(b) * a.Hkv + h) * a.budget;
  for (int64_t j = tid + left; j < a.budget; j += kThreads) kept[j] = -1;
  if (n <= a.budget || left == 0) {
    for (int j = tid; j < left; j += kThreads) {
      kept[j] = j;
      carry(a, row, h, j, j);
    }
    return;
  }

  int newest = -2147483647 - 1;
  for (int t = tid; t < n; t += kThreads) {
    const Place p = place(a, row, t);
    if (p.ok) newest = max(newest, position_at(a, h, p));
  }
#pragma unroll
  for (int s = 1; s < 64; s *= 2) newest = max(newest, __shfl_xor(newest, s));
  if (lane == 0) red[wave] = newest;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) newest = max(newest, red[i]);
  const int64_t since = int64_t(newest) - a.recent;

  auto key = [&](int t) -> uint32_t {
    const Place p = place(a, row, t);
    if (!p.ok) return 0;
    return int64_t(position_at(a, h, p)) > since ? kFirst : weight_key(weight_at(a, h, p));
  };

  // The key of rank `budget` from the top, eight bits at a time; `want` of the
  // keys that share the bits found so far are still to be taken.
  uint32_t prefix = 0, want = uint32_t(a.budget);
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
    __syncthreads();
    for (int t = tid; t < n; t += kThreads) {
      const uint32_t x = key(t);
      if (shift == 24 || (x >> (shift + 8)) == prefix) atomicAdd(&hist[(x >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (wave == 0) {  // lane l holds bins 255 - 4l .. 252 - 4l
      uint32_t c[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += c[i] = hist[255 - 4 * lane - i];
      uint32_t upto = sum;
#pragma unroll
      for (int s = 1; s < 64; s *= 2) {
        const uint32_t o = __shfl_up(upto, s);
        if (lane >= s) upto += o;
      }
      uint32_t above = upto - sum;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (above < want && above + c[i] >= want) {
          chosen[0] = 255 - 4 * lane - i;
          chosen[1] = want - above;
        }
        above += c[i];
      }
    }
    __syncthreads();
    prefix = (prefix << 8) | chosen[0];
    want = chosen[1];
  }
  const uint32_t last = prefix;  // keys above stay; of the equal ones the first `want`

  // Equal keys below the budget come first.
  int equal = 0;
  for (int t0 = 0; t0 < a.budget; t0 += kThreads) {
    int total;
    rank_of(scan_a, t0 + tid < a.budget && key(t0 + tid) == last, &total);
    equal += total;
  }
  const int equal_below = equal;

  // The movers, in order, into the first entries of the map's row.
  int movers = 0;
  for (int t0 = a.budget; t0 < n; t0 += kThreads) {
    const int t = t0 + tid;
    const uint32_t x = t < n ? key(t) : 0;
    int total;
    const int r = equal + rank_of(scan_a, t < n && x == last, &total);
    equal += total;
    const bool stays = t < n && (x > last || (x == last && uint32_t(r) < want));
    const int i = movers + rank_of(scan_b, stays, &total);
    movers += total;
    if (stays) kept[i] = t;
  }
  __syncthreads();

  // The free slots from the top down: as many as there are movers.
  equal = equal_below;
  for (int t0 = (a.budget - 1) / kThreads * kThreads; t0 >= 0; t0 -= kThreads) {
    const int t = t0 + tid;
    const bool in = t < a.budget;
    const uint32_t x = in ? key(t) : 0;
    int total;
    int r = rank_of(scan_a, in && x == last, &total);
    equal -= total;
    r += equal;
    const bool stays = in && (x > last || (x == last && uint32_t(r) < want));
    int i = rank_of(scan_b, in && !stays, &total);
    movers -= total;
    i += movers;
    int from = t;
    if (in && !stays) from = kept[i];
    __syncthreads();  // every entry that this chunk overwrites has been read
    if (in) {
      kept[t] = from;
      carry(a, row, h, from, t);
    }
  }
}

// Set lanes of b before this one.
__device__ __forceinline__ uint32_t lanes_before(uint64_t b) {
  return __builtin_amdgcn_mbcnt_hi(uint32_t(b >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(b), 0u));
}

// Copies rows of one head.  Each lane names one pair of slots (from < 0: none);
// their places are looked up together and gathered into the first lanes (a pair
// with a slot on no page is left out).  Then lanes 0..31 copy key rows and 32..63
// value rows, as many pairs at a time as their rows fill lanes, eight such loads
// in flight (past the last pair, that one is read again): a CU's rate is what it
// has in flight (one pair a load: 32 x 2048 to 512, 32 heads of 64 79 us, 67 so; 8
// ragged x 4096 to 1024 of 128 49, 47).
__device__ __forceinline__ void move_rows(const EvictArgs& a, const int32_t* row, int h, int from, int to) {
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int shift = a.D <= 64 ? 3 : a.D <= 128 ? 4 : 5;  // of the lanes of a row
  const int per = 32 >> shift, sub = (lane & 31) >> shift, d = (lane & ((1 << shift) - 1)) * 8;
  uint16_t* base = half ? a.v + int64_t(h) * a.v_h : a.k + int64_t(h) * a.k_h;
  const int64_t sp = half ? a.v_p : a.k_p, ss = half ? a.v_s : a.k_s;
  const Place p0 = place(a, row, max(from, 0)), p1 = place(a, row, to);
  const bool on = from >= 0 && p0.ok && p1.ok;
  const uint64_t pairs = __builtin_amdgcn_ballot_w64(on);
  const int n = __popcll(pairs), rank = int(lanes_before(pairs));
  const int lane4 = 4 * (on ? rank : n + lane - rank);
  const int from_page = __builtin_amdgcn_ds_permute(lane4, p0.page);
  const int from_slot = __builtin_amdgcn_ds_permute(lane4, p0.slot);
  const int to_page = __builtin_amdgcn_ds_permute(lane4, p1.page);
  const int to_slot = __builtin_amdgcn_ds_permute(lane4, p1.slot);
  const int dl = d < a.D ? d : 0;  // lanes past the row read its start and store nothing
  constexpr int kRows = 8;
  for (int i0 = 0; i0 < n; i0 += kRows * per) {
    u32x4 x[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int i = min(i0 + u * per + sub, n - 1);
      x[u] = *reinterpret_cast<const u32x4*>(base + int64_t(__shfl(from_page, i)) * sp +
                                             int64_t(__shfl(from_slot, i)) * ss + dl);
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int i = i0 + u * per + sub, j = min(i, n - 1);
      const int page = __shfl(to_page, j), slot = __shfl(to_slot, j);
      if (i < n && d < a.D) *reinterpret_cast<u32x4*>(base + int64_t(page) * sp + int64_t(slot) * ss + d) = x[u];
    }
  }
}

constexpr int kDigit = 11;        // bits of a histogram
constexpr int kBins = 1 << kDigit;
constexpr int kCandidates = 512;  // keys ranked by counting

// Histogram entries, one word of padding per 32: 64 lanes that read 32 bins
// each then hit different banks.
__device__ __forceinline__ uint32_t bin_at(uint32_t bin) { return bin + (bin >> 5); }

// Counts the active lanes' bins.  Lanes that share the first one's bin (recent
// tokens, tokens nothing looked at) count once together: an atomic per lane
// would queue up on one address.
__device__ __forceinline__ void count_bins(uint32_t* hist, uint32_t bin, bool active) {
  const uint64_t all = __builtin_amdgcn_ballot_w64(active);
  if (all == 0) return;
  const int leader = __builtin_ctzll(all);
  const uint32_t first = uint32_t(__builtin_amdgcn_readlane(int(bin), leader));
  const uint64_t same = __builtin_amdgcn_ballot_w64(active && bin == first);
  if (int(threadIdx.x & 63) == leader)
    atomicAdd(&hist[bin_at(first)], uint32_t(__popcll(same)));
  else if (active && bin != first)
    atomicAdd(&hist[bin_at(bin)], 1u);
}

// Weights, positions and places of the four tokens from t on (clamped to last).
// vec: a page holds a multiple of four slots and both arrays are aligned for
// 16-byte loads, so one place and two loads do.
__device__ __forceinline__ void load4(const EvictArgs& a, const int32_t* row, int h, int t, int last, Place (&at)[4],
                                      float (&w)[4], int32_t (&pos)[4]) {
  if (a.vec) {
    at[0] = place(a, row, min(t, last & ~3));
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
    const f32x4 wv = *reinterpret_cast<const f32x4*>(entry(a.w, a.w_h, a.w_p, h, at[0]));
    const i32x4 pv = *reinterpret_cast<const i32x4*>(entry(a.pos, a.p_h, a.p_p, h, at[0]));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      at[e] = Place{at[0].page, at[0].slot + e, at[0].ok};
      w[e] = wv[e];
      pos[e] = pv[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) at[e] = place(a, row, min(t + e, last));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[e] = weight_at(a, h, at[e]);
      pos[e] = position_at(a, h, at[e]);
    }
  }
}

// Thread i holds tokens 4 (q kThreads + i) .. + 3 for q < kQ: a chunk of 256
// tokens per wave and q, in order.  move: also copy the rows.
template <int kThreads, int kQ>
__global__ __launch_bounds__(kThreads, kThreads / 256) void evict_kernel(EvictArgs a, int move) {
  constexpr int kWaves = kThreads / 64, kChunks = kWaves * kQ;
  constexpr bool kHold = kQ <= 2;  // weights and positions stay in registers for the end
  static_assert(kChunks <= 128, "");
  extern __shared__ uint16_t lists[];  // movers, then free slots: list_len entries each
  __shared__ uint32_t hist[kBins + kBins / 32];
  __shared__ uint64_t cand[kCandidates];
  __shared__ uint32_t chunk[kChunks];
  __shared__ uint32_t listed, chosen[3];
  __shared__ int32_t red[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int h = blockIdx.x, b = blockIdx.y;
  const int32_t* row = a.table + int64_t(b) * a.table_b;
  const int n = min(max(a.lengths[b], 0), a.cap);
  const int left = min(n, a.budget);
  if (h == 0 && tid == 0) a.lengths_out[b] = left;
  int32_t* kept = a.kept + (int64_t(b) * a.Hkv + h) * a.budget;
  for (int64_t j = tid + left; j < a.budget; j += kThreads) kept[j] = -1;
  if (n <= a.budget || left == 0) {
    for (int j = tid; j < left; j += kThreads) {
      kept[j] = j;
      carry(a, row, h, j, j);
    }
    return;
  }

  float w[kQ][4];
  int32_t pos[kQ][4];
  uint32_t key[kQ][4];
  uint32_t there = 0;  // bit 4q + e: the token is below the length and on a page
  {
    Place at[kQ][4];
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      if (4 * q * kThreads >= n) continue;  // the same for every thread, here and below
      load4(a, row, h, 4 * (q * kThreads + tid), n - 1, at[q], w[q], pos[q]);
    }
    int newest = -2147483647 - 1;
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      if (4 * q * kThreads >= n) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool ok = 4 * (q * kThreads + tid) + e < n && at[q][e].ok;
        there |= uint32_t(ok) << (4 * q + e);
        newest = ok ? max(newest, pos[q][e]) : newest;
      }
    }
    newest = wave_max(newest);
    if (lane == 0) red[wave] = newest;
    if (tid == 0) listed = 0;
    for (int i = tid; i < kBins + kBins / 32; i += kThreads) hist[i] = 0;
    __syncthreads();
    newest = wave_max(red[min(lane, kWaves - 1)]);
    // positions above `since` are recent (none if it would be below the smallest number)
    const int64_t since = int64_t(newest) - a.recent;
    const bool all = since < -2147483647 - 1;
#pragma unroll
    for (int q = 0; q < kQ; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        key[q][e] = 0;
        if (4 * q * kThreads >= n) continue;
        const uint32_t k = all || pos[q][e] > int32_t(since) ? kFirst : weight_key(w[q][e]);
        key[q][e] = (there >> (4 * q + e)) & 1 ? k : 0u;
      }
  }

  // The key of rank `budget` from the top, 11, 11 and 10 bits at a time:
  // `prefix` holds the bits found so far (those above `shift`), `sharing` keys
  // have them, of which `want` stay.
  uint32_t prefix = 0, want = uint32_t(a.budget), sharing = 0;
  int shift = 32;
#pragma unroll 1
  do {
    const int bits = min(kDigit, shift), over = shift;
    shift -= bits;
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      if (4 * q * kThreads >= n) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        count_bins(hist, (key[q][e] >> shift) & ((1u << bits) - 1),
                   4 * (q * kThreads + tid) + e < n && (over == 32 || (key[q][e] >> over) == prefix));
    }
    __syncthreads();
    if (wave == 0) {  // lane l holds the 32 bins from kBins - 1 - 32 l downwards
      uint32_t sum = 0;
#pragma unroll
      for (int i = 0; i < 32; ++i) sum += hist[bin_at(kBins - 1 - 32 * lane) - i];
      const uint32_t upto = scan_wave(sum);
      const uint64_t reach = __builtin_amdgcn_ballot_w64(upto >= want);
      const int l = __builtin_ctzll(reach);  // the lane whose bins hold the budget's end
      const uint32_t before = uint32_t(__builtin_amdgcn_readlane(int(upto - sum), l));
      const uint32_t c = lane < 32 ? hist[bin_at(kBins - 1 - 32 * l) - lane] : 0;
      const uint32_t u = before + scan_wave(c);
      if (u >= want && u - c < want && lane < 32) {
        chosen[0] = uint32_t(kBins - 1 - 32 * l - lane);
        chosen[1] = want - (u - c);
        chosen[2] = c;
      }
    }
    __syncthreads();
    prefix = (prefix << bits) | chosen[0];
    want = chosen[1];
    sharing = chosen[2];
    if (shift > 0 && sharing > kCandidates) {
      for (int i = tid; i < kBins + kBins / 32; i += kThreads) hist[i] = 0;
      __syncthreads();
    }
  } while (shift > 0 && sharing > kCandidates);

  // Keys above stay; of those that share the prefix the `want` best, by their
  // key and then the lower slot.
  uint32_t taken = ~0u;  // bit 4q + e: if it shares the prefix, the token stays
  if (sharing == want) {
    // all of them
  } else if (sharing <= kCandidates) {
    uint32_t at[kQ][4];
#pragma unroll
    for (int q = 0; q < kQ; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 4 * (q * kThreads + tid) + e;
        at[q][e] = ~0u;
        if (t < n && (key[q][e] >> shift) == prefix) {
          at[q][e] = atomicAdd(&listed, 1u);
          cand[at[q][e]] = uint64_t(key[q][e]) << 32 | (0xffffffffu - uint32_t(t));
        }
      }
    __syncthreads();
    // four lanes to a candidate, each counting a quarter of the list
    for (uint32_t i = tid / 4; i < sharing; i += kThreads / 4) {
      const uint64_t mine = cand[i];
      uint32_t rank = 0;
#pragma unroll 8
      for (uint32_t j = tid % 4; j < sharing; j += 4) rank += cand[j] > mine;
      rank += uint32_t(__builtin_amdgcn_mov_dpp(int(rank), 0xb1, 0xf, 0xf, true));  // lanes 1 0 3 2
      rank += uint32_t(__builtin_amdgcn_mov_dpp(int(rank), 0x4e, 0xf, 0xf, true));  // lanes 2 3 0 1
      if (tid % 4 == 0) hist[i] = rank < want;  // the counts have been read
    }
    __syncthreads();
    taken = 0;
#pragma unroll
    for (int q = 0; q < kQ; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (at[q][e] != ~0u && hist[at[q][e]]) taken |= 1u << (4 * q + e);
  } else {  // more equal keys than that: in slot order
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      uint32_t c = 0;
#pragma unroll
      for (int e = 0; e < 4 && 4 * q * kThreads < n; ++e)
        c += __popcll(__builtin_amdgcn_ballot_w64(4 * (q * kThreads + tid) + e < n && key[q][e] == prefix));
      if (lane == 0) chunk[q * kWaves + wave] = c;
    }
    __syncthreads();
    const uint32_t c0 = lane < kChunks ? chunk[lane] : 0, c1 = 64 + lane < kChunks ? chunk[min(64 + lane, kChunks - 1)] : 0;
    const uint32_t u0 = scan_wave(c0), u1 = __shfl(u0, 63) + scan_wave(c1) - c1;  // u1: before the second 64
    taken = 0;
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      if (4 * q * kThreads >= n) continue;
      const int i = q * kWaves + wave;
      uint32_t rank = i < 64 ? __shfl(u0 - c0, i) : __shfl(u1, i - 64);
      bool equal[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        equal[e] = 4 * (q * kThreads + tid) + e < n && key[q][e] == prefix;
        rank += lanes_before(__builtin_amdgcn_ballot_w64(equal[e]));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (equal[e] && rank < want) taken |= 1u << (4 * q + e);
        rank += equal[e];
      }
    }
    __syncthreads();  // chunk is written again
  }

  // Who stays, and how many movers and free slots each chunk has.
  uint32_t mine = 0;
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    uint32_t movers = 0, holes = 0;
#pragma unroll
    for (int e = 0; e < 4 && 4 * q * kThreads < n; ++e) {
      const int t = 4 * (q * kThreads + tid) + e;
      const uint32_t x = key[q][e] >> shift;
      const bool on = t < n && (x > prefix || (x == prefix && ((taken >> (4 * q + e)) & 1)));
      mine |= uint32_t(on) << (4 * q + e);
      movers += __popcll(__builtin_amdgcn_ballot_w64(on && t >= a.budget));
      holes += __popcll(__builtin_amdgcn_ballot_w64(!on && t < a.budget));
    }
    if (lane == 0) chunk[q * kWaves + wave] = movers << 16 | holes;
  }
  __syncthreads();
  // every wave adds the chunks up for itself
  const uint32_t c0 = lane < kChunks ? chunk[lane] : 0, u0 = scan_wave(c0);
  uint32_t total = uint32_t(__builtin_amdgcn_readlane(int(u0), 63)), c1 = 0, u1 = 0;
  if (kChunks > 64) {
    c1 = chunk[min(64 + lane, kChunks - 1)];
    u1 = total + scan_wave(c1);
    total = uint32_t(__builtin_amdgcn_readlane(int(u1), 63));
  }
  const int movers = int(total >> 16);
  uint16_t* from = lists;
  uint16_t* freed = lists + a.list_len;
  uint32_t number[kQ];  // of the thread's first mover and free slot of the group
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    number[q] = 0;
    if (4 * q * kThreads >= n) continue;
    const int i = q * kWaves + wave;
    uint32_t r = uint32_t(i < 64 ? __builtin_amdgcn_readlane(int(u0 - c0), i) : __builtin_amdgcn_readlane(int(u1 - c1), i - 64));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = 4 * (q * kThreads + tid) + e;
      const bool on = (mine >> (4 * q + e)) & 1;
      r += lanes_before(__builtin_amdgcn_ballot_w64(on && t >= a.budget)) << 16;
      r += lanes_before(__builtin_amdgcn_ballot_w64(!on && t < a.budget));
    }
    number[q] = r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = 4 * (q * kThreads + tid) + e;
      const bool on = (mine >> (4 * q + e)) & 1;
      if (t < a.budget && on) kept[t] = t;
      if (t < a.budget && !on) {
        freed[r & 0xffffu] = uint16_t(t);
        r += 1;
      }
      if (t >= a.budget && on) {
        from[r >> 16] = uint16_t(t);
        r += 1u << 16;
      }
    }
  }
  __syncthreads();
  // Every token that stays tells its slot where it is from.
  const bool copy = a.w_out != a.w || a.pos_out != a.pos;
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    const int t0 = 4 * (q * kThreads + tid);
    if (4 * q * kThreads >= n) continue;
    // nothing to do for a wave without movers (and without a copy)
    const uint32_t on4 = (mine >> (4 * q)) & 15u;
    if (!__builtin_amdgcn_ballot_w64(on4 != 0 && (copy || t0 + 3 >= a.budget))) continue;
    Place at[4];
    float w4[4];
    int32_t p4[4];
    if (!kHold) load4(a, row, h, t0, n - 1, at, w4, p4);
    uint32_t r = number[q] >> 16;
    int to[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool on = (on4 >> e) & 1, moves = on && t0 + e >= a.budget;
      to[e] = moves ? int(freed[r]) : on && copy ? t0 + e : -1;
      r += moves;
      at[e] = place(a, row, max(to[e], 0));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (to[e] < 0) continue;
      if (t0 + e >= a.budget) kept[to[e]] = t0 + e;
      if (at[e].ok && ((there >> (4 * q + e)) & 1))
        put(a, h, at[e], kHold ? w[q][e] : w4[e], kHold ? pos[q][e] : p4[e]);
    }
  }
  if (move) {
    // the pairs dealt evenly: at most 64 a wave and round
    const int share = min((movers + kWaves - 1) / kWaves, 64);
    for (int i0 = 0; i0 < movers; i0 += share * kWaves) {
      const int i = i0 + wave * share + lane;
      const bool on = lane < share && i < movers;
      move_rows(a, row, h, on ? int(from[i]) : -1, on ? int(freed[i]) : 0);
    }
  }
}

// The rows alone, a wave per 64 slots of the map.
__global__ __launch_bounds__(256) void evict_move_kernel(EvictArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int h = blockIdx.y, b = blockIdx.z;
  const int j0 = (blockIdx.x * 4 + wave) * 64;
  if (j0 >= a.budget) return;
  const int32_t* row = a.table + int64_t(b) * a.table_b;
  const int32_t* kept = a.kept + (int64_t(b) * a.Hkv + h) * a.budget;
  const int from = j0 + lane < a.budget ? kept[j0 + lane] : -1;
  move_rows(a, row, h, from >= a.budget ? from : -1, j0 + lane);
}

template <int kThreads, int kQ>
hipError_t launch_one(const EvictArgs& a, int move, hipStream_t s) {
  const size_t lds = 4 * size_t(a.list_len);
  if (lds > 56 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(evict_kernel<kThreads, kQ>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, int(lds));
    if (e != hipSuccess) return e;
  }
  evict_kernel<kThreads, kQ><<<dim3(a.Hkv, a.B), kThreads, lds, s>>>(a, move);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_evict(const KvView& c, const EvictCall& r, int num_cus, hipStream_t s) {
  EvictArgs a{};
  a.k = c.k;
  a.v = c.v;
  a.table = c.table;
  a.lengths = c.lengths;
  a.w = r.weights;
  a.pos = r.positions;
  a.w_out = r.weights_out;
  a.pos_out = r.positions_out;
  a.lengths_out = r.lengths_out;
  a.kept = r.kept;
  a.k_p = c.k_p;
  a.k_s = c.k_s;
  a.k_h = c.k_h;
  a.v_p = c.v_p;
  a.v_s = c.v_s;
  a.v_h = c.v_h;
  a.table_b = c.table_b;
  a.w_p = r.w_p;
  a.w_h = r.w_h;
  a.p_p = r.p_p;
  a.p_h = r.p_h;
  a.wo_p = r.wo_p;
  a.wo_h = r.wo_h;
  a.po_p = r.po_p;
  a.po_h = r.po_h;
  a.B = int(c.B);
  a.Hkv = int(c.Hkv);
  a.D = int(c.D);
  a.S = int(c.S);
  a.pages = int(c.pages);
  a.per_seq = int(c.per_seq);
  a.cap = int(c.per_seq * c.S);
  a.budget = int(r.budget);
  a.recent = int(r.recent);
  a.div = page_div(c.S);
  a.vec = c.S % 4 == 0 && (r.w_p | r.w_h | r.p_p | r.p_h) % 4 == 0 &&
          ((reinterpret_cast<uintptr_t>(r.weights) | reinterpret_cast<uintptr_t>(r.positions)) & 15) == 0;
  a.list_len = std::max(0, std::min(a.budget, a.cap - a.budget));
  // The workgroup that selects also moves, unless workgroups are too few to
  // move many rows at the memory's rate (15 x 8 heads, 7098 to 3549 tokens: 65
  // us against 47 with a launch of its own; 16 x 8, 2176 to 2048: 19 against 24;
  // 32 x 32, 2048 to 512: 8 less than with one).
  const bool move = int64_t(a.Hkv) * a.B >= num_cus || a.list_len <= 512;
  // The fewest threads that hold all keys, eight each at most up to 8192 tokens:
  // 16 x 32 heads, 2000 tokens by 512 x 4 keys 21 us, by 1024 x 8 31; 8 x 32,
  // 8000 tokens by 1024 x 8 32, by 1024 x 16 41.  Above 32768 tokens the keys
  // would not fit; reading them again takes 70-180% longer (4 x 8, 30000: 95
  // and 181).
  hipError_t e;
  if (a.cap <= 1024) {
    e = launch_one<256, 1>(a, move, s);
  } else if (a.cap <= 2048) {
    e = launch_one<512, 1>(a, move, s);
  } else if (a.cap <= 8192) {
    e = launch_one<1024, 2>(a, move, s);
  } else if (a.cap <= kMaxTokens) {
    e = a.cap <= kMaxTokens / 2 ? launch_one<1024, 4>(a, move, s) : launch_one<1024, 8>(a, move, s);
  } else {
    evict_long_kernel<1024><<<dim3(a.Hkv, a.B), 1024, 0, s>>>(a);
    e = hipGetLastError();
  }
  if (e != hipSuccess || a.list_len == 0 || (move && a.cap <= kMaxTokens)) return e;
  evict_move_kernel<<<dim3((a.budget + 255) / 256, a.Hkv, a.B), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace swm
