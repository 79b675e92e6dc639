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
// First launch, one workgroup per (sequence, head): the key of rank `budget`
// by a radix selection of eight bits at a time (histograms in LDS), then two
// ordered passes of ballots that number the movers and the free slots.  The
// list of movers is kept in the map's own row until the second pass, which
// runs from the top slot down: the i-th free slot j has j >= i, so an entry is
// read before anything overwrites it.  Second launch: the rows, a wave per 64
// slots of the map.
//
// Bound: the weights and positions are read once (8 bytes per token and
// head; from LDS after that), the moved rows once; at serving sizes the chain
// of passes inside a workgroup is what takes the time.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kernels.h"

namespace swm {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kFirst = 0xffffffffu;  // key of the tokens that stay before all others
constexpr int kLdsTokens = 32768;         // tokens whose keys fit in LDS (128 KiB of the CU's 160)

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
  double inv_s;
};

// Page and slot of token t < capacity; false where the table names no page.
__device__ __forceinline__ bool place(const EvictArgs& a, const int32_t* row, int t, int* page, int* slot) {
  const int i = int((double(t) + 0.5) * a.inv_s);
  *slot = t - i * a.S;
  *page = row[min(i, a.per_seq - 1)];
  return *page >= 0 && *page < a.pages;
}

// Weights by size as whole numbers: NaN and +inf before all, -0 like +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t b = __float_as_uint(w + 0.f);
  if ((b & 0x7fffffffu) > 0x7f800000u || b == 0x7f800000u) return kFirst;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
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

template <int kThreads, bool kLds>
__global__ __launch_bounds__(kThreads) void evict_select_kernel(EvictArgs a) {
  extern __shared__ uint32_t keys[];
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
  const float* w = a.w + int64_t(h) * a.w_h;
  const int32_t* pos = a.pos + int64_t(h) * a.p_h;
  float* wo = a.w_out + int64_t(h) * a.wo_h;
  int32_t* po = a.pos_out + int64_t(h) * a.po_h;
  const bool copy = a.w_out != a.w, copy_p = a.pos_out != a.pos;

  // weight and position of the token in slot `from` become those of slot `to`
  auto carry = [&](int from, int to) {
    int p0, s0, p1, s1;
    if (!place(a, row, from, &p0, &s0) || !place(a, row, to, &p1, &s1)) return;
    if (from != to || copy) wo[int64_t(p1) * a.wo_p + s1] = w[int64_t(p0) * a.w_p + s0];
    if (from != to || copy_p) po[int64_t(p1) * a.po_p + s1] = pos[int64_t(p0) * a.p_p + s0];
  };

  for (int j = tid + left; j < a.budget; j += kThreads) kept[j] = -1;
  if (n <= a.budget || left == 0) {
    for (int j = tid; j < left; j += kThreads) {
      kept[j] = j;
      carry(j, j);
    }
    return;
  }

  int newest = -2147483647 - 1;
  for (int t = tid; t < n; t += kThreads) {
    int p, s;
    if (place(a, row, t, &p, &s)) newest = max(newest, pos[int64_t(p) * a.p_p + s]);
  }
#pragma unroll
  for (int s = 1; s < 64; s *= 2) newest = max(newest, __shfl_xor(newest, s));
  if (lane == 0) red[wave] = newest;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) newest = max(newest, red[i]);
  const int64_t since = int64_t(newest) - a.recent;

  auto key_of = [&](int t) -> uint32_t {
    int p, s;
    if (!place(a, row, t, &p, &s)) return 0;
    if (int64_t(pos[int64_t(p) * a.p_p + s]) > since) return kFirst;
    return weight_key(w[int64_t(p) * a.w_p + s]);
  };
  if (kLds) {
    for (int t = tid; t < n; t += kThreads) keys[t] = key_of(t);
    __syncthreads();
  }
  auto key = [&](int t) -> uint32_t { return kLds ? keys[t] : key_of(t); };

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
      carry(from, t);
    }
  }
}

// A wave per 64 slots of the map; lanes 0..31 carry a key row, 32..63 the value
// row.
__global__ __launch_bounds__(256) void evict_move_kernel(EvictArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int h = blockIdx.y, b = blockIdx.z;
  const int j0 = (blockIdx.x * 4 + wave) * 64;
  if (j0 >= a.budget) return;
  const int32_t* row = a.table + int64_t(b) * a.table_b;
  const int32_t* kept = a.kept + (int64_t(b) * a.Hkv + h) * a.budget;
  const int j = j0 + lane;
  const int from = j < a.budget ? kept[j] : -1;
  // both places of the lane's own slot, as element offsets; -1 where it stays
  int64_t ks = -1, kd = 0, vs = 0, vd = 0;
  if (from >= a.budget) {
    int p0, s0, p1, s1;
    if (place(a, row, from, &p0, &s0) && place(a, row, j, &p1, &s1)) {
      ks = int64_t(p0) * a.k_p + int64_t(s0) * a.k_s;
      kd = int64_t(p1) * a.k_p + int64_t(s1) * a.k_s;
      vs = int64_t(p0) * a.v_p + int64_t(s0) * a.v_s;
      vd = int64_t(p1) * a.v_p + int64_t(s1) * a.v_s;
    }
  }
  uint64_t todo = __builtin_amdgcn_ballot_w64(ks >= 0);
  const int half = lane >> 5, d = (lane & 31) * 8;
  uint16_t* base = half ? a.v + int64_t(h) * a.v_h : a.k + int64_t(h) * a.k_h;
  while (todo) {
    constexpr int kRows = 4;  // rows in flight
    u32x4 x[kRows];
    int64_t to[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      to[i] = -1;
      if (todo) {
        const int l = __builtin_ctzll(todo);
        todo &= todo - 1;
        const int64_t k0 = __shfl(ks, l), k1 = __shfl(kd, l), v0 = __shfl(vs, l), v1 = __shfl(vd, l);
        const int64_t src = half ? v0 : k0;
        to[i] = half ? v1 : k1;
        if (d < a.D) x[i] = *reinterpret_cast<const u32x4*>(base + src + d);
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (to[i] >= 0 && d < a.D) *reinterpret_cast<u32x4*>(base + to[i] + d) = x[i];
  }
}

}  // namespace

hipError_t launch_evict(const KvView& c, const EvictCall& r, hipStream_t s) {
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
  a.inv_s = 1.0 / double(c.S);
  constexpr int kThreads = 1024;
  const dim3 grid(a.Hkv, a.B);
  if (a.cap <= kLdsTokens) {
    const size_t lds = 4 * size_t(std::max(a.cap, 1));
    if (lds > 60 * 1024) {
      const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(evict_select_kernel<kThreads, true>),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, int(lds));
      if (e != hipSuccess) return e;
    }
    evict_select_kernel<kThreads, true><<<grid, kThreads, lds, s>>>(a);
  } else {
    evict_select_kernel<kThreads, false><<<grid, kThreads, 0, s>>>(a);
  }
  hipError_t e = hipGetLastError();
  // nothing can move unless the capacity is beyond the budget
  if (e != hipSuccess || a.cap <= a.budget || a.budget == 0) return e;
  evict_move_kernel<<<dim3((a.budget + 255) / 256, a.Hkv, a.B), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace swm
