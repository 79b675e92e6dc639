// What brings tokens into a paged cache: their pages and slots, and their rows.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kernels.h"
#include "paging.h"
#include "wave.h"

namespace swm {
namespace {

// ---------------------------------------------------------------- reserve
//
// Sequence b goes from n_b to n_b + c_b tokens, from h_b = ceil(n_b / S) pages
// to g_b.  Pages from g_b to h_b go back, in order of sequence and place, on top
// of the free ones; then sequence b takes g_b - h_b from the top, in order:
//   upto_b = sum_{a <= b} max(g_a - h_a, 0);  granted if upto_b <= free pages,
// so what a sequence gets follows from prefix sums, and one workgroup has them
// in registers.  The slots of the added tokens read the table that it wrote.

constexpr int kThreads = 1024;  // of the planning workgroup: sequences of a round
constexpr int kOwnSlots = 4 * kThreads;  // slots that it fills itself
constexpr int kFill = 256;      // threads of a workgroup that fills slots, and tokens of it
constexpr int kHeld = 4096;     // sequences whose starts it holds in LDS

struct ReserveArgs {
  int32_t *table, *lengths;
  const int32_t* counts;
  int32_t *free_pages, *free_count, *starts, *granted;
  int64_t* slots;
  int64_t table_b, tokens;
  int32_t B, S, pages, per_seq, cap, room;  // room: entries of free_pages
  PageDiv div;
};

struct Step {
  int old, want, had, has;
};
__device__ __forceinline__ Step step_of(const ReserveArgs& a, int b) {
  Step s{0, 0, 0, 0};
  if (b >= a.B) return s;
  s.old = min(max(a.lengths[b], 0), a.cap);
  const int64_t want = int64_t(s.old) + a.counts[b];
  s.want = want > a.cap ? s.old : int(max(want, int64_t(0)));
  s.had = s.old > 0 ? page_index(a.div, s.old - 1) + 1 : 0;
  s.has = s.want > 0 ? page_index(a.div, s.want - 1) + 1 : 0;
  return s;
}

// Sums of the workgroup's threads up to and including this one; *all: of all.
// sums: kThreads / 64 entries that nothing else uses until the next barrier but one.
__device__ __forceinline__ int64_t scan_block(int64_t v, int64_t* sums, int64_t* all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int o = 1; o < 64; o *= 2) {
    const int64_t x = __shfl_up(v, o);
    if (lane >= o) v += x;
  }
  __syncthreads();
  if (lane == 63) sums[wave] = v;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int w = 0; w < kThreads / 64; ++w) {
    const int64_t x = sums[w];
    if (w < wave) before += x;
    total += x;
  }
  *all = total;
  return v + before;
}

// The entry of a rising list whose value is the first above i.
template <typename T>
__device__ __forceinline__ int first_above(const T* list, int n, int64_t i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (list[mid] > i)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// Slot of token `at` of a sequence, -1 where the table names no page.
__device__ __forceinline__ int64_t slot_of(const ReserveArgs& a, int b, int at) {
  const int i = page_index(a.div, at);
  const int page = a.table[int64_t(b) * a.table_b + i];
  return page >= 0 && page < a.pages ? int64_t(page) * a.S + (at - i * a.S) : -1;
}

__global__ __launch_bounds__(kThreads) void reserve_kernel(ReserveArgs a) {
  __shared__ int64_t upto[kThreads];
  __shared__ int64_t sums[kThreads / 64];
  __shared__ int32_t first[kThreads];
  const int tid = threadIdx.x, lane = tid & 63;
  int64_t have = min(max(a.free_count[0], 0), a.room);
  // pages that come back
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const Step s = step_of(a, b0 + tid);
    int64_t total;
    const int64_t u = scan_block(max(s.had - s.has, 0), sums, &total);
    if (total == 0) continue;
    upto[tid] = u;
    first[tid] = s.has;
    __syncthreads();
    for (int64_t i0 = 0; i0 < total; i0 += kThreads) {
      const int64_t i = i0 + tid;
      int page = -1;
      if (i < total) {
        const int x = first_above(upto, kThreads, i);
        const int64_t begin = x ? upto[x - 1] : 0;
        int32_t* e = a.table + int64_t(b0 + x) * a.table_b + first[x] + (i - begin);
        page = *e;
        *e = -1;
      }
      const bool is = page >= 0 && page < a.pages;
      int64_t some;
      const int64_t at = have + scan_block(is, sums, &some) - 1;
      if (is && at < a.room) a.free_pages[at] = page;
      have = min(have + some, int64_t(a.room));
    }
  }
  __threadfence_block();
  __syncthreads();
  // pages that are taken, lengths, starts
  int64_t taken = 0, asked = 0, packed = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + tid;
    const Step s = step_of(a, b);
    const int count = b < a.B ? a.counts[b] : 0;
    int64_t total, rows;
    const int need = max(s.has - s.had, 0);
    const int64_t u = asked + scan_block(need, sums, &total);
    const int64_t p = packed + scan_block(max(count, 0), sums, &rows);
    const bool fits = need == 0 || u <= have;
    if (b < a.B) {
      if (fits) a.lengths[b] = s.want;
      else if (a.lengths[b] != s.old) a.lengths[b] = s.old;
      a.granted[b] = fits ? s.want - s.old : 0;
      a.starts[b + 1] = int32_t(min(p, int64_t(0x7fffffff)));
      if (b == 0) a.starts[0] = 0;
    }
    int64_t here;
    upto[tid] = u;
    first[tid] = s.had;
    scan_block(fits ? need : 0, sums, &here);  // the barriers of the lists too
    for (int64_t i = asked + tid; i < asked + here; i += kThreads) {
      const int x = first_above(upto, kThreads, i);
      const int64_t begin = x ? upto[x - 1] : asked;
      a.table[int64_t(b0 + x) * a.table_b + first[x] + (i - begin)] = a.free_pages[have - 1 - i];
    }
    __syncthreads();
    taken += here;
    asked += total;
    packed += rows;
  }
  if (tid == 0) {
    a.free_count[0] = int32_t(have - taken);
    if (a.B == 0) a.starts[0] = 0;
  }
  if (a.tokens > kOwnSlots) return;
  __threadfence_block();
  __syncthreads();
  for (int64_t i = tid; i < a.tokens; i += kThreads) {
    int64_t slot = -1;
    if (i < packed) {
      const int b = first_above(a.starts + 1, a.B, i);
      const int g = a.granted[b];
      if (g > 0) slot = slot_of(a, b, a.lengths[b] - g + int(i - a.starts[b]));
    }
    a.slots[i] = slot;
  }
}

__global__ __launch_bounds__(kFill) void slots_kernel(ReserveArgs a) {
  __shared__ int32_t starts[kHeld];
  const bool held = a.B <= kHeld;
  if (held) {
    for (int b = threadIdx.x; b < a.B; b += kFill) starts[b] = a.starts[b + 1];
    __syncthreads();
  }
  const int64_t i = int64_t(blockIdx.x) * kFill + threadIdx.x;
  if (i >= a.tokens) return;
  int64_t slot = -1;
  if (a.B > 0 && i < a.starts[a.B]) {
    const int b = held ? first_above(starts, a.B, i) : first_above(a.starts + 1, a.B, i);
    const int g = a.granted[b];
    if (g > 0) slot = slot_of(a, b, a.lengths[b] - g + int(i - a.starts[b]));
  }
  a.slots[i] = slot;
}

// ---------------------------------------------------------------- append

constexpr int kCopy = 256;  // threads of a workgroup
constexpr int kEach = 4;    // chunks of keys and as many of values a thread has in flight

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct AppendArgs {
  const uint16_t *k, *v;
  uint16_t *pool_k, *pool_v;
  const int64_t* slots;
  float* weights;
  int32_t* positions;
  const int32_t* at;
  int64_t k_t, k_h, v_t, v_h;
  int64_t k_p, k_s, k_ph, v_p, v_s, v_ph;
  int64_t w_p, w_h, p_p, p_h;
  int64_t T;
  int32_t S, C, per;  // C: 16-byte chunks of a row, per: of a token
  int64_t limit;      // slots of the pool
  PageDiv div_per, div_c, div_s;
};

// A chunk of a key row and the same of a value row a thread, consecutive
// threads along a token's rows.
__global__ __launch_bounds__(kCopy) void append_kernel(AppendArgs a) {
  const int64_t i0 = int64_t(blockIdx.x) * (kCopy * kEach);
  const int64_t t0 = i0 / a.per;
  const int rest = int(i0 - t0 * a.per);
  u32x4 k[kEach], v[kEach];
  int64_t slot[kEach];
  int head[kEach], chunk[kEach];
  int64_t token[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int x = rest + e * kCopy + int(threadIdx.x);
    const int dt = page_index(a.div_per, x);
    const int y = x - dt * a.per;
    head[e] = page_index(a.div_c, y);
    chunk[e] = y - head[e] * a.C;
    token[e] = t0 + dt;
    const bool in = token[e] < a.T;
    const int64_t t = in ? token[e] : 0;
    slot[e] = in ? a.slots[t] : -1;
    k[e] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(a.k + t * a.k_t + head[e] * a.k_h + 8 * chunk[e]));
    v[e] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(a.v + t * a.v_t + head[e] * a.v_h + 8 * chunk[e]));
  }
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    if (slot[e] < 0 || slot[e] >= a.limit) continue;
    const int64_t page = a.limit < (int64_t(1) << 31) ? page_index(a.div_s, int(slot[e])) : slot[e] / a.S;
    const int64_t s = slot[e] - page * a.S;
    *reinterpret_cast<u32x4*>(a.pool_k + page * a.k_p + s * a.k_s + head[e] * a.k_ph + 8 * chunk[e]) = k[e];
    *reinterpret_cast<u32x4*>(a.pool_v + page * a.v_p + s * a.v_s + head[e] * a.v_ph + 8 * chunk[e]) = v[e];
    if (chunk[e] == 0) {
      if (a.weights) a.weights[page * a.w_p + head[e] * a.w_h + s] = 0.f;
      if (a.positions) a.positions[page * a.p_p + head[e] * a.p_h + s] = a.at[token[e]];
    }
  }
}

}  // namespace

hipError_t launch_reserve(const KvView& c, const ReserveCall& r, hipStream_t s) {
  ReserveArgs a{};
  a.table = const_cast<int32_t*>(c.table);
  a.lengths = const_cast<int32_t*>(c.lengths);
  a.counts = r.counts;
  a.free_pages = r.free_pages;
  a.free_count = r.free_count;
  a.starts = r.starts;
  a.granted = r.granted;
  a.slots = r.slots;
  a.table_b = c.table_b;
  a.tokens = r.tokens;
  a.B = int(c.B);
  a.S = int(c.S);
  a.pages = int(c.pages);
  a.per_seq = int(c.per_seq);
  a.cap = int(c.per_seq * c.S);
  a.room = int(r.free_size);
  a.div = page_div(c.S);
  reserve_kernel<<<1, kThreads, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.tokens <= kOwnSlots) return e;
  slots_kernel<<<dim3(uint32_t((a.tokens + kFill - 1) / kFill)), kFill, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_append(const KvView& c, const AppendCall& r, hipStream_t s) {
  AppendArgs a{};
  a.k = r.k;
  a.v = r.v;
  a.k_t = r.k_t;
  a.k_h = r.k_h;
  a.v_t = r.v_t;
  a.v_h = r.v_h;
  a.pool_k = c.k;
  a.pool_v = c.v;
  a.k_p = c.k_p;
  a.k_s = c.k_s;
  a.k_ph = c.k_h;
  a.v_p = c.v_p;
  a.v_s = c.v_s;
  a.v_ph = c.v_h;
  a.slots = r.slots;
  a.weights = r.weights;
  a.positions = r.positions;
  a.at = r.at;
  a.w_p = r.w_p;
  a.w_h = r.w_h;
  a.p_p = r.p_p;
  a.p_h = r.p_h;
  a.T = r.T;
  a.S = int(c.S);
  a.C = int(c.D / 8);
  a.per = int(c.Hkv * a.C);
  a.limit = c.pages * c.S;
  a.div_per = page_div(a.per);
  a.div_c = page_div(a.C);
  a.div_s = page_div(c.S);
  const int64_t blocks = (r.T * a.per + kCopy * kEach - 1) / (kCopy * kEach);
  append_kernel<<<dim3(uint32_t(blocks)), kCopy, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace swm
