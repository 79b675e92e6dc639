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
// in registers.  The slots of the added tokens follow from the same sums: a page just
// taken is read from the list of free ones, not from the table.  All of it is a
// chain of a few latencies: 16 sequences 5.1 us (8.0 with the sums by shuffles and
// the slots by the table); 256 of which a quarter ends and a quarter begins, 8192 pages
// back and 8192 out, 14 us (28 with one page a thread at a time).  More than 4096
// slots are filled by a second launch (4 us) from the table.

constexpr int kThreads = 1024;  // of the planning workgroup: sequences of a round
constexpr int kOwnSlots = 4 * kThreads;  // slots that it fills itself
constexpr int kRun = 4;         // pages a thread takes or gives back at a time
constexpr int kFill = 256;      // threads of a workgroup that fills slots, and tokens of it
constexpr int kHeld = 4096;     // sequences whose starts it holds in LDS

struct ReserveArgs {
  int32_t *table, *lengths;
  const int32_t* counts;
  int32_t *free_pages, *free_count, *starts, *granted;
  int64_t* slots;
  int64_t table_b, tokens;
  int32_t B, S, pages, cap, room;  // room: entries of free_pages
  PageDiv div;
};

struct Step {
  int old, want, had, has;
};
__device__ __forceinline__ Step step_of(const ReserveArgs& a, int b, int* count) {
  Step s{0, 0, 0, 0};
  *count = 0;
  if (b >= a.B) return s;
  *count = a.counts[b];
  s.old = min(max(a.lengths[b], 0), a.cap);
  const int64_t want = int64_t(s.old) + *count;
  s.want = want > a.cap ? s.old : int(max(want, int64_t(0)));
  s.had = s.old > 0 ? page_index(a.div, s.old - 1) + 1 : 0;
  s.has = s.want > 0 ? page_index(a.div, s.want - 1) + 1 : 0;
  return s;
}

// Sums of three numbers below 2^31 over the workgroup's threads up to and
// including this one, and of all, by halves of 16 bits, so that 1024 of them
// stay within 32 bits.  part: where the waves leave theirs, another half every
// other time, so that one barrier is enough.
constexpr int kParts = kThreads / 64;  // 16, a row of lanes
struct Three {
  int64_t upto[3], all[3];
};
__device__ __forceinline__ Three scan_three(int x, int y, int z, uint32_t (*part)[6 * kParts], int* turn) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t* p = part[*turn];
  *turn ^= 1;
  uint32_t v[6] = {uint32_t(x) & 0xffffu, uint32_t(x) >> 16, uint32_t(y) & 0xffffu,
                   uint32_t(y) >> 16,     uint32_t(z) & 0xffffu, uint32_t(z) >> 16};
#pragma unroll
  for (int e = 0; e < 6; ++e) {
    v[e] = scan_wave(v[e]);
    if (lane == 63) p[e * kParts + wave] = v[e];
  }
  __syncthreads();
  // lanes 16 e .. + 15: the waves' sums of half e (e < 4), and of 4 and 5
  const uint32_t a = scan_wave_rows(p[lane]), b = scan_wave_rows(p[4 * kParts + (lane & 31)]);
  Three r;
#pragma unroll
  for (int e = 0; e < 3; ++e) {
    uint32_t before[2], all[2];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int row = 2 * e + f;
      const uint32_t sums = row < 4 ? a : b;
      const int first = 16 * (row < 4 ? row : row - 4);
      all[f] = __builtin_amdgcn_readlane(sums, first + kParts - 1);
      before[f] = wave ? __builtin_amdgcn_readlane(sums, first + (wave ? wave - 1 : 0)) : 0;
    }
    r.upto[e] = ((int64_t(before[1]) + v[2 * e + 1]) << 16) + before[0] + v[2 * e];
    r.all[e] = (int64_t(all[1]) << 16) + all[0];
  }
  return r;
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
  __shared__ int64_t upto[kThreads];   // pages of the round's sequences, summed
  __shared__ int64_t rows[kThreads];   // added tokens, summed
  __shared__ int32_t first[kThreads];  // where a sequence's pages go
  __shared__ int32_t old[kThreads], got[kThreads];
  __shared__ uint32_t part[2][6 * kParts];
  const int tid = threadIdx.x;
  const bool one = a.B <= kThreads;  // all sequences in one round: nothing is read again
  int turn = 0;
  int64_t have = min(max(a.free_count[0], 0), a.room);
  Step s{};
  int count = 0;
  Three sums{};
  // pages that come back
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    s = step_of(a, b0 + tid, &count);
    sums = scan_three(max(s.had - s.has, 0), max(s.has - s.had, 0), max(count, 0), part, &turn);
    const int64_t total = sums.all[0];
    if (total == 0) continue;
    upto[tid] = sums.upto[0];
    first[tid] = s.has;
    __syncthreads();
    for (int64_t i0 = 0; i0 < total; i0 += kRun * kThreads) {
      const int64_t i = i0 + kRun * tid;
      int page[kRun], some = 0;
      int x = i < total ? first_above(upto, kThreads, i) : 0;
#pragma unroll
      for (int e = 0; e < kRun; ++e) {
        page[e] = -1;
        if (i + e >= total) continue;
        while (upto[x] <= i + e) ++x;
        int32_t* entry = a.table + int64_t(b0 + x) * a.table_b + first[x] + (i + e - (x ? upto[x - 1] : 0));
        page[e] = *entry;
        *entry = -1;
      }
#pragma unroll
      for (int e = 0; e < kRun; ++e) some += page[e] >= 0 && page[e] < a.pages;
      const Three p = scan_three(some, 0, 0, part, &turn);
      int64_t at = have + p.upto[0] - some;
#pragma unroll
      for (int e = 0; e < kRun; ++e)
        if (page[e] >= 0 && page[e] < a.pages) {
          if (at < a.room) a.free_pages[at] = page[e];
          ++at;
        }
      have = min(have + p.all[0], int64_t(a.room));
    }
    __syncthreads();
  }
  __threadfence_block();
  __syncthreads();
  // pages that are taken, lengths, starts
  int64_t taken = 0, asked = 0, packed = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + tid;
    if (!one) {
      s = step_of(a, b, &count);
      sums = scan_three(0, max(s.has - s.had, 0), max(count, 0), part, &turn);
    }
    const int need = max(s.has - s.had, 0);
    const int64_t u = asked + sums.upto[1], p = packed + sums.upto[2];
    const bool fits = need == 0 || u <= have;
    const int more = fits ? s.want - s.old : 0;
    if (b < a.B) {
      a.lengths[b] = s.old + more;
      a.granted[b] = more;
      a.starts[b + 1] = int32_t(min(p, int64_t(0x7fffffff)));
      if (b == 0) a.starts[0] = 0;
    }
    upto[tid] = u;
    rows[tid] = p;
    first[tid] = s.had;
    old[tid] = s.old;
    got[tid] = more;
    const Three f = scan_three(fits ? need : 0, 0, 0, part, &turn);  // its barrier is the lists' too
    const int64_t here = asked + f.all[0];
    for (int64_t i = asked + kRun * tid; i < here; i += kRun * kThreads) {
      int x = first_above(upto, kThreads, i);
#pragma unroll
      for (int e = 0; e < kRun; ++e) {
        if (i + e >= here) break;
        while (upto[x] <= i + e) ++x;
        a.table[int64_t(b0 + x) * a.table_b + first[x] + (i + e - (x ? upto[x - 1] : asked))] =
            a.free_pages[have - 1 - (i + e)];
      }
    }
    if (!one) __syncthreads();
    taken += f.all[0];
    asked += sums.all[1];
    packed += sums.all[2];
  }
  if (tid == 0) {
    a.free_count[0] = int32_t(have - taken);
    if (a.B == 0) a.starts[0] = 0;
  }
  if (a.tokens > kOwnSlots) return;
  if (!one) {
    __threadfence_block();
    __syncthreads();
  }
  for (int64_t i = tid; i < a.tokens; i += kThreads) {
    int64_t slot = -1;
    if (i < packed) {
      if (one) {
        const int b = first_above(rows, a.B, i);
        if (got[b] > 0) {
          const int at = old[b] + int(i - (b ? rows[b - 1] : 0)), x = page_index(a.div, at);
          // a page just taken comes from the list of free ones: the table's entry may be on its way
          const int page = x >= first[b] ? a.free_pages[have - 1 - ((b ? upto[b - 1] : 0) + x - first[b])]
                                         : a.table[int64_t(b) * a.table_b + x];
          if (page >= 0 && page < a.pages) slot = int64_t(page) * a.S + (at - x * a.S);
        }
      } else {
        const int b = first_above(a.starts + 1, a.B, i);
        const int g = a.granted[b];
        if (g > 0) slot = slot_of(a, b, a.lengths[b] - g + int(i - a.starts[b]));
      }
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
// threads along a token's rows, four of each on their way: bound by memory (8 x
// 2048 tokens, 8 heads of 128: 134 MB read and written in 23.5 us), or by one
// latency and a launch (16 tokens 4.2 us).
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
