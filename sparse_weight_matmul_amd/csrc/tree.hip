// Attention of drafted tokens over a paged key-value cache that holds their
// keys and values behind the sequence's own.
//
//   x_it = scale * q_i . k_t ;  o_i = sum_t e^(x_it - m_i) v_t / sum_t e^(x_it - m_i)
//
// over the tokens t before the drafted ones, i itself, its parent, the parent's
// parent and so on, as far as they are live (on a page of the pool, not masked).
//
// The rows of one key-value head, drafted tokens x query heads of its group, go
// over the same tokens.  Up to 32 of them are bound by the read of the cache (16
// ragged x 4096 tokens, 8 drafted: 528 MB in 103 us, 5.1 TB/s; a wave waits for
// its tile and nothing else, so 128 KiB of a CU's LDS are on their way), hundreds by
// the matrix cores (2 x 131072, 64 drafted, eight heads to a group: 550 GFLOP in
// 590 to 620 us, and 12 for the join).  Which of the two kernels runs goes by the
// rows that max_tokens allows.  16 x 4096 tokens, 32 heads on 8: 32 rows 72 us (3.8
// TB/s), 36 rows 64, 64 rows 68, 96 rows 74, 128 rows 79.  Rows above 128 halves leave
// room for one workgroup of four waves on a CU: 16 x 4096, 8 drafted, 32 heads of 192
// 312 us (5.2 TB/s), of 256 379 (5.7); 2 x 32768, 32 drafted, 32 heads of 256 on 8 152
// (0.45 PFLOP/s).  Registers spill where these instances for rows above 192 halves
// have no more (16 to 24 of a lane), and 6 or 8 in those for few query rows of up to 64
// halves, which keep four waves on a SIMD: 16 ragged x 4096, 32 heads of 64 82 us (3.2 TB/s).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "flash.h"
#include "kernels.h"
#include "paging.h"
#include "wave.h"

namespace swm {
namespace {

using namespace flash;

constexpr int kBlock = 4 * kRows;  // query rows of a workgroup of four waves
// waves over few query rows, so that their tiles fill LDS
constexpr int few_waves(int chunks) { return chunks == 32 ? 4 : 8; }
constexpr int max_of(int a, int b) { return a > b ? a : b; }
constexpr int kMaxCut = 128;            // sequences whose lengths a wave holds, two a lane

struct TreeArgs {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  const int32_t *starts, *parents, *table, *lengths;
  const uint8_t* mask;
  int32_t* plan;  // first piece and number of pieces of each sequence
  float* ml;      // [piece][key-value head][row][2] maximum (in units of log2) and sum
  float* part;    // [piece][key-value head][row][D] unnormalised outputs
  int64_t q_t, q_h, o_t, o_h;
  int64_t k_p, k_s, k_h, v_p, v_s, v_h;
  int64_t table_b, mask_b;
  // Which of these are neighbours decides how they are loaded: with room here and order
  // behind it, 35 drafted tokens over 3 x 92955, eight heads of 64 on two, take 70.0 us for 67.0.
  int32_t B, T, Hq, Hkv, G, D, S, pages, cap, most;
  int32_t order;        // whole sequences, the longest first
  int32_t room;         // pieces of all sequences at most; 0: every sequence is one
  int32_t tiles, rows;  // workgroups along a unit's rows; rows of a piece in the workspace
  float c;
  uint32_t flip;
  bool zero;
  PageDiv div, per_g, per_pair, per_hkv;
};

// A sequence's drafted tokens: packed rows *first .. + *n - 1.
__device__ __forceinline__ void drafted(const TreeArgs& a, int b, int* first, int* n) {
  const int s0 = min(max(a.starts[b], 0), a.T), s1 = min(max(a.starts[b + 1], 0), a.T);
  *first = s0;
  *n = min(max(s1 - s0, 0), a.most);
}

// Lane `from`'s value.
__device__ __forceinline__ uint64_t pick(uint64_t v, int from) {
  return uint64_t(uint32_t(__shfl(uint32_t(v >> 32), from))) << 32 | uint32_t(__shfl(uint32_t(v), from));
}

// Which drafted tokens the lane's one sees: bit j for token j.  Every lane
// starts with itself and its parent; each round adds what the farthest one seen
// so far sees: 2, 4, .. generations.  A parent that is not before its child is none.
__device__ __forceinline__ int parent_of(const TreeArgs& a, int first, int n, int lane) {
  return lane < n ? a.parents ? a.parents[first + lane] : lane - 1 : -1;
}
__device__ __forceinline__ uint64_t ancestors(int up, int lane) {
  uint64_t sees = uint64_t(1) << lane;
  if (up >= lane) up = -1;
#pragma unroll
  for (int r = 0; r < 6; ++r) {
    const int from = max(up, 0);
    const uint64_t more = pick(sees, from);
    const int next = __shfl(up, from);
    if (up >= 0) {
      sees |= more;
      up = next;
    }
  }
  return sees;
}

// What lane l holds of sequences 2 l and 2 l + 1: the packed rows of their drafted
// tokens, how many they are, and their tokens (none of all that past the batch).
struct Held {
  int first[2], drafts[2], n[2];
};
__device__ __forceinline__ Held hold(const TreeArgs& a, int lane) {
  Held x;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int b = min(2 * lane + e, a.B - 1);
    drafted(a, b, &x.first[e], &x.drafts[e]);
    x.n[e] = min(max(a.lengths[b], 0), a.cap);
    if (2 * lane + e >= a.B) x.drafts[e] = x.n[e] = 0;
  }
  return x;
}
// Tokens of a sequence in units of kUnit (64 or more), one at least where it has
// drafted ones: below 2^25, so that 128 of them add up in 32 bits.
template <int kUnit>
__device__ __forceinline__ uint32_t units_of(const Held& x, int e) {
  return x.drafts[e] ? max((x.n[e] + kUnit - 1) / kUnit, 1) : 0;
}

// The pieces that the sequences are cut into: `each` units, the fewest (two at
// least) with which they are a.room in all.  Lane l has sequences 2 l and 2 l +
// 1, pieces first .. mid - 1 and mid .. last - 1.  A quotient that is one off
// only moves the last piece's end.
struct Cuts {
  uint32_t each;
  int first, mid, last;
};
template <int kUnit>
__device__ __forceinline__ Cuts cut(const TreeArgs& a, const Held& x) {
  const uint32_t t0 = units_of<kUnit>(x, 0), t1 = units_of<kUnit>(x, 1);
  const uint32_t total = wave_sum(t0 + t1), room = a.room;
  uint32_t c0, c1;
  auto count = [&](uint32_t q) {
    const float inv = 1.f / float(q);
    c0 = t0 ? max(uint32_t(float(t0 + q - 1) * inv), 1u) : 0;
    c1 = t1 ? max(uint32_t(float(t1 + q - 1) * inv), 1u) : 0;
    return wave_sum(c0 + c1);
  };
  uint32_t q = max((total + room - 1) / room, 2u);
  if (count(q) > room) {
    uint32_t low = q;
    q = max(uint32_t(wave_max(int(max(t0, t1)))), low + 1);  // whole sequences fit
    while (q - low > max(low / 16, 1u)) {
      const uint32_t mid = low + (q - low) / 2;
      if (count(mid) > room)
        low = mid;
      else
        q = mid;
    }
    count(q);
  }
  Cuts r;
  const uint32_t upto = scan_wave(c0 + c1);
  r.each = q;
  r.last = int(upto);
  r.mid = int(upto - c1);
  r.first = int(upto - c1 - c0);
  return r;
}

// The sequence that comes i-th by length, the longest first.
template <int kUnit>
__device__ __forceinline__ int by_length(const TreeArgs& a, const Held& x, int lane, int i) {
  // unique keys: units, then the lower sequence; those past the batch have none below them
  auto key = [&](int e) {
    const int b = 2 * lane + e;
    return b < a.B ? units_of<kUnit>(x, e) << 7 | uint32_t(127 - b) : 0u;
  };
  const uint32_t k0 = key(0), k1 = key(1);
  int r0 = 0, r1 = 0;
  for (int l = 0; l < (a.B + 1) / 2; ++l) {
    const uint32_t y = __builtin_amdgcn_readlane(k0, l), z = __builtin_amdgcn_readlane(k1, l);
    r0 += int(y > k0) + int(z > k0);
    r1 += int(y > k1) + int(z > k1);
  }
  const uint64_t in0 = __builtin_amdgcn_ballot_w64(2 * lane < a.B && r0 == i);
  const uint64_t in1 = __builtin_amdgcn_ballot_w64(2 * lane + 1 < a.B && r1 == i);
  return in0 ? 2 * __builtin_ctzll(in0) : 2 * __builtin_ctzll(in1) + 1;
}

// What a workgroup does: tokens begin .. end - 1 of sequence b (n in all) and
// key-value head hkv, for the query rows from m0 on of the sequence's `rows`.
struct Work {
  int b, hkv, m0, rows, first, drafts, n, begin, end;
  int piece, count;  // which piece of all sequences' this is, and how many the sequence has
};
template <int kUnit, int kBlock>
__device__ __forceinline__ bool find_work(const TreeArgs& a, int lane, int wave, Work* w) {
  // Workgroups go round the eight XCDs: those that read the same tokens are
  // eight apart, so that they share an L2.
  const int group = page_index(a.per_pair, blockIdx.x), rest = blockIdx.x - group * 8 * a.tiles;
  const int pair = group * 8 + (rest & 7);
  w->m0 = (rest >> 3) * kBlock;
  w->piece = page_index(a.per_hkv, pair);
  w->hkv = pair - w->piece * a.Hkv;
  if (w->piece >= (a.room > 0 ? a.room : a.B)) return false;
  int b = w->piece, nth = 0;
  w->count = 1;
  uint32_t each = 0;
  if (a.room > 0 || a.order) {
    const Held x = hold(a, lane);
    if (a.room > 0) {
      const Cuts c = cut<kUnit>(a, x);
      if (blockIdx.x == 0 && wave == 0) {
        if (2 * lane < a.B) {
          a.plan[4 * lane] = c.first;
          a.plan[4 * lane + 1] = c.mid - c.first;
        }
        if (2 * lane + 1 < a.B) {
          a.plan[4 * lane + 2] = c.mid;
          a.plan[4 * lane + 3] = c.last - c.mid;
        }
      }
      const uint64_t in = __builtin_amdgcn_ballot_w64(w->piece >= c.first && w->piece < c.last);
      if (in == 0) return false;  // more workgroups than pieces
      const int l = __builtin_ctzll(in);
      const int from = __builtin_amdgcn_readlane(c.first, l), mid = __builtin_amdgcn_readlane(c.mid, l);
      const bool second = w->piece >= mid;
      b = 2 * l + second;
      nth = w->piece - (second ? mid : from);
      w->count = second ? __builtin_amdgcn_readlane(c.last, l) - mid : mid - from;
      each = __builtin_amdgcn_readfirstlane(c.each) * kUnit;
    } else {
      b = by_length<kUnit>(a, x, lane, w->piece);
    }
    w->b = b = __builtin_amdgcn_readfirstlane(b);
    const bool odd = b & 1;
    w->first = __builtin_amdgcn_readlane(odd ? x.first[1] : x.first[0], b >> 1);
    w->drafts = __builtin_amdgcn_readlane(odd ? x.drafts[1] : x.drafts[0], b >> 1);
    w->n = __builtin_amdgcn_readlane(odd ? x.n[1] : x.n[0], b >> 1);
  } else {
    w->b = b = __builtin_amdgcn_readfirstlane(b);
    drafted(a, b, &w->first, &w->drafts);
    w->first = __builtin_amdgcn_readfirstlane(w->first);
    w->drafts = __builtin_amdgcn_readfirstlane(w->drafts);
    w->n = __builtin_amdgcn_readfirstlane(min(max(a.lengths[b], 0), a.cap));
  }
  w->rows = w->drafts * a.G;
  w->begin = __builtin_amdgcn_readfirstlane(int(min(int64_t(nth) * each, int64_t(w->n))));
  w->end = __builtin_amdgcn_readfirstlane(
      nth == w->count - 1 ? w->n : int(min(int64_t(nth + 1) * each, int64_t(w->n))));
  return w->m0 < w->rows;
}

// A query row: token `token` of the drafted ones, query head `head`.
struct Row {
  int token, head;
};
__device__ __forceinline__ Row row_of(const TreeArgs& a, const Work& w, int m) {
  Row r;
  r.token = page_index(a.per_g, m);
  r.head = w.hkv * a.G + m - r.token * a.G;
  return r;
}
__device__ __forceinline__ const uint16_t* query_of(const TreeArgs& a, const Work& w, const Row& r) {
  return a.q + int64_t(w.first + r.token) * a.q_t + int64_t(r.head) * a.q_h;
}

// The cache as one workgroup sees it.
struct Source {
  const int32_t* row;
  const uint8_t* mask;
  const uint16_t *k, *v;
  int end;
};
__device__ __forceinline__ Source source_of(const TreeArgs& a, const Work& w) {
  Source s;
  s.row = a.table + int64_t(w.b) * a.table_b;
  s.mask = a.mask ? a.mask + int64_t(w.b) * a.mask_b : nullptr;
  s.k = a.k + int64_t(w.hkv) * a.k_h;
  s.v = a.v + int64_t(w.hkv) * a.v_h;
  s.end = w.end;
  return s;
}
// The page of token t, always one of the pool; the top bit is set where the token is not live.
constexpr int kDead = int(0x80000000u), kPage = 0x7fffffff;
__device__ __forceinline__ int place_of(const TreeArgs& a, int id, bool on) {
  return id < 0 || id >= a.pages ? kDead : on ? id : id | kDead;
}
__device__ __forceinline__ int place(const TreeArgs& a, const Source& s, int t) {
  if (t >= s.end) return kDead;
  return place_of(a, s.row[page_index(a.div, t)], !s.mask || s.mask[t] != 0);
}

// A tile's loads into LDS, straight, N of 1 KiB from the keys and as many from the
// values: load i brings rows r0 + i step .. + 64 / C - 1 of the tile from token t0 on,
// where lane l holds the place of token t0 + l.  Every lane finds the addresses of its
// token's rows (a scalar calculation for every load, 50 instructions each, took
// a third of the time); kUniform: the rows of a load are on one page, so that its
// first row's address serves.  Value rows of tokens that are not live become
// zeros, as their weight is.
template <int C, int N, bool kUniform>
__device__ __forceinline__ void load_tile(const TreeArgs& a, const Source& s, int t0, int places, int lane, int r0,
                                          int step, uint16_t* dk, uint16_t* dv) {
  const uint64_t live = __builtin_amdgcn_ballot_w64(places >= 0);
  const int t = t0 + lane, slot = t - page_index(a.div, t) * a.S, page = places & kPage;
  const uint64_t ka = reinterpret_cast<uint64_t>(s.k + page * a.k_p + slot * a.k_s);
  const uint64_t va = reinterpret_cast<uint64_t>(s.v + page * a.v_p + slot * a.v_s);
  const int lr = lane / C, lc = lane % C;
  const uint32_t to_k = lds_address(dk), to_v = lds_address(dv);
  auto offsets = [&](int i, uint32_t* k, uint32_t* v) {  // from the row's address, or that of the load's first row
    const int rw = r0 + i * step + lr;
    *k = key_chunk<C>(rw, lc) * 16 + (kUniform ? uint32_t(lr * int(a.k_s)) * 2 : 0);
    *v = value_chunk<C>(rw, lc) * 16 + (kUniform ? uint32_t(lr * int(a.v_s)) * 2 : 0);
  };
  auto from = [&](uint64_t at, int i) -> uint64_t {
    const int r = r0 + i * step;
    if (kUniform)
      return uint64_t(uint32_t(__builtin_amdgcn_readlane(int(at >> 32), r))) << 32 |
             uint32_t(__builtin_amdgcn_readlane(int(at), r));
    return pick(at, r + lr);
  };
  if (~live == 0 && a.D == C * 8) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint32_t k, v;
      offsets(i, &k, &v);
      if (kUniform) {
        to_lds(from(ka, i), k, to_k + i * step * C * 16);
        to_lds(from(va, i), v, to_v + i * step * C * 16);
      } else {
        to_lds(from(ka, i) + k, to_k + i * step * C * 16);
        to_lds(from(va, i) + v, to_v + i * step * C * 16);
      }
    }
    return;
  }
  // Keys of tokens that are not live may hold anything: their scores are not used.
  bool none = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t k, v;
    offsets(i, &k, &v);
    const int rw = r0 + i * step + lr;
    const bool on = (live >> rw) & 1;
    to_lds_some(from(ka, i) + k, to_k + i * step * C * 16,
                __builtin_amdgcn_ballot_w64(key_chunk<C>(rw, lc) * 8 < a.D));
    const uint64_t v_on = __builtin_amdgcn_ballot_w64(on && value_chunk<C>(rw, lc) * 8 < a.D);
    const uint64_t vi = from(va, i) + v;
    if (v_on)
      to_lds_some(vi, to_v + i * step * C * 16, v_on);
    else
      none = true;
    if (!on) *reinterpret_cast<u32x4*>(dv + i * step * C * 8 + lane * 8) = u32x4{0, 0, 0, 0};
  }
  if (none) wait_vm<0>();  // fewer are on their way than those who count them think
}

// Scores of tokens that the lane's row does not see become -inf: those that
// are not live, and drafted ones that are none of its ancestors.  own: tokens before
// the drafted ones.
template <int NB>
__device__ __forceinline__ void hide(f32x16 (&s)[NB], uint64_t live, uint64_t sees, int t0, int own, int h) {
  if (t0 + 32 * NB > own) {
    const int rel = own - t0;  // drafted token j is token rel + j of the tile, rel < 64
    uint64_t tree = rel >= 0 ? sees << rel : rel > -64 ? sees >> -rel : 0;
    if (rel > 0) tree |= (uint64_t(1) << rel) - 1;
    live &= tree;
  }
  live >>= 4 * h;
#pragma unroll
  for (int e = 0; e < NB; ++e)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (!((uint32_t(live >> (32 * e)) >> (8 * (i >> 2) + (i & 3))) & 1)) s[e][i] = neg_inf();
}

// What clear_odd took out of the value row of drafted token t, for the rows that see it.
template <int ND>
__device__ __forceinline__ void add_odd(const TreeArgs& a, const Source& s, uint64_t sees, int t, int own, int h,
                                        State<ND>& st) {
  const int p = place(a, s, t);
  if (p < 0 || !((sees >> (t - own)) & 1)) return;
  const uint16_t* src = s.v + p * a.v_p + (t - page_index(a.div, t) * a.S) * a.v_s;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int e = 32 * d + 8 * (i >> 2) + 4 * h + (i & 3);
      if (e >= a.D) continue;
      const uint16_t x = src[e];
      if ((x & 0x7c00) == 0x7c00) st.o[d][i] += float(__builtin_bit_cast(_Float16, x));
    }
}

// Many query rows, 32 a wave, over tiles of 64 tokens that the waves share:
// kBufs of them in LDS, all but one on their way.  Table entries and mask bytes
// come through LDS too, kAhead tiles ahead: a wave that waited for one in a
// register would wait for every tile requested before it (2 x 131072 tokens: 822
// us, 697 without reading the table at all).
constexpr int kRing = 8;  // tiles whose entries LDS holds
template <int NK, int ND, int C, int W, int kBufs, bool kUniform>
__global__ __launch_bounds__(64 * W, ND <= 4 ? 2 : 1) void tree_kernel(TreeArgs a) {
  constexpr int kTile = kTokens * C * 8;  // halves
  extern __shared__ uint16_t smem[];
  uint16_t* sk = smem;                  // [kBufs][kTile]
  uint16_t* sv = smem + kBufs * kTile;  // [kBufs][kTile]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, h = lane >> 5;
  Work w;
  if (!find_work<kTokens, W * kRows>(a, lane, wave, &w)) return;
  const Source src = source_of(a, w);
  const int begin = w.begin, end = w.end;
  const int own = w.n - w.drafts;  // negative where the length does not count all the drafted ones
  const int m = w.m0 + wave * kRows + r;
  const bool idle = w.m0 + wave * kRows >= w.rows;
  // requested before the tiles, which whoever waits for these would wait for too
  const Row mine = row_of(a, w, min(m, w.rows - 1));
  const int parent = parent_of(a, w.first, w.drafts, lane);
  half8 q[NK];
  load_query(query_of(a, w, mine), a.D, h, q);

  // Key dimensions that only pad the products: zeros, never loaded.
  if (a.D < 16 * NK) {
    for (int i = threadIdx.x; i < kBufs * kTile / 8; i += 64 * W)
      *reinterpret_cast<u32x4*>(sk + i * 8) = u32x4{0, 0, 0, 0};
    __syncthreads();
  }
  auto load = [&](int t0, int places, int buf) {
    constexpr int kSpan = 64 / C;  // rows of a load
    load_tile<C, C / W, kUniform>(a, src, t0, places, lane, wave * kSpan, W * kSpan,
                                  sk + buf * kTile + wave * 512, sv + buf * kTile + wave * 512);
  };
  // Table entries and mask of a tile, 64 / W tokens a wave.
  constexpr int kAhead = 2 * kBufs - 1, kShare = 64 / W;
  const int32_t* ring = reinterpret_cast<const int32_t*>(smem + 2 * kBufs * kTile);  // [kRing][2][64]
  const uint32_t ring_to = lds_address(smem + 2 * kBufs * kTile);
  const bool masked = src.mask != nullptr;
  auto request = [&](int t0) {  // past the end the last token's, so that there is always something to count
    const int t = t0 + wave * kShare + lane;
    const uint64_t on = __builtin_amdgcn_ballot_w64(lane < kShare);
    const uint32_t to = ring_to + (uint32_t(t0 - begin) / kTokens % kRing * 2 * 64 + wave * kShare) * 4;
    const int x = min(t, end - 1);
    word_to_lds(src.row + page_index(a.div, x), to, on);
    if (masked) byte_to_lds(src.mask + x, to + 64 * 4, on);
  };
  auto requested = [&](int t0) {
    const int32_t* e = ring + uint32_t(t0 - begin) / kTokens % kRing * 2 * 64 + lane;
    const int id = e[0], on = masked ? e[64] : 1;
    return t0 + lane < end ? place_of(a, id, on != 0) : kDead;
  };
  // places of the tile at hand and of the kBufs - 1 after it
  int places[kBufs];
#pragma unroll
  for (int i = 0; i < kBufs; ++i) places[i] = place(a, src, begin + i * kTokens + lane);
#pragma unroll
  for (int i = kBufs; i < kAhead; ++i)
    if (begin < end) request(begin + i * kTokens);
#pragma unroll
  for (int i = 0; i < kBufs - 1; ++i)
    if (begin + i * kTokens < end) load(begin + i * kTokens, places[i], i);

  const uint64_t sees = pick(ancestors(parent, lane), mine.token);
  mend_query(a.D, h, a.zero, a.flip, q);
  const Reads<NK, ND, C> at(smem, lane, kBufs * kTile * 2);
  State<ND> st;
  st.clear();
  bool odd = false;
  // One tile, in buffer `buf`.
  auto step = [&](int t0, auto constant) {
    constexpr int buf = decltype(constant)::value;
    const uint64_t live = __builtin_amdgcn_ballot_w64(places[0] >= 0);
    // what was requested after this tile may be on its way, as long as it is the same every time
    constexpr int kTiles = (kBufs - 2) * 2 * (C / W);
    if (kBufs == 2 || t0 + (kBufs - 2) * kTokens >= end)
      wait_vm<0>();
    else if (masked)
      wait_vm<kTiles + 2 * (kBufs - 2)>();
    else
      wait_vm<kTiles + (kBufs - 2)>();
    __syncthreads();
    request(t0 + kAhead * kTokens);
    if (t0 + (kBufs - 1) * kTokens < end) load(t0 + (kBufs - 1) * kTokens, places[kBufs - 1], (buf + kBufs - 1) % kBufs);
#pragma unroll
    for (int i = 0; i + 1 < kBufs; ++i) places[i] = places[i + 1];
    places[kBufs - 1] = requested(t0 + kBufs * kTokens);
    const bool drafts_here = t0 + kTokens > own;
    if (drafts_here) {
      // A drafted token's infinity or NaN must not reach rows that do not see
      // it (its weight there is zero): zeros in its place, added at the end.
      uint16_t* vt = sv + buf * kTile;
      bool bad = false;
      for (int i = threadIdx.x; i < kTokens * C; i += 64 * W)
        if (t0 + i / C >= own && value_chunk<C>(i / C, i % C) * 8 < a.D) bad |= clear_odd(vt + i * 8);
      odd |= __syncthreads_or(bad);
    }
    if (idle) return;
    f32x16 s[2];
    scores(at, buf * kTile * 2, q, s);
    if (drafts_here || ~live) hide(s, live, sees, t0, own, h);
    half8 p[4];
    weights(st, s, a.c, buf == 0 && t0 == begin, p);
    outputs(st, at, buf * kTile * 2, p);
  };
  if (kBufs > 2) wait_vm<0>();  // the first tiles are followed by fewer requests than later ones
  for (int t0 = begin; t0 < end; t0 += kBufs * kTokens) {
    step(t0, std::integral_constant<int, 0>());
    if (t0 + kTokens < end) step(t0 + kTokens, std::integral_constant<int, 1>());
    if constexpr (kBufs == 4) {
      if (t0 + 2 * kTokens < end) step(t0 + 2 * kTokens, std::integral_constant<int, 2>());
      if (t0 + 3 * kTokens < end) step(t0 + 3 * kTokens, std::integral_constant<int, 3>());
    }
  }
  if (idle) return;
  const float l = sum_halves(st.l);
  if (odd)
    for (int t = max(begin, own); t < end; ++t) add_odd(a, src, sees, t, own, h, st);
  if (m >= w.rows) return;
  if (w.count > 1) {
    const int64_t to = (int64_t(w.piece) * a.Hkv + w.hkv) * a.rows + m;
    if (h == 0) {
      a.ml[2 * to] = st.m * a.c;
      a.ml[2 * to + 1] = l;
    }
    float* dst = a.part + to * a.D;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int e = 32 * d + 2 * i + 4 * h;
        if (e < a.D)
          *reinterpret_cast<float4*>(dst + e) = float4{st.o[d][i], st.o[d][i + 1], st.o[d][i + 2], st.o[d][i + 3]};
      }
    return;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  write_row(st, inv, a.out + int64_t(w.first + mine.token) * a.o_t + int64_t(mine.head) * a.o_h, a.D, h);
}

// Four dimensions of an output row.
__device__ __forceinline__ void write_four(uint16_t* dst, const float4& o, float inv) {
  const half2v lo = __builtin_convertvector(f32x2{o.x * inv, o.y * inv}, half2v);
  const half2v hi = __builtin_convertvector(f32x2{o.z * inv, o.w * inv}, half2v);
  const u32x2 w = {__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
  if ((reinterpret_cast<uintptr_t>(dst) & 7) == 0) {
    *reinterpret_cast<u32x2*>(dst) = w;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) dst[e] = uint16_t(w[e >> 1] >> (16 * (e & 1)));
  }
}

// Few query rows, 32 at most: bound by the read of the cache.  Every wave has
// tiles of its own, 32 tokens in LDS that no other wave looks at, so that there
// is no barrier in the loop and as many bytes on their way as LDS holds; the
// waves' sums are joined at the end.
template <int NK, int ND, int C, int W, bool kUniform>
__global__ __launch_bounds__(64 * W, C == 8 ? 4 : W / 4) void tree_few_kernel(TreeArgs a) {
  constexpr int kTile = 32 * C * 8;  // halves
  constexpr int kRow = 32 * ND + 4;  // floats, off the bank stride
  extern __shared__ uint16_t smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, h = lane >> 5;
  uint16_t* sk = smem + wave * 2 * kTile;
  uint16_t* sv = sk + kTile;
  Work w;
  if (!find_work<32 * W, 32>(a, lane, wave, &w)) return;
  const Source src = source_of(a, w);
  const int end = w.end, own = w.n - w.drafts;
  const int t_first = w.begin + 32 * wave;
  // requested before the tiles, which whoever waits for these would wait for too
  const Row mine = row_of(a, w, min(r, w.rows - 1));
  const int parent = parent_of(a, w.first, w.drafts, lane);
  half8 q[NK];
  load_query(query_of(a, w, mine), a.D, h, q);

  if (a.D < 16 * NK) {
    for (int i = lane; i < kTile / 8; i += 64) *reinterpret_cast<u32x4*>(sk + i * 8) = u32x4{0, 0, 0, 0};
    __syncthreads();
  }
  auto load = [&](int t0, int places) {  // both halves of the wave hold the same places
    load_tile<C, C / 2, kUniform>(a, src, t0, places, lane, 0, 64 / C, sk, sv);
  };
  int now = place(a, src, t_first + r), next = place(a, src, t_first + 32 * W + r);
  if (t_first < end) load(t_first, now);

  const uint64_t sees = pick(ancestors(parent, lane), mine.token);
  mend_query(a.D, h, a.zero, a.flip, q);
  const Reads<NK, ND, C> at(sk, lane, kTile * 2);
  State<ND> st;
  st.clear();
  bool odd = false;
  for (int t0 = t_first; t0 < end; t0 += 32 * W) {
    const uint64_t live = __builtin_amdgcn_ballot_w64(now >= 0) & 0xffffffffu;
    now = next;
    wait_vm<0>();
    asm volatile("" ::: "memory");  // no barrier follows: reads of the tile stay below
    __builtin_amdgcn_sched_barrier(0);
    const bool drafts_here = t0 + 32 > own;
    if (drafts_here) {
      bool bad = false;
      for (int i = lane; i < 32 * C; i += 64)
        if (t0 + i / C >= own && value_chunk<C>(i / C, i % C) * 8 < a.D) bad |= clear_odd(sv + i * 8);
      odd |= __builtin_amdgcn_ballot_w64(bad) != 0;
    }
    f32x16 s[1];
    scores(at, 0, q, s);
    if (drafts_here || live != 0xffffffffu) hide(s, live, sees, t0, own, h);
    half8 p[2];
    weights(st, s, a.c, t0 == t_first, p);
    outputs(st, at, 0, p);
    __builtin_amdgcn_sched_barrier(0);  // the tile has been read: the next one takes its place
    if (t0 + 32 * W < end) load(t0 + 32 * W, now);
    next = place(a, src, t0 + 64 * W + r);
  }
  if (odd)
    for (int t = max(w.begin, own); t < end; ++t)
      if ((t - w.begin) / 32 % W == wave) add_odd(a, src, sees, t, own, h, st);
  const float l = sum_halves(st.l);

  // The waves' sums: four dimensions of a row a thread.
  __syncthreads();
  float* sm_m = reinterpret_cast<float*>(smem);  // [W][32]
  float* sm_l = sm_m + 32 * W;
  float* sm_o = sm_l + 32 * W;  // [W][32][kRow]
  if (h == 0) {
    sm_m[32 * wave + r] = st.m * a.c;
    sm_l[32 * wave + r] = l;
  }
  if (r < w.rows) {
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4*>(sm_o + (32 * wave + r) * kRow + 32 * d + 2 * i + 4 * h) =
            float4{st.o[d][i], st.o[d][i + 1], st.o[d][i + 2], st.o[d][i + 3]};
  }
  __syncthreads();
  constexpr int kPer = 8 * ND;  // threads of a row
  for (int i = threadIdx.x; i < w.rows * kPer; i += 64 * W) {
    const int m = i / kPer, d = i % kPer * 4;
    if (d >= a.D) continue;
    float top = neg_inf();
#pragma unroll
    for (int x = 0; x < W; ++x) top = fmaxf(top, sm_m[32 * x + m]);
    const float base = top == neg_inf() ? 0.f : top;
    float sum = 0.f;
    float4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < W; ++x) {
      const float f = __builtin_amdgcn_exp2f(sm_m[32 * x + m] - base);
      const float4 v = *reinterpret_cast<const float4*>(sm_o + (32 * x + m) * kRow + d);
      sum += f * sm_l[32 * x + m];
      o.x += f * v.x;
      o.y += f * v.y;
      o.z += f * v.z;
      o.w += f * v.w;
    }
    if (w.count > 1) {
      const int64_t to = (int64_t(w.piece) * a.Hkv + w.hkv) * a.rows + m;
      if (d == 0) {
        a.ml[2 * to] = top;
        a.ml[2 * to + 1] = sum;
      }
      *reinterpret_cast<float4*>(a.part + to * a.D + d) = o;
    } else {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const Row it = row_of(a, w, m);
      write_four(a.out + int64_t(w.first + it.token) * a.o_t + int64_t(it.head) * a.o_h + d, o, inv);
    }
  }
}

constexpr int kJoin = 256;

// The pieces of a row added up by a wave: lane p has the maximum and the sum of
// piece p, then `per` lanes take four dimensions each of a piece's outputs, all
// groups of them another piece.  Everything that does not depend on the row's
// place is requested at once.
__global__ __launch_bounds__(kJoin) void tree_join_kernel(TreeArgs a, int per) {
  const int lane = threadIdx.x & 63;
  const int64_t at = int64_t(blockIdx.x) * (kJoin / 64) + (threadIdx.x >> 6);  // packed row and query head
  const int64_t t = at / a.Hq;
  const int qh = int(at - t * a.Hq);
  if (t >= a.T) return;
  // the row's sequence: the last that starts at or before it
  const int s0 = 2 * lane < a.B ? a.starts[2 * lane] : 0x7fffffff;
  const int s1 = 2 * lane + 1 < a.B ? a.starts[2 * lane + 1] : 0x7fffffff;
  const uint64_t in0 = __builtin_amdgcn_ballot_w64(s0 <= t), in1 = __builtin_amdgcn_ballot_w64(s1 <= t);
  if (!(in0 | in1)) return;
  const int b = max(in0 ? 2 * (63 - __builtin_clzll(in0)) : -1, in1 ? 2 * (63 - __builtin_clzll(in1)) + 1 : -1);
  int first, drafts;
  drafted(a, b, &first, &drafts);
  const int from_piece = a.plan[2 * b], pieces = a.plan[2 * b + 1];
  const int i = int(t) - first;
  if (i < 0 || i >= drafts || pieces < 2) return;  // one piece: written already
  const int hkv = page_index(a.per_g, qh);
  const int64_t next = int64_t(a.Hkv) * a.rows;
  const int64_t from = (int64_t(from_piece) * a.Hkv + hkv) * a.rows + int64_t(i) * a.G + (qh - hkv * a.G);
  const float* ml = a.ml + 2 * from;
  float m = neg_inf();
  for (int p = lane; p < pieces; p += 64) m = fmaxf(m, ml[2 * next * p]);
  m = wave_max(m);
  const float base = m == neg_inf() ? 0.f : m;
  float l = 0.f;
  for (int p = lane; p < pieces; p += 64) l += __builtin_amdgcn_exp2f(ml[2 * next * p] - base) * ml[2 * next * p + 1];
  l = wave_sum(l);
  const int d = lane % per * 4, part = lane / per, parts = 64 / per;
  float4 o = {0.f, 0.f, 0.f, 0.f};
  if (d < a.D) {
    const float* src = a.part + from * a.D + d;
    constexpr int kUnroll = 8;
    for (int p0 = part; p0 < pieces; p0 += kUnroll * parts) {
      float4 v[kUnroll];
      float f[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int p = min(p0 + u * parts, pieces - 1);
        v[u] = *reinterpret_cast<const float4*>(src + p * next * a.D);
        f[u] = p0 + u * parts < pieces ? __builtin_amdgcn_exp2f(ml[2 * next * p] - base) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (p0 + u * parts >= pieces) continue;
        o.x += f[u] * v[u].x;
        o.y += f[u] * v[u].y;
        o.z += f[u] * v[u].z;
        o.w += f[u] * v[u].w;
      }
    }
  }
  for (int s = per; s < 64; s *= 2) {
    o.x += __shfl_xor(o.x, s);
    o.y += __shfl_xor(o.y, s);
    o.z += __shfl_xor(o.z, s);
    o.w += __shfl_xor(o.w, s);
  }
  if (part > 0 || d >= a.D) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  write_four(a.out + t * a.o_t + int64_t(qh) * a.o_h + d, o, inv);
}

template <int NK, int ND, int C, bool kUniform>
hipError_t launch_as(const TreeArgs& a, bool few, bool wide, uint32_t grid, hipStream_t s) {
  if (few) {
    constexpr int W = few_waves(C);
    constexpr int kLds = max_of(W * 2 * 32 * C * 16, W * 32 * 4 * (2 + 32 * ND + 4));
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(tree_few_kernel<NK, ND, C, W, kUniform>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
    tree_few_kernel<NK, ND, C, W, kUniform><<<grid, 64 * W, kLds, s>>>(a);
    return hipGetLastError();
  }
  constexpr int kEntries = kRing * 2 * 64 * 4;
  constexpr int kTwo = 4 * kTokens * C * 16 + kEntries, kFour = 8 * kTokens * C * 16 + kEntries;
  if constexpr (C == 16) {
    if (wide) {
      const hipError_t e =
          hipFuncSetAttribute(reinterpret_cast<const void*>(tree_kernel<NK, ND, C, 8, 4, kUniform>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, kFour);
      if (e != hipSuccess) return e;
      tree_kernel<NK, ND, C, 8, 4, kUniform><<<grid, 64 * 8, kFour, s>>>(a);
      return hipGetLastError();
    }
  }
  if (kTwo > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(tree_kernel<NK, ND, C, 4, 2, kUniform>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, kTwo);
    if (e != hipSuccess) return e;
  }
  tree_kernel<NK, ND, C, 4, 2, kUniform><<<grid, 64 * 4, kTwo, s>>>(a);
  return hipGetLastError();
}

template <int NK, int ND, int C>
hipError_t launch(const TreeArgs& a, bool few, bool wide, uint32_t grid, hipStream_t s) {
  return a.S % (64 / C) == 0 ? launch_as<NK, ND, C, true>(a, few, wide, grid, s)
                             : launch_as<NK, ND, C, false>(a, few, wide, grid, s);
}

}  // namespace

// How the work is dealt.  The lengths are in device memory, so the host decides by
// the capacity alone whether sequences are cut and into how many pieces at most; the
// kernel sizes them.  Up to twice as many units as workgroups at a time and more
// than four steps: cut (1 x 1024 tokens, 32 heads, four steps: 18.6 us whole, 20.4
// as two pieces and a join); of several sequences into up to four pieces a place, so
// that unlike lengths even out.  More units: whole sequences, the longest first (16
// ragged x 4096, 32 heads 103 us; cut, with the tiles shared, 134).
// 256 rows a workgroup rather than 128 where there are more than 128: 606 us for 642
// at 2 x 131072.
TreePlan plan_tree(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t cap, int64_t most, int num_cus) {
  TreePlan p;
  const int64_t rows = most * (Hq / Hkv);
  p.few = rows <= kRows;
  const int chunks = D <= 64 ? 8 : D <= 128 ? 16 : 32;
  p.wide = chunks == 16 && rows > kBlock;
  const int64_t block = p.few ? kRows : p.wide ? 2 * kBlock : kBlock;
  p.tiles = std::max<int64_t>(1, (rows + block - 1) / block);
  const int64_t units = B * Hkv * p.tiles;
  const int64_t unit = p.few ? 32 * few_waves(chunks) : kTokens;
  const int64_t steps = (cap + unit - 1) / unit;
  // workgroups at a time
  const int64_t slots = num_cus * int64_t(p.few ? (chunks == 8 ? 2 : 1) : (chunks == 32 || p.wide ? 1 : 2));
  if (B >= 1 && B <= kMaxCut && steps > 4) {
    if (units < 2 * slots) {
      int64_t k = 1;
      while (B > 1 && k < 4 && k * slots < 4 * units) ++k;
      p.room = int(std::min<int64_t>(k * slots * B / units, (steps + 1) / 2 * B));
      if (p.room <= B) p.room = 0;
    }
    p.order = p.room == 0 && B > 1 && units > slots;
  }
  const int64_t pairs = (p.room ? p.room : B) * Hkv;
  p.grid = (pairs + 7) / 8 * 8 * p.tiles;
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  if (p.room) {
    p.off_ml = up(size_t(B) * 8);
    const size_t all = size_t(pairs) * size_t(p.tiles * block);
    p.off_part = p.off_ml + up(all * 8);
    p.bytes = p.off_part + all * size_t(D) * 4;
  }
  return p;
}

hipError_t launch_tree(const KvView& c, const TreeCall& r, const TreePlan& p, void* ws, hipStream_t s) {
  TreeArgs a{};
  a.q = r.q;
  a.out = r.out;
  a.starts = r.starts;
  a.parents = r.parents;
  a.mask = r.mask;
  a.q_t = r.q_t;
  a.q_h = r.q_h;
  a.o_t = r.o_t;
  a.o_h = r.o_h;
  a.mask_b = r.mask_b;
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
  a.B = int(c.B);
  a.T = int(r.T);
  a.Hq = int(r.Hq);
  a.Hkv = int(c.Hkv);
  a.G = int(r.Hq / c.Hkv);
  a.D = int(c.D);
  a.S = int(c.S);
  a.pages = int(c.pages);
  a.cap = int(c.per_seq * c.S);
  a.most = int(r.most);
  a.room = p.room;
  a.tiles = int(p.tiles);
  a.rows = int(p.tiles) * (p.few ? kRows : p.wide ? 2 * kBlock : kBlock);
  a.order = p.order;
  a.zero = r.scale == 0.f;
  a.c = a.zero ? 1.f : std::abs(r.scale) * 1.44269504088896340736f;
  a.flip = r.scale < 0.f ? 0x80008000u : 0u;
  a.div = page_div(c.S);
  a.per_g = page_div(a.G);
  a.per_pair = page_div(8 * p.tiles);
  a.per_hkv = page_div(c.Hkv);
  if (p.room) {
    uint8_t* w = static_cast<uint8_t*>(ws);
    a.plan = reinterpret_cast<int32_t*>(w);
    a.ml = reinterpret_cast<float*>(w + p.off_ml);
    a.part = reinterpret_cast<float*>(w + p.off_part);
  }
  const uint32_t grid = uint32_t(p.grid);
  const hipError_t e = a.D <= 64    ? launch<4, 2, 8>(a, p.few, p.wide, grid, s)
                       : a.D <= 96  ? launch<6, 3, 16>(a, p.few, p.wide, grid, s)
                       : a.D <= 128 ? launch<8, 4, 16>(a, p.few, p.wide, grid, s)
                       : a.D <= 192 ? launch<12, 6, 32>(a, p.few, p.wide, grid, s)
                                    : launch<16, 8, 32>(a, p.few, p.wide, grid, s);
  if (e != hipSuccess || !p.room) return e;
  const int per = a.D <= 64 ? 16 : a.D <= 128 ? 32 : 64;
  const int64_t rows = r.T * r.Hq;
  tree_join_kernel<<<dim3(uint32_t((rows + kJoin / 64 - 1) / (kJoin / 64))), kJoin, 0, s>>>(a, per);
  return hipGetLastError();
}

}  // namespace swm
