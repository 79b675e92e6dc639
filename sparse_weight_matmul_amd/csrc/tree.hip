// Attention of drafted tokens over a paged key-value cache that holds their
// keys and values behind the sequence's own.
//
//   x_it = scale * q_i . k_t ;  o_i = sum_t e^(x_it - m_i) v_t / sum_t e^(x_it - m_i),  m_i = max x_it
//
// over the tokens t before the drafted ones, i itself, its parent, the parent's
// parent and so on, as far as they are live (on a page of the pool, not masked).
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

constexpr int kWaves = 4;
constexpr int kBlock = kWaves * kRows;  // query rows of a workgroup
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
  int32_t B, T, Hq, Hkv, G, D, S, pages, cap, per_seq, most;
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

// Which drafted tokens the lane's one sees: bit j for token j.  Every lane
// starts with itself and its parent; each round adds what the farthest one seen
// so far sees: 2, 4, .. generations.  A parent that is not before its child is none.
__device__ __forceinline__ uint64_t ancestors(const TreeArgs& a, int first, int n, int lane) {
  uint64_t sees = uint64_t(1) << lane;
  int up = -1;
  if (lane < n) {
    up = a.parents ? a.parents[first + lane] : lane - 1;
    if (up < 0 || up >= lane) up = -1;
  }
#pragma unroll
  for (int r = 0; r < 6; ++r) {
    const int from = max(up, 0);
    const uint32_t lo = __shfl(uint32_t(sees), from), hi = __shfl(uint32_t(sees >> 32), from);
    const int next = __shfl(up, from);
    if (up >= 0) {
      sees |= uint64_t(hi) << 32 | lo;
      up = next;
    }
  }
  return sees;
}

// The pieces that the sequences are cut into: `each` tiles of 64 tokens, the
// fewest (two at least) with which they are a.room in all.  Lane l has sequences 2 l and
// 2 l + 1, pieces first .. mid - 1 and mid .. last - 1.  A quotient that is
// one off only moves the last piece's end.
struct Cuts {
  uint32_t each;
  int first, mid, last;
};
__device__ __forceinline__ uint32_t tiles_of(const TreeArgs& a, int b) {
  if (b >= a.B) return 0;
  int first, n;
  drafted(a, b, &first, &n);
  return n ? max((min(max(a.lengths[b], 0), a.cap) + kTokens - 1) / kTokens, 1) : 0;
}
__device__ __forceinline__ Cuts cut(const TreeArgs& a, int lane) {
  const uint32_t t0 = tiles_of(a, 2 * lane), t1 = tiles_of(a, 2 * lane + 1);
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

// One workgroup: 128 query rows (drafted token x query head of the group) of a
// sequence and key-value head, over a piece of its tokens.  kUniform: the rows of
// one load instruction are on one page, so that its address is scalar.
template <int NK, int ND, int C, bool kUniform>
__global__ __launch_bounds__(64 * kWaves, ND <= 4 ? 2 : 1) void tree_kernel(TreeArgs a) {
  constexpr int kTile = kTokens * C * 8;  // halves
  constexpr int kLoads = C / kWaves;      // 1 KiB each, of a wave and tile
  constexpr int kSpan = 64 / C;           // rows of one
  extern __shared__ uint16_t smem[];
  uint16_t* sk = smem;              // [2][kTile]
  uint16_t* sv = smem + 2 * kTile;  // [2][kTile]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, h = lane >> 5;
  // Workgroups go round the eight XCDs: those that read the same tokens are
  // eight apart, so that they share an L2.
  const int group = page_index(a.per_pair, blockIdx.x), rest = blockIdx.x - group * 8 * a.tiles;
  const int tile = rest >> 3, pair = group * 8 + (rest & 7);
  const int piece = page_index(a.per_hkv, pair), hkv = pair - piece * a.Hkv;
  if (piece >= (a.room > 0 ? a.room : a.B)) return;
  int b = piece, nth = 0, count = 1;
  uint32_t each = 0;
  if (a.room > 0) {
    const Cuts c = cut(a, lane);
    if (blockIdx.x == 0 && wave == 0) {
      if (2 * lane < a.B) a.plan[4 * lane] = c.first, a.plan[4 * lane + 1] = c.mid - c.first;
      if (2 * lane + 1 < a.B) a.plan[4 * lane + 2] = c.mid, a.plan[4 * lane + 3] = c.last - c.mid;
    }
    const uint64_t in = __builtin_amdgcn_ballot_w64(piece >= c.first && piece < c.last);
    if (in == 0) return;  // more workgroups than pieces
    const int l = __builtin_ctzll(in);
    const int mid = __builtin_amdgcn_readlane(c.mid, l);
    const bool second = piece >= mid;
    b = 2 * l + second;
    nth = piece - (second ? mid : __builtin_amdgcn_readlane(c.first, l));
    count = second ? __builtin_amdgcn_readlane(c.last, l) - mid : mid - __builtin_amdgcn_readlane(c.first, l);
    each = __builtin_amdgcn_readfirstlane(c.each);
  }
  b = __builtin_amdgcn_readfirstlane(b);
  int first, drafts;
  drafted(a, b, &first, &drafts);
  first = __builtin_amdgcn_readfirstlane(first);
  drafts = __builtin_amdgcn_readfirstlane(drafts);
  const int rows = drafts * a.G;
  if (tile * kBlock >= rows) return;
  const int n = __builtin_amdgcn_readfirstlane(min(max(a.lengths[b], 0), a.cap));
  const int own = n - drafts;  // tokens before the drafted ones; negative where the length does not count them all
  const int begin = __builtin_amdgcn_readfirstlane(min(int64_t(nth) * each * kTokens, int64_t(n)));
  const int end = __builtin_amdgcn_readfirstlane(
      nth == count - 1 ? n : min(int64_t(nth + 1) * each * kTokens, int64_t(n)));
  const int32_t* row = a.table + int64_t(b) * a.table_b;
  const uint8_t* mask = a.mask ? a.mask + int64_t(b) * a.mask_b : nullptr;
  const uint16_t* kh = a.k + int64_t(hkv) * a.k_h;
  const uint16_t* vh = a.v + int64_t(hkv) * a.v_h;

  // the lane's query row: token i of the drafted ones, query head g of the group
  const int m0 = tile * kBlock + wave * kRows;
  const int mi = min(m0 + r, rows - 1);
  const int qi = page_index(a.per_g, mi), qh = hkv * a.G + mi - qi * a.G;
  const bool idle = m0 >= rows;
  half8 q[NK];
  {
    const uint16_t* src = a.q + int64_t(first + qi) * a.q_t + int64_t(qh) * a.q_h;
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      const int d = 16 * k + 8 * h;
      u32x4 w = *reinterpret_cast<const u32x4*>(src + (d < a.D ? d : 0));
      if (d >= a.D || a.zero) w = u32x4{0, 0, 0, 0};
      q[k] = __builtin_bit_cast(half8, w ^ a.flip);
    }
  }
  uint64_t sees = ancestors(a, first, drafts, lane);
  {
    const uint32_t lo = __shfl(uint32_t(sees), qi), hi = __shfl(uint32_t(sees >> 32), qi);
    sees = uint64_t(hi) << 32 | lo;
  }

  // Key dimensions that only pad the products: zeros, never loaded.
  if (a.D < 16 * NK) {
    for (int i = threadIdx.x; i < 2 * kTile / 8; i += 64 * kWaves)
      *reinterpret_cast<u32x4*>(sk + i * 8) = u32x4{0, 0, 0, 0};
  }

  // The page of token t0 + lane, always one of the pool; the top bit is set
  // where the token is not live.
  constexpr int kDead = int(0x80000000u), kPage = 0x7fffffff;
  auto place = [&](int t0) {
    const int t = t0 + lane;
    int page = kDead;
    if (t < end) {
      const int id = row[page_index(a.div, t)];
      if (id >= 0 && id < a.pages) page = mask && mask[t] == 0 ? id | kDead : id;
    }
    return page;
  };
  // Of the wave's loads: the row of a tile and the lane's bytes in it, by the first row of each.
  const int lr = lane / C, lc = lane % C;
  uint32_t k_off[kLoads], v_off[kLoads];
  bool k_in[kLoads], v_in[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int rw = (i * kWaves + wave) * kSpan + lr;
    const int kc = key_chunk<C>(rw, lc) * 8, vc = value_chunk<C>(rw, lc) * 8;
    k_in[i] = kc < a.D;
    v_in[i] = vc < a.D;
    k_off[i] = uint32_t(lr * int(a.k_s) + kc) * 2;
    v_off[i] = uint32_t(lr * int(a.v_s) + vc) * 2;
  }
  // A tile into buffer buf; rows that are not live become zeros.
  auto load = [&](int t0, int pages, int buf) {
    const uint64_t live = __builtin_amdgcn_ballot_w64(pages >= 0);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r0 = (i * kWaves + wave) * kSpan, rw = r0 + lr;
      uint16_t* dk = sk + buf * kTile + (i * kWaves + wave) * 512;
      uint16_t* dv = sv + buf * kTile + (i * kWaves + wave) * 512;
      const uint8_t *ks, *vs;
      if (kUniform) {
        const int page = __builtin_amdgcn_readlane(pages, r0) & kPage, t = t0 + r0, slot = t - page_index(a.div, t) * a.S;
        ks = reinterpret_cast<const uint8_t*>(kh + page * a.k_p + slot * a.k_s) + k_off[i];
        vs = reinterpret_cast<const uint8_t*>(vh + page * a.v_p + slot * a.v_s) + v_off[i];
      } else {
        const int page = __shfl(pages, rw) & kPage, t = t0 + rw, slot = t - page_index(a.div, t) * a.S;
        ks = reinterpret_cast<const uint8_t*>(kh + page * a.k_p + (slot - lr) * a.k_s) + k_off[i];
        vs = reinterpret_cast<const uint8_t*>(vh + page * a.v_p + (slot - lr) * a.v_s) + v_off[i];
      }
      if (~live == 0 && a.D == C * 8) {
        __builtin_amdgcn_global_load_lds(ks, (lds_ptr)dk, 16, 0, 0);
        __builtin_amdgcn_global_load_lds(vs, (lds_ptr)dv, 16, 0, 0);
      } else {
        const bool on = (live >> rw) & 1;
        if (on && k_in[i]) __builtin_amdgcn_global_load_lds(ks, (lds_ptr)dk, 16, 0, 0);
        if (on && v_in[i]) __builtin_amdgcn_global_load_lds(vs, (lds_ptr)dv, 16, 0, 0);
        if (!on) *reinterpret_cast<u32x4*>(dv + lane * 8) = u32x4{0, 0, 0, 0};
      }
    }
  };

  const Reads<NK, ND, C> at(smem, lane);
  State<ND> st;
  st.clear();
  bool odd = false;
  int now = place(begin), next = place(begin + kTokens);
  if (a.D < 16 * NK) __syncthreads();
  if (begin < end) load(begin, now, 0);
  // One tile, in buffer `buf`.
  auto step = [&](int t0, auto constant) {
    constexpr int buf = decltype(constant)::value;
    const uint64_t live = __builtin_amdgcn_ballot_w64(now >= 0);
    now = next;
    wait_vm<0>();
    __syncthreads();
    if (t0 + kTokens < end) load(t0 + kTokens, now, buf ^ 1);
    next = place(t0 + 2 * kTokens);
    const bool drafts_here = t0 + kTokens > own;
    if (drafts_here) {
      // A drafted token's infinity or NaN must not reach rows that do not see
      // it (its weight there is zero): zeros in its place, added at the end.
      uint16_t* vt = sv + buf * kTile;
      bool bad = false;
      for (int i = threadIdx.x; i < kTokens * C; i += 64 * kWaves)
        if (t0 + i / C >= own && value_chunk<C>(i / C, i % C) * 8 < a.D) bad |= clear_odd(vt + i * 8);
      odd |= __syncthreads_or(bad);
    }
    if (idle) return;
    f32x16 s[2];
    scores(at, buf * kTile * 2, q, s);
    if (drafts_here || ~live) {
      uint64_t on = live;
      if (drafts_here) {
        const int rel = own - t0;  // drafted token j is token rel + j of the tile
        uint64_t tree = rel >= 0 ? sees << rel : rel > -64 ? sees >> -rel : 0;  // rel < kTokens
        if (rel > 0) tree |= (uint64_t(1) << rel) - 1;
        on &= tree;
      }
      on >>= 4 * h;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (!((uint32_t(on >> (32 * e)) >> (8 * (i >> 2) + (i & 3))) & 1)) s[e][i] = neg_inf();
    }
    half8 p[4];
    weights(st, s, a.c, p);
    outputs(st, at, (2 + buf) * kTile * 2, p);
  };
  for (int t0 = begin; t0 < end; t0 += 2 * kTokens) {
    step(t0, std::integral_constant<int, 0>());
    if (t0 + kTokens < end) step(t0 + kTokens, std::integral_constant<int, 1>());
  }
  if (idle) return;
  const float l = sum_halves(st.l);
  if (odd) {
    for (int t = max(begin, own); t < end; ++t) {
      const int page = row[page_index(a.div, t)], slot = t - page_index(a.div, t) * a.S;
      if (!((sees >> (t - own)) & 1) || page < 0 || page >= a.pages || (mask && mask[t] == 0)) continue;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int e = 32 * d + 8 * (i >> 2) + 4 * h + (i & 3);
          if (e >= a.D) continue;
          const uint16_t w = vh[page * a.v_p + slot * a.v_s + e];
          if ((w & 0x7c00) == 0x7c00) st.o[d][i] += float(__builtin_bit_cast(_Float16, w));
        }
    }
  }
  if (m0 + r >= rows) return;
  if (count > 1) {
    const int64_t to = (int64_t(piece) * a.Hkv + hkv) * a.rows + m0 + r;
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
  uint16_t* dst = a.out + int64_t(first + qi) * a.o_t + int64_t(qh) * a.o_h;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int e = 32 * d + 2 * i + 4 * h;
      if (e >= a.D) continue;
#pragma unroll
      for (int f = 0; f < 4; ++f) dst[e + f] = __builtin_bit_cast(uint16_t, _Float16(st.o[d][i + f] * inv));
    }
}

constexpr int kJoin = 256;

// The pieces of a row added up, four dimensions a thread, `per` threads a row.
__global__ __launch_bounds__(kJoin) void tree_join_kernel(TreeArgs a, int per) {
  const int tid = threadIdx.x;
  const int64_t at = int64_t(blockIdx.x) * (kJoin / per) + tid / per;  // packed row and query head
  const int d = tid % per * 4;
  const int64_t t = at / a.Hq;
  const int qh = int(at - t * a.Hq);
  if (t >= a.T || d >= a.D) return;
  // the row's sequence: the last that starts at or before it
  int lo = 0, hi = a.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (a.starts[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  int first, drafts;
  drafted(a, lo, &first, &drafts);
  const int i = int(t) - first;
  if (i < 0 || i >= drafts) return;
  const int pieces = a.plan[2 * lo + 1];
  if (pieces < 2) return;  // written already
  const int hkv = page_index(a.per_g, qh);
  const int64_t next = int64_t(a.Hkv) * a.rows;
  const int64_t from = (int64_t(a.plan[2 * lo]) * a.Hkv + hkv) * a.rows + int64_t(i) * a.G + (qh - hkv * a.G);
  float m = neg_inf();
  for (int p = 0; p < pieces; ++p) m = fmaxf(m, a.ml[2 * (from + p * next)]);
  const float base = m == neg_inf() ? 0.f : m;
  float l = 0.f;
  float4 o = {0.f, 0.f, 0.f, 0.f};
  for (int p = 0; p < pieces; ++p) {
    const int64_t x = from + p * next;
    const float f = __builtin_amdgcn_exp2f(a.ml[2 * x] - base);
    const float4 v = *reinterpret_cast<const float4*>(a.part + x * a.D + d);
    l += f * a.ml[2 * x + 1];
    o.x += f * v.x;
    o.y += f * v.y;
    o.z += f * v.z;
    o.w += f * v.w;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint16_t* dst = a.out + t * a.o_t + int64_t(qh) * a.o_h + d;
  dst[0] = __builtin_bit_cast(uint16_t, _Float16(o.x * inv));
  dst[1] = __builtin_bit_cast(uint16_t, _Float16(o.y * inv));
  dst[2] = __builtin_bit_cast(uint16_t, _Float16(o.z * inv));
  dst[3] = __builtin_bit_cast(uint16_t, _Float16(o.w * inv));
}

template <int NK, int ND, int C, bool kUniform>
hipError_t launch_as(const TreeArgs& a, uint32_t grid, hipStream_t s) {
  constexpr int kLds = 4 * kTokens * C * 16;
  if (kLds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(tree_kernel<NK, ND, C, kUniform>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
  }
  tree_kernel<NK, ND, C, kUniform><<<grid, 64 * kWaves, kLds, s>>>(a);
  return hipGetLastError();
}

template <int NK, int ND, int C>
hipError_t launch(const TreeArgs& a, uint32_t grid, hipStream_t s) {
  return a.S % (64 / C) == 0 ? launch_as<NK, ND, C, true>(a, grid, s) : launch_as<NK, ND, C, false>(a, grid, s);
}

}  // namespace

// How the work is dealt: see the kernel.
TreePlan plan_tree(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t cap, int64_t most, int num_cus) {
  TreePlan p;
  const int64_t rows = most * (Hq / Hkv);
  p.tiles = std::max<int64_t>(1, (rows + kBlock - 1) / kBlock);
  const int64_t units = Hkv * p.tiles;  // of a sequence
  const int64_t steps = (cap + kTokens - 1) / kTokens;
  const int64_t slots = (D <= 128 ? 2 : 1) * int64_t(num_cus);  // workgroups at a time
  if (B >= 1 && B <= kMaxCut && steps > 2 && units * B <= 4 * slots) {
    int64_t k = 1;
    while (B > 1 && k < 4 && k * slots < 4 * B * units) ++k;
    p.room = int(std::min<int64_t>(k * slots / units, (steps + 1) / 2 * B));
    if (p.room <= B) p.room = 0;
  }
  const int64_t pairs = (p.room ? p.room : B) * Hkv;
  p.grid = (pairs + 7) / 8 * 8 * p.tiles;
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  if (p.room) {
    p.off_ml = up(size_t(B) * 8);
    const size_t all = size_t(pairs) * size_t(p.tiles) * kBlock;
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
  a.per_seq = int(c.per_seq);
  a.cap = int(c.per_seq * c.S);
  a.most = int(r.most);
  a.room = p.room;
  a.tiles = int(p.tiles);
  a.rows = int(p.tiles) * kBlock;
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
  const hipError_t e = a.D <= 64    ? launch<4, 2, 8>(a, grid, s)
                       : a.D <= 96  ? launch<6, 3, 16>(a, grid, s)
                       : a.D <= 128 ? launch<8, 4, 16>(a, grid, s)
                       : a.D <= 192 ? launch<12, 6, 32>(a, grid, s)
                                    : launch<16, 8, 32>(a, grid, s);
  if (e != hipSuccess || !p.room) return e;
  const int per = a.D <= 64 ? 16 : a.D <= 128 ? 32 : 64;
  const int64_t rows = r.T * r.Hq;
  tree_join_kernel<<<dim3(uint32_t((rows + kJoin / per - 1) / (kJoin / per))), kJoin, 0, s>>>(a, per);
  return hipGetLastError();
}

}  // namespace swm
