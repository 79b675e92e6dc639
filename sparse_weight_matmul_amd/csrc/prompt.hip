// Attention over whole prompts, packed one behind the other.
//
//   x_ij = scale * q_i . k_j ;  o_i = sum_j e^(x_ij - m_i) v_j / sum_j e^(x_ij - m_i)
//
// over the tokens j of the row's own sequence, j <= i if causal; m_i is any
// number near the row's largest score (flash.h says which).
//
// Four D operations for every row and token it sees, against 4 D bytes a token and
// head: bound by the matrix cores but for the shortest prompts.  A workgroup has
// 128 rows of a head, 32 a wave, and goes once over the keys and values they see,
// tile by tile through LDS, the next tile on its way meanwhile.  Key fragments are
// read once per 32 rows, so that LDS reads (128 bytes a cycle and CU) take as long
// as the products; together with the power limit that is what holds long prompts at
// about 1.05 PFLOP/s: 1 x 16384 tokens, 32 heads on 8, 2055 to 2135 us by the card (with
// zeros for inputs, which draw less power, 1480; a library's product of 8192^3 runs at
// 1.34 to 1.53 PFLOP/s with random inputs and at 2.2 with zeros).  Shorter ones pay 5 us
// a workgroup for its first tile, which two or three workgroups to a CU
// hide in part: 16 ragged x 2048, 32 heads 268 to 280 us (0.7 PFLOP/s).  Rows above 128
// halves leave room for one workgroup on a CU: 1 x 4096 tokens, 32 heads on 8, of 64
// 94 us (0.73 PFLOP/s), of 128 159 (0.87), of 192 353 (0.58), of 256 420 (0.66).
// Tried: eight waves in two groups that take turns on the matrix cores (1 x 16384 1 to
// 4% faster, but 352 us for 280 for the ragged batch), 64 rows a wave (half the LDS
// reads, but the accumulators do not fit beside the rest without copies: 2490), all blocks
// of a batch by their tokens (see pick_of_few).
#include <hip/hip_runtime.h>

#include <algorithm>
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
// Workgroups per CU from which tiles are small.  Measured with 32 heads of 128, us,
// tiles of 64 / 32 tokens: 8 x 1024 tokens (9 a CU) 121 / 129, 64 x 100 (14) 81 /
// 64, 1 x 16384 (16) 2079 / 2081, 16 ragged x 2048 (19) 292 / 279, 32 x 512 (20)
// 179 / 174, 64 x 256 (24) 167 / 153, 1 x 512 (0.6) 17.5 / 20.6.
constexpr int kMany = 12;
// Mean length below which a wave has a block of 32 rows by itself, where there are
// two workgroups per CU and more.  us, as blocks of 128 / so: 64 x 10 tokens, 160 heads of
// 64 103 / 27, 32 heads of 128: 64 x 10 37 / 13, 64 x 32 42 / 22, 64 x 64 42 / 39,
// 64 x 100 61 / 63; 8 x 40, 32 of 256 (1.2 a CU) 13.5 / 14.6.
constexpr int kShort = 80;
// Tokens up to which a sequence of such a batch is dealt out so.  32 heads of 128, us,
// by 32 rows / by 128: 255 empty places and 1 x 512 23 / 21, 1 x 1024 41 / 33, 1 x 2048
// 82 / 60, 1 x 16384 2990 / 2260 (2130 in a batch of its own, whose tiles leave room for
// three workgroups on a CU); 60 x 5 and 4 x 300 25 / 28, 200 x 5 and 30 x 300 120 / 133.
constexpr int kLong = 512;

struct PromptArgs {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  const int32_t* starts;
  int64_t q_t, q_h, k_t, k_h, v_t, v_h, o_t, o_h;
  int32_t B, T, Hq, G, D;
  float c;        // |scale| log2(e), or 1 where the scale is 0
  uint32_t flip;  // sign bits that turn q where the scale is negative
  bool zero;      // the scale is 0
  PageDiv per_hq;
};

// The sequence's part of the packed rows, whatever `starts` holds.
__device__ __forceinline__ void rows_of(const PromptArgs& a, int s, int* first, int* n) {
  const int s0 = min(max(a.starts[s], 0), a.T), s1 = min(max(a.starts[s + 1], 0), a.T);
  *first = s0;
  *n = max(s1 - s0, 0);
}

struct Block {
  int first, n, j;  // the sequence's rows, and which block of them
};
// Block j of the sequence that lane l holds; false for one that it does not have.
template <int kBlock>
__device__ __forceinline__ bool take(int first, int n, int l, int j, Block* out) {
  out->first = __builtin_amdgcn_readlane(first, l);
  out->n = __builtin_amdgcn_readlane(n, l);
  out->j = j;
  return j >= 0 && j < (out->n + kBlock - 1) / kBlock;
}

// The block of query rows that comes at place u: sequence after sequence, of up
// to 64 the longest first, so that short ones fill the end; a sequence's last
// block first.  (All blocks by their tokens, whatever their sequence, is worse, 298
// us for 281 at 16 ragged x 2048: the workgroups at work then read keys of so many
// sequences that no L2 holds them.)  Of up to 64 sequences lane l holds number l,
// its rows and how many blocks of it count.
template <int kBlock>
__device__ __forceinline__ bool pick_of_few(const PromptArgs& a, int u, int lane, int first, int n, int blocks,
                                            Block* out) {
  int before = 0;  // blocks of longer sequences, and of equal ones with a lower index
  for (int l = 0; l < a.B; ++l) {
    const int x = __builtin_amdgcn_readlane(blocks, l);
    before += x + int(l < lane) > blocks ? x : 0;
  }
  const uint64_t in = __builtin_amdgcn_ballot_w64(before <= u && u < before + blocks);
  if (!in) return false;
  const int l = __builtin_ctzll(in);
  return take<kBlock>(first, n, l, __builtin_amdgcn_readlane(before + blocks, l) - 1 - u, out);
}

// Of more, every lane has added up a 64th, whose bounds are requested one behind
// the other, then the wave goes through the one part that has place u.
template <typename F>
__device__ __forceinline__ void each_of_part(const PromptArgs& a, int lane, F f) {
  const int per = (a.B + 63) / 64, own = min(lane * per, a.B), next = min(own + per, a.B);
  int from = own < a.B ? min(max(a.starts[own], 0), a.T) : 0;
#pragma unroll 8
  for (int s = own; s < next; ++s) {
    const int to = min(max(a.starts[s + 1], 0), a.T);
    f(max(to - from, 0));
    from = to;
  }
}
template <int kBlock, typename F>
__device__ __forceinline__ bool pick_of_many(const PromptArgs& a, int u, int lane, int sum, F blocks_of, Block* out) {
  const int per = (a.B + 63) / 64, own = min(lane * per, a.B), next = min(own + per, a.B);
  const int upto = int(scan_wave(uint32_t(sum)));
  const uint64_t part = __builtin_amdgcn_ballot_w64(u < upto);
  if (!part) return false;
  const int l = __builtin_ctzll(part);
  int base = __builtin_amdgcn_readlane(upto - sum, l);
  const int end = __builtin_amdgcn_readlane(next, l);
  for (int s0 = __builtin_amdgcn_readlane(own, l); s0 < end; s0 += 64) {
    int first = 0, n = 0;
    if (s0 + lane < end) rows_of(a, s0 + lane, &first, &n);
    const int last = base + int(scan_wave(uint32_t(blocks_of(n))));
    const uint64_t in = __builtin_amdgcn_ballot_w64(u < last);
    if (in) {
      const int i = __builtin_ctzll(in);
      return take<kBlock>(first, n, i, __builtin_amdgcn_readlane(last, i) - 1 - u, out);
    }
    base = __builtin_amdgcn_readlane(last, 63);
  }
  return false;
}

__device__ __forceinline__ bool held_by_lanes(const PromptArgs& a) { return a.B > 1 && a.B <= 64; }

// Blocks of 128 rows, a workgroup each.
__device__ __forceinline__ bool find_wide(const PromptArgs& a, int u, int lane, Block* out) {
  auto blocks_of = [](int n) { return (n + kBlock - 1) / kBlock; };
  if (held_by_lanes(a)) {
    int first = 0, n = 0;
    if (lane < a.B) rows_of(a, lane, &first, &n);
    return pick_of_few<kBlock>(a, u, lane, first, n, blocks_of(n), out);
  }
  int sum = 0;
  each_of_part(a, lane, [&](int n) { sum += blocks_of(n); });
  return pick_of_many<kBlock>(a, u, lane, sum, blocks_of, out);
}

// Where prompts are short in the mean: blocks of 32 rows, a wave each, but of sequences
// of more than kLong tokens, which the mean hides among short and empty ones; those
// keep their blocks of 128 rows, which come first.  Without such sequences the place is
// the wave's own, known before the bounds come.  With the code for both, more than 64
// sequences take 1 to 3% longer than with that for 32 rows alone (1024 x 10 tokens 137
// us for 132).
struct Place {
  int u, head;
  bool wide;  // a workgroup's block of 128 rows
};
__device__ __forceinline__ bool find_mixed(const PromptArgs& a, int lane, int wave, Place* p, Block* out) {
  auto small_at = [&](int before) {  // behind so many workgroups of wide ones
    const int i = (int(blockIdx.x) - before) * kWaves + wave, u = page_index(a.per_hq, i);
    return Place{u, i - u * a.Hq, false};
  };
  auto place = [&](int blocks) {  // by the number of wide ones; a grid has less than 2^24 workgroups
    const int before = int(min(uint32_t(blocks), (1u << 24) / a.Hq + 1)) * a.Hq;
    if (int(blockIdx.x) >= before) return small_at(before);
    const int u = page_index(a.per_hq, blockIdx.x);
    return Place{u, int(blockIdx.x) - u * a.Hq, true};
  };
  auto all = [](int n) { return (n + kRows - 1) / kRows; };
  auto wide = [](int n) { return n > kLong ? (n + kBlock - 1) / kBlock : 0; };
  auto small = [&](int n) { return n > kLong ? 0 : all(n); };
  *p = small_at(0);
  if (held_by_lanes(a)) {
    int first = 0, n = 0;
    if (lane < a.B) rows_of(a, lane, &first, &n);
    if (__builtin_amdgcn_ballot_w64(n > kLong)) {
      *p = place(int(wave_sum(uint32_t(wide(n)))));
      if (p->wide) return pick_of_few<kBlock>(a, p->u, lane, first, n, wide(n), out);
    }
    return pick_of_few<kRows>(a, p->u, lane, first, n, small(n), out);
  }
  int sum = 0, longest = 0;
  each_of_part(a, lane, [&](int n) {
    sum += all(n);
    longest = max(longest, n);
  });
  if (__builtin_amdgcn_ballot_w64(longest > kLong)) {
    int blocks = 0;
    sum = 0;
    each_of_part(a, lane, [&](int n) {
      blocks += wide(n);
      sum += small(n);
    });
    *p = place(int(wave_sum(uint32_t(blocks))));
    if (p->wide) return pick_of_many<kBlock>(a, p->u, lane, blocks, wide, out);
    return pick_of_many<kRows>(a, p->u, lane, sum, small, out);
  }
  return pick_of_many<kRows>(a, p->u, lane, sum, all, out);
}

// The head of workgroup `i` of those over one block of rows: they go round the eight
// XCDs, and neighbouring heads, which share keys, to one of them.
__device__ __forceinline__ int head_of(const PromptArgs& a, int i) {
  return a.Hq % 8 == 0 ? (i & 7) * (a.Hq >> 3) + (i >> 3) : i;
}

// A row's output; what clear_odd took out of the value rows `from` .. `end` - 1
// goes to the rows that see them.
template <int ND>
__device__ __forceinline__ void finish(const PromptArgs& a, State<ND>& st, const uint16_t* vh, bool odd, int from,
                                       int end, int qi, int n, int first, int head, int h) {
  const float l = sum_halves(st.l);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (odd) {
    int D = a.D;
    for (int t = from; t < end; ++t) {
      asm volatile("" : "+s"(D));  // its comparisons stay here: before the loop they would take 64 pairs of registers
      if (t > qi) continue;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int x = 32 * d + 8 * (i >> 2) + 4 * h + (i & 3);
          if (x >= D) continue;
          const uint16_t w = vh[int64_t(t) * a.v_t + x];
          if ((w & 0x7c00) == 0x7c00) st.o[d][i] += float(__builtin_bit_cast(_Float16, w));
        }
    }
  }
  if (qi >= n) return;
  write_row(st, inv, a.out + int64_t(first + qi) * a.o_t + int64_t(head) * a.o_h, a.D, h);
}

// A workgroup's block of 128 rows, over tiles of 32 NB tokens.
template <int NK, int ND, int C, bool kCausal, int NB>
__device__ __forceinline__ void wide_block(const PromptArgs& a, const Block& block, int head, uint16_t* smem) {
  constexpr int kTokens = 32 * NB;
  constexpr int kTile = kTokens * C * 8;        // halves
  constexpr int kLoads = C * NB / 2 / kWaves;  // 1 KiB each, of a wave and tile
  uint16_t* sv = smem + 2 * kTile;  // two key tiles, then two value tiles
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = block.first, n = block.n, j = block.j;
  const int q0 = j * kBlock + wave * kRows;  // the wave's first row
  const int end = kCausal ? min(n, (j + 1) * kBlock) : n;
  const int hkv = head / a.G;
  const int r = lane & 31, h = lane >> 5;
  const int qi = q0 + r;

  const uint16_t* kh = a.k + int64_t(first) * a.k_t + int64_t(hkv) * a.k_h;
  const uint16_t* vh = a.v + int64_t(first) * a.v_t + int64_t(hkv) * a.v_h;
  uint32_t k_off[kLoads], v_off[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int at = (i * kWaves + wave) * 64 + lane, row = at / C, c = at % C;
    const int kc = key_chunk<C>(row, c) * 8, vc = value_chunk<C>(row, c) * 8;
    k_off[i] = kc < a.D ? uint32_t(row * int(a.k_t) + kc) * 2 : 0x80000000u;
    v_off[i] = vc < a.D ? uint32_t(row * int(a.v_t) + vc) * 2 : 0x80000000u;
  }
  const uint32_t to = lds_address(smem);
  auto load = [&](int t0, int buf) {  // rows behind the sequence's end are zeros
    const int left = min(n - t0, kTokens);
    load_tile(kh + int64_t(t0) * a.k_t, ((left - 1) * int(a.k_t) + a.D) * 2, k_off, kLoads,
              to + (buf * kTile + wave * 512) * 2, kWaves * 1024);
    load_tile(vh + int64_t(t0) * a.v_t, ((left - 1) * int(a.v_t) + a.D) * 2, v_off, kLoads,
              to + ((2 + buf) * kTile + wave * 512) * 2, kWaves * 1024);
  };

  load(0, 0);
  half8 q[NK];
  load_query(a.q + int64_t(first + min(qi, n - 1)) * a.q_t + int64_t(head) * a.q_h, a.D, h, q);
  const Reads<NK, ND, C> at(smem, lane, 2 * kTile * 2);
  State<ND> st;
  st.clear();
  bool odd = false;  // a value that is no number, in a tile that some rows see only a part of
  // One tile, in buffer `buf`, a constant so that it is part of the reads' offsets.
  auto step = [&](int t0, auto constant) {
    constexpr int buf = decltype(constant)::value;
    wait_vm<0>();
    __syncthreads();
    if (t0 + kTokens < end) load(t0 + kTokens, buf ^ 1);
    if (buf == 0 && t0 == 0) mend_query(a.D, h, a.zero, a.flip, q);
    if (kCausal && t0 + kTokens > j * kBlock) {
      // An infinity or NaN times a weight of zero would reach rows that do not
      // see its token: zeros in its place here, added to the rows that do at the end.
      uint16_t* vt = sv + buf * kTile;
      bool bad = false;
      for (int i = threadIdx.x; i < kTokens * C; i += 64 * kWaves) bad |= clear_odd(vt + i * 8);
      odd |= __syncthreads_or(bad);
    }
    if (kCausal && t0 > q0 + kRows - 1) return;
    f32x16 s[NB];
    scores(at, buf * kTile * 2, q, s);
    if (t0 + kTokens > n || (kCausal && t0 + kTokens - 1 > q0)) {
      const int last = (kCausal ? min(qi, n - 1) : n - 1) - t0 - 4 * h;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (32 * b + 8 * (i >> 2) + (i & 3) > last) s[b][i] = neg_inf();
    }
    half8 p[2 * NB];
    weights(st, s, a.c, buf == 0 && t0 == 0, p);
    outputs(st, at, buf * kTile * 2, p);
  };
  for (int t0 = 0; t0 < end; t0 += 2 * kTokens) {
    step(t0, std::integral_constant<int, 0>());
    if (t0 + kTokens < end) step(t0 + kTokens, std::integral_constant<int, 1>());
  }
  finish(a, st, vh, kCausal && odd, j * kBlock, end, qi, n, first, head, h);
}

// With tiles of 64 tokens two workgroups share a CU, with 32 three, whose waves
// fill more of each other's gaps, but each alone takes longer.
template <int NK, int ND, int C, bool kCausal, int NB>
__global__ __launch_bounds__(64 * kWaves, ND > 4 ? 1 : NB == 1 ? 3 : 2) void prompt_kernel(PromptArgs a) {
  extern __shared__ uint16_t smem[];
  const int u = page_index(a.per_hq, blockIdx.x);
  Block block;
  if (!find_wide(a, u, threadIdx.x & 63, &block)) return;
  wide_block<NK, ND, C, kCausal, NB>(a, block, head_of(a, blockIdx.x - u * a.Hq), smem);
}

// Short prompts: a wave has 32 rows of a head by itself, with a tile of 32 tokens
// of its own, so that no wave is there for rows that a sequence does not have.
template <int NK, int ND, int C, bool kCausal>
__device__ __forceinline__ void small_block(const PromptArgs& a, const Block& block, int head, uint16_t* smem) {
  constexpr int kTile = kRows * C * 8;  // halves
  constexpr int kLoads = C / 2;         // 1 KiB each, of a tile
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint16_t* sk = smem + wave * 2 * kTile;  // no other wave looks at these
  uint16_t* sv = sk + kTile;
  const int first = block.first, n = block.n, q0 = block.j * kRows;
  const int end = kCausal ? min(n, q0 + kRows) : n;
  const int hkv = head / a.G;
  const int r = lane & 31, h = lane >> 5, qi = q0 + r;
  const uint16_t* kh = a.k + int64_t(first) * a.k_t + int64_t(hkv) * a.k_h;
  const uint16_t* vh = a.v + int64_t(first) * a.v_t + int64_t(hkv) * a.v_h;
  uint32_t k_off[kLoads], v_off[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int at = i * 64 + lane, row = at / C, c = at % C;
    const int kc = key_chunk<C>(row, c) * 8, vc = value_chunk<C>(row, c) * 8;
    k_off[i] = kc < a.D ? uint32_t(row * int(a.k_t) + kc) * 2 : 0x80000000u;
    v_off[i] = vc < a.D ? uint32_t(row * int(a.v_t) + vc) * 2 : 0x80000000u;
  }
  const uint32_t to = lds_address(sk);
  auto load = [&](int t0) {
    const int left = min(n - t0, kRows);
    load_tile(kh + int64_t(t0) * a.k_t, ((left - 1) * int(a.k_t) + a.D) * 2, k_off, kLoads, to, 1024);
    load_tile(vh + int64_t(t0) * a.v_t, ((left - 1) * int(a.v_t) + a.D) * 2, v_off, kLoads, to + kTile * 2, 1024);
  };
  load(0);
  half8 q[NK];
  load_query(a.q + int64_t(first + min(qi, n - 1)) * a.q_t + int64_t(head) * a.q_h, a.D, h, q);
  const Reads<NK, ND, C> at(sk, lane, kTile * 2);
  State<ND> st;
  st.clear();
  bool odd = false;
  for (int t0 = 0; t0 < end; t0 += kRows) {
    wait_vm<0>();
    asm volatile("" ::: "memory");  // no barrier follows: reads of the tile stay below
    __builtin_amdgcn_sched_barrier(0);
    if (t0 == 0) mend_query(a.D, h, a.zero, a.flip, q);
    if (kCausal && t0 == q0) {  // see prompt_kernel
      bool bad = false;
      for (int i = lane; i < kRows * C; i += 64) bad |= clear_odd(sv + i * 8);
      odd = __builtin_amdgcn_ballot_w64(bad) != 0;
    }
    f32x16 s[1];
    scores(at, 0, q, s);
    if (t0 + kRows > n || (kCausal && t0 == q0)) {
      const int last = (kCausal ? min(qi, n - 1) : n - 1) - t0 - 4 * h;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (8 * (i >> 2) + (i & 3) > last) s[0][i] = neg_inf();
    }
    half8 p[2];
    weights(st, s, a.c, t0 == 0, p);
    outputs(st, at, 0, p);
    __builtin_amdgcn_sched_barrier(0);  // the tile has been read: the next one takes its place
    if (t0 + kRows < end) load(t0 + kRows);
  }
  finish(a, st, vh, odd, q0, end, qi, n, first, head, h);
}

// Both, a workgroup of one kind or the other.
template <int NK, int ND, int C, bool kCausal>
__global__ __launch_bounds__(64 * kWaves, ND > 4 ? 1 : 2) void prompt_mixed_kernel(PromptArgs a) {
  extern __shared__ uint16_t smem[];
  Place p;
  Block block;
  if (!find_mixed(a, threadIdx.x & 63, __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), &p, &block)) return;
  if (p.wide)
    wide_block<NK, ND, C, kCausal, 1>(a, block, head_of(a, p.head), smem);
  else
    small_block<NK, ND, C, kCausal>(a, block, p.head, smem);
}

template <int NK, int ND, int C, bool kCausal, int NB>
hipError_t launch_as(const PromptArgs& a, uint32_t grid, hipStream_t s) {
  constexpr int kLds = 4 * 32 * NB * C * 16;
  if (kLds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(prompt_kernel<NK, ND, C, kCausal, NB>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
  }
  prompt_kernel<NK, ND, C, kCausal, NB><<<grid, 64 * kWaves, kLds, s>>>(a);
  return hipGetLastError();
}

template <int NK, int ND, int C, bool kCausal>
hipError_t launch_mixed(const PromptArgs& a, hipStream_t s) {
  constexpr int kLds = kWaves * 2 * kRows * C * 16;  // of the small blocks, more than the wide ones use
  if (kLds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(prompt_mixed_kernel<NK, ND, C, kCausal>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
  }
  // Of m sequences with tokens up to x are long: T / 128 + x workgroups for whole blocks and long ends, a quarter
  // of one for a short end.
  const int64_t m = std::min(a.T, a.B), x = std::min<int64_t>(m, a.T / (kLong + 1));
  const int64_t quarters = a.T / kRows + 1 + 4 * x + (m - x);  // of a workgroup, for each head
  const uint32_t grid = uint32_t((quarters * a.Hq + kWaves - 1) / kWaves);
  prompt_mixed_kernel<NK, ND, C, kCausal><<<grid, 64 * kWaves, kLds, s>>>(a);
  return hipGetLastError();
}

template <int NK, int ND, int C>
hipError_t launch(const PromptArgs& a, bool causal, uint32_t grid, int num_cus, hipStream_t s) {
  if (a.T / a.B < kShort && grid >= 2u * num_cus)
    return causal ? launch_mixed<NK, ND, C, true>(a, s) : launch_mixed<NK, ND, C, false>(a, s);
  if constexpr (C == 16) {  // shorter rows leave room for three anyway, longer ones for one
    if (grid >= uint32_t(kMany) * num_cus)
      return causal ? launch_as<NK, ND, C, true, 1>(a, grid, s) : launch_as<NK, ND, C, false, 1>(a, grid, s);
  }
  return causal ? launch_as<NK, ND, C, true, 2>(a, grid, s) : launch_as<NK, ND, C, false, 2>(a, grid, s);
}

}  // namespace

int64_t prompt_grid(int64_t T, int64_t B, int64_t Hq) { return (T / kBlock + std::min(T, B)) * Hq; }

hipError_t launch_prompt(const PromptCall& r, int num_cus, hipStream_t s) {
  PromptArgs a{};
  a.q = r.q;
  a.k = r.k;
  a.v = r.v;
  a.out = r.out;
  a.starts = r.starts;
  a.q_t = r.q_t;
  a.q_h = r.q_h;
  a.k_t = r.k_t;
  a.k_h = r.k_h;
  a.v_t = r.v_t;
  a.v_h = r.v_h;
  a.o_t = r.o_t;
  a.o_h = r.o_h;
  a.B = int(r.B);
  a.T = int(r.T);
  a.Hq = int(r.Hq);
  a.G = int(r.Hq / r.Hkv);
  a.D = int(r.D);
  a.zero = r.scale == 0.f;
  a.c = a.zero ? 1.f : std::abs(r.scale) * 1.44269504088896340736f;
  a.per_hq = page_div(r.Hq);
  a.flip = r.scale < 0.f ? 0x80008000u : 0u;
  const uint32_t grid = uint32_t(prompt_grid(r.T, r.B, r.Hq));
  if (a.D <= 64) return launch<4, 2, 8>(a, r.causal, grid, num_cus, s);
  if (a.D <= 96) return launch<6, 3, 16>(a, r.causal, grid, num_cus, s);
  if (a.D <= 128) return launch<8, 4, 16>(a, r.causal, grid, num_cus, s);
  if (a.D <= 192) return launch<12, 6, 32>(a, r.causal, grid, num_cus, s);
  return launch<16, 8, 32>(a, r.causal, grid, num_cus, s);
}

}  // namespace swm
