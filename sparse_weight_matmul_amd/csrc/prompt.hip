// Attention over whole prompts, packed one behind the other.
//
//   x_ij = scale * q_i . k_j ;  o_i = sum_j e^(x_ij - m_i) v_j / sum_j e^(x_ij - m_i),  m_i = max x_ij
//
// over the tokens j of the row's own sequence, j <= i if causal.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "flash.h"
#include "kernels.h"
#include "wave.h"

namespace swm {
namespace {

using namespace flash;

constexpr int kWaves = 4;
constexpr int kBlock = kWaves * kRows;  // query rows of a workgroup

struct PromptArgs {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  const int32_t* starts;
  int64_t q_t, q_h, k_t, k_h, v_t, v_h, o_t, o_h;
  int32_t B, T, Hq, G, D;
  float c;        // |scale| log2(e), or 1 where the scale is 0
  uint32_t flip;  // sign bits that turn q where the scale is negative
  bool zero;      // the scale is 0
};

// The sequence's part of the packed rows, whatever `starts` holds.
__device__ __forceinline__ void rows_of(const PromptArgs& a, int s, int* first, int* n) {
  const int s0 = min(max(a.starts[s], 0), a.T), s1 = min(max(a.starts[s + 1], 0), a.T);
  *first = s0;
  *n = max(s1 - s0, 0);
}

// The block of query rows that comes at place u: block *j of sequence *s.
// Long blocks go first where every sequence has a lane's register.
template <int kBlock>
__device__ __forceinline__ bool find_block(const PromptArgs& a, int u, int lane, int* s, int* j) {
  int base = 0;
  for (int s0 = 0; s0 < a.B; s0 += 64) {
    int first, n = 0;
    if (s0 + lane < a.B) rows_of(a, s0 + lane, &first, &n);
    const int blocks = (n + kBlock - 1) / kBlock;
    const int upto = base + int(scan_wave(uint32_t(blocks)));
    const uint64_t in = __builtin_amdgcn_ballot_w64(u < upto);
    if (in) {
      const int l = __builtin_ctzll(in);
      *s = s0 + l;
      *j = __builtin_amdgcn_readlane(upto, l) - 1 - u;  // the last block of a sequence first
      return true;
    }
    base = __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
}

template <int NK>
__device__ __forceinline__ void load_query(const PromptArgs& a, int row, int head, int h, half8 (&q)[NK]) {
  const uint16_t* src = a.q + int64_t(row) * a.q_t + int64_t(head) * a.q_h;
#pragma unroll
  for (int x = 0; x < NK; ++x) {
    const int d = 16 * x + 8 * h;
    u32x4 w = *reinterpret_cast<const u32x4*>(src + (d < a.D ? d : 0));
    if (d >= a.D || a.zero) w = u32x4{0, 0, 0, 0};
    q[x] = __builtin_bit_cast(half8, w ^ a.flip);
  }
}

// A row's output; what clear_odd took out of the value rows `from` .. `end` - 1
// goes to the rows that see them.
template <int ND>
__device__ __forceinline__ void finish(const PromptArgs& a, State<ND>& st, const uint16_t* vh, bool odd, int from,
                                       int end, int qi, int n, int first, int head, int h) {
  const float l = sum_halves(st.l);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (odd) {
    for (int t = from; t < end; ++t) {
      if (t > qi) continue;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int x = 32 * d + 8 * (i >> 2) + 4 * h + (i & 3);
          if (x >= a.D) continue;
          const uint16_t w = vh[int64_t(t) * a.v_t + x];
          if ((w & 0x7c00) == 0x7c00) st.o[d][i] += float(__builtin_bit_cast(_Float16, w));
        }
    }
  }
  if (qi >= n) return;
  uint16_t* dst = a.out + int64_t(first + qi) * a.o_t + int64_t(head) * a.o_h;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int x = 32 * d + 2 * i + 4 * h;
      if (x >= a.D) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[x + e] = __builtin_bit_cast(uint16_t, _Float16(st.o[d][i + e] * inv));
    }
}

template <int NK, int ND, int C, bool kCausal>
__global__ __launch_bounds__(64 * kWaves, ND <= 4 ? 2 : 1) void prompt_kernel(PromptArgs a) {
  constexpr int kTile = kTokens * C * 8;  // halves
  constexpr int kLoads = C / kWaves;      // 1 KiB each, of a wave and tile
  extern __shared__ uint16_t smem[];
  uint16_t* sv = smem + 2 * kTile;  // two key tiles, then two value tiles
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int u = blockIdx.x / a.Hq;
  int head = blockIdx.x - u * a.Hq;
  if (a.Hq % 8 == 0) head = (head & 7) * (a.Hq >> 3) + (head >> 3);
  int seq, j;
  if (!find_block<kBlock>(a, u, lane, &seq, &j)) return;
  int first, n;
  rows_of(a, seq, &first, &n);
  first = __builtin_amdgcn_readfirstlane(first);
  n = __builtin_amdgcn_readfirstlane(n);
  const int q0 = j * kBlock + wave * kRows;  // the wave's first row
  const int end = kCausal ? min(n, (j + 1) * kBlock) : n;
  const int hkv = head / a.G;
  const int r = lane & 31, h = lane >> 5;
  const int qi = q0 + r;

  half8 q[NK];
  load_query<NK>(a, first + min(qi, n - 1), head, h, q);

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
  auto load = [&](int t0, int buf) {
    const int left = min(n - t0, kTokens);
    load_tile(kh + int64_t(t0) * a.k_t, ((left - 1) * int(a.k_t) + a.D) * 2, k_off, kLoads,
              to + (buf * kTile + wave * 512) * 2, kWaves * 1024);
    load_tile(vh + int64_t(t0) * a.v_t, ((left - 1) * int(a.v_t) + a.D) * 2, v_off, kLoads,
              to + ((2 + buf) * kTile + wave * 512) * 2, kWaves * 1024);
  };

  // Bytes from the start of LDS: two key tiles, then two value tiles.
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
    if (kCausal && t0 + kTokens > j * kBlock) {
      // An infinity or NaN times a weight of zero would reach rows that do not
      // see its token: zeros in its place here, added to the rows that do at the end.
      uint16_t* vt = sv + buf * kTile;
      bool bad = false;
      for (int i = threadIdx.x; i < kTokens * C; i += 64 * kWaves) bad |= clear_odd(vt + i * 8);
      odd |= __syncthreads_or(bad);
    }
    if (kCausal && t0 > q0 + kRows - 1) return;
    f32x16 s[2];
    scores(at, buf * kTile * 2, q, s);
    if (t0 + kTokens > n || (kCausal && t0 + kTokens - 1 > q0)) {
      const int last = (kCausal ? min(qi, n - 1) : n - 1) - t0 - 4 * h;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (32 * b + 8 * (i >> 2) + (i & 3) > last) s[b][i] = neg_inf();
    }
    half8 p[4];
    weights(st, s, a.c, p);
    outputs(st, at, buf * kTile * 2, p);
  };
  load(0, 0);
  for (int t0 = 0; t0 < end; t0 += 2 * kTokens) {
    step(t0, std::integral_constant<int, 0>());
    if (t0 + kTokens < end) step(t0 + kTokens, std::integral_constant<int, 1>());
  }
  finish(a, st, vh, kCausal && odd, j * kBlock, end, qi, n, first, head, h);
}

// Long prompts: 256 rows, two groups of four waves that take turns on the matrix
// cores.  While one group forms the scores of its next tile and the outputs of
// the one before, the other turns its scores into weights; a barrier after each.
// Tiles of keys and values go round four places in LDS each.
constexpr int kWide = 8;
constexpr int kLong = 512;
constexpr int kWideBlock = kWide * kRows;

__device__ __forceinline__ void turn() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

template <int NK, int ND, int C, bool kCausal>
__global__ __launch_bounds__(64 * kWide, 2) void prompt_wide_kernel(PromptArgs a) {
  constexpr int kTile = kTokens * C * 8;  // halves
  constexpr int kLoads = C / kWide;       // 1 KiB each, of a wave and tile
  extern __shared__ uint16_t smem[];      // four key tiles, four value tiles
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool late = wave >= kWide / 2;  // the group that begins a turn later
  const int u = blockIdx.x / a.Hq;
  int head = blockIdx.x - u * a.Hq;
  if (a.Hq % 8 == 0) head = (head & 7) * (a.Hq >> 3) + (head >> 3);
  int seq, j;
  if (!find_block<kWideBlock>(a, u, lane, &seq, &j)) return;
  int first, n;
  rows_of(a, seq, &first, &n);
  first = __builtin_amdgcn_readfirstlane(first);
  n = __builtin_amdgcn_readfirstlane(n);
  const int q0 = j * kWideBlock + wave * kRows;  // the wave's first row
  const int end = kCausal ? min(n, (j + 1) * kWideBlock) : n;
  const int tiles = (end + kTokens - 1) / kTokens;  // of the workgroup
  const int mine = kCausal ? min(tiles, (q0 + kRows - 1) / kTokens + 1) : tiles;
  const int hkv = head / a.G;
  const int r = lane & 31, h = lane >> 5;
  const int qi = q0 + r;
  half8 q[NK];
  load_query<NK>(a, first + min(qi, n - 1), head, h, q);

  const uint16_t* kh = a.k + int64_t(first) * a.k_t + int64_t(hkv) * a.k_h;
  const uint16_t* vh = a.v + int64_t(first) * a.v_t + int64_t(hkv) * a.v_h;
  uint32_t k_off[kLoads], v_off[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int at = (i * kWide + wave) * 64 + lane, row = at / C, c = at % C;
    const int kc = key_chunk<C>(row, c) * 8, vc = value_chunk<C>(row, c) * 8;
    k_off[i] = kc < a.D ? uint32_t(row * int(a.k_t) + kc) * 2 : 0x80000000u;
    v_off[i] = vc < a.D ? uint32_t(row * int(a.v_t) + vc) * 2 : 0x80000000u;
  }
  const uint32_t to = lds_address(smem);
  // tile i into place i % 4; rows behind the sequence's end are zeros
  auto load_k = [&](int i, int place) {
    const int t0 = i * kTokens, left = min(n - t0, kTokens);
    load_tile(kh + int64_t(t0) * a.k_t, ((left - 1) * int(a.k_t) + a.D) * 2, k_off, kLoads,
              to + (place * kTile + wave * 512) * 2, kWide * 1024);
  };
  auto load_v = [&](int i, int place) {
    const int t0 = i * kTokens, left = min(n - t0, kTokens);
    load_tile(vh + int64_t(t0) * a.v_t, ((left - 1) * int(a.v_t) + a.D) * 2, v_off, kLoads,
              to + ((4 + place) * kTile + wave * 512) * 2, kWide * 1024);
  };
  // Value tile i is here as far as this wave loaded it.  In tiles that some rows
  // see a part of, see prompt_kernel.
  bool odd = false;
  auto arrived = [&](int i, int place) {
    if (!kCausal || i >= tiles || (i + 1) * kTokens <= j * kWideBlock) return;
    uint16_t* vt = smem + (4 + place) * kTile;
#pragma unroll
    for (int x = 0; x < kLoads; ++x) odd |= clear_odd(vt + (x * kWide + wave) * 512 + lane * 8);
  };

  const Reads<NK, ND, C> at(smem, lane, 4 * kTile * 2);
  State<ND> st;
  st.clear();
  f32x16 s[2];
  half8 p[4], k[NK];
  auto softmax = [&] {
    weights(st, s, a.c, p);
    asm volatile("" ::"v"(p[0]), "v"(p[1]), "v"(p[2]), "v"(p[3]), "v"(st.l));  // here, not where they are used
  };
  auto hide = [&](int i) {  // what the rows do not see of tile i
    const int t0 = i * kTokens;
    if (t0 + kTokens > n || (kCausal && t0 + kTokens - 1 > q0)) {
      const int last = (kCausal ? min(qi, n - 1) : n - 1) - t0 - 4 * h;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (32 * b + 8 * (e >> 2) + (e & 3) > last) s[b][e] = neg_inf();
    }
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < tiles) load_k(i, i);
    if (i < 3 && i < tiles) load_v(i, i);
  }
  if (tiles > 3)
    wait_vm<6 * kLoads>();
  else
    wait_vm<0>();
  turn();
  scores(at, 0, q, s);
  hide(0);
  softmax();
  wait_vm<0>();
  arrived(0, 0);
  arrived(1, 1);
  turn();
  if (late) turn();
  // One tile: the products of tile i, then the weights of tile i + 1.  While every
  // row sees all of the tiles up to i + 2 and there are four more of them:
  int i = 0;
  auto step = [&](auto constant) {
    constexpr int x = decltype(constant)::value;  // i % 4
    load_k(i + 4, x);
    load_v(i + 3, (x + 3) % 4);
    __builtin_amdgcn_s_setprio(1);
    scores_and_outputs(st, at, (x + 1) % 4 * kTile * 2, x * kTile * 2, k, q, s, p);
    __builtin_amdgcn_s_setprio(0);
    turn();
    read_first(at, (x + 2) % 4 * kTile * 2, k);  // for the products of the next turn but one
    softmax();
    // the late group reads keys i + 3 and values i + 2 a turn after the early one has
    wait_vm<2 * kLoads>();
    turn();
    ++i;
  };
  const int whole = min((kCausal ? min(j * kWideBlock, n) : n) / kTokens - 2, tiles - 4);
  if (whole >= 4) read_first(at, kTile * 2, k);
  while (i + 4 <= whole) {
    step(std::integral_constant<int, 0>());
    step(std::integral_constant<int, 1>());
    step(std::integral_constant<int, 2>());
    step(std::integral_constant<int, 3>());
  }
#pragma clang loop unroll(disable)
  for (; i < tiles; ++i) {
    const int x = i & 3;
    if (i + 4 < tiles) load_k(i + 4, x);
    if (i + 3 < tiles) load_v(i + 3, (x + 3) & 3);
    if (i + 1 < mine) {
      read_first(at, ((x + 1) & 3) * kTile * 2, k);
      scores_and_outputs(st, at, ((x + 1) & 3) * kTile * 2, x * kTile * 2, k, q, s, p);
    } else if (i < mine)
      outputs(st, at, x * kTile * 2, p);
    turn();
    if (i + 1 < mine) {
      hide(i + 1);
      softmax();
    }
    if (i + 4 < tiles)
      wait_vm<2 * kLoads>();
    else
      wait_vm<0>();
    arrived(i + 2, (x + 2) & 3);
    turn();
  }
  if (!late) turn();
  if (kCausal) odd = __syncthreads_or(odd);
  finish(a, st, vh, odd, j * kWideBlock, end, qi, n, first, head, h);
}

template <int NK, int ND, int C, bool kCausal>
hipError_t launch_as(const PromptArgs& a, uint32_t grid, hipStream_t s) {
  constexpr int kLds = 4 * kTokens * C * 16;
  if (kLds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(prompt_kernel<NK, ND, C, kCausal>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
  }
  prompt_kernel<NK, ND, C, kCausal><<<grid, 64 * kWaves, kLds, s>>>(a);
  return hipGetLastError();
}

template <int NK, int ND, int C, bool kCausal>
hipError_t launch_wide(const PromptArgs& a, uint32_t grid, hipStream_t s) {
  constexpr int kLds = 8 * kTokens * C * 16;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(prompt_wide_kernel<NK, ND, C, kCausal>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (e != hipSuccess) return e;
  prompt_wide_kernel<NK, ND, C, kCausal><<<grid, 64 * kWide, kLds, s>>>(a);
  return hipGetLastError();
}

template <int NK, int ND, int C>
hipError_t launch(const PromptArgs& a, bool causal, uint32_t grid, hipStream_t s) {
  if constexpr (C == 16) {
    if (a.T / a.B >= kLong) {
      const uint32_t blocks = uint32_t(a.T / kWideBlock + std::min(a.T, a.B)) * a.Hq;
      return causal ? launch_wide<NK, ND, C, true>(a, blocks, s) : launch_wide<NK, ND, C, false>(a, blocks, s);
    }
  }
  return causal ? launch_as<NK, ND, C, true>(a, grid, s) : launch_as<NK, ND, C, false>(a, grid, s);
}

}  // namespace

int64_t prompt_grid(int64_t T, int64_t B, int64_t Hq) { return (T / kBlock + std::min(T, B)) * Hq; }

hipError_t launch_prompt(const PromptCall& r, hipStream_t s) {
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
  a.flip = r.scale < 0.f ? 0x80008000u : 0u;
  const uint32_t grid = uint32_t(prompt_grid(r.T, r.B, r.Hq));
  if (a.D <= 64) return launch<4, 2, 8>(a, r.causal, grid, s);
  if (a.D <= 96) return launch<6, 3, 16>(a, r.causal, grid, s);
  if (a.D <= 128) return launch<8, 4, 16>(a, r.causal, grid, s);
  if (a.D <= 192) return launch<12, 6, 32>(a, r.causal, grid, s);
  return launch<16, 8, 32>(a, r.causal, grid, s);
}

}  // namespace swm
