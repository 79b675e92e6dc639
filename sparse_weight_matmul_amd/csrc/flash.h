// Pieces of an attention with many query rows, on v_mfma_f32_32x32x16_f16: a
// wave takes 32 query rows and 32 or 64 tokens at a time, from key and value tiles
// in LDS.
//
// Scores are formed transposed, S^T = K Q^T (A: 32 tokens, B: 32 query rows):
// lane l of the result holds, for the one row l % 32, the tokens 8 (i / 4) + 4
// (l / 32) + i % 4 of its registers i.  Sums and maxima are then per lane but
// for one exchange with lane l ^ 32, and the weights are the second product's
// B operand as they stand, O^T = V^T P^T: step s of 16 tokens takes registers
// 8 (s % 2) .. + 7 of score block s / 2, which are tokens 16 s + 8 (e / 4) + 4
// (l / 32) + e % 4.  Its A operand, the same tokens of dimension l % 32, is
// read from the row-major value tile by the transposing LDS read
// (ds_read_b64_tr_b16: of 16 lanes, lane j gets element j of four rows).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace swm {
namespace flash {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr;

constexpr int kTokens = 64;  // of a tile
constexpr int kRows = 32;    // query rows of a wave

// The weights e^(x - m) go into the second product as fp16, once rounded (2^-11
// of each, as large as the output's own rounding), times 2^kUp.  The sum that
// divides is that of the rounded weights, so that what they lose together
// cancels.  m is the largest score when it was last looked for: a row's scores may
// outgrow it by a factor of 2^(16 - kUp) before a weight leaves fp16's range,
// which the sum shows, and only then is the largest looked for again (looking in
// every tile took a quarter of its vector instructions).  Weights down to 2^-24
// of the largest keep their relative precision; smaller ones are off by 2^-35 of it at most.
// Measured over prompts and trees of all sizes, in the 2-norm of the outputs: 2.1 to
// 2.7e-4 from the result in 64 bits, which rounded once to fp16 is 1.7 to 2.1e-4 away.
constexpr float kUp = 10.f;

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// Where a tile's 16-byte chunk c of a row is kept: the row's chunks are
// permuted so that the reads of eight or sixteen rows meet all banks.
// C: chunks of a row in LDS, 8, 16 or 32.
template <int C>
__device__ __forceinline__ int key_chunk(int row, int c) {
  return C == 8 ? c ^ ((row >> 1) & 7) : c ^ (row & 15);
}
template <int C>
__device__ __forceinline__ int value_chunk(int row, int c) {
  return C == 8 ? c ^ (((row >> 1) & 1) << 2) : c ^ ((row & 3) << 2 | ((row >> 2) & 3));
}

__device__ __forceinline__ void both_halves(float v, float* a, float* b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  *a = __uint_as_float(r[0]);
  *b = __uint_as_float(r[1]);
}
__device__ __forceinline__ float max_halves(float v) {
  float a, b;
  both_halves(v, &a, &b);
  return fmaxf(a, b);
}
__device__ __forceinline__ float sum_halves(float v) {
  float a, b;
  both_halves(v, &a, &b);
  return a + b;
}

// A wave's running state for 32 rows: m (of the unscaled scores), what it adds to
// a score in units of log2 (infinity while there is none, so that the first tile
// looks for it), the sum per lane's row over the lane's own tokens; O^T.
template <int ND>
struct State {
  float m, base, l;
  f32x16 o[ND];
  __device__ __forceinline__ void clear() {
    m = neg_inf();
    base = __builtin_inff();
    l = 0.f;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  }
};

// What a lane reads of a tile, in bytes from the tile's start: key chunks 2 x +
// h of row r, and value chunks of four rows (e: of eight).  The rest of an
// address is the same for all lanes and goes into the instruction.
typedef const __attribute__((address_space(3))) uint8_t* lds_bytes;
template <int NK, int ND, int C>
struct Reads {
  lds_bytes base;
  uint32_t k[NK], v[2][ND];
  // values: bytes from the first key tile to the first value tile
  __device__ __forceinline__ Reads(const uint16_t* lds, int lane, int values) : base((lds_bytes)lds) {
    const int r = lane & 31, j = lane & 15, d16 = (lane >> 4) & 1, h = lane >> 5;
#pragma unroll
    for (int x = 0; x < NK; ++x) k[x] = (r * C + key_chunk<C>(r, 2 * x + h)) * 16;
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        const int row = 8 * e + 4 * h + (j >> 2);
        v[e][d] = values + (row * C + value_chunk<C>(row, 4 * d + 2 * d16 + ((j & 3) >> 1))) * 16 + 8 * (j & 1);
      }
  }
};

// A query row's fragments, and what the scale's sign and a D that is no multiple
// of 16 make of them: apart, so that nothing waits for the loads before it has to.
template <int NK>
__device__ __forceinline__ void load_query(const uint16_t* row, int D, int h, half8 (&q)[NK]) {
#pragma unroll
  for (int x = 0; x < NK; ++x) {
    const int d = 16 * x + 8 * h;
    q[x] = *reinterpret_cast<const half8*>(row + (d < D ? d : 0));
  }
}
template <int NK>
__device__ __forceinline__ void mend_query(int D, int h, bool zero, uint32_t flip, half8 (&q)[NK]) {
  if (D == 16 * NK && !zero && !flip) return;
#pragma unroll
  for (int x = 0; x < NK; ++x) {
    u32x4 w = __builtin_bit_cast(u32x4, q[x]);
    if (16 * x + 8 * h >= D || zero) w = u32x4{0, 0, 0, 0};
    q[x] = __builtin_bit_cast(half8, w ^ flip);
  }
}

// Key fragment x of 32 tokens at `at` (bytes), and value fragment d of 16.
template <int NK, int ND, int C>
__device__ __forceinline__ half8 read_keys(const Reads<NK, ND, C>& a, int at, int x) {
  return *reinterpret_cast<const __attribute__((address_space(3))) half8*>(a.base + a.k[x] + at);
}
template <int NK, int ND, int C>
__device__ __forceinline__ half8 read_values(const Reads<NK, ND, C>& a, int at, int d) {
  u32x4 w;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const s16x4 t =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(a.base + a.v[e][d] + at));
    const u32x2 u = __builtin_bit_cast(u32x2, t);
    w[2 * e] = u[0];
    w[2 * e + 1] = u[1];
  }
  return __builtin_bit_cast(half8, w);
}

// Scores of 32 NB tokens of the key tile at `at` (bytes), before the scale.
template <int NB, int NK, int ND, int C>
__device__ __forceinline__ void scores(const Reads<NK, ND, C>& a, int at, const half8 (&q)[NK], f32x16 (&s)[NB]) {
  half8 f[NB][NK];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int x = 0; x < NK; ++x)  // rows 32 apart have their chunks in the same order
      f[b][x] = read_keys(a, at + b * 32 * C * 16, x);
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    s[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[b][0], q[0], f32x16{}, 0, 0, 0);
#pragma unroll
    for (int x = 1; x < NK; ++x) s[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[b][x], q[x], s[b], 0, 0, 0);
  }
  if (NB < 2 || NK > 8) return;  // nothing to overlap, or no registers for it
  // half of the fragments are on their way before the first product
  __builtin_amdgcn_sched_group_barrier(0x100, NK, 0);
#pragma unroll
  for (int x = 0; x < NK; ++x) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, NK, 0);
}

// 2^(s c + base) as fp16, and their sum; c > 0: scale in units of log2.
template <int NB>
__device__ __forceinline__ float powers(const f32x16 (&s)[NB], float c, float base, half8 (&p)[2 * NB]) {
  float sum[2 * NB];
#pragma unroll
  for (int x = 0; x < 2 * NB; ++x) {
    u32x4 w;
    sum[x] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x >> 1][8 * (x & 1) + e], c, base));
      const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x >> 1][8 * (x & 1) + e + 1], c, base));
      const half2v h = __builtin_convertvector(f32x2{p0, p1}, half2v);
      sum[x] = __builtin_amdgcn_fdot2(h, half2v{_Float16(1.f), _Float16(1.f)}, sum[x], false);
      w[e >> 1] = __builtin_bit_cast(uint32_t, h);
    }
    p[x] = __builtin_bit_cast(half8, w);
  }
#pragma unroll
  for (int x = 1; x < 2 * NB; ++x) sum[0] += sum[x];
  return sum[0];
}

// The weights of a tile's scores, and the running sum.  fresh: it is the first tile.
template <int NB, int ND>
__device__ __forceinline__ void weights(State<ND>& st, const f32x16 (&s)[NB], float c, bool fresh, half8 (&p)[2 * NB]) {
  float sum = __builtin_inff();
  if (!fresh) sum = powers(s, c, st.base, p);
  if (__builtin_amdgcn_ballot_w64(!(sum < __builtin_inff()))) {
    float mx = s[0][0];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[b][i]);
    const float m = fmaxf(max_halves(mx), st.m);
    const float f = m == st.m ? 1.f : __builtin_amdgcn_exp2f((st.m - m) * c);
    st.m = m;
    st.l *= f;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) st.o[d][i] *= f;
    const bool none = m == neg_inf();  // nothing live so far: weights of 2^-inf
    const float base = none ? 0.f : kUp - m * c;
    st.base = none ? __builtin_inff() : base;
    sum = powers(s, c, base, p);
  }
  st.l += sum;
}

// O^T += V^T P^T over the 16 NX tokens of the value tile at `at` (bytes).
template <int NX, int NK, int ND, int C>
__device__ __forceinline__ void outputs(State<ND>& st, const Reads<NK, ND, C>& a, int at, const half8 (&p)[NX]) {
  half8 f[NX][ND];
#pragma unroll
  for (int x = 0; x < NX; ++x)
#pragma unroll
    for (int d = 0; d < ND; ++d)  // rows 16 apart have their chunks in the same order
      f[x][d] = read_values(a, at + x * 16 * C * 16, d);
#pragma unroll
  for (int x = 0; x < NX; ++x)
#pragma unroll
    for (int d = 0; d < ND; ++d) st.o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[x][d], p[x], st.o[d], 0, 0, 0);
  if (ND > 4) return;
  __builtin_amdgcn_sched_group_barrier(0x100, 2 * ND, 0);
#pragma unroll
  for (int x = 0; x < (NX - 1) * ND; ++x) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, ND, 0);
}

// Loads of 16 bytes a lane straight into LDS, lane l's to `to` + 16 l.  In
// assembly, so that the compiler does not wait for them before the next
// transposing read, of another tile; who reads what they bring waits for it
// himself (wait_vm).  They have no register for a result.  The counter that
// the compiler's own waits look at runs in order, so that these only make them
// longer.  Their place in LDS is an operand in m0, which the compiler writes
// itself: a statement that wrote it would have to name it, and m0 cannot be named
// as clobbered.
__device__ __forceinline__ uint32_t lds_address(const uint16_t* p) {
  return __builtin_amdgcn_readfirstlane(uint32_t(reinterpret_cast<uintptr_t>((lds_ptr)(const_cast<uint16_t*>(p)))));
}
__device__ __forceinline__ void to_lds(uint64_t at, uint32_t to) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(at), "{m0}"(to) : "memory");
}
__device__ __forceinline__ void to_lds(uint64_t base, uint32_t off, uint32_t to) {  // base: of the whole wave
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(to) : "memory");
}
// The same for the lanes of `on` alone, one at least, so that it is always counted:
// a branch round it would change how many are on their way.
__device__ __forceinline__ void to_lds_some(uint64_t at, uint32_t to, uint64_t on) {
  uint64_t all;
  asm volatile(
      "s_and_saveexec_b64 %0, %3\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, off\n\ts_mov_b64 exec, %0"
      : "=&s"(all)
      : "v"(at), "{m0}"(to), "s"(on)
      : "memory", "scc");
}
// A word, or a byte as a word, of each lane of `on`: lane l's to `to` + 4 l.
__device__ __forceinline__ void word_to_lds(const void* at, uint32_t to, uint64_t on) {
  uint64_t all;
  asm volatile(
      "s_and_saveexec_b64 %0, %3\n\ts_nop 4\n\tglobal_load_lds_dword %1, off\n\ts_mov_b64 exec, %0"
      : "=&s"(all)
      : "v"(at), "{m0}"(to), "s"(on)
      : "memory", "scc");
}
__device__ __forceinline__ void byte_to_lds(const void* at, uint32_t to, uint64_t on) {
  uint64_t all;
  asm volatile(
      "s_and_saveexec_b64 %0, %3\n\ts_nop 4\n\tglobal_load_lds_ubyte %1, off\n\ts_mov_b64 exec, %0"
      : "=&s"(all)
      : "v"(at), "{m0}"(to), "s"(on)
      : "memory", "scc");
}

// A wave's part of a tile, n such loads of 1 KiB: 16 bytes at `off` from `src` a
// lane, those from `bytes` on as zeros.
__device__ __forceinline__ void load_tile(const uint16_t* src, int bytes, const uint32_t* off, int n, uint32_t to,
                                          int step) {
  const uint64_t base = reinterpret_cast<uint64_t>(src);
  const u32x4 resource = {uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(base))),
                          uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(base >> 32))) & 0xffffu,
                          uint32_t(__builtin_amdgcn_readfirstlane(bytes)), 0x00020000u};
#pragma unroll
  for (int i = 0; i < n; ++i)
    asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(off[i]), "s"(resource),
                 "{m0}"(to + i * step)
                 : "memory");
}

// A row's output, O^T times `inv`, rounded; four dimensions a store where rows
// are aligned to them.
template <int ND>
__device__ __forceinline__ void write_row(const State<ND>& st, float inv, uint16_t* dst, int D, int h) {
  const bool wide = (reinterpret_cast<uintptr_t>(dst) & 7) == 0;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int x = 32 * d + 2 * i + 4 * h;
      const half2v lo = __builtin_convertvector(f32x2{st.o[d][i] * inv, st.o[d][i + 1] * inv}, half2v);
      const half2v hi = __builtin_convertvector(f32x2{st.o[d][i + 2] * inv, st.o[d][i + 3] * inv}, half2v);
      const u32x2 w = {__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
      if (D < 32 * ND && x >= D) continue;
      if (wide) {
        *reinterpret_cast<u32x2*>(dst + x) = w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[x + e] = uint16_t(w[e >> 1] >> (16 * (e & 1)));
      }
    }
}

// Zeros for the infinities and NaN among eight halves in LDS; whether there were any.
__device__ __forceinline__ bool clear_odd(uint16_t* at) {
  u32x4 w = *reinterpret_cast<u32x4*>(at);
  bool any = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const bool lo = (w[e] & 0x7c00u) == 0x7c00u, hi = (w[e] & 0x7c000000u) == 0x7c000000u;
    any |= lo | hi;
    w[e] &= (lo ? 0xffff0000u : ~0u) & (hi ? 0x0000ffffu : ~0u);
  }
  if (any) *reinterpret_cast<u32x4*>(at) = w;
  return any;
}

// s_waitcnt: at most n vector memory operations of this wave outstanding.
template <int n>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((n & 15) | (7 << 4) | (15 << 8) | (((n >> 4) & 3) << 14));
}

}  // namespace flash
}  // namespace swm
