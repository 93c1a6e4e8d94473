// Device-side pieces shared by the latent-attention kernels (gfx950).
//
// Both attention kernels compute the transposed products
//   S^T = K Q^T   (rows: keys, columns: query rows)
//   O^T = V^T P^T (rows: value columns, columns: query rows)
// so that a lane's MFMA results all belong to ONE query row (column l%16 of
// a 16 x 16 result, l%32 of a 32 x 32 one): the softmax's maximum, sum and
// rescaling are per-lane values, and the probabilities a lane computes are
// already its B operand of the second product.  The contraction over keys
// may run in any order as long as both operands agree: a lane holds the
// keys its S^T registers hold, and V^T is read from LDS for those keys by
// the transposing read (ds_read_b64_tr_b16: within 16 lanes, lane i supplies
// the address of 4 consecutive 16-bit values of key i/4, columns 4 (i%4)..,
// and receives column i of the 4 keys; lane layout measured on MI355X).
//
// Key and value rows reach LDS by direct loads (global_load_lds_dwordx4:
// lane l's 16 bytes land at the wave's LDS base + 16 l), issued by inline
// assembly so that the compiler does not wait for them before every LDS
// read; the kernels wait by hand.  A row's 16-byte chunks are permuted when
// they are fetched (the lane that fills LDS chunk p fetches chunk
// p ^ swizzle(row)), so that equal chunks of neighbouring rows, which the
// 16-byte reads of K and the transposing reads of V take together, lie in
// different banks.  The forms of 32 query rows a wave read without conflicts.
// The 16-row form does not: lanes l and l ^ 16 take two chunks of one row
// there, which the permutation does not keep apart, and the counters show 144
// cycles of conflicts a tile, 4 for each of its 36 K reads, a third of its LDS
// cycles (memory bounds that form; its LDS is busy 13% of the time).
#pragma once

#include <type_traits>
#include <utility>

#include "mxfp4_device.h"

namespace mxfp4 {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4s* lds_v4s_t;
typedef __attribute__((address_space(3))) v8s* lds_v8s_t;
typedef __attribute__((address_space(3))) v4f* lds_v4f_t;
typedef __attribute__((address_space(3))) float* lds_f32_t;
typedef __attribute__((address_space(3))) int* lds_i32_t;
typedef __attribute__((address_space(3))) int64_t* lds_i64_t;

// LDS by byte address (a kernel's only __shared__ array starts at 0).
__device__ __forceinline__ v8bf lds_read16(uint32_t a) {
  return __builtin_bit_cast(v8bf, *(lds_v8s_t)(uintptr_t)a);
}
__device__ __forceinline__ v4s lds_read_tr(uint32_t a) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t)(uintptr_t)a);
}
__device__ __forceinline__ v8bf join_keys(v4s a, v4s b) {
  return __builtin_bit_cast(v8bf, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Reverses 3 bits of the row's pair number: the swizzle of 128-byte rows, of
// which a 256-byte bank line holds two.  16 rows' equal chunks fall on 16
// different slots, and so do the chunk pairs of 8 rows and the chunk quads of
// 4 rows.
__host__ __device__ constexpr uint32_t swizzle128(uint32_t row) {
  return ((row & 2) << 1) | ((row & 4) >> 1) | ((row & 8) >> 3);
}
// Reverses 4 bits: the swizzle of rows whose length is a multiple of 256
// bytes.  16 rows' equal chunks fall on 16 different slots (K reads), and so
// do the chunk pairs of 8 rows and the chunk quads of 4 rows (V reads): no
// conflicts measured.
__host__ __device__ constexpr uint32_t bitrev4(uint32_t r) {
  return ((r & 1) << 3) | ((r & 2) << 1) | ((r & 4) >> 1) | ((r & 8) >> 3);
}

// Direct loads of 16 bytes per lane to LDS at `lds` + 16 lane, from a
// uniform base plus a lane's byte offset, or OFF bytes past a lane's own
// address.  (M0 holds the LDS base; one wait state after it is written;
// nothing else in these kernels uses it.  A
// base that a vector instruction wrote would need five: the compiler does
// not count them into an assembly statement, so there are four here.)
__device__ __forceinline__ void dma16(uint32_t lds, const void* base, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2"
               :: "s"(lds), "v"(voff), "s"(base) : "memory");
}
// (The instruction adds its immediate offset to the LDS address too.)
// STREAM: rows that nothing reads again are loaded past the caches.
template <int OFF, bool STREAM>
__device__ __forceinline__ void dma16_at(uint32_t lds, const void* p) {
  lds -= OFF;
  if constexpr (STREAM)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off offset:%2 nt"
                 :: "s"(lds), "v"(p), "i"(OFF) : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off offset:%2"
                 :: "s"(lds), "v"(p), "i"(OFF) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" :: "i"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void wave_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// A barrier for LDS alone: stores to memory stay under way across it.
__device__ __forceinline__ void lds_barrier() {
  wait_lds();
  wave_barrier();
}

// The larger / the sum of x over the lanes that share a query row: lanes
// l, l ^ 32 (RW = 32), and l ^ 16 too (RW = 16).  The lane-swap
// instructions on two copies of x give each lane both halves' values.
template <int RW>
__device__ __forceinline__ float rows_max(float x) {
  if constexpr (RW == 16) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  }
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
template <int RW>
__device__ __forceinline__ float rows_sum(float x) {
  if constexpr (RW == 16) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  }
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// The larger / the sum of x over the 64 lanes, by lane permutations (no LDS):
// the lane's pair, quad, half row and row of 16, then the two swaps.
template <typename T, typename Op>
__device__ __forceinline__ T wave_reduce(T x, Op op) {
  static_assert(sizeof(T) == 4, "one register");
  auto with = [&](int y) { x = op(x, __builtin_bit_cast(T, y)); };
  with(__builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), 0xB1, 0xF, 0xF, true));   // lane ^ 1
  with(__builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), 0x4E, 0xF, 0xF, true));   // lane ^ 2
  with(__builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), 0x141, 0xF, 0xF, true));  // mirrored in 8
  with(__builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), 0x140, 0xF, 0xF, true));  // mirrored in 16
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  x = op(__builtin_bit_cast(T, (uint32_t)a[0]), __builtin_bit_cast(T, (uint32_t)a[1]));
  const uint32_t w = __builtin_bit_cast(uint32_t, x);
  const auto c = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return op(__builtin_bit_cast(T, (uint32_t)c[0]), __builtin_bit_cast(T, (uint32_t)c[1]));
}
template <typename T>
__device__ __forceinline__ T wave_sum(T x) {
  return wave_reduce(x, [](T a, T b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float x) {
  return wave_reduce(x, [](float a, float b) { return fmaxf(a, b); });
}

// MFMA by the number of query rows (columns): K = 32 of 16 x 16, K = 16 of
// 32 x 32.  Either way a lane's operand is 8 bf16.
__device__ __forceinline__ v4f mfma_rows(v8bf a, v8bf b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ v16f mfma_rows(v8bf a, v8bf b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// A chain of 32 x 32 products with its sum in vector registers, for kernels
// whose other accumulators fill all accumulation registers.  The compiler
// counts no wait states after an assembly statement, so the last product
// carries the wait that its sum's first reader (or copy) needs.
template <bool FIRST, bool LAST>
__device__ __forceinline__ void mfma_vgpr(v16f& c, v8bf a, v8bf b) {
  static_assert(!(FIRST && LAST), "a chain has two products at least");
  if constexpr (FIRST) asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, 0" : "=&v"(c) : "v"(a), "v"(b));
  else if constexpr (LAST)
    asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0\n\ts_nop 15\n\ts_nop 3" : "+v"(c) : "v"(a), "v"(b));
  else asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
}

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The running maximum may lag the true one by this many powers of two
// before the accumulators are rescaled: probabilities then reach 2^8, which
// changes no relative rounding, and most tiles rescale nothing.
constexpr float kLag = 8.0f;

// A row's sums of probabilities: of the exact ones, for the log-sum-exp, and
// of the bf16 ones the value product takes, for the output's division.  What
// rounding does to a probability then moves the weights but not their sum: a
// row that one key dominates keeps that key's value to the last bit.
struct RowSums {
  float exact = 0, used = 0;
  __device__ __forceinline__ void scale(float f) {
    exact *= f;
    used *= f;
  }
  __device__ __forceinline__ float inverse() const { return used == 0 ? 0.0f : 1.0f / used; }
  __device__ __forceinline__ float log_sum_exp(float m) const {  // m: the maximum, in units of log2
    return exact > 0 ? (m + __builtin_amdgcn_logf(exact)) * kLn2 : exact == 0 ? kNegInf : exact;
  }
};
// Two rounded probabilities a step: their dot product with ones.
__device__ __forceinline__ float add_rounded(const v8bf& p, float sum) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const v2bf one = {(__bf16)1.0f, (__bf16)1.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) sum = __builtin_amdgcn_fdot2_f32_bf16(v2bf{p[2 * i], p[2 * i + 1]}, one, sum, false);
  return sum;
}

// Probabilities of a tile from its scores x (one query row per lane):
// updates the row's maximum m (in units of log2, scores times c) and the
// lane's share of the row's sums, rounds to bf16 operands.  True if any
// row's maximum rose: the caller then rescales its accumulators by alpha.
// (bf16 is what the matrix units multiply with the bf16 values at full rate; a
// second product with the roundings' rests would double the value side.  The
// outputs' error against 64 bits, relative norm, beside that of exact results
// rounded to bf16: decode 1.7e-3 and 1.7e-3, prompts 2.0e-3 to 2.3e-3 and
// 1.6e-3.)
template <int RW, int NX>
__device__ __forceinline__ bool softmax_step(float (&x)[NX], float c, float& m, RowSums& l, float& alpha,
                                             v8bf (&p)[NX / 8]) {
  float mx = x[0];
#pragma unroll
  for (int i = 1; i < NX; ++i) mx = fmaxf(mx, x[i]);
  mx = rows_max<RW>(mx) * c;
  bool grew = false;
  if (__builtin_amdgcn_ballot_w64(mx > m + kLag)) {
    const float mn = fmaxf(m, mx);
    alpha = m == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
    grew = __builtin_amdgcn_ballot_w64(alpha != 1.0f) != 0;  // (no row's first keys: zeros need no scaling)
    m = mn;
    l.scale(alpha);
  }
  const float mu = m == kNegInf ? 0.0f : m;  // a row that has seen nothing yet
#pragma unroll
  for (int i = 0; i < NX; ++i) {
    x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], c, -mu));
    l.exact += x[i];
  }
#pragma unroll
  for (int i = 0; i < NX / 8; ++i) {
    v8bf t;
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = (__bf16)x[8 * i + j];
    p[i] = t;
    l.used = add_rounded(t, l.used);
  }
  return grew;
}

// Accumulators that stay in accumulation registers: vector instructions
// cannot take those, and where plain C++ reads them the compiler moves all of
// them through vector registers ahead of any branch, in the loop on every
// tile.  So they are read and written one by one, by assembly statements,
// behind a wait for matrix results still in flight (which the compiler does
// not count for assembly statements).
__device__ __forceinline__ void acc_settle() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 15\n\ts_nop 7" ::: "memory");
}
__device__ __forceinline__ float acc_read(float a) {
  float v;
  asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a));
  return v;
}
// o *= alpha
template <typename V, int N>
__device__ __forceinline__ void rescale(V (&o)[N], float alpha) {
  acc_settle();
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int j = 0; j < (int)(sizeof(V) / 4); ++j) {
      const float t = acc_read(o[i][j]) * alpha;
      float r;
      asm volatile("v_accvgpr_write_b32 %0, %1" : "=a"(r) : "v"(t));
      o[i][j] = r;
    }
  }
  asm volatile("s_nop 3" ::: "memory");
}

// A run of N matrix steps whose operands come from LDS in groups of G: the
// next group's reads are issued before this group's products, and nothing
// moves between groups, so that a wave alone on its SIMD hides the LDS
// latency behind G products and no more than two groups are in registers.
// read(i) gives step i's operand, mul(i, operand) uses it, i a compile-time
// constant; `now` holds group 0, read ahead by the caller.  (Recursion, not
// a loop: the operand registers need constant indices, and the compiler does
// not unroll every such loop.)
template <int AT, typename T, int G, typename Mul, int... I>
__device__ __forceinline__ void multiply_group(T (&now)[G], Mul& mul, std::integer_sequence<int, I...>) {
  (mul(std::integral_constant<int, AT + I>{}, now[I]), ...);
}
template <int AT, typename T, int G, typename Read, int... I>
__device__ __forceinline__ void read_group_at(T (&next)[G], Read& read, std::integer_sequence<int, I...>) {
  ((next[I] = read(AT + I)), ...);
}
template <int N, int G, int AT = 0, typename T, typename Read, typename Mul>
__device__ __forceinline__ void pipeline(T (&now)[G], Read read, Mul mul) {
  static_assert(N % G == 0, "whole groups");
  T next[G];
  if constexpr (AT + G < N) read_group_at<AT + G>(next, read, std::make_integer_sequence<int, G>{});
  multiply_group<AT>(now, mul, std::make_integer_sequence<int, G>{});
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (AT + G < N) pipeline<N, G, AT + G>(next, read, mul);
}
template <int G, typename T, typename Read>
__device__ __forceinline__ void read_group(T (&first)[G], Read read) {
  read_group_at<0>(first, read, std::make_integer_sequence<int, G>{});
  __builtin_amdgcn_sched_barrier(0);
}

// Key (within a 32-key tile) of a lane's score register i.
template <int RW>
__device__ __forceinline__ int key_of(int i, uint32_t lane) {
  if constexpr (RW == 16) return 16 * (i >> 2) + 4 * (int)(lane >> 4) + (i & 3);
  else return 8 * (i >> 2) + 4 * (int)(lane >> 5) + (i & 3);
}

}  // namespace mxfp4
