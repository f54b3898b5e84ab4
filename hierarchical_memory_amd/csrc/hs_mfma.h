// What the two attention kernels share: types, loads past the registers into LDS, LDS places, accumulators (gfx950).
#pragma once

#include "hs_internal.h"

namespace hs {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef short s8 __attribute__((ext_vector_type(8)));
typedef float f16 __attribute__((ext_vector_type(16)));
typedef float f4 __attribute__((ext_vector_type(4)));
#define HS_LDS __attribute__((address_space(3)))

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The running maximum moves only when a score passes it by more than this (in powers of two): weights above one are as
// exact (bf16 has the exponents of 32 bits, and only ratios count), and moving it means touching every accumulator.
constexpr float kSlack = 16.0f;

// The tiles' loads go from memory to LDS past the registers, and past the compiler: it would wait for all of them before
// any read of LDS. They are counted here instead. Loads end in their order, so N or fewer on their way means that the
// older ones are in LDS; the wave's own LDS reads have ended too when it passes.
template <int N>
__device__ __forceinline__ void wait_loads_and_meet() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// 16 bytes of each lane's address + kOffset to LDS at lds + 16 * lane (the instruction adds its offset to both). It takes the LDS
// address from m0, a register that is reserved: the compiler keeps nothing in it (a clobber list may not name it), and no other
// instruction of these kernels uses it.
template <int kOffset>
__device__ __forceinline__ void load_to_lds(const char* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off offset:%2" ::"s"(lds - kOffset), "v"(p),
               "n"(kOffset)
               : "memory");
}

// A tile in LDS: its rows' columns in groups of 64 values (128 bytes), one group of all rows after another, and the eight
// 16-byte chunks of a group changing places by the row: 16 rows read at one chunk, and 4 rows at four chunks, meet no bank of
// the 64 twice. A wave's asynchronous load (16 bytes a lane, in order, into LDS) fills eight rows of one group.
__device__ __forceinline__ int swizzle(int row) { return ((row >> 1) & 1) << 2 | ((row >> 2) & 3); }

// A query's eight values, their signs turned where the scale is negative: scores are then scaled by its magnitude, which
// keeps their order.
constexpr uint32_t kSigns = 0x80008000u;
__device__ __forceinline__ bf8 turned(v4u x, uint32_t sign) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] ^= sign;
  return __builtin_bit_cast(bf8, x);
}

// A scale of zero is applied to the queries: as a factor of scores it would make a masked one, -infinity, NaN.
template <int kN>
__device__ __forceinline__ void zero_scaled(bf8 (&q)[kN]) {
#pragma unroll
  for (int s = 0; s < kN; ++s)
#pragma unroll
    for (int i = 0; i < 8; ++i) q[s][i] = (__bf16)((float)q[s][i] * 0.0f);
}

// The magnitude of the scale, to base 2, for such queries. (Below 2^-126 it has fewer digits; what that changes of an exponent
// is less than 2^-22.)
__device__ __forceinline__ float scale_of(float scale) { return scale == 0.0f ? 1.0f : fabsf(scale) * kLog2e; }

// The running maximum m is a score, unscaled, and weights are relative to m times the scale in 32 bits, which one fma takes off
// a scaled score. Its rounding cancels, being the same for all of them, as long as it is small beside the exponents' range:
// from kFar on (where it reaches one) a weight is that of the score's distance from m instead, which any two scores have
// (2^(s scale - m scale) would end at 0 or infinity for the maximum itself from about 2^30 on).
constexpr float kFar = 16777216.0f;
__device__ __forceinline__ bool is_far(float m, float scale) { return fabsf(m * scale) >= kFar; }

// What the product of m and the scale lost in rounding, where the weights are relative to it.
__device__ __forceinline__ float rest_of(float m, float scale) {
  return is_far(m, scale) ? 0.0f : fmaf(m, scale, -(m * scale));
}

// The factor that takes weights relative to the maximum `from` to those relative to `to` (zero from -infinity, no score yet).
__device__ __forceinline__ float rebase(float from, float to, float scale) {
  return from == -INFINITY ? 0.0f
                           : __builtin_amdgcn_exp2f((from - to) * scale + (rest_of(to, scale) - rest_of(from, scale)));
}

// The weights 2^(s scale - m) of two of a lane's scores, rounded to bf16 in p[i] and p[i + 1] for the second product; their
// sum is added to `sum`, that of the rounded ones, one dot product with ones, to `rsum`.
__device__ __forceinline__ void weigh_pair(float s0, float s1, float scale, float m, bf8& p, int i, float& sum,
                                           float& rsum) {
  const bf2 ones = {(__bf16)1.0f, (__bf16)1.0f};
  const float a = __builtin_amdgcn_exp2f(fmaf(s0, scale, -m)), b = __builtin_amdgcn_exp2f(fmaf(s1, scale, -m));
  const bf2 r = {(__bf16)a, (__bf16)b};
  sum += a;
  sum += b;
  rsum = __builtin_amdgcn_fdot2_f32_bf16(r, ones, rsum, false);
  p[i] = r[0];
  p[i + 1] = r[1];
}

// The larger of a lane's value and that of the lane 32 away.
__device__ __forceinline__ float max_of_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// The largest of the values of the four lanes 16 apart.
__device__ __forceinline__ float max_of_quarters(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return max_of_halves(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}

// The matrix unit's first operand read across a tile's rows: lane (column d = lane % 32 of the 32 that `lo` begins) gets rows
// 4 half + 0..3 (from lo) and 8 + 4 half + 0..3 (from hi) of the 16 that begin there, half = lane / 32.
__device__ __forceinline__ s4 read_across(const char* at) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((HS_LDS s4*)(const HS_LDS char*)at);
}
__device__ __forceinline__ bf8 read_across(const char* lo, const char* hi) {
  return __builtin_bit_cast(bf8, __builtin_shufflevector(read_across(lo), read_across(hi), 0, 1, 2, 3, 4, 5, 6, 7));
}

// Where read_across reads in a group of columns for this lane: its row and chunk, for the first and second 32 columns and
// the rows from 0 and from 8 on.
__device__ __forceinline__ int across_place(int lane, int second, int from) {
  const int row = from + 4 * (lane >> 5) + ((lane & 15) >> 2), x = 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
  return row * 128 + (((x ^ swizzle(row)) ^ (4 * second)) << 4) + 8 * (lane & 1);
}

}  // namespace hs
