// What the two ways of the Newton-Schulz products (newton.hip, newton_small.hip) share.
#pragma once

#include "dense.h"

namespace moe {

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4_t __attribute__((ext_vector_type(4)));

// X is stored times this: its values are at least about 2^-14 at the largest size, its singular values at most about 1.2,
// so that neither end leaves fp16's normal range.
constexpr float kXScale = 256.0f;
constexpr int kNormBlocks = 256;  // partial sums of |G|^2 at most

__device__ __forceinline__ uint32_t f16x2_rne(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){a, b}, f16x2_t));
}
__device__ __forceinline__ uint2 pack4_f16(const f32x4_t& v) {
  return make_uint2(f16x2_rne(v[0], v[1]), f16x2_rne(v[2], v[3]));
}
__device__ __forceinline__ f32x4_t unpack4_f16(const uint2& p) {
  return __builtin_convertvector(__builtin_bit_cast(f16x4_t, p), f32x4_t);
}

// Value i of G as stored, and as fp32 (exact). A lane outside the matrix reads a value inside it and takes 0 afterwards:
// a load with its conversion behind a branch is waited for there, one after another (a stack of 3 x 1001 x 600 fp32 took
// 13.6 us for its first X so).
template <int DT>
__device__ __forceinline__ uint32_t stored_at(const void* p, size_t i) {
  if constexpr (DT == kDtF32) return static_cast<const uint32_t*>(p)[i];
  return static_cast<const uint16_t*>(p)[i];
}
template <int DT>
__device__ __forceinline__ float stored_value(uint32_t v) {
  if constexpr (DT == kDtF32) return __uint_as_float(v);
  return DT == kDtBf16 ? __uint_as_float(v << 16) : f16_bits_to_f32(v);
}

// Sum over a block of WAVES waves in a fixed order; every thread has it.
template <int WAVES>
__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) s += lds[w];
  return s;
}

// Matrices with a side of at most kNewtonSmall, taken as m x n with m <= n (newton_small.hip).
constexpr int kNewtonSmall = 256;
struct SmallArgs {
  int m, n, steps;
  int tall;          // G is [n][m], else [m][n]
  const void* g;
  uint16_t* out;     // as G
  float ca, cb, cc;  // a, b, c
  double eps;
  int panels, per_block;
  const double* norm;  // [matrix][norm_parts] parts of |G|^2
  int norm_parts;
  u32x4_t* state;    // X, both parts
  uint16_t* square;  // A, padded
  f32x4_t* part;     // the blocks' parts of A
};
struct SmallLayout {
  size_t state, square, norm, part, total;
};
bool newton_in_one(int m, int n, int batch);
SmallLayout newton_small_layout(int m, int n, int batch);
hipError_t launch_newton_one(SmallArgs a, int batch, int dtype, hipStream_t st);     // all of it
hipError_t launch_newton_panels(SmallArgs a, int batch, int dtype, hipStream_t st);  // from |G|^2 on

}  // namespace moe
