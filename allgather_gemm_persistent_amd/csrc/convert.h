// Conversions between a chunk of 8 elements in memory and 8 floats, for the row operators.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace agg {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ inline void widen(const u32x4& p, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __builtin_bit_cast(float, p[i] << 16);
    v[2 * i + 1] = __builtin_bit_cast(float, p[i] & 0xFFFF0000u);
  }
}

// eight floats as bfloat16, nearest even
__device__ inline u32x4 narrow(const float (&v)[8]) {
  u32x4 p;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    p[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[2 * i], v[2 * i + 1]}, bf16x2));
  return p;
}

// eight floats as e4m3, nearest even (beyond 464 a NaN: the caller keeps them inside)
__device__ inline u32x2 narrow_e4m3(const float (&v)[8]) {
  u32x2 p;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int q = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h], v[4 * h + 1], 0, false);
    p[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2], v[4 * h + 3], q, true);
  }
  return p;
}

// a float inside e4m3's range; a NaN stays one
__device__ inline float clamp_e4m3(float v) { return v != v ? v : fminf(fmaxf(v, -448.0f), 448.0f); }

constexpr float kNormal = 1.17549435e-38f;   // the least float of full precision, 2^-126

}  // namespace agg
