// mx_format.hpp -- the microscaled formats on the device: a group's scale byte, and codes of its elements.
#pragma once

#include <hip/hip_runtime.h>

#include "dash_internal.hpp"

namespace dash {
namespace {

typedef float f32x8 __attribute__((ext_vector_type(8), aligned(16)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int GROUP = MX_GROUP;

// The format's scale byte for a group whose largest magnitude has the bits `top`
template <int F>
__device__ __forceinline__ unsigned scale_byte(unsigned top) {
  constexpr int lead = F == DASH_MX_E2M1 ? 2 : 8;                       // m = 1.5 2^2 or 1.75 2^8
  constexpr unsigned frac = F == DASH_MX_E2M1 ? 0x400000u : 0x600000u;  // the fraction of m
  const int e = (int)(top >> 23) - lead + ((top & 0x7fffffu) > frac ? 1 : 0);
  return top >= 0x7f800000u ? 255u : (unsigned)(e < 0 ? 0 : e);
}

// Codes of 8 values of a group with that scale byte: 8 bytes (E4M3) or 4 (E2M1)
template <int F>
struct Codes;
template <>
struct Codes<DASH_MX_E4M3> {
  typedef u32x2 type;
  static constexpr int BITS = 8;
  static __device__ __forceinline__ type encode(const f32x8& x, unsigned byte) {
    float y[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) y[q] = byte == 255u ? 0.f : ldexpf(x[q], 127 - (int)byte);
    type c;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      s16x2 v = {0, 0};
      v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v, y[4 * w], y[4 * w + 1], 1.f, false);
      v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v, y[4 * w + 2], y[4 * w + 3], 1.f, true);
      c[w] = __builtin_bit_cast(unsigned, v);
    }
    return c;
  }
  typedef unsigned raw4;
  // codes of 4 values of a group with that scale byte
  static __device__ __forceinline__ raw4 encode4(const float* x, unsigned byte) {
    float y[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) y[q] = byte == 255u ? 0.f : ldexpf(x[q], 127 - (int)byte);
    s16x2 v = {0, 0};
    v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v, y[0], y[1], 1.f, false);
    v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v, y[2], y[3], 1.f, true);
    return __builtin_bit_cast(unsigned, v);
  }
  // the values of 4 codes
  static __device__ __forceinline__ f32x4 decode(raw4 c) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, 1.f, false);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, 1.f, true);
    return f32x4{a[0], a[1], b[0], b[1]};
  }
};
template <>
struct Codes<DASH_MX_E2M1> {
  typedef unsigned type;
  static constexpr int BITS = 4;
  static __device__ __forceinline__ type encode(const f32x8& x, unsigned byte) {
    float y[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) y[q] = byte == 255u ? 0.f : ldexpf(x[q], 127 - (int)byte);
    type c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[0], y[1], 1.f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[2], y[3], 1.f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[4], y[5], 1.f, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[6], y[7], 1.f, 3);
    return c;
  }
  typedef uint16_t raw4;
  static __device__ __forceinline__ raw4 encode4(const float* x, unsigned byte) {
    float y[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) y[q] = byte == 255u ? 0.f : ldexpf(x[q], 127 - (int)byte);
    unsigned c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[0], y[1], 1.f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[2], y[3], 1.f, 1);
    return (raw4)c;
  }
  static __device__ __forceinline__ f32x4 decode(raw4 c) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4((unsigned)c, 1.f, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4((unsigned)c, 1.f, 1);
    return f32x4{a[0], a[1], b[0], b[1]};
  }
};

__device__ __forceinline__ unsigned mag_bits(float x) { return __builtin_bit_cast(unsigned, x) & 0x7fffffffu; }

__device__ __forceinline__ unsigned umax(unsigned a, unsigned b) { return a > b ? a : b; }
__device__ __forceinline__ unsigned umin(unsigned a, unsigned b) { return a < b ? a : b; }

}  // namespace
}  // namespace dash
