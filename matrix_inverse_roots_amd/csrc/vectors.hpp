// vectors.hpp -- 16-byte pieces of rows of fp32, binary16 or bfloat16 on the device.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

namespace dash {
namespace {

// 16 bytes of elements that start on any element: the hardware takes such loads and stores whole
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  typedef float type __attribute__((ext_vector_type(4), aligned(4)));
};
template <>
struct Vec<__bf16> {
  typedef __bf16 type __attribute__((ext_vector_type(8), aligned(2)));
};
template <>
struct Vec<_Float16> {
  typedef _Float16 type __attribute__((ext_vector_type(8), aligned(2)));
};
template <typename T>
using vec_of = typename Vec<T>::type;
template <typename T>
constexpr int EACH = 16 / (int)sizeof(T);

// w >> (8 BYTES - bits): the last elements of w come first, zeros follow.  0 < bits < 8 BYTES.
__device__ __forceinline__ uint64_t last_first(uint64_t w, int bits) { return w >> (64 - bits); }
struct Bytes16 {
  uint64_t lo, hi;
};
__device__ __forceinline__ Bytes16 last_first(Bytes16 w, int bits) {
  const int by = 128 - bits;
  if (by >= 64) return {w.hi >> (by - 64), 0};
  return {(w.lo >> by) | (w.hi << (64 - by)), w.hi >> by};
}

// The N elements from c on of a row of n, zero beyond it: one load, where the row ends inside the piece of the
// row's last N elements.  n >= N, or 0 (nothing is loaded).  PAST, here and below: past the caches, for what is far
// larger than they are and used once.
template <int N, bool PAST = false, typename T>
__device__ __forceinline__ auto load_elements(const T* row, int64_t c, int64_t n) {
  typedef T piece_t __attribute__((ext_vector_type(N), aligned(sizeof(T))));
  typedef std::conditional_t<N * sizeof(T) == 16, Bytes16, uint64_t> bytes_t;
  piece_t v = {};
  if (c < n) {
    const int64_t at = c + N <= n ? c : n - N;
    const piece_t* p = (const piece_t*)(row + at);
    v = PAST ? __builtin_nontemporal_load(p) : *p;
    if (at != c)
      v = __builtin_bit_cast(piece_t, last_first(__builtin_bit_cast(bytes_t, v), (int)(n - c) * 8 * (int)sizeof(T)));
  }
  return v;
}
// A piece of -0, which changes nothing that it is added to
template <typename T>
__device__ __forceinline__ vec_of<T> minus_zeros() {
  typedef unsigned words_t __attribute__((ext_vector_type(4)));
  const unsigned w = sizeof(T) == 4 ? 0x80000000u : 0x80008000u;
  return __builtin_bit_cast(vec_of<T>, words_t{w, w, w, w});
}
// Elements c .. c + EACH - 1 of a row of n, zero beyond it; n >= EACH, or 0
template <bool PAST = false, typename T>
__device__ __forceinline__ vec_of<T> load_piece(const T* row, int64_t c, int64_t n) {
  return __builtin_bit_cast(vec_of<T>, load_elements<EACH<T>, PAST>(row, c, n));
}
// The same for a row of any length
template <bool PAST = false, typename T>
__device__ __forceinline__ vec_of<T> load_short(const T* row, int64_t c, int64_t n) {
  if (n >= EACH<T>) return load_piece<PAST>(row, c, n);
  vec_of<T> v;
#pragma unroll
  for (int q = 0; q < EACH<T>; ++q) v[q] = c + q < n ? row[c + q] : (T)0.f;
  return v;
}

// The EACH values at x, each rounded once, to c .. of a row of n; what lies beyond it is not written.  The row's
// last piece goes out in halves: at most three stores for eight elements where one for each would be seven.
template <bool PAST = false, typename T>
__device__ __forceinline__ void store_piece(T* row, int64_t c, int64_t n, const float* x) {
  vec_of<T> v;
#pragma unroll
  for (int q = 0; q < EACH<T>; ++q) v[q] = (T)x[q];
  if (c + EACH<T> <= n) {
    vec_of<T>* p = (vec_of<T>*)(row + c);
    if (PAST)
      __builtin_nontemporal_store(v, p);
    else
      *p = v;
  } else if (c < n) {
    typedef uint64_t __attribute__((aligned(2), may_alias)) u64;
    typedef uint32_t __attribute__((aligned(2), may_alias)) u32;
    typedef uint16_t __attribute__((may_alias)) u16;
    Bytes16 w = __builtin_bit_cast(Bytes16, v);
    char* p = (char*)(row + c);
    const int left = (int)(n - c) * (int)sizeof(T);  // bytes
    if (left & 8) {
      *(u64*)p = w.lo;
      w.lo = w.hi;
      p += 8;
    }
    if (left & 4) {
      *(u32*)p = (uint32_t)w.lo;
      w.lo >>= 32;
      p += 4;
    }
    if (sizeof(T) == 2 && (left & 2)) *(u16*)p = (uint16_t)w.lo;
  }
}

// v of the lane whose number differs in the bits `o`; one instruction a word (__shfl_xor checks the number, too)
template <typename S>
__device__ __forceinline__ S of_lane_xor(S v, int o) {
  const int from = (int)(((threadIdx.x & 63) ^ (unsigned)o) << 2);
  if constexpr (sizeof(S) == 8) {
    const uint64_t w = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)(uint32_t)w);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)(uint32_t)(w >> 32));
    return __builtin_bit_cast(S, (uint64_t)hi << 32 | lo);
  } else {
    return __builtin_bit_cast(S, __builtin_amdgcn_ds_bpermute(from, __builtin_bit_cast(int, v)));
  }
}

// x_0^2 + ... + x_{E-1}^2 in 64 bits.  Formed in 32 bits where neither the sum leaves their range nor a term
// that matters falls below it (the sum is then off by at most E roundings of 2^-24 of it); else term by term in
// 64, on a branch that a wave takes only if a lane needs it (as a choice of two values it would always pay).
template <int E>
__device__ __forceinline__ double sum_squares(const float* x) {
  float s = x[0] * x[0];
#pragma unroll
  for (int q = 1; q < E; ++q) s = fmaf(x[q], x[q], s);
  const bool out = !(s >= 0x1p-96f && s <= 0x1p126f);
  double d = (double)s;
  if (__ballot(out)) {
    unsigned any = 0;
#pragma unroll
    for (int q = 0; q < E; ++q) any |= __builtin_bit_cast(unsigned, x[q]) << 1;
    if (__ballot(out && any != 0)) {
      double t = 0.;
#pragma unroll
      for (int q = 0; q < E; ++q) t = fma((double)x[q], (double)x[q], t);
      if (out) d = t;
    }
  }
  return d;
}

// The factor of a norm: 1 up to `most`, most / norm beyond it, NaN for a NaN
__device__ __forceinline__ float clip_factor(const float* norm, float most) {
  const float v = *norm;
  return v <= most ? 1.f : most / v;
}

}  // namespace
}  // namespace dash
