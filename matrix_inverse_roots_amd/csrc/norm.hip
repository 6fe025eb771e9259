// norm.hip -- the root-mean-square norm of a layer's input, written as the microscaled rows that
// dash_grad_stack_mx reads, and its gradient.
//
//   h = x + res,  rstd = (sum h^2 / n + eps)^{-1/2},  y = h rstd gain          (a row of n elements)
//   m = dy gain,  xhat = h rstd,  c = sum m xhat / n:
//   dx = dh + rstd (m - xhat c),  dgain = sum over rows of dy xhat
//
// Both are a few operations per element: the bytes in and out over the memory bandwidth is their time.  A row
// is read once and stays in the registers of the `lanes` threads that share it (K pieces of 16 bytes each)
// until its sum is known; longer rows are read twice.  Neighbouring threads take neighbouring pieces, so that a
// wave's access is one run and a group of 32 lies in neighbouring lanes.
#include <hip/hip_runtime.h>

#include "dash_internal.hpp"
#include "mx_format.hpp"
#include "vectors.hpp"

namespace dash {
namespace {

struct NormArgs {
  const void *x, *res, *gain;
  void *h, *y;
  uint8_t *codes, *scales;
  float* rstd;
  int64_t ldx, ldr, ldh, ldy;
  int64_t T, n, first_wg;
  double over_n, eps;
  dash_prec gain_type;
  int lanes, per;  // threads of a row (a power of two up to 64, or whole waves), and rows of a workgroup
  bool past;       // outputs past the caches (which hold no part of them until they are read)
};

// Elements c .. c + E - 1 of the gain (1 where there is none), zero beyond n; n >= E
template <int E>
__device__ __forceinline__ void load_gain(const void* gain, dash_prec type, int64_t c, int64_t n, float* g) {
  if (!gain) {
#pragma unroll
    for (int q = 0; q < E; ++q) g[q] = 1.f;
  } else if (type == DASH_FP32) {
#pragma unroll
    for (int p = 0; p < E / 4; ++p) {
      const vec_of<float> v = load_piece((const float*)gain, c + 4 * p, n);
#pragma unroll
      for (int q = 0; q < 4; ++q) g[4 * p + q] = v[q];
    }
  } else {
    const auto v = load_elements<E>((const uint16_t*)gain, c, n);
#pragma unroll
    for (int q = 0; q < E; ++q)
      g[q] = type == DASH_BF16 ? (float)__builtin_bit_cast(__bf16, (uint16_t)v[q])
                               : (float)__builtin_bit_cast(_Float16, (uint16_t)v[q]);
  }
}
__device__ __forceinline__ float gain_at(const void* gain, dash_prec type, int64_t c) {
  if (!gain) return 1.f;
  if (type == DASH_FP32) return ((const float*)gain)[c];
  return type == DASH_BF16 ? (float)((const __bf16*)gain)[c] : (float)((const _Float16*)gain)[c];
}

// The sum over the `lanes` threads of a row, the same bits in each.  Every thread of the workgroup calls it;
// `shared` holds a value per wave.
template <typename S>
__device__ __forceinline__ S row_sum(S v, int lanes, S* shared) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2)
    if (o < lanes) v += of_lane_xor(v, o);
  if (lanes > 64) {
    const int wave = threadIdx.x >> 6, waves = lanes >> 6;
    const int first = waves == (int)(blockDim.x >> 6) ? 0 : wave / waves * waves;
    __syncthreads();  // (the last row's values have been read)
    if ((threadIdx.x & 63) == 0) shared[wave] = v;
    __syncthreads();
    v = 0;
    for (int i = 0; i < waves; ++i) v += shared[first + i];
  }
  return v;
}

// rstd, and what its rounding lost times 2^24, so that the two hold 47 bits of it down to fp32's least normal number
struct Root {
  float rstd, rest;
  __device__ __forceinline__ Root(double square) {
    const double r = rsqrt(square);
    rstd = (float)r;
    rest = (float)(0x1p24 * (r - (double)rstd));
  }
  // y = h rstd g, off by at most four roundings (of h, of rstd and of two products)
  __device__ __forceinline__ float times(float h, float g) const { return h * rstd * g; }
  // The same as the fp32 number that rounds to the code that h rstd g itself rounds to: formed in 64 bits, cut off, and
  // made odd if anything was lost, so that it is on y's side of each border of codes and of scales (they end in 19
  // zeros).  y carries up to 2^-47 of itself (the sum of up to 32 squares a thread and its joins 2^-48.6, what is left
  // of rstd 2^-49, a few roundings): if it is within 64 steps of 2^-53 to 2^-52 of an fp32 number, it is that one, as
  // where the row's elements have one magnitude.  h: the sum before its rounding.
  __device__ __forceinline__ float odd_times(double h, float g) const {
    const double root = fma((double)rest, 0x1p-24, (double)rstd);
    uint64_t y = __builtin_bit_cast(uint64_t, h * root * (double)g);
    const unsigned low = (1u << 29) - 1, within = 64;  // (what fp32 does not hold)
    if ((((unsigned)y + within) & low) > 2 * within) y = (y & ~(uint64_t)low) | (low + 1);
    return (float)__builtin_bit_cast(double, y);
  }
};

// One piece of y as codes; the scale byte from the first lane of its group
template <int F, int E, bool PAST>
__device__ __forceinline__ void store_codes(const float* y, int64_t group0, int64_t c, uint8_t* codes, uint8_t* scales) {
  unsigned top = 0;
#pragma unroll
  for (int q = 0; q < E; ++q) top = umax(top, mag_bits(y[q]));
#pragma unroll
  for (int o = 1; o < GROUP / E; o *= 2) top = umax(top, of_lane_xor(top, o));
  const unsigned byte = scale_byte<F>(top);
  typedef typename Codes<F>::raw4 raw4;
  typedef raw4 raw_t __attribute__((ext_vector_type(E / 4)));
  raw_t raw;
#pragma unroll
  for (int p = 0; p < E / 4; ++p) raw[p] = Codes<F>::encode4(y + 4 * p, byte);
  raw_t* out = (raw_t*)(codes + (group0 * GROUP + c) * Codes<F>::BITS / 8);
  if (PAST)
    __builtin_nontemporal_store(raw, out);
  else
    *out = raw;
  if (c % GROUP == 0) scales[group0 + c / GROUP] = (uint8_t)byte;
}

// A piece of y made ready for its codes.  Four roundings move an element across a border only if its last 19 bits are
// next to zeros: once in a hundred waves, which form the piece again, one element after the other (the registers are
// few).  The sum x + res of fp32 elements is rounded as often as not; of 16-bit ones next to never.
template <typename T>
__device__ __forceinline__ void settle(const NormArgs& a, int64_t row, int64_t c, float* y, const float* h,
                                       const float* g, const Root& root) {
  constexpr int E = EACH<T>;
  constexpr unsigned NEAR = 4;
  const auto border = [](float v) { return (__builtin_bit_cast(unsigned, v) + NEAR) << 13; };
  unsigned least = ~0u;
#pragma unroll
  for (int q = 0; q < E; ++q) least = umin(least, border(y[q]));
  if (__builtin_expect(!__ballot(least <= 2 * NEAR << 13), 1)) return;
#pragma unroll
  for (int q = 0; q < E; ++q) {
    // (zeros, Inf and NaN are where they belong)
    const bool near = border(y[q]) <= 2 * NEAR << 13 && y[q] != 0.f && isfinite(y[q]);
    if (__builtin_expect(!__ballot(near), 1)) continue;
    float hq = h[q];
    asm volatile("" : "+v"(hq));
    double sum = hq;
    if (sizeof(T) == 4 && a.res && near && c + q < a.n) {
      asm volatile("" : "+v"(row));
      sum = (double)((const float*)a.x)[row * a.ldx + c + q] + (double)((const float*)a.res)[row * a.ldr + c + q];
    }
    const float odd = root.odd_times(sum, g[q]);
    if (near) y[q] = odd;
  }
}

// One piece of h = x + res; what its squares lack of those of the fp32 sums themselves, 2 sum h rest, is added to `more`
// (in 64 bits: its terms lie 2^-24 below squares that may be anywhere in their range)
template <typename T, int K>
__device__ __forceinline__ void add_up(const vec_of<T>& x, const vec_of<T>& res, bool sum, float* h, double* more) {
#pragma unroll
  for (int q = 0; q < EACH<T>; ++q) h[q] = sum ? (float)x[q] + (float)res[q] : (float)x[q];
  if (sizeof(T) == 2 || !sum) return;
#pragma unroll
  for (int q = 0; q < EACH<T>; ++q) {
    const double rest = ((double)(float)x[q] + (double)(float)res[q]) - (double)h[q];
    *more = fma(2. * (double)h[q], rest, *more);
  }
  if (K >= 4) asm volatile("" : "+v"(*more));  // (here, and not with x and res in registers until the gain is there)
}
template <int E>
__device__ __forceinline__ double squares64(const float* h) {
  double s = 0.;
#pragma unroll
  for (int q = 0; q < E; ++q) s = fma((double)h[q], (double)h[q], s);
  asm volatile("" : "+v"(s));  // (one piece at a time in 64 bits: the registers are few)
  return s;
}

// Rows side by side in a workgroup, each in the registers of its `lanes` threads from its only read on.  HBM bounds it:
// 8192 x 2048 bfloat16 with residual, y and codes 30.6 us (152 MB, 5.0 TB/s), 65536 x 4096 390 us (6.2 TB/s), 32768 x
// 8192 fp32 without y 599 us (5.8 TB/s).  Codes alone, where more instructions come to a byte: 65536 x 4096 bfloat16
// 208 us (3.9 TB/s).
template <typename T, int F, int K, bool PAST>
__global__ __launch_bounds__(1024) void rmsnorm_kernel(NormArgs a) {
  constexpr int E = EACH<T>;
  __shared__ double shared[16];
  const int slot = (int)(threadIdx.x / (unsigned)a.lanes), lane = (int)threadIdx.x - slot * a.lanes;
  const int64_t row = (a.first_wg + blockIdx.x) * a.per + slot;
  const bool live = row < a.T;  // (the others go along to the barriers)
  const int64_t groups = (a.n + GROUP - 1) / GROUP;
  const T* x = (const T*)a.x + row * a.ldx;
  const T* res = (const T*)a.res + row * a.ldr;
  float h[K][E], g[K][E];
  double more = 0.;
  {
    vec_of<T> vx[K], vr[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const unsigned c = (unsigned)E * (lane + k * a.lanes);
      vx[k] = load_piece(x, c, live ? a.n : 0);
      if (a.res) vr[k] = load_piece(res, c, live ? a.n : 0);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) add_up<T, K>(vx[k], vr[k], a.res != nullptr, h[k], &more);
  }
  double s = isfinite(more) ? more : 0.;  // (an h that is not finite makes the sum what it is)
#pragma unroll
  for (int k = 0; k < K; ++k) {  // (the gain on its way before the sums: 8192 x 2048 bfloat16 36 -> 32 us)
    load_gain<E>(a.gain, a.gain_type, (int64_t)E * (lane + k * a.lanes), a.n, g[k]);
    s += squares64<E>(h[k]);
  }
  s = row_sum(s, a.lanes, shared);
  if (!live) return;
  const Root root(fma(s, a.over_n, a.eps));
  if (a.rstd && lane == 0) a.rstd[row] = root.rstd;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const unsigned c = (unsigned)E * (lane + k * a.lanes);
    if (c >= groups * GROUP) break;  // (the lanes of a group together)
    float y[E];
#pragma unroll
    for (int q = 0; q < E; ++q) y[q] = root.times(h[k][q], g[k][q]);
    if (a.y) store_piece<PAST>((T*)a.y + row * a.ldy, c, a.n, y);
    if (a.codes) {
      settle<T>(a, row, c, y, h[k], g[k], root);
      store_codes<F, E, PAST>(y, row * groups, c, a.codes, a.scales);
    }
    if (a.h) store_piece<PAST>((T*)a.h + row * a.ldh, c, a.n, h[k]);  // (last: it may take the place of x or res)
  }
}

// Rows that the registers of a workgroup do not hold: x and res are read twice, the second time from the caches (2000
// x 40000 bfloat16 with residual, y and codes 172 us; 723 MB at the rate of a copy 153)
template <typename T, int F>
__global__ __launch_bounds__(1024) void rmsnorm_long_kernel(NormArgs a) {
  constexpr int E = EACH<T>;
  __shared__ double shared[16];
  const int64_t row = a.first_wg + blockIdx.x;
  const int64_t groups = (a.n + GROUP - 1) / GROUP;
  const T* x = (const T*)a.x + row * a.ldx;
  const T* res = (const T*)a.res + row * a.ldr;
  double s = 0.;
  for (int64_t c = (int64_t)E * threadIdx.x; c < a.n; c += E * 1024) {
    const vec_of<T> vx = load_piece(x, c, a.n);
    vec_of<T> vr;
    if (a.res) vr = load_piece(res, c, a.n);
    float h[E];
    double more = 0.;
    add_up<T, 1>(vx, vr, a.res != nullptr, h, &more);
    s += squares64<E>(h) + (isfinite(more) ? more : 0.);
  }
  s = row_sum(s, 1024, shared);
  const Root root(fma(s, a.over_n, a.eps));
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = root.rstd;
  for (int64_t c = (int64_t)E * threadIdx.x; c < groups * GROUP; c += E * 1024) {
    const vec_of<T> vx = load_piece(x, c, a.n);
    float h[E], g[E], y[E];
    load_gain<E>(a.gain, a.gain_type, c, a.n, g);
#pragma unroll
    for (int q = 0; q < E; ++q) h[q] = (float)vx[q];
    if (a.res) {
      const vec_of<T> vr = load_piece(res, c, a.n);
#pragma unroll
      for (int q = 0; q < E; ++q) h[q] += (float)vr[q];
    }
#pragma unroll
    for (int q = 0; q < E; ++q) y[q] = root.times(h[q], g[q]);
    if (a.y) store_piece((T*)a.y + row * a.ldy, c, a.n, y);
    if (a.codes) {
      settle<T>(a, row, c, y, h, g, root);
      store_codes<F, E, false>(y, row * groups, c, a.codes, a.scales);
    }
    if (a.h) store_piece((T*)a.h + row * a.ldh, c, a.n, h);
  }
}

// Rows of fewer than 8 elements, which no 16-byte piece fits: a thread each.  A wave's access is not one run, and a group
// of codes is mostly padding: 2^21 x 4 fp32 with residual, y and codes 65 us (212 MB at the rate of a copy 45).
constexpr int TINY = 8;
template <typename T, int F>
__global__ __launch_bounds__(256) void rmsnorm_tiny_kernel(NormArgs a) {
  const int64_t row = (a.first_wg + blockIdx.x) * 256 + threadIdx.x;
  if (row >= a.T) return;
  const int n = (int)a.n;
  double h[TINY];
  float y[GROUP];
  double s = 0.;
#pragma unroll
  for (int q = 0; q < TINY; ++q) {
    h[q] = q < n ? (double)(float)((const T*)a.x)[row * a.ldx + q] : 0.;
    if (a.res && q < n) h[q] += (double)(float)((const T*)a.res)[row * a.ldr + q];
    // (h is fp32's sum: of 16-bit elements as longer rows take it, and beyond fp32 an Inf)
    if (sizeof(T) == 2 || !isfinite((float)h[q])) h[q] = (double)(float)h[q];
    s = fma(h[q], h[q], s);
  }
  const Root root(fma(s, a.over_n, a.eps));
  if (a.rstd) a.rstd[row] = root.rstd;
  unsigned top = 0;
#pragma unroll
  for (int q = 0; q < GROUP; ++q) {
    y[q] = 0.f;
    if (q < TINY && q < n) {
      const float g = gain_at(a.gain, a.gain_type, q);
      const float rounded = (float)h[q], plain = root.times(rounded, g), odd = root.odd_times(h[q], g);
      y[q] = isfinite(plain) ? odd : plain;
      if (a.h) ((T*)a.h)[row * a.ldh + q] = (T)rounded;
      if (a.y) ((T*)a.y)[row * a.ldy + q] = (T)plain;
    }
    top = umax(top, mag_bits(y[q]));
  }
  if (!a.codes) return;
  const unsigned byte = scale_byte<F>(top);
  typedef typename Codes<F>::raw4 raw4;
#pragma unroll
  for (int p = 0; p < GROUP / 4; ++p) ((raw4*)a.codes)[row * (GROUP / 4) + p] = Codes<F>::encode4(y + 4 * p, byte);
  a.scales[row] = (uint8_t)byte;
}

// `grid` workgroups, in as many launches as they take
template <typename K, typename A>
hipError_t launch_rows(K kernel, int64_t grid, int block, A& a, hipStream_t stream) {
  const int64_t most = most_workgroups(block);
  for (a.first_wg = 0; a.first_wg < grid; a.first_wg += most) {
    const int64_t n = grid - a.first_wg < most ? grid - a.first_wg : most;
    hipLaunchKernelGGL(kernel, dim3((unsigned)n), dim3(block), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, int F, int K>
hipError_t rmsnorm_rows(NormArgs& a, hipStream_t stream) {
  return launch_rows(a.past ? rmsnorm_kernel<T, F, K, true> : rmsnorm_kernel<T, F, K, false>,
                     (a.T + a.per - 1) / a.per, a.per * a.lanes, a, stream);
}

// Threads for a row of `pieces`, k each: whole waves, or within one a power of two
int row_lanes(int64_t pieces, int k) {
  const int64_t need = (pieces + k - 1) / k;
  if (need > 64) return (int)((need + 63) / 64 * 64);
  int lanes = 1;
  while (lanes < need) lanes *= 2;
  return lanes;
}

// Pieces of a thread, where at most `threads` share a row.  One, so that many waves have loads under way (8192 x
// 2048 bfloat16 with 1 / 2 / 4: 30.7 / 36.0 / 37.3 us; its gradient 31.1 / 33.4); but two where the last
// one of a row is cut, which the wave that holds it pays for (one / two: 50001 x 263 binary16 34.3 / 30.7, gradient 34.4
// / 30.2; 12001 x 1001 bfloat16 23.3 / 21.4, 26.5 / 24.3; 12001 x 2047 40 / 39, 46 / 41; 50001 x 263 fp32 51 / 46, 56 /
// 44; 12001 x 3001 fp32 the same).
int row_pieces(int64_t pieces, bool whole, int threads, int least = 1) {
  int k = whole || least > 1 ? least : 2;
  while (pieces > (int64_t)threads * k) k *= 2;
  return k;
}

template <typename T, int F>
hipError_t rmsnorm(NormArgs& a, hipStream_t stream) {
  constexpr int E = EACH<T>;
  const int64_t pieces = (a.n + GROUP - 1) / GROUP * (GROUP / E);
  if (a.n < TINY) return launch_rows(rmsnorm_tiny_kernel<T, F>, (a.T + 255) / 256, 256, a, stream);
  if (pieces > 1024 * (32 / E)) return launch_rows(rmsnorm_long_kernel<T, F>, a.T, 1024, a, stream);
  // Threads of a row at most: 1024; fp32, with half as many elements each, sooner takes more of them (16384 x 4096 with
  // 512 / 1024 threads 198 / 206 us; codes alone of 4096 x 12288 with 384 / 768 80 / 58, 4096 x 16384 with 512 / 1024
  // 81 / 100).
  const int most = E == 8 || pieces > 6144 ? 1024 : pieces > 2048 ? 768 : 512;
  // Without a residual a piece is one load and not two, and needs more of them a thread: with codes alone 16 elements
  // (65536 x 4096 bfloat16 with 1 / 2 pieces 254 / 205 us, fp32 with 2 / 4 298 / 252), with y from 512 pieces on two
  // (287 / 249 us; 8192 x 2048 19.1 / 19.9).
  const int least = a.res ? 1 : !a.y && !a.h ? 16 / E : pieces >= 512 ? 2 : 1;
  const int k = row_pieces(pieces, a.n % E == 0, most, least);
  a.lanes = row_lanes(pieces, k);
  if (a.lanes < GROUP / E) a.lanes = GROUP / E;
  a.per = a.lanes < 256 ? 256 / a.lanes : 1;
  const int streams = 1 + (a.res != nullptr) + (a.h != nullptr) + (a.y != nullptr);
  a.past = a.T * a.n * (int64_t)sizeof(T) * streams > LARGE_BYTES;
  switch (k) {
    case 1: return rmsnorm_rows<T, F, 1>(a, stream);
    case 2: return rmsnorm_rows<T, F, 2>(a, stream);
    case 4: return rmsnorm_rows<T, F, 4>(a, stream);
  }
  if constexpr (E == 4) return rmsnorm_rows<T, F, 8>(a, stream);
  return hipErrorInvalidValue;
}

// ------------------------------------------------------------------------------------------------
// The gradient
// ------------------------------------------------------------------------------------------------

struct BackArgs {
  const void *dy, *h, *dh, *gain;
  const float* rstd;
  void* dx;
  float* dgain;
  float* part;  // [workgroups, n]: the sums that are joined into it
  int64_t lddy, ldh, lddh, lddx;
  int64_t T, n;
  float over_n;
  dash_prec gain_type;
  int lanes, per;  // threads of a row, and rows side by side
  bool accumulate, sums;  // sums: dgain is wanted
};

constexpr int BACK_BLOCK = 512;

// The compiler takes v for a new value here, so that it keeps the 16 bytes and not what it widened them to
template <typename V>
__device__ __forceinline__ V keep_packed(V v) {
  typedef unsigned words_t __attribute__((ext_vector_type(4)));
  words_t w = __builtin_bit_cast(words_t, v);
  asm volatile("" : "+v"(w));
  return __builtin_bit_cast(V, w);
}

// The largest power of two below x (0 for 1)
__host__ __device__ inline int half_of(int x) {
  int h = 1;
  while (2 * h < x) h *= 2;
  return x > 1 ? h : 0;
}

// One row of dx, and (SUMS) its part of the thread's column sums.  Every thread of the workgroup calls it; rows
// behind the last are zeros.
template <typename T, int K, bool SUMS, bool PAST>
__device__ __forceinline__ void back_row(const BackArgs& a, int64_t row, int lane, const float (&g)[K][EACH<T>],
                                         float (&dg)[K][EACH<T>], float* shared) {
  constexpr int E = EACH<T>;
  const int64_t n = row < a.T ? a.n : 0;
  vec_of<T> dy[K], h[K], dh[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t c = (int64_t)E * (lane + k * a.lanes);
    dy[k] = load_piece<PAST>((const T*)a.dy + row * a.lddy, c, n);
    h[k] = load_piece<PAST>((const T*)a.h + row * a.ldh, c, n);
    dh[k] = minus_zeros<T>();
    if (a.dh) dh[k] = load_piece<PAST>((const T*)a.dh + row * a.lddh, c, n);
  }
  const float rstd = row < a.T ? a.rstd[row] : 0.f;
  float dot = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int q = 0; q < E; ++q) {
      const float d = (float)dy[k][q], xhat = (float)h[k][q] * rstd;
      if (SUMS) dg[k][q] = fmaf(d, xhat, dg[k][q]);
      dot = fmaf(d * g[k][q], xhat, dot);
    }
  const float mean = row_sum(dot, a.lanes, shared) * a.over_n;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t c = (int64_t)E * (lane + k * a.lanes);
    if (c >= n) break;
    dy[k] = keep_packed(dy[k]);  // (kept as they were loaded until here, and widened again)
    h[k] = keep_packed(h[k]);
    float dx[E];
#pragma unroll
    for (int q = 0; q < E; ++q) {
      const float xhat = (float)h[k][q] * rstd;
      dx[q] = fmaf(rstd, fmaf(-xhat, mean, (float)dy[k][q] * g[k][q]), (float)dh[k][q]);
    }
    store_piece<PAST>((T*)a.dx + row * a.lddx, c, n, dx);
  }
}

// `per` rows side by side, then the next ones a grid further (the workgroups together read one run of rows:
// 32768 x 8192 bfloat16 417 -> 395 us over a run of rows for each).  Every thread keeps the sums dy xhat of
// its columns in registers, and the workgroup stores one row of them at the end: equal calls add in the same
// order.  HBM bounds it: that case now takes 375 us (2.15 GB, 5.7 TB/s); 50001 x 263 fp32, whose rows start on 4
// bytes, 50 us (211 MB, 4.2 TB/s).
template <typename T, int K, bool PAST>
__global__ __launch_bounds__(BACK_BLOCK) void rmsnorm_back_kernel(BackArgs a) {
  constexpr int E = EACH<T>;
  extern __shared__ __attribute__((aligned(16))) float columns[];
  __shared__ float shared[BACK_BLOCK / 64];
  const int per = a.per, slot = (int)(threadIdx.x / (unsigned)a.lanes), lane = (int)threadIdx.x - slot * a.lanes;
  float g[K][E], dg[K][E];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    load_gain<E>(a.gain, a.gain_type, (int64_t)E * (lane + k * a.lanes), a.n, g[k]);
#pragma unroll
    for (int q = 0; q < E; ++q) dg[k][q] = 0.f;
  }
  for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < a.T; r0 += (int64_t)gridDim.x * per)
    back_row<T, K, true, PAST>(a, r0 + slot, lane, g, dg, shared);
  if (!a.sums) return;
  // the rows side by side, halving (slot by slot 64 of them took 10 us)
  for (int half = half_of(per); half; half /= 2) {
    __syncthreads();
    float* with = columns + (slot & (half - 1)) * (K * E) * a.lanes + lane;
    if (slot >= half && slot < 2 * half)
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int q = 0; q < E; ++q) with[(k * E + q) * a.lanes] = dg[k][q];
    __syncthreads();
    if (slot < half && slot + half < per)
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int q = 0; q < E; ++q) dg[k][q] += with[(k * E + q) * a.lanes];
  }
  if (slot) return;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t c = (int64_t)E * (lane + k * a.lanes);
#pragma unroll
    for (int p = 0; p < E / 4; ++p) store_piece(a.part + blockIdx.x * a.n, c + 4 * p, a.n, dg[k] + 4 * p);
  }
}

// Few rows, dy not replaced: the first row_wgs workgroups take `per` rows each, and the others 16 pieces of columns
// each, whose sums they form from dy and h themselves (the caches hold them): no second launch.  The launch and one
// row's latency bound it: 16 x 2048 bfloat16 4.0 us, 9.4 with the call around it (13.4 with a launch for the join).
template <typename T, int K>
__global__ __launch_bounds__(BACK_BLOCK) void rmsnorm_back_few_kernel(BackArgs a, int row_wgs) {
  constexpr int E = EACH<T>, WIDE = 16, SHARES = BACK_BLOCK / WIDE;
  __shared__ float shared[2 * (BACK_BLOCK / 64)];  // (of a row that the workgroup's last waves would begin, too)
  __shared__ float sums[SHARES][WIDE * E + 1];
  if ((int)blockIdx.x < row_wgs) {
    const int slot = (int)(threadIdx.x / (unsigned)a.lanes), lane = (int)threadIdx.x - slot * a.lanes;
    float g[K][E];
#pragma unroll
    for (int k = 0; k < K; ++k) load_gain<E>(a.gain, a.gain_type, (int64_t)E * (lane + k * a.lanes), a.n, g[k]);
    // (threads behind the workgroup's last row go along to the barriers with a row of zeros)
    const int64_t row = slot < a.per ? (int64_t)blockIdx.x * a.per + slot : a.T;
    back_row<T, K, false, false>(a, row, lane, g, g, shared);
    return;
  }
  const int piece = threadIdx.x % WIDE, share = threadIdx.x / WIDE;
  const int64_t c0 = (int64_t)((int)blockIdx.x - row_wgs) * (WIDE * E), c = c0 + piece * E;
  float s[E];
#pragma unroll
  for (int q = 0; q < E; ++q) s[q] = 0.f;
#pragma unroll 4
  for (int64_t row = share; row < a.T; row += SHARES) {
    const vec_of<T> dy = load_piece((const T*)a.dy + row * a.lddy, c, a.n);
    const vec_of<T> h = load_piece((const T*)a.h + row * a.ldh, c, a.n);
    const float rstd = a.rstd[row];
#pragma unroll
    for (int q = 0; q < E; ++q) s[q] = fmaf((float)dy[q], (float)h[q] * rstd, s[q]);
  }
#pragma unroll
  for (int q = 0; q < E; ++q) sums[share][piece * E + q] = s[q];
  __syncthreads();
  const int64_t out = c0 + threadIdx.x;
  if (threadIdx.x >= WIDE * E || out >= a.n) return;
  double all = a.accumulate ? (double)a.dgain[out] : 0.;
#pragma unroll
  for (int i = 0; i < SHARES; ++i) all += (double)sums[i][threadIdx.x];
  a.dgain[out] = (float)all;
}

// Rows that the registers of a workgroup do not hold: each is read twice, its mean summed in 64 bits from pieces on (a
// thread may have thousands of them), and the column sums stay in the workgroup's row of `part`, which is read and
// written for every row (2000 x 40000 bfloat16 267 us; 640 MB at the rate of a copy 135)
template <typename T>
__global__ __launch_bounds__(1024) void rmsnorm_back_long_kernel(BackArgs a) {
  constexpr int E = EACH<T>;
  __shared__ double shared[16];
  float* part = a.part + blockIdx.x * a.n;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const T* dy = (const T*)a.dy + row * a.lddy;
    const T* h = (const T*)a.h + row * a.ldh;
    const float rstd = a.rstd[row];
    double dot = 0.;
    for (int64_t c = (int64_t)E * threadIdx.x; c < a.n; c += E * 1024) {
      const vec_of<T> vd = load_piece(dy, c, a.n), vh = load_piece(h, c, a.n);
      float g[E], sum = 0.f;
      load_gain<E>(a.gain, a.gain_type, c, a.n, g);
#pragma unroll
      for (int q = 0; q < E; ++q) sum = fmaf((float)vd[q] * g[q], (float)vh[q] * rstd, sum);
      dot += (double)sum;
    }
    const float mean = (float)(row_sum(dot, 1024, shared) * (double)a.over_n);
    for (int64_t c = (int64_t)E * threadIdx.x; c < a.n; c += E * 1024) {
      const vec_of<T> vd = load_piece(dy, c, a.n), vh = load_piece(h, c, a.n);
      float g[E], dx[E];
      load_gain<E>(a.gain, a.gain_type, c, a.n, g);
#pragma unroll
      for (int q = 0; q < E; ++q) dx[q] = rstd * fmaf(-((float)vh[q] * rstd), mean, (float)vd[q] * g[q]);
      if (a.dh) {
        const vec_of<T> vr = load_piece((const T*)a.dh + row * a.lddh, c, a.n);
#pragma unroll
        for (int q = 0; q < E; ++q) dx[q] += (float)vr[q];
      }
      store_piece((T*)a.dx + row * a.lddx, c, a.n, dx);
      if (a.sums) {
#pragma unroll
        for (int p = 0; p < E / 4; ++p) {
          float v[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = (float)vd[4 * p + q] * ((float)vh[4 * p + q] * rstd);
          if (row > blockIdx.x) {
            const vec_of<float> old = load_piece(part, c + 4 * p, a.n);
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] += old[q];
          }
          store_piece(part, c + 4 * p, a.n, v);
        }
      }
    }
  }
}

// Rows of fewer than 8 elements: a thread each, whose sums a workgroup joins in order (2^21 x 4 fp32 63 us; 143 MB at
// the rate of a copy 30)
template <typename T>
__global__ __launch_bounds__(256) void rmsnorm_back_tiny_kernel(BackArgs a) {
  __shared__ float sums[TINY][256];
  const int n = (int)a.n;
  float dg[TINY];
#pragma unroll
  for (int q = 0; q < TINY; ++q) dg[q] = 0.f;
  for (int64_t row = blockIdx.x * 256 + threadIdx.x; row < a.T; row += gridDim.x * 256) {
    const float rstd = a.rstd[row];
    float m[TINY], xhat[TINY], dot = 0.f;
#pragma unroll
    for (int q = 0; q < TINY; ++q) {
      const float d = q < n ? (float)((const T*)a.dy)[row * a.lddy + q] : 0.f;
      xhat[q] = q < n ? (float)((const T*)a.h)[row * a.ldh + q] * rstd : 0.f;
      m[q] = q < n ? d * gain_at(a.gain, a.gain_type, q) : 0.f;
      dg[q] = fmaf(d, xhat[q], dg[q]);
      dot = fmaf(m[q], xhat[q], dot);
    }
    const float mean = dot * a.over_n;
#pragma unroll
    for (int q = 0; q < TINY; ++q) {
      if (q >= n) break;
      float dx = rstd * fmaf(-xhat[q], mean, m[q]);
      if (a.dh) dx += (float)((const T*)a.dh)[row * a.lddh + q];
      ((T*)a.dx)[row * a.lddx + q] = (T)dx;
    }
  }
  if (!a.sums) return;
#pragma unroll
  for (int q = 0; q < TINY; ++q) sums[q][threadIdx.x] = dg[q];
  __syncthreads();
  if ((int)threadIdx.x >= n) return;
  double s = 0.;
  for (int i = 0; i < 256; ++i) s += (double)sums[threadIdx.x][i];
  a.part[blockIdx.x * a.n + threadIdx.x] = (float)s;
}

// dgain (+)= the sum of the workgroups' rows: 32 columns x 32 threads with a share of the rows each, which are
// joined across a wave (512 rows of 263 4.4 us, 256 rows of 8192 4.8: latency).
__global__ __launch_bounds__(1024) void rmsnorm_join_kernel(const float* part, int parts, int64_t n, float* dgain,
                                                            bool accumulate) {
  __shared__ double sums[32][33];
  const int col = threadIdx.x & 31, share = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + col;
  double s = 0.;
  if (c < n)
#pragma unroll 16
    for (int p = share; p < parts; p += 32) s += (double)part[p * n + c];
  sums[share][col] = s;
  __syncthreads();
  s = sums[col][share];
#pragma unroll
  for (int o = 1; o < 32; o *= 2) s += __shfl_xor(s, o, 64);
  const int64_t out = (int64_t)blockIdx.x * 32 + share;
  if (col == 0 && out < n) dgain[out] = (float)(accumulate ? s + (double)dgain[out] : s);
}

// How the rows are shared out, over at most MOST_PARTS workgroups
constexpr int64_t MOST_PARTS = 512;
struct BackPlan {
  int k, lanes, per;  // pieces of a thread (0: the kernels of long and of tiny rows), threads of a row, rows abreast
  int64_t wgs;
  bool few = false;  // rmsnorm_back_few_kernel
};
// Rows whose gradient is one launch, though their columns' workgroups read dy and h once more: 16 x 2048 bfloat16 3.0
// us (in two launches 5.9), 512 x 64 4.8 (6.7), 512 x 2048 5.7 (9.2), 512 x 16384 16.5 (22.1), in fp32 31.8 (30.2).
constexpr int64_t FEW_ROWS = 512;
BackPlan back_plan(int64_t T, int64_t n, int E) {
  BackPlan p;
  const int64_t pieces = (n + E - 1) / E;
  if (n < TINY || pieces > (int64_t)BACK_BLOCK * (32 / E)) {
    p.k = p.lanes = 0;
    p.per = n < TINY ? 256 : 1;
  } else {
    // (16-bit rows that end inside a piece: up to four pieces a thread, 12001 x 8001 198 -> 188 us, whole ones of
    // 8192 are 2 % the other way)
    const bool whole = n % E == 0;
    p.k = row_pieces(pieces, whole, E == 8 && !whole ? 256 : BACK_BLOCK);
    if (p.k > 32 / E) p.k = 32 / E;
    p.lanes = row_lanes(pieces, p.k);
    p.per = BACK_BLOCK / p.lanes;
  }
  // With four pieces a thread one workgroup fills a compute unit's registers (fp32 16384 x 6144 with 256 / 512 of
  // them 288 / 299 us, 12001 x 8001 289 / 297); with fewer, two (50001 x 263 bfloat16 with 256 / 512 49 / 38).
  const int64_t most = p.k >= 4 ? MOST_PARTS / 2 : MOST_PARTS;
  p.wgs = (T + p.per - 1) / p.per;
  if (p.wgs > most) p.wgs = most;
  return p;
}

template <typename T, int K>
hipError_t back_rows(const BackArgs& a, const BackPlan& p, hipStream_t stream) {
  if (p.few) {
    const int64_t wide = 16 * EACH<T>;
    hipLaunchKernelGGL((rmsnorm_back_few_kernel<T, K>), dim3((unsigned)(p.wgs + (a.n + wide - 1) / wide)),
                       dim3(BACK_BLOCK), 0, stream, a, (int)p.wgs);
  } else {
    const size_t lds = a.sums ? (size_t)half_of(p.per) * p.lanes * K * EACH<T> * sizeof(float) : 0;
    const bool past = a.T * a.n * (int64_t)sizeof(T) * (a.dh ? 4 : 3) > LARGE_BYTES;
    hipLaunchKernelGGL((past ? rmsnorm_back_kernel<T, K, true> : rmsnorm_back_kernel<T, K, false>),
                       dim3((unsigned)p.wgs), dim3(p.per * p.lanes), lds, stream, a);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t back(BackArgs& a, void* ws, hipStream_t stream) {
  BackPlan p = back_plan(a.T, a.n, EACH<T>);
  p.few = p.k && a.sums && a.T <= FEW_ROWS && a.dx != a.dy;
  if (p.few) p.wgs = (a.T + p.per - 1) / p.per;
  a.lanes = p.lanes;
  a.per = p.per;
  a.part = (float*)ws;
  hipError_t e = hipErrorInvalidValue;
  if (p.k == 0) {
    if (a.n < TINY)
      hipLaunchKernelGGL(rmsnorm_back_tiny_kernel<T>, dim3((unsigned)p.wgs), dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL(rmsnorm_back_long_kernel<T>, dim3((unsigned)p.wgs), dim3(1024), 0, stream, a);
    e = hipGetLastError();
  } else if (p.k == 1) {
    e = back_rows<T, 1>(a, p, stream);
  } else if (p.k == 2) {
    e = back_rows<T, 2>(a, p, stream);
  } else if (p.k == 4) {
    e = back_rows<T, 4>(a, p, stream);
  } else {
    if constexpr (EACH<T> == 4) e = back_rows<T, 8>(a, p, stream);
  }
  if (e != hipSuccess || !a.sums || p.few) return e;
  hipLaunchKernelGGL(rmsnorm_join_kernel, dim3((unsigned)((a.n + 31) / 32)), dim3(1024), 0, stream, a.part, (int)p.wgs,
                     a.n, a.dgain, a.accumulate);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm(const RmsNorm& p, dash_prec type, dash_mx_fmt fmt, hipStream_t stream) {
  NormArgs a{p.x.p, p.res.p, p.gain, p.h.p, p.y.p, p.codes, p.scales, p.rstd, p.x.ld, p.res.ld, p.h.ld, p.y.ld,
             p.T, p.n, 0, 1.0 / (double)p.n, (double)p.eps, p.gain_type, 0, 0, false};
  const bool e4 = fmt == DASH_MX_E4M3;
  if (type == DASH_FP32) return e4 ? rmsnorm<float, DASH_MX_E4M3>(a, stream) : rmsnorm<float, DASH_MX_E2M1>(a, stream);
  if (type == DASH_BF16) return e4 ? rmsnorm<__bf16, DASH_MX_E4M3>(a, stream) : rmsnorm<__bf16, DASH_MX_E2M1>(a, stream);
  return e4 ? rmsnorm<_Float16, DASH_MX_E4M3>(a, stream) : rmsnorm<_Float16, DASH_MX_E2M1>(a, stream);
}

// a row of partial sums for every workgroup that any smaller T may have
size_t rmsnorm_back_workspace_bytes(int64_t T, int64_t n) {
  return (size_t)(T < MOST_PARTS ? T : MOST_PARTS) * (size_t)n * sizeof(float);
}

hipError_t launch_rmsnorm_back(const RmsNormBack& p, dash_prec type, void* ws, hipStream_t stream) {
  BackArgs a{p.dy.p, p.h.p, p.dh.p, p.gain, p.rstd, p.dx.p, p.dgain, nullptr, p.dy.ld, p.h.ld, p.dh.ld, p.dx.ld,
             p.T, p.n, 1.f / (float)p.n, p.gain_type, 0, 0, p.accumulate, p.dgain != nullptr};
  if (type == DASH_FP32) return back<float>(a, ws, stream);
  if (type == DASH_BF16) return back<__bf16>(a, ws, stream);
  return back<_Float16>(a, ws, stream);
}

}  // namespace dash
