// mx.hip -- microscaled storage: quantisation by rows and by columns, and back.
//
// A row of a microscaled matrix is cut into groups of 32 consecutive elements that share a power of
// two 2^e, stored as one byte e + 127; an element is an E2M1 value (1 sign, 2 exponent, 1 mantissa
// bit: 0, .5, 1, 1.5, 2, 3, 4, 6) or an E4M3 value (largest 448).  e is the least integer with
// max|x| <= m 2^e, m the largest element value (6 = 1.5 2^2 or 448 = 1.75 2^8), so nothing
// saturates: with max|x| = 1.f 2^E it is E - 2 or E - 8, plus one when 1.f exceeds 1.5 or 1.75; below
// -127 it is -127.  x 2^-e is exact (or rounds to a zero code anyway) and the conversion instruction
// rounds it to the element grid once, to nearest, ties to even.  A group that holds an Inf or a NaN
// gets byte 255 and zero codes, which reads back as NaN throughout.
//
// Both directions stream: bytes in plus bytes out over the memory bandwidth is their time.
#include <hip/hip_runtime.h>

#include "dash_internal.hpp"
#include "mx_format.hpp"

namespace dash {
namespace {

template <typename T>
using v8 = T __attribute__((ext_vector_type(8), aligned(16)));

// Elements c0 .. c0 + 7 of a row of `cols` (zero beyond it), widened to fp32.  vec: the row's start and
// pitch are 16-byte aligned.
template <typename T>
__device__ __forceinline__ f32x8 load8(const T* row, int64_t c0, int64_t cols, bool vec) {
  f32x8 x;
  if (vec && c0 + 8 <= cols) {
    const v8<T> r = *(const v8<T>*)(row + c0);
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = (float)r[q];
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = c0 + q < cols ? (float)row[c0 + q] : 0.f;
  }
  return x;
}

struct QuantArgs {
  const void* src;
  int64_t N, rows, cols, ld;
  uint8_t *codes, *scales, *codes_t, *scales_t;
  float* diag;
  bool vec;
  int lanes;         // rows kernel: threads of a workgroup on one row (a power of two, 4 .. 256)
  int64_t col_wgs;   // and workgroups along a row
  int64_t first_wg;  // of this launch
};

// Quantises the thread's 8 values of a group held by 4 neighbouring lanes; the scale byte in every one.
template <int F>
__device__ __forceinline__ typename Codes<F>::type encode_group(const f32x8& x, unsigned& byte) {
  unsigned top = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) top = umax(top, mag_bits(x[q]));
  top = umax(top, __shfl_xor(top, 1, 64));
  top = umax(top, __shfl_xor(top, 2, 64));
  byte = scale_byte<F>(top);
  return Codes<F>::encode(x, byte);
}

// The diagonal element of a square matrix's row r among columns c0 .. c0 + 7 goes to diag, and 0 into
// its place.
__device__ __forceinline__ void take_diag(f32x8& x, int64_t r, int64_t c0, float* out) {
#pragma unroll
  for (int q = 0; q < 8; ++q)
    if (c0 + q == r) {
      *out = x[q];
      x[q] = 0.f;
    }
}

// Rows a thread takes a piece of, their loads under way together: 2 from 16-bit sources (65536 x 4096
// bfloat16 to E4M3 166 -> 151 us) and 1 from fp32 (192 x 1024 x 1024 to E2M1 160 us; 2: 163); on the way
// back 2 (65536 x 4096 to bfloat16 with 1 / 2 / 4 154 / 130 / 139 us, 192 x 1024 x 1024 E4M3 to fp32
// 219 / 162 / 170).
template <typename T>
constexpr int ROWS_IN = sizeof(T) == 2 ? 2 : 1;
constexpr int ROWS_BACK = 2;

// Rows only: 4 threads per group; rows of all matrices are one list.
template <typename T, int F>
__global__ __launch_bounds__(256) void mx_rows_kernel(QuantArgs a) {
  const int64_t wg = a.first_wg + blockIdx.x, rb = wg / a.col_wgs, cb = wg - rb * a.col_wgs;
  const int per = 256 / a.lanes;
  const int64_t first = rb * per * ROWS_IN<T> + threadIdx.x / a.lanes;
  const int64_t c0 = 8 * (cb * a.lanes + threadIdx.x % a.lanes);
  const int64_t groups = (a.cols + GROUP - 1) / GROUP;
  if (c0 >= groups * GROUP) return;  // (the 4 lanes of a group leave together)
  f32x8 x[ROWS_IN<T>];
#pragma unroll
  for (int i = 0; i < ROWS_IN<T>; ++i) {
    const int64_t r = first + i * per;
    x[i] = r < a.N * a.rows ? load8((const T*)a.src + r * a.ld, c0, a.cols, a.vec) : f32x8{};
  }
#pragma unroll
  for (int i = 0; i < ROWS_IN<T>; ++i) {
    const int64_t r = first + i * per;
    if (r >= a.N * a.rows) return;  // (as above)
    if (a.diag) take_diag(x[i], r % a.rows, c0, a.diag + r);
    unsigned byte;
    const typename Codes<F>::type c = encode_group<F>(x[i], byte);
    *(typename Codes<F>::type*)(a.codes + (r * groups * GROUP + c0) * Codes<F>::BITS / 8) = c;
    if (threadIdx.x % 4 == 0) a.scales[r * groups + c0 / GROUP] = (uint8_t)byte;
  }
}

// Columns, and rows from the same read: a QT x QT tile goes through LDS.  QT / 32 neighbouring lanes take
// the 32-row groups of one column, so that with QT = 128 a wave writes 16 columns' 128 (64) contiguous
// bytes; a row's columns are xored with 16 (row / 32), which puts the groups on different banks.
template <typename T, int F, bool ROWS, int QT>
__global__ __launch_bounds__(256) void mx_cols_kernel(QuantArgs a) {
  constexpr int CHUNKS = QT / 8, STEP = 256 / CHUNKS, EACH = QT / STEP;  // 8-column pieces per row; a thread's rows
  constexpr int GROUPS = QT / GROUP;
  __shared__ __attribute__((aligned(16))) float tile[QT * QT];
  const int64_t tr = (a.rows + QT - 1) / QT, tc = (a.cols + QT - 1) / QT;
  const int64_t wg = a.first_wg + blockIdx.x, n = wg / (tr * tc), t = wg - n * (tr * tc);
  const int64_t r0 = t / tc * QT, c0 = t % tc * QT;
  const T* src = (const T*)a.src + n * a.rows * a.ld;
  const int64_t gc = (a.cols + GROUP - 1) / GROUP, gr = (a.rows + GROUP - 1) / GROUP;
  f32x8 x[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int64_t r = r0 + threadIdx.x / CHUNKS + STEP * i, c = c0 + 8 * (threadIdx.x % CHUNKS);
    x[i] = r < a.rows ? load8(src + r * a.ld, c, a.cols, a.vec) : f32x8{};
  }
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int lr = threadIdx.x / CHUNKS + STEP * i, lc = 8 * (threadIdx.x % CHUNKS);
    const int64_t r = r0 + lr, c = c0 + lc;
    if (a.diag && r < a.rows) take_diag(x[i], r, c, a.diag + n * a.rows + r);
    *(f32x8*)&tile[lr * QT + (lc ^ (16 * (lr >> 5)))] = x[i];
    if (ROWS) {
      unsigned byte;
      const typename Codes<F>::type code = encode_group<F>(x[i], byte);
      if (r < a.rows && c < gc * GROUP) {
        *(typename Codes<F>::type*)(a.codes + ((n * a.rows + r) * gc * GROUP + c) * Codes<F>::BITS / 8) = code;
        if (threadIdx.x % 4 == 0) a.scales[(n * a.rows + r) * gc + c / GROUP] = (uint8_t)byte;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int task = threadIdx.x; task < QT * GROUPS; task += 256) {
    const int g = task % GROUPS, lc = task / GROUPS;
    const int64_t c = c0 + lc, r = r0 + GROUP * g;
    if (c >= a.cols || r >= a.rows) continue;
    f32x8 y[4];
    unsigned top = 0;
#pragma unroll
    for (int k = 0; k < GROUP; ++k) {
      const float v = tile[(GROUP * g + k) * QT + (lc ^ (16 * g))];
      y[k >> 3][k & 7] = v;
      top = umax(top, mag_bits(v));
    }
    const unsigned byte = scale_byte<F>(top);
    uint8_t* out = a.codes_t + ((n * a.cols + c) * gr * GROUP + r) * Codes<F>::BITS / 8;
    typename Codes<F>::type code[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) code[k] = Codes<F>::encode(y[k], byte);
    if constexpr (F == DASH_MX_E4M3) {
      *(u32x4*)out = u32x4{code[0][0], code[0][1], code[1][0], code[1][1]};
      *(u32x4*)(out + 16) = u32x4{code[2][0], code[2][1], code[3][0], code[3][1]};
    } else {
      *(u32x4*)out = u32x4{code[0], code[1], code[2], code[3]};
    }
    a.scales_t[(n * a.cols + c) * gr + r / GROUP] = (uint8_t)byte;
  }
}

struct DequantArgs {
  const uint8_t *codes, *scales;
  const float* diag;
  int64_t N, rows, cols, ld;
  void* dst;
  bool vec;
  int lanes;
  int64_t col_wgs, first_wg;
};

// The values: element times 2^e in fp32 (ldexp is exact down to fp32's subnormals), the diagonal's own
// value in its place, rounded to the output type once.  A thread makes 16 bytes of output per row, so
// that a wave's store is one run of whole lines.
template <typename T, int F>
__global__ __launch_bounds__(256) void mx_values_kernel(DequantArgs a) {
  constexpr int EACH = 16 / sizeof(T), QUADS = EACH / 4;
  typedef typename Codes<F>::raw4 raw4;
  typedef T out_t __attribute__((ext_vector_type(EACH)));
  struct alignas(sizeof(raw4) * QUADS) Raw {
    raw4 q[QUADS];
  };
  const int64_t wg = a.first_wg + blockIdx.x, rb = wg / a.col_wgs, cb = wg - rb * a.col_wgs;
  const int per = 256 / a.lanes;
  const int64_t first = rb * per * ROWS_BACK + threadIdx.x / a.lanes;
  const int64_t c0 = EACH * (cb * a.lanes + threadIdx.x % a.lanes);
  if (c0 >= a.cols) return;
  const int64_t groups = (a.cols + GROUP - 1) / GROUP;
  Raw c[ROWS_BACK];
  int byte[ROWS_BACK];
#pragma unroll
  for (int i = 0; i < ROWS_BACK; ++i) {
    const int64_t r = first + i * per;
    c[i] = Raw{};
    byte[i] = 0;
    if (r < a.N * a.rows) {
      c[i] = *(const Raw*)(a.codes + (r * groups * GROUP + c0) * Codes<F>::BITS / 8);
      byte[i] = a.scales[r * groups + c0 / GROUP];
    }
  }
#pragma unroll
  for (int i = 0; i < ROWS_BACK; ++i) {
    const int64_t r = first + i * per;
    if (r >= a.N * a.rows) return;
    float x[EACH];
#pragma unroll
    for (int w = 0; w < QUADS; ++w) {
      const f32x4 v = Codes<F>::decode(c[i].q[w]);
#pragma unroll
      for (int q = 0; q < 4; ++q) x[4 * w + q] = byte[i] == 255 ? __builtin_nanf("") : ldexpf(v[q], byte[i] - 127);
    }
    if (a.diag) {
      const int64_t d = r % a.rows;
#pragma unroll
      for (int q = 0; q < EACH; ++q)
        if (c0 + q == d) x[q] += a.diag[r];
    }
    T* out = (T*)a.dst + r * a.ld + c0;
    if (a.vec && c0 + EACH <= a.cols) {
      out_t v;
#pragma unroll
      for (int q = 0; q < EACH; ++q) v[q] = (T)x[q];
      *(out_t*)out = v;
    } else {
#pragma unroll
      for (int q = 0; q < EACH; ++q)
        if (c0 + q < a.cols) out[q] = (T)x[q];
    }
  }
}

// Threads of a 256-thread workgroup on one row of `chunks` pieces, and workgroups along it
void row_split(int64_t chunks, int& lanes, int64_t& col_wgs) {
  lanes = 4;
  while (lanes < 256 && lanes < chunks) lanes *= 2;
  col_wgs = (chunks + lanes - 1) / lanes;
}

// `grid` workgroups of 256 threads, in as many launches as they take (one, below 2^24)
template <typename K, typename A>
hipError_t launch_all(K kernel, int64_t grid, A& a, hipStream_t stream) {
  const int64_t most = most_workgroups(256);
  for (a.first_wg = 0; a.first_wg < grid; a.first_wg += most) {
    const int64_t n = grid - a.first_wg < most ? grid - a.first_wg : most;
    hipLaunchKernelGGL(kernel, dim3((unsigned)n), dim3(256), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename K>
hipError_t launch_cols(K kernel, int64_t side, QuantArgs& a, hipStream_t stream) {
  return launch_all(kernel, a.N * ((a.rows + side - 1) / side) * ((a.cols + side - 1) / side), a, stream);
}

template <typename T, int F>
hipError_t quantize(QuantArgs& a, hipStream_t stream) {
  if (a.codes_t) {
    // 64-wide tiles, but 128-wide ones (whole lines written per column) for large stacks of fp32 that fill
    // them.  Both measured, rows and columns to E4M3, calls back to back (us, 64 / 128): 1777 x 1001 fp16 7.3 /
    // 11.5; fp32 60 x 320 x 320 7.8 / 12.6, 48 x 1024 x 1024 58 / 62, 96 x 1024 x 1024 129 / 114, 192 x 1024 x
    // 1024 270 / 218, 4000 x 192 x 192 174 / 255, 20000 x 6437 315 / 284; 16384 x 16384 bfloat16 325 / 373.
    if constexpr (sizeof(T) == 4) {
      const int64_t tiles = a.N * ((a.rows + 127) / 128) * ((a.cols + 127) / 128);
      if (tiles >= 4096 && (double)tiles * (128 * 128) <= 1.1 * (double)a.N * (double)a.rows * (double)a.cols)
        return a.codes ? launch_cols(mx_cols_kernel<T, F, true, 128>, 128, a, stream)
                       : launch_cols(mx_cols_kernel<T, F, false, 128>, 128, a, stream);
    }
    return a.codes ? launch_cols(mx_cols_kernel<T, F, true, 64>, 64, a, stream)
                   : launch_cols(mx_cols_kernel<T, F, false, 64>, 64, a, stream);
  }
  row_split((a.cols + GROUP - 1) / GROUP * 4, a.lanes, a.col_wgs);
  const int per = 256 / a.lanes * ROWS_IN<T>;
  return launch_all(mx_rows_kernel<T, F>, (a.N * a.rows + per - 1) / per * a.col_wgs, a, stream);
}

template <typename T, int F>
hipError_t dequantize(DequantArgs& a, hipStream_t stream) {
  constexpr int EACH = 16 / sizeof(T);
  row_split((a.cols + EACH - 1) / EACH, a.lanes, a.col_wgs);
  const int per = 256 / a.lanes * ROWS_BACK;
  return launch_all(mx_values_kernel<T, F>, (a.N * a.rows + per - 1) / per * a.col_wgs, a, stream);
}

bool row_aligned(const void* p, int64_t ld, size_t size) {
  return ((uintptr_t)p & 15) == 0 && ((size_t)ld * size) % 16 == 0;
}

}  // namespace

hipError_t launch_mx_quantize(const void* src, dash_prec type, int64_t N, int64_t rows, int64_t cols, int64_t ld,
                              dash_mx_fmt fmt, void* codes, void* scales, void* codes_t, void* scales_t, float* diag,
                              hipStream_t stream) {
  QuantArgs a{src, N, rows, cols, ld, (uint8_t*)codes, (uint8_t*)scales, (uint8_t*)codes_t, (uint8_t*)scales_t, diag,
              row_aligned(src, ld, type == DASH_FP32 ? 4 : 2), 0, 0, 0};
  const bool e4 = fmt == DASH_MX_E4M3;
  if (type == DASH_FP32)
    return e4 ? quantize<float, DASH_MX_E4M3>(a, stream) : quantize<float, DASH_MX_E2M1>(a, stream);
  if (type == DASH_BF16)
    return e4 ? quantize<__bf16, DASH_MX_E4M3>(a, stream) : quantize<__bf16, DASH_MX_E2M1>(a, stream);
  return e4 ? quantize<_Float16, DASH_MX_E4M3>(a, stream) : quantize<_Float16, DASH_MX_E2M1>(a, stream);
}

hipError_t launch_mx_dequantize(const void* codes, const void* scales, const float* diag, int64_t N, int64_t rows,
                                int64_t cols, dash_mx_fmt fmt, dash_prec type, int64_t ld, void* dst,
                                hipStream_t stream) {
  DequantArgs a{(const uint8_t*)codes, (const uint8_t*)scales, diag, N, rows, cols, ld, dst,
                row_aligned(dst, ld, type == DASH_FP32 ? 4 : 2), 0, 0, 0};
  const bool e4 = fmt == DASH_MX_E4M3;
  if (type == DASH_FP32)
    return e4 ? dequantize<float, DASH_MX_E4M3>(a, stream) : dequantize<float, DASH_MX_E2M1>(a, stream);
  if (type == DASH_BF16)
    return e4 ? dequantize<__bf16, DASH_MX_E4M3>(a, stream) : dequantize<__bf16, DASH_MX_E2M1>(a, stream);
  return e4 ? dequantize<_Float16, DASH_MX_E4M3>(a, stream) : dequantize<_Float16, DASH_MX_E2M1>(a, stream);
}

}  // namespace dash
