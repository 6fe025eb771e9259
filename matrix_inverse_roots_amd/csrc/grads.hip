// grads.hip -- the global norm of many gradients, and clipping them by it.
//
//   |g_i|^2 = sum x^2,  norm = (sum_i |g_i|^2)^{1/2},  g_i <- g_i min(1, most / norm)
//
// One read for the norm, one read and one write for the clipping: the bytes over the memory bandwidth is
// their time.  The tensors' descriptors travel as kernel arguments, GROUP_TENSORS to a launch; every tensor is cut into
// pieces of 16 bytes along its rows, and `per_wg` of them go to a workgroup.  Sums are kept
// in 64 bits, so that neither large nor small elements leave their range, and joined in a fixed order: equal
// calls give equal bits.
#include <hip/hip_runtime.h>

#include "dash_internal.hpp"
#include "vectors.hpp"

namespace dash {
namespace {

// (as many as the kernel arguments' 4 KiB hold: a launch of few small tensors costs what one of many does)
constexpr int GROUP_TENSORS = 160;
struct Tensors {
  uint64_t where[GROUP_TENSORS];     // address, and the type in the highest byte
  uint64_t size[GROUP_TENSORS];      // elements; or those of a row, and its pitch in the high half
  uint32_t rows[GROUP_TENSORS];      // 0: one run of elements
  int32_t wg_base[GROUP_TENSORS];    // first workgroup
  int32_t n, first;                  // `first`: number of the launch's first tensor
  int64_t wg_first;                  // and workgroup
  int64_t per_wg;
};
static_assert(sizeof(Tensors) <= 4000, "kernel arguments hold 4 KiB");

// The tensor of this workgroup, the last whose first workgroup is not behind it: every lane looks at some
__device__ __forceinline__ int find_tensor(const Tensors& g) {
  int below = 0;
#pragma unroll
  for (int i = 0; i < (GROUP_TENSORS + 63) / 64; ++i) {
    const int t = i * 64 + (threadIdx.x & 63);
    below += __popcll(__ballot(t < g.n && g.wg_base[t < GROUP_TENSORS ? t : 0] <= (int)blockIdx.x));
  }
  return __builtin_amdgcn_readfirstlane(below - 1);
}

// One tensor in pieces of 16 bytes
template <typename T>
struct Pieces {
  T* p;
  int64_t len, pieces;  // elements of a row (or of all), pieces of all
  uint32_t row_pieces, ld;
  bool flat;
  __device__ __forceinline__ Pieces(const Tensors& g, int t) {
    constexpr int E = EACH<T>;
    p = (T*)(g.where[t] & 0x00ffffffffffffffull);
    const uint64_t size = g.size[t];
    const uint32_t rows = g.rows[t];
    flat = rows == 0;
    len = flat ? (int64_t)size : (int64_t)(uint32_t)size;
    ld = (uint32_t)(size >> 32);
    row_pieces = (uint32_t)((len + E - 1) / E);
    pieces = flat ? (len + E - 1) / E : (int64_t)rows * row_pieces;
  }
};

// Calls f(row pointers, columns, row lengths) for DEPTH pieces at a time out of [first, first + most), every
// `threads`-th from `thread` on; pieces that there are not have length 0
template <int DEPTH, typename T, typename F>
__device__ __forceinline__ void each_piece(const Pieces<T>& v, int64_t first, int64_t most, int thread, int threads,
                                           F f) {
  constexpr int E = EACH<T>;
  const int64_t left = v.pieces - first, mine = left < most ? left : most;
  T* p = v.p;
  uint32_t at0 = 0;
  if (v.flat) {
    p += first * E;
  } else {  // (a row has fewer than 2^31 pieces, a workgroup fewer than 2^30)
    const int64_t row0 = first / v.row_pieces;
    at0 = (uint32_t)(first - row0 * v.row_pieces);
    p += row0 * (int64_t)v.ld;
  }
  for (int64_t i = thread; i < mine; i += (int64_t)threads * DEPTH) {
    T* row[DEPTH];
    int64_t c[DEPTH], len[DEPTH];
#pragma unroll
    for (int k = 0; k < DEPTH; ++k) {
      const int64_t at = i + (int64_t)threads * k;
      row[k] = p;
      c[k] = at * E;
      len[k] = v.flat ? v.len - first * E : v.len;
      if (!v.flat) {
        const uint32_t a = at0 + (uint32_t)at, r = a / v.row_pieces;
        row[k] = p + (int64_t)r * v.ld;
        c[k] = (int64_t)(a - r * v.row_pieces) * E;
      }
      if (at >= mine) len[k] = 0;
    }
    f(row, c, len);
  }
}

// Pieces that a thread has under way together (the norm of 6.4 GB with 2 / 4: 935 / 961 us)
constexpr int READ_DEPTH = 2, WRITE_DEPTH = 2;

template <bool PAST, typename T>
__device__ __forceinline__ double squares(const Tensors& g, int t, int64_t first, int64_t most, int thread,
                                          int threads) {
  double s = 0.;
  each_piece<READ_DEPTH>(Pieces<T>(g, t), first, most, thread, threads, [&](T* const* row, const int64_t* c,
                                                                       const int64_t* len) {
    vec_of<T> v[READ_DEPTH];
#pragma unroll
    for (int k = 0; k < READ_DEPTH; ++k) v[k] = load_short<PAST>(row[k], c[k], len[k]);
#pragma unroll
    for (int k = 0; k < READ_DEPTH; ++k) {
      float x[EACH<T>];
#pragma unroll
      for (int q = 0; q < EACH<T>; ++q) x[q] = (float)v[k][q];
      s += sum_squares<EACH<T>>(x);
    }
  });
  return s;
}
template <bool PAST>
__device__ __forceinline__ double squares_of(const Tensors& g, int t, int64_t first, int64_t most, int thread,
                                             int threads) {
  const int type = (int)(g.where[t] >> 56);
  if (type == DASH_FP32) return squares<PAST, float>(g, t, first, most, thread, threads);
  if (type == DASH_BF16) return squares<PAST, __bf16>(g, t, first, most, thread, threads);
  return squares<PAST, _Float16>(g, t, first, most, thread, threads);
}
__device__ __forceinline__ double wave_sum(double s) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) s += __shfl_xor(s, o, 64);
  return s;
}

// part[w] = the sum of squares of workgroup w's pieces; base[t] = tensor t's first workgroup.  HBM bounds it: 6.4 GB
// of fp32 in two launches 920 us (7.0 TB/s)
template <bool PAST>
__global__ __launch_bounds__(256) void grad_squares_kernel(Tensors g, double* part, int64_t* base) {
  const int t = find_tensor(g), w = (int)blockIdx.x - g.wg_base[t];
  const double s = wave_sum(squares_of<PAST>(g, t, w * g.per_wg, g.per_wg, threadIdx.x, 256));
  __shared__ double waves[4];
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x) return;
  part[g.wg_first + blockIdx.x] = (waves[0] + waves[1]) + (waves[2] + waves[3]);
  if (w == 0) base[g.first + t] = g.wg_first + blockIdx.x;
}

// A few small tensors: a wave takes one after the other, and their norm is ready with this launch (9 tensors of up to
// 2048 elements 4.5 us)
__global__ __launch_bounds__(1024) void grad_norm_small_kernel(Tensors g, float* norm, float* norms) {
  __shared__ double waves[16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  double all = 0.;
  for (int t = wave; t < g.n; t += 16) {
    const double s = wave_sum(squares_of<false>(g, t, 0, INT64_MAX, lane, 64));
    if (norms && lane == 0) norms[t] = (float)sqrt(s);
    all += s;
  }
  if (lane == 0) waves[wave] = all;
  __syncthreads();
  if (threadIdx.x) return;
  for (int i = 1; i < 16; ++i) all += waves[i];
  *norm = (float)sqrt(all);
}

// Workgroup 0: the norm of all; the others: each wave one tensor's (65536 sums 9 us: latency)
__global__ __launch_bounds__(1024) void grad_norm_kernel(const double* part, const int64_t* base, int64_t parts, int n,
                                                         float* norm, float* norms) {
  __shared__ double waves[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double s = 0.;
  if (blockIdx.x == 0) {
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < parts; i += 1024) s += part[i];
  } else {
    const int64_t t = (int64_t)(blockIdx.x - 1) * 16 + wave;
    if (t >= n) return;
    const int64_t end = t + 1 < n ? base[t + 1] : parts;
    for (int64_t i = base[t] + lane; i < end; i += 64) s += part[i];
  }
  s = wave_sum(s);
  if (blockIdx.x) {
    if (lane == 0) norms[(int64_t)(blockIdx.x - 1) * 16 + wave] = (float)sqrt(s);
    return;
  }
  if (lane == 0) waves[wave] = s;
  __syncthreads();
  if (threadIdx.x) return;
  for (int i = 1; i < 16; ++i) s += waves[i];
  *norm = (float)sqrt(s);
}

template <bool PAST, typename T>
__device__ __forceinline__ void clip_tensor(const Tensors& g, int t, float factor) {
  const int64_t first = (int64_t)((int)blockIdx.x - g.wg_base[t]) * g.per_wg;
  each_piece<WRITE_DEPTH>(Pieces<T>(g, t), first, g.per_wg, threadIdx.x, 256, [&](T* const* row, const int64_t* c,
                                                                            const int64_t* len) {
    vec_of<T> v[WRITE_DEPTH];
#pragma unroll
    for (int k = 0; k < WRITE_DEPTH; ++k) v[k] = load_short<PAST>(row[k], c[k], len[k]);
#pragma unroll
    for (int k = 0; k < WRITE_DEPTH; ++k) {
      float x[EACH<T>];
#pragma unroll
      for (int q = 0; q < EACH<T>; ++q) x[q] = (float)v[k][q] * factor;
      store_piece<PAST>(row[k], c[k], len[k], x);
    }
  });
}

// HBM bounds it: 0.8 GB of bfloat16 251 us (6.4 TB/s); a launch of 160 ragged tensors of up to 2^20 elements (62 MB)
// 17 us.
template <bool PAST>
__global__ __launch_bounds__(256) void grad_clip_kernel(Tensors g, const float* norm, float most) {
  const float factor = clip_factor(norm, most);
  if (factor == 1.f) return;  // (the gradients stay as they are)
  const int t = find_tensor(g), type = (int)(g.where[t] >> 56);
  if (type == DASH_FP32)
    clip_tensor<PAST, float>(g, t, factor);
  else if (type == DASH_BF16)
    clip_tensor<PAST, __bf16>(g, t, factor);
  else
    clip_tensor<PAST, _Float16>(g, t, factor);
}

// A tensor as the kernels take it: one run where nothing lies between its rows
struct Shape {
  int64_t rows, len;  // rows 0: one run
  int64_t pieces;
  Shape(const dash_tensor& g) {
    const int each = g.type == DASH_FP32 ? 4 : 8;
    rows = 0;
    len = g.rows * g.cols;
    if (len && g.rows > 1 && g.ld != g.cols) {
      rows = g.rows;
      len = g.cols;
    }
    pieces = (len + each - 1) / each * (rows ? rows : 1);
  }
  int64_t workgroups(int64_t per_wg) const { return pieces ? (pieces + per_wg - 1) / per_wg : 1; }
};

// How a list is shared out: pieces of a workgroup, and workgroups in all.  Clipping takes one pass of every thread (0.8
// GB of bfloat16 257 us; 16384 workgroups that loop 300), up to 2^22 workgroups; where nothing is clipped they read the
// norm and leave (0.8 GB 23 us, 6.4 GB of fp32 168).  The norm takes two passes, up to
// 65536 workgroups, whose sums one more launch adds (6.4 GB: 923 us, with 16384 of them 935, with 393216 1159).
struct Share {
  int64_t per_wg, wgs;
  bool small;  // for grad_norm_small_kernel
  bool past;   // the caches: they hold no part of it until the next pass
};
// One workgroup or two launches (tensors x bfloat16 elements, us): 9 x 512 3.1 / 5.2, 9 x 4096 4.5 / 5.1, 32 x 512 4.5 /
// 5.2, 32 x 4096 7.7 / 5.1, 64 x 512 7.3 / 5.3, 64 x 4096 13.8 / 5.2: at the rule's end the other way is the shorter one.
constexpr int64_t SMALL_PIECES = 512;
Share share_out(const dash_tensor* g, int n, bool write) {
  int64_t all = 0, most = 0;
  for (int i = 0; i < n; ++i) {
    const int64_t p = Shape(g[i]).pieces;
    all += p;
    if (p > most) most = p;
  }
  Share s;
  const int64_t step = 256 * (write ? WRITE_DEPTH : READ_DEPTH), least = write ? step : 2 * step;
  const int64_t even = (all / (write ? 1 << 22 : 1 << 16) + step - 1) / step * step;
  s.per_wg = even > least ? even : least;
  s.past = all * (write ? 32 : 16) > LARGE_BYTES;
  s.small = n <= 64 && most <= SMALL_PIECES;
  s.wgs = 0;
  for (int i = 0; i < n; ++i) s.wgs += Shape(g[i]).workgroups(s.per_wg);
  return s;
}

// f(group, its workgroups) for every launch
template <typename F>
hipError_t each_group(const dash_tensor* t, int n, const Share& s, F f) {
  int64_t wgs = 0;
  for (int i0 = 0; i0 < n;) {
    Tensors g;
    g.n = 0;
    g.first = i0;
    g.wg_first = wgs;
    g.per_wg = s.per_wg;
    int64_t here = 0;
    for (; i0 + g.n < n && g.n < GROUP_TENSORS; ++g.n) {
      const dash_tensor& m = t[i0 + g.n];
      const Shape r(m);
      const int64_t more = r.workgroups(s.per_wg);
      if (here + more > most_workgroups(256)) break;
      g.where[g.n] = (uint64_t)(uintptr_t)m.ptr | (uint64_t)m.type << 56;
      g.size[g.n] = r.rows ? (uint64_t)r.len | (uint64_t)m.ld << 32 : (uint64_t)r.len;
      g.rows[g.n] = (uint32_t)r.rows;
      g.wg_base[g.n] = (int32_t)here;
      here += more;
    }
    if (g.n == 0) return hipErrorInvalidValue;
    f(g, here);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    i0 += g.n;
    wgs += here;
  }
  return hipSuccess;
}

}  // namespace

size_t grad_norm_workspace_bytes(const dash_tensor* t, int n) {
  return align_up((size_t)share_out(t, n, false).wgs * sizeof(double), 256) + (size_t)n * sizeof(int64_t);
}

hipError_t launch_grad_norm(const dash_tensor* t, int n, float* norm, float* norms, void* ws, hipStream_t stream) {
  const Share s = share_out(t, n, false);
  if (s.small && n) {
    return each_group(t, n, s, [&](const Tensors& g, int64_t) {
      hipLaunchKernelGGL(grad_norm_small_kernel, dim3(1), dim3(1024), 0, stream, g, norm, norms);
    });
  }
  double* part = (double*)ws;
  int64_t* base = (int64_t*)((char*)ws + align_up((size_t)s.wgs * sizeof(double), 256));
  const hipError_t e = each_group(t, n, s, [&](const Tensors& g, int64_t wgs) {
    hipLaunchKernelGGL(s.past ? grad_squares_kernel<true> : grad_squares_kernel<false>, dim3((unsigned)wgs), dim3(256),
                       0, stream, g, part, base);
  });
  if (e != hipSuccess) return e;
  const int64_t grid = 1 + (norms ? ((int64_t)n + 15) / 16 : 0);
  hipLaunchKernelGGL(grad_norm_kernel, dim3((unsigned)grid), dim3(1024), 0, stream, part, base, s.wgs, n, norm, norms);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const dash_tensor* t, int n, const float* norm, float most, hipStream_t stream) {
  const Share s = share_out(t, n, true);
  return each_group(t, n, s, [&](const Tensors& g, int64_t wgs) {
    hipLaunchKernelGGL(s.past ? grad_clip_kernel<true> : grad_clip_kernel<false>, dim3((unsigned)wgs), dim3(256), 0,
                       stream, g, norm, most);
  });
}

}  // namespace dash
