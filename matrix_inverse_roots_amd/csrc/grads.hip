// grads.hip -- the global norm of many gradients, and clipping them by it.
//
//   |g_i|^2 = sum x^2,  norm = (sum_i |g_i|^2)^{1/2},  g_i <- g_i min(1, most / norm)
//
// One read for the norm, one read and one write for the clipping: the bytes over the memory bandwidth is
// their time.  The tensors' descriptors travel as kernel arguments, GROUP_TENSORS to a launch; every tensor is cut into
// pieces of 16 bytes along its rows and shared out evenly over workgroups, `per_wg` pieces each.  Sums are kept
// in 64 bits, so that neither large nor small elements leave their range, and joined in a fixed order: equal
// calls give equal bits.
#include <hip/hip_runtime.h>

#include "dash_internal.hpp"
#include "vectors.hpp"

namespace dash {
namespace {

constexpr int GROUP_TENSORS = 80;
struct Tensors {
  void* ptr[GROUP_TENSORS];
  int64_t pieces[GROUP_TENSORS];  // of all rows
  int64_t row_pieces[GROUP_TENSORS];
  int64_t len[GROUP_TENSORS], ld[GROUP_TENSORS];  // elements of a row, and its pitch
  int32_t wg_base[GROUP_TENSORS + 1];             // first workgroup
  uint8_t type[GROUP_TENSORS];
  int32_t n, first;  // `first`: number of the launch's first tensor
  int64_t wg_first;  // and workgroup
  int64_t per_wg;
};
static_assert(sizeof(Tensors) <= 4000, "kernel arguments hold 4 KiB");

// The tensor of this workgroup
__device__ __forceinline__ int find_tensor(const Tensors& g) {
  int lo = 0, hi = g.n;  // wg_base[lo] <= workgroup < wg_base[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((int)blockIdx.x >= g.wg_base[mid])
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Calls f(row pointer, column, row length) for every piece of this workgroup, DEPTH of them together
template <typename T, int DEPTH, typename F>
__device__ __forceinline__ void each_piece(const Tensors& g, int t, F f) {
  constexpr int E = EACH<T>;
  const int64_t first = (int64_t)((int)blockIdx.x - g.wg_base[t]) * g.per_wg;
  const int64_t left = g.pieces[t] - first, mine = left < g.per_wg ? left : g.per_wg;
  const int64_t row0 = first / g.row_pieces[t], at0 = first - row0 * g.row_pieces[t];
  T* const p = (T*)g.ptr[t] + row0 * g.ld[t];
  const bool flat = g.row_pieces[t] == g.pieces[t];  // (one row)
  for (int64_t i = threadIdx.x; i < mine; i += 256 * DEPTH) {
    T* row[DEPTH];
    int64_t c[DEPTH];
    bool in[DEPTH];
#pragma unroll
    for (int k = 0; k < DEPTH; ++k) {
      const int64_t at = at0 + i + 256 * k;
      in[k] = i + 256 * k < mine;
      if (flat) {
        row[k] = p;
        c[k] = at * E;
      } else {  // (at < 2^32: a row has fewer than 2^31 pieces, and so has a workgroup)
        const unsigned r = (unsigned)at / (unsigned)g.row_pieces[t];
        row[k] = p + r * g.ld[t];
        c[k] = (int64_t)((unsigned)at - r * (unsigned)g.row_pieces[t]) * E;
      }
    }
    f(row, c, in, g.len[t]);
  }
}

constexpr int DEPTH = 4;

template <typename T>
__device__ __forceinline__ double tensor_squares(const Tensors& g, int t) {
  double s = 0.;
  each_piece<T, DEPTH>(g, t, [&](T* const* row, const int64_t* c, const bool* in, int64_t len) {
    vec_of<T> v[DEPTH];
#pragma unroll
    for (int k = 0; k < DEPTH; ++k) v[k] = load_short(row[k], c[k], in[k] ? len : 0);
#pragma unroll
    for (int k = 0; k < DEPTH; ++k) {
      float x[EACH<T>];
#pragma unroll
      for (int q = 0; q < EACH<T>; ++q) x[q] = (float)v[k][q];
      s += sum_squares<EACH<T>>(x);
    }
  });
  return s;
}

// part[w] = the sum of squares of workgroup w's pieces; base[t] = tensor t's first workgroup
__global__ __launch_bounds__(256) void grad_squares_kernel(Tensors g, double* part, int64_t* base) {
  const int t = find_tensor(g);
  double s;
  if (g.type[t] == DASH_FP32)
    s = tensor_squares<float>(g, t);
  else if (g.type[t] == DASH_BF16)
    s = tensor_squares<__bf16>(g, t);
  else
    s = tensor_squares<_Float16>(g, t);
  __shared__ double waves[4];
#pragma unroll
  for (int o = 1; o < 64; o *= 2) s += __shfl_xor(s, o, 64);
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x) return;
  part[g.wg_first + blockIdx.x] = (waves[0] + waves[1]) + (waves[2] + waves[3]);
  if ((int)blockIdx.x == g.wg_base[t]) base[g.first + t] = g.wg_first + blockIdx.x;
}

// Workgroup 0: the norm of all; the others: each wave one tensor's
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
#pragma unroll
  for (int o = 1; o < 64; o *= 2) s += __shfl_xor(s, o, 64);
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

template <typename T>
__device__ __forceinline__ void clip_tensor(const Tensors& g, int t, float factor) {
  each_piece<T, DEPTH>(g, t, [&](T* const* row, const int64_t* c, const bool* in, int64_t len) {
    vec_of<T> v[DEPTH];
#pragma unroll
    for (int k = 0; k < DEPTH; ++k) v[k] = load_short(row[k], c[k], in[k] ? len : 0);
#pragma unroll
    for (int k = 0; k < DEPTH; ++k) {
      float x[EACH<T>];
#pragma unroll
      for (int q = 0; q < EACH<T>; ++q) x[q] = (float)v[k][q] * factor;
      store_piece(row[k], c[k], in[k] ? len : 0, x);
    }
  });
}

__global__ __launch_bounds__(256) void grad_clip_kernel(Tensors g, const float* norm, float most) {
  const float factor = clip_factor(norm, most);
  if (factor == 1.f) return;  // (the gradients stay as they are)
  const int t = find_tensor(g);
  if (g.type[t] == DASH_FP32)
    clip_tensor<float>(g, t, factor);
  else if (g.type[t] == DASH_BF16)
    clip_tensor<__bf16>(g, t, factor);
  else
    clip_tensor<_Float16>(g, t, factor);
}

// A tensor as rows: one where nothing lies between them
struct Rows {
  int64_t rows, len, ld, row_pieces;
  Rows(const dash_tensor& g) {
    const int each = g.type == DASH_FP32 ? 4 : 8;
    rows = g.rows;
    len = g.cols;
    ld = g.ld;
    if (rows == 0 || len == 0) {
      rows = 1;
      len = 0;
    } else if (ld == len || rows == 1) {
      len *= rows;
      rows = 1;
    }
    row_pieces = (len + each - 1) / each;
    if (row_pieces == 0) row_pieces = 1;  // (an empty tensor has a piece of no elements)
  }
  int64_t pieces() const { return rows * row_pieces; }
};

// Pieces of a workgroup: enough to hide the latency of its start (16 for each thread, 64 KiB a workgroup), more
// where that would make over 16384 workgroups
int64_t pieces_per_wg(const dash_tensor* g, int n) {
  int64_t all = 0;
  for (int i = 0; i < n; ++i) all += Rows(g[i]).pieces();
  const int64_t least = 256 * 16;
  const int64_t even = (all / 16384 + 256 * DEPTH - 1) / (256 * DEPTH) * (256 * DEPTH);
  return even > least ? even : least;
}

// f(group, its workgroups) for every launch
template <typename F>
hipError_t each_group(const dash_tensor* t, int n, F f) {
  const int64_t per_wg = pieces_per_wg(t, n);
  int64_t wgs = 0;
  for (int i0 = 0; i0 < n;) {
    Tensors g{};
    g.first = i0;
    g.wg_first = wgs;
    g.per_wg = per_wg;
    int64_t here = 0;
    for (; i0 + g.n < n && g.n < GROUP_TENSORS; ++g.n) {
      const dash_tensor& m = t[i0 + g.n];
      const Rows r(m);
      const int64_t more = (r.pieces() + per_wg - 1) / per_wg;
      if (here + more > most_workgroups(256)) break;
      g.ptr[g.n] = m.ptr;
      g.pieces[g.n] = r.pieces();
      g.row_pieces[g.n] = r.row_pieces;
      g.len[g.n] = r.len;
      g.ld[g.n] = r.ld;
      g.type[g.n] = (uint8_t)m.type;
      here += more;
      g.wg_base[g.n + 1] = (int32_t)here;
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

int64_t all_workgroups(const dash_tensor* t, int n) {
  const int64_t per_wg = pieces_per_wg(t, n);
  int64_t wgs = 0;
  for (int i = 0; i < n; ++i) wgs += (Rows(t[i]).pieces() + per_wg - 1) / per_wg;
  return wgs;
}

}  // namespace

size_t grad_norm_workspace_bytes(const dash_tensor* t, int n) {
  return align_up((size_t)all_workgroups(t, n) * sizeof(double), 256) + (size_t)n * sizeof(int64_t);
}

hipError_t launch_grad_norm(const dash_tensor* t, int n, float* norm, float* norms, void* ws, hipStream_t stream) {
  const int64_t parts = all_workgroups(t, n);
  double* part = (double*)ws;
  int64_t* base = (int64_t*)((char*)ws + align_up((size_t)parts * sizeof(double), 256));
  const hipError_t e = each_group(t, n, [&](const Tensors& g, int64_t wgs) {
    hipLaunchKernelGGL(grad_squares_kernel, dim3((unsigned)wgs), dim3(256), 0, stream, g, part, base);
  });
  if (e != hipSuccess) return e;
  const int64_t grid = 1 + (norms ? ((int64_t)n + 15) / 16 : 0);
  hipLaunchKernelGGL(grad_norm_kernel, dim3((unsigned)grid), dim3(1024), 0, stream, part, base, parts, n, norm, norms);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const dash_tensor* t, int n, const float* norm, float most, hipStream_t stream) {
  return each_group(t, n, [&](const Tensors& g, int64_t wgs) {
    hipLaunchKernelGGL(grad_clip_kernel, dim3((unsigned)wgs), dim3(256), 0, stream, g, norm, most);
  });
}

}  // namespace dash
