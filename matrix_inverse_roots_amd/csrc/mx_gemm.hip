// mx_gemm.hip -- batched products with microscaled operands: the Shampoo statistics from
// microscaled gradient tiles, the preconditioned update with microscaled roots, and gradient tiles
// from a layer's microscaled input.
//
// A microscaled element is c 2^(s - 127) with c an E2M1 or E4M3 value (at most 4 significant bits)
// and s its group's scale byte.  bfloat16 has 8 significant bits and fp32's exponent range, so every
// element is a bfloat16 number exactly (elements below 2^-126 lose their lowest bits to bfloat16's
// subnormals), scale included, and the 32x32x16 bfloat16 MFMA forms products of two elements exactly
// and sums them in fp32.  (The scaled 8-bit MFMA, at twice the rate, drops bits below the largest
// addend of its 64: sums of 4096 positive E4M3 products came out 7e-5 low, a hundred times fp32's own
// error, so it is not used; the 4-bit one sums exactly within a group, and the E2M1 statistics use it.)
// A floating operand beside a microscaled one is cut into bfloat16 pieces that add up to it exactly
// (one for bfloat16, two for binary16, three for fp32), or into two binary16 pieces (the update), and
// each piece multiplies the one microscaled piece: exact products again, accumulated in fp32.
//
// One frame: an output tile of TILE x TILE, 2 TILE threads, k-slices of 32 (one scale group along k), a
// register ring of slices under way and an LDS double buffer of 16-bit planes, one per piece.  An operand
// whose k is contiguous in memory sits in LDS as [row][32 k], one whose k is the slow axis as [k][TILE],
// read back k-major by the transposing LDS load.
#include <hip/hip_runtime.h>

#include <cmath>
#include <type_traits>

#include "gemm_common.hpp"

namespace dash {
namespace gemm {
namespace {

template <int V>
using IC = std::integral_constant<int, V>;

constexpr int BK = 32;  // k-slice: one scale group

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------------------------------------
// Elements
// ------------------------------------------------------------------------------------------------

// The scale as the conversion instructions take it: only the exponent field of the fp32 operand
// counts, so a scale byte in that field is the scale (255 makes the results NaN).
__device__ __forceinline__ float scale_of(unsigned byte) { return __builtin_bit_cast(float, byte << 23); }

// Two elements to bfloat16 or binary16: the two of a byte (E2M1, byte I of w) or of half a word (E4M3,
// half I of w)
template <typename TE>
struct Pair;
template <>
struct Pair<__bf16> {
  typedef bf16x2 type;
  template <int I>
  static __device__ __forceinline__ type e4m3(unsigned w, float s) {
    return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, I);
  }
  template <int I>
  static __device__ __forceinline__ type e2m1(unsigned w, float s) {
    return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, I);
  }
};
template <>
struct Pair<_Float16> {
  typedef f16x2 type;
  template <int I>
  static __device__ __forceinline__ type e4m3(unsigned w, float s) {
    return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, s, I);
  }
  template <int I>
  static __device__ __forceinline__ type e2m1(unsigned w, float s) {
    return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, I);
  }
};

// 8 consecutive elements, from 8 bytes (E4M3) or 4 (E2M1).  TOP: the exponent t for which the largest
// element value times 2^t is in [2^13, 2^14)
template <int F>
struct Elem;
template <>
struct Elem<DASH_MX_E4M3> {
  typedef u32x2 raw8;
  static constexpr int BITS = 8, TOP = 5;
  template <typename TE>
  static __device__ __forceinline__ typename Half<TE>::v8 decode(raw8 r, float s) {
    const auto a = Pair<TE>::template e4m3<0>(r[0], s), b = Pair<TE>::template e4m3<1>(r[0], s);
    const auto c = Pair<TE>::template e4m3<0>(r[1], s), d = Pair<TE>::template e4m3<1>(r[1], s);
    return typename Half<TE>::v8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  }
};
template <>
struct Elem<DASH_MX_E2M1> {
  typedef unsigned raw8;
  static constexpr int BITS = 4, TOP = 11;
  template <typename TE>
  static __device__ __forceinline__ typename Half<TE>::v8 decode(raw8 r, float s) {
    const auto a = Pair<TE>::template e2m1<0>(r, s), b = Pair<TE>::template e2m1<1>(r, s);
    const auto c = Pair<TE>::template e2m1<2>(r, s), d = Pair<TE>::template e2m1<3>(r, s);
    return typename Half<TE>::v8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  }
};

// x = p[0] + p[1] + ... for the 8 elements lo[0..3], hi[0..3]: each piece the nearest bfloat16 to what is
// left, every difference exact in fp32.  Three pieces hold fp32's bits (split3), two binary16's 11.  An Inf, or
// a magnitude that rounds to one, leaves Inf - Inf, NaN, in the second piece; and the products of two pieces
// that differ in sign may overflow to infinities that do.
// INF: pieces of one sign, cut off instead of rounded (8 bits each, so they hold x all the same), with an Inf
// or a NaN in the first alone.  Their products' sum is finite, Inf or NaN where x's product is.
template <int P, bool INF>
__device__ __forceinline__ void pieces(const f32x4& lo, const f32x4& hi, bf16x8 (&p)[P]) {
  static_assert(P == 2 || P == 3, "binary16 or fp32");
  if constexpr (INF) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      float left = q < 4 ? lo[q] : hi[q - 4];
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const bool finite = fabsf(left) < __builtin_inff();
        const float a = finite ? __builtin_bit_cast(float, __builtin_bit_cast(unsigned, left) & 0xffff0000u) : left;
        p[i][q] = (__bf16)a;
        left = finite ? left - a : 0.f;
      }
    }
  } else if constexpr (P == 3) {
    split3(lo, hi, p[0], p[1], p[2]);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float x = q < 4 ? lo[q] : hi[q - 4];
      p[0][q] = (__bf16)x;
      p[1][q] = (__bf16)(x - (float)p[0][q]);
    }
  }
}

// ------------------------------------------------------------------------------------------------
// LDS planes: TILE x 32 elements of 16 bits
// ------------------------------------------------------------------------------------------------

// [row][32 k]: rows of four 16-byte chunks; the chunk index is xored with bits 2-3 and bit 1 of the row.
// The 16-byte reads of 16 rows then fall on 16 distinct slots of 256 bytes, and the 16-byte writes of 8
// lanes (two chunks of four rows, or four of two) on 8 distinct slots of 128 bytes
__device__ __forceinline__ int kc_at(int row, int chunk) {
  return row * BK + 8 * (chunk ^ ((row >> 2) & 3) ^ ((row >> 1) & 1));
}

// [k][TILE]: the 64-byte block of 32 columns is xored with k % 4 (with 64 columns, two blocks to a row
// of half the banks, with bit 1 of k), so the four rows that one transposing load reads fall on distinct
// banks
template <int TILE>
__device__ __forceinline__ int ks_at(int k, int col) {
  const int turn = TILE == 64 ? (k >> 1) & 1 : k & 3;
  return k * TILE + ((((col >> 5) ^ turn) << 5) | (col & 31));
}

// The MFMA operand of rows (columns) base .. base + 31, k = 16 ks .. 16 ks + 15: lane l holds row
// l % 32, k = 8 (l / 32) .. + 7.
template <int TILE, bool KS, typename TE>
__device__ __forceinline__ typename Half<TE>::v8 fragment(const TE* plane, int base, int ks, int lane) {
  if constexpr (!KS) {
    return *(const typename Half<TE>::v8*)&plane[kc_at(base + (lane & 31), 2 * ks + (lane >> 5))];
  } else {
    // transposing load: in each group of 16 lanes, lane 4 r + c points at four columns of row r; lane i
    // receives column i of the group's four rows
    const int k = 16 * ks + 8 * (lane >> 5) + ((lane & 15) >> 2);
    const int col = base + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    typedef __attribute__((address_space(3))) s16x4* lds_ptr;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)&plane[ks_at<TILE>(k, col)]);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)&plane[ks_at<TILE>(k + 4, col)]);
    return __builtin_bit_cast(typename Half<TE>::v8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
}

// ------------------------------------------------------------------------------------------------
// Operand loaders.  init: the thread's place in the tile whose first row (column) is r0; load: slice
// kt into ring slot SLOT (CHECK: with the matrix's edges minded; the others are whole); store: a slot
// into LDS planes.  An address is a wave-uniform base that moves with kt plus a 32-bit lane offset.
// ------------------------------------------------------------------------------------------------

// DEPTH: slices in the register ring, 4, but 2 beside an fp32 operand in 256 x 256 tiles (where four
// spill) and in the update (where four changed nothing at any width).

// Microscaled, k contiguous: thread t holds 16 k of row t / 2.  Rows beyond the matrix are zero.
// shift: added to the scale bytes (a power of two on every element).
template <int F, int TILE, int D, typename E>
struct CodesK {
  typedef E TE;
  static constexpr int DEPTH = D;
  static constexpr int PIECES = 1;
  static constexpr bool KS = false;
  typedef typename Elem<F>::raw8 raw8;
  const uint8_t *c, *s;
  unsigned off_c, off_s;
  raw8 r[DEPTH][2];
  unsigned sc[DEPTH];
  int row, half, shift;
  bool in;
  __device__ __forceinline__ void init(const MxCodes& q, int64_t b, int64_t r0, int tid, int shift_ = 0) {
    row = tid >> 1;
    in = r0 + row < q.rows;
    half = tid & 1;
    shift = shift_;
    const int64_t at = b * q.rows + r0;
    c = q.codes + at * q.row_bytes;
    s = q.scales + at * q.row_groups;
    off_c = (unsigned)row * (unsigned)q.row_bytes + half * (2 * Elem<F>::BITS);
    off_s = (unsigned)row * (unsigned)q.row_groups;
  }
  template <int SLOT, bool CHECK>
  __device__ __forceinline__ void load(int64_t kt) {
    if (CHECK) {
      r[SLOT][0] = r[SLOT][1] = raw8{};
      sc[SLOT] = 0;
      if (!in) return;
    }
    const raw8* p = (const raw8*)(c + kt * (BK * Elem<F>::BITS / 8) + off_c);
    r[SLOT][0] = p[0];
    r[SLOT][1] = p[1];
    sc[SLOT] = (s + kt)[off_s];
  }
  template <int SLOT>
  __device__ __forceinline__ void store(TE* planes) const {
    unsigned byte = sc[SLOT];
    if (!std::is_same<TE, __bf16>::value) {
      const int moved = (int)byte + shift;
      byte = byte == 255u ? 255u : moved > 0 ? (unsigned)moved : 0u;
    }
    const float f = scale_of(byte);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *(typename Half<TE>::v8*)&planes[kc_at(row, 2 * half + i)] = Elem<F>::template decode<TE>(r[SLOT][i], f);
  }
};

// Microscaled, k the slow axis (rows of the stored matrix are k): thread t holds 8 columns of two of the
// slice's rows, 16 apart.  Columns beyond the stored row and rows beyond K are zero.
template <int F, int TILE, int D>
struct CodesCol {
  typedef __bf16 TE;
  static constexpr int DEPTH = D;
  static constexpr int PIECES = 1;
  static constexpr bool KS = true;
  typedef typename Elem<F>::raw8 raw8;
  const uint8_t *c, *s;
  unsigned off_c, off_s;
  raw8 r[DEPTH][2];
  unsigned sc[DEPTH][2];
  int64_t row_c, row_s, left;  // left: rows from this thread's first one to the last
  int k, col;
  __device__ __forceinline__ void init(const MxCodes& q, int64_t c0, int64_t k0, int64_t k1, int tid) {
    col = 8 * (tid % (TILE / 8));
    k = tid / (TILE / 8);
    row_c = q.row_bytes;
    row_s = q.row_groups;
    c = q.codes + k0 * row_c + c0 * Elem<F>::BITS / 8;
    s = q.scales + k0 * row_s + c0 / 32;
    off_c = (unsigned)k * (unsigned)row_c + col * Elem<F>::BITS / 8;
    off_s = (unsigned)k * (unsigned)row_s + col / 32;
    left = c0 + col < row_s * 32 ? k1 - k0 - k : 0;
  }
  template <int SLOT, bool CHECK>
  __device__ __forceinline__ void load(int64_t kt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t at = kt * BK + 16 * i;
      if (CHECK) {
        r[SLOT][i] = raw8{};
        sc[SLOT][i] = 0;
        if (at >= left) continue;
      }
      r[SLOT][i] = *(const raw8*)(c + at * row_c + off_c);
      sc[SLOT][i] = (s + at * row_s)[off_s];
    }
  }
  template <int SLOT>
  __device__ __forceinline__ void store(__bf16* planes) const {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *(bf16x8*)&planes[ks_at<TILE>(k + 16 * i, col)] =
          Elem<F>::template decode<TE>(r[SLOT][i], scale_of(sc[SLOT][i]));
  }
};

// fp32, k contiguous, two binary16 pieces of 2^e x: thread t holds 8 k of rows t / 4 and t / 4 + TILE / 2
// (four lanes read a row's 128 bytes).  Rows from x.cols on (the matrices are square) are zero.  m1 is
// -1 (see split2).
template <int TILE>
struct FloatK {
  typedef _Float16 TE;
  static constexpr int DEPTH = 2;
  static constexpr int PIECES = 2;
  static constexpr bool KS = false;
  const float* p;
  unsigned off;
  f32x4 r[DEPTH][2][2];
  int64_t half;  // elements from one of the thread's rows to the other
  int row, chunk, e;
  bool in[2];
  float m1;
  __device__ __forceinline__ void init(const MxFloats& x, int64_t b, int64_t r0, int tid, int e_, float m1_) {
    row = tid >> 2;
    chunk = tid & 3;
    e = e_;
    m1 = m1_;
    in[0] = r0 + row < x.cols;
    in[1] = r0 + row + TILE / 2 < x.cols;
    p = (const float*)x.p + b * x.stride + r0 * x.ld;
    half = x.ld * (TILE / 2);
    off = (unsigned)row * (unsigned)x.ld + 8 * chunk;
  }
  template <int SLOT, bool CHECK>
  __device__ __forceinline__ void load(int64_t kt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (CHECK) {
        r[SLOT][i][0] = r[SLOT][i][1] = f32x4{};
        if (!in[i]) continue;
      }
      const float* q = p + kt * BK + i * half + off;
      r[SLOT][i][0] = *(const f32x4*)q;
      r[SLOT][i][1] = *(const f32x4*)(q + 4);
    }
  }
  template <int SLOT>
  __device__ __forceinline__ void store(TE* planes) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f16x8 p0, p1;
      split2(r[SLOT][i][0], r[SLOT][i][1], e, m1, p0, p1);
      TE* at = planes + kc_at(row + i * (TILE / 2), chunk);
      *(f16x8*)at = p0;
      *(f16x8*)(at + TILE * BK) = p1;
    }
  }
};

// fp32, k the slow axis, two binary16 pieces of 2^e x: thread t holds 8 columns of two of the slice's
// rows, 16 apart.  Columns beyond the matrix are zero; the slices' rows all exist.
template <int TILE>
struct FloatCol16 {
  typedef _Float16 TE;
  static constexpr int DEPTH = 2;
  static constexpr int PIECES = 2;
  static constexpr bool KS = true;
  const float* p;
  unsigned off;
  f32x4 r[DEPTH][2][2];
  int64_t ld;
  int k, col, e;
  bool in;
  float m1;
  __device__ __forceinline__ void init(const MxFloats& x, int64_t b, int64_t c0, int tid, int e_, float m1_) {
    col = 8 * (tid % (TILE / 8));
    k = tid / (TILE / 8);
    ld = x.ld;
    e = e_;
    m1 = m1_;
    in = c0 + col < x.cols;
    p = (const float*)x.p + b * x.stride + c0;
    off = (unsigned)k * (unsigned)ld + col;
  }
  template <int SLOT, bool CHECK>
  __device__ __forceinline__ void load(int64_t kt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (CHECK) {
        r[SLOT][i][0] = r[SLOT][i][1] = f32x4{};
        if (!in) continue;
      }
      const float* q = p + (kt * BK + 16 * i) * ld + off;
      r[SLOT][i][0] = *(const f32x4*)q;
      r[SLOT][i][1] = *(const f32x4*)(q + 4);
    }
  }
  template <int SLOT>
  __device__ __forceinline__ void store(TE* planes) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f16x8 p0, p1;
      split2(r[SLOT][i][0], r[SLOT][i][1], e, m1, p0, p1);
      TE* at = planes + ks_at<TILE>(k + 16 * i, col);
      *(f16x8*)at = p0;
      *(f16x8*)(at + TILE * BK) = p1;
    }
  }
};

// fp32, bfloat16 or binary16, k the slow axis, in bfloat16 pieces: thread t holds 8 columns of two of the slice's rows, 16
// apart.  Columns and rows beyond the matrix are zero; only elements of the matrix are read.
template <typename T>
struct Pieces {
  static constexpr int N = std::is_same<T, float>::value ? 3 : std::is_same<T, _Float16>::value ? 2 : 1;
};
template <typename T, int TILE, int D, bool INF>
struct FloatCol {
  typedef __bf16 TE;
  static constexpr int DEPTH = D;
  static constexpr int PIECES = Pieces<T>::N;
  static constexpr bool KS = true;
  typedef T v8 __attribute__((ext_vector_type(8), aligned(16)));
  const T* p;
  unsigned off;
  v8 r[DEPTH][2];
  int64_t ld, left;
  int k, col, wide;  // wide: elements of the thread's 8 columns that exist
  bool vec;          // all 8, in rows that start on 16 bytes
  __device__ __forceinline__ void init(const MxFloats& x, int64_t b, int64_t c0, int64_t k0, int64_t k1, int tid) {
    col = 8 * (tid % (TILE / 8));
    k = tid / (TILE / 8);
    ld = x.ld;
    p = (const T*)x.p + b * x.stride + k0 * ld + c0;
    off = (unsigned)k * (unsigned)ld + col;
    const int64_t in = x.cols - c0 - col;
    wide = in >= 8 ? 8 : in > 0 ? (int)in : 0;
    vec = x.vec && wide == 8;
    left = wide ? k1 - k0 - k : 0;
  }
  template <int SLOT, bool CHECK>
  __device__ __forceinline__ void load(int64_t kt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t at = kt * BK + 16 * i;
      const T* q = p + at * ld + off;
      if (!CHECK) {
        r[SLOT][i] = *(const v8*)q;
        continue;
      }
      r[SLOT][i] = v8{};
      if (at >= left) continue;
      if (vec) {
        r[SLOT][i] = *(const v8*)q;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < wide) r[SLOT][i][e] = q[e];
      }
    }
  }
  template <int SLOT>
  __device__ __forceinline__ void store(__bf16* planes) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      bf16x8 v[PIECES];
      if constexpr (PIECES == 1) {
        v[0] = __builtin_bit_cast(bf16x8, r[SLOT][i]);
      } else {
        f32x4 lo, hi;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          lo[q] = (float)r[SLOT][i][q];
          hi[q] = (float)r[SLOT][i][4 + q];
        }
        pieces<PIECES, INF>(lo, hi, v);
      }
#pragma unroll
      for (int q = 0; q < PIECES; ++q) *(bf16x8*)&planes[q * TILE * BK + ks_at<TILE>(k + 16 * i, col)] = v[q];
    }
  }
};

// ------------------------------------------------------------------------------------------------
// The product of one tile: acc = sum over slices of A's rows times B's columns
// ------------------------------------------------------------------------------------------------

// Waves of a tile: 256 -> 2 x 4 waves of 128 x 64, 128 -> 2 x 2 of 64 x 64, 64 -> 2 x 1 of 32 x 64
template <int TILE>
struct Shape;
template <>
struct Shape<256> {
  static constexpr int WN = 4, MTM = 4, MTN = 2;
};
template <>
struct Shape<128> {
  static constexpr int WN = 2, MTM = 2, MTN = 2;
};
template <>
struct Shape<64> {
  static constexpr int WN = 1, MTM = 1, MTN = 2;
};

// One slice: PA planes of A at st, PB planes of B at stb
template <int TILE, int PA, int PB, bool KSA, bool KSB, typename TE>
__device__ __forceinline__ void multiply_slice(const TE* st, const TE* stb, int wm, int wn, int lane,
                                               f32x16 (&acc)[Shape<TILE>::MTM][Shape<TILE>::MTN]) {
  constexpr int MTM = Shape<TILE>::MTM, MTN = Shape<TILE>::MTN;
  constexpr int PLANE = TILE * BK;
#pragma unroll
  for (int ks = 0; ks < 2; ++ks)
#pragma unroll
    for (int pb = 0; pb < PB; ++pb) {
      typename Half<TE>::v8 bv[MTN];
#pragma unroll
      for (int nt = 0; nt < MTN; ++nt)
        bv[nt] = fragment<TILE, KSB>(stb + pb * PLANE, (wn * MTN + nt) * 32, ks, lane);
#pragma unroll
      for (int pa = 0; pa < PA; ++pa)
#pragma unroll
        for (int mt = 0; mt < MTM; ++mt) {
          const auto av = fragment<TILE, KSA>(st + pa * PLANE, (wm * MTM + mt) * 32, ks, lane);
#pragma unroll
          for (int nt = 0; nt < MTN; ++nt) acc[mt][nt] = Half<TE>::mfma(av, bv[nt], acc[mt][nt]);
        }
    }
}

template <int MTM, int MTN>
__device__ __forceinline__ void clear(f32x16 (&acc)[MTM][MTN]) {
#pragma unroll
  for (int mt = 0; mt < MTM; ++mt)
#pragma unroll
    for (int nt = 0; nt < MTN; ++nt)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[mt][nt][r] = 0.f;
}

// Time of a launch by tile width, in us per k-slice: `lat` is what a slice takes in a compute unit with
// one workgroup or few, `thr` each workgroup's share where a unit holds `cap` of them.  A launch is full
// rounds of 256 cap workgroups and a last one.
struct TileRate {
  int tile;
  double lat, thr;
  int cap;
};
inline double slice_time(const TileRate& r, double workgroups) {
  const double w = workgroups / 256, full = floor(w / r.cap), rest = w - full * r.cap;
  return full * r.thr * r.cap + (rest > 0 ? (r.lat > r.thr * rest ? r.lat : r.thr * rest) : 0);
}

// slices: of k; whole: the leading ones that need no checks
template <int TILE, typename LA, typename LB>
__device__ __forceinline__ void multiply(LA& la, LB& lb, int64_t slices, int64_t whole, typename LA::TE* stage0,
                                         typename LA::TE* stage1, int wm, int wn, int lane,
                                         f32x16 (&acc)[Shape<TILE>::MTM][Shape<TILE>::MTN]) {
  constexpr int PLANE = TILE * BK;
  constexpr int PA = LA::PIECES, PB = LB::PIECES;
  typedef typename LA::TE TE;
  static_assert(std::is_same<TE, typename LB::TE>::value, "operands of one type");
  constexpr int DEPTH = LA::DEPTH;
  static_assert(DEPTH == LB::DEPTH && (DEPTH == 2 || DEPTH == 4), "the loops below step through 2 or 4 slots");
  clear(acc);
  if (slices <= 0) return;

  auto compute = [&](const TE* st) {
    multiply_slice<TILE, PA, PB, LA::KS, LB::KS>(st, st + PA * PLANE, wm, wn, lane, acc);
  };
  auto load = [&](auto slot_c, auto check_c, int64_t kt) {
    la.template load<decltype(slot_c)::value, decltype(check_c)::value>(kt);
    lb.template load<decltype(slot_c)::value, decltype(check_c)::value>(kt);
  };
  auto store = [&](auto slot_c) {  // (slices alternate between the stages)
    constexpr int slot = decltype(slot_c)::value;
    TE* st = slot & 1 ? stage1 : stage0;
    la.template store<slot>(st);
    lb.template store<slot>(st + PA * PLANE);
  };
  // steady state: the loads of slice kt + DEPTH go into the registers that slice kt left, slice kt + 1 moves
  // from registers to the other stage, slice kt is multiplied
  auto step = [&](auto slot_c, int64_t kt) {
    constexpr int slot = decltype(slot_c)::value;
    load(slot_c, IC<0>{}, kt + DEPTH);
    store(IC<(slot + 1) % DEPTH>{});
    compute(slot & 1 ? stage1 : stage0);
    // two binary16 pieces: asks for the split's arithmetic between the products instead of before them
    // (384 x 1024 4.19 -> 4.03 ms; the gradient tiles came out level or 1 % slower)
    if constexpr (TILE == 256 && std::is_same<TE, _Float16>::value) {
      constexpr int PRODUCTS = 2 * PA * PB * Shape<TILE>::MTM * Shape<TILE>::MTN;
      constexpr int VALU = 0x2, MFMA = 0x8, VMEM_READ = 0x20, DS_READ = 0x100, DS_WRITE = 0x200;
      __builtin_amdgcn_sched_group_barrier(VMEM_READ, 16, 0);
      __builtin_amdgcn_sched_group_barrier(DS_READ, 6, 0);
#pragma unroll
      for (int m = 0; m < PRODUCTS; ++m) {
        __builtin_amdgcn_sched_group_barrier(MFMA, 1, 0);
        __builtin_amdgcn_sched_group_barrier(VALU, 4, 0);
        __builtin_amdgcn_sched_group_barrier(DS_READ, 1, 0);
        if (m >= PRODUCTS / 4) __builtin_amdgcn_sched_group_barrier(DS_WRITE, 1, 0);
      }
    }
    __syncthreads();
  };
  auto last_step = [&](auto slot_c, int64_t kt) {
    constexpr int slot = decltype(slot_c)::value;
    if (kt >= slices) return;
    if (kt + DEPTH < slices) load(slot_c, IC<1>{}, kt + DEPTH);
    if (kt + 1 < slices) store(IC<(slot + 1) % DEPTH>{});
    compute(slot & 1 ? stage1 : stage0);
    __syncthreads();
  };
  load(IC<0>{}, IC<1>{}, 0);
  if (slices > 1) load(IC<1>{}, IC<1>{}, 1);
  if constexpr (DEPTH == 4) {
    if (slices > 2) load(IC<2>{}, IC<1>{}, 2);
    if (slices > 3) load(IC<3>{}, IC<1>{}, 3);
  }
  store(IC<0>{});
  __syncthreads();
  int64_t kt = 0;
  for (; kt + 2 * DEPTH <= whole; kt += DEPTH) {
    step(IC<0>{}, kt);
    step(IC<1>{}, kt + 1);
    if constexpr (DEPTH == 4) {
      step(IC<2>{}, kt + 2);
      step(IC<3>{}, kt + 3);
    }
  }
  for (; kt < slices; kt += DEPTH) {
    last_step(IC<0>{}, kt);
    last_step(IC<1>{}, kt + 1);
    if constexpr (DEPTH == 4) {
      last_step(IC<2>{}, kt + 2);
      last_step(IC<3>{}, kt + 3);
    }
  }
}

// ------------------------------------------------------------------------------------------------
// Two E4M3 operands, k contiguous in both
// ------------------------------------------------------------------------------------------------
//
// A 32-k slice of a row is 32 bytes: loaded slice by slice, every load touches one cache line per row
// and uses a quarter of it, and the lines per load bounded the product.  So 128 k of a row are loaded at
// once, 16 consecutive k by each of 8 neighbouring lanes, and slice s of the four takes k = 4 s .. 4 s + 3
// of every lane's 16: any 32 k make a slice as long as both operands agree.  A thread holds such pieces
// of four rows, 32 apart.  Rows and k beyond B (a multiple of 64) are zero.
// EDGE: B is not a multiple of 128.
template <int TILE, bool EDGE>
struct CodesWide {
  static_assert(TILE == 128, "the passes of 32 rows lie inside or outside B as a whole");
  const uint8_t *c, *s;
  unsigned off_c, off_s;
  int64_t row_c, row_s;  // 32 rows
  u32x4 r[4];
  unsigned sc[4];
  int row, lane8, B, rows;  // rows: of the tile that exist
  __device__ __forceinline__ void init(const MxCodes& q, int64_t b, int r0, int B_, int tid) {
    row = tid >> 3;
    lane8 = tid & 7;
    B = B_;
    rows = B - r0;
    const int64_t at = b * q.rows + r0;
    c = q.codes + at * q.row_bytes;
    s = q.scales + at * q.row_groups;
    row_c = q.row_bytes * 32;
    row_s = q.row_groups * 32;
    off_c = (unsigned)row * (unsigned)q.row_bytes + 16 * lane8;
    off_s = (unsigned)row * (unsigned)q.row_groups + lane8 / 2;
  }
  __device__ __forceinline__ void load(int quad) {  // k = 128 quad .. 128 quad + 127
    auto piece = [&](int i) {
      r[i] = *(const u32x4*)(c + i * row_c + quad * 128 + off_c);
      sc[i] = (s + i * row_s + quad * 4)[off_s];
    };
    if (!EDGE || (rows >= TILE && 128 * quad + 128 <= B)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) piece(i);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r[i] = u32x4{};
        sc[i] = 0;
        if (32 * i < rows && 128 * quad + 16 * lane8 < B) piece(i);
      }
    }
  }
  template <int SLICE>
  __device__ __forceinline__ void store(__bf16* plane) const {
    typedef __bf16 v4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = scale_of(sc[i]);
      const bf16x2 lo = Pair<__bf16>::e4m3<0>(r[i][SLICE], f), hi = Pair<__bf16>::e4m3<1>(r[i][SLICE], f);
      *(v4*)&plane[kc_at(row + i * 32, lane8 >> 1) + 4 * (lane8 & 1)] = v4{lo[0], lo[1], hi[0], hi[1]};
    }
  }
};

// quads: of 128 k.  same: both operands are the same rows (B's plane is then A's)
template <int TILE, bool EDGE>
__device__ __forceinline__ void multiply_wide(CodesWide<TILE, EDGE>& la, CodesWide<TILE, EDGE>& lb, bool same, int quads,
                                              __bf16* stage0, __bf16* stage1, int wm, int wn, int lane,
                                              f32x16 (&acc)[Shape<TILE>::MTM][Shape<TILE>::MTN]) {
  constexpr int PLANE = TILE * BK;
  const int second = same ? 0 : PLANE;
  clear(acc);
  auto load = [&](int quad) {
    la.load(quad);
    if (!same) lb.load(quad);
  };
  auto store = [&](auto slice_c) {
    constexpr int slice = decltype(slice_c)::value;
    __bf16* st = slice & 1 ? stage1 : stage0;
    la.template store<slice>(st);
    if (!same) lb.template store<slice>(st + PLANE);
  };
  auto compute = [&](const __bf16* st) {
    multiply_slice<TILE, 1, 1, false, false>(st, st + second, wm, wn, lane, acc);
  };
  load(0);
  store(IC<0>{});
  __syncthreads();
  // each slice is multiplied while the next moves to the other stage; the next quad is loaded as soon as
  // the last slice has left the registers (a second set of them would cost the third workgroup per
  // compute unit, which hides more: 1.51 -> 1.35 ms for 384 tiles of 1024)
  for (int quad = 0; quad < quads; ++quad) {
    store(IC<1>{});
    compute(stage0);
    __syncthreads();
    store(IC<2>{});
    compute(stage1);
    __syncthreads();
    store(IC<3>{});
    if (quad + 1 < quads) load(quad + 1);
    compute(stage0);
    __syncthreads();
    if (quad + 1 < quads) store(IC<0>{});
    compute(stage1);
    __syncthreads();
  }
}

// ------------------------------------------------------------------------------------------------
// Statistics: L <- beta L + (1 - beta) Q Q^T from row codes, R from column codes (two problems)
// ------------------------------------------------------------------------------------------------

struct StatsArgs {
  GemmArgs g;
  MxCodes q[2];
};

// A <- beta A + (1 - beta) acc for the tile and its mirror, the arithmetic and the accesses of epilogue_split
// (32 x 32 sub-blocks; on a diagonal tile those below the diagonal store nothing and those on it their
// upper part and its mirror).  A wave's old values are all under way before its first store (each sub-block's
// loaded at its turn, 384 x 1024 1272 -> 1299 us in E4M3 and 918 -> 963 in E2M1).
template <int TILE, bool EDGE>
__device__ __forceinline__ void stats_epilogue(const StatsArgs& a, const TileCoord& tc, float* A,
                                               const f32x16 (&acc)[Shape<TILE>::MTM][Shape<TILE>::MTN], int wm, int wn,
                                               int lane, float* mlds) {
  constexpr int MTM = Shape<TILE>::MTM, MTN = Shape<TILE>::MTN, SUBS = MTM * MTN;
  // non-temporal: A passes through once (cached, 384 x 1024 1272 -> 1306 us in E4M3 and 918 -> 963 in E2M1,
  // 60 x 1600 716 -> 759 and 426 -> 486; but 20000 x 64 469 -> 267)
  constexpr int NT = 2;
  const int B = a.g.B;
  const float al = a.g.epi.alpha, be = a.g.epi.delta;
  const uint64_t at = (uint64_t)(A + tc.b * (int64_t)B * B);  // (the same in every lane: say so)
  const uint64_t base = ((uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(at >> 32)) << 32) |
                        (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)at);
  const __amdgpu_buffer_rsrc_t rs =
      __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, B * B * 4, BUFFER_RSRC_WORD3);
  const int li = lane & 31, h = lane >> 5;
  const int swm = __builtin_amdgcn_readfirstlane(wm), swn = __builtin_amdgcn_readfirstlane(wn);
  const int vlane = (4 * h * B + li) * 4;                   // lane part: row 4 h, column li
  const int vmir = ((lane >> 3) * B + 4 * (lane & 7)) * 4;  // mirror: row lane / 8, column 4 (lane % 8)
  const bool diag = tc.ti == tc.tj;
  auto row_of = [&](int t) { return (swm * MTM + t / MTN) * 32; };
  auto col_of = [&](int t) { return (swn * MTN + t % MTN) * 32; };
  // (sub-blocks lie inside or outside B as a whole)
  auto kept = [&](int t) {
    return !(diag && row_of(t) > col_of(t)) &&
           (!EDGE || (tc.ti * TILE + row_of(t) < B && tc.tj * TILE + col_of(t) < B));
  };
  float old[SUBS][16];
  auto load = [&](int t, float (&ev)[16]) {
    if (!kept(t)) return;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int i = tc.ti * TILE + row_of(t) + 8 * (r >> 2) + (r & 3);
      ev[r] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                            rs, vlane, (i * B + tc.tj * TILE + col_of(t)) * 4, NT));
    }
  };
#pragma unroll
  for (int t = 0; t < SUBS; ++t) load(t, old[t]);
#pragma unroll
  for (int t = 0; t < SUBS; ++t) {
    const int ib = row_of(t), jb = col_of(t);
    if (kept(t)) {
      const int row0 = tc.ti * TILE + ib, col0 = tc.tj * TILE + jb;
      const bool masked = row0 == col0;
      float v[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        v[r] = al * acc[t / MTN][t % MTN][r] + be * old[t][r];
        if (!masked || 8 * (r >> 2) + (r & 3) + 4 * h <= li)
          __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, v[r]), rs, vlane,
                                                ((row0 + 8 * (r >> 2) + (r & 3)) * B + col0) * 4, NT);
      }
      // the transposed sub-block through the wave's own LDS
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(f32x4*)&mlds[li * MLDS_PITCH + 8 * q + 4 * h] = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int rr = 8 * q + (lane >> 3), cc = 4 * (lane & 7);
        const f32x4 x = *(const f32x4*)&mlds[rr * MLDS_PITCH + cc];
        const int so = ((col0 + 8 * q) * B + row0) * 4;
        if (!masked) {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), rs, vmir, so, NT);
        } else {  // only the mirror's strict lower part
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float y = x[e];  // (a bit cast of a vector's element itself takes element 0)
            if (cc + e < rr)
              __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, y), rs, vmir + 4 * e, so, NT);
          }
        }
      }
    }
  }
}

// E4M3: 128-wide tiles, three workgroups to a compute unit: one's loads and stores of A run under the others'
// products.  (256-wide ones, one to a unit, took 1.50 ms where these take 1.37 at B = 1024, 394 us against
// 327 at 200 x 768, and 3 % less at B = 4096; with B an odd multiple of 64, 64-wide tiles took 6 % more at
// B = 192 and 86 % more at 1600.)  Both formats at B = 64: one 64-wide tile.
template <int F, int TILE, bool EDGE>
__global__ __launch_bounds__(2 * TILE, 3) void mx_stats_kernel(StatsArgs a) {
  constexpr int MTM = Shape<TILE>::MTM, MTN = Shape<TILE>::MTN, WAVES = TILE / 32;
  constexpr int STAGE = 2 * TILE * BK;
  __shared__ __attribute__((aligned(16))) __bf16 stage0[STAGE];
  __shared__ __attribute__((aligned(16))) __bf16 stage1[STAGE];
  const TileCoord tc = decode_tile(a.g, true);
  const MxCodes q = tc.prob ? a.q[1] : a.q[0];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / Shape<TILE>::WN, wn = wave % Shape<TILE>::WN;
  f32x16 acc[MTM][MTN];
  if constexpr (TILE == 128) {
    CodesWide<TILE, EDGE> la, lb;
    la.init(q, tc.b, tc.ti * TILE, a.g.B, tid);
    lb.init(q, tc.b, tc.tj * TILE, a.g.B, tid);
    multiply_wide(la, lb, tc.ti == tc.tj, (a.g.B + 127) / 128, stage0, stage1, wm, wn, lane, acc);
  } else {
    CodesK<F, TILE, 4, __bf16> la, lb;
    la.init(q, tc.b, tc.ti * TILE, tid);
    lb.init(q, tc.b, tc.tj * TILE, tid);
    multiply<TILE>(la, lb, a.g.B / BK, a.g.B / BK, stage0, stage1, wm, wn, lane, acc);
  }
  constexpr int PER = WAVES / 2 * MLDS_FLOATS * 4;
  static_assert(PER <= STAGE * 2, "LDS for the mirror");
  float* mlds = (float*)(wave < WAVES / 2 ? (void*)stage0 : (void*)stage1) + (wave % (WAVES / 2)) * MLDS_FLOATS;
  stats_epilogue<TILE, EDGE>(a, tc, (float*)(tc.prob ? a.g.p1.D : a.g.p0.D), acc, wm, wn, lane, mlds);
}

// ------------------------------------------------------------------------------------------------
// E2M1 statistics: the scaled 4-bit MFMA
// ------------------------------------------------------------------------------------------------
//
// The 32x32x64 scaled MFMA multiplies E2M1 codes as they are stored, at four times the bfloat16 rate: lane l
// takes row l % 32, k = 32 (l / 32) .. + 31, one scale group, and its scale byte.  Products of two E2M1
// values are whole quarters up to 36, so its sum of a group is exact; the sums across groups are fp32's
// (against 64 bits as near as the bfloat16 kernel's).  Stages hold codes, 128 k of a row in its 64
// bytes, laid out like 32 bfloat16 k; a thread loads one group of a row and its scale.  Three workgroups
// of 128-wide tiles to a compute unit (four, in 128 registers, took 1.24 ms where these take 1.06 at
// B = 1024).  Against the bfloat16 kernel on the same codes: B = 1024 1450 -> 1062 us (4.96 TB/s), 2048 1140
// -> 717, 4096 915 -> 574, 256 593 -> 588; at B = 64 49 -> 53, so that stays with the bfloat16 one.
template <bool EDGE>
struct Codes4 {
  static constexpr int TILE = 128;
  const uint8_t *c, *s;
  unsigned off_c, off_s;
  int64_t row_c, row_s;  // TILE / 2 rows
  u32x4 r[2];
  unsigned sc[2];
  int row, group, B, rows;
  __device__ __forceinline__ void init(const MxCodes& q, int64_t b, int r0, int B_, int tid) {
    row = tid >> 2;
    group = tid & 3;
    B = B_;
    rows = B - r0;
    const int64_t at = b * q.rows + r0;
    c = q.codes + at * q.row_bytes;
    s = q.scales + at * q.row_groups;
    row_c = q.row_bytes * (TILE / 2);
    row_s = q.row_groups * (TILE / 2);
    off_c = (unsigned)row * (unsigned)q.row_bytes + 16 * group;
    off_s = (unsigned)row * (unsigned)q.row_groups + group;
  }
  __device__ __forceinline__ void load(int slice) {  // k = 128 slice .. 128 slice + 127
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (EDGE) {
        r[i] = u32x4{};
        sc[i] = 0;
        if (row + i * (TILE / 2) >= rows || 128 * slice + 32 * group >= B) continue;
      }
      r[i] = *(const u32x4*)(c + i * row_c + slice * 64 + off_c);
      sc[i] = (s + i * row_s + slice * 4)[off_s];
    }
  }
  __device__ __forceinline__ void store(__bf16* plane, uint8_t* scales) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      *(u32x4*)&plane[kc_at(row + i * (TILE / 2), group)] = r[i];
      scales[4 * (row + i * (TILE / 2)) + group] = (uint8_t)sc[i];
    }
  }
};

template <bool EDGE>
__global__ __launch_bounds__(256, 3) void mx_stats4_kernel(StatsArgs a) {
  constexpr int TILE = 128;
  constexpr int MTM = Shape<TILE>::MTM, MTN = Shape<TILE>::MTN, WAVES = TILE / 32;
  constexpr int PLANE = TILE * BK, STAGE = 2 * PLANE;
  typedef int v8i __attribute__((ext_vector_type(8)));
  __shared__ __attribute__((aligned(16))) __bf16 stage[2][STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t scale[2][2][4 * TILE];
  const TileCoord tc = decode_tile(a.g, true);
  const MxCodes q = tc.prob ? a.q[1] : a.q[0];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / Shape<TILE>::WN, wn = wave % Shape<TILE>::WN;
  const bool same = tc.ti == tc.tj;
  const int sb = same ? 0 : 1;  // B's plane
  Codes4<EDGE> la, lb;
  la.init(q, tc.b, tc.ti * TILE, a.g.B, tid);
  lb.init(q, tc.b, tc.tj * TILE, a.g.B, tid);
  f32x16 acc[MTM][MTN];
  clear(acc);
  auto load = [&](int slice) {
    la.load(slice);
    if (!same) lb.load(slice);
  };
  auto store = [&](int to) {
    la.store(stage[to], scale[to][0]);
    if (!same) lb.store(stage[to] + PLANE, scale[to][1]);
  };
  auto operand = [&](const __bf16* plane, int base, int ks) {
    const u32x4 x = *(const u32x4*)&plane[kc_at(base + (lane & 31), 2 * ks + (lane >> 5))];
    return v8i{(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
  };
  // the row's four scale bytes, moved so that byte 2 ks is the lane's
  auto scales = [&](const uint8_t* s, int base) {
    return (int)(*(const unsigned*)&s[4 * (base + (lane & 31))] >> (8 * (lane >> 5)));
  };
  auto compute = [&](int from) {
    const __bf16 *pa = stage[from], *pb = stage[from] + sb * PLANE;
    int xa[MTM], xb[MTN];
#pragma unroll
    for (int mt = 0; mt < MTM; ++mt) xa[mt] = scales(scale[from][0], (wm * MTM + mt) * 32);
#pragma unroll
    for (int nt = 0; nt < MTN; ++nt) xb[nt] = scales(scale[from][sb], (wn * MTN + nt) * 32);
    constexpr int FP4 = 4;
#pragma unroll
    for (int mt = 0; mt < MTM; ++mt)
#pragma unroll
      for (int nt = 0; nt < MTN; ++nt)
        acc[mt][nt] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            operand(pa, (wm * MTM + mt) * 32, 0), operand(pb, (wn * MTN + nt) * 32, 0), acc[mt][nt], FP4, FP4, 0, xa[mt],
            0, xb[nt]);
#pragma unroll
    for (int mt = 0; mt < MTM; ++mt)
#pragma unroll
      for (int nt = 0; nt < MTN; ++nt)
        acc[mt][nt] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            operand(pa, (wm * MTM + mt) * 32, 1), operand(pb, (wn * MTN + nt) * 32, 1), acc[mt][nt], FP4, FP4, 2, xa[mt],
            2, xb[nt]);
  };
  const int slices = (a.g.B + 127) / 128;
  load(0);
  store(0);
  if (slices > 1) load(1);
  __syncthreads();
  for (int k = 0; k < slices; ++k) {
    if (k + 1 < slices) store((k + 1) & 1);
    if (k + 2 < slices) load(k + 2);
    compute(k & 1);
    __syncthreads();
  }
  static_assert(WAVES / 2 * MLDS_FLOATS * 4 <= STAGE * 2, "LDS for the mirror");
  float* mlds = (float*)stage[wave < WAVES / 2 ? 0 : 1] + (wave % (WAVES / 2)) * MLDS_FLOATS;
  stats_epilogue<TILE, EDGE>(a, tc, (float*)(tc.prob ? a.g.p1.D : a.g.p0.D), acc, wm, wn, lane, mlds);
}

template <int TILE, typename K>
hipError_t launch_stats(K kernel, StatsArgs& a, hipStream_t stream) {
  a.g.tdim = (a.g.B + TILE - 1) / TILE;
  a.g.tiles = a.g.tdim * (a.g.tdim + 1) / 2;
  const int64_t grid = 2 * a.g.N * a.g.tiles;
  if (grid > most_workgroups(2 * TILE)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(2 * TILE), 0, stream, a);
  return hipGetLastError();
}

// ------------------------------------------------------------------------------------------------
// Update: T = XL G and U = T XR^T, each with the root's diagonal added in fp32
// ------------------------------------------------------------------------------------------------
//
// The floating operand is brought to binary16's upper range by a power of two per block (2^13 <= 2^e
// max|x| < 2^14) and cut into two binary16 pieces, which hold 22 of its 24 significant bits (see
// gemm_split.hip); the root's elements are binary16 numbers under a power of two per block (the largest
// scale's elements below 2^14; elements 2^-38 of the block's largest lose bits to binary16's
// subnormals).  Two matrix passes per product, where bfloat16 pieces would take three.

struct ApplyArgs {
  GemmArgs g;  // N, B and the tile map only
  MxCodes q;
  MxFloats x;
  const float* diag;      // [N, B] or null: + diag[i] x[i][j] (LEFT) or + x[i][j] diag[j]
  float* out;
  const float* amax;      // [N, parts]: bounds of x's finite magnitudes
  int parts;
  const unsigned* bytes;  // [N, byte_parts]: the largest scale byte short of 255 of XL and (<< 8) of XR
  int byte_parts;
  float* amax_out;        // LEFT: [N, tiles, waves]: the largest finite |out| each wave stored
};

// Bounds of a block are taken over its finite elements: an Inf (or a row of XL G beyond fp32) would leave no
// scale to the others, which meet it in no sum.  `scan` folds a function over some elements; the plain
// maximum (NaN passed over) is theirs unless it is Inf, and only then a second scan leaves the infinities
// out (tested per element in the first, 2 x 128 15.7 -> 17.1 us, 20 x 960 249 -> 257).
template <typename S>
__device__ __forceinline__ float finite_max(S scan) {
  const float inf = __builtin_inff();
  float m = scan([](float m, float x) { return fmaxf(m, fabsf(x)); });
  if (m == inf) m = scan([=](float m, float x) { return fabsf(x) < inf ? fmaxf(m, fabsf(x)) : m; });
  return m;
}

// The largest v and c over a workgroup's threads, in all of them
template <int WAVES>
__device__ __forceinline__ void block_max(float& v, unsigned& c) {
  __shared__ float vs[WAVES];
  __shared__ unsigned cs[WAVES];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const unsigned x = __shfl_xor(c, o, 64);
    v = fmaxf(v, __shfl_xor(v, o, 64));
    c = x > c ? x : c;
  }
  if ((threadIdx.x & 63) == 0) {
    vs[threadIdx.x >> 6] = v;
    cs[threadIdx.x >> 6] = c;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    v = fmaxf(v, vs[w]);
    c = cs[w] > c ? cs[w] : c;
  }
}

// LEFT: out = Q X (Q's rows, X's columns); else out = X Q^T (X's rows, Q's rows as columns).  OWN: no launch
// went before for the bounds; each workgroup takes G's (LEFT) and the root's scale bytes' from the block
// itself
template <int F, int TILE, bool LEFT, bool OWN>
__global__ __launch_bounds__(2 * TILE) void mx_apply_kernel(ApplyArgs a) {
  constexpr int MTM = Shape<TILE>::MTM, MTN = Shape<TILE>::MTN, WAVES = TILE / 32;
  constexpr int STAGE = 3 * TILE * BK;
  __shared__ __attribute__((aligned(16))) _Float16 stage0[STAGE];
  __shared__ __attribute__((aligned(16))) _Float16 stage1[STAGE];
  const TileCoord tc = decode_tile(a.g, false);
  const int B = a.g.B;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / Shape<TILE>::WN, wn = wave % Shape<TILE>::WN;
  float m = 0.f;
  unsigned top = 0;
  if (!(OWN && LEFT))
    for (int p = lane; p < a.parts; p += 64) m = fmaxf(m, a.amax[tc.b * a.parts + p]);
  if constexpr (OWN) {
    const int n = B * B;
    if (LEFT) {
      const f32x4* g = (const f32x4*)((const float*)a.x.p + tc.b * n);
      m = finite_max([&](auto f) {
        float s = 0.f;
#pragma unroll 4
        for (int i = tid; i < n / 4; i += 2 * TILE) {
          const f32x4 v = g[i];
          s = f(f(f(f(s, v[0]), v[1]), v[2]), v[3]);
        }
        return s;
      });
    }
    for (int i = tid; i < n / MX_GROUP; i += 2 * TILE) {
      const unsigned c = a.q.scales[tc.b * (n / MX_GROUP) + i];
      top = c != 255u && c > top ? c : top;
    }
    block_max<WAVES>(m, top);
  } else {
    for (int p = lane; p < a.byte_parts; p += 64) {
      const unsigned v = a.bytes[tc.b * a.byte_parts + p];
      const unsigned c = LEFT ? v & 255u : v >> 8;
      top = c > top ? c : top;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const unsigned c = __shfl_xor(top, o, 64);
      m = fmaxf(m, __shfl_xor(m, o, 64));
      top = c > top ? c : top;
    }
  }
  const int ex = __builtin_amdgcn_readfirstlane(top_exp(m));
  const int shift = __builtin_amdgcn_readfirstlane(127 + Elem<F>::TOP - (int)top);
  float m1 = -1.f;
  asm("" : "+s"(m1));  // (no instruction: hides the constant -1 from the optimiser)
  const int whole = (tc.ti + 1) * TILE <= B && (tc.tj + 1) * TILE <= B ? B / BK : 0;
  f32x16 acc[MTM][MTN];
  CodesK<F, TILE, 2, _Float16> lq;
  lq.init(a.q, tc.b, (LEFT ? tc.ti : tc.tj) * TILE, tid, shift);
  if constexpr (LEFT) {
    FloatCol16<TILE> lx;
    lx.init(a.x, tc.b, tc.tj * TILE, tid, ex, m1);
    multiply<TILE>(lq, lx, B / BK, whole, stage0, stage1, wm, wn, lane, acc);
  } else {
    FloatK<TILE> lx;
    lx.init(a.x, tc.b, tc.ti * TILE, tid, ex, m1);
    multiply<TILE>(lx, lq, B / BK, whole, stage0, stage1, wm, wn, lane, acc);
  }
  const int64_t off = tc.b * (int64_t)B * B;
  const float* x = (const float*)a.x.p + off;
  const float* dg = a.diag ? a.diag + tc.b * B : nullptr;
  float* out = a.out + off;
  const int es = -ex - shift;
  float most = 0.f;
#pragma unroll
  for (int mt = 0; mt < MTM; ++mt)
#pragma unroll
    for (int nt = 0; nt < MTN; ++nt) {
      // (sub-blocks lie inside or outside B as a whole)
      if (tc.ti * TILE + (wm * MTM + mt) * 32 >= B || tc.tj * TILE + (wn * MTN + nt) * 32 >= B) continue;
      const int i0 = tc.ti * TILE + (wm * MTM + mt) * 32 + 4 * (lane >> 5);
      const int j = tc.tj * TILE + (wn * MTN + nt) * 32 + (lane & 31);
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[mt][nt][r] = ldexpf(acc[mt][nt][r], es);
      // (all loads of a sub-block before its stores)
      if (dg) {
        float xv[16], dv[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int i = i0 + 8 * (r >> 2) + (r & 3);
          xv[r] = x[i * B + j];
          dv[r] = dg[LEFT ? i : j];
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[mt][nt][r] += xv[r] * dv[r];
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) out[(i0 + 8 * (r >> 2) + (r & 3)) * B + j] = acc[mt][nt][r];
      if (LEFT) most = fmaxf(most, finite_max([&](auto f) {
                               float s = 0.f;
#pragma unroll
                               for (int r = 0; r < 16; ++r) s = f(s, acc[mt][nt][r]);
                               return s;
                             }));
    }
  if (LEFT) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor(most, o, 64));
    if (lane == 0) a.amax_out[(tc.b * a.g.tiles + tc.ti * a.g.tdim + tc.tj) * WAVES + wave] = most;
  }
}

// Bounds of a block in `parts` pieces: max|G| over its finite elements, and both roots' largest scale bytes
__global__ __launch_bounds__(256) void mx_bounds_kernel(const float* G, const uint8_t* sl, const uint8_t* sr, int B,
                                                        int parts, float* amax, unsigned* bytes) {
  const int64_t b = blockIdx.x / parts;
  const int p = (int)(blockIdx.x - b * parts);
  const int64_t n = (int64_t)B * B / parts, ns = (int64_t)B * B / MX_GROUP / parts;
  const f32x4* g = (const f32x4*)(G + b * B * B + p * n);
  float m = finite_max([&](auto f) {
    float s = 0.f;
#pragma unroll 8
    for (int i = threadIdx.x; i < n / 4; i += 256) {
      const f32x4 v = g[i];
      s = f(f(f(f(s, v[0]), v[1]), v[2]), v[3]);
    }
    return s;
  });
  const int64_t s0 = b * B * B / MX_GROUP + p * ns;
  unsigned l = 0, r = 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < ns; i += 256) {
    const unsigned x = sl[s0 + i], y = sr[s0 + i];
    l = x != 255u && x > l ? x : l;
    r = y != 255u && y > r ? y : r;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const unsigned x = __shfl_xor(l, o, 64), y = __shfl_xor(r, o, 64);
    m = fmaxf(m, __shfl_xor(m, o, 64));
    l = x > l ? x : l;
    r = y > r ? y : r;
  }
  __shared__ float ms[4];
  __shared__ unsigned bs[4];
  if ((threadIdx.x & 63) == 0) {
    ms[threadIdx.x >> 6] = m;
    bs[threadIdx.x >> 6] = l | r << 8;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 4; ++w) {
      m = fmaxf(m, ms[w]);
      l = (bs[w] & 255u) > l ? bs[w] & 255u : l;
      r = (bs[w] >> 8) > r ? bs[w] >> 8 : r;
    }
    amax[blockIdx.x] = m;
    bytes[blockIdx.x] = l | r << 8;
  }
}

template <int F, int TILE, bool OWN>
hipError_t launch_apply_tile(ApplyArgs& a, const MxApply& p, hipStream_t stream) {
  a.g.tdim = (p.B + TILE - 1) / TILE;
  a.g.tiles = a.g.tdim * a.g.tdim;
  const int64_t grid = p.N * a.g.tiles;
  if (grid > most_workgroups(2 * TILE)) return hipErrorInvalidConfiguration;
  a.q = p.xl;
  a.diag = p.xl_diag;
  a.x.p = p.G;
  a.out = p.T;
  a.amax = p.amax_g;
  a.parts = p.parts;
  a.amax_out = p.amax_t;
  hipLaunchKernelGGL((mx_apply_kernel<F, TILE, true, OWN>), dim3((unsigned)grid), dim3(2 * TILE), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  a.q = p.xr;
  a.diag = p.xr_diag;
  a.x.p = p.T;
  a.out = p.U;
  a.amax = p.amax_t;
  a.parts = a.g.tiles * (TILE / 32);
  hipLaunchKernelGGL((mx_apply_kernel<F, TILE, false, OWN>), dim3((unsigned)grid), dim3(2 * TILE), 0, stream, a);
  return hipGetLastError();
}

// The tile with the least predicted time.  Measured with tiles of 64 / 128 / 256 (both products and the
// bounds, us): 2 x 128 24 / 26 / 33, 30 x 704 200 / 187 / 219, 16 x 1024 295 / 195 / 175, 100 x 1088
// 2137 / 1739 / 1622, 384 x 1024 6831 / 5028 / 4275; the rates are fitted to 22 such shapes, B 64 .. 3136.
constexpr TileRate APPLY_RATES[3] = {{64, 0.9, 0.28, 4}, {128, 1.0, 0.8, 2}, {256, 1.85, 2.5, 1}};
int apply_tile(int64_t N, int B) {
  int best = 64;
  double least = INFINITY;
  for (const TileRate& r : APPLY_RATES) {
    const double side = (B + r.tile - 1) / r.tile, t = slice_time(r, (double)N * side * side);
    if (t < least) {
      least = t;
      best = r.tile;
    }
  }
  return best;
}

// Up to this B a block is 64 KiB or less, and its workgroups find the bounds themselves: with / without a
// launch for them, 2 x 128 22 / 19 us, 3000 x 128 258 / 240, 20000 x 64 403 / 357; but 1000 x 192 257 / 323.
constexpr int APPLY_OWN_BOUNDS = 128;

template <int F>
hipError_t launch_apply_fmt(ApplyArgs& a, const MxApply& p, hipStream_t stream) {
  const int tile = apply_tile(p.N, p.B);
  if (p.B <= APPLY_OWN_BOUNDS)  // (a 256-wide tile is never the cheapest there)
    return tile > 64 ? launch_apply_tile<F, 128, true>(a, p, stream) : launch_apply_tile<F, 64, true>(a, p, stream);
  return tile == 256   ? launch_apply_tile<F, 256, false>(a, p, stream)
         : tile == 128 ? launch_apply_tile<F, 128, false>(a, p, stream)
                       : launch_apply_tile<F, 64, false>(a, p, stream);
}

// ------------------------------------------------------------------------------------------------
// Gradient tiles: G = dY^T Q, dY [T, out], Q [T, in], in the order of launch_tile_copy
// ------------------------------------------------------------------------------------------------

struct GradArgs {
  MxFloats dy;      // ld, cols = out
  MxCodes q;        // rows = T
  int64_t T, out, in;
  int B;            // tiles of the stack
  int64_t tr, tc;   // tile rows and columns of the stack
  int64_t gm, gn;   // kernel tiles along out and in
  int splits;       // of the token axis
  int64_t chunk;    // tokens per split, a multiple of BK
  int accumulate;
  float* G;
  float* part;      // [splits, gm TILE, gn TILE] when splits > 1
};

template <typename T, int F, int TILE>
__global__ __launch_bounds__(2 * TILE) void mx_grad_kernel(GradArgs a) {
  constexpr int MTM = Shape<TILE>::MTM, MTN = Shape<TILE>::MTN;
  constexpr int STAGE = (Pieces<T>::N + 1) * TILE * BK;
  __shared__ __attribute__((aligned(16))) __bf16 stage0[STAGE];
  __shared__ __attribute__((aligned(16))) __bf16 stage1[STAGE];
  const int64_t lid = xcd_remap(blockIdx.x, gridDim.x);
  const int64_t tiles = a.gm * a.gn;
  const int split = (int)(lid / tiles);
  const int64_t rem = lid - split * tiles;
  const int64_t ti = rem / a.gn, tj = rem - ti * a.gn;
  const int64_t i0 = ti * TILE, j0 = tj * TILE;
  const int64_t k0 = split * a.chunk, k1 = k0 + a.chunk < a.T ? k0 + a.chunk : a.T;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / Shape<TILE>::WN, wn = wave % Shape<TILE>::WN;
  f32x16 acc[MTM][MTN];
  constexpr int D = sizeof(T) == 4 && TILE == 256 ? 2 : 4;
  FloatCol<T, TILE, D, false> la;
  CodesCol<F, TILE, D> lb;
  la.init(a.dy, 0, i0, k0, k1, tid);
  lb.init(a.q, j0, k0, k1, tid);
  // a tile of padding alone has no products
  const int64_t slices = i0 < a.out && j0 < a.in ? (k1 - k0 + BK - 1) / BK : 0;
  const bool inside = a.dy.vec && i0 + TILE <= a.out && j0 + TILE <= a.q.row_groups * 32;
  const int64_t whole = inside ? (k1 - k0) / BK : 0;
  multiply<TILE>(la, lb, slices, whole, stage0, stage1, wm, wn, lane, acc);
  if constexpr (Pieces<T>::N > 1) {
    // Infinities among the pieces' products have left NaN: a tile with a NaN is formed once more, slice by
    // slice, in pieces that mind them.  (Minded at once, 16384 x 2048 x 8192 took 6 % more in binary16 and 5 %
    // in fp32; this test takes 2 % of 50000 x 520 x 264 in fp32 and up to 1.4 % elsewhere, a call full of NaN
    // 2.3 times as long.  The pipelined loop again in its place cost the first loop registers: 3 %.)
    float sum[4] = {0.f, 0.f, 0.f, 0.f};  // NaN if an addend is (or from Inf - Inf)
#pragma unroll
    for (int mt = 0; mt < MTM; ++mt)
#pragma unroll
      for (int nt = 0; nt < MTN; ++nt)
#pragma unroll
        for (int r = 0; r < 16; ++r) sum[r & 3] += acc[mt][nt][r];
    const float all = sum[0] + sum[1] + (sum[2] + sum[3]);
    if (__syncthreads_or(all != all)) {
      FloatCol<T, TILE, D, true> li;
      li.init(a.dy, 0, i0, k0, k1, tid);
      lb.init(a.q, j0, k0, k1, tid);
      clear(acc);
      for (int64_t kt = 0; kt < slices; ++kt) {
        li.template load<0, true>(kt);
        lb.template load<0, true>(kt);
        li.template store<0>(stage0);
        lb.template store<0>(stage0 + Pieces<T>::N * TILE * BK);
        __syncthreads();
        multiply_slice<TILE, Pieces<T>::N, 1, true, true>(stage0, stage0 + Pieces<T>::N * TILE * BK, wm, wn, lane, acc);
        __syncthreads();
      }
    }
  }
#pragma unroll
  for (int mt = 0; mt < MTM; ++mt)
#pragma unroll
    for (int nt = 0; nt < MTN; ++nt) {
      // a 32 x 32 sub-block lies in one tile of the stack (B is a multiple of 64)
      const int64_t is = i0 + (wm * MTM + mt) * 32, js = j0 + (wn * MTN + nt) * 32;
      if (is >= a.tr * a.B || js >= a.tc * a.B) continue;
      const int64_t j = js + (lane & 31);
      float* base;
      int64_t ld;
      if (a.splits > 1) {
        ld = a.gn * TILE;
        base = a.part + (split * a.gm * TILE + is) * ld + j;
      } else {
        ld = a.B;
        const int64_t t = is / a.B * a.tc + js / a.B;
        base = a.G + (t * a.B + is % a.B) * a.B + j % a.B;
      }
      auto row = [&](int r) { return 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3); };
      float v[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) v[r] = is + row(r) < a.out && j < a.in ? acc[mt][nt][r] : 0.f;
      if (a.splits == 1 && a.accumulate) {  // (all loads of a sub-block before its stores)
        float old[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) old[r] = base[row(r) * ld];
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] += old[r];
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) base[row(r) * ld] = v[r];
    }
}

// The splits' partial sums added in order, into the stack's tiles; one thread per 4 columns.
__global__ __launch_bounds__(256) void mx_grad_join_kernel(GradArgs a, int64_t pm, int64_t pn) {
  const int64_t quads = a.tc * a.B / 4;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= a.tr * a.B * quads) return;
  const int64_t i = e / quads, j = 4 * (e - i * quads);
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (i < a.out && j < a.in) {
    const float* p = a.part + i * pn + j;
    const int64_t step = pm * pn;
    int s = 0;
    for (; s + 8 <= a.splits; s += 8) {  // (eight loads under way at a time)
      f32x4 x[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = *(const f32x4*)(p + (s + q) * step);
#pragma unroll
      for (int q = 0; q < 8; ++q) v += x[q];
    }
    for (; s < a.splits; ++s) v += *(const f32x4*)(p + s * step);
  }
  const int64_t t = i / a.B * a.tc + j / a.B;
  f32x4* at = (f32x4*)(a.G + (t * a.B + i % a.B) * a.B + j % a.B);
  *at = a.accumulate ? *at + v : v;
}

// The launch's shape: kernel tile, tiles, and splits of the token axis so that few tiles still fill the
// chip, joined by a second launch: the pair with the least predicted time.  Measured with the best
// split for tiles of 64 / 128 / 256 (us, E4M3, bfloat16 dY unless said): 1 x 256 x 192 (tokens x out x in)
// 9 / 10 / 13, 2048 x 1024 x 1024 21 / 25 / 34, 65536 x 256 x 256 32 / 27 / 50, 4096 x 2048 x 2048 68 / 50 /
// 59, 50000 x 520 x 264 fp32 138 / 103 / 139, 4096 x 2048 x 8192 294 / 166 / 129.  The rates (each further
// piece of dY adds half of one; 1.4 slices to start and end; a join 3.2 us and 1.2 per 10^6 partial sums)
// are fitted to 20 such shapes, over which the choice is 2 % from the best on average.
constexpr TileRate GRAD_RATES[3] = {{64, 0.19, 0.17, 4}, {128, 0.47, 0.365, 2}, {256, 1.15, 1.15, 1}};
struct GradShape {
  int tile = 64;
  int64_t gm = 1, gn = 1, chunk = 0;
  int splits = 1;
};
GradShape grad_shape(int64_t T, int64_t out, int64_t in, dash_prec type) {
  const int pieces = type == DASH_FP32 ? 3 : type == DASH_FP16 ? 2 : 1;
  GradShape best;
  double least = INFINITY;
  for (const TileRate& r : GRAD_RATES) {
    const int64_t gm = (out + r.tile - 1) / r.tile, gn = (in + r.tile - 1) / r.tile, tiles = gm * gn;
    for (int round = 0; round <= 2 * r.cap; ++round) {  // one split, or splits that fill `round` per unit
      int64_t s = round == 0 ? 1 : 256 * round / tiles;
      if (s > (T + 2 * BK - 1) / (2 * BK)) s = (T + 2 * BK - 1) / (2 * BK);
      if (s < 1 || (round > 0 && s == 1)) s = 1;
      const int64_t chunk = ((T + s - 1) / s + BK - 1) / BK * BK;
      const int splits = chunk ? (int)((T + chunk - 1) / chunk) : 1;
      double t = (chunk / BK + 1.4) * (1 + 0.5 * (pieces - 1)) * slice_time(r, (double)tiles * splits);
      if (splits > 1) t += 3.2 + 1.2e-6 * (double)tiles * r.tile * r.tile * splits;
      if (t < least) {
        least = t;
        best.tile = r.tile;
        best.gm = gm;
        best.gn = gn;
        best.chunk = chunk;
        best.splits = splits;
      }
    }
  }
  return best;
}

template <typename T, int F, int TILE>
hipError_t launch_grad_one(GradArgs& a, const GradShape& g, hipStream_t stream) {
  // one split: the launch also writes the padding of the stack's edge tiles
  if (g.splits == 1) {
    a.gm = (a.tr * a.B + TILE - 1) / TILE;
    a.gn = (a.tc * a.B + TILE - 1) / TILE;
  } else {
    a.gm = g.gm;
    a.gn = g.gn;
  }
  const int64_t grid = a.gm * a.gn * g.splits;
  if (grid > most_workgroups(2 * TILE)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((mx_grad_kernel<T, F, TILE>), dim3((unsigned)grid), dim3(2 * TILE), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || g.splits == 1) return e;
  const int64_t joins = (a.tr * a.B * (a.tc * a.B / 4) + 255) / 256;
  if (joins > most_workgroups(256)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(mx_grad_join_kernel, dim3((unsigned)joins), dim3(256), 0, stream, a, g.gm * TILE, g.gn * TILE);
  return hipGetLastError();
}

template <typename T, int F>
hipError_t launch_grad_tile(GradArgs& a, const GradShape& g, hipStream_t stream) {
  if (g.tile == 256) return launch_grad_one<T, F, 256>(a, g, stream);
  if (g.tile == 128) return launch_grad_one<T, F, 128>(a, g, stream);
  return launch_grad_one<T, F, 64>(a, g, stream);
}

template <typename T>
hipError_t launch_grad_fmt(GradArgs& a, const GradShape& g, dash_mx_fmt fmt, hipStream_t stream) {
  return fmt == DASH_MX_E4M3 ? launch_grad_tile<T, DASH_MX_E4M3>(a, g, stream)
                             : launch_grad_tile<T, DASH_MX_E2M1>(a, g, stream);
}

}  // namespace
}  // namespace gemm

using namespace gemm;

hipError_t launch_mx_stats(const MxCodes& rows, const MxCodes& cols, int64_t NG, int B, dash_mx_fmt fmt, float beta,
                           float* A, hipStream_t stream) {
  StatsArgs a;
  a.g.N = NG;
  a.g.B = B;
  a.g.nprob = 2;
  a.g.epi.alpha = 1.f - beta;
  a.g.epi.delta = beta;
  a.g.p0.D = A;
  a.g.p1.D = A + NG * (int64_t)B * B;
  a.q[0] = rows;
  a.q[1] = cols;
  const bool edge = B % 128 != 0;
  if (fmt == DASH_MX_E4M3)
    return B == 64 ? launch_stats<64>(mx_stats_kernel<DASH_MX_E4M3, 64, false>, a, stream)
           : edge  ? launch_stats<128>(mx_stats_kernel<DASH_MX_E4M3, 128, true>, a, stream)
                   : launch_stats<128>(mx_stats_kernel<DASH_MX_E4M3, 128, false>, a, stream);
  return B == 64 ? launch_stats<64>(mx_stats_kernel<DASH_MX_E2M1, 64, false>, a, stream)
         : edge  ? launch_stats<128>(mx_stats4_kernel<true>, a, stream)
                 : launch_stats<128>(mx_stats4_kernel<false>, a, stream);
}

hipError_t launch_mx_apply(const MxApply& p, dash_mx_fmt fmt, hipStream_t stream) {
  if (p.B > APPLY_OWN_BOUNDS) {
    const int64_t grid = p.N * p.parts;
    if (grid > most_workgroups(256)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(mx_bounds_kernel, dim3((unsigned)grid), dim3(256), 0, stream, p.G, p.xl.scales, p.xr.scales,
                       p.B, p.parts, p.amax_g, p.bytes);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  ApplyArgs a;
  a.g.N = p.N;
  a.g.B = p.B;
  a.g.nprob = 1;
  a.x.ld = p.B;
  a.x.stride = (int64_t)p.B * p.B;
  a.x.cols = p.B;
  a.bytes = p.bytes;
  a.byte_parts = p.parts;
  return fmt == DASH_MX_E4M3 ? launch_apply_fmt<DASH_MX_E4M3>(a, p, stream)
                             : launch_apply_fmt<DASH_MX_E2M1>(a, p, stream);
}

size_t mx_grad_workspace_bytes(int64_t T, int64_t out, int64_t in, dash_prec type) {
  const GradShape g = grad_shape(T, out, in, type);
  return g.splits > 1 ? (size_t)g.splits * g.gm * g.gn * g.tile * g.tile * sizeof(float) : 0;
}

hipError_t launch_mx_grad(const void* dY, dash_prec type, int64_t ldy, const MxCodes& q, dash_mx_fmt fmt, int64_t T,
                          int64_t out, int64_t in, int B, bool accumulate, float* G, void* ws, hipStream_t stream) {
  const GradShape g = grad_shape(T, out, in, type);
  GradArgs a;
  a.dy.p = dY;
  a.dy.ld = ldy;
  a.dy.stride = 0;
  a.dy.cols = out;
  a.dy.vec = ((uintptr_t)dY & 15) == 0 && (T <= 1 || ldy * (type == DASH_FP32 ? 4 : 2) % 16 == 0);
  a.q = q;
  a.T = T;
  a.out = out;
  a.in = in;
  a.B = B;
  a.tr = (out + B - 1) / B;
  a.tc = (in + B - 1) / B;
  a.splits = g.splits;
  a.chunk = g.chunk;
  a.accumulate = accumulate;
  a.G = G;
  a.part = (float*)ws;
  if (type == DASH_FP32) return launch_grad_fmt<float>(a, g, fmt, stream);
  if (type == DASH_BF16) return launch_grad_fmt<__bf16>(a, g, fmt, stream);
  return launch_grad_fmt<_Float16>(a, g, fmt, stream);
}

}  // namespace dash
