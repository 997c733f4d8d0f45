// Pieces of rows in memory and the row quantizer, shared by the row-wise
// operators (rows.hip) and the product that quantizes its own rows (int8.hip).
// The quantizer's results are compared bit for bit: sources that include this
// must not have products and sums fused behind their back in it.
#pragma once

#include "common.h"

namespace qlora {
namespace {

constexpr float kAmaxFloor = 1e-30f;

// A launch has fewer than 2^32 threads in a dimension: workgroups (of up to
// 1024 threads) past kGridX go on in the second one, whose last line is filled
// up with workgroups that have nothing to do.
constexpr int64_t kGridX = 1 << 21;
inline dim3 grid_of(int64_t blocks) {
  return dim3((uint32_t)(blocks < kGridX ? blocks : kGridX), (uint32_t)((blocks + kGridX - 1) / kGridX));
}
__device__ __forceinline__ int64_t block_of(uint32_t x, uint32_t y) { return (int64_t)y * kGridX + x; }

// One fp32 of a 16- or 32-bit element type.
struct F32 {};
template <typename T> struct Elem { typedef uint16_t type; };
template <> struct Elem<F32> { typedef float type; };

// 16 bytes at any element's address: rows that are not 16-byte aligned (an odd
// width, a slice of a wider matrix) are still loaded and stored 16 bytes at a
// time, which the hardware takes at any alignment; only a row's end goes
// in smaller parts.  777 x 2500 in fp16, norm forward and backward: 24 us, and
// 54 us with such rows loaded element by element.
struct __attribute__((packed, aligned(2))) Bytes16 {
  uint32_t x, y, z, w;
};

// A row-major input whose rows are `ld` elements apart.
template <typename T>
struct Mat {
  typedef typename Elem<T>::type E;
  const E* p;
  int64_t ld, n;  // n: elements from p to the end of the last row
};

template <typename T>
Mat<T> mat(const void* p, int64_t ld, int64_t m, int64_t k) {
  Mat<T> a;
  a.p = static_cast<const typename Elem<T>::type*>(p);
  a.ld = ld;
  a.n = m > 0 ? (m - 1) * ld + k : 0;
  return a;
}

// The first nd (< DW) dwords at p, at any 2-byte boundary; zeros after them.
// By the bits of nd: a load of DW/2 dwords, of DW/4 ..., each to its place.
// (A load for each element would keep 16 addresses and masks alive and make
// the kernels spill.  The places are picked with masks: as selects the compiler
// makes an indexed array of them, puts it into LDS, and for that reads the
// launch's dimensions from host memory, 10 us a launch.)
__device__ __forceinline__ uint32_t only_if(bool b) { return b ? ~0u : 0u; }

template <int B, int DW>
__device__ __forceinline__ void load_some_from(const uint8_t* p, int nd, uint32_t (&d)[DW]) {
  if (nd & B) {
    const int at = nd & ~(2 * B - 1);
    uint32_t v[B];
    __builtin_memcpy(v, p + 4 * at, 4 * B);
#pragma unroll
    for (int o = 0; o + 2 * B <= DW; o += 2 * B)
#pragma unroll
      for (int i = 0; i < B; ++i) d[o + i] |= v[i] & only_if(at == o);
  }
  if constexpr (B > 1) load_some_from<B / 2>(p, nd, d);
}
template <int DW>
__device__ __forceinline__ void load_some(const uint8_t* p, int nd, uint32_t (&d)[DW]) {
#pragma unroll
  for (int i = 0; i < DW; ++i) d[i] = 0;
  load_some_from<DW / 2>(p, nd, d);
}
template <int B, int DW>
__device__ __forceinline__ void store_some_from(uint8_t* p, int nd, const uint32_t (&d)[DW]) {
  if (nd & B) {
    const int at = nd & ~(2 * B - 1);
    uint32_t v[B];
#pragma unroll
    for (int i = 0; i < B; ++i) v[i] = 0;
#pragma unroll
    for (int o = 0; o + 2 * B <= DW; o += 2 * B)
#pragma unroll
      for (int i = 0; i < B; ++i) v[i] |= d[o + i] & only_if(at == o);
    __builtin_memcpy(p + 4 * at, v, 4 * B);
  }
  if constexpr (B > 1) store_some_from<B / 2>(p, nd, d);
}
template <int DW>
__device__ __forceinline__ void store_some(uint8_t* p, int nd, const uint32_t (&d)[DW]) {
  store_some_from<DW / 2>(p, nd, d);
}

// Elements c .. c + 15 of a row, as 16-byte parts: 8 dwords of pairs of a
// 16-bit type or 16 dwords of fp32.  WHOLE: all of them are there; otherwise
// (the end of a row whose length is no multiple of 16) n = k - c are, and
// zeros follow.
template <typename T>
struct Piece {
  static constexpr int kDw = sizeof(typename Elem<T>::type) * 4;
  uint32_t d[kDw];
  __device__ __forceinline__ float at(int i) const {
    if constexpr (kDw == 8) return T::widen((uint16_t)(d[i >> 1] >> (16 * (i & 1))));
    else return __builtin_bit_cast(float, d[i]);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kDw; ++i) d[i] = 0;
  }
  // Drops the first n (0 .. 15) elements and fills up with zeros: what makes
  // the end of a row out of the 16 elements before its end.
  __device__ __forceinline__ void shift(int n) {
    if constexpr (kDw == 8) {
      if (n & 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = __builtin_amdgcn_alignbit(i + 1 < 8 ? d[i + 1] : 0u, d[i], 16);
      }
      n >>= 1;
    }
    shift_dwords<kDw / 2>(n);
  }
  template <int B>
  __device__ __forceinline__ void shift_dwords(int n) {
    const uint32_t yes = only_if(n & B);
#pragma unroll
    for (int i = 0; i < kDw; ++i) d[i] = (d[i] & ~yes) | ((i + B < kDw ? d[i + B] : 0u) & yes);
    if constexpr (B > 1) shift_dwords<B / 2>(n);
  }
  template <bool WHOLE>
  __device__ __forceinline__ void load(const Mat<T>& a, int64_t row, int64_t c, int64_t k) {
    const int64_t e = row * a.ld + c;
    const uint8_t* p = reinterpret_cast<const uint8_t*>(a.p + e);
    constexpr int PER = 16 / sizeof(typename Elem<T>::type);
    if constexpr (WHOLE) {
#pragma unroll
      for (int j = 0; j < kDw / 4; ++j) {
        const Bytes16 u = in_bounds(e + j * PER, PER, a.n) ? *reinterpret_cast<const Bytes16*>(p + 16 * j)
                                                           : Bytes16{0, 0, 0, 0};
        d[4 * j] = u.x;
        d[4 * j + 1] = u.y;
        d[4 * j + 2] = u.z;
        d[4 * j + 3] = u.w;
      }
    } else {
      int n = (int)(k - c);
      if (!in_bounds(e, n, a.n)) n = 0;
      load_some(p, kDw == 8 ? n >> 1 : n, d);
      if (kDw == 8 && (n & 1)) {
        const uint32_t last = a.p[e + n - 1];
#pragma unroll
        for (int i = 0; i < kDw; ++i) d[i] |= last & only_if(i == n >> 1);
      }
    }
  }
};

__device__ __forceinline__ uint32_t abs_bits(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }

// Quantizer of one row from its largest absolute value: code = RNE(a / b)
// with a = c x, b the row's amax and c = 127, both scaled down by 2^32 where
// 127 x could overflow.  The quotient is a y (y = 1 / b), corrected once by
// its exact remainder, which makes it the correctly rounded one (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990): exact ties are met exactly, with 3 operations a value
// where a division has about 10.
struct RowQuant {
  float c, b, y;
};

__device__ __forceinline__ RowQuant row_quant(float amax) {
  const float f = amax >= 0x1p+96f ? 0x1p-32f : 1.f;
  RowQuant q;
  q.c = 127.f * f;
  q.b = amax * f;
  q.y = 1.f / q.b;
  return q;
}

// Four codes as one dword.  Adding 1.5 * 2^23 rounds to nearest even and
// leaves the code in the low byte.
__device__ __forceinline__ uint32_t code_bits(const RowQuant& q, float x) {
  const float a = q.c * x;
  const float q0 = a * q.y;
  const float q1 = __builtin_fmaf(__builtin_fmaf(-q0, q.b, a), q.y, q0);
  return __builtin_bit_cast(uint32_t, q1 + 12582912.f);
}
__device__ __forceinline__ uint32_t codes4(const RowQuant& q, float a, float b, float c, float d) {
  const uint32_t lo = __builtin_amdgcn_perm(code_bits(q, b), code_bits(q, a), 0x0c0c0400u);
  const uint32_t hi = __builtin_amdgcn_perm(code_bits(q, d), code_bits(q, c), 0x04000c0cu);
  return lo | hi;
}

// The 16 codes of a piece.
__device__ __forceinline__ uint4 codes16(const RowQuant& q, const float (&v)[16]) {
  return make_uint4(codes4(q, v[0], v[1], v[2], v[3]), codes4(q, v[4], v[5], v[6], v[7]),
                    codes4(q, v[8], v[9], v[10], v[11]), codes4(q, v[12], v[13], v[14], v[15]));
}

// ---- what a row is made of --------------------------------------------------
// Raw: what is loaded for a piece; load(): the loads alone, so that those of
// all a thread's pieces are in flight together; value(): 16 fp32 values.

template <typename T>
struct QuantSrc {
  static constexpr bool kNorm = false, kHeavy = false;
  Mat<T> x;
  const float* col_scale;
  struct Raw {
    Piece<T> x;
    __device__ __forceinline__ void shift(int n) { x.shift(n); }
  };
  template <bool WHOLE>
  __device__ __forceinline__ void load(int64_t row, int64_t c, int64_t k, Raw& r) const {
    r.x.template load<WHOLE>(x, row, c, k);
  }
  __device__ __forceinline__ void value(const Raw& r, int64_t, int64_t c, int64_t k, float (&v)[16], float&) const {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = r.x.at(i);
    if (col_scale) {
      Piece<F32> f;
      const Mat<F32> a{col_scale, k, k};
      if (c + 16 <= k) f.template load<true>(a, 0, c, k);
      else f.template load<false>(a, 0, c, k);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] *= f.at(i);
    }
  }
};

// One piece by itself, whole or not (c < k).
template <typename Src>
__device__ __forceinline__ void piece(const Src& src, int64_t row, int64_t c, int64_t k, float (&v)[16], float& sum) {
  typename Src::Raw r;
  if (c + 16 <= k) src.template load<true>(row, c, k, r);
  else src.template load<false>(row, c, k, r);
  src.value(r, row, c, k, v, sum);
}

}  // namespace
}  // namespace qlora
