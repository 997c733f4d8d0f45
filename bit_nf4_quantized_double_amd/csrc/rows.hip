// Row-wise operators around the linears of a decoder block: RMS norm with the
// residual's addition, SwiGLU, and quantization of rows to 8 bits.
//
//   quantize   amax = max(max |x|, 1e-30), scale = amax / 127,
//              code = 127 x / amax rounded to nearest, ties to even
//   RMS norm   h = E(x + residual), rstd = 1 / sqrt(mean h^2 + eps),
//              y = h gamma rstd
//   backward   hat = h rstd, g = dy gamma,
//              dx = dh + rstd (g - hat mean(g hat)), dgamma = sum_m dy hat
//   SwiGLU     y = gate u / (1 + e^-gate)
//
// All of them move a few bytes per operation and are bound by memory: each
// input is read once, kept in registers as fp32 across the row's reductions,
// and each output written once.  The 8-bit output goes straight into the
// operand tiles that the int8 product reads (int8_layout.h).
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "int8_layout.h"

namespace qlora {
namespace {

constexpr float kAmaxFloor = 1e-30f;

// One fp32 of a 16- or 32-bit element type.
struct F32 {};
template <typename T> struct Elem { typedef uint16_t type; };
template <> struct Elem<F32> { typedef float type; };
template <typename T> __device__ __forceinline__ float widen(uint16_t b) { return T::widen(b); }
template <typename T> __device__ __forceinline__ float widen(float f) { return f; }

// 16 bytes at any element's address: rows that are not 16-byte aligned (an odd
// width, a slice of a wider matrix) are still loaded and stored 16 bytes at a
// time, which the hardware takes at any alignment; only a row's end goes
// element by element.  A row 2500 wide in fp16, norm forward and backward at
// 777 rows: TODO.
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

// Elements c .. c + W - 1 of a row as fp32, zeros from k on.
template <int W, typename T>
__device__ __forceinline__ void load_row(const Mat<T>& a, int64_t row, int64_t c, int64_t k, float (&v)[W]) {
  typedef typename Elem<T>::type E;
  const int64_t e = row * a.ld + c;
  if (c + W <= k) {
    constexpr int PER = 16 / sizeof(E);
    Bytes16 u[W / PER];
#pragma unroll
    for (int j = 0; j < W / PER; ++j)
      u[j] = in_bounds(e + j * PER, PER, a.n) ? *reinterpret_cast<const Bytes16*>(a.p + e + j * PER)
                                              : Bytes16{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < W / PER; ++j) {
      const uint32_t d[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if constexpr (sizeof(E) == 2) v[j * PER + i] = widen<T>((uint16_t)(d[i >> 1] >> (16 * (i & 1))));
        else v[j * PER + i] = __builtin_bit_cast(float, d[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = c + i < k && in_bounds(e + i, 1, a.n) ? widen<T>(a.p[e + i]) : 0.f;
  }
}

// The same 16 elements of a 16-bit row, packed in pairs.
template <typename T>
__device__ __forceinline__ void load_packed(const Mat<T>& a, int64_t row, int64_t c, int64_t k, uint32_t (&d)[8]) {
  const int64_t e = row * a.ld + c;
  if (c + 16 <= k) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const Bytes16 u = in_bounds(e + 8 * j, 8, a.n) ? *reinterpret_cast<const Bytes16*>(a.p + e + 8 * j)
                                                     : Bytes16{0, 0, 0, 0};
      d[4 * j] = u.x;
      d[4 * j + 1] = u.y;
      d[4 * j + 2] = u.z;
      d[4 * j + 3] = u.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (c + i < k && in_bounds(e + i, 1, a.n)) d[i >> 1] |= (uint32_t)a.p[e + i] << (16 * (i & 1));
  }
}
template <typename T>
__device__ __forceinline__ float unpack(const uint32_t (&d)[8], int i) {
  return T::widen((uint16_t)(d[i >> 1] >> (16 * (i & 1))));
}

// A row-major contiguous 16-bit output of n elements.
struct Out16 {
  uint16_t* p;
  int64_t ld, n;
};
Out16 out16(uint16_t* p, int64_t m, int64_t k) { return Out16{p, k, m * k}; }

template <typename T, int W>
__device__ __forceinline__ void store_row(const Out16& o, int64_t row, int64_t c, int64_t k, const float (&v)[W]) {
  const int64_t e = row * o.ld + c;
  if (c + W <= k) {
#pragma unroll
    for (int j = 0; j < W; j += 8)
      if (in_bounds(e + j, 8, o.n))
        *reinterpret_cast<Bytes16*>(o.p + e + j) =
            Bytes16{T::pack2(v[j], v[j + 1]), T::pack2(v[j + 2], v[j + 3]), T::pack2(v[j + 4], v[j + 5]),
                    T::pack2(v[j + 6], v[j + 7])};
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (c + i < k && in_bounds(e + i, 1, o.n)) o.p[e + i] = (uint16_t)T::pack2(v[i], 0.f);
  }
}

// Sum and maximum (of non-negative fp32 bit patterns, so that a NaN or an
// infinity wins) over the TPR threads of a row; every thread gets both.
// `lds` has two words for each wave of the workgroup.
template <int TPR>
__device__ __forceinline__ void row_reduce(float& sum, uint32_t& top, uint32_t* lds) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    sum += __shfl_xor(sum, d);
    top = max(top, (uint32_t)__shfl_xor((int)top, d));
  }
  if constexpr (TPR > 64) {
    constexpr int NW = TPR / 64;
    const int wave = threadIdx.x >> 6, first = wave & ~(NW - 1);
    __syncthreads();  // an earlier reduction's reads are done
    if ((threadIdx.x & 63) == 0) {
      lds[2 * wave] = __builtin_bit_cast(uint32_t, sum);
      lds[2 * wave + 1] = top;
    }
    __syncthreads();
    sum = 0.f;
    top = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      sum += __builtin_bit_cast(float, lds[2 * (first + i)]);
      top = max(top, lds[2 * (first + i) + 1]);
    }
  }
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }

// Where a row's codes go.
struct Out8 {
  int8_t* codes;
  float* scale;
  int64_t kp, bytes, nscale;
  bool weight;
};

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

__device__ __forceinline__ void store_codes(const Out8& o, int64_t row, int64_t piece, bool finite, const RowQuant& q,
                                            const float (&v)[16]) {
  if (piece * 16 >= o.kp) return;
  const int64_t at = int8_piece(o.weight ? int8_weight_row(row) : row, piece, o.kp);
  uint4 u = make_uint4(codes4(q, v[0], v[1], v[2], v[3]), codes4(q, v[4], v[5], v[6], v[7]),
                       codes4(q, v[8], v[9], v[10], v[11]), codes4(q, v[12], v[13], v[14], v[15]));
  if (!finite) u = make_uint4(0, 0, 0, 0);
  if (in_bounds(at, 16, o.bytes)) *reinterpret_cast<uint4*>(o.codes + at) = u;
}

// ---- what a row is made of --------------------------------------------------
// load(): 16 values of a row as fp32.

template <typename T>
struct QuantSrc {
  static constexpr bool kNorm = false;
  Mat<T> x;
  const float* col_scale;
  __device__ __forceinline__ void load(int64_t row, int64_t c, int64_t k, float (&v)[16], float&) const {
    load_row<16>(x, row, c, k, v);
    if (col_scale) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] *= c + i < k && in_bounds(c + i, 1, k) ? col_scale[c + i] : 0.f;
    }
  }
};

__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.f + __expf(-g)); }

template <typename T>
struct SwigluSrc {
  static constexpr bool kNorm = false;
  Mat<T> g, u;
  __device__ __forceinline__ void load(int64_t row, int64_t c, int64_t k, float (&v)[16], float&) const {
    float w[16];
    load_row<16>(g, row, c, k, v);
    load_row<16>(u, row, c, k, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = v[i] * sigmoid(v[i]) * w[i];
  }
};

// load() gives h gamma and adds up h^2: y is that times rstd, whose factor
// the codes do not see and the scale gets at the end, so that one reduction
// serves both.
template <typename T, typename G>
struct NormSrc {
  static constexpr bool kNorm = true;
  Mat<T> x, r;
  Mat<G> gamma;
  Out16 h;
  float eps;
  __device__ __forceinline__ void load(int64_t row, int64_t c, int64_t k, float (&v)[16], float& sum) const {
    float w[16];
    load_row<16>(x, row, c, k, v);
    if (r.p) {
      load_row<16>(r, row, c, k, w);
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        // what is normalised is the hidden state as it is stored, in 16 bits
        const uint32_t b = T::pack2(v[i] + w[i], v[i + 1] + w[i + 1]);
        v[i] = T::widen((uint16_t)b);
        v[i + 1] = T::widen((uint16_t)(b >> 16));
      }
      store_row<T>(h, row, c, k, v);
    }
    load_row<16>(gamma, 0, c, k, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      sum = __builtin_fmaf(v[i], v[i], sum);
      v[i] *= w[i];
    }
  }
};

// One row per TPR threads, blockDim.x / TPR rows per workgroup.  A thread
// holds NCH pieces of 16 values (piece j: TPR j + its index in the row);
// NCH == 0 (rows too long for that) reads the row a second time instead, from
// the cache.
template <typename Src, int TPR, int NCH, bool Y16, typename T>
__global__ __launch_bounds__(1024) void k_rows(Src src, Out8 o8, Out16 o16, float* rstd_out, int64_t m, int64_t k) {
  __shared__ uint32_t s_red[32];
  const int t = threadIdx.x & (TPR - 1);
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / TPR) + threadIdx.x / TPR;
  const bool live = row < m;
  const int64_t npieces = Y16 ? (k + 15) / 16 : o8.kp / 16;
  float sum = 0.f;
  uint32_t top = 0;
  constexpr int NV = NCH ? NCH : 1;
  float v[NV][16];
  if (live) {
    if constexpr (NCH > 0) {
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const int64_t p = t + (int64_t)j * TPR;
        if (p * 16 < k) {
          src.load(row, p * 16, k, v[j], sum);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[j][i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) top = max(top, abs_bits(v[j][i]));
      }
    } else {
      for (int64_t p = t; p * 16 < k; p += TPR) {
        src.load(row, p * 16, k, v[0], sum);
#pragma unroll
        for (int i = 0; i < 16; ++i) top = max(top, abs_bits(v[0][i]));
      }
    }
  }
  row_reduce<TPR>(sum, top, s_red);
  if (!live) return;
  float rstd = 1.f;
  // 1 / sqrt in full: it is once a row, and every value of the row has it
  if constexpr (Src::kNorm) rstd = 1.f / sqrtf(sum / (float)k + src.eps);
  if constexpr (Y16) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t p = t + (int64_t)j * TPR;
      if (p < npieces) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[j][i] *= rstd;
        store_row<T>(o16, row, p * 16, k, v[j]);
      }
    }
    if (t == 0 && in_bounds(row, 1, m)) rstd_out[row] = rstd;
  } else {
    // the floor is on the amax of the output, top * rstd
    float amax = __builtin_bit_cast(float, top);
    if constexpr (Src::kNorm) amax = fmaxf(amax, kAmaxFloor / rstd);
    else amax = fmaxf(amax, kAmaxFloor);
    const bool finite = top < 0x7f800000u && amax < __builtin_inff();
    const RowQuant q = row_quant(finite ? amax : 1.f);
    if constexpr (NCH > 0) {
#pragma unroll
      for (int j = 0; j < NCH; ++j) store_codes(o8, row, t + (int64_t)j * TPR, finite, q, v[j]);
    } else {
      for (int64_t p = t; p < npieces; p += TPR) {
        float again = 0.f;
        if (p * 16 < k) {
          src.load(row, p * 16, k, v[0], again);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[0][i] = 0.f;
        }
        store_codes(o8, row, p, finite, q, v[0]);
      }
    }
    // a row with an infinity or a NaN: zero codes and a NaN scale, so that
    // every value and product of it is NaN
    if (t == 0 && in_bounds(row, 1, o8.nscale))
      o8.scale[row] = finite ? amax * rstd / 127.f : __builtin_nanf("");
  }
}

// Threads for a row: enough that two pieces each hold it, as many as there
// are for few rows; then as many rows in a workgroup as keep one for each
// compute unit, at most a strip of 16 (whose codes share cache lines).
template <typename Src, bool Y16, typename T>
hipError_t launch_rows(const Src& src, const Out8& o8, const Out16& o16, float* rstd, int64_t m, int64_t k, int cus,
                       hipStream_t st) {
  const int64_t pieces = Y16 ? (k + 15) / 16 : o8.kp / 16;
  auto go = [&](auto tpr, auto nch) {
    constexpr int TPR = decltype(tpr)::value, NCH = decltype(nch)::value;
    int64_t r = 1;
    while (r * 2 * TPR <= 1024 && r < 16 && r * 2 * cus <= m) r *= 2;
    const int64_t grid = (m + r - 1) / r;
    k_rows<Src, TPR, NCH, Y16, T><<<dim3((uint32_t)grid), dim3((uint32_t)(TPR * r)), 0, st>>>(src, o8, o16, rstd, m, k);
    return hipGetLastError();
  };
  if (pieces <= 64) return go(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  if (pieces <= 128) return go(std::integral_constant<int, 128>{}, std::integral_constant<int, 1>{});
  if (pieces <= 256) return go(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
  if (pieces <= 512) return go(std::integral_constant<int, 512>{}, std::integral_constant<int, 1>{});
  if (pieces <= 1024) return go(std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
  if (pieces <= 2048) return go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
  if constexpr (!Src::kNorm) return go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 0>{});
  return hipErrorInvalidValue;  // the entry points refuse norms of longer rows
}

Out8 out8(int8_t* codes, float* scale, int64_t m, int64_t k, bool weight) {
  return Out8{codes, scale, int8_kp(k), (int64_t)(weight ? int8_weight_bytes(m, k) : int8_rows_bytes(m, k)), m, weight};
}

template <typename T, typename G>
hipError_t norm_typed(const NormArgs& a, int cus, hipStream_t st) {
  NormSrc<T, G> s;
  s.x = mat<T>(a.x, a.ldx, a.m, a.k);
  s.r = mat<T>(a.residual, a.ldr, a.residual ? a.m : 0, a.k);
  s.gamma = mat<G>(a.gamma, a.k, 1, a.k);
  s.h = out16(a.h, a.m, a.k);
  s.eps = a.eps;
  if (a.y) return launch_rows<NormSrc<T, G>, true, T>(s, Out8{}, out16(a.y, a.m, a.k), a.rstd, a.m, a.k, cus, st);
  return launch_rows<NormSrc<T, G>, false, T>(s, out8(a.codes, a.scale, a.m, a.k, false), Out16{}, nullptr, a.m, a.k,
                                              cus, st);
}

// ---- RMS norm, backward -----------------------------------------------------
// Workgroup b takes rows b, b + groups, ...; a thread keeps its columns
// throughout, so the dgamma of its rows adds up in registers (in row order)
// and leaves once, as one row of partial sums; k_norm_dgamma adds the groups
// up in a fixed order.  No atomics: the same inputs give the same bits.
template <typename T, typename G, int TPR, int NCH>
__global__ __launch_bounds__(TPR) void k_norm_bwd(Mat<T> dy, Mat<T> h, Mat<T> dh, Mat<G> gamma, const float* rstd,
                                                  Out16 dx, float* part, int64_t m, int64_t k) {
  __shared__ uint32_t s_red[32];
  const int t = threadIdx.x;
  float acc[NCH][16];
#pragma unroll
  for (int j = 0; j < NCH; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[j][i] = 0.f;
  for (int64_t row = blockIdx.x; row < m; row += gridDim.x) {
    const float rs = in_bounds(row, 1, m) ? rstd[row] : 0.f;
    // the row's values stay packed across the reduction: half the registers
    uint32_t hp[NCH][8], dp[NCH][8];
    float dot = 0.f;
    uint32_t none = 0;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int64_t c = ((int64_t)j * TPR + t) * 16;
      load_packed(h, row, c, k, hp[j]);
      load_packed(dy, row, c, k, dp[j]);
    }
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      float gm[16];
      load_row<16>(gamma, 0, ((int64_t)j * TPR + t) * 16, k, gm);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float hat = unpack<T>(hp[j], i) * rs, d = unpack<T>(dp[j], i);
        acc[j][i] = __builtin_fmaf(d, hat, acc[j][i]);
        dot = __builtin_fmaf(d * gm[i], hat, dot);
      }
    }
    row_reduce<TPR>(dot, none, s_red);
    dot /= (float)k;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int64_t c = ((int64_t)j * TPR + t) * 16;
      if (c >= k) continue;
      float g[16];
      load_row<16>(gamma, 0, c, k, g);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        g[i] = rs * __builtin_fmaf(-(unpack<T>(hp[j], i) * rs), dot, unpack<T>(dp[j], i) * g[i]);
      if (dh.p) {
        uint32_t e[8];
        load_packed(dh, row, c, k, e);
#pragma unroll
        for (int i = 0; i < 16; ++i) g[i] += unpack<T>(e, i);
      }
      store_row<T>(dx, row, c, k, g);
    }
  }
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    const int64_t c = ((int64_t)j * TPR + t) * 16;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (c + i < k && in_bounds((int64_t)blockIdx.x * k + c + i, 1, (int64_t)gridDim.x * k))
        part[(int64_t)blockIdx.x * k + c + i] = acc[j][i];
  }
}

// dgamma[c] = sum over the groups of part[g][c]: 64 columns a workgroup, 16
// waves that each add every 16th group, then the waves in order.
__global__ __launch_bounds__(1024) void k_norm_dgamma(const float* part, int groups, float* dgamma, int64_t k) {
  __shared__ float s[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float v = 0.f;
  if (c < k)
    for (int g = w; g < groups; g += 16)
      v += in_bounds(g * k + c, 1, groups * k) ? part[g * k + c] : 0.f;
  s[w][lane] = v;
  __syncthreads();
  if (w == 0 && c < k) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += s[i][lane];
    if (in_bounds(c, 1, k)) dgamma[c] = v;
  }
}

template <typename T, typename G>
hipError_t norm_bwd_typed(const NormBwdArgs& a, int cus, hipStream_t st) {
  const Mat<T> dy = mat<T>(a.dy, a.lddy, a.m, a.k), h = mat<T>(a.h, a.ldh, a.m, a.k),
               dh = mat<T>(a.dh, a.lddh, a.dh ? a.m : 0, a.k);
  const Mat<G> gamma = mat<G>(a.gamma, a.k, 1, a.k);
  const Out16 dx = out16(a.dx, a.m, a.k);
  const int groups = a.m > 0 ? norm_bwd_groups(a.m, a.k, cus) : 0;
  auto go = [&](auto tpr, auto nch) {
    constexpr int TPR = decltype(tpr)::value, NCH = decltype(nch)::value;
    k_norm_bwd<T, G, TPR, NCH><<<dim3(groups), dim3(TPR), 0, st>>>(dy, h, dh, gamma, a.rstd, dx, a.part, a.m, a.k);
    return hipGetLastError();
  };
  const int64_t pieces = (a.k + 15) / 16;
  hipError_t e = hipSuccess;
  if (groups == 0) {  // no rows: dgamma is an empty sum
  } else if (pieces <= 64) e = go(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  else if (pieces <= 256) e = go(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
  else if (pieces <= 512) e = go(std::integral_constant<int, 512>{}, std::integral_constant<int, 1>{});
  else if (pieces <= 1024) e = go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 1>{});
  else e = go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
  if (e != hipSuccess) return e;
  k_norm_dgamma<<<dim3((uint32_t)((a.k + 63) / 64)), dim3(1024), 0, st>>>(a.part, groups, a.dgamma, a.k);
  return hipGetLastError();
}

// ---- SwiGLU in 16 bits, elementwise -----------------------------------------
// 8 values a thread; `per` pieces of 8 in a row.
template <typename T>
__global__ __launch_bounds__(256) void k_swiglu(Mat<T> g, Mat<T> u, Out16 y, uint32_t per, uint32_t total, int64_t k) {
  const uint32_t id = blockIdx.x * 256u + threadIdx.x;
  if (id >= total) return;
  const int64_t row = id / per, c = (int64_t)(id % per) * 8;
  float a[8], b[8];
  load_row<8>(g, row, c, k, a);
  load_row<8>(u, row, c, k, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = a[i] * sigmoid(a[i]) * b[i];
  store_row<T>(y, row, c, k, a);
}

template <typename T>
__global__ __launch_bounds__(256) void k_swiglu_bwd(Mat<T> dy, Mat<T> g, Mat<T> u, Out16 dg, Out16 du, uint32_t per,
                                                    uint32_t total, int64_t k) {
  const uint32_t id = blockIdx.x * 256u + threadIdx.x;
  if (id >= total) return;
  const int64_t row = id / per, c = (int64_t)(id % per) * 8;
  float d[8], a[8], b[8];
  load_row<8>(dy, row, c, k, d);
  load_row<8>(g, row, c, k, a);
  load_row<8>(u, row, c, k, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = sigmoid(a[i]);
    const float dup = d[i] * a[i] * s;
    a[i] = d[i] * b[i] * s * (1.f + a[i] * (1.f - s));
    b[i] = dup;
  }
  store_row<T>(dg, row, c, k, a);
  store_row<T>(du, row, c, k, b);
}

}  // namespace

hipError_t launch_quant_rows(const QuantArgs& a, int cus, hipStream_t st) {
  const Out8 o = out8(a.codes, a.scale, a.m, a.k, a.weight);
  auto go = [&](auto type) {
    typedef decltype(type) T;
    const QuantSrc<T> s{mat<T>(a.x, a.ldx, a.m, a.k), a.col_scale};
    return launch_rows<QuantSrc<T>, false, T>(s, o, Out16{}, nullptr, a.m, a.k, cus, st);
  };
  return a.type == kRowF32 ? go(F32{}) : a.type == kRowF16 ? go(F16{}) : go(Bf16{});
}

hipError_t launch_norm(const NormArgs& a, int cus, hipStream_t st) {
  if (a.gamma_type == kRowF32) return a.type == kRowF16 ? norm_typed<F16, F32>(a, cus, st) : norm_typed<Bf16, F32>(a, cus, st);
  return a.type == kRowF16 ? norm_typed<F16, F16>(a, cus, st) : norm_typed<Bf16, Bf16>(a, cus, st);
}

// Two workgroups a compute unit where there are rows for them: more partial
// sums would cost more than the rows they spread.
int norm_bwd_groups(int64_t m, int64_t k, int cus) {
  const int64_t per = k > 8192 ? 1 : 2;
  return (int)std::max<int64_t>(1, std::min<int64_t>(m, per * cus));
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, int cus, hipStream_t st) {
  if (a.gamma_type == kRowF32)
    return a.type == kRowF16 ? norm_bwd_typed<F16, F32>(a, cus, st) : norm_bwd_typed<Bf16, F32>(a, cus, st);
  return a.type == kRowF16 ? norm_bwd_typed<F16, F16>(a, cus, st) : norm_bwd_typed<Bf16, Bf16>(a, cus, st);
}

hipError_t launch_swiglu_rows(const SwigluArgs& a, int cus, hipStream_t st) {
  const Out8 o = out8(a.codes, a.scale, a.m, a.k, false);
  auto go = [&](auto type) {
    typedef decltype(type) T;
    const SwigluSrc<T> s{mat<T>(a.g, a.ldg, a.m, a.k), mat<T>(a.u, a.ldu, a.m, a.k)};
    return launch_rows<SwigluSrc<T>, false, T>(s, o, Out16{}, nullptr, a.m, a.k, cus, st);
  };
  return a.type == kRowF16 ? go(F16{}) : go(Bf16{});
}

hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t st) {
  const uint32_t per = (uint32_t)((a.k + 7) / 8), total = (uint32_t)(per * a.m);
  auto go = [&](auto type) {
    typedef decltype(type) T;
    k_swiglu<T><<<dim3((total + 255u) / 256u), dim3(256), 0, st>>>(
        mat<T>(a.g, a.ldg, a.m, a.k), mat<T>(a.u, a.ldu, a.m, a.k), out16(a.y, a.m, a.k), per, total, a.k);
    return hipGetLastError();
  };
  return a.type == kRowF16 ? go(F16{}) : go(Bf16{});
}

hipError_t launch_swiglu_bwd(const SwigluArgs& a, hipStream_t st) {
  const uint32_t per = (uint32_t)((a.k + 7) / 8), total = (uint32_t)(per * a.m);
  auto go = [&](auto type) {
    typedef decltype(type) T;
    k_swiglu_bwd<T><<<dim3((total + 255u) / 256u), dim3(256), 0, st>>>(
        mat<T>(a.dy, a.lddy, a.m, a.k), mat<T>(a.g, a.ldg, a.m, a.k), mat<T>(a.u, a.ldu, a.m, a.k),
        out16(a.dg, a.m, a.k), out16(a.du, a.m, a.k), per, total, a.k);
    return hipGetLastError();
  };
  return a.type == kRowF16 ? go(F16{}) : go(Bf16{});
}

QLORA_OOB_READER(oob_count_rows)

}  // namespace qlora
