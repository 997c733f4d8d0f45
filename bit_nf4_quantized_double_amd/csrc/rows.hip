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
#include "rows_common.h"

namespace qlora {
namespace {

// Floats in a row of dgamma's partial sums: whole 16-byte pieces.
__host__ __device__ constexpr int64_t part_pitch(int64_t k) { return (k + 15) / 16 * 16; }

// A row-major contiguous 16-bit output of n elements.
struct Out16 {
  uint16_t* p;
  int64_t ld, n;
};
Out16 out16(uint16_t* p, int64_t m, int64_t k) { return Out16{p, k, m * k}; }

template <typename T>
__device__ __forceinline__ void store_row(const Out16& o, int64_t row, int64_t c, int64_t k, const float (&v)[16]) {
  const int64_t e = row * o.ld + c;
  uint8_t* p = reinterpret_cast<uint8_t*>(o.p + e);
  uint32_t d[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) d[i] = T::pack2(v[2 * i], v[2 * i + 1]);
  if (c + 16 <= k) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (in_bounds(e + 8 * j, 8, o.n))
        *reinterpret_cast<Bytes16*>(p + 16 * j) = Bytes16{d[4 * j], d[4 * j + 1], d[4 * j + 2], d[4 * j + 3]};
  } else {
    int n = (int)(k - c);
    if (!in_bounds(e, n, o.n)) n = 0;
    store_some(p, n >> 1, d);
    if (n & 1) {
      uint32_t last = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) last |= d[i] & only_if(i == n >> 1);
      o.p[e + n - 1] = (uint16_t)last;
    }
  }
}

// Sum and maximum (of non-negative fp32 bit patterns, so that a NaN or an
// infinity wins) over the threads that share a row; each of them gets both.
// RW rows share a wave (64 / RW lanes each, one after another), NW consecutive
// waves share them; `lds` has 2 RW words for each wave of the workgroup.
template <int NW, int RW>
__device__ __forceinline__ void row_reduce(float& sum, uint32_t& top, uint32_t* lds) {
#pragma unroll
  for (int d = 32 / RW; d > 0; d >>= 1) {
    sum += __shfl_xor(sum, d);
    top = max(top, (uint32_t)__shfl_xor((int)top, d));
  }
  if constexpr (NW > 1) {
    const int wave = threadIdx.x >> 6, first = wave / NW * NW, lane = threadIdx.x & 63, r = lane / (64 / RW);
    __syncthreads();  // an earlier reduction's reads are done
    if (lane % (64 / RW) == 0) {
      lds[2 * (RW * wave + r)] = __builtin_bit_cast(uint32_t, sum);
      lds[2 * (RW * wave + r) + 1] = top;
    }
    __syncthreads();
    sum = 0.f;
    top = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      sum += __builtin_bit_cast(float, lds[2 * (RW * (first + w) + r)]);
      top = max(top, lds[2 * (RW * (first + w) + r) + 1]);
    }
  }
}

// Where a row's codes go.
struct Out8 {
  int8_t* codes;
  float* scale;
  int64_t kp, bytes, nscale;
  bool weight;
};

__device__ __forceinline__ void store_codes(const Out8& o, int64_t row, int64_t piece, uint4 u) {
  if (row >= o.nscale || piece * 16 >= o.kp) return;
  const int64_t at = int8_piece(o.weight ? int8_weight_row(row) : row, piece, o.kp);
  if (in_bounds(at, 16, o.bytes)) *reinterpret_cast<uint4*>(o.codes + at) = u;
}

// ---- sources of rows (QuantSrc: rows_common.h) -------------------------------

// 1 / (1 + e^-g).  The reciprocal instruction flushes results below 2^-126, so
// it is taken of 2^-32 (1 + e^-g) and scaled back: powers of two, which change
// no other result.
__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(__builtin_fmaf(__expf(-g), 0x1p-32f, 0x1p-32f)) * 0x1p-32f;
}

template <typename T>
struct SwigluSrc {
  static constexpr bool kNorm = false, kHeavy = false;
  Mat<T> g, u;
  struct Raw {
    Piece<T> g, u;
    __device__ __forceinline__ void shift(int n) {
      g.shift(n);
      u.shift(n);
    }
  };
  template <bool WHOLE>
  __device__ __forceinline__ void load(int64_t row, int64_t c, int64_t k, Raw& r) const {
    r.g.template load<WHOLE>(g, row, c, k);
    r.u.template load<WHOLE>(u, row, c, k);
  }
  __device__ __forceinline__ void value(const Raw& r, int64_t, int64_t, int64_t, float (&v)[16], float&) const {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = r.g.at(i) * sigmoid(r.g.at(i)) * r.u.at(i);
  }
};

// value() gives h gamma and adds up h^2: y is that times rstd, whose factor
// the codes do not see and the scale gets at the end, so that one reduction
// serves both.
template <typename T, typename G>
struct NormSrc {
  static constexpr bool kNorm = true, kHeavy = Piece<G>::kDw == 16;  // heavy: 32 registers a piece in flight
  Mat<T> x, r;
  Mat<G> gamma;
  Out16 h;
  float eps;
  struct Raw {
    Piece<T> x, r;
    Piece<G> g;
    __device__ __forceinline__ void shift(int n) {
      x.shift(n);
      r.shift(n);
      g.shift(n);
    }
  };
  template <bool WHOLE>
  __device__ __forceinline__ void load(int64_t row, int64_t c, int64_t k, Raw& w) const {
    w.x.template load<WHOLE>(x, row, c, k);
    if (r.p) w.r.template load<WHOLE>(r, row, c, k);
    else w.r.zero();
    w.g.template load<WHOLE>(gamma, 0, c, k);
  }
  __device__ __forceinline__ void value(const Raw& w, int64_t row, int64_t c, int64_t k, float (&v)[16],
                                        float& sum) const {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = w.x.at(i);
    if (r.p) {
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        // what is normalised is the hidden state as it is stored, in 16 bits
        const uint32_t b = T::pack2(v[i] + w.r.at(i), v[i + 1] + w.r.at(i + 1));
        v[i] = T::widen((uint16_t)b);
        v[i + 1] = T::widen((uint16_t)(b >> 16));
      }
      store_row<T>(h, row, c, k, v);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      sum = __builtin_fmaf(v[i], v[i], sum);
      v[i] *= w.g.at(i);
    }
  }
};

// TPR threads share a row, RW rows share a wave, and a workgroup of kBlock
// threads takes kBlock / TPR rows.  A thread holds NCH pieces of 16 values
// (piece j: TPR j + its index in the row); NCH == 0 (rows too long for that)
// reads the row a second time instead, from the cache.
//
// WIDE: k is at least 16.  All of a thread's loads then go out together, with
// no branch between them: where a row's length is no multiple of 16 its last
// piece is made from the 16 values before its end.
//
// RW = 4 for 8-bit output of many rows: a piece's codes are 16 bytes of a
// strip whose neighbours are the next rows', so one row alone scatters its
// stores, 64 cache lines an instruction.  With four rows in a wave the codes
// change lanes before they are stored, so that neighbouring lanes hold
// neighbouring rows and store runs of 64 bytes, while the loads stay runs of
// 512 bytes of one row.  SwiGLU at 8192 x 14336: 130 us, 163 us with a row to
// a workgroup (two sets of inputs in turn, in part from the last-level cache).
// Rows interleaved by lanes instead, for loads and stores alike, do as well at
// aligned widths, and take 107 us for 57 at 8192 x 7167.
//
// Measured in bf16 at 8192 x 4096 on fresh inputs, median times of the kernel:
// quantize 19 us (5.2 TB/s), SwiGLU in 8 bits 32 us (5.2), norm with the
// residual 45 us (5.9), the same in 8 bits 42 us (5.6; 47 us with the values
// read back between the calls).  Rows of 14336 are 1024 threads to a workgroup
// and one of those to a compute unit, so loads and stores take turns: SwiGLU at
// 8192 x 14336 144 to 150 us (4.0 TB/s).  Walking over the rows, with the next
// ones loaded into the registers that finished pieces leave, spills: 175 us for
// 131 under the conditions of the 130 above.  The norm with four pieces a
// thread spills 3 registers as it is: 2048 x 16384 56 us, in 16 bits 46 us.
template <int TPR, int RW> constexpr int kBlock = TPR * RW < 256 ? 256 : TPR * RW;

template <typename Src, int TPR, int RW, int NCH, bool WIDE, bool Y16, typename T>
__global__ __launch_bounds__((kBlock<TPR, RW>)) void k_rows(Src src, Out8 o8, Out16 o16, float* rstd_out, int64_t m,
                                                           int64_t k) {
  constexpr int NW = TPR * RW / 64;  // waves that share RW rows
  __shared__ uint32_t s_red[2 * RW * kBlock<TPR, RW> / 64];
  constexpr int LR = 64 / RW;  // lanes of a row in a wave
  const int lane = threadIdx.x & 63, wave = threadIdx.x % (TPR * RW) / 64;
  const int t = wave * LR + lane % LR;
  const int64_t row0 = (block_of(blockIdx.x, blockIdx.y) * (kBlock<TPR, RW> / (TPR * RW)) + threadIdx.x / (TPR * RW)) * RW;
  const int64_t row = row0 + lane / LR;
  const bool live = row < m;
  const int64_t npieces = Y16 ? (k + 15) / 16 : o8.kp / 16;
  float sum = 0.f;
  uint32_t top = 0;
  constexpr int NV = NCH ? NCH : 1;
  float v[NV][16];
  if constexpr (NCH > 0) {
    typename Src::Raw raw[NCH];
    if constexpr (WIDE) {
      // a thread past the row's end reads its last 16 values and drops them
#pragma unroll
      for (int j = 0; j < NCH; ++j)
        src.template load<true>(live ? row : m - 1, min((t + (int64_t)j * TPR) * 16, k - 16), k, raw[j]);
    }
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int64_t c = (t + (int64_t)j * TPR) * 16;
      if (live && c < k) {
        if constexpr (WIDE) {
          if (c + 16 > k) raw[j].shift((int)(c + 16 - k));
          src.value(raw[j], row, c, k, v[j], sum);
        } else {
          piece(src, row, c, k, v[j], sum);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[j][i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) top = max(top, abs_bits(v[j][i]));
    }
  } else if (live) {
    for (int64_t p = t; p * 16 < k; p += TPR) {
      piece(src, row, p * 16, k, v[0], sum);
#pragma unroll
      for (int i = 0; i < 16; ++i) top = max(top, abs_bits(v[0][i]));
    }
  }
  row_reduce<NW, RW>(sum, top, s_red);
  if (RW == 1 && !live) return;
  float rstd = 1.f;
  // 1 / sqrt in full: it is once a row, and every value of the row has it (a
  // row of no values has the mean 0)
  if constexpr (Src::kNorm) rstd = 1.f / sqrtf(sum / (float)max(k, (int64_t)1) + src.eps);
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
    if constexpr (RW > 1) {
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        // lane RW i + r takes row r's piece i from lane LR r + i
        uint4 u = finite ? codes16(q, v[j]) : make_uint4(0, 0, 0, 0);
        const int from = (lane % RW * LR + lane / RW) * 4;
        u.x = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)u.x);
        u.y = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)u.y);
        u.z = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)u.z);
        u.w = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)u.w);
        store_codes(o8, row0 + lane % RW, wave * LR + lane / RW + (int64_t)j * TPR, u);
      }
    } else if constexpr (NCH > 0) {
#pragma unroll
      for (int j = 0; j < NCH; ++j)
        store_codes(o8, row, t + (int64_t)j * TPR, finite ? codes16(q, v[j]) : make_uint4(0, 0, 0, 0));
    } else {
      for (int64_t p = t; p < npieces; p += TPR) {
        float again = 0.f;
        if (p * 16 < k) {
          piece(src, row, p * 16, k, v[0], again);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[0][i] = 0.f;
        }
        store_codes(o8, row, p, finite ? codes16(q, v[0]) : make_uint4(0, 0, 0, 0));
      }
    }
    // a row with an infinity or a NaN: zero codes and a NaN scale, so that
    // every value and product of it is NaN
    if (live && t == 0 && in_bounds(row, 1, o8.nscale))
      o8.scale[row] = finite ? amax * rstd / 127.f : __builtin_nanf("");
  }
}

template <typename Src, bool Y16, typename T>
hipError_t launch_rows(const Src& src, const Out8& o8, const Out16& o16, float* rstd, int64_t m, int64_t k, int cus,
                       hipStream_t st) {
  const int64_t pieces = Y16 ? (k + 15) / 16 : o8.kp / 16;
  auto go = [&](auto tpr, auto rw, auto nch) {
    constexpr int TPR = decltype(tpr)::value, RW = decltype(rw)::value, NCH = decltype(nch)::value;
    constexpr int per = kBlock<TPR, RW> / TPR;
    const dim3 grid = grid_of((m + per - 1) / per), block(kBlock<TPR, RW>);
    if constexpr (TPR == 64 && RW == 1) {
      if (k < 16) {
        k_rows<Src, TPR, RW, NCH, false, Y16, T><<<grid, block, 0, st>>>(src, o8, o16, rstd, m, k);
        return hipGetLastError();
      }
    }
    k_rows<Src, TPR, RW, NCH, (NCH > 0), Y16, T><<<grid, block, 0, st>>>(src, o8, o16, rstd, m, k);
    return hipGetLastError();
  };
  using std::integral_constant;
  constexpr integral_constant<int, 0> c0{};
  constexpr integral_constant<int, 1> c1{};
  constexpr integral_constant<int, 2> c2{};
  constexpr integral_constant<int, 4> c4{};
  constexpr integral_constant<int, 64> c64{};
  constexpr integral_constant<int, 128> c128{};
  constexpr integral_constant<int, 256> c256{};
  constexpr integral_constant<int, 512> c512{};
  constexpr integral_constant<int, 1024> c1024{};
  if constexpr (!Y16) {
    // four rows side by side where that still leaves each compute unit some
    if (m >= 4 * cus && k >= 16) {
      if (pieces <= 64) return go(c64, c4, c1);
      if (pieces <= 128) return go(c128, c4, c1);
      if (pieces <= 256) return go(c128, c4, c2);
      if (pieces <= 512) return go(c256, c4, c2);
      if (pieces <= 768) return go(c256, c4, integral_constant<int, 3>{});
      if (pieces <= 1024) {
        if constexpr (Src::kHeavy) return go(c512, c2, c2);  // four pieces of it would spill
        else return go(c256, c4, c4);
      }
      if constexpr (!Src::kNorm) {
        if (pieces <= 2048) return go(c512, c2, c4);
      }
    }
  }
  if (pieces <= 64) return go(c64, c1, c1);
  if (pieces <= 128) return go(c128, c1, c1);
  if (pieces <= 256) return go(c256, c1, c1);
  if (pieces <= 512) return go(c512, c1, c1);
  if (pieces <= 1024) return go(c512, c1, c2);
  if (pieces <= 2048) return go(c1024, c1, c2);
  if constexpr (!Src::kNorm) return go(c1024, c1, c0);
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
  // (y is NULL where rows have no values)
  if (a.rstd) return launch_rows<NormSrc<T, G>, true, T>(s, Out8{}, out16(a.y, a.m, a.k), a.rstd, a.m, a.k, cus, st);
  return launch_rows<NormSrc<T, G>, false, T>(s, out8(a.codes, a.scale, a.m, a.k, false), Out16{}, nullptr, a.m, a.k,
                                              cus, st);
}

// ---- RMS norm, backward -----------------------------------------------------
// A workgroup has SUB teams of TPR threads.  Team i of all of them takes rows
// i, i + teams, ...; a thread keeps its columns throughout, so the dgamma of
// its rows adds up in registers (in row order), the teams' sums meet in LDS
// (in team order), and one row of partial sums leaves each workgroup;
// k_norm_dgamma adds those up in a fixed order.  No atomics: the same inputs
// give the same bits.  The next row's h and dY are loaded before the current
// row's reduction, whose latency would otherwise bound the kernel; they stay
// packed in pairs.  8192 x 4096: 56 us (4.8 TB/s); without the loads ahead, four
// rows to a workgroup's turn, 70 us.  Every instance is short of registers: with
// one piece a thread 8 to 13 of them are spilled, 12 to 20 with gamma in fp32,
// most of them reloaded once a turn (8192 x 4096 with gamma in fp32: 62 us; 2048
// x 16384: 61 and 73 us); with two pieces 61 and 123.
template <typename T, typename G, int TPR, int NCH, bool WIDE>
__global__ __launch_bounds__(1024) void k_norm_bwd(Mat<T> dy, Mat<T> h, Mat<T> dh, Mat<G> gamma, const float* rstd,
                                                   Out16 dx, float* part, float* dgamma, int64_t m, int64_t k) {
  constexpr int SUB = 1024 / TPR, NW = TPR / 64;
  __shared__ uint32_t s_red[2 * 16];
  __shared__ __attribute__((aligned(16))) float s_acc[SUB > 1 ? SUB * TPR * 16 : 4];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int64_t step = (int64_t)gridDim.x * SUB;
  auto col = [&](int j) { return ((int64_t)j * TPR + t) * 16; };
  // one piece of a row; rows past the last read the last.  WIDE: as in k_rows,
  // made good by fix() when it is used, so that nothing waits for it before.
  auto get = [&](auto& p, const auto& a, int64_t r, int64_t c) {
    r = r < m ? r : m - 1;
    if constexpr (WIDE) {
      p.template load<true>(a, r, min(c, k - 16), k);
    } else {
      if (c + 16 <= k) p.template load<true>(a, r, c, k);
      else if (c < k) p.template load<false>(a, r, c, k);
      else p.zero();
    }
  };
  auto fix = [&](auto& p, int64_t c) {
    if (WIDE && c + 16 > k) {
      if (c < k) p.shift((int)(c + 16 - k));
      else p.zero();
    }
  };
  float acc[NCH][16];
  Piece<G> gm[NCH];
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    get(gm[j], gamma, 0, col(j));
    fix(gm[j], col(j));
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[j][i] = 0.f;
  }
  constexpr bool AHEAD = NCH == 1;  // two pieces a thread and the next row's would spill far more
  Piece<T> hp[NCH], dp[NCH], hn[NCH], dn[NCH], ep[NCH];
  int64_t row = (int64_t)blockIdx.x * SUB + sub;
#pragma unroll
  for (int j = 0; j < NCH && AHEAD; ++j) {
    get(hp[j], h, row, col(j));
    get(dp[j], dy, row, col(j));
  }
  // every team makes the same number of turns: they share the barriers
  for (int64_t first = (int64_t)blockIdx.x * SUB; first < m; first += step, row += step) {
    const bool live = row < m;
    const float rs = live && in_bounds(row, 1, m) ? rstd[row] : 0.f;
    auto mend = [&] {
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        fix(hp[j], col(j));
        fix(dp[j], col(j));
        if (!live) {  // a row past the last adds nothing, also where the last one's dY is infinite
          hp[j].zero();
          dp[j].zero();
        }
      }
    };
    if (AHEAD) mend();
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      if (dh.p && AHEAD) get(ep[j], dh, row, col(j));
      get(AHEAD ? hn[j] : hp[j], h, AHEAD ? row + step : row, col(j));
      get(AHEAD ? dn[j] : dp[j], dy, AHEAD ? row + step : row, col(j));
    }
    if (!AHEAD) mend();
    float dot = 0.f;
    uint32_t none = 0;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      float part_dot = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float hat = hp[j].at(i) * rs, d = dp[j].at(i);
        acc[j][i] = __builtin_fmaf(d, hat, acc[j][i]);
        part_dot = __builtin_fmaf(d * gm[j].at(i), hat, part_dot);
      }
      dot += part_dot;
    }
    row_reduce<NW, 1>(dot, none, s_red);
    const float mean = dot / (float)k;
    // unpack again rather than keep 48 unpacked values across the reduction:
    // the compiler would find them equal, and spill
#pragma unroll
    for (int j = 0; j < NCH; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        asm volatile("" : "+v"(hp[j].d[i]), "+v"(dp[j].d[i]));
        if constexpr (Piece<G>::kDw == 8) asm volatile("" : "+v"(gm[j].d[i]));
      }
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int64_t c = col(j);
      if (live && c < k) {
        float g[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          g[i] = rs * __builtin_fmaf(-(hp[j].at(i) * rs), mean, dp[j].at(i) * gm[j].at(i));
        if (dh.p) {
          if (!AHEAD) get(ep[j], dh, row, c);
          fix(ep[j], c);
#pragma unroll
          for (int i = 0; i < 16; ++i) g[i] += ep[j].at(i);
        }
        store_row<T>(dx, row, c, k, g);
      }
      if (AHEAD) {
        hp[j] = hn[j];
        dp[j] = dn[j];
      }
    }
  }
  if constexpr (SUB > 1) {
    // [team][4-column group][thread]: conflict-free both ways
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(s_acc + ((sub * 4 + i) * TPR + t) * 4) =
          make_float4(acc[0][4 * i], acc[0][4 * i + 1], acc[0][4 * i + 2], acc[0][4 * i + 3]);
    __syncthreads();
    if (sub > 0) return;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[0][i] = 0.f;
#pragma unroll 2
    for (int w = 0; w < SUB; ++w)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 f = *reinterpret_cast<const float4*>(s_acc + ((w * 4 + i) * TPR + t) * 4);
        acc[0][4 * i] += f.x;
        acc[0][4 * i + 1] += f.y;
        acc[0][4 * i + 2] += f.z;
        acc[0][4 * i + 3] += f.w;
      }
  }
  // a workgroup alone has the whole dgamma (two pieces a thread: 4 us slower
  // at 32768 for the registers that this takes)
  if constexpr (NCH == 1) {
    if (gridDim.x == 1) {
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int64_t c = col(0) + i;
        if (c + 4 <= k) {
          if (in_bounds(c, 4, k))
            *reinterpret_cast<float4*>(dgamma + c) = make_float4(acc[0][i], acc[0][i + 1], acc[0][i + 2], acc[0][i + 3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + e < k && in_bounds(c + e, 1, k)) dgamma[c + e] = acc[0][i + e];
        }
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    const int64_t c = col(j);
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int64_t e = (int64_t)blockIdx.x * part_pitch(k) + c + i;
      if (c + i < k && in_bounds(e, 4, (int64_t)gridDim.x * part_pitch(k)))
        *reinterpret_cast<float4*>(part + e) = make_float4(acc[j][i], acc[j][i + 1], acc[j][i + 2], acc[j][i + 3]);
    }
  }
}

// dgamma[c] = sum over the groups of part[g][c]: 32 columns a workgroup, 32
// partial sums of every 32nd group each, then those in order.
__global__ __launch_bounds__(1024) void k_norm_dgamma(const float* part, int groups, float* dgamma, int64_t k) {
  __shared__ float s[32][32];
  const int col = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + col, pitch = part_pitch(k);
  float v = 0.f;
  if (c < k) {
#pragma unroll 8
    for (int g = w; g < groups; g += 32) v += in_bounds(g * pitch + c, 1, groups * pitch) ? part[g * pitch + c] : 0.f;
  }
  s[w][col] = v;
  __syncthreads();
  if (w == 0 && c < k) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += s[i][col];
    if (in_bounds(c, 1, k)) dgamma[c] = v;
  }
}

// Threads for a row of the backward.
int norm_bwd_threads(int64_t k) { return k <= 1024 ? 64 : k <= 2048 ? 128 : k <= 4096 ? 256 : k <= 8192 ? 512 : 1024; }

template <typename T, typename G>
hipError_t norm_bwd_typed(const NormBwdArgs& a, int cus, hipStream_t st) {
  const Mat<T> dy = mat<T>(a.dy, a.lddy, a.m, a.k), h = mat<T>(a.h, a.ldh, a.m, a.k),
               dh = mat<T>(a.dh, a.lddh, a.dh ? a.m : 0, a.k);
  const Mat<G> gamma = mat<G>(a.gamma, a.k, 1, a.k);
  const Out16 dx = out16(a.dx, a.m, a.k);
  const int groups = a.m > 0 ? norm_bwd_groups(a.m, a.k, cus) : 0;
  auto go = [&](auto tpr, auto nch) {
    constexpr int TPR = decltype(tpr)::value, NCH = decltype(nch)::value;
    if constexpr (TPR == 64) {
      if (a.k < 16) {
        k_norm_bwd<T, G, TPR, NCH, false><<<dim3(groups), dim3(1024), 0, st>>>(dy, h, dh, gamma, a.rstd, dx, a.part, a.dgamma,
                                                                            a.m, a.k);
        return hipGetLastError();
      }
    }
    k_norm_bwd<T, G, TPR, NCH, true><<<dim3(groups), dim3(1024), 0, st>>>(dy, h, dh, gamma, a.rstd, dx, a.part, a.dgamma,
                                                                            a.m, a.k);
    return hipGetLastError();
  };
  using std::integral_constant;
  constexpr integral_constant<int, 1> c1{};
  hipError_t e = hipSuccess;
  if (groups > 0) {  // without rows dgamma is an empty sum
    switch (norm_bwd_threads(a.k)) {
      case 64: e = go(integral_constant<int, 64>{}, c1); break;
      case 128: e = go(integral_constant<int, 128>{}, c1); break;
      case 256: e = go(integral_constant<int, 256>{}, c1); break;
      case 512: e = go(integral_constant<int, 512>{}, c1); break;
      default:
        e = a.k <= 16384 ? go(integral_constant<int, 1024>{}, c1)
                         : go(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
    }
  }
  // k_norm_bwd's own condition for having written dgamma
  if (e != hipSuccess || (groups == 1 && a.k <= 16384)) return e;
  k_norm_dgamma<<<dim3((uint32_t)((a.k + 31) / 32)), dim3(1024), 0, st>>>(a.part, groups, a.dgamma, a.k);
  return hipGetLastError();
}

// ---- SwiGLU in 16 bits, elementwise -----------------------------------------
// 16 values a thread; `per` pieces in a row.  8192 x 4096 in bf16: forward 32 us
// (6.3 TB/s), backward 57 us (5.9).
template <typename T>
__global__ __launch_bounds__(256) void k_swiglu(SwigluSrc<T> s, Out16 y, uint32_t per, uint32_t total, int64_t k) {
  const uint32_t id = blockIdx.x * 256u + threadIdx.x;
  if (id >= total) return;
  const int64_t row = id / per, c = (int64_t)(id % per) * 16;
  float v[16], none = 0.f;
  piece(s, row, c, k, v, none);
  store_row<T>(y, row, c, k, v);
}

template <typename T>
__global__ __launch_bounds__(256) void k_swiglu_bwd(Mat<T> dy, SwigluSrc<T> s, Out16 dg, Out16 du, uint32_t per,
                                                    uint32_t total, int64_t k) {
  const uint32_t id = blockIdx.x * 256u + threadIdx.x;
  if (id >= total) return;
  const int64_t row = id / per, c = (int64_t)(id % per) * 16;
  typename SwigluSrc<T>::Raw r;
  Piece<T> d;
  if (c + 16 <= k) {
    s.template load<true>(row, c, k, r);
    d.template load<true>(dy, row, c, k);
  } else {
    s.template load<false>(row, c, k, r);
    d.template load<false>(dy, row, c, k);
  }
  float a[16], b[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float g = r.g.at(i), sg = sigmoid(g), dyi = d.at(i);
    a[i] = dyi * r.u.at(i) * sg * (1.f + g * (1.f - sg));
    b[i] = dyi * g * sg;
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

// One workgroup of 1024 threads a compute unit, where there are rows for them;
// a single one for the rows of two turns, which then needs no second kernel to
// add up dgamma (on the device 4 x 4096: 6.0 us for 8.9, 8 x 4096: 8.3; at a
// third turn they are level).  From 8192 values on a row has a turn of its own
// and a second one costs what the kernel does.
int norm_bwd_groups(int64_t m, int64_t k, int cus) {
  const int64_t sub = 1024 / norm_bwd_threads(k);
  if (k <= 4096 && m <= 2 * sub) return 1;
  return (int)std::max<int64_t>(1, std::min<int64_t>((m + sub - 1) / sub, cus));
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
  const uint32_t per = (uint32_t)((a.k + 15) / 16), total = (uint32_t)(per * a.m);
  auto go = [&](auto type) {
    typedef decltype(type) T;
    const SwigluSrc<T> s{mat<T>(a.g, a.ldg, a.m, a.k), mat<T>(a.u, a.ldu, a.m, a.k)};
    k_swiglu<T><<<dim3((total + 255u) / 256u), dim3(256), 0, st>>>(s, out16(a.y, a.m, a.k), per, total, a.k);
    return hipGetLastError();
  };
  return a.type == kRowF16 ? go(F16{}) : go(Bf16{});
}

hipError_t launch_swiglu_bwd(const SwigluArgs& a, hipStream_t st) {
  const uint32_t per = (uint32_t)((a.k + 15) / 16), total = (uint32_t)(per * a.m);
  auto go = [&](auto type) {
    typedef decltype(type) T;
    const SwigluSrc<T> s{mat<T>(a.g, a.ldg, a.m, a.k), mat<T>(a.u, a.ldu, a.m, a.k)};
    k_swiglu_bwd<T><<<dim3((total + 255u) / 256u), dim3(256), 0, st>>>(
        mat<T>(a.dy, a.lddy, a.m, a.k), s, out16(a.dg, a.m, a.k), out16(a.du, a.m, a.k), per, total, a.k);
    return hipGetLastError();
  };
  return a.type == kRowF16 ? go(F16{}) : go(Bf16{});
}

QLORA_OOB_READER(oob_count_rows)

}  // namespace qlora
